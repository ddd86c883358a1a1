// Host preparation of 8-bit (e4m3) weights with one scale per 128 x 128 block.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/svdq.h"
#include "host_internal.hpp"

using namespace svdq;

namespace {

// Nearest e4m3 code, ties to even; |v| is at most 448 (1 + 2^-22) or not finite.
// 1 sign, 4 exponent bits (bias 7), 3 fraction bits; below 2^-6 the step is 2^-9.
uint8_t to_e4m3(float v) {
  const uint8_t sign = std::signbit(v) ? 0x80 : 0;
  const float a = std::fabs(v);
  if (!std::isfinite(a)) return sign | 0x7F;
  int e = 0;
  std::frexp(a, &e);                       // a = f * 2^e, f in [1/2, 1)
  const int step = a < 0x1p-6f ? -9 : e - 4;
  int q = static_cast<int>(std::nearbyint(std::ldexp(a, -step)));   // 0 .. 16, exact scaling
  if (step == -9) return sign | static_cast<uint8_t>(q);            // q = 8 is the first normal
  int ex = e - 1;
  if (q == 16) {
    q = 8;
    ++ex;
  }
  return sign | static_cast<uint8_t>(((ex + 7) << 3) + (q - 8));
}

}  // namespace

extern "C" int svdq_prepare_weights_fp8(const float* W, int64_t K, int64_t N, uint8_t* w_codes,
                                        float* w_scales) {
  clear_error();
  const char* fn = "svdq_prepare_weights_fp8";
  if (!W || !w_codes || !w_scales) {
    set_error("%s: null pointer", fn);
    return SVDQ_ERR_NULL;
  }
  if (K < 1 || N < 1 || K > (int64_t{1} << 22) || N > (int64_t{1} << 31)) {
    set_error("%s: K=%lld N=%lld", fn, (long long)K, (long long)N);
    return SVDQ_ERR_SHAPE;
  }
  const int64_t B = SVDQ_FP8_BLOCK, G = (K + B - 1) / B, Kp = G * B, NB = (N + B - 1) / B;
#pragma omp parallel for collapse(2) schedule(static)
  for (int64_t nb = 0; nb < NB; ++nb) {
    for (int64_t g = 0; g < G; ++g) {
      const int64_t n1 = nb * B + B < N ? nb * B + B : N, k1 = g * B + B < K ? g * B + B : K;
      float a = 0.f;
      for (int64_t k = g * B; k < k1; ++k)
        for (int64_t n = nb * B; n < n1; ++n) a = std::fmax(a, std::fabs(W[k * N + n]));
      const float s = std::fmax(a / 448.0f, 0x1p-126f);
      const float inv = 1.0f / s;
      w_scales[nb * G + g] = s;
      for (int64_t n = nb * B; n < n1; ++n) {
        uint8_t* c = w_codes + n * Kp + g * B;
        for (int64_t k = g * B; k < k1; ++k) c[k - g * B] = to_e4m3(W[k * N + n] * inv);
        std::memset(c + (k1 - g * B), 0, static_cast<size_t>(B - (k1 - g * B)));
      }
    }
  }
  return SVDQ_OK;
}
