// Attention of new tokens over a paged cache (gfx950).
//
//   x_ij = scale * s_k * q_i . k_j;  with a cap: x_ij = cap * tanh(x_ij / cap);
//   with slopes: x_ij -= slope_h * |pos_i - j|;
//   o_i = s_v * sum_j exp(x_ij) v_j / sum_j exp(x_ij) over the keys j that row i sees:
//   j < length of its sequence, in a page of the pool, and, if causal, j <= pos_i,
//   where the sequence's n new tokens are its last: pos_i = length - n + i.
// s_k and s_v are the head's scales of e4m3 codes (1 of 16-bit pages).
//
// A wave takes one query head of one token. Its lanes hold a key each for the
// scores and two channels each for the outputs; one pass over the keys with the
// running maximum and sum of the softmax. All arithmetic is fp32.
#include <hip/hip_runtime.h>

#include "../../include/svdq.h"
#include "block_common.hpp"
#include "block_launch.hpp"
#include "paged_attention.hpp"

namespace svdq {

namespace {

constexpr int kWaves = 4;
constexpr float kNegInf = -__builtin_inff();

template <class T>
__device__ __forceinline__ float element(const void* p, int64_t i) {
  return static_cast<float>(static_cast<const T*>(p)[i]);
}
template <>
__device__ __forceinline__ float element<uint8_t>(const void* p, int64_t i) {
  return __builtin_amdgcn_cvt_f32_fp8(static_cast<const uint8_t*>(p)[i], 0);
}

template <class T, class E>
__global__ __launch_bounds__(64 * kWaves) void paged_attention_kernel(const PagedArgs g) {
  __shared__ float qs[kWaves][128];
  __shared__ float ps[kWaves][64];
  __shared__ int64_t rows[kWaves][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int Hq = g.Hkv * g.G;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWaves + w;
  const int t = static_cast<int>(unit / Hq), head = static_cast<int>(unit % Hq);
  if (t >= g.T) return;
  // the last sequence that starts at or before t
  int lo = 0, hi = g.B;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (g.starts[mid] <= t) lo = mid + 1;
    else hi = mid;
  }
  const int b = lo - 1;
  if (b < 0 || t >= g.starts[b + 1]) return;       // no sequence's token
  const int n = g.starts[b + 1] - g.starts[b], i = t - g.starts[b];
  int length = g.lengths[b] < g.capacity ? g.lengths[b] : g.capacity;
  const int pos = length - n + i;
  int end = g.causal && pos + 1 < length ? pos + 1 : length;
  const int hk = head / g.G;
  const Pages& pg = g.pages;
  const float ks = g.scale * (pg.k_scales != nullptr ? pg.k_scales[hk] : 1.f);
  const float vs = pg.v_scales != nullptr ? pg.v_scales[hk] : 1.f;
  const float slope = g.slopes != nullptr ? g.slopes[head] : 0.f;
  const T* q = static_cast<const T*>(g.q) + t * g.q_t + head * g.q_h;
  for (int c = lane; c < 128; c += 64) qs[w][c] = c < g.D ? static_cast<float>(q[c]) : 0.f;
  float m = kNegInf, l = 0.f, o[2] = {0.f, 0.f};
  for (int j0 = 0; j0 < end; j0 += 64) {
    const int j = j0 + lane;
    int64_t page = -1;
    if (j < end) page = g.tables[static_cast<int64_t>(b) * g.width + (j >> pg.page_log2)];
    const bool seen = page >= 0 && page < pg.count;
    const int64_t row = ((static_cast<int64_t>(hk) << pg.page_log2) + (j & ((1 << pg.page_log2) - 1))) * g.D;
    float x = kNegInf;
    if (seen) {
      const char* k = static_cast<const char*>(pg.k) + page * pg.k_stride;
      float sum = 0.f;
      for (int c = 0; c < g.D; ++c) sum = __builtin_fmaf(qs[w][c], element<E>(k, row + c), sum);
      x = sum * ks;
      if (g.softcap > 0.f) x = g.softcap * tanhf(x / g.softcap);
      if (slope != 0.f) x = x - slope * fabsf(static_cast<float>(pos - j));
    }
    float top = x;
    for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
    const float m_new = fmaxf(m, top);
    const float base = m_new == kNegInf ? 0.f : m_new;
    const float alpha = expf(m - base);
    // 2^-24: sums of values near fp32's largest stay finite for up to 2^24 keys
    const float p = seen ? expf(x - base) * 0x1p-24f : 0.f;
    float add = p;
    for (int d = 1; d < 64; d *= 2) add += __shfl_xor(add, d);
    l = l * alpha + add;
    m = m_new;
    ps[w][lane] = p;
    rows[w][lane] = seen ? page * pg.v_stride / static_cast<int64_t>(sizeof(E)) + row : -1;
    __builtin_amdgcn_wave_barrier();
    o[0] *= alpha;
    o[1] *= alpha;
    for (int k = 0; k < 64; ++k) {
      const int64_t at = rows[w][k];
      if (at < 0) continue;
      for (int e = 0; e < 2; ++e)
        if (lane + 64 * e < g.D)
          o[e] = __builtin_fmaf(ps[w][k], element<E>(pg.v, at + lane + 64 * e), o[e]);
    }
    __builtin_amdgcn_wave_barrier();
  }
  const float inv = l == 0.f ? 0.f : vs / l;
  T* out = static_cast<T*>(g.out) + t * g.o_t + head * g.o_h;
  for (int e = 0; e < 2; ++e)
    if (lane + 64 * e < g.D) out[lane + 64 * e] = static_cast<T>(o[e] * inv);
}

template <class T>
hipError_t launch_t(const PagedArgs& g, hipStream_t stream) {
  const int64_t units = static_cast<int64_t>(g.T) * g.Hkv * g.G;
  const unsigned grid = static_cast<unsigned>((units + kWaves - 1) / kWaves);
  if (g.pages.coded)
    hipLaunchKernelGGL((paged_attention_kernel<T, uint8_t>), dim3(grid), dim3(64 * kWaves), 0, stream, g);
  else
    hipLaunchKernelGGL((paged_attention_kernel<T, T>), dim3(grid), dim3(64 * kWaves), 0, stream, g);
  return hipGetLastError();
}

}  // namespace

bool paged_attention_fits(int64_t T, int64_t Hq) { return grid_fits(T * Hq / kWaves + 1, 64 * kWaves); }

hipError_t launch_paged_attention(const PagedArgs& g, int dtype, hipStream_t stream) {
  return dtype == SVDQ_F16 ? launch_t<_Float16>(g, stream) : launch_t<__bf16>(g, stream);
}

}  // namespace svdq
