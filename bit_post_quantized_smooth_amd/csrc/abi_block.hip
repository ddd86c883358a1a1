// C ABI of the 8-bit attention block: argument checks, workspace carving and
// kernel launches. Every check runs on the host before anything is enqueued;
// on an error nothing is launched or written.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <limits>
#include <utility>

#include "../../include/svdq.h"
#include "abi_checks.hpp"
#include "attention.hpp"
#include "block_launch.hpp"
#include "host_internal.hpp"

using namespace svdq;

namespace {

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxK = int64_t{1} << 22;      // 256 rows of codes stay below 2^31 bytes

size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

bool known(int dtype) { return dtype == SVDQ_F16 || dtype == SVDQ_F32 || dtype == SVDQ_BF16; }
uintptr_t esize(int dtype) { return dtype == SVDQ_F32 ? 4 : 2; }

int check_quant(const char* fn, const void* X, const void* residual, int dtype, int64_t M,
                int64_t K, int64_t ldx, int64_t ldr, const float* gain, const uint8_t* a_codes,
                const float* a_scales, const void* residual_out, int64_t ldo) {
  if (!known(dtype)) return fail(SVDQ_ERR_DTYPE, fn, "dtype is not f16, bf16 or f32");
  if (M < 0 || M > kMaxRows || K < 1 || K > kMaxK) {
    set_error("%s: M=%lld K=%lld out of range", fn, (long long)M, (long long)K);
    return SVDQ_ERR_SHAPE;
  }
  if (ldx < K || ldx > kMaxStride || (residual && (ldr < K || ldr > kMaxStride)) ||
      (residual_out && (ldo < K || ldo > kMaxStride)))
    return fail(SVDQ_ERR_SHAPE, fn, "a row stride is smaller than K or out of range");
  if (M == 0) return SVDQ_OK;
  if (!X || !a_codes || !a_scales) return fail(SVDQ_ERR_NULL, fn, "null pointer");
  const uintptr_t e = esize(dtype);
  if (!aligned(X, e) || !aligned(residual, e) || !aligned(residual_out, e) ||
      !aligned(a_codes, 16) || !aligned(a_scales, 16) || !aligned(gain, 16))
    return fail(SVDQ_ERR_ALIGN, fn,
                "X, residual and residual_out need their element's alignment, codes, scales "
                "and gain 16 bytes");
  if ((residual_out == X && ldo != ldx) || (residual && residual_out == residual && ldo != ldr))
    return fail(SVDQ_ERR_SHAPE, fn, "in-place residual_out with another row stride");
  return SVDQ_OK;
}

int check_gemm(const char* fn, const uint8_t* a_codes, const float* a_scales,
               const uint8_t* w_codes, const float* w_scales, const float* bias, const void* Y,
               int y_dtype, int64_t M, int64_t N, int64_t Kp, int64_t ldy, int32_t activation) {
  if (!known(y_dtype)) return fail(SVDQ_ERR_DTYPE, fn, "y_dtype is not f16, bf16 or f32");
  if (activation != SVDQ_ACT_NONE && activation != SVDQ_ACT_GELU_TANH)
    return fail(SVDQ_ERR_ACT, fn, "unknown activation");
  if (Kp < SVDQ_FP8_BLOCK || Kp % SVDQ_FP8_BLOCK != 0)
    return fail(SVDQ_ERR_GROUP, fn, "Kp is not a positive multiple of 128");
  if (Kp > kMaxK || M < 0 || M > kMaxRows || N < 1 || N > kMaxRows || ldy < N ||
      ldy > kMaxStride || ((M + 63) / 64) * ((N + 63) / 64) > (int64_t{1} << 26) ||
      !gemm_fp8_fits(M, N, y_dtype)) {
    set_error("%s: M=%lld N=%lld Kp=%lld ldy=%lld out of range", fn, (long long)M, (long long)N,
              (long long)Kp, (long long)ldy);
    return SVDQ_ERR_SHAPE;
  }
  if (M == 0) return SVDQ_OK;
  if (!a_codes || !a_scales || !w_codes || !w_scales || !Y)
    return fail(SVDQ_ERR_NULL, fn, "null pointer");
  if (!aligned(a_codes, 16) || !aligned(w_codes, 16) || !aligned(a_scales, 4) ||
      !aligned(w_scales, 4) || !aligned(bias, 4) || !aligned(Y, esize(y_dtype)))
    return fail(SVDQ_ERR_ALIGN, fn,
                "codes must be 16-byte aligned, scales, bias and Y aligned to their elements");
  return SVDQ_OK;
}

// The workspace of svdq_linear_fp8: codes, scales, the split product's partials.
struct LinearWs {
  size_t scales, part;
};
LinearWs linear_ws(int64_t M, int64_t K) {
  const int64_t Kp = fp8_padded(K);
  LinearWs w;
  w.scales = round_up(static_cast<size_t>(M) * Kp, 256);
  w.part = w.scales + round_up(static_cast<size_t>(M) * (Kp / SVDQ_FP8_BLOCK) * 4, 256);
  return w;
}

}  // namespace

extern "C" {

int svdq_rmsnorm_quantize_fp8(const void* X, const void* residual, int dtype, int64_t M, int64_t K,
                              int64_t ldx, int64_t ldr, const float* gain, float eps,
                              uint8_t* a_codes, float* a_scales, void* residual_out, int64_t ldo,
                              hipStream_t stream) {
  clear_error();
  const char* fn = "svdq_rmsnorm_quantize_fp8";
  if (int s = check_quant(fn, X, residual, dtype, M, K, ldx, ldr, gain, a_codes, a_scales,
                          residual_out, ldo))
    return s;
  if (!(eps >= 0.f) || std::isinf(eps)) return fail(SVDQ_ERR_SHAPE, fn, "eps is not a finite value >= 0");
  if (M == 0) return SVDQ_OK;
  if (int s = device_ready(fn)) return s;
  return check_hip(launch_quantize_fp8(X, residual, dtype, M, K, ldx, ldr, true, gain, eps, a_codes,
                                       a_scales, residual_out, ldo, stream),
                   fn);
}

int svdq_quantize_act_fp8(const void* X, int dtype, int64_t M, int64_t K, int64_t ldx,
                          uint8_t* a_codes, float* a_scales, hipStream_t stream) {
  clear_error();
  const char* fn = "svdq_quantize_act_fp8";
  if (int s = check_quant(fn, X, nullptr, dtype, M, K, ldx, 0, nullptr, a_codes, a_scales, nullptr,
                          0))
    return s;
  if (M == 0) return SVDQ_OK;
  if (int s = device_ready(fn)) return s;
  return check_hip(launch_quantize_fp8(X, nullptr, dtype, M, K, ldx, 0, false, nullptr, 0.f,
                                       a_codes, a_scales, nullptr, 0, stream),
                   fn);
}

size_t svdq_gemm_fp8_workspace_bytes(int64_t M, int64_t N, int64_t Kp) {
  if (M < 1 || N < 1 || Kp < SVDQ_FP8_BLOCK || Kp % SVDQ_FP8_BLOCK != 0) return 0;
  return gemm_fp8_split_bytes(M, N, Kp);
}

int svdq_gemm_fp8(const uint8_t* a_codes, const float* a_scales, const uint8_t* w_codes,
                  const float* w_scales, const float* bias, void* Y, int y_dtype, int64_t M,
                  int64_t N, int64_t Kp, int64_t ldy, int32_t activation, void* ws,
                  size_t ws_bytes, hipStream_t stream) {
  clear_error();
  const char* fn = "svdq_gemm_fp8";
  if (int s = check_gemm(fn, a_codes, a_scales, w_codes, w_scales, bias, Y, y_dtype, M, N, Kp, ldy,
                         activation))
    return s;
  if (!aligned(ws, 16)) return fail(SVDQ_ERR_ALIGN, fn, "the workspace must be 16-byte aligned");
  if (M == 0) return SVDQ_OK;
  if (int s = device_ready(fn)) return s;
  return check_hip(launch_gemm_fp8(a_codes, a_scales, w_codes, w_scales, bias, Y, y_dtype, M, N, Kp,
                                   ldy, activation == SVDQ_ACT_GELU_TANH, static_cast<float*>(ws),
                                   ws ? ws_bytes : 0, stream),
                   fn);
}

size_t svdq_linear_fp8_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  if (M < 1 || K < 1 || N < 1) return 0;
  return linear_ws(M, K).part + gemm_fp8_split_bytes(M, N, fp8_padded(K));
}

int svdq_linear_fp8(const void* X, int x_dtype, int64_t ldx, const uint8_t* w_codes,
                    const float* w_scales, const float* bias, void* Y, int y_dtype, int64_t ldy,
                    int64_t M, int64_t K, int64_t N, void* ws, size_t ws_bytes,
                    int32_t activation, hipStream_t stream) {
  clear_error();
  const char* fn = "svdq_linear_fp8";
  if (M < 0 || M > kMaxRows || K < 1 || K > kMaxK || N < 1 || N > kMaxRows) {
    set_error("%s: M=%lld K=%lld N=%lld out of range", fn, (long long)M, (long long)K,
              (long long)N);
    return SVDQ_ERR_SHAPE;
  }
  if (M > 0) {
    if (!ws) return fail(SVDQ_ERR_NULL, fn, "null workspace");
    if (!aligned(ws, 256)) return fail(SVDQ_ERR_ALIGN, fn, "workspace must be 256-byte aligned");
  }
  const LinearWs L = linear_ws(M, K);
  if (ws_bytes < L.part) {
    set_error("%s: workspace %zu bytes < %zu needed", fn, ws_bytes, L.part);
    return SVDQ_ERR_WORKSPACE;
  }
  uint8_t* base = static_cast<uint8_t*>(ws);
  uint8_t* codes = base;
  float* scales = reinterpret_cast<float*>(base + L.scales);
  if (int s = check_quant(fn, X, nullptr, x_dtype, M, K, ldx, 0, nullptr, codes, scales, nullptr, 0))
    return s;
  if (int s = check_gemm(fn, codes, scales, w_codes, w_scales, bias, Y, y_dtype, M, N,
                         fp8_padded(K), ldy, activation))
    return s;
  if (M == 0) return SVDQ_OK;
  if (int s = device_ready(fn)) return s;
  if (int s = check_hip(launch_quantize_fp8(X, nullptr, x_dtype, M, K, ldx, 0, false, nullptr, 0.f,
                                            codes, scales, nullptr, 0, stream),
                        fn))
    return s;
  return check_hip(launch_gemm_fp8(codes, scales, w_codes, w_scales, bias, Y, y_dtype, M, N,
                                   fp8_padded(K), ldy, activation == SVDQ_ACT_GELU_TANH,
                                   reinterpret_cast<float*>(base + L.part), ws_bytes - L.part,
                                   stream),
                   fn);
}

namespace {

constexpr int64_t kMaxLen = int64_t{1} << 30;

int check_attention_sizes(const char* fn, int64_t B, int64_t Lq, int64_t Lk, int64_t Hq,
                          int64_t Hkv, int64_t D) {
  if (B < 0 || B > kMaxLen || Lq < 0 || Lq > kMaxLen || Lk < 0 || Lk > kMaxLen || Hkv < 1 ||
      Hkv > 65536 || Hq < Hkv || Hq > 65536 || Hq % Hkv != 0 || Lq * (Hq / Hkv) > kMaxLen ||
      (Lq > 0 && B * Hkv > kMaxLen / Lq)) {
    set_error("%s: B=%lld Lq=%lld Lk=%lld Hq=%lld Hkv=%lld out of range", fn, (long long)B,
              (long long)Lq, (long long)Lk, (long long)Hq, (long long)Hkv);
    return SVDQ_ERR_SHAPE;
  }
  if (D < 8 || D > 128 || D % 8 != 0)
    return fail(SVDQ_ERR_SHAPE, fn, "D is not a multiple of 8 up to 128");
  return SVDQ_OK;
}

// Whether tokens of B x L x H heads of D channels at these strides may share elements:
// dimensions by growing stride, each has to step over all that the smaller ones span.
bool overlaps(const int64_t* strides, int64_t B, int64_t L, int64_t H, int64_t D) {
  std::pair<int64_t, int64_t> dims[3] = {{strides[0], B}, {strides[1], L}, {strides[2], H}};
  std::sort(dims, dims + 3);
  __int128 span = D;                   // 2^30 of 2^40 would not fit 64 bits
  for (const auto& [stride, count] : dims) {
    if (count < 2) continue;
    if (stride < span) return true;
    span += static_cast<__int128>(count - 1) * stride;
  }
  return false;
}

// Per split and row: the maximum and sum, then D outputs.
size_t attention_ml_bytes(int64_t B, int64_t Lq, int64_t Hq, int splits) {
  return round_up(static_cast<size_t>(splits) * B * Lq * Hq * 8, 256);
}
size_t attention_bytes(int64_t B, int64_t Lq, int64_t Hq, int64_t D, int splits) {
  if (splits < 2) return 0;
  return attention_ml_bytes(B, Lq, Hq, splits) + static_cast<size_t>(splits) * B * Lq * Hq * D * 4;
}

}  // namespace

size_t svdq_attention_workspace_bytes(int64_t B, int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hkv,
                                      int64_t D) {
  const int s = check_attention_sizes("svdq_attention_workspace_bytes", B, Lq, Lk, Hq, Hkv, D);
  clear_error();                       // a size query reports by its 0 alone
  if (s != SVDQ_OK || B == 0 || Lq == 0) return 0;
  return attention_bytes(B, Lq, Hq, D, attention_plan(B, Lq, Lk, Hq, Hkv, D, true).splits);
}

int svdq_attention(const void* Q, const void* K, const void* V, void* Out, int dtype, int64_t B,
                   int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hkv, int64_t D,
                   const int64_t* strides, float scale, float softcap, const float* slopes,
                   int32_t causal, const int32_t* prefix, const int32_t* key_ranges,
                   int64_t key_ranges_batch, void* ws, size_t ws_bytes, hipStream_t stream) {
  clear_error();
  const char* fn = "svdq_attention";
  if (dtype != SVDQ_F16 && dtype != SVDQ_BF16)
    return fail(SVDQ_ERR_DTYPE, fn, "dtype is not f16 or bf16");
  if (int s = check_attention_sizes(fn, B, Lq, Lk, Hq, Hkv, D)) return s;
  if (!std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.f)
    return fail(SVDQ_ERR_SHAPE, fn, "scale and softcap must be finite, softcap not negative");
  if (prefix && !causal) return fail(SVDQ_ERR_SHAPE, fn, "a prefix needs causal");
  if (key_ranges_batch < 0 || key_ranges_batch > kMaxStride)
    return fail(SVDQ_ERR_SHAPE, fn, "batch stride of key_ranges out of range");
  if (!strides) return fail(SVDQ_ERR_NULL, fn, "null strides");
  for (int i = 0; i < 12; ++i)
    if (strides[i] < 0 || strides[i] > kMaxStride || strides[i] % 8 != 0)
      return fail(SVDQ_ERR_ALIGN, fn, "a stride is negative, too large or not a multiple of 8");
  const int64_t *sk = strides + 3, *sv = strides + 6;
  if (sk[1] > kMaxK || sv[1] > kMaxK || (Lk > 1 && (sk[1] < D || sv[1] < D)))
    return fail(SVDQ_ERR_SHAPE, fn, "token strides of K and V must lie in D .. 2^22");
  if (B == 0 || Lq == 0) return SVDQ_OK;
  if (overlaps(strides + 9, B, Lq, Hq, D))
    return fail(SVDQ_ERR_SHAPE, fn, "the strides of Out make it overlap itself");
  AttnPlan p = attention_plan(B, Lq, Lk, Hq, Hkv, D, true);
  if (p.grid == 0) return fail(SVDQ_ERR_SHAPE, fn, "more rows than one launch can cover");
  if (!Q || !Out || (Lk > 0 && (!K || !V))) return fail(SVDQ_ERR_NULL, fn, "null pointer");
  if (!aligned(Q, 16) || !aligned(K, 16) || !aligned(V, 16) || !aligned(Out, 16) ||
      !aligned(slopes, 4) || !aligned(prefix, 4) || !aligned(key_ranges, 4) || !aligned(ws, 16))
    return fail(SVDQ_ERR_ALIGN, fn,
                "Q, K, V, Out and the workspace must be 16-byte aligned, the rest 4-byte");
  if (int s = device_ready(fn)) return s;
  if (p.splits > 1 && (ws == nullptr || ws_bytes < attention_bytes(B, Lq, Hq, D, p.splits)))
    p = attention_plan(B, Lq, Lk, Hq, Hkv, D, false);
  AttnArgs g{};
  g.q = Q;
  g.k = K;
  g.v = V;
  g.out = Out;
  int64_t* to[12] = {&g.q_b, &g.q_l, &g.q_h, &g.k_b, &g.k_l, &g.k_h,
                     &g.v_b, &g.v_l, &g.v_h, &g.o_b, &g.o_l, &g.o_h};
  for (int i = 0; i < 12; ++i) *to[i] = strides[i];
  g.slopes = slopes;
  g.prefix = prefix;
  g.ranges = key_ranges;
  g.range_b = key_ranges_batch;
  g.part_ml = static_cast<float*>(ws);
  g.part_o = p.splits > 1 ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                                     attention_ml_bytes(B, Lq, Hq, p.splits))
                          : nullptr;
  constexpr float kLog2e = 1.4426950408889634f;
  g.q_sign = scale > 0.f ? 1 : scale < 0.f ? -1 : 0;
  g.scale2 = g.q_sign != 0 ? std::fabs(scale) * kLog2e : 1.f;
  // finite at any cap: a score of 0 times an infinity would be NaN
  constexpr float kMost = std::numeric_limits<float>::max();
  g.cap = softcap == 0.f ? kNoCap : softcap <= kNearest ? kNearCap : kAnyCap;
  g.cap_in = softcap > 0.f ? std::fmin(2.0f * kLog2e * (std::fabs(scale) / softcap), kMost) : 0.f;
  g.cap2 = std::fmin(softcap * kLog2e, kMost);
  g.B = static_cast<int>(B);
  g.Lq = static_cast<int>(Lq);
  g.Lk = static_cast<int>(Lk);
  g.Hkv = static_cast<int>(Hkv);
  g.G = static_cast<int>(Hq / Hkv);
  g.D = static_cast<int>(D);
  g.rows = static_cast<int>(Lq * (Hq / Hkv));
  g.causal = causal != 0;
  return check_hip(launch_attention(g, dtype, p, stream), fn);
}

}  // extern "C"
