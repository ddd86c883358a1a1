// C ABI of the paged key-value cache: argument checks and kernel launches.
// Every check runs on the host before anything is enqueued; on an error nothing
// is launched or written. Page numbers, slots, lengths and starts lie on the
// device: the kernels bound each before they use it.
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
#include "paged.hpp"
#include "paged_attention.hpp"

using namespace svdq;

namespace {

constexpr int64_t kMaxTokens = int64_t{1} << 30;
constexpr int64_t kMaxHeads = 65536;

int check_heads(const char* fn, int dtype, int64_t T, int64_t Hq, int64_t Hkv, int64_t D) {
  if (dtype != SVDQ_F16 && dtype != SVDQ_BF16)
    return fail(SVDQ_ERR_DTYPE, fn, "dtype is not f16 or bf16");
  if (T < 0 || T > kMaxTokens || Hq < 0 || Hq > kMaxHeads || Hkv < 0 || Hkv > kMaxHeads) {
    set_error("%s: %lld tokens of %lld and %lld heads out of range", fn, (long long)T, (long long)Hq,
              (long long)Hkv);
    return SVDQ_ERR_SHAPE;
  }
  if (D < 8 || D > 128 || D % 8 != 0)
    return fail(SVDQ_ERR_SHAPE, fn, "D is not a multiple of 8 up to 128");
  return SVDQ_OK;
}

int check_strides(const char* fn, const int64_t* strides, int n) {
  if (!strides) return fail(SVDQ_ERR_NULL, fn, "null strides");
  for (int i = 0; i < n; ++i)
    if (strides[i] < 0 || strides[i] > kMaxStride || strides[i] % 8 != 0)
      return fail(SVDQ_ERR_ALIGN, fn, "a stride is negative, too large or not a multiple of 8");
  return SVDQ_OK;
}

// Whether counts x D channels at these strides may share elements: dimensions by
// growing stride, each has to step over all that the smaller ones span.
template <int N>
bool overlaps(std::pair<int64_t, int64_t> (&dims)[N], int64_t D) {
  std::sort(dims, dims + N);
  __int128 span = D;
  for (const auto& [stride, count] : dims)
    if (count == 0) return false;
  for (const auto& [stride, count] : dims) {
    if (count < 2) continue;
    if (stride < span) return true;
    span += static_cast<__int128>(count - 1) * stride;
  }
  return false;
}
bool rows_overlap(const int64_t* s, int64_t T, int64_t H, int64_t D) {
  std::pair<int64_t, int64_t> dims[] = {{s[0], T}, {s[1], H}};
  return overlaps(dims, D);
}

int check_rotation(const char* fn, const int32_t* positions, const double* freqs, int64_t pairs,
                   float factor, int64_t D, const float* q_gain, const float* k_gain, float eps) {
  if (pairs < 0 || 2 * pairs > D)
    return fail(SVDQ_ERR_SHAPE, fn, "the rotated channels are not 0 .. D");
  if (!std::isfinite(factor)) return fail(SVDQ_ERR_SHAPE, fn, "factor is not finite");
  if (pairs > 0 && (!positions || !freqs)) return fail(SVDQ_ERR_NULL, fn, "null pointer");
  if (!std::isfinite(eps)) return fail(SVDQ_ERR_SHAPE, fn, "eps is not finite");
  // the reciprocal root takes a subnormal mean for 0: a head of zeros would become NaN
  if (std::fpclassify(eps) == FP_SUBNORMAL)
    return fail(SVDQ_ERR_SHAPE, fn, "eps is below fp32's normal numbers");
  if (eps < 0.f && (q_gain || k_gain)) return fail(SVDQ_ERR_SHAPE, fn, "a gain needs the norm");
  if (!aligned(positions, 4) || !aligned(freqs, 8) || !aligned(q_gain, 4) || !aligned(k_gain, 4))
    return fail(SVDQ_ERR_ALIGN, fn, "positions, freqs and gains need their element's alignment");
  return SVDQ_OK;
}

// Fills pg; the pointers are checked by check_pool_pointers, since calls on no
// tokens need none.
int check_pool(const char* fn, void* k, void* v, int cache_dtype, int dtype, int64_t count,
               int64_t page_size, int64_t k_stride, int64_t v_stride, int64_t Hkv, int64_t D,
               const float* k_scales, const float* v_scales, Pages& pg) {
  if (cache_dtype != SVDQ_E4M3 && cache_dtype != dtype)
    return fail(SVDQ_ERR_DTYPE, fn, "pages are neither e4m3 nor of the tokens' dtype");
  int log2 = 0;
  while (log2 < 10 && (int64_t{1} << log2) < page_size) ++log2;
  if (page_size != (int64_t{1} << log2) || page_size < 16)
    return fail(SVDQ_ERR_SHAPE, fn, "the page size is not a power of two in 16 .. 1024");
  if (Hkv < 1) return fail(SVDQ_ERR_SHAPE, fn, "no key heads");
  const bool coded = cache_dtype == SVDQ_E4M3;
  const int64_t bytes = Hkv * page_size * D * (coded ? 1 : 2);
  if (count < 0 || count > ((int64_t{1} << 31) >> log2))
    return fail(SVDQ_ERR_SHAPE, fn, "a pool holds 2^31 tokens at most");
  if (k_stride > kMaxStride || v_stride > kMaxStride || k_stride < bytes || v_stride < bytes ||
      k_stride % 16 != 0 || v_stride % 16 != 0)
    return fail(SVDQ_ERR_SHAPE, fn, "a page stride is smaller than a page, too large or not a multiple of 16 bytes");
  if (!coded && (k_scales || v_scales)) return fail(SVDQ_ERR_SHAPE, fn, "16-bit pages have no scales");
  pg = Pages{k, v, k_stride, v_stride, count, k_scales, v_scales, log2, coded ? 1 : 0};
  return SVDQ_OK;
}

int check_pool_pointers(const char* fn, const Pages& pg) {
  if (pg.count > 0 && (!pg.k || !pg.v)) return fail(SVDQ_ERR_NULL, fn, "null pages");
  if (!aligned(pg.k, 16) || !aligned(pg.v, 16) || !aligned(pg.k_scales, 4) || !aligned(pg.v_scales, 4))
    return fail(SVDQ_ERR_ALIGN, fn, "pages must be 16-byte aligned, scales 4-byte");
  return SVDQ_OK;
}

}  // namespace

extern "C" {

int svdq_norm_rotary(const void* Q, const void* K, void* Q_out, void* K_out, int dtype, int64_t T,
                     int64_t Hq, int64_t Hkv, int64_t D, const int64_t* strides,
                     const int32_t* positions, const double* freqs, int64_t pairs, float factor,
                     int32_t interleaved, const float* q_gain, const float* k_gain, float eps,
                     hipStream_t stream) {
  clear_error();
  const char* fn = "svdq_norm_rotary";
  if (int s = check_heads(fn, dtype, T, Hq, Hkv, D)) return s;
  if (int s = check_strides(fn, strides, 8)) return s;
  if (!heads_fit(T, Hq + Hkv)) return fail(SVDQ_ERR_SHAPE, fn, "more heads than one launch can cover");
  if (T == 0 || Hq + Hkv == 0) return SVDQ_OK;
  if (int s = check_rotation(fn, positions, freqs, pairs, factor, D, q_gain, k_gain, eps)) return s;
  if ((Hq > 0 && (!Q || !Q_out)) || (Hkv > 0 && (!K || !K_out)))
    return fail(SVDQ_ERR_NULL, fn, "null pointer");
  if (!aligned(Q, 16) || !aligned(K, 16) || !aligned(Q_out, 16) || !aligned(K_out, 16))
    return fail(SVDQ_ERR_ALIGN, fn, "heads must be 16-byte aligned");
  if (rows_overlap(strides + 4, T, Hq, D) || rows_overlap(strides + 6, T, Hkv, D))
    return fail(SVDQ_ERR_SHAPE, fn, "the strides of an output make it overlap itself");
  if ((Q == Q_out && Hq > 0 && (strides[0] != strides[4] || strides[1] != strides[5])) ||
      (K == K_out && Hkv > 0 && (strides[2] != strides[6] || strides[3] != strides[7])))
    return fail(SVDQ_ERR_SHAPE, fn, "in place with other strides");
  if (Hq > 0 && Hkv > 0 && Q_out == K_out)
    return fail(SVDQ_ERR_SHAPE, fn, "queries and keys into the same output");
  if (int s = device_ready(fn)) return s;
  HeadsArgs g{};
  g.q = Q;
  g.k = K;
  g.q_out = Q_out;
  g.k_out = K_out;
  int64_t* to[8] = {&g.q_t, &g.q_h, &g.k_t, &g.k_h, &g.qo_t, &g.qo_h, &g.ko_t, &g.ko_h};
  for (int i = 0; i < 8; ++i) *to[i] = strides[i];
  g.positions = positions;
  g.freqs = freqs;
  g.q_gain = q_gain;
  g.k_gain = k_gain;
  g.factor = factor;
  g.eps = eps;
  g.pairs = static_cast<int>(pairs);
  g.interleaved = interleaved != 0;
  g.norm = eps >= 0.f;
  g.T = static_cast<int>(T);
  g.Hq = static_cast<int>(Hq);
  g.Hkv = static_cast<int>(Hkv);
  g.D = static_cast<int>(D);
  return check_hip(launch_heads(g, dtype, stream), fn);
}

int svdq_paged_write(const void* Q, const void* K, const void* V, void* Q_out, int dtype, int64_t T,
                     int64_t Hq, int64_t Hkv, int64_t D, const int64_t* strides,
                     const int32_t* positions, const double* freqs, int64_t pairs, float factor,
                     int32_t interleaved, const float* q_gain, const float* k_gain, float eps,
                     const int32_t* slots, void* k_pages, void* v_pages, int cache_dtype,
                     int64_t pages, int64_t page_size, int64_t k_page_stride,
                     int64_t v_page_stride, const float* k_scales, const float* v_scales,
                     hipStream_t stream) {
  clear_error();
  const char* fn = "svdq_paged_write";
  if (int s = check_heads(fn, dtype, T, Hq, Hkv, D)) return s;
  if (int s = check_strides(fn, strides, 8)) return s;
  HeadsArgs g{};
  if (int s = check_pool(fn, k_pages, v_pages, cache_dtype, dtype, pages, page_size, k_page_stride,
                         v_page_stride, Hkv, D, k_scales, v_scales, g.pages))
    return s;
  if (!heads_fit(T, Hq + 2 * Hkv))
    return fail(SVDQ_ERR_SHAPE, fn, "more heads than one launch can cover");
  if (T == 0) return SVDQ_OK;
  if (int s = check_rotation(fn, positions, freqs, pairs, factor, D, q_gain, k_gain, eps)) return s;
  if ((Hq > 0 && (!Q || !Q_out)) || !K || !V || !slots) return fail(SVDQ_ERR_NULL, fn, "null pointer");
  if (int s = check_pool_pointers(fn, g.pages)) return s;
  if (!aligned(Q, 16) || !aligned(K, 16) || !aligned(V, 16) || !aligned(Q_out, 16) || !aligned(slots, 4))
    return fail(SVDQ_ERR_ALIGN, fn, "heads must be 16-byte aligned, slots 4-byte");
  if (rows_overlap(strides + 6, T, Hq, D))
    return fail(SVDQ_ERR_SHAPE, fn, "the strides of Q_out make it overlap itself");
  if (pages > 0 && k_pages == v_pages)
    return fail(SVDQ_ERR_SHAPE, fn, "keys and values into the same pages");
  if (Q == Q_out && Hq > 0 && (strides[0] != strides[6] || strides[1] != strides[7]))
    return fail(SVDQ_ERR_SHAPE, fn, "in place with other strides");
  if (int s = device_ready(fn)) return s;
  g.q = Q;
  g.k = K;
  g.v = V;
  g.q_out = Q_out;
  int64_t* to[8] = {&g.q_t, &g.q_h, &g.k_t, &g.k_h, &g.v_t, &g.v_h, &g.qo_t, &g.qo_h};
  for (int i = 0; i < 8; ++i) *to[i] = strides[i];
  g.positions = positions;
  g.freqs = freqs;
  g.q_gain = q_gain;
  g.k_gain = k_gain;
  g.slots = slots;
  g.factor = factor;
  g.eps = eps;
  g.pairs = static_cast<int>(pairs);
  g.interleaved = interleaved != 0;
  g.norm = eps >= 0.f;
  g.T = static_cast<int>(T);
  g.Hq = static_cast<int>(Hq);
  g.Hkv = static_cast<int>(Hkv);
  g.D = static_cast<int>(D);
  return check_hip(launch_heads(g, dtype, stream), fn);
}

int svdq_paged_read(const void* k_pages, const void* v_pages, int cache_dtype, int64_t pages,
                    int64_t page_size, int64_t k_page_stride, int64_t v_page_stride,
                    const float* k_scales, const float* v_scales, const int32_t* tables,
                    int64_t width, const int32_t* lengths, int64_t B, int64_t L, int64_t Hkv,
                    int64_t D, void* K_out, void* V_out, int dtype, const int64_t* strides,
                    hipStream_t stream) {
  clear_error();
  const char* fn = "svdq_paged_read";
  if (int s = check_heads(fn, dtype, L, 0, Hkv, D)) return s;
  if (int s = check_strides(fn, strides, 6)) return s;
  ReadArgs g{};
  if (int s = check_pool(fn, const_cast<void*>(k_pages), const_cast<void*>(v_pages), cache_dtype,
                         dtype, pages, page_size, k_page_stride, v_page_stride, Hkv, D, k_scales,
                         v_scales, g.pages))
    return s;
  if (B < 0 || B > kMaxTokens || width < 0 || width > kMaxTokens >> g.pages.page_log2 ||
      !read_fits(B, L, Hkv)) {
    set_error("%s: %lld sequences of %lld tokens and %lld pages out of range", fn, (long long)B,
              (long long)L, (long long)width);
    return SVDQ_ERR_SHAPE;
  }
  if (B == 0 || L == 0) return SVDQ_OK;
  if (!lengths || !K_out || !V_out || (width > 0 && !tables))
    return fail(SVDQ_ERR_NULL, fn, "null pointer");
  if (int s = check_pool_pointers(fn, g.pages)) return s;
  if (!aligned(K_out, 16) || !aligned(V_out, 16) || !aligned(tables, 4) || !aligned(lengths, 4))
    return fail(SVDQ_ERR_ALIGN, fn, "outputs must be 16-byte aligned, tables and lengths 4-byte");
  for (int i = 0; i < 2; ++i) {
    std::pair<int64_t, int64_t> dims[] = {
        {strides[3 * i], B}, {strides[3 * i + 1], L}, {strides[3 * i + 2], Hkv}};
    if (overlaps(dims, D))
      return fail(SVDQ_ERR_SHAPE, fn, "the strides of an output make it overlap itself");
  }
  if (K_out == V_out) return fail(SVDQ_ERR_SHAPE, fn, "keys and values into the same output");
  if (int s = device_ready(fn)) return s;
  g.tables = tables;
  g.lengths = lengths;
  g.k_out = K_out;
  g.v_out = V_out;
  int64_t* to[6] = {&g.k_b, &g.k_t, &g.k_h, &g.v_b, &g.v_t, &g.v_h};
  for (int i = 0; i < 6; ++i) *to[i] = strides[i];
  g.width = static_cast<int>(width);
  g.B = static_cast<int>(B);
  g.L = static_cast<int>(L);
  g.Hkv = static_cast<int>(Hkv);
  g.D = static_cast<int>(D);
  return check_hip(launch_read(g, dtype, stream), fn);
}

namespace {

int check_paged_attention_sizes(const char* fn, int64_t T, int64_t B, int64_t capacity, int64_t Hq,
                                int64_t Hkv, int64_t D) {
  if (T < 0 || B < 0 || B > kMaxTokens || capacity < 0 || capacity > kMostKeys || Hkv < 1 ||
      Hkv > kMaxHeads || Hq < Hkv || Hq > kMaxHeads || Hq % Hkv != 0 || Hq / Hkv > kMostGroup ||
      T > kMaxTokens / Hq) {
    set_error("%s: %lld tokens of %lld sequences, %lld keys, %lld over %lld heads out of range", fn,
              (long long)T, (long long)B, (long long)capacity, (long long)Hq, (long long)Hkv);
    return SVDQ_ERR_SHAPE;
  }
  if (D < 8 || D > 128 || D % 8 != 0)
    return fail(SVDQ_ERR_SHAPE, fn, "D is not a multiple of 8 up to 128");
  return SVDQ_OK;
}

}  // namespace

size_t svdq_paged_attention_workspace_bytes(int64_t T, int64_t B, int64_t capacity, int64_t Hq,
                                            int64_t Hkv, int64_t D) {
  const int s = check_paged_attention_sizes("svdq_paged_attention_workspace_bytes", T, B, capacity,
                                            Hq, Hkv, D);
  clear_error();                       // a size query reports by its 0 alone
  if (s != SVDQ_OK) return 0;
  return paged_attention_parts(T, B, capacity, Hkv, Hq / Hkv, D).all();
}

int svdq_paged_attention(const void* Q, void* Out, int dtype, int64_t T, int64_t Hq, int64_t Hkv,
                         int64_t D, const int64_t* strides, const void* k_pages,
                         const void* v_pages, int cache_dtype, int64_t pages, int64_t page_size,
                         int64_t k_page_stride, int64_t v_page_stride, const float* k_scales,
                         const float* v_scales, const int32_t* tables, int64_t width,
                         const int32_t* lengths, const int32_t* starts, int64_t B, float scale,
                         float softcap, const float* slopes, int32_t causal, void* ws,
                         size_t ws_bytes, hipStream_t stream) {
  clear_error();
  const char* fn = "svdq_paged_attention";
  if (int s = check_heads(fn, dtype, T, Hq, Hkv, D)) return s;
  if (int s = check_strides(fn, strides, 4)) return s;
  PagedArgs g{};
  if (int s = check_pool(fn, const_cast<void*>(k_pages), const_cast<void*>(v_pages), cache_dtype,
                         dtype, pages, page_size, k_page_stride, v_page_stride, Hkv, D, k_scales,
                         v_scales, g.pages))
    return s;
  if (width < 0 || width > kMaxTokens >> g.pages.page_log2)
    return fail(SVDQ_ERR_SHAPE, fn, "the tables' width is out of range");
  const int64_t capacity = width << g.pages.page_log2;
  if (int s = check_paged_attention_sizes(fn, T, B, capacity, Hq, Hkv, D)) return s;
  if (!std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.f)
    return fail(SVDQ_ERR_SHAPE, fn, "scale and softcap must be finite, softcap not negative");
  // Slopes are kept in units of the scores, and key scales (2^-64 .. 2^64, on the device)
  // multiply the scale: neither may leave fp32. A product of 0 would make a masked score
  // -inf * 0, an infinite one a score of 0.
  if ((slopes || k_scales) && scale != 0.f && std::fabs(scale) < 0x1p-40f)
    return fail(SVDQ_ERR_SHAPE, fn, "a scale below 2^-40 with slopes or key scales");
  if (k_scales && std::fabs(scale) > 0x1p60f)
    return fail(SVDQ_ERR_SHAPE, fn, "a scale above 2^60 with key scales");
  if (T == 0 || B == 0) return SVDQ_OK;
  if (rows_overlap(strides + 2, T, Hq, D))
    return fail(SVDQ_ERR_SHAPE, fn, "the strides of Out make it overlap itself");
  if (!Q || !Out || !lengths || !starts || (width > 0 && !tables))
    return fail(SVDQ_ERR_NULL, fn, "null pointer");
  if (int s = check_pool_pointers(fn, g.pages)) return s;
  if (!aligned(Q, 16) || !aligned(Out, 16) || !aligned(ws, 16) || !aligned(tables, 4) ||
      !aligned(lengths, 4) || !aligned(starts, 4) || !aligned(slopes, 4))
    return fail(SVDQ_ERR_ALIGN, fn, "Q, Out and the workspace must be 16-byte aligned, the rest 4-byte");
  if (int s = device_ready(fn)) return s;
  g.q = Q;
  g.out = Out;
  int64_t* to[4] = {&g.q_t, &g.q_h, &g.o_t, &g.o_h};
  for (int i = 0; i < 4; ++i) *to[i] = strides[i];
  g.tables = tables;
  g.lengths = lengths;
  g.starts = starts;
  g.slopes = slopes;
  constexpr float kLog2e = 1.4426950408889634f;
  g.q_sign = scale > 0.f ? 1 : scale < 0.f ? -1 : 0;
  g.scale2 = g.q_sign != 0 ? std::fabs(scale) * kLog2e : 1.f;
  // finite at any cap: a score of 0 times an infinity would be NaN
  constexpr float kMost = std::numeric_limits<float>::max();
  g.cap = softcap == 0.f ? kNoCap : softcap <= kNearest ? kNearCap : kAnyCap;
  g.cap_in = softcap > 0.f ? std::fmin(2.0f * kLog2e * (std::fabs(scale) / softcap), kMost) : 0.f;
  g.cap2 = std::fmin(softcap * kLog2e, kMost);
  g.causal = causal != 0;
  g.width = static_cast<int>(width);
  g.B = static_cast<int>(B);
  g.T = static_cast<int>(T);
  g.Hkv = static_cast<int>(Hkv);
  g.G = static_cast<int>(Hq / Hkv);
  g.D = static_cast<int>(D);
  g.capacity = static_cast<int>(capacity);
  const PartBytes parts = paged_attention_parts(T, B, capacity, Hkv, Hq / Hkv, D);
  if (parts.o > 0 && ws != nullptr && ws_bytes >= parts.all()) {
    uint8_t* base = static_cast<uint8_t*>(ws);
    g.part_rows = T * (Hq / Hkv) <= 32 ? 32 : 128;
    g.cuts = reinterpret_cast<Cut*>(base);
    g.part_ml = reinterpret_cast<float*>(base + parts.cuts);
    g.part_o = reinterpret_cast<float*>(base + parts.cuts + parts.ml);
  }
  return check_hip(launch_paged_attention(g, dtype, stream), fn);
}

}  // extern "C"
