// Norm and rotation of query and key heads, and the cache's pages (gfx950).
//
//   u = x / sqrt(mean(x^2) + eps) * gain        (over the head's D channels; optional)
//   a pair (a, b) of the first 2 * pairs channels, at the token's position:
//     (a, b) <- factor * (a cos - b sin, a sin + b cos)
//   queries, and keys without pages: rounded to 16 bits;
//   keys and values with pages: rounded to 16 bits, or to codes
//     e4m3_rne(clamp(u * fp32(1 / s), -448, 448)) with the head's scale s.
//
// Sums, norms and rotations are fp32 and a value is rounded once. A code keeps a
// relative precision of 2^-4 over 2^15 of range, so one scale per head, chosen
// beforehand, serves all tokens: a scale per token would have to be read with its
// row and would turn the scores' one factor into one per key. Finite values beyond
// 448 s are clamped to it, infinities become the NaN code, so that they are not lost.
//
// Bound by memory: each element is read once and written once. 16 lanes (8 up to
// 64 channels) hold a head, 8 channels each, and take several heads of one token
// in turn, so that the angles' sines and cosines are computed once for them and
// their loads are in flight together.
#include <hip/hip_runtime.h>

#include "../../include/svdq.h"
#include "block_common.hpp"
#include "block_launch.hpp"
#include "head_rotation.hpp"
#include "paged.hpp"

namespace svdq {

namespace {

constexpr int VEC = 8;
constexpr int kThreads = 256;

template <class T>
struct Vec8 {
  typedef T vec __attribute__((ext_vector_type(8)));
};

// Where a channel's partner lies: the next or last channel, 8 channels of another
// lane, or (pairs not a multiple of 8) anywhere, read from memory again.
enum { kStay = 0, kNext = 1, kLanes = 2, kFar = 3 };

// e4m3 codes of 8 values, two dwords
__device__ __forceinline__ int2 codes8(const float (&u)[VEC], float inv) {
  float x[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    const float y = u[e] * inv;
    const float kept = fminf(fmaxf(y, -448.f), 448.f);
    x[e] = fabsf(u[e]) < __builtin_inff() ? kept : __builtin_nanf("");
  }
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], hi, true);
  return make_int2(lo, hi);
}

template <class T>
__device__ __forceinline__ void store16(T* p, const float (&u)[VEC]) {
  typename Vec8<T>::vec y;
#pragma unroll
  for (int e = 0; e < VEC; ++e) y[e] = static_cast<T>(u[e]);
  *reinterpret_cast<typename Vec8<T>::vec*>(p) = y;
}

// LPR lanes per head, HPG heads of a token per group of lanes.
template <class T, int STORE, int LPR, int HPG>
__global__ __launch_bounds__(kThreads) void heads_kernel(const HeadsArgs g) {
  typedef typename Vec8<T>::vec vec;
  const int64_t group = static_cast<int64_t>(blockIdx.x) * (kThreads / LPR) + threadIdx.x / LPR;
  const int t = static_cast<int>(group / g.chunks);
  if (t >= g.T) return;                            // all lanes of a group together
  const int head0 = static_cast<int>(group % g.chunks) * HPG;
  const int rl = threadIdx.x % LPR, c0 = VEC * rl;
  const bool active = c0 < g.D;
  const int64_t slot = STORE != kNoPages ? g.slots[t] : -1;
  const bool stored = STORE == kNoPages ||
                      (slot >= 0 && slot < (g.pages.count << g.pages.page_log2));

  // source of head h of the list queries, keys, values
  auto source = [&](int h) {
    const bool is_q = h < g.Hq, is_k = h < g.Hq + g.Hkv;
    const T* base = static_cast<const T*>(is_q ? g.q : is_k ? g.k : g.v);
    const int64_t st = is_q ? g.q_t : is_k ? g.k_t : g.v_t, sh = is_q ? g.q_h : is_k ? g.k_h : g.v_h;
    const int hh = is_q ? h : is_k ? h - g.Hq : h - g.Hq - g.Hkv;
    return base + t * st + hh * sh;
  };
  vec raw[HPG];
#pragma unroll
  for (int i = 0; i < HPG; ++i) {
    const int h = head0 + i;
#pragma unroll
    for (int e = 0; e < VEC; ++e) raw[i][e] = static_cast<T>(0.f);
    if (active && h < g.heads && (h < g.Hq || stored))
      raw[i] = *reinterpret_cast<const vec*>(source(h) + c0);
  }

  const int R = 2 * g.pairs;
  const int mode = R == 0 ? kStay : g.interleaved ? kNext : g.pairs % VEC == 0 ? kLanes : kFar;
  // cosine and signed sine of each channel; the channels behind R stay as they are
  float cs[VEC], sn[VEC];
  int other[VEC];                                  // the partner's channel
  if (mode != kStay) {
    const int32_t position = g.positions[t];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int c = c0 + e;
      const bool first = mode == kNext ? (e & 1) == 0 : c < g.pairs;
      const int pair = mode == kNext ? c / 2 : first ? c : c - g.pairs;
      other[e] = mode == kNext ? c ^ 1 : first ? c + g.pairs : c - g.pairs;
      cs[e] = 1.f;
      sn[e] = 0.f;
      if (c < R) {
        if (mode == kNext && !first) {
          cs[e] = cs[e - (e & 1)];
          sn[e] = -sn[e - (e & 1)];
        } else {
          cos_sin(position, g.freqs[pair], cs[e], sn[e]);
          cs[e] = cs[e] * g.factor;
          sn[e] = sn[e] * (first ? -g.factor : g.factor);
        }
      }
    }
  }
  float gq[VEC], gk[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) gq[e] = gk[e] = 1.f;
  if (g.norm && active) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if (g.q_gain != nullptr) gq[e] = g.q_gain[c0 + e];
      if (g.k_gain != nullptr) gk[e] = g.k_gain[c0 + e];
    }
  }

#pragma unroll
  for (int i = 0; i < HPG; ++i) {
    const int h = head0 + i;
    if (h >= g.heads) break;
    const bool is_q = h < g.Hq, is_v = h >= g.Hq + g.Hkv;
    if (!is_q && !stored) continue;
    float u[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) u[e] = static_cast<float>(raw[i][e]);
    float rstd = 1.f;
    if (g.norm && !is_v) {
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) sum = __builtin_fmaf(u[e], u[e], sum);
#pragma unroll
      for (int d = 1; d < LPR; d *= 2) sum += __shfl_xor(sum, d);
      rstd = 1.0f / sqrtf(sum / static_cast<float>(g.D) + g.eps);
#pragma unroll
      for (int e = 0; e < VEC; ++e) u[e] = u[e] * rstd * (is_q ? gq[e] : gk[e]);
    }
    if (mode != kStay && !is_v) {
      float p[VEC];
      if (mode == kNext) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) p[e] = u[e ^ 1];
      } else if (mode == kLanes) {
        const int step = g.pairs / VEC;
        const int from = rl < step ? rl + step : rl - step;
        const int lane = static_cast<int>(threadIdx.x & 63) - rl + (from < LPR ? from : rl);
#pragma unroll
        for (int e = 0; e < VEC; ++e) p[e] = __shfl(u[e], lane);
      } else {
        const T* x = source(h);
        const float* gain = is_q ? g.q_gain : g.k_gain;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          p[e] = 0.f;
          if (active && c0 + e < R) {
            p[e] = static_cast<float>(x[other[e]]);
            if (g.norm) p[e] = p[e] * rstd * (gain != nullptr ? gain[other[e]] : 1.f);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (c0 + e < R) u[e] = __builtin_fmaf(u[e], cs[e], p[e] * sn[e]);
    }
    if (!active) continue;
    if (is_q) {
      store16(static_cast<T*>(g.q_out) + t * g.qo_t + h * g.qo_h + c0, u);
      continue;
    }
    const int hh = is_v ? h - g.Hq - g.Hkv : h - g.Hq;
    if constexpr (STORE == kNoPages) {
      store16(static_cast<T*>(g.k_out) + t * g.ko_t + hh * g.ko_h + c0, u);
    } else {
      const Pages& pg = g.pages;
      const int64_t row = (static_cast<int64_t>(hh) << pg.page_log2) +
                          (slot & ((1 << pg.page_log2) - 1));
      char* page = static_cast<char*>(is_v ? pg.v : pg.k) +
                   (slot >> pg.page_log2) * (is_v ? pg.v_stride : pg.k_stride);
      if constexpr (STORE == kHalfPages) {
        store16(reinterpret_cast<T*>(page) + row * g.D + c0, u);
      } else {
        const float* scales = is_v ? pg.v_scales : pg.k_scales;
        const float inv = scales != nullptr ? 1.0f / scales[hh] : 1.f;
        *reinterpret_cast<int2*>(page + row * g.D + c0) = codes8(u, inv);
      }
    }
  }
}

template <class T, int STORE, int LPR>
hipError_t launch_l(HeadsArgs g, hipStream_t stream) {
  // One head per group of lanes while that leaves lanes idle.
  constexpr int kPer = 8;
  const bool many = static_cast<int64_t>(g.T) * g.heads * LPR >= int64_t{kPer} * 2048 * 64;
  g.chunks = many ? (g.heads + kPer - 1) / kPer : g.heads;
  const int64_t groups = static_cast<int64_t>(g.T) * g.chunks;
  const unsigned grid = static_cast<unsigned>((groups + kThreads / LPR - 1) / (kThreads / LPR));
  if (many)
    hipLaunchKernelGGL((heads_kernel<T, STORE, LPR, kPer>), dim3(grid), dim3(kThreads), 0, stream, g);
  else
    hipLaunchKernelGGL((heads_kernel<T, STORE, LPR, 1>), dim3(grid), dim3(kThreads), 0, stream, g);
  return hipGetLastError();
}

template <class T>
hipError_t launch_t(const HeadsArgs& g, int store, hipStream_t stream) {
  if (g.D > 64)
    return store == kNoPages     ? launch_l<T, kNoPages, 16>(g, stream)
           : store == kHalfPages ? launch_l<T, kHalfPages, 16>(g, stream)
                                 : launch_l<T, kCodePages, 16>(g, stream);
  return store == kNoPages     ? launch_l<T, kNoPages, 8>(g, stream)
         : store == kHalfPages ? launch_l<T, kHalfPages, 8>(g, stream)
                               : launch_l<T, kCodePages, 8>(g, stream);
}

// Rows back from their pages: LPR lanes per row, kPerRead heads of a token each.
constexpr int kPerRead = 4;

template <class T, bool CODED, int LPR>
__global__ __launch_bounds__(kThreads) void read_kernel(const ReadArgs g) {
  const int64_t group = static_cast<int64_t>(blockIdx.x) * (kThreads / LPR) + threadIdx.x / LPR;
  const int64_t token = group / g.chunks;
  const int head0 = static_cast<int>(group % g.chunks) * kPerRead;
  const int64_t b = token / g.L;
  if (b >= g.B) return;
  const int j = static_cast<int>(token % g.L), c0 = VEC * (threadIdx.x % LPR);
  const Pages& pg = g.pages;
  if (j >= g.lengths[b] || j >> pg.page_log2 >= g.width || c0 >= g.D) return;
  const int64_t page = g.tables[b * g.width + (j >> pg.page_log2)];
  if (page < 0 || page >= pg.count) return;
  typedef typename Vec8<T>::vec vec;
  const int64_t in_page = j & ((1 << pg.page_log2) - 1);
#pragma unroll
  for (int i = 0; i < 2 * kPerRead; ++i) {
    const int h = head0 + i / 2;
    if (h >= g.Hkv) break;
    const bool is_v = i & 1;
    const char* base = static_cast<const char*>(is_v ? pg.v : pg.k) +
                       page * (is_v ? pg.v_stride : pg.k_stride);
    const int64_t at = ((static_cast<int64_t>(h) << pg.page_log2) + in_page) * g.D + c0;
    T* out = is_v ? static_cast<T*>(g.v_out) + b * g.v_b + j * g.v_t + h * g.v_h + c0
                  : static_cast<T*>(g.k_out) + b * g.k_b + j * g.k_t + h * g.k_h + c0;
    if constexpr (CODED) {
      const float* scales = is_v ? pg.v_scales : pg.k_scales;
      const float s = scales != nullptr ? scales[h] : 1.f;
      const int2 w = *reinterpret_cast<const int2*>(base + at);
      float u[VEC];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int word = e ? w.y : w.x;
        const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8(word, false);
        const v2f hi = __builtin_amdgcn_cvt_pk_f32_fp8(word, true);
        u[4 * e] = lo[0] * s;
        u[4 * e + 1] = lo[1] * s;
        u[4 * e + 2] = hi[0] * s;
        u[4 * e + 3] = hi[1] * s;
      }
      store16(out, u);
    } else {
      *reinterpret_cast<vec*>(out) = *reinterpret_cast<const vec*>(reinterpret_cast<const T*>(base) + at);
    }
  }
}

template <class T, bool CODED, int LPR>
hipError_t launch_r(const ReadArgs& g, hipStream_t stream) {
  const int64_t groups = static_cast<int64_t>(g.B) * g.L * g.chunks;
  const unsigned grid = static_cast<unsigned>((groups + kThreads / LPR - 1) / (kThreads / LPR));
  hipLaunchKernelGGL((read_kernel<T, CODED, LPR>), dim3(grid), dim3(kThreads), 0, stream, g);
  return hipGetLastError();
}

template <class T>
hipError_t launch_rt(const ReadArgs& g, hipStream_t stream) {
  if (g.D > 64)
    return g.pages.coded ? launch_r<T, true, 16>(g, stream) : launch_r<T, false, 16>(g, stream);
  return g.pages.coded ? launch_r<T, true, 8>(g, stream) : launch_r<T, false, 8>(g, stream);
}

}  // namespace

bool heads_fit(int64_t T, int64_t heads) {
  return heads <= (int64_t{1} << 20) && T <= 0x7FFFFFFFll && grid_fits(T * heads / (kThreads / 16) + 1, kThreads);
}
bool read_fits(int64_t B, int64_t L, int64_t Hkv) {
  const int64_t per = (Hkv + kPerRead - 1) / kPerRead;
  return L == 0 || (B <= (int64_t{1} << 40) / L && grid_fits(B * L * per / (kThreads / 16) + 1, kThreads));
}

hipError_t launch_heads(HeadsArgs g, int dtype, int store, hipStream_t stream) {
  g.heads = g.Hq + (store == kNoPages ? 1 : 2) * g.Hkv;
  return dtype == SVDQ_F16 ? launch_t<_Float16>(g, store, stream) : launch_t<__bf16>(g, store, stream);
}

hipError_t launch_read(ReadArgs g, int dtype, hipStream_t stream) {
  g.chunks = (g.Hkv + kPerRead - 1) / kPerRead;
  return dtype == SVDQ_F16 ? launch_rt<_Float16>(g, stream) : launch_rt<__bf16>(g, stream);
}

}  // namespace svdq
