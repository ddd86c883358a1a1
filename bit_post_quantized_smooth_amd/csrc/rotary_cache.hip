// Norm and rotation of query and key heads, and the cache's pages (gfx950).
//
//   u = x / sqrt(mean(x^2) + eps) * gain        (over the head's D channels; optional)
//   a pair (a, b) of the first 2 * pairs channels, at the token's position:
//     (a, b) <- factor * (a cos - b sin, a sin + b cos)
//   queries, and keys without pages: rounded to 16 bits;
//   keys and values with pages: rounded to 16 bits, or to codes
//     e4m3_rne(clamp(u * fp32(1 / s), -448, 448)) with the head's scale s (two roundings of
//     2^-24 where a division has one, so that a value as near a midpoint of two codes may
//     take the other, for one instruction an element instead of ten; 1 / s is in fp32 for
//     scales in 2^-64 .. 2^64).
//
// Sums, norms and rotations are fp32 and a value is rounded once. A code keeps a
// relative precision of 2^-4 over 2^15 of range, so one scale per head, chosen
// beforehand, serves all tokens: a scale per token would have to be read with its
// row and would turn the scores' one factor into one per key. Finite values beyond
// 448 s are clamped to it, infinities become the NaN code, so that they are not lost.
//
// Bound by memory: each element is read once and written once. 16 lanes (8 up to
// 64 channels) hold a head, 8 channels each. A workgroup takes one operand's heads, up to
// four of a token per lane, so that the angles' sines and cosines are computed once for
// them and their loads are in flight together. Sums over a head and the exchange of halves are
// lane moves inside the vector unit; only a rotation of part of the head goes through LDS, and
// one whose halves begin inside a lane's channels reads the partners from memory again.
//
// Measured: 4608 tokens of 24 + 24 heads of 128, fp16, norm and rotation: 24.5 to 25 us, 4.6 TB/s (a
// copy of as many bytes 23.3); 8191 tokens, 32/8 heads into e4m3 pages: 42.8 us, 4.3 TB/s (35.8);
// one token 3.4 us, and 5.9 to 6.4 with its call. Operands chosen per lane, with branches around each load:
// 49 and 98 us. Reads of 8 sequences of up to 8191 out of e4m3 pages: 65.7 us, 4.8 TB/s (59.1).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

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

// Where a channel's partner lies: there is none; the next or last channel; in the lane
// half a head away, where all LPR lanes' channels turn; in another lane; or (pairs not a
// multiple of 8) anywhere, read from memory again.
enum { kStay, kNext, kOpposite, kLanes, kFar };

template <int CTRL, int BANKS>
__device__ __forceinline__ float dpp(float old, float x) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, old), __builtin_bit_cast(int, x), CTRL,
                                         0xF, BANKS, false));
}
// The value of the lane half of LPR lanes away, within 16 lanes' registers.
template <int LPR>
__device__ __forceinline__ float opposite(float x) {
  if constexpr (LPR == 16) return dpp<0x128, 0xF>(x, x);             // rotate by 8
  return dpp<0x114, 0xA>(dpp<0x104, 0x5>(x, x), x);                  // 4 up, 4 down
}
// The sum over LPR lanes: neighbours, pairs, mirrored fours, mirrored eights.
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
  x += dpp<0xB1, 0xF>(x, x);
  x += dpp<0x4E, 0xF>(x, x);
  x += dpp<0x141, 0xF>(x, x);
  if constexpr (LPR == 16) x += dpp<0x140, 0xF>(x, x);
  return x;
}
template <int LPR>
__device__ __forceinline__ float row_max(float x) {
  x = fmaxf(x, dpp<0xB1, 0xF>(x, x));
  x = fmaxf(x, dpp<0x4E, 0xF>(x, x));
  x = fmaxf(x, dpp<0x141, 0xF>(x, x));
  if constexpr (LPR == 16) x = fmaxf(x, dpp<0x140, 0xF>(x, x));
  return x;
}

// e4m3 codes of 8 values, two dwords
__device__ __forceinline__ int2 codes8(const float (&u)[VEC], float inv) {
  float x[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    const float kept = __builtin_amdgcn_fmed3f(u[e] * inv, -448.f, 448.f);
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

// LPR lanes per head; a workgroup takes up to HPG heads of one operand for 256 / LPR tokens,
// so that which operand it is, and whether it turns, is the same for all its lanes. Loads
// have no branch around them: what lies behind the last token, head or channel reads the
// last one again and is not stored.
template <class T, int MODE, int LPR, int HPG>
__global__ __launch_bounds__(kThreads) void heads_kernel(const HeadsArgs g) {
  typedef typename Vec8<T>::vec vec;
  const int chunk = static_cast<int>(blockIdx.x) % g.chunks;
  const int tokens = static_cast<int>(blockIdx.x) / g.chunks;
  const bool is_q = chunk < g.q_chunks, is_v = chunk >= g.q_chunks + g.k_chunks;
  const int head0 = HPG * (is_q ? chunk : is_v ? chunk - g.q_chunks - g.k_chunks : chunk - g.q_chunks);
  const int H = is_q ? g.Hq : g.Hkv;
  const T* src = static_cast<const T*>(is_q ? g.q : is_v ? g.v : g.k);
  const int64_t src_t = is_q ? g.q_t : is_v ? g.v_t : g.k_t;
  const int64_t src_h = is_q ? g.q_h : is_v ? g.v_h : g.k_h;
  const bool turn = MODE != kStay && !is_v, norm = g.norm && !is_v;

  const int rl = threadIdx.x % LPR, c0 = VEC * rl;
  const int64_t t0 = static_cast<int64_t>(tokens) * (kThreads / LPR) + threadIdx.x / LPR;
  const int64_t t = t0 < g.T ? t0 : g.T - 1;
  const bool inside = c0 < g.D;
  const int c = inside ? c0 : 0;

  src += t * src_t + c;
  vec raw[HPG];
#pragma unroll
  for (int i = 0; i < HPG; ++i) {
    const int h = head0 + i < H ? head0 + i : H - 1;
    raw[i] = *reinterpret_cast<const vec*>(src + h * src_h);
  }
  const int64_t slot = g.slots != nullptr && !is_q ? g.slots[t] : 0;
  const float* gain = is_q ? g.q_gain : g.k_gain;
  float gains[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) gains[e] = 1.f;
  if (norm && gain != nullptr) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) gains[e] = gain[c + e];
  }
  // cosine and signed sine of each channel; the channels behind R stay as they are
  const int R = 2 * g.pairs;
  float cs[VEC], sn[VEC];
  if (turn) {
    const int32_t position = g.positions[t];
    double freq[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if (MODE == kNext && (e & 1)) continue;
      const int ch = c0 + e;
      const int pair = ch >= R ? 0 : MODE == kNext ? ch / 2 : ch < g.pairs ? ch : ch - g.pairs;
      freq[e] = g.freqs[pair];
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const bool first = MODE == kNext ? (e & 1) == 0 : c0 + e < g.pairs;
      if (MODE == kNext && (e & 1)) {
        cs[e] = cs[e - 1];
        sn[e] = -sn[e - 1];
        continue;
      }
      cos_sin(position, freq[e], cs[e], sn[e]);
      cs[e] = cs[e] * g.factor;
      sn[e] = sn[e] * (first ? -g.factor : g.factor);
    }
  }

  // where the rows go
  const Pages& pg = g.pages;
  const bool paged = g.slots != nullptr && !is_q;
  const bool stored = inside && t0 < g.T && (!paged || (slot >= 0 && slot < (pg.count << pg.page_log2)));
  char* to;
  int64_t to_h;
  if (paged) {
    const int esize = pg.coded ? 1 : 2;
    to = static_cast<char*>(is_v ? pg.v : pg.k) + (slot >> pg.page_log2) * (is_v ? pg.v_stride : pg.k_stride) +
         ((slot & ((1 << pg.page_log2) - 1)) * g.D + c) * esize;
    to_h = static_cast<int64_t>(g.D * esize) << pg.page_log2;
  } else {
    to = static_cast<char*>(is_q ? g.q_out : g.k_out) + (t * (is_q ? g.qo_t : g.ko_t) + c) * 2;
    to_h = (is_q ? g.qo_h : g.ko_h) * 2;
  }
  const float* scales = is_v ? pg.v_scales : pg.k_scales;

#pragma unroll
  for (int i = 0; i < HPG; ++i) {
    const int h = head0 + i;
    if (h >= H) break;
    float u[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) u[e] = static_cast<float>(raw[i][e]);
    float root = 1.f, unit = 1.f;
    if (norm) {
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) sum = __builtin_fmaf(u[e], u[e], sum);
      float mean = __builtin_fmaf(row_sum<LPR>(inside ? sum : 0.f), g.inv_D, g.eps);
      // squares beyond fp32 (bf16 values above 2^63) or below it (with an eps as small):
      // of values in units of the row's largest. The values take the unit before the root:
      // the two multiplied can leave fp32 (a row below 2^-128).
      const bool far = !(mean >= 0x1p-100f && mean < __builtin_inff());
      if (__builtin_amdgcn_ballot_w64(far) != 0) {
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) top = fmaxf(top, fabsf(u[e]));
        top = row_max<LPR>(inside ? top : 0.f);
        if (far && top > 0.f && top < __builtin_inff()) {
          unit = __builtin_ldexpf(1.f, min(max(-__builtin_amdgcn_frexp_expf(top), -126), g.most_unit));
          sum = 0.f;
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            u[e] = u[e] * unit;
            sum = __builtin_fmaf(u[e], u[e], sum);
          }
        }
        sum = row_sum<LPR>(inside ? sum : 0.f);
        if (unit != 1.f) mean = __builtin_fmaf(sum, g.inv_D, g.eps * unit * unit);
      }
      root = __builtin_amdgcn_rsqf(mean);
#pragma unroll
      for (int e = 0; e < VEC; ++e) u[e] = u[e] * root * gains[e];
    }
    if (turn) {
      float p[VEC];
      if constexpr (MODE == kNext) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) p[e] = u[e ^ 1];
      } else if constexpr (MODE == kOpposite) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) p[e] = opposite<LPR>(u[e]);
      } else if constexpr (MODE == kLanes) {
        const int step = g.pairs / VEC, from = rl < step ? rl + step : rl - step;
        const int lane = static_cast<int>(threadIdx.x & 63) - rl + (from < LPR ? from : rl);
#pragma unroll
        for (int e = 0; e < VEC; ++e) p[e] = __shfl(u[e], lane);
      } else if constexpr (MODE == kFar) {
        const T* x = src + h * src_h - c;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int ch = c0 + e, other = ch >= R ? 0 : ch < g.pairs ? ch + g.pairs : ch - g.pairs;
          p[e] = static_cast<float>(x[other]);
          if (norm) p[e] = p[e] * unit * root * (gain != nullptr ? gain[other] : 1.f);
        }
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float v = __builtin_fmaf(u[e], cs[e], p[e] * sn[e]);
        u[e] = MODE == kOpposite || c0 + e < R ? v : u[e];
      }
    }
    if (stored) {
      if (paged && pg.coded)
        *reinterpret_cast<int2*>(to + h * to_h) = codes8(u, scales != nullptr ? 1.0f / scales[h] : 1.f);
      else
        store16(reinterpret_cast<T*>(to + h * to_h), u);
    }
  }
}

template <class T, int MODE, int LPR>
hipError_t launch_l(HeadsArgs g, hipStream_t stream) {
  // Four heads per lane share the angles and have their loads in flight together (8191
  // tokens of 32/8 heads into codes 44 us; one head 80, two 52, eight 44; 4608 of 48: 25.5, 32,
  // 26 and 28), where that leaves 1024 waves (1031 tokens of 24 heads: 5.6 us, one head 6.9);
  // else one (777 tokens of 10 heads: 3.0 us, four 3.4).
  constexpr int kPer = 4;
  const bool many = static_cast<int64_t>(g.T) * g.heads * LPR >= int64_t{kPer} * 1024 * 64;
  const int per = many ? kPer : 1;
  g.q_chunks = (g.Hq + per - 1) / per;
  g.k_chunks = (g.Hkv + per - 1) / per;
  g.chunks = g.q_chunks + (g.slots != nullptr ? 2 : 1) * g.k_chunks;
  g.inv_D = 1.0f / static_cast<float>(g.D);
  g.most_unit = g.eps > 0.f ? std::min(126, (100 - std::ilogb(g.eps)) / 2) : 126;   // eps * 2^(2 unit) stays finite
  const int64_t blocks = (static_cast<int64_t>(g.T) + kThreads / LPR - 1) / (kThreads / LPR) * g.chunks;
  const unsigned grid = static_cast<unsigned>(blocks);
  if (many)
    hipLaunchKernelGGL((heads_kernel<T, MODE, LPR, kPer>), dim3(grid), dim3(kThreads), 0, stream, g);
  else
    hipLaunchKernelGGL((heads_kernel<T, MODE, LPR, 1>), dim3(grid), dim3(kThreads), 0, stream, g);
  return hipGetLastError();
}

template <class T, int LPR>
hipError_t launch_m(const HeadsArgs& g, hipStream_t stream) {
  if (g.pairs == 0) return launch_l<T, kStay, LPR>(g, stream);
  if (g.interleaved) return launch_l<T, kNext, LPR>(g, stream);
  if (2 * g.pairs == VEC * LPR) return launch_l<T, kOpposite, LPR>(g, stream);
  return g.pairs % VEC == 0 ? launch_l<T, kLanes, LPR>(g, stream) : launch_l<T, kFar, LPR>(g, stream);
}

template <class T>
hipError_t launch_t(const HeadsArgs& g, hipStream_t stream) {
  return g.D > 64 ? launch_m<T, 16>(g, stream) : launch_m<T, 8>(g, stream);
}

// Rows back from their pages: a group of lanes takes kPerRead heads of a token, keys and
// values, with the loads of all on their way together; 8 channels a lane, so that 16
// bytes of one lane's are stored beside the next one's (16 codes a lane, whose 32 bytes are
// stored in two halves: 76 us where these take 66, 8 sequences of up to 8191).
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
  constexpr int esize = CODED ? 1 : 2;
  const int64_t in_page = (j & ((1 << pg.page_log2) - 1)) * g.D + c0, per_head = static_cast<int64_t>(g.D) << pg.page_log2;
  const char* from[2] = {static_cast<const char*>(pg.k) + page * pg.k_stride + in_page * esize,
                         static_cast<const char*>(pg.v) + page * pg.v_stride + in_page * esize};
  T* to[2] = {static_cast<T*>(g.k_out) + b * g.k_b + j * g.k_t + c0, static_cast<T*>(g.v_out) + b * g.v_b + j * g.v_t + c0};
  typedef int loaded __attribute__((ext_vector_type(CODED ? 2 : 4)));
  loaded x[2][kPerRead];
#pragma unroll
  for (int i = 0; i < kPerRead; ++i) {
    const int h = min(head0 + i, g.Hkv - 1);
#pragma unroll
    for (int o = 0; o < 2; ++o) x[o][i] = *reinterpret_cast<const loaded*>(from[o] + h * per_head * esize);
  }
#pragma unroll
  for (int i = 0; i < kPerRead; ++i) {
    const int h = head0 + i;
    if (h >= g.Hkv) break;
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      T* out = to[o] + h * (o ? g.v_h : g.k_h);
      if constexpr (CODED) {
        const float* scales = o ? pg.v_scales : pg.k_scales;
        const float s = scales != nullptr ? scales[h] : 1.f;
        float u[VEC];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int word = x[o][i][e];
          const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8(word, false);
          const v2f hi = __builtin_amdgcn_cvt_pk_f32_fp8(word, true);
          u[4 * e] = lo[0] * s;
          u[4 * e + 1] = lo[1] * s;
          u[4 * e + 2] = hi[0] * s;
          u[4 * e + 3] = hi[1] * s;
        }
        store16(out, u);
      } else {
        *reinterpret_cast<v4i*>(out) = x[o][i];
      }
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
  return heads <= (int64_t{1} << 20) && T <= 0x7FFFFFFFll && grid_fits((T / (kThreads / 16) + 1) * heads, kThreads);
}
bool read_fits(int64_t B, int64_t L, int64_t Hkv) {
  const int64_t per = (Hkv + kPerRead - 1) / kPerRead;
  return L == 0 || (B <= (int64_t{1} << 40) / L && grid_fits(B * L * per / (kThreads / 16) + 1, kThreads));
}

hipError_t launch_heads(HeadsArgs g, int dtype, hipStream_t stream) {
  g.heads = g.Hq + (g.slots != nullptr ? 2 : 1) * g.Hkv;
  return dtype == SVDQ_F16 ? launch_t<_Float16>(g, stream) : launch_t<__bf16>(g, stream);
}

hipError_t launch_read(ReadArgs g, int dtype, hipStream_t stream) {
  g.chunks = (g.Hkv + kPerRead - 1) / kPerRead;
  return dtype == SVDQ_F16 ? launch_rt<_Float16>(g, stream) : launch_rt<__bf16>(g, stream);
}

}  // namespace svdq
