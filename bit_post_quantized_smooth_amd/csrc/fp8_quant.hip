// Residual addition, RMS norm and 8-bit quantization in one pass (gfx950).
//
//   h = x + r (fp32);  residual_out = round(h);
//   u = h * (1 / sqrt(mean(h^2) + eps)) * gain;
//   per group of 128 channels: a = max|u|, s = max(fp32(a / 448), 2^-126),
//   q = e4m3_rne(u * fp32(1 / s)); channels K .. Kp-1 of the last group: q = 0.
//
// The sums are fp32 and the norm uses the unrounded h. u * fp32(1/s) is at most
// 448 (1 + 2^-22), below the 464 where rounding to nearest would leave e4m3's
// range, so no clamp is needed; a NaN stays a NaN code, and an infinity becomes
// one (its group's scale is infinite and 1/s zero).
//
// Bound by memory: every element is read once and its code written once. A
// row stays in registers between the sum and the quantization. A lane holds
// runs of 8 channels, so 16 neighbouring lanes hold one group and the group's
// maximum is four cross-lane steps. Rows of up to 2048 channels take one wave
// each (no barrier); longer ones a workgroup of 256 threads, up to 16384
// channels in registers; beyond that the row is read twice.
//
// Measured (bf16 with residual, its sum and a gain): 4608 x 12288 in 76 us, 5.2
// TB/s, which is what a large copy reaches; 96 us when each run's loads waited
// behind a branch for the row's end, and 79 us when the gain was read behind the
// sum instead of with the row. fp32 8192 x 4096: 78 us, 5.6 TB/s. 4608 x 12283,
// whose rows start at odd addresses: 100 us. One row of 5120: 4 us, all latency.
#include <hip/hip_runtime.h>

#include "../../include/svdq.h"
#include "block_common.hpp"
#include "block_launch.hpp"

namespace svdq {

namespace {

constexpr int VEC = 8;              // channels per lane and step

// 8 elements of a row whose start is only aligned to its element type: gfx950
// loads and stores global vectors at any dword or half-word address
template <class T>
struct RowVec {
  typedef T vec __attribute__((ext_vector_type(8), aligned(alignof(T))));
};

template <class T>
__device__ __forceinline__ void load8(const T* p, int64_t k, int64_t K,
                                      float (&v)[VEC]) {
  if (k + VEC <= K) {
    const auto x = *reinterpret_cast<const typename RowVec<T>::vec*>(p + k);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = static_cast<float>(x[e]);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = k + e < K ? static_cast<float>(p[k + e]) : 0.f;
  }
}

template <class T>
__device__ __forceinline__ void store8(T* p, int64_t k, int64_t K,
                                       const float (&v)[VEC]) {
  if (k + VEC <= K) {
    typename RowVec<T>::vec x;
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = static_cast<T>(v[e]);
    *reinterpret_cast<typename RowVec<T>::vec*>(p + k) = x;
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (k + e < K) p[k + e] = static_cast<T>(v[e]);
  }
}

// The maximum over the 16 lanes that hold one group.
__device__ __forceinline__ float group_max(float a) {
#pragma unroll
  for (int d = 1; d < 16; d *= 2) a = fmaxf(a, __shfl_xor(a, d));
  return a;
}

// Quantizes the 8 values u of channels k .. k+7 (k a multiple of 8, below Kp);
// lane k/8 % 16 of the group's 16.
__device__ __forceinline__ void quantize8(const float (&u)[VEC], int64_t k,
                                          uint8_t* __restrict__ codes,
                                          float* __restrict__ scales) {
  float a = 0.f;
#pragma unroll
  for (int e = 0; e < VEC; ++e) a = fmaxf(a, fabsf(u[e]));
  a = group_max(a);
  const float s = fmaxf(a / 448.0f, 1.17549435e-38f);
  const float inv = 1.0f / s;
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(u[0] * inv, u[1] * inv, lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(u[2] * inv, u[3] * inv, lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(u[4] * inv, u[5] * inv, hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(u[6] * inv, u[7] * inv, hi, true);
  *reinterpret_cast<int2*>(codes + k) = make_int2(lo, hi);
  if ((k / VEC) % (kFp8Block / VEC) == 0) scales[k / kFp8Block] = s;
}

struct QuantArgs {
  const void* X;
  const void* residual;
  const float* gain;
  uint8_t* codes;
  float* scales;
  void* residual_out;
  int64_t M, K, Kp, ldx, ldr, ldo;
  float eps;
};

template <class T>
__device__ __forceinline__ void load_h(const T* x, const T* r, int64_t k, int64_t K,
                                       float (&h)[VEC]) {
  load8(x, k, K, h);
  if (r != nullptr) {
    float t[VEC];
    load8(r, k, K, t);
#pragma unroll
    for (int e = 0; e < VEC; ++e) h[e] = h[e] + t[e];
  }
}

// u = h * rstd * gain for one run of 8 channels; channels past K come out 0
__device__ __forceinline__ void normalize8(float (&h)[VEC], float rstd, const float* gain,
                                           int64_t k, int64_t K) {
  if (gain != nullptr) {
    float g[VEC];
    load8(gain, k, K, g);
#pragma unroll
    for (int e = 0; e < VEC; ++e) h[e] = h[e] * rstd * g[e];
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) h[e] = h[e] * rstd;
  }
}

// The sum over the lanes of a row: TPR is 64 (one wave) or 256 (a workgroup).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* sums) {
#pragma unroll
  for (int d = 32; d >= 1; d /= 2) v += __shfl_xor(v, d);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = v;
    __syncthreads();
    v = sums[0];
#pragma unroll
    for (int i = 1; i < TPR / 64; ++i) v += sums[i];
  }
  return v;
}

// TPR threads per row, NV runs of 8 channels per thread in registers; NV = 0:
// any row length, read again after the sum.
//
// In registers, all of a thread's loads go out at once, without a branch for a
// run past the row or ending inside it: such a run reads the row's last 8
// channels instead (K >= 8), and afterwards takes zeros or its own few. The gain
// comes with them rather than behind the sum.
template <class T, bool NORM, int TPR, int NV>
__global__ __launch_bounds__(256) void quantize_fp8_kernel(const QuantArgs q) {
  __shared__ float sums[4];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / TPR) + threadIdx.x / TPR;
  if (row >= q.M) return;                          // whole waves only when TPR is 64
  const int t = threadIdx.x % TPR;
  const T* x = static_cast<const T*>(q.X) + row * q.ldx;
  const T* r = q.residual ? static_cast<const T*>(q.residual) + row * q.ldr : nullptr;
  T* o = q.residual_out ? static_cast<T*>(q.residual_out) + row * q.ldo : nullptr;
  uint8_t* codes = q.codes + row * q.Kp;
  float* scales = q.scales + row * (q.Kp / kFp8Block);
  constexpr int64_t step = VEC * TPR;
  if constexpr (NV > 0) {
    typedef typename RowVec<T>::vec V;
    typedef typename RowVec<float>::vec G;
    float h[NV][VEC];
    V xv[NV], rv[NV];
    G gv[NV];
    int64_t at[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t k = VEC * t + i * step;
      at[i] = k + VEC <= q.K ? k : q.K - VEC;
      xv[i] = *reinterpret_cast<const V*>(x + at[i]);
    }
    if (r != nullptr) {
#pragma unroll
      for (int i = 0; i < NV; ++i) rv[i] = *reinterpret_cast<const V*>(r + at[i]);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) rv[i][e] = static_cast<T>(-0.f);   // x + -0 is x
    }
    if constexpr (NORM) {
      if (q.gain != nullptr) {
#pragma unroll
        for (int i = 0; i < NV; ++i) gv[i] = *reinterpret_cast<const G*>(q.gain + at[i]);
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < VEC; ++e) gv[i][e] = 1.f;
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t k = VEC * t + i * step;
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        h[i][e] = at[i] == k ? static_cast<float>(xv[i][e]) + static_cast<float>(rv[i][e]) : 0.f;
      if (k < q.K && at[i] != k) load_h(x, r, k, q.K, h[i]);
    }
    float rstd = 1.f;
    if constexpr (NORM) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss = __builtin_fmaf(h[i][e], h[i][e], ss);
      rstd = 1.0f / sqrtf(row_sum<TPR>(ss, sums) / static_cast<float>(q.K) + q.eps);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t k = VEC * t + i * step;
      if (k < q.Kp) {
        if (o != nullptr) store8(o, k, q.K, h[i]);
        if constexpr (NORM) {
          if (at[i] == k || k >= q.K) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) h[i][e] = h[i][e] * rstd * gv[i][e];
          } else {
            normalize8(h[i], rstd, q.gain, k, q.K);
          }
        }
        quantize8(h[i], k, codes, scales);
      }
    }
  } else {
    float h[VEC];
    float rstd = 1.f;
    if constexpr (NORM) {
      float ss = 0.f;
      for (int64_t k = VEC * t; k < q.Kp; k += step) {
        load_h(x, r, k, q.K, h);
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss = __builtin_fmaf(h[e], h[e], ss);
      }
      rstd = 1.0f / sqrtf(row_sum<TPR>(ss, sums) / static_cast<float>(q.K) + q.eps);
    }
    for (int64_t k = VEC * t; k < q.Kp; k += step) {
      load_h(x, r, k, q.K, h);
      if (o != nullptr) store8(o, k, q.K, h);
      if constexpr (NORM) normalize8(h, rstd, q.gain, k, q.K);
      quantize8(h, k, codes, scales);
    }
  }
}

template <class T, bool NORM>
void launch_t(const QuantArgs& q, hipStream_t stream) {
  const int64_t per_wave = 64 * VEC, per_wg = 256 * VEC;
  // as many launches as the rows need, each of a grid that fits
  constexpr int64_t kMaxWgs = 0xFFFFFFFFll / 256;
  auto go = [&](auto kernel, int rows) {
    QuantArgs p = q;
    for (int64_t at = 0; at < q.M; at += kMaxWgs * rows) {
      p.X = static_cast<const T*>(q.X) + at * q.ldx;
      if (q.residual) p.residual = static_cast<const T*>(q.residual) + at * q.ldr;
      if (q.residual_out) p.residual_out = static_cast<T*>(q.residual_out) + at * q.ldo;
      p.codes = q.codes + at * q.Kp;
      p.scales = q.scales + at * (q.Kp / kFp8Block);
      p.M = q.M - at < kMaxWgs * rows ? q.M - at : kMaxWgs * rows;
      hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>((p.M + rows - 1) / rows)), dim3(256),
                         0, stream, p);
    }
  };
  if (q.K < VEC) go(quantize_fp8_kernel<T, NORM, 256, 0>, 1);
  else if (q.Kp <= per_wave) go(quantize_fp8_kernel<T, NORM, 64, 1>, 4);
  else if (q.Kp <= 2 * per_wave) go(quantize_fp8_kernel<T, NORM, 64, 2>, 4);
  else if (q.Kp <= 3 * per_wave) go(quantize_fp8_kernel<T, NORM, 64, 3>, 4);
  else if (q.Kp <= 4 * per_wave) go(quantize_fp8_kernel<T, NORM, 64, 4>, 4);
  else if (q.Kp <= 2 * per_wg) go(quantize_fp8_kernel<T, NORM, 256, 2>, 1);
  else if (q.Kp <= 3 * per_wg) go(quantize_fp8_kernel<T, NORM, 256, 3>, 1);
  else if (q.Kp <= 4 * per_wg) go(quantize_fp8_kernel<T, NORM, 256, 4>, 1);
  else if (q.Kp <= 6 * per_wg) go(quantize_fp8_kernel<T, NORM, 256, 6>, 1);
  else if (q.Kp <= 8 * per_wg) go(quantize_fp8_kernel<T, NORM, 256, 8>, 1);
  else go(quantize_fp8_kernel<T, NORM, 256, 0>, 1);
}

template <class T>
void launch_n(const QuantArgs& q, bool norm, hipStream_t stream) {
  norm ? launch_t<T, true>(q, stream) : launch_t<T, false>(q, stream);
}

}  // namespace

hipError_t launch_quantize_fp8(const void* X, const void* residual, int dtype, int64_t M,
                               int64_t K, int64_t ldx, int64_t ldr, bool norm, const float* gain,
                               float eps, uint8_t* codes, float* scales, void* residual_out,
                               int64_t ldo, hipStream_t stream) {
  const QuantArgs q{X, residual, gain, codes, scales, residual_out, M, K, fp8_padded(K),
                    ldx, ldr, ldo, eps};
  if (dtype == SVDQ_F16) launch_n<_Float16>(q, norm, stream);
  else if (dtype == SVDQ_BF16) launch_n<__bf16>(q, norm, stream);
  else launch_n<float>(q, norm, stream);
  return hipGetLastError();
}

}  // namespace svdq
