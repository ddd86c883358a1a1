// Host-side launchers of the 8-bit attention block's kernels (abi_block.hip
// validates every argument before it calls them).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace svdq {

constexpr int kFp8Block = 128;      // channels per e4m3 scale

// A launch takes fewer than 2^32 threads: more are not refused, their number is cut
// to 32 bits and the rest of the grid never runs.
inline bool grid_fits(int64_t wgs, int threads) { return wgs <= 0xFFFFFFFFll / threads; }

inline int64_t fp8_padded(int64_t K) { return (K + kFp8Block - 1) / kFp8Block * kFp8Block; }

// norm: the RMS norm (gain may be null, eps); else the rows are quantized as
// they are. residual and residual_out may be null. dtype: SVDQ_F16, SVDQ_F32
// or SVDQ_BF16, of X, residual and residual_out.
hipError_t launch_quantize_fp8(const void* X, const void* residual, int dtype, int64_t M,
                               int64_t K, int64_t ldx, int64_t ldr, bool norm, const float* gain,
                               float eps, uint8_t* codes, float* scales, void* residual_out,
                               int64_t ldo, hipStream_t stream);

// part: part_bytes (16-byte aligned) for the fp32 partial tiles of a product
// that is split along K; with fewer than gemm_fp8_split_bytes(M, N, Kp), or a
// null pointer, the product may run unsplit.
hipError_t launch_gemm_fp8(const uint8_t* a_codes, const float* a_scales, const uint8_t* w_codes,
                           const float* w_scales, const float* bias, void* Y, int y_dtype,
                           int64_t M, int64_t N, int64_t Kp, int64_t ldy, bool gelu, float* part,
                           size_t part_bytes, hipStream_t stream);
size_t gemm_fp8_split_bytes(int64_t M, int64_t N, int64_t Kp);
// Whether a kernel's grid can cover M x N.
bool gemm_fp8_fits(int64_t M, int64_t N, int y_dtype);

}  // namespace svdq
