// Device-side pieces shared by the 8-bit attention block's kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"

namespace svdq {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// s_waitcnt immediates: all vector memory done (n = 0), or all but the newest
// n (n < 16), LDS counters left alone.
constexpr int wait_vmem(int n) { return 0x0F70 | n; }

// A raw buffer over `bytes` bytes at a wave-uniform base: lanes whose offset
// lies past the end read zero.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_buffer(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, static_cast<int>(bytes),
                                           0x00020000);
}

// 16 bytes per lane from `buf` straight into LDS at dst + 16 * lane.
__device__ __forceinline__ void buffer_to_lds16(__amdgpu_buffer_rsrc_t buf, void* dst,
                                                uint32_t offset, uint32_t soffset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      buf, (__attribute__((address_space(3))) void*)dst, 16, static_cast<int>(offset),
      static_cast<int>(soffset), 0, 0);
}

}  // namespace svdq
