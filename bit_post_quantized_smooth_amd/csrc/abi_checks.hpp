// What the entry points of the 8-bit block and of the paged cache check and report alike.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/svdq.h"
#include "host_internal.hpp"

namespace svdq {

constexpr int64_t kMaxStride = int64_t{1} << 40;

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int fail(int status, const char* fn, const char* what) {
  set_error("%s: %s", fn, what);
  return status;
}

inline int device_ready(const char* fn) {
  int dev = -1;
  const hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess || dev < 0) {
    (void)hipGetLastError();
    set_error("%s: no usable GPU: %s", fn, hipGetErrorString(e));
    return SVDQ_ERR_NO_DEVICE;
  }
  return SVDQ_OK;
}

inline int check_hip(hipError_t e, const char* fn) {
  if (e != hipSuccess) {
    set_error("%s launch: %s", fn, hipGetErrorString(e));
    return SVDQ_ERR_HIP;
  }
  return SVDQ_OK;
}

}  // namespace svdq
