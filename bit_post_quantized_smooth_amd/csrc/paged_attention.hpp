// Host-side launcher of the attention over a paged cache (abi_paged.hip
// validates every argument before it calls it).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "paged.hpp"

namespace svdq {

// Strides in elements: _t token, _h head; channels are contiguous.
struct PagedArgs {
  const void* q;
  void* out;
  int64_t q_t, q_h, o_t, o_h;
  Pages pages;
  const int32_t* tables;     // B x width page numbers
  const int32_t* lengths;    // B: tokens of each sequence in the cache
  const int32_t* starts;     // B + 1: each sequence's first token among the T
  const float* slopes;       // per query head, or null
  float scale, softcap;
  int causal;
  int width, B, T, Hkv, G, D;
  int capacity;              // width << page_log2
};

bool paged_attention_fits(int64_t T, int64_t Hq);
hipError_t launch_paged_attention(const PagedArgs& g, int dtype, hipStream_t stream);

}  // namespace svdq
