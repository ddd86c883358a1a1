// Host-side launchers of the paged key-value cache's kernels (abi_paged.hip
// validates every argument before it calls them).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace svdq {

// Pages of one pool: page p at base + p * stride bytes, in it Hkv heads of
// 2^page_log2 tokens of D channels, 16 bits or e4m3 codes. A slot is
// page << page_log2 | token in the page.
struct Pages {
  void* k;
  void* v;
  int64_t k_stride, v_stride;      // bytes between pages
  int64_t count;                   // pages in the pool
  const float* k_scales;           // per head, of e4m3 codes; null: 1
  const float* v_scales;
  int page_log2;
  int coded;                       // e4m3 codes; else the type of the queries
};

// Strides in elements: _t token, _h head; channels are contiguous.
struct HeadsArgs {
  const void* q;
  const void* k;
  const void* v;                   // null without pages
  void* q_out;
  void* k_out;                     // null with pages
  int64_t q_t, q_h, k_t, k_h, v_t, v_h, qo_t, qo_h, ko_t, ko_h;
  const int32_t* positions;
  const double* freqs;             // radians per position of each pair
  const float* q_gain;
  const float* k_gain;
  const int32_t* slots;            // per token; null: no pages
  Pages pages;
  float factor, eps;
  int pairs;                       // 0: no rotation
  int interleaved, norm;
  int T, Hq, Hkv, D;
  int heads, q_chunks, k_chunks, chunks;   // set by launch_heads
  float inv_D;
  int most_unit;
};

// Whether one launch covers T tokens of this many heads.
bool heads_fit(int64_t T, int64_t heads);
hipError_t launch_heads(HeadsArgs g, int dtype, hipStream_t stream);

struct ReadArgs {
  Pages pages;
  const int32_t* tables;           // B x width page numbers
  const int32_t* lengths;          // B
  void* k_out;
  void* v_out;
  int64_t k_b, k_t, k_h, v_b, v_t, v_h;
  int width, B, L, Hkv, D;
  int chunks;                      // set by launch_read
};
bool read_fits(int64_t B, int64_t L, int64_t Hkv);
hipError_t launch_read(ReadArgs g, int dtype, hipStream_t stream);

}  // namespace svdq
