// Host-side launcher of the attention over a paged cache (abi_paged.hip
// validates every argument before it calls it).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "paged.hpp"

namespace svdq {

// The tile that a workgroup is the first to have a part of; parts 0: it has none. Its own
// part is the second of its two, those of the workgroups behind it are their first.
struct Cut {
  int32_t parts, hk;
  int32_t first;             // the sequence's first token
  int32_t row, rows;         // the tile's first row and number of rows
  int32_t pad[3];
};

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
  Cut* cuts;                 // per workgroup
  float* part_ml;            // parts, two per workgroup: maximum and sum per row
  float* part_o;             // parts: unnormalized outputs, D per row
  // as in AttnArgs, without the head's scale
  int q_sign;
  float scale2;
  int cap;
  float cap_in, cap2;
  int causal;
  int width, B, T, Hkv, G, D;
  int capacity;              // width << page_log2
  int part_rows;             // rows of a part; 0: tiles are not split
};

// Largest group of query heads, and most keys of a sequence: their products with
// 2^30 rows fit the 64 bits that work is counted in.
constexpr int64_t kMostGroup = 256;
constexpr int64_t kMostKeys = int64_t{1} << 26;

// Bytes of the cuts, the parts' maxima and sums, and their outputs, on the current device.
struct PartBytes {
  size_t cuts, ml, o;
  size_t all() const { return cuts + ml + o; }
};
PartBytes paged_attention_parts(int64_t T, int64_t B, int64_t capacity, int64_t Hkv, int64_t G,
                                int64_t D);
// The kernel of heads of up to DP channels (64 or 128); a source file each.
template <class T, int DP>
void launch_paged_tiles(const PagedArgs& g, unsigned grid, hipStream_t stream);
hipError_t launch_paged_attention(PagedArgs g, int dtype, hipStream_t stream);

}  // namespace svdq
