// Host-side launcher of the attention kernels (abi_block.hip validates every
// argument before it calls them).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace svdq {

// Caps of the scores: none; up to kNearest, whose tanh may be off by 2^-23 of 1; any.
enum { kNoCap = 0, kNearCap = 1, kAnyCap = 2 };
constexpr float kNearest = 64.f;

// Strides in elements: _b batch, _l token, _h head; channels are contiguous.
struct AttnArgs {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  int64_t q_b, q_l, q_h, k_b, k_l, k_h, v_b, v_l, v_h, o_b, o_l, o_h;
  const float* slopes;       // per query head, or null
  const int32_t* prefix;     // per batch entry, or null
  const int32_t* ranges;     // [begin, end) per query row, or null
  int64_t range_b;           // batch stride of ranges (elements; 0: shared)
  float* part_ml;            // splits: maximum and sum per row
  float* part_o;             // splits: unnormalized outputs, D per row
  // the kernel's scale is positive: its sign, or 0, goes into Q
  int q_sign;
  float scale2;              // |scale| * log2(e), 1 for a scale of 0
  int cap;                   // kNoCap, kNearCap or kAnyCap
  float cap_in, cap2;        // 2 log2(e) |scale| / cap, cap * log2(e)
  int B, Lq, Lk, Hkv, G, D;  // G query heads per key head
  int rows;                  // Lq * G
  int causal;
  int row_tiles, splits;     // set by launch_attention
};

struct AttnPlan {
  bool few;                  // row tiles of 32 rows: the waves split a tile's keys
  int64_t row_tiles, wgs;
  int splits;                // workgroups along the keys
  unsigned grid;
};

// grid 0: no row tile's grid can cover the rows.
AttnPlan attention_plan(int64_t B, int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hkv, int64_t D,
                        bool split);
hipError_t launch_attention(AttnArgs g, int dtype, const AttnPlan& p, hipStream_t stream);

}  // namespace svdq
