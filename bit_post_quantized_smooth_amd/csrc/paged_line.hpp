// The line of work of the attention over a paged cache (gfx950): which tiles there are,
// what each is worth, and which of them a workgroup has.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "paged_attention.hpp"

namespace svdq {

namespace {

constexpr int kFew = 32, kMany = 128;     // rows of a tile
constexpr int kGroupKeys = 16;            // keys that lie in one page together

// Work is counted in keys of a tile of few rows, times G. A tile of many takes twice as
// long per key; its start and end as long as kStart keys.
constexpr int kStart = 128;
constexpr int kWhole = 512;               // tiles up to this are not split
constexpr int kLeast = 256;               // the smallest share of a workgroup

struct Sequence {
  int first, n, length;                   // tokens among the T; tokens in the cache
  bool few;
  int tiles;                              // of one key head
  int64_t fixed, step;                    // tile r: fixed + step * (r + 1)

  __device__ __forceinline__ int64_t cost(int r) const { return fixed + step * (r + 1); }
  __device__ __forceinline__ int64_t before(int r) const {
    return r * fixed + step * ((static_cast<int64_t>(r) * (r + 1)) / 2);
  }
};

__device__ __forceinline__ Sequence sequence(const PagedArgs& g, int b) {
  Sequence s;
  s.first = min(max(g.starts[b], 0), g.T);
  s.n = min(max(g.starts[b + 1], s.first), g.T) - s.first;
  s.length = g.pages.count > 0 ? min(max(g.lengths[b], 0), g.capacity) : 0;
  const int rows = s.n * g.G;
  s.few = rows <= kFew;
  s.tiles = s.few ? (rows > 0 ? 1 : 0) : (rows + kMany - 1) / kMany;
  const bool steps = g.causal && !s.few;
  const int64_t keys = steps ? max(s.length - s.n, 0) : s.length;
  s.fixed = static_cast<int64_t>(g.G) * (kStart + (s.few ? 1 : 2) * keys);
  s.step = steps ? 2 * kMany : 0;
  return s;
}

// Sequences 64 at a time, one a lane.
__device__ __forceinline__ int64_t own_work(const PagedArgs& g, int b) {
  if (b >= g.B) return 0;
  const Sequence s = sequence(g, b);
  return s.before(s.tiles);
}
__device__ __forceinline__ int64_t running_sum(int64_t x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int64_t y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  return x;
}
__device__ __forceinline__ int64_t uniform(int64_t x) {
  const int lo = __builtin_amdgcn_readfirstlane(static_cast<int>(x));
  const int hi = __builtin_amdgcn_readfirstlane(static_cast<int>(x >> 32));
  return static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(hi)) << 32 |
                              static_cast<uint32_t>(lo));
}

// The work of one key head.
__device__ __forceinline__ int64_t head_work(const PagedArgs& g) {
  int64_t sum = 0;
  for (int b0 = 0; b0 < g.B; b0 += 64)
    sum += uniform(__shfl(running_sum(own_work(g, b0 + (threadIdx.x & 63))), 63));
  return sum;
}

// A workgroup's place on the line: the tile that position c falls into.
struct Place {
  int hk, b, r;
  int64_t start;                          // the tile's
};
__device__ __forceinline__ Place place(const PagedArgs& g, int64_t per_head, int64_t c) {
  Place p;
  p.hk = static_cast<int>(c / per_head);
  int64_t left = c - p.hk * per_head;
  p.b = 0;
  p.r = 0;
  for (int b0 = 0; b0 < g.B; b0 += 64) {
    const int64_t upto = running_sum(own_work(g, b0 + (threadIdx.x & 63)));
    const uint64_t behind = __builtin_amdgcn_ballot_w64(upto > left);
    if (behind != 0) {
      const int at = __builtin_ctzll(behind);
      if (at > 0) left -= uniform(__shfl(upto, at - 1));
      p.b = b0 + at;
      break;
    }
    left -= uniform(__shfl(upto, 63));
  }
  const Sequence s = sequence(g, p.b);
  int lo = 0, hi = s.tiles - 1;           // the last tile that starts at or before left
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (s.before(mid) <= left) lo = mid;
    else hi = mid - 1;
  }
  p.b = __builtin_amdgcn_readfirstlane(p.b);
  p.r = __builtin_amdgcn_readfirstlane(lo);
  p.start = uniform(c - (left - s.before(lo)));
  return p;
}
// The next tile, if there is one.
__device__ __forceinline__ bool next_place(const PagedArgs& g, const Sequence& s, Place& p) {
  p.start += s.cost(p.r);
  if (++p.r < s.tiles) return true;
  p.r = 0;
  int heads = 2;                          // none holds tokens: one round is enough
  while (heads > 0) {
    if (++p.b == g.B) {
      p.b = 0;
      --heads;
      if (++p.hk == g.Hkv) return false;
    }
    if (sequence(g, p.b).tiles > 0) return true;
  }
  return false;
}

__device__ __forceinline__ int64_t share(const PagedArgs& g, int64_t work, int wgs) {
  return max((work + wgs - 1) / wgs, static_cast<int64_t>(kLeast) * g.G);
}
__device__ __forceinline__ bool left_whole(const PagedArgs& g, int64_t cost) {
  return g.part_rows == 0 || cost <= static_cast<int64_t>(kWhole) * g.G;
}

}  // namespace

}  // namespace svdq
