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

// Work is counted in keys of a tile of few rows, times G. A tile of many rows takes twice
// as long per key (per workgroup, two on a compute unit: 64 keys 2.4 us, where few rows take
// 128 in 2.2). A tile's start and end take 8 us, as long as 448 keys (measured, one token for
// each of 8 sequences of up to 8191, 32/8 heads: 36 us counting 128 of them, 33 with 384, 31
// with 448 to 640). Tiles up to kWhole are not cut (8 prompts of 300 at the end of 900: 67 us;
// 1024: 80), and a share is not below kLeast (3 sequences of 1000: 13.7 us, with 256 15.5;
// one of 8191: 21.9 and 20.9).
constexpr int kStart = 448;
constexpr int kWholeFew = 960, kWholeMany = 768;
constexpr int kLeast = 192;

// The arguments, which lie in memory as far away as the host's, in one round of loads
// instead of one where each is first needed.
__device__ __forceinline__ void fetch_arguments(const PagedArgs& g) {
  asm volatile("" ::"s"(g.q), "s"(g.o_t), "s"(g.pages.k_stride), "s"(g.pages.v_scales), "s"(g.tables),
               "s"(g.part_ml), "s"(g.scale2), "s"(g.B), "s"(g.part_rows));
}

struct Sequence {
  int first, n, length;                   // tokens among the T; tokens in the cache
  bool few;
  int tiles;                              // of one key head
  int64_t fixed, step;                    // tile r: fixed + step * (r + 1)

  __device__ __forceinline__ void set(const PagedArgs& g) {
    const int rows = n * g.G;
    few = rows <= kFew;
    tiles = few ? (rows > 0 ? 1 : 0) : (rows + kMany - 1) / kMany;
    const bool steps = g.causal && !few;
    const int64_t keys = steps ? max(length - n, 0) : length;
    fixed = static_cast<int64_t>(g.G) * (kStart + (few ? 1 : 2) * keys);
    step = steps ? 2 * kMany : 0;
  }

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
  s.set(g);
  return s;
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
__device__ __forceinline__ int64_t of_lane(int64_t x, int lane) {
  const int lo = __builtin_amdgcn_readlane(static_cast<int>(x), lane);
  const int hi = __builtin_amdgcn_readlane(static_cast<int>(x >> 32), lane);
  return static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(hi)) << 32 |
                              static_cast<uint32_t>(lo));
}

// The wave's one value of x, in scalar registers: what comes out of vector arithmetic stays
// in vector registers otherwise, and every load by an address made of it becomes a loop.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
  const int lo = uniform(static_cast<int>(x)), hi = uniform(static_cast<int>(x >> 32));
  return static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(hi)) << 32 |
                              static_cast<uint32_t>(lo));
}

// a / b and what is left, for quotients below 2^24 (one multiplication by a reciprocal that
// is good to that, put right by one; a division of 64 bits takes 130 instructions).
__device__ __forceinline__ int quotient(int64_t a, int64_t b, int64_t& left) {
  int q = uniform(static_cast<int>(static_cast<double>(a) * __builtin_amdgcn_rcp(static_cast<double>(b))));
  left = a - q * b;
  if (left < 0) {
    left += b;
    --q;
  } else if (left >= b) {
    left -= b;
    ++q;
  }
  return q;
}

// The line as a wave sees it. Each lane sums up `span` sequences, one after the other (one
// each where there are up to 64: 1000 take 4 rounds of loads instead of 16), and 64 of
// them are held at a time, one a lane.
struct Line {
  Sequence own;
  int at;                                 // the first of those held
  int span;
  int64_t upto;                           // work of the lanes' sequences up to this lane's end
  int64_t per_head;                       // work of one key head

  __device__ __forceinline__ void hold(const PagedArgs& g, int first) {
    at = first;
    const int b = first + static_cast<int>(threadIdx.x & 63);
    own = sequence(g, b < g.B ? b : g.B - 1);
    if (b >= g.B) own.tiles = 0;
  }
  __device__ __forceinline__ Line(const PagedArgs& g) {
    span = (g.B + 63) / 64;
    int64_t sum = 0;
    if (span == 1) {
      hold(g, 0);
      sum = own.before(own.tiles);
    } else {
      at = -64;                           // none
      const int b0 = static_cast<int>(threadIdx.x & 63) * span;
#pragma unroll 4
      for (int i = 0; i < span; ++i) {
        const Sequence s = sequence(g, min(b0 + i, g.B - 1));
        if (b0 + i < g.B) sum += s.before(s.tiles);
      }
    }
    upto = running_sum(sum);
    per_head = of_lane(upto, 63);
  }
  // Sequence b, the same for the whole wave.
  __device__ __forceinline__ Sequence get(const PagedArgs& g, int b) {
    if (b < at || b >= at + 64) hold(g, b);
    const int lane = b - at;
    Sequence s;
    s.first = __builtin_amdgcn_readlane(own.first, lane);
    s.n = __builtin_amdgcn_readlane(own.n, lane);
    s.length = __builtin_amdgcn_readlane(own.length, lane);
    s.set(g);
    return s;
  }
};

// A workgroup's place on the line: the tile that position c falls into.
struct Place {
  int hk, b, r;
  int64_t start;                          // the tile's
};
// The first lane whose sum exceeds left, which is taken on from there.
__device__ __forceinline__ int lane_of(int64_t upto, int64_t& left) {
  const uint64_t behind = __builtin_amdgcn_ballot_w64(upto > left);
  const int lane = behind != 0 ? __builtin_ctzll(behind) : 63;
  if (lane > 0) left -= of_lane(upto, lane - 1);
  return lane;
}
__device__ __forceinline__ Place place(const PagedArgs& g, Line& line, int64_t c, Sequence& s) {
  Place p;
  int64_t left;
  p.hk = quotient(c, line.per_head, left);
  p.b = lane_of(line.upto, left) * line.span;
  if (line.span > 1) {
    while (true) {
      line.hold(g, p.b);
      const int64_t upto = running_sum(line.own.before(line.own.tiles));
      const int64_t all = of_lane(upto, 63);
      if (all > left || p.b + 64 >= g.B) {
        p.b += lane_of(upto, left);
        break;
      }
      left -= all;
      p.b += 64;
    }
  }
  s = line.get(g, p.b);
  int lo = 0, hi = s.tiles - 1;           // the last tile that starts at or before left
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (s.before(mid) <= left) lo = mid;
    else hi = mid - 1;
  }
  p.r = lo;
  p.start = c - (left - s.before(lo));
  return p;
}
// The next tile and its sequence, if there is one.
__device__ __forceinline__ bool next_place(const PagedArgs& g, Line& line, Place& p, Sequence& s) {
  p.start += s.cost(p.r);
  if (++p.r < s.tiles) return true;
  p.r = 0;
  while (true) {
    if (++p.b == g.B) {
      p.b = 0;
      if (++p.hk == g.Hkv) return false;
    }
    s = line.get(g, p.b);
    if (s.tiles > 0) return true;         // some are, or there was no place
  }
}

// What a workgroup takes of the line: no less than work / wgs.
__device__ __forceinline__ int64_t share(const PagedArgs& g, int64_t work, int wgs) {
  const double part = static_cast<double>(work) * __builtin_amdgcn_rcp(static_cast<double>(wgs));
  const int64_t each = uniform(static_cast<int64_t>(part * (1.0 + 0x1p-20))) + 1;
  return max(each, static_cast<int64_t>(kLeast) * g.G);
}
// A place x on a tile's stretch of work at which it may be cut: a tile's start is not divided.
__device__ __forceinline__ int64_t cut_at(const PagedArgs& g, int64_t x) {
  return x <= static_cast<int64_t>(kStart) * g.G ? 0 : x;
}
// The steps of a tile that lie before place x, 0 < x < cost: the same for the workgroups on
// both sides of it.
__device__ __forceinline__ int steps_before(const PagedArgs& g, int steps, int64_t x, int64_t cost) {
  const int64_t start = static_cast<int64_t>(kStart) * g.G;
  const double part = static_cast<double>(x - start) * __builtin_amdgcn_rcp(static_cast<double>(cost - start));
  return min(steps, uniform(static_cast<int>(static_cast<double>(steps) * part)));
}
__device__ __forceinline__ bool left_whole(const PagedArgs& g, const Sequence& s, int64_t cost) {
  return g.part_rows == 0 || cost <= static_cast<int64_t>(s.few ? kWholeFew : kWholeMany) * g.G;
}

}  // namespace

}  // namespace svdq
