// Attention of new tokens over a paged cache (gfx950).
//
//   x_ij = scale * s_k * q_i . k_j;  with a cap: x_ij = cap * tanh(x_ij / cap);
//   with slopes: x_ij -= slope_h * |pos_i - j|;
//   o_i = s_v * sum_j exp(x_ij) v_j / sum_j exp(x_ij) over the keys j that row i sees:
//   j < length of its sequence, in a page of the pool, and, if causal, j <= pos_i,
//   where the sequence's n new tokens are its last: pos_i = length - n + i.
// s_k and s_v are the head's scales of e4m3 codes (1 of 16-bit pages): s_k is part of
// the scores' scale and s_v of the division by the weights' sum, so that codes enter
// the products as they are (every one is exact in fp16 and bf16).
//
// The softmax in one pass, its roundings and the matrix products are those of
// attention_core.hpp: a wave owns 32 rows (query and head of one key head) and its
// tiles of K and V lie in LDS as 16-bit values.
//
// Two kinds of row tiles, by a sequence's own rows, in one launch, so that single
// tokens and chunks of prompts run side by side:
//   up to 32 rows (single tokens): the waves of a workgroup take blocks of 32 keys in
//   turn. Each has its own part of LDS and fetches its next block into registers before
//   it works on one (64 KB of codes in flight per compute unit, 128 KB of 16 bits; two
//   blocks of codes ahead do not fit the registers), with no barrier until the four add
//   up their outputs at the end;
//   more rows: 128 per workgroup, 32 a wave, sharing tiles of 64 keys in two stages;
//   16-bit tiles go straight into LDS, codes through registers, widened on the way.
//
// The lengths are only known on the device. So the tiles, over all sequences and key
// heads, are laid end to end by an estimate of their work, and each workgroup of a
// fixed number, as many as are resident, takes an equal share of the line: the shares
// balance whatever the lengths are. Where a share's border falls into a tile the keys
// are split there, each part writes fp32 outputs with their maxima and sums, and a
// second kernel joins them in order. Tiles of little work are left whole.
//
// What bounds it. Single tokens: memory, and a tile's start (the lengths, a place on the
// line, page numbers and the first keys are loads behind each other: 7 us) and end (2 us).
// One token for each of 8 sequences of up to 8191, 32/8 heads of 128, e4m3: 25 us, of them
// 15 at 7 TB/s (105 MB, part of them in the last-level cache), and 4.5 to join; 16-bit pages 54
// us with the join. 64 sequences of 8191: 194 us, 5.5 TB/s (16 bits 373, 5.8); 1024 of 300,
// whose tiles are all start and end: 199 us, 3.25 TB/s (268, 4.75). The join is launched where
// the table could hold a sequence long enough to cut, whatever the lengths are: one token over
// 333 keys takes 9.4 us with a table of 336 places, 12.0 with one of 8192.
// Chunks: neither unit alone; the vector unit is busy 41% of the time (the softmax, with 7
// vector instructions per matrix instruction, and the issue of these) and the matrix cores
// 36%, for the most part one after the other. 4095 tokens at the end of 16383, 32/8 heads, e4m3,
// 1.08 to 1.12 ms with 17 us to join the parts, 860 to 890 TFLOP/s. Widening codes takes 1 to 4% of
// it (16-bit pages: fp16 1101 us beside 1113, bf16 1041 beside 1083). Its LDS writes meet in
// banks; in another order they do not, and the kernel takes as long (1136 us beside 1137).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/svdq.h"
#include "attention_core.hpp"
#include "block_common.hpp"
#include "k2_common.hpp"
#include "paged_attention.hpp"
#include "paged_line.hpp"

namespace svdq {

namespace {

// Page numbers of 64 groups of 16 keys, one a lane, and of the 64 before them, which are
// on their way while these are used. -1: not in the pool.
struct PageWindow {
  const PagedArgs* g;
  const int32_t* table;
  int at, now, then;
  uint64_t there;

  __device__ __forceinline__ int fetch(int group) const {
    const int i = (group + static_cast<int>(threadIdx.x & 63)) >> (g->pages.page_log2 - 4);
    if (i < 0 || i >= g->width) return -1;
    return table[i];
  }
  __device__ __forceinline__ void begin(const PagedArgs& args, int b, int group) {
    g = &args;
    table = args.tables + static_cast<int64_t>(b) * args.width;
    at = group & ~63;
    now = fetch(at);
    then = fetch(at - 64);
  }
  // Once they are needed: whoever begins may have other loads to send first.
  __device__ __forceinline__ void see() {
    there = __builtin_amdgcn_ballot_w64(now >= 0 && now < g->pages.count);
  }
  // Groups are asked for in descending order.
  __device__ __forceinline__ void seek(int group) {
    while (group < at) {
      now = then;
      at -= 64;
      then = fetch(at - 64);
      see();
    }
  }
  __device__ __forceinline__ bool has(int group) const { return there >> (group - at) & 1; }
  __device__ __forceinline__ int page(int group) const {
    return __builtin_amdgcn_readlane(now, group - at);
  }
};

struct Scores {
  float scale2, cap_in, cap2;
};

// What the two kinds of tiles share. CODED: pages of e4m3 codes.
template <class T, int DP, int RW, int CAP, bool SLOPES, bool CODED>
struct PagedTile : AttentionCore<T, DP, RW, CAP, SLOPES, 128, Scores, true> {
  typedef AttentionCore<T, DP, RW, CAP, SLOPES, 128, Scores, true> Core;
  using typename Core::Lds;
  using typename Core::vec;
  using Core::DB, Core::DS, Core::KB, Core::KT, Core::UNITS;
  using Core::g, Core::lds, Core::lane, Core::wave, Core::rl, Core::h, Core::qf, Core::o, Core::m,
      Core::l, Core::lo, Core::pos, Core::width, Core::large, Core::w_lo, Core::w_hi,
      Core::w_lo_max, Core::w_hi_min, Core::slope2, Core::kb0, Core::vb0, Core::holes;
  static constexpr int ESIZE = CODED ? 1 : 2;
  static constexpr int LPR = DP * ESIZE / 16;       // lanes that fetch a row
  static constexpr int RPI = 64 / LPR;              // rows of one fetch of a wave

  const PagedArgs& a;
  PageWindow pages;
  int hk, last;                                     // last: keys that any row of the tile sees
  float vscale;
  // the lane's share of a fetch: its place in the rows (beyond any buffer past D) and in LDS
  uint32_t fetch_at;
  int put_at;

  __device__ __forceinline__ PagedTile(const PagedArgs& args, const Scores& scores, Lds& shared)
      : Core(scores, shared), a(args) {}

  // Rows 16 * group .. of K or V: base and bytes; none of a page outside the pool.
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows(const void* pool, int64_t stride, int group) const {
    const int key = group * kGroupKeys;
    const int in_page = key & ((1 << a.pages.page_log2) - 1);
    const int n = min(last - key, kGroupKeys);
    const bool there = n > 0 && pages.has(group);
    const int64_t page = there ? pages.page(group) : 0;
    const char* base = static_cast<const char*>(pool) + page * stride +
                       ((static_cast<int64_t>(hk) << a.pages.page_log2) + in_page) * a.D * ESIZE;
    return make_buffer(base, there ? static_cast<uint32_t>(n * a.D * ESIZE) : 0u);
  }

  // 16 codes or 8 values a lane, of RPI rows from row `row0` of the group on
  __device__ __forceinline__ v4i fetch(__amdgpu_buffer_rsrc_t buf, int row0) const {
    return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(
                                       buf, static_cast<int>(fetch_at), row0 * a.D * ESIZE, 0));
  }
  // The same into LDS rows from `to` on (16-byte units from its start; row `row0` of them),
  // widened. The twist of a row is the exclusive or of its bits' twists, and a fetch's
  // rows lie within RPI: one address per lane, a constant each.
  __device__ __forceinline__ void put(uint8_t* to, int row0, v4i x) const {
    uint8_t* p = to + row0 * DP * 2 + (put_at ^ (Core::twist(row0) * 16));
    if constexpr (CODED) {
      v4i w[2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int word = x[i];
        w[i >> 1][2 * (i & 1)] = widen<false>(word);
        w[i >> 1][2 * (i & 1) + 1] = widen<true>(word);
      }
      // the second 8 may lie behind D: the next row's
      if (16 * (lane % LPR) + 8 >= a.D) w[1] = v4i{0, 0, 0, 0};
      *reinterpret_cast<v4i*>(p) = w[0];
      *reinterpret_cast<v4i*>(to + row0 * DP * 2 + (put_at ^ ((Core::twist(row0) ^ 1) * 16))) = w[1];
    } else {
      *reinterpret_cast<v4i*>(p) = x;
    }
  }
  template <bool HIGH>
  static __device__ __forceinline__ int widen(int word) {
    if constexpr (__is_same(T, _Float16))
      return __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(word, 1.0f, HIGH));
    else
      return __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(word, 1.0f, HIGH));
  }

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[d][e] = 0.f;
    m = kNegInf;
    l = 0.f;
    large = false;
  }

  // The lane's row r of sequence s: what it sees, its slope, its queries.
  __device__ __forceinline__ void rows_of(const Sequence& s, const Place& p, int r) {
    lane = Core::opaque(threadIdx.x & 63);   // nothing of a lane's is kept from tile to tile
    wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    rl = lane & 31;
    h = lane >> 5;
    hk = uniform(p.hk);
    holes = 0;
    vscale = a.pages.v_scales != nullptr ? a.pages.v_scales[hk] : 1.f;
    fetch_at = 16 * (lane % LPR) < a.D * ESIZE
                   ? static_cast<uint32_t>((lane / LPR) * a.D * ESIZE + 16 * (lane % LPR))
                   : 0x80000000u;
    const int row = lane / LPR;
    put_at = row * DP * 2 + (((CODED ? 2 : 1) * (lane % LPR)) ^ Core::twist(row)) * 16;
    kb0 = Core::k_base();
    vb0 = Core::v_base();
    const bool real = r < s.n * a.G;
    const int i = real ? r / a.G : 0;
    const int head = hk * a.G + (real ? r % a.G : 0);
    pos = s.length - s.n + i;
    slope2 = SLOPES ? a.slopes[head] * kLog2e / (Core::RAW ? g.scale2 : 1.f) : 0.f;
    const int hi = a.causal ? min(s.length, pos + 1) : s.length;
    lo = 0;
    width = real && hi > 0 ? static_cast<uint32_t>(hi) : 0u;
    // Loads without a branch, from the first row and channels where there is nothing to
    // load; queries() makes operands of them when the first keys are on their way.
    const T* qp = static_cast<const T*>(a.q) + (s.first + static_cast<int64_t>(i)) * a.q_t + head * a.q_h;
#pragma unroll
    for (int t = 0; t < DS; ++t) {
      const int c = (2 * t + h) * 8;
      qf[t] = __builtin_bit_cast(vec, *reinterpret_cast<const v4i*>(qp + (c < a.D ? c : 0)));
    }
  }
  // Negated for a negative scale, 0 for a scale of 0 and where nothing was loaded.
  __device__ __forceinline__ void queries(bool real) {
    const int sign = a.q_sign < 0 ? static_cast<int>(0x80008000u) : 0;
#pragma unroll
    for (int t = 0; t < DS; ++t) {
      const int c = (2 * t + h) * 8, keep = real && c < a.D && a.q_sign != 0 ? -1 : 0;
      v4i z = __builtin_bit_cast(v4i, qf[t]);
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] = (z[e] ^ sign) & keep;
      qf[t] = __builtin_bit_cast(vec, z);
    }
  }
  __device__ __forceinline__ bool not_finite() const {
    bool odd = false;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) odd |= !(fabsf(o[d][e]) < __builtin_inff());
    return __builtin_amdgcn_ballot_w64(odd) != 0;
  }

  // Channels ch .. ch + 3 of row r (row in_tile of the tile), whose weights sum to l, under
  // the reference m: the outputs, or in the part `slot`.
  __device__ __forceinline__ void store(const Sequence& s, int r, int in_tile, int slot, int ch, v4f x) {
    if (ch >= a.D) return;
    if (slot >= 0) {
      const int64_t row = static_cast<int64_t>(slot) * a.part_rows + in_tile;
      if (ch == 0) {
        a.part_ml[2 * row] = m;
        a.part_ml[2 * row + 1] = l;
      }
      // the join reads no outputs of a row without weights
      if (l != 0.f) *reinterpret_cast<v4f*>(a.part_o + row * a.D + ch) = x;
      return;
    }
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    T* op = static_cast<T*>(a.out) + (s.first + static_cast<int64_t>(r / a.G)) * a.o_t +
            (hk * a.G + r % a.G) * a.o_h;
    typedef T vec4 __attribute__((ext_vector_type(4)));
    vec4 y;
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] = static_cast<T>(x[c] * inv * vscale);
    *reinterpret_cast<vec4*>(op + ch) = y;
  }
};

// Up to 32 rows: blocks of 32 keys, a wave's own.
template <class T, int DP, int CAP, bool SLOPES, bool CODED>
struct FewRows : PagedTile<T, DP, 1, CAP, SLOPES, CODED> {
  typedef PagedTile<T, DP, 1, CAP, SLOPES, CODED> Tile;
  using Tile::a, Tile::lds, Tile::wave, Tile::lane, Tile::rl, Tile::h, Tile::o, Tile::m, Tile::l,
      Tile::last, Tile::holes, Tile::pages, Tile::DB, Tile::RPI;
  static constexpr int NF = 32 / RPI;               // fetches of a block and operand

  struct Ahead {
    v4i k[NF], v[NF];
    uint32_t gone;
  };

  __device__ __forceinline__ FewRows(const PagedArgs& args, const Scores& scores, typename Tile::Lds& shared)
      : Tile(args, scores, shared) {}

  __device__ __forceinline__ void get(Ahead& x, int block) {
    pages.seek(2 * block);
    x.gone = 0;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int group = 2 * block + half;
      const auto kb = Tile::rows(a.pages.k, a.pages.k_stride, group);
      const auto vb = Tile::rows(a.pages.v, a.pages.v_stride, group);
      if (!pages.has(group)) x.gone |= 1u << half;
#pragma unroll
      for (int i = 0; i < NF / 2; ++i) {
        x.k[half * (NF / 2) + i] = Tile::fetch(kb, i * RPI);
        x.v[half * (NF / 2) + i] = Tile::fetch(vb, i * RPI);
      }
    }
  }
  __device__ __forceinline__ void set(const Ahead& x) {
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      Tile::put(&lds.k[32 * wave][0], i * RPI, x.k[i]);
      Tile::put(&lds.v[32 * wave][0], i * RPI, x.v[i]);
    }
    holes = x.gone;
  }

  // Blocks block1 - 1 - wave, 4 before it, ... from block0 on, whose page numbers are on
  // their way. (From the last keys to the first: with slopes the largest scores come first.)
  template <bool CAREFUL>
  __device__ __forceinline__ void pass(int block0, int block1, bool real) {
    int i = block1 - 1 - wave;
    Ahead x;
    if (i >= block0) {
      pages.see();
      get(x, i);
    }
    if constexpr (!CAREFUL) Tile::queries(real);
    Tile::zero();
    for (; i >= block0; i -= kWaves) {
      set(x);
      if (i - kWaves >= block0) get(x, i - kWaves);
      this->template block<CAREFUL>(0, 32 * wave, 32 * i);
    }
  }

  __device__ __forceinline__ void run(const Sequence& s, const Place& p, int64_t x0, int64_t x1,
                                      int64_t cost, int slot) {
    wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    last = uniform(s.length);            // the last query sees them all
    const int blocks = (last + 31) / 32;
    const int b0 = uniform(x0 > 0 ? steps_before(a, blocks, x0, cost) : 0);
    const int b1 = uniform(x1 < cost ? steps_before(a, blocks, x1, cost) : blocks);
    pages.begin(a, p.b, 2 * (b1 - 1 - wave));
    const int rows = s.n * a.G;
    Tile::rows_of(s, p, Tile::opaque(threadIdx.x & 31));
    pass<false>(b0, b1, rl < rows);
    if (Tile::not_finite()) {
      pages.begin(a, p.b, 2 * (b1 - 1 - wave));
      pass<true>(b0, b1, rl < rows);
    }
    l = half_sum(l);
    join(s, slot, rows);
  }

  // Adds the waves' outputs in wave order, scaled to the common maximum: the rows that
  // there are, 32 lanes a row, 4 channels each.
  static constexpr int STRIDE = DP + 4;             // floats; rows on different banks
  static constexpr size_t JOIN_BYTES = (kWaves * 32 * STRIDE + kWaves * 32 * 2) * 4;

  __device__ __forceinline__ void join(const Sequence& s, int slot, int rows) {
    float* mem = reinterpret_cast<float*>(&lds);
    float* ml = mem + kWaves * 32 * STRIDE;
    __syncthreads();                     // the tiles are no longer read
    if (rl < rows) {
      if (h == 0) {
        ml[(wave * 32 + rl) * 2] = m;
        ml[(wave * 32 + rl) * 2 + 1] = l;
      }
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<v4f*>(mem + (wave * 32 + rl) * STRIDE + 32 * d + 8 * e + 4 * h) =
              v4f{o[d][4 * e], o[d][4 * e + 1], o[d][4 * e + 2], o[d][4 * e + 3]};
    }
    __syncthreads();
    const int ch = 4 * (lane & 31);
    for (int r = 2 * wave + h; r < rows; r += 2 * kWaves) {
      float f[kWaves], top = kNegInf;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        f[w] = ml[(w * 32 + r) * 2];
        top = fmaxf(top, f[w]);
      }
      // two above the largest: the sum of four finite partial outputs is finite
      const float base = top == kNegInf ? 0.f : top + 2.f;
      m = top == kNegInf ? top : base;
      l = 0.f;
      v4f sum = v4f{0.f, 0.f, 0.f, 0.f};
      if (ch < DP) {
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          f[w] = __builtin_amdgcn_exp2f(f[w] - base);
          l = __builtin_fmaf(ml[(w * 32 + r) * 2 + 1], f[w], l);
          const v4f x = *reinterpret_cast<const v4f*>(mem + (w * 32 + r) * STRIDE + ch);
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] = __builtin_fmaf(x[e], f[w], sum[e]);
        }
        Tile::store(s, r, r, slot, ch, sum);
      }
    }
    __syncthreads();                     // the next tile's rows may come
  }
};

// 128 rows, 32 a wave: tiles of 64 keys for all, in two stages.
template <class T, int DP, int CAP, bool SLOPES, bool CODED>
struct ManyRows : PagedTile<T, DP, 4, CAP, SLOPES, CODED> {
  typedef PagedTile<T, DP, 4, CAP, SLOPES, CODED> Tile;
  using Tile::a, Tile::lds, Tile::wave, Tile::lane, Tile::rl, Tile::h, Tile::o, Tile::m, Tile::l,
      Tile::last, Tile::holes, Tile::pages, Tile::DB, Tile::RPI, Tile::KT, Tile::width, Tile::LPR;
  static constexpr int NF = 16 / RPI;               // fetches of a wave, tile and operand
  v4i kx[CODED ? NF : 1], vx[CODED ? NF : 1];
  uint32_t copy_at[CODED ? 1 : NF];
  uint32_t gone;                                    // the next tile's holes
  int hi, hi_min;                                   // keys that a row, all rows of the wave see

  __device__ __forceinline__ ManyRows(const PagedArgs& args, const Scores& scores, typename Tile::Lds& shared)
      : Tile(args, scores, shared) {}

  // Tile t's 16 rows of this wave: on their way into registers (codes) or stage s.
  __device__ __forceinline__ void get(int t, int s) {
    const int group = t * (KT / kGroupKeys) + wave;
    pages.seek(t * (KT / kGroupKeys));
    gone = 0xFu & ~static_cast<uint32_t>(pages.there >> (t * (KT / kGroupKeys) - pages.at));
    const auto kb = Tile::rows(a.pages.k, a.pages.k_stride, group);
    const auto vb = Tile::rows(a.pages.v, a.pages.v_stride, group);
    if constexpr (CODED) {
#pragma unroll
      for (int i = 0; i < NF; ++i) kx[i] = Tile::fetch(kb, i * RPI);
#pragma unroll
      for (int i = 0; i < NF; ++i) vx[i] = Tile::fetch(vb, i * RPI);
    } else {
#pragma unroll
      for (int i = 0; i < NF; ++i)
        buffer_to_lds16(kb, &lds.k[s * KT + 16 * wave + i * RPI][0], copy_at[i],
                        static_cast<uint32_t>(i * RPI * a.D * 2));
#pragma unroll
      for (int i = 0; i < NF; ++i)
        buffer_to_lds16(vb, &lds.v[s * KT + 16 * wave + i * RPI][0], copy_at[i],
                        static_cast<uint32_t>(i * RPI * a.D * 2));
    }
  }
  __device__ __forceinline__ void set(int s) {
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      Tile::put(&lds.k[s * KT + 16 * wave][0], i * RPI, kx[i]);
      Tile::put(&lds.v[s * KT + 16 * wave][0], i * RPI, vx[i]);
    }
  }

  template <bool CAREFUL>
  __device__ __forceinline__ void pass(int t0, int t1, bool real) {
    pages.see();
    int t = t1 - 1;
    get(t, 0);
    uint32_t now = gone;
    if constexpr (!CAREFUL) Tile::queries(real);
    Tile::zero();
    if constexpr (CODED) {
      set(0);
      if (t > t0) get(t - 1, 1);
    }
    // From the last tile to the first: with slopes the largest scores come first, and the
    // outputs are not rescaled for every tile (13 single tokens beside 3 chunks, slopes of 24
    // heads: 138 -> 117 us). The wave sees nothing from tile `off` on; all its rows see all keys
    // of the tiles before `out`, but for pages that are missing: from the first of those on every
    // tile is masked. A loop for each, as one with branches would copy the outputs.
    const int off = max(t0, min(t1, (hi + KT - 1) / KT)), out = CAREFUL ? t0 : max(t0, min(off, hi_min / KT));
    auto begin = [&]() {
      const int s = (t1 - 1 - t) & 1;
      if constexpr (CODED) {
        __syncthreads();                 // the tile is in stage s, stage s ^ 1 is free
        holes = now;
        if (t > t0) {
          now = gone;
          set(s ^ 1);
          if (t - 1 > t0) get(t - 2, s);
        }
      } else {
        __builtin_amdgcn_s_waitcnt(wait_vmem(0));
        __syncthreads();
        holes = now;
        if (t > t0) {
          get(t - 1, s ^ 1);
          now = gone;
        }
      }
      return s;
    };
    auto masked = [&]() {
      const int s = begin();
      if constexpr (!CAREFUL) {
        this->template pair<true>(s, 0, t * KT);
      } else {
        const uint32_t both = holes;
#pragma unroll 1
        for (int kb = 0; kb < 2; ++kb) {
          holes = both >> (2 * kb);
          this->template block<CAREFUL>(s, 32 * kb, t * KT + 32 * kb);
        }
      }
    };
    for (; t >= off; --t) begin();
    for (; t >= out; --t) masked();
    if constexpr (!CAREFUL) {
      for (; t >= t0 && now == 0; --t) this->template pair<false>(begin(), 0, t * KT);
      for (; t >= t0; --t) masked();
    }
    __syncthreads();                     // the tiles are no longer read
  }

  __device__ __forceinline__ void run(const Sequence& s, const Place& p, int64_t x0, int64_t x1,
                                      int64_t cost, int slot) {
    const int top = min(s.n, ((p.r + 1) * kMany + a.G - 1) / a.G);  // queries before the tile's end
    last = uniform(a.causal ? max(0, min(s.length, s.length - s.n + top)) : s.length);
    const int tiles = (last + KT - 1) / KT;
    const int t0 = uniform(x0 > 0 ? steps_before(a, tiles, x0, cost) : 0);
    const int t1 = uniform(x1 < cost ? steps_before(a, tiles, x1, cost) : tiles);
    pages.begin(a, p.b, (t1 - 1) * (KT / kGroupKeys));
    const int in_tile = Tile::opaque(32 * static_cast<int>(threadIdx.x >> 6) + static_cast<int>(threadIdx.x & 31));
    const int r = p.r * kMany + in_tile;
    Tile::rows_of(s, p, r);
    const bool real = r < s.n * a.G;
    hi = static_cast<int>(width);
    hi_min = real ? hi : last;           // rows past the end ask for no mask
#pragma unroll
    for (int d = 16; d >= 1; d /= 2) {
      hi = max(hi, __shfl_xor(hi, d));
      hi_min = min(hi_min, __shfl_xor(hi_min, d));
    }
    hi = __builtin_amdgcn_readfirstlane(hi);
    hi_min = __builtin_amdgcn_readfirstlane(hi_min);
    if constexpr (!CODED) {
#pragma unroll
      for (int i = 0; i < NF; ++i) {
        const int row = lane / LPR, unit = (lane % LPR) ^ Tile::twist(i * RPI + row);
        copy_at[i] = unit * 8 < a.D ? static_cast<uint32_t>(row * a.D * 2 + unit * 16) : 0x80000000u;
      }
    }
    if (t0 < t1) {
      pass<false>(t0, t1, real);
      const bool again = Tile::not_finite();      // asked of all lanes
      if (lane == 0) lds.odd[wave] = again;
      __syncthreads();
      bool any = false;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) any |= lds.odd[w] != 0;
      if (__builtin_amdgcn_readfirstlane(any)) {
        pages.begin(a, p.b, (t1 - 1) * (KT / kGroupKeys));
        pass<true>(t0, t1, real);
      }
    } else {
      Tile::zero();
    }
    l = half_sum(l);
    if (real)
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          Tile::store(s, r, in_tile, slot, 32 * d + 8 * e + 4 * h,
                      v4f{o[d][4 * e], o[d][4 * e + 1], o[d][4 * e + 2], o[d][4 * e + 3]});
    __syncthreads();                     // lds.odd is read
  }
};

template <class T, int DP, int CAP, bool SLOPES, bool CODED>
__global__ __launch_bounds__(64 * kWaves, 2) void paged_attention_kernel(const PagedArgs g) {
  typedef FewRows<T, DP, CAP, SLOPES, CODED> Few;
  typedef ManyRows<T, DP, CAP, SLOPES, CODED> Many;
  static_assert(sizeof(typename Few::Tile::Lds) == sizeof(typename Many::Tile::Lds));
  constexpr size_t kTiles = sizeof(typename Few::Tile::Lds);
  __shared__ alignas(16) uint8_t mem[kTiles > Few::JOIN_BYTES ? kTiles : Few::JOIN_BYTES];
  fetch_arguments(g);
  Line line(g);
  const int64_t work = line.per_head * g.Hkv;
  const int wgs = static_cast<int>(gridDim.x);
  const int w = xcd_contiguous(static_cast<int>(blockIdx.x), wgs);
  const int64_t each = share(g, work, wgs), c0 = w * each, c1 = min(c0 + each, work);
  if (g.part_rows > 0 && threadIdx.x == 0) g.cuts[w].parts = 0;
  if (c0 >= work) return;
  Sequence s;
  Place p = place(g, line, c0, s);
  for (bool more = true; more && p.start < c1; more = next_place(g, line, p, s)) {
    const int64_t cost = s.cost(p.r);
    int64_t x0 = 0, x1 = cost;
    int slot = -1;
    if (left_whole(g, s, cost)) {
      if (p.start < c0) continue;        // the workgroup before has it
    } else {
      x0 = cut_at(g, c0 - p.start);
      x1 = cut_at(g, min(c1 - p.start, cost));
      if (x1 == 0) continue;             // the workgroup behind has it all
      if (x0 > 0 || x1 < cost) slot = 2 * w + (x0 == 0 ? 1 : 0);
      if (x0 == 0 && x1 < cost && threadIdx.x == 0) {
        const int rows = s.few ? kFew : kMany;
        Cut& cut = g.cuts[w];
        int64_t left;
        cut.parts = quotient(p.start + cost - 1, each, left) - w + 1;
        cut.first = s.first;
        cut.row = p.r * rows;
        cut.rows = min(rows, s.n * g.G - p.r * rows);
        cut.hk = p.hk;
      }
    }
    Scores scores;
    const float ks = g.pages.k_scales != nullptr ? g.pages.k_scales[p.hk] : 1.f;
    scores.scale2 = g.scale2 * ks;
    scores.cap_in = fminf(g.cap_in * ks, 3.4028235e38f);
    scores.cap2 = g.cap2;
    if (s.few) {
      Few t(g, scores, *reinterpret_cast<typename Few::Tile::Lds*>(mem));
      t.run(s, p, x0, x1, cost, slot);
    } else {
      Many t(g, scores, *reinterpret_cast<typename Many::Tile::Lds*>(mem));
      t.run(s, p, x0, x1, cost, slot);
    }
  }
}

template <class T, int DP, int CAP, bool SLOPES>
void launch_e(const PagedArgs& g, unsigned grid, hipStream_t stream) {
  if (g.pages.coded)
    hipLaunchKernelGGL((paged_attention_kernel<T, DP, CAP, SLOPES, true>), dim3(grid), dim3(64 * kWaves), 0,
                       stream, g);
  else
    hipLaunchKernelGGL((paged_attention_kernel<T, DP, CAP, SLOPES, false>), dim3(grid), dim3(64 * kWaves), 0,
                       stream, g);
}
template <class T, int DP, int CAP>
void launch_s(const PagedArgs& g, unsigned grid, hipStream_t stream) {
  g.slopes != nullptr ? launch_e<T, DP, CAP, true>(g, grid, stream) : launch_e<T, DP, CAP, false>(g, grid, stream);
}

}  // namespace

template <class T, int DP>
void launch_paged_tiles(const PagedArgs& g, unsigned grid, hipStream_t stream) {
  g.cap == kNoCap     ? launch_s<T, DP, kNoCap>(g, grid, stream)
  : g.cap == kNearCap ? launch_s<T, DP, kNearCap>(g, grid, stream)
                      : launch_s<T, DP, kAnyCap>(g, grid, stream);
}

}  // namespace svdq
