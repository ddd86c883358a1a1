// Masked attention with grouped heads (gfx950).
//
//   x_ij = scale * q_i . k_j;  with a cap: x_ij = cap * tanh(x_ij / cap);
//   with slopes: x_ij -= slope_h * |pos_i - j|,  pos_i = i + Lk - Lq;
//   o_i = sum_j exp(x_ij) v_j / sum_j exp(x_ij) over the keys j that row i sees.
//
// Every mask is an interval of keys per query row, [lo_i, hi_i): the caller's
// ranges (documents, padding, filled part of a cache), cut by the causal rule
// j <= pos_i, which the first `prefix` keys escape. A row that sees no key
// comes out 0, and a key that a row does not see never reaches its output,
// whatever its K and V hold.
//
// One pass over the keys with the running maximum and sum of the softmax, in
// base 2 (log2 e goes into the scale). The query heads that share a key head
// are rows of one problem, so each K and V tile is read once for all of them:
// row r is query r / G of head hk*G + r % G. A wave owns 32 rows and computes
//   S^T = K Q^T   (v_mfma_f32_32x32x16, K the first operand),
// so a lane holds scores of one row only (row lane % 32): the softmax needs one
// exchange between the wave's halves, and the rescaling factor of a row is in
// the lane that holds its outputs. The same registers, rounded to 16 bits, are
// the second operand of
//   O^T += V^T P^T;
// the matrix core sums over the keys in any order, so V^T is read in the order
// in which S^T leaves the keys: a transposing LDS read (ds_read_b64_tr_b16) of
// 4 keys x 16 channels per 16 lanes. Scores, maxima, sums and outputs are fp32;
// P is rounded to the type of V (nearest even), the precision of the result, and summed
// as rounded, so that an average of equal values is that value.
//
// K and V go from global memory straight into LDS (two stages), rows of DP
// channels with their 16-byte units XOR-swizzled by the row; channels past D
// and keys outside the tile read as zero. A workgroup takes 128 rows (RW = 4: a
// wave each 32, all sharing the tiles of 64 keys) or 32 (RW = 1: the waves share
// out tiles of 128 keys and add their outputs at the end), and work may be split
// along the keys over workgroups, which then write fp32 outputs with their maxima
// and sums for a second kernel that joins them in order.
//
// The maximum that the exponents refer to is raised only when a score exceeds it by
// kGrow (4 or 8, base 2): the outputs are then rescaled, otherwise they stay in place. The
// products of one half of a tile go out beside the exponents of the other. Tiles
// that no row sees in part run a loop without masks; tiles cut by a mask, and a
// wave's tiles of which it sees nothing, have loops of their own, since a branch
// inside one loop moves the outputs between registers. V of a hidden key times a
// weight of 0 is NaN where V is not finite: only if an output comes out so is the
// pass repeated with hidden keys' V taken out.
//
// Measured (D = 128). 24 heads of 4608 x 4608, fp16: 286 to 313 us by card, 830 to
// 910 TFLOP/s; the matrix core is busy 41% of the time, beside 6.5 vector
// instructions per matrix instruction, and 864 workgroups are 1.69 rounds of the
// 512 that fit. Packed documents of the same length: 130 to 140 us. 16 heads over 4,
// 8191 causal rows with a prefix, bf16: 298 us, with scores capped at 30 338 to 383 us
// by card (350 beside the 298), 11 vector instructions per matrix instruction. One
// token, 32 heads over 8, 8 caches of 8191: 42 us plus 5 us to join, 210 MB at 5.0 TB/s.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/svdq.h"
#include "attention.hpp"
#include "attention_core.hpp"
#include "block_common.hpp"
#include "block_launch.hpp"
#include "k2_common.hpp"

namespace svdq {

namespace {

// RW waves along the rows, 4 / RW along the keys of a tile.
template <class T, int DP, int RW, int CAP, bool SLOPES>
struct Attention
    : AttentionCore<T, DP, RW, CAP, SLOPES, RW == 4 ? 128 : 256, AttnArgs> {
  typedef AttentionCore<T, DP, RW, CAP, SLOPES, RW == 4 ? 128 : 256, AttnArgs> Core;
  using typename Core::Lds;
  using typename Core::vec;
  using Core::DB, Core::DS, Core::KB, Core::KT, Core::KW, Core::UNITS;
  using Core::g, Core::lds, Core::lane, Core::wave, Core::rl, Core::h, Core::qf, Core::o, Core::m,
      Core::l, Core::lo, Core::pos, Core::width, Core::large, Core::w_lo, Core::w_hi,
      Core::w_lo_max, Core::w_hi_min, Core::slope2, Core::kb0, Core::vb0;
  using Core::k_base, Core::twist, Core::v_base;
  static constexpr int RPC = 64 / UNITS;            // rows per copy instruction
  static constexpr int CPW = KT / RPC / kWaves;     // copy instructions per wave and operand
  static_assert(KW == 1 || sizeof(Lds::k) + sizeof(Lds::v) >=
                               static_cast<size_t>(kWaves) * 32 * (DP + 2) * 4,
                "the waves' partial outputs are joined in the tiles' memory");

  int kw;
  int64_t b;
  int hk;
  uint32_t krow, vrow, unit_at[CPW];                // a lane's share of the copies

  __device__ __forceinline__ Attention(const AttnArgs& args, Lds& shared) : Core(args, shared) {}

  __device__ __forceinline__ void copy_k(int s, int key0, int keys) {
    const char* base = static_cast<const char*>(g.k) + (b * g.k_b + hk * g.k_h + key0 * g.k_l) * 2;
    const int n = keys < KT ? keys : KT;
    const __amdgpu_buffer_rsrc_t buf =
        make_buffer(base, static_cast<uint32_t>(((n - 1) * g.k_l + g.D) * 2));
#pragma unroll
    for (int i = 0; i < CPW; ++i)
      buffer_to_lds16(buf, &lds.k[s * KT + (CPW * wave + i) * RPC][0], krow + unit_at[i],
                      static_cast<uint32_t>(i * RPC * 2 * g.k_l));
  }
  __device__ __forceinline__ void copy_v(int s, int key0, int keys) {
    const char* base = static_cast<const char*>(g.v) + (b * g.v_b + hk * g.v_h + key0 * g.v_l) * 2;
    const int n = keys < KT ? keys : KT;
    const __amdgpu_buffer_rsrc_t buf =
        make_buffer(base, static_cast<uint32_t>(((n - 1) * g.v_l + g.D) * 2));
#pragma unroll
    for (int i = 0; i < CPW; ++i)
      buffer_to_lds16(buf, &lds.v[s * KT + (CPW * wave + i) * RPC][0], vrow + unit_at[i],
                      static_cast<uint32_t>(i * RPC * 2 * g.v_l));
  }

  // Tiles t0 .. t1-1 of the keys from `first` on, the first of them on its way to
  // stage 0, into o, m and l.
  template <bool CAREFUL>
  __device__ __forceinline__ void pass(int first, int last, int t0, int t1) {
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[d][e] = 0.f;
    m = kNegInf;
    l = 0.f;
    large = false;
    // The wave's keys of tile tt are f + tt * KT .. + 32 * KB - 1. It has no part in
    // tiles before `on` and from `off` on; every row sees all of its keys in tiles
    // `in` .. `out` - 1. A loop for each: with one loop and branches the outputs
    // are copied where the paths meet.
    const int row0 = 32 * KB * kw, f = first + row0;
    auto upto = [&](int x) {           // tiles that begin before key x, within t0 .. t1
      const int n = x > f ? (x - f + KT - 1) / KT : 0;
      return n < t0 ? t0 : n < t1 ? n : t1;
    };
    const int on = upto(w_lo + 1 - 32 * KB), off = max(on, upto(w_hi));
    int in = max(on, upto(w_lo_max)), out = min(off, upto(w_hi_min - 32 * KB + 1));
    if (CAREFUL || KB != 2 || in >= out) in = out = off;
    int tt = t0;
    auto begin = [&]() {
      const int key0 = first + tt * KT, s = (tt - t0) & 1;
      __builtin_amdgcn_s_waitcnt(wait_vmem(0));
      __syncthreads();                 // the tile is in stage s, stage s ^ 1 is free
      if (tt + 1 < t1) {
        copy_k(s ^ 1, key0 + KT, last - (key0 + KT));
        copy_v(s ^ 1, key0 + KT, last - (key0 + KT));
      }
      return s;
    };
    auto masked = [&]() {
      const int s = begin();
      if constexpr (KB == 2 && !CAREFUL) {
        this->template pair<true>(s, row0, f + tt * KT);
      } else {
#pragma unroll 1
        for (int kb = 0; kb < KB; ++kb)
          this->template block<CAREFUL>(s, row0 + 32 * kb, f + tt * KT + 32 * kb);
      }
    };
    for (; tt < on; ++tt) begin();
    for (; tt < in; ++tt) masked();
    if constexpr (KB == 2 && !CAREFUL) {
      for (; tt < out; ++tt) this->template pair<false>(begin(), row0, f + tt * KT);
      for (; tt < off; ++tt) masked();
    }
    for (; tt < t1; ++tt) begin();
    __syncthreads();                   // the tiles are no longer read
  }

  __device__ __forceinline__ void run() {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    rl = lane & 31;
    h = lane >> 5;
    kw = wave % KW;
    const int rw = wave / KW;
    int t, rt;
    if (RW > 1 && (g.causal || g.ranges != nullptr)) {
      // Row tiles of unequal work: heads next to each other, so that each of the 8
      // XCDs (to which workgroups are dealt in turn) gets long and short rows alike,
      // and the last rows first. Under the causal rule those see the most keys, so
      // that what is left at the end is short: prefix mask, 8191 tokens: 555 -> 415
      // us; causal, 8192: 350 -> 288 us. Ranges alone follow no order: heads side by
      // side take 4608 tokens in documents of 744, 1488 and 2232 from 154 to 135 us,
      // of falling length from 157 to 125, and 12 of growing or falling length from
      // 74 and 67 to 57 and 63; the first rows first would give 127, 132, 65 and 57.
      const int heads = g.B * g.Hkv * g.splits;
      t = static_cast<int>(blockIdx.x) % heads;
      rt = g.row_tiles - 1 - static_cast<int>(blockIdx.x) / heads;
    } else {
      // Equal work: the row tiles of a head on one XCD, for its K and V in that
      // L2 (42 heads of 4608 tokens: 509 -> 489 us).
      t = xcd_contiguous(static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
      rt = t % g.row_tiles;
      t /= g.row_tiles;
    }
    const int split = t % g.splits;
    t /= g.splits;
    hk = t % g.Hkv;
    b = t / g.Hkv;

    const int r = (rt * RW + rw) * 32 + rl;
    const bool real = r < g.rows;
    const int i = real ? r / g.G : 0;
    const int head = hk * g.G + (real ? r % g.G : 0);
    pos = i + g.Lk - g.Lq;
    slope2 = SLOPES ? g.slopes[head] * kLog2e : 0.f;
    lo = 0;
    int hi = g.Lk;
    if (g.ranges != nullptr) {
      const int32_t* p = g.ranges + b * g.range_b + 2 * static_cast<int64_t>(i);
      lo = p[0] > 0 ? p[0] : 0;
      hi = p[1] < hi ? p[1] : hi;
    }
    if (g.causal) {
      const int pre = g.prefix != nullptr ? g.prefix[b] : 0;
      const int c = pos + 1 > pre ? pos + 1 : pre;
      hi = c < hi ? c : hi;
    }
    width = real && hi > lo ? static_cast<uint32_t>(hi - lo) : 0u;
    if (width == 0) {                 // sees nothing
      lo = g.Lk;
      hi = 0;
    }
    // the wave's bounds; rows past the end ask for no mask
    w_lo = lo;
    w_hi = hi;
    w_lo_max = real ? lo : 0;
    w_hi_min = real ? hi : g.Lk;
#pragma unroll
    for (int d = 16; d >= 1; d /= 2) {
      w_lo = min(w_lo, __shfl_xor(w_lo, d));
      w_hi = max(w_hi, __shfl_xor(w_hi, d));
      w_lo_max = max(w_lo_max, __shfl_xor(w_lo_max, d));
      w_hi_min = min(w_hi_min, __shfl_xor(w_hi_min, d));
    }
    w_lo = __builtin_amdgcn_readfirstlane(w_lo);
    w_hi = __builtin_amdgcn_readfirstlane(w_hi);
    w_lo_max = __builtin_amdgcn_readfirstlane(w_lo_max);
    w_hi_min = __builtin_amdgcn_readfirstlane(w_hi_min);
    if (lane == 0) {
      lds.bounds[wave][0] = w_lo;
      lds.bounds[wave][1] = w_hi;
    }
    __syncthreads();
    int first = lds.bounds[0][0], last = lds.bounds[0][1];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
      first = min(first, lds.bounds[w][0]);
      last = max(last, lds.bounds[w][1]);
    }
    first = __builtin_amdgcn_readfirstlane(first);
    last = __builtin_amdgcn_readfirstlane(last);
    // this workgroup's share of the tiles
    const int tiles = last > first ? (last - first + KT - 1) / KT : 0;
    const int t0 = static_cast<int>(static_cast<int64_t>(tiles) * split / g.splits);
    const int t1 = static_cast<int>(static_cast<int64_t>(tiles) * (split + 1) / g.splits);

    kb0 = k_base();
    vb0 = v_base();
    // the first of the wave's rows that this lane copies; units past D (a multiple
    // of 8 channels) get an offset beyond any buffer
    const int copied = CPW * wave * RPC + lane / UNITS;
    krow = static_cast<uint32_t>(copied * g.k_l * 2);
    vrow = static_cast<uint32_t>(copied * g.v_l * 2);
#pragma unroll
    for (int c = 0; c < CPW; ++c) {
      const int unit = (lane % UNITS) ^ twist(copied + c * RPC);
      unit_at[c] = unit * 8 < g.D ? static_cast<uint32_t>(unit * 16) : 0x80000000u;
    }
    const int start = first + t0 * KT;
    if (t0 < t1) {
      copy_k(0, start, last - start);
      copy_v(0, start, last - start);
    }

    const T* qp = static_cast<const T*>(g.q) + b * g.q_b + static_cast<int64_t>(i) * g.q_l +
                  static_cast<int64_t>(head) * g.q_h;
#pragma unroll
    for (int s = 0; s < DS; ++s) {
      const int c = (2 * s + h) * 8;
      v4i z = v4i{0, 0, 0, 0};
      if (real && c < g.D && g.q_sign != 0) {
        z = *reinterpret_cast<const v4i*>(qp + c);
        if (g.q_sign < 0) z = z ^ static_cast<int>(0x80008000u);
      }
      qf[s] = __builtin_bit_cast(vec, z);
    }
    // A hidden key has P = 0, but 0 times an infinity or a NaN in V would reach the
    // rows that do not see it, and a sum of bf16 values can overflow where their average
    // does not. Both leave an output that is not finite, so the first pass does not look
    // at V; only then a second one does, with lower weights.
    pass<false>(first, last, t0, t1);
    bool odd = false;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) odd |= !(fabsf(o[d][e]) < __builtin_inff());
    const bool again = __builtin_amdgcn_ballot_w64(odd) != 0;
    if (lane == 0) lds.odd[wave] = again;
    __syncthreads();
    bool any = false;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) any |= lds.odd[w] != 0;
    if (__builtin_amdgcn_readfirstlane(any)) {
      if (t0 < t1) {
        copy_k(0, start, last - start);
        copy_v(0, start, last - start);
      }
      pass<true>(first, last, t0, t1);
    }
    l = half_sum(l);
    if constexpr (KW > 1) join_waves();
    if (KW == 1 || wave == 0) store(real, split, r, i, head);
  }

  // Adds the partial results of the workgroup's waves, in wave order, into
  // wave 0: o in fp32 scaled to the common maximum.
  __device__ __forceinline__ void join_waves() {
    float* mem = reinterpret_cast<float*>(&lds);
    float* ml = mem + kWaves * 32 * DP;
    if (h == 0) {
      ml[(wave * 32 + rl) * 2] = m;
      ml[(wave * 32 + rl) * 2 + 1] = l;
    }
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) mem[((wave * DB + d) * 16 + e) * 64 + lane] = o[d][e];
    __syncthreads();
    if (wave != 0) return;
    float top = kNegInf;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, ml[(w * 32 + rl) * 2]);
    // two above the largest: the sum of four finite partial outputs is finite
    const float base = top == kNegInf ? 0.f : top + 2.f;
    float f[kWaves];
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      f[w] = __builtin_amdgcn_exp2f(ml[(w * 32 + rl) * 2] - base);
      l = __builtin_fmaf(ml[(w * 32 + rl) * 2 + 1], f[w], l);
    }
    m = top == kNegInf ? top : base;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
          v = __builtin_fmaf(mem[((w * DB + d) * 16 + e) * 64 + lane], f[w], v);
        o[d][e] = v;
      }
  }

  __device__ __forceinline__ void store(bool real, int split, int r, int i, int head) {
    if (!real) return;
    if (g.splits > 1) {
      const int64_t row = ((static_cast<int64_t>(split) * g.B + b) * g.Hkv + hk) * g.rows + r;
      if (h == 0) {
        g.part_ml[2 * row] = m;
        g.part_ml[2 * row + 1] = l;
      }
      if (l == 0.f) return;            // the join reads no outputs of such a row
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int ch = 32 * d + 8 * e + 4 * h;
          if (ch < g.D)
            *reinterpret_cast<v4f*>(g.part_o + row * g.D + ch) =
                v4f{o[d][4 * e], o[d][4 * e + 1], o[d][4 * e + 2], o[d][4 * e + 3]};
        }
      return;
    }
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    T* op = static_cast<T*>(g.out) + b * g.o_b + static_cast<int64_t>(i) * g.o_l +
            static_cast<int64_t>(head) * g.o_h;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int ch = 32 * d + 8 * e + 4 * h;
        if (ch < g.D) {
          typedef T vec4 __attribute__((ext_vector_type(4)));
          vec4 y;
#pragma unroll
          for (int c = 0; c < 4; ++c) y[c] = static_cast<T>(o[d][4 * e + c] * inv);
          *reinterpret_cast<vec4*>(op + ch) = y;
        }
      }
  }
};

template <class T, int DP, int RW, int CAP, bool SLOPES>
__global__ __launch_bounds__(64 * kWaves, 2) void attention_kernel(const AttnArgs g) {
  using A = Attention<T, DP, RW, CAP, SLOPES>;
  __shared__ typename A::Lds lds;
  A a(g, lds);
  a.run();
}

// Joins the splits of one output row in a workgroup: 32 lanes hold its channels,
// 4 each, and 8 groups of lanes take the splits in turn; their sums are added in
// order. Every load is issued before the first is needed, the row being short.
constexpr int kJoin = 8;
constexpr int kMaxSplits = 64;

template <class T>
__global__ __launch_bounds__(32 * kJoin) void attention_join(const AttnArgs g) {
  __shared__ v4f sums[kJoin][32];
  __shared__ float weights[kJoin];
  const int64_t all = static_cast<int64_t>(g.B) * g.Hkv * g.rows;
  const int64_t row = blockIdx.x;
  const int group = threadIdx.x / 32, ch = 4 * (threadIdx.x % 32);
  // the row's maxima and sums, one split per lane
  const int lane = threadIdx.x % 64;
  float m = kNegInf, l = 0.f;
  if (lane < g.splits) {
    m = g.part_ml[2 * (lane * all + row)];
    l = g.part_ml[2 * (lane * all + row) + 1];
  }
  float top = m;
#pragma unroll
  for (int d = 32; d >= 1; d /= 2) top = fmaxf(top, __shfl_xor(top, d));
  // 2^6 splits at most: the sum of their finite partial outputs is finite
  const float f = l == 0.f ? 0.f : __builtin_amdgcn_exp2f(m - (top == kNegInf ? 0.f : top + 6.f));
  v4f o = v4f{0.f, 0.f, 0.f, 0.f};
  float n = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxSplits / kJoin; ++i) {
    const int s = group + i * kJoin;
    const float fs = __shfl(f, s), ls = __shfl(l, s);
    if (s >= g.splits || ls == 0.f) continue;      // nothing was written for it
    n = __builtin_fmaf(ls, fs, n);
    if (ch < g.D) {
      const v4f p = *reinterpret_cast<const v4f*>(g.part_o + (s * all + row) * g.D + ch);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(p[e], fs, o[e]);
    }
  }
  sums[group][threadIdx.x % 32] = o;
  if (threadIdx.x % 32 == 0) weights[group] = n;
  __syncthreads();
  if (group != 0 || ch >= g.D) return;
#pragma unroll
  for (int i = 1; i < kJoin; ++i) {
    const v4f p = sums[i][threadIdx.x];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = o[e] + p[e];
    n = n + weights[i];
  }
  const float inv = n == 0.f ? 0.f : 1.0f / n;
  const int64_t r = row % g.rows, bh = row / g.rows;
  const int64_t b = bh / g.Hkv, hk = bh % g.Hkv;
  T* op = static_cast<T*>(g.out) + b * g.o_b + (r / g.G) * g.o_l + (hk * g.G + r % g.G) * g.o_h + ch;
  typedef T vec4 __attribute__((ext_vector_type(4)));
  vec4 y;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = static_cast<T>(o[e] * inv);
  *reinterpret_cast<vec4*>(op) = y;
}

template <class T, int DP, int RW, int CAP>
void launch_s(const AttnArgs& g, unsigned grid, hipStream_t stream) {
  if (g.slopes != nullptr)
    hipLaunchKernelGGL((attention_kernel<T, DP, RW, CAP, true>), dim3(grid), dim3(64 * kWaves), 0,
                       stream, g);
  else
    hipLaunchKernelGGL((attention_kernel<T, DP, RW, CAP, false>), dim3(grid), dim3(64 * kWaves), 0,
                       stream, g);
}

template <class T, int DP, int RW>
void launch_c(const AttnArgs& g, unsigned grid, hipStream_t stream) {
  g.cap == kNoCap     ? launch_s<T, DP, RW, kNoCap>(g, grid, stream)
  : g.cap == kNearCap ? launch_s<T, DP, RW, kNearCap>(g, grid, stream)
                      : launch_s<T, DP, RW, kAnyCap>(g, grid, stream);
}

template <class T>
hipError_t launch_t(const AttnArgs& g, const AttnPlan& p, hipStream_t stream) {
  if (p.few)
    g.D > 64 ? launch_c<T, 128, 1>(g, p.grid, stream) : launch_c<T, 64, 1>(g, p.grid, stream);
  else
    g.D > 64 ? launch_c<T, 128, 4>(g, p.grid, stream) : launch_c<T, 64, 4>(g, p.grid, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || g.splits == 1) return e;
  const int64_t rows = static_cast<int64_t>(g.B) * g.Hkv * g.rows;
  hipLaunchKernelGGL(attention_join<T>, dim3(static_cast<unsigned>(rows)), dim3(32 * kJoin), 0,
                     stream, g);
  return hipGetLastError();
}

}  // namespace

// The row tile (128 rows, a wave each 32 of them, or 32, the waves sharing a
// tile's keys) and the split along the keys of least estimated time, in
// microseconds measured at D = 128: a tile of a workgroup that has its compute
// unit to itself takes 1.8 (128 keys, 32 rows) or 1.2 (64 keys, 128 rows); 32 rows
// are bound by memory from about 150 workgroups on, 128 rows share their unit
// beyond one workgroup each; a workgroup's start and end take 2.5, and joining
// splits 6 and their outputs written and read at 4 TB/s. One token, 32 heads over
// 8, 8 caches of 8191: 55 us with 4 splits, 124 with one, 65 with 16; one cache: 17,
// 78 (32 splits). 32 rows against 128: 500 causal tokens of 8 heads 9.4 against
// 16.8 us, 1000 of 4 heads 17 against 23, 77 of 24 heads alike.
AttnPlan attention_plan(int64_t B, int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hkv, int64_t D,
                        bool split) {
  AttnPlan p{};
  const int64_t rows = Lq * (Hq / Hkv);
  const int cus = resident_slots() / 2;
  float least = -1.f;
  constexpr int kTried[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, kMaxSplits};
  for (const bool few : {true, false}) {
    if (!few && rows <= 32) break;
    const int64_t row_tiles = (rows + (few ? 31 : 127)) / (few ? 32 : 128);
    const int64_t wgs = row_tiles * B * Hkv;
    const int64_t tiles = (Lk + (few ? 127 : 63)) / (few ? 128 : 64);
    const int slots = few && D > 64 ? cus : 2 * cus;
    for (const int s : kTried) {
      if (s > 1 && (!split || s > tiles)) break;
      // the grids of the kernel and of the join of its rows
      if (!grid_fits(wgs * s, 64 * kWaves) || (s > 1 && !grid_fits(B * Hkv * rows, 32 * kJoin)))
        break;
      const float all = static_cast<float>(wgs) * static_cast<float>(s);
      const float active = all < slots ? all : static_cast<float>(slots);
      const float rounds = std::ceil(all / static_cast<float>(slots));
      float tile;
      if (few) {
        tile = 0.0124f * active * (D > 64 ? 1.f : 0.5f);
        if (tile < 1.8f) tile = 1.8f;
      } else {
        tile = active <= cus ? 1.2f : 1.2f + 1.3f * (active - cus) / cus;
      }
      float us = rounds * (static_cast<float>((tiles + s - 1) / s) * tile + 2.5f);
      if (s > 1)
        us += 6.f + static_cast<float>(B * Lq) * static_cast<float>(Hq * D) * s * 8.f / 4e6f;
      if (least < 0.f || us < least) {
        least = us;
        p.few = few;
        p.row_tiles = row_tiles;
        p.wgs = wgs * s;
        p.splits = s;
      }
    }
  }
  p.grid = static_cast<unsigned>(p.wgs);
  return p;
}

hipError_t launch_attention(AttnArgs g, int dtype, const AttnPlan& p, hipStream_t stream) {
  g.row_tiles = static_cast<int>(p.row_tiles);
  g.splits = p.splits;
  return dtype == SVDQ_F16 ? launch_t<_Float16>(g, p, stream) : launch_t<__bf16>(g, p, stream);
}

}  // namespace svdq
