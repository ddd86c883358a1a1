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
#include "block_common.hpp"
#include "block_launch.hpp"
#include "k2_common.hpp"

namespace svdq {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_inff();
constexpr int kWaves = 4;
constexpr float kLarge = 1e6f;       // logits (base 2); their rounding is below 2^-4

template <class T>
struct Half;
template <>
struct Half<_Float16> {
  typedef v8h vec;
  static __device__ __forceinline__ v16f mfma(v8h a, v8h b, v16f c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
  // c plus elements i and i + 1 of x, read from their halves of the register (a
  // conversion of each to fp32 first: DiT 312 us instead of 295; the two-element dot
  // product: 298)
  static __device__ __forceinline__ float add2(v8h x, int i, float c) {
    typedef _Float16 v2 __attribute__((ext_vector_type(2)));
    const uint32_t u = __builtin_bit_cast(uint32_t, v2{x[i], x[i + 1]});
    asm("v_fma_mix_f32 %0, %1, 1.0, %0 op_sel_hi:[1,0,0]" : "+v"(c) : "v"(u));
    asm("v_fma_mix_f32 %0, %1, 1.0, %0 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "+v"(c) : "v"(u));
    return c;
  }
  static constexpr uint16_t kInf = 0x7C00;
  // What is far below a row's largest weight falls among fp16's subnormal numbers, so
  // the largest is not 1 but up to 2^11: a weight's step is at most 2^-34 of it, where
  // it was 2^-24. 2^4 above that the outputs are rescaled, below 65504.
  static constexpr float kLift = 11.f, kGrow = 4.f;
  static constexpr float kCarefulLift = kLift;      // no sum of fp16 values is that large
};
template <>
struct Half<__bf16> {
  typedef v8bf vec;
  static __device__ __forceinline__ v16f mfma(v8bf a, v8bf b, v16f c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  // (in place of one addition of the unrounded weight each: prefix 367 -> 338 us)
  static __device__ __forceinline__ float add2(v8bf x, int i, float c) {
    typedef __bf16 v2 __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_fdot2_f32_bf16(v2{x[i], x[i + 1]}, v2{1.f, 1.f}, c, false);
  }
  static constexpr uint16_t kInf = 0x7F80;
  static constexpr float kLift = 0.f, kGrow = 8.f;
  // In the careful pass: sums of values near the type's (and fp32's) largest stay finite
  // where each weight is at most 2^-24, for up to 2^24 keys.
  static constexpr float kCarefulLift = -32.f;
};

typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef unsigned short v8u __attribute__((ext_vector_type(8)));

// max over the two lanes that share a row (lane and lane ^ 32); sum likewise
__device__ __forceinline__ void half_pair(float x, float& a, float& b) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t r0 = r[0], r1 = r[1];   // scalars: a bit cast of an element takes element 0
  a = __builtin_bit_cast(float, r0);
  b = __builtin_bit_cast(float, r1);
}
__device__ __forceinline__ float half_max(float x) {
  float a, b;
  half_pair(x, a, b);
  return fmaxf(a, b);
}
__device__ __forceinline__ float half_sum(float x) {
  float a, b;
  half_pair(x, a, b);
  return a + b;
}

// A transposing read: 16 lanes bring 4 rows x 16 channels, lane i gets channel i
// of the 4 rows. The restrict pointer is there for the compiler's alias
// information: without any, it makes the read wait for every copy in flight.
__device__ __forceinline__ v4s read_tr(const uint8_t* __restrict__ p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(p));
}

// RW waves along the rows, 4 / RW along the keys of a tile.
template <class T, int DP, int RW, int CAP, bool SLOPES>
struct Attention {
  static constexpr int KW = kWaves / RW;
  static constexpr int KB = KW == 1 ? 2 : 1;        // blocks of 32 keys per wave and tile
  static constexpr int KT = 32 * KB * KW;           // keys per tile
  static constexpr int DB = DP / 32, DS = DP / 16;  // output blocks, steps of the dot product
  static constexpr int UNITS = DP / 8;              // 16-byte units per row
  static constexpr int RPC = 64 / UNITS;            // rows per copy instruction
  static constexpr int CPW = KT / RPC / kWaves;     // copy instructions per wave and operand
  typedef typename Half<T>::vec vec;

  // one object, and reads through plain vector types: with several, or
  // through a struct, the compiler makes every read wait for every copy
  struct alignas(16) Lds {
    uint8_t k[2][KT][DP * 2];
    uint8_t v[2][KT][DP * 2];
    int bounds[kWaves][2];
    int odd[kWaves];
  };
  static_assert(KW == 1 || sizeof(Lds::k) + sizeof(Lds::v) >=
                               static_cast<size_t>(kWaves) * 32 * (DP + 2) * 4,
                "the waves' partial outputs are joined in the tiles' memory");

  const AttnArgs& g;
  Lds& lds;
  int lane, wave, rl, h, kw;
  int64_t b;
  int hk;
  vec qf[DS];
  v16f o[DB];
  // the row's reference (base 2) and this half's sum. The reference is the running
  // maximum rounded up to a whole number, so that rescaling multiplies by a power of
  // two, which rounds nothing, less kLift. It only follows the maximum when that has
  // grown by more than kGrow: until then exp2(x - m) stays below 2^(kLift + kGrow) and
  // nothing needs rescaling.
  float m, l;
  int lo, pos;                                      // the row's first key, its own position
  uint32_t width;                                   // keys it sees, from lo on
  bool large;                                       // a reference beyond kLarge
  int w_lo, w_hi, w_lo_max, w_hi_min;               // over the wave's rows
  float slope2;
  int kb0, vb0;                                     // k_base(), v_base()
  uint32_t krow, vrow, unit_at[CPW];                // a lane's share of the copies

  __device__ __forceinline__ Attention(const AttnArgs& args, Lds& shared) : g(args), lds(shared) {}

  __device__ __forceinline__ void copy_k(int s, int key0, int keys) {
    const char* base = static_cast<const char*>(g.k) + (b * g.k_b + hk * g.k_h + key0 * g.k_l) * 2;
    const int n = keys < KT ? keys : KT;
    const __amdgpu_buffer_rsrc_t buf =
        make_buffer(base, static_cast<uint32_t>(((n - 1) * g.k_l + g.D) * 2));
#pragma unroll
    for (int i = 0; i < CPW; ++i)
      buffer_to_lds16(buf, &lds.k[s][(CPW * wave + i) * RPC][0], krow + unit_at[i],
                      static_cast<uint32_t>(i * RPC * 2 * g.k_l));
  }
  __device__ __forceinline__ void copy_v(int s, int key0, int keys) {
    const char* base = static_cast<const char*>(g.v) + (b * g.v_b + hk * g.v_h + key0 * g.v_l) * 2;
    const int n = keys < KT ? keys : KT;
    const __amdgpu_buffer_rsrc_t buf =
        make_buffer(base, static_cast<uint32_t>(((n - 1) * g.v_l + g.D) * 2));
#pragma unroll
    for (int i = 0; i < CPW; ++i)
      buffer_to_lds16(buf, &lds.v[s][(CPW * wave + i) * RPC][0], vrow + unit_at[i],
                      static_cast<uint32_t>(i * RPC * 2 * g.v_l));
  }

  // Unit u of row r lies at u ^ twist(r). LDS has 64 banks of 4 bytes. A read of
  // the K operand takes one unit of 16 consecutive rows at a time, one of V^T 64
  // bytes of 4 consecutive rows (starting at a multiple of 4): the twist has to
  // differ in all of 16 rows (rows of 256 bytes) or in 8 of one parity (128
  // bytes), and in its bit of 64 bytes between rows that share banks among 4.
  static __device__ __forceinline__ int twist(int r) {
    return UNITS == 16 ? 4 * (r & 3) + ((r >> 2) & 3) : 2 * (r & 2) + ((r >> 2) & 3);
  }

  // Addresses within a stage. Rows are 2 * DP bytes and a multiple of 16 rows
  // apart the twist is the same, so all operands of a tile come from two base
  // addresses per lane: the unit's bits are flipped by constants and whole groups
  // of rows are added. (Kept in registers each, they would not fit beside the
  // outputs; opaque() stops the compiler from doing that.)
  static __device__ __forceinline__ int opaque(int x) {
    asm volatile("" : "+v"(x));
    return x;
  }
  __device__ __forceinline__ int k_at(int s) const { return opaque(kb0 + s * KT * DP * 2); }
  __device__ __forceinline__ int v_at(int s) const { return opaque(vb0 + s * KT * DP * 2); }
  // K: row rl, unit h.
  __device__ __forceinline__ int k_base() const { return rl * DP * 2 + ((h ^ twist(rl)) << 4); }
  // V: row 4h + a/4, the 4 channels at 16 * (group & 1) + 4 * (a & 3), a = lane % 16.
  __device__ __forceinline__ int v_base() const {
    const int a = lane & 15, row = 4 * h + (a >> 2), ch = (lane & 16) + 4 * (a & 3);
    return row * DP * 2 + (((ch >> 3) ^ twist(row)) << 4) + (ch & 4) * 2;
  }

  // The V^T operand of 16 keys (from LDS row `row`, a multiple of 16) and output
  // block d: lane (d, h) gets keys 4h .. 4h+3 and 8+4h .. 8+4h+3 of channel 32 d +
  // lane % 32. at: the stage's base address.
  __device__ __forceinline__ v8s v_frag(int at, int row, int d) const {
    const uint8_t* p = &lds.v[0][0][0] + row * DP * 2;
    // rows 8 apart differ in one bit of their twist
    const v4s lo4 = read_tr(p + (at ^ (d * 64)));
    const v4s hi4 = read_tr(p + 8 * DP * 2 + (at ^ (d * 64) ^ 32));
    return __builtin_shufflevector(lo4, hi4, 0, 1, 2, 3, 4, 5, 6, 7);
  }

  // Without a cap and slopes a score stays as the products give it and its scale
  // goes into the exponential; with them it is made a base-2 logit here.
  static constexpr bool RAW = CAP == kNoCap && !SLOPES;

  // x = K Q^T of the 32 keys from LDS row `row0` on; at: the stage's base address
  __device__ __forceinline__ v16f products(int at, int row0) {
    v16f x;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
    const uint8_t* p = &lds.k[0][0][0] + row0 * DP * 2;
#pragma unroll
    for (int t = 0; t < DS; ++t) {
      const v4i kf = *reinterpret_cast<const v4i*>(p + (at ^ (t * 32)));
      x = Half<T>::mfma(__builtin_bit_cast(vec, kf), qf[t], x);
    }
    return x;
  }

  // cap * tanh(y) of a score, with an error relative to itself. The difference from 1
  // loses what is small beside the cap (2^-23 of it, 5e-6 of a logit at a cap of 64,
  // but 0.1 at 1e6), so below |y| = 1/4 it is y (1 + u (c1 + c2 u)), u = y^2, with the
  // coefficients of least largest error over that range (5e-7). c1 and c2 are those for
  // t = (2 log2(e) y)^2. Both forms for every score cost more vector work (16 heads over
  // 4, 8191 causal rows with a prefix, bf16: 435 us against 350), so caps up to kNearest
  // keep the one.
  __device__ __forceinline__ float any_cap(float v) const {
    constexpr float kSmall = 0.25f * 2.0f * kLog2e, c1 = -0.04002727f, c2 = 0.001857806f;
    const float z = v * g.cap_in, t = z * z;
    const float e = __builtin_amdgcn_exp2f(z);
    const float far = g.cap2 * __builtin_fmaf(-2.0f, __builtin_amdgcn_rcpf(e + 1.0f), 1.0f);
    const float x = v * g.scale2;
    const float near = __builtin_fmaf(x * t, __builtin_fmaf(c2, t, c1), x);
    return fabsf(z) < kSmall ? near : far;
  }

  // Scores to logits (see RAW) with the masked ones at -inf; the largest of this
  // lane's in base 2. key0: the block's first key.
  template <bool MASK>
  __device__ __forceinline__ float logits(v16f& x, int key0) {
    float top = kNegInf;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int key = key0 + (i & 3) + 8 * (i >> 2) + 4 * h;
      float v = x[i];
      if constexpr (CAP == kNearCap) {
        // cap * tanh(y) with tanh(y) = 1 - 2 / (exp(2 y) + 1)
        const float e = __builtin_amdgcn_exp2f(v * g.cap_in);
        v = __builtin_fmaf(-2.0f * g.cap2, __builtin_amdgcn_rcpf(e + 1.0f), g.cap2);
      } else if constexpr (CAP == kAnyCap) {
        v = any_cap(v);
      } else if constexpr (SLOPES) {
        v = v * g.scale2;
      }
      if constexpr (SLOPES)
        v = __builtin_fmaf(-slope2, fabsf(static_cast<float>(pos - key)), v);
      if constexpr (MASK) v = static_cast<uint32_t>(key - lo) < width ? v : kNegInf;
      x[i] = v;
      top = fmaxf(top, v);
    }
    return RAW ? top * g.scale2 : top;
  }

  // Whether a block's largest logits (the row's, of both halves) outgrow the
  // reference in any row; the new reference if so.
  template <bool CAREFUL>
  static constexpr float lift() {
    return CAREFUL ? Half<T>::kCarefulLift : Half<T>::kLift;
  }
  template <bool CAREFUL>
  __device__ __forceinline__ bool outgrows(float top) const {
    return __builtin_amdgcn_ballot_w64(top > m + (lift<CAREFUL>() + Half<T>::kGrow)) != 0;
  }
  template <bool CAREFUL>
  __device__ __forceinline__ float raise(float top) {
    const float m_new = fmaxf(m, __builtin_ceilf(top) - lift<CAREFUL>());
    const float alpha = m_new == kNegInf ? 1.f : __builtin_amdgcn_exp2f(m - m_new);
    m = m_new;
    large = __builtin_amdgcn_ballot_w64(m > kLarge || (m < -kLarge && m != kNegInf)) != 0;
    l = l * alpha;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] = o[d][i] * alpha;
    return alpha;                        // what everything under the old reference is worth
  }
  // what the exponentials subtract; -inf: a row that has seen no key yet
  __device__ __forceinline__ float base() const { return m == kNegInf ? 0.f : m; }

  // The scale of the exponentials' exp2(scale * x - base) in one rounding. The
  // maximum that base comes from was rounded as a product: it can lie below the
  // product that goes in here, by 2^-4 up to a base of kLarge, but by enough to
  // overflow beyond. Then the product is rounded first, as the maximum was.
  __device__ __forceinline__ float exp_scale(v16f& x) {
    if constexpr (!RAW) return 1.f;
    if (!large) return g.scale2;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = x[i] * g.scale2;
    return 1.f;
  }

  // x -> P in 16 bits (the operands of 16 keys each)
  __device__ __forceinline__ void exponentials(const v16f& x, float scale, vec (&p)[2]) {
    const float sub = base();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float e = __builtin_amdgcn_exp2f(RAW ? __builtin_fmaf(x[i], scale, -sub) : x[i] - sub);
      p[i >> 3][i & 7] = static_cast<T>(e);
    }
  }
  // l += P as it was rounded: a row's weights then add up to 1 whatever their rounding
  __device__ __forceinline__ void add_weights(const vec (&p)[2]) {
#pragma unroll
    for (int i = 0; i < 16; i += 2) l = Half<T>::add2(p[i >> 3], i & 7, l);
  }

  // O^T += V^T P^T over the 32 keys from row0 on, every key seen
  __device__ __forceinline__ void pv(int at, int row0, const vec (&p)[2]) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int d = 0; d < DB; ++d)
        o[d] = Half<T>::mfma(__builtin_bit_cast(vec, v_frag(at, row0 + 16 * t, d)), p[t], o[d]);
  }

  // The same with the infinities and NaN of V taken out of the operands;
  // add_special() brings them to the rows that see their keys.
  __device__ __forceinline__ void pv_careful(int s, int at, int row0, int key0, const vec (&p)[2]) {
    bool special = false;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      v8s v[DB];
      v8u big = v8u{0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        v[d] = v_frag(at, row0 + 16 * t, d);
        big = __builtin_elementwise_max(big, __builtin_bit_cast(v8u, v[d] & short{0x7FFF}));
      }
      uint16_t most = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) most = most > big[e] ? most : big[e];
      if (__builtin_amdgcn_ballot_w64(most >= Half<T>::kInf) != 0) {
        special = true;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if ((static_cast<uint16_t>(v[d][e]) & 0x7FFF) >= Half<T>::kInf) v[d][e] = 0;
      }
#pragma unroll
      for (int d = 0; d < DB; ++d)
        o[d] = Half<T>::mfma(__builtin_bit_cast(vec, v[d]), p[t], o[d]);
    }
    if (special) add_special(s, row0, key0);
  }

  // o += every infinity and NaN of V in the block's keys that the row sees (as
  // often as each is looked at; the sum is the same).
  __device__ __forceinline__ void add_special(int s, int row0, int key0) {
#pragma unroll 1
    for (int k = 0; k < 32; ++k) {
      const bool seen = static_cast<uint32_t>(key0 + k - lo) < width;
      const uint8_t* row = &lds.v[s][row0 + k][0];
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int ch = 32 * d + 8 * e + 4 * h, unit = (ch >> 3) ^ twist(row0 + k);
          typedef T vec4 __attribute__((ext_vector_type(4)));
          const v4s bits = *reinterpret_cast<const v4s*>(row + unit * 16 + (ch & 4) * 2);
          const vec4 val = __builtin_bit_cast(vec4, bits);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const bool take = seen && (static_cast<uint16_t>(bits[c]) & 0x7FFF) >= Half<T>::kInf;
            o[d][4 * e + c] = o[d][4 * e + c] + (take ? static_cast<float>(val[c]) : 0.f);
          }
        }
    }
  }

  // One block of 32 keys, whose first row in stage s is row0 and first key key0.
  template <bool CAREFUL>
  __device__ __forceinline__ void block(int s, int row0, int key0) {
    v16f x = products(k_at(s), row0);
    const float top = half_max(logits<true>(x, key0));
    if (outgrows<CAREFUL>(top)) raise<CAREFUL>(top);
    vec p[2];
    const float scale = exp_scale(x);
    exponentials(x, scale, p);
    add_weights(p);
    if constexpr (CAREFUL) pv_careful(s, v_at(s), row0, key0, p);
    else pv(v_at(s), row0, p);
  }

  // Two blocks: the softmax of one runs on the vector unit beside the products of
  // the other on the matrix cores. The branches are rare and change registers in
  // place, so that the outputs stay where they are.
  template <bool MASK>
  __device__ __forceinline__ void pair(int s, int row0, int key0) {
    const int ka = k_at(s), va = v_at(s);
    v16f x = products(ka, row0);
    vec p[2], r[2];
    float top = half_max(logits<MASK>(x, key0));
    if (outgrows<false>(top)) raise<false>(top);
    float scale = exp_scale(x);
    v16f y = products(ka, row0 + 32);
    exponentials(x, scale, p);
    __builtin_amdgcn_sched_barrier(0);
    add_weights(p);                      // while y's products are on their way
    top = half_max(logits<MASK>(y, key0 + 32));
    if (outgrows<false>(top)) {          // x's exponentials are not in o yet; exact
      const float alpha = raise<false>(top);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        p[i >> 3][i & 7] = static_cast<T>(static_cast<float>(p[i >> 3][i & 7]) * alpha);
    }
    scale = exp_scale(y);
    pv(va, row0, p);
    exponentials(y, scale, r);
    add_weights(r);
    pv(va, row0 + 32, r);
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
        pair<true>(s, row0, f + tt * KT);
      } else {
#pragma unroll 1
        for (int kb = 0; kb < KB; ++kb)
          block<CAREFUL>(s, row0 + 32 * kb, f + tt * KT + 32 * kb);
      }
    };
    for (; tt < on; ++tt) begin();
    for (; tt < in; ++tt) masked();
    if constexpr (KB == 2 && !CAREFUL) {
      for (; tt < out; ++tt) pair<false>(begin(), row0, f + tt * KT);
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
