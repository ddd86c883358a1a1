// The arithmetic of the attention kernels (gfx950): scores, softmax and weighted sums of
// tiles of K and V that lie in LDS, for one wave of 32 rows. The kernels bring the tiles
// there, say which keys a row sees, and store the outputs.
#pragma once

#include <hip/hip_runtime.h>

#include "attention.hpp"
#include "block_common.hpp"

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

// RW waves along the rows, 4 / RW along the keys of a tile; ROWS rows of K and V in LDS
// (whole stages of a tile's KT keys). ARGS holds scale2, cap_in and cap2. With HOLES,
// bit n of `holes` hides the tile's keys 16 n .. 16 n + 15 from every row.
template <class T, int DP, int RW, int CAP, bool SLOPES, int ROWS, class ARGS, bool HOLES = false>
struct AttentionCore {
  static constexpr int KW = kWaves / RW;
  static constexpr int KB = KW == 1 ? 2 : 1;        // blocks of 32 keys per wave and tile
  static constexpr int KT = 32 * KB * KW;           // keys per tile
  static constexpr int DB = DP / 32, DS = DP / 16;  // output blocks, steps of the dot product
  static constexpr int UNITS = DP / 8;              // 16-byte units per row
  typedef typename Half<T>::vec vec;

  // one object, and reads through plain vector types: with several, or
  // through a struct, the compiler makes every read wait for every copy
  struct alignas(16) Lds {
    uint8_t k[ROWS][DP * 2];
    uint8_t v[ROWS][DP * 2];
    int bounds[kWaves][2];
    int odd[kWaves];
  };

  const ARGS& g;
  Lds& lds;
  int lane, wave, rl, h;
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
  uint32_t holes;

  __device__ __forceinline__ AttentionCore(const ARGS& args, Lds& shared) : g(args), lds(shared) {}

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
    const uint8_t* p = &lds.v[0][0] + row * DP * 2;
    // rows 8 apart differ in one bit of their twist
    const v4s lo4 = read_tr(p + (at ^ (d * 64)));
    const v4s hi4 = read_tr(p + 8 * DP * 2 + (at ^ (d * 64) ^ 32));
    return __builtin_shufflevector(lo4, hi4, 0, 1, 2, 3, 4, 5, 6, 7);
  }

  // Without a cap and slopes a score stays as the products give it and its scale
  // goes into the exponential; with them it is made a base-2 logit here. (With HOLES
  // slopes too leave it so: slope2 is then in the scores' units, and the distance of a
  // key is one subtraction of whole numbers in fp32.)
  static constexpr bool RAW = CAP == kNoCap && (!SLOPES || HOLES);

  // x = K Q^T of the 32 keys from LDS row `row0` on; at: the stage's base address
  __device__ __forceinline__ v16f products(int at, int row0) {
    v16f x;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
    const uint8_t* p = &lds.k[0][0] + row0 * DP * 2;
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
  // lane's in base 2. key0: the block's first key; gone: its bits of `holes`.
  template <bool MASK>
  __device__ __forceinline__ float logits(v16f& x, int key0, uint32_t gone) {
    float top = kNegInf;
    const float away = SLOPES && HOLES ? static_cast<float>(pos - key0 - 4 * h) : 0.f;
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
      } else if constexpr (SLOPES && !HOLES) {
        v = v * g.scale2;
      }
      if constexpr (SLOPES && HOLES)
        v = __builtin_fmaf(-slope2, fabsf(away - static_cast<float>((i & 3) + 8 * (i >> 2))), v);
      else if constexpr (SLOPES)
        v = __builtin_fmaf(-slope2, fabsf(static_cast<float>(pos - key)), v);
      if constexpr (MASK) v = static_cast<uint32_t>(key - lo) < width ? v : kNegInf;
      if constexpr (MASK && HOLES) v = (gone >> (i >> 3) & 1) != 0 ? kNegInf : v;
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

  // x -> P in 16 bits (the operands of 16 keys each). The rounding is a choice: weights
  // in fp32 would need two 16-bit operands each, twice the second product's matrix
  // instructions. A bf16 output is off by 0.0022 to 0.0024 of its norm with it, 0.0017 by its own
  // rounding alone; fp16 0.00026 to 0.0003 and 0.00021 (prompts and single tokens).
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
      const uint8_t* row = &lds.v[s * KT + row0 + k][0];
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
    const float top = half_max(logits<true>(x, key0, holes));
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
    float top = half_max(logits<MASK>(x, key0, holes));
    if (outgrows<false>(top)) raise<false>(top);
    float scale = exp_scale(x);
    v16f y = products(ka, row0 + 32);
    exponentials(x, scale, p);
    __builtin_amdgcn_sched_barrier(0);
    add_weights(p);                      // while y's products are on their way
    top = half_max(logits<MASK>(y, key0 + 32, holes >> 2));
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
};

}  // namespace

}  // namespace svdq
