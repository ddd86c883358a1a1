// Matrix product in e4m3 with block scales (gfx950):
//
//   Y[m, n] = act( sum_g sa[m, g] * sw[n/128, g] * P_g[m, n] + bias[n] ),
//   P_g[m, n] = sum over the 128 channels k of group g of a[m, k] * w[n, k].
//
// A matrix instruction takes one group: v_mfma_f32_16x16x128 with both
// operands in e4m3 gives P_g of a 16 x 16 block, and four fp32 multiply-adds
// per lane add it, scaled, to the accumulators. The weight block is the first
// operand, so a lane ends up with 4 consecutive columns of one row of Y and
// one activation scale serves all its columns; the weight scale is the same
// for the whole wave.
//
// Precision. The 8-bit matrix instructions align the products of one
// instruction to the largest before they add them. What is lost goes by the
// group's largest |a w|, not by its sum: at most 2^-13 of it in 60000 sums against
// fp64, which was 1e-5 to 5e-5 of |P_g| on Gaussian and heavy-tailed groups and is
// more where a group's products cancel (the accumulators across groups are fp32).
// 16-bit outputs accept that; an fp32 output takes the variant that widens the
// codes to fp16 (exact) and multiplies with v_mfma_f32_16x16x32_f16, whose
// sums are good to 1e-7, at half the matrix rate (EXACT below).
//
// Three kernels:
// - tiles: a workgroup computes BM x BN outputs, both operands copied from
//   global memory straight into LDS, one 128-byte row piece per row and chunk,
//   its 16-byte units XOR-swizzled so that the operand reads of 16 lanes cover
//   all banks. From 256 x 256 (the fewest bytes read again per product) to 64 x
//   64 (the most workgroups), chosen by estimated time; optionally split along K,
//   each slice writing fp32 partial tiles.
// - few rows (M <= 16): bound by reading the weights once. A workgroup owns 16
//   columns, its waves take the groups in turn, operands go straight to
//   registers, and the waves' accumulators are added through LDS in order.
// - the sums of a product split along K, in slice order.
//
// Measured. 4608 x 9216 x 3072 to fp16: 136 to 147 us by card, 1.8 to 1.9 PFLOP/s;
// the matrix core is busy 42% of the time, the clock falls to 1.9 GHz under it, and
// 648 tiles are 2.53 rounds of the 256 compute units. A chunk of a 256 x 256 tile
// takes 1.55 us, which is the rate of a large library product without group
// scales; what is lost is the last round and 7 us of start and end per tile. One
// row, 10240 x 1280: 4.8 us for 13 MB. 24 x 3072 x 12288: 10 to 11 us the tiles of 16
// slices (3.5 TB/s) and 2 to 4 us their sums. 1023 x 1283 x 1272 to fp32: 15 us, of which
// 7 are a launch, a tile's start and its end, the rest 10 chunks of 0.65 us that
// wait for their copies and LDS reads (without the widening 0.55).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "../../include/svdq.h"
#include "block_common.hpp"
#include "block_launch.hpp"
#include "k2_common.hpp"

namespace svdq {

namespace {

constexpr int kMaxSlices = 16;      // of a product split along K
constexpr int kChunk = kFp8Block;   // K values per group and matrix instruction
// vmcnt(n) expcnt(7) lgkmcnt(0)
constexpr int wait_copies(int n) { return (n & 15) | ((n >> 4) << 14) | 0x70; }

struct GemmArgs {
  const uint8_t* a;
  const uint8_t* w;
  const float* sa;
  const float* sw;
  const float* bias;
  void* Y;
  float* part;                      // split along K: [slice][M][part_ld(N)] fp32
  int64_t M, N, Kp, ldy;
  int slices;
};

// Row stride of the partial tiles: 4 columns move in one access.
__host__ __device__ constexpr int64_t part_ld(int64_t N) { return (N + 3) / 4 * 4; }

template <int N, int I = 0, class F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<N, I + 1>(f);
  }
}

__device__ __forceinline__ v8h widen8(int lo, int hi) {
  const v2h a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
  const v2h b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
  const v2h c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
  const v2h d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
  return v8h{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// One lane's 32 codes of a 16-row block and one group, as the 8-bit
// instruction takes them, or widened to fp16.
template <bool EXACT>
struct Frag;
template <>
struct Frag<false> {
  v8i v;
  __device__ __forceinline__ void set(v4i x, v4i y) {
    v = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};
template <>
struct Frag<true> {
  v8h v[4];
  __device__ __forceinline__ void set(v4i x, v4i y) {
    v[0] = widen8(x[0], x[1]);
    v[1] = widen8(x[2], x[3]);
    v[2] = widen8(y[0], y[1]);
    v[3] = widen8(y[2], y[3]);
  }
};

__device__ __forceinline__ v4f mfma_group(const Frag<false>& w, const Frag<false>& a) {
  const v4f zero = v4f{0.f, 0.f, 0.f, 0.f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, a.v, zero, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ v4f mfma_group(const Frag<true>& w, const Frag<true>& a) {
  v4f p = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int t = 0; t < 4; ++t) p = mfma_f16_16x16x32(w.v[t], a.v[t], p);
  return p;
}

// Global vectors may lie at any address that their elements may.
typedef int v4i_any __attribute__((ext_vector_type(4), aligned(2)));

// The 4 bias values of columns n .. n+3 (0 without a bias and past the end).
__device__ __forceinline__ v4f bias4(const GemmArgs& g, int64_t n) {
  v4f b = v4f{0.f, 0.f, 0.f, 0.f};
  if (g.bias != nullptr) {
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = g.bias[n + e < g.N ? n + e : g.N - 1];
  }
  return b;
}

template <int YT>
__device__ __forceinline__ uint16_t bits16(float x) {
  if constexpr (YT == SVDQ_F16) return f2h(x);
  else return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}

// The bias, the optional GELU and the one rounding to a 16-bit output.
template <int YT, bool GELU>
__device__ __forceinline__ uint2 round4(v4f v, v4f b) {
  uint32_t h[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float x = v[e] + b[e];
    if constexpr (GELU) x = gelu_tanh_f32(x);
    h[e] = bits16<YT>(x);
  }
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// Columns n .. n+3 of row m of Y (of type YT) from the fp32 sums v, in one
// store where Y's alignment allows it.
template <int YT, bool GELU>
__device__ __forceinline__ void finish4(const GemmArgs& g, v4f v, v4f b, int64_t m, int64_t n) {
  if (m >= g.M || n >= g.N) return;
  constexpr int ES = YT == SVDQ_F32 ? 4 : 2;
  const bool vec =
      n + 3 < g.N && ((reinterpret_cast<uintptr_t>(g.Y) | (g.ldy * ES)) % (4 * ES)) == 0;
  if constexpr (YT == SVDQ_F32) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = v[e] + b[e];
      if constexpr (GELU) v[e] = gelu_tanh_f32(v[e]);
    }
    float* y = static_cast<float*>(g.Y) + m * g.ldy + n;
    if (vec) {
      *reinterpret_cast<v4f*>(y) = v;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < g.N) y[e] = v[e];
    }
  } else {
    const uint2 h = round4<YT, GELU>(v, b);
    uint16_t* y = static_cast<uint16_t*>(g.Y) + m * g.ldy + n;
    if (vec) {
      *reinterpret_cast<uint2*>(y) = h;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < g.N) y[e] = static_cast<uint16_t>((e < 2 ? h.x : h.y) >> (16 * (e & 1)));
    }
  }
}

// ---------------------------------------------------------------------------
// Tiles: WM x WN waves, each of 16*NBM rows and 16*NBN columns; NST chunks in
// LDS. Two stages are all that fits with a large tile, whose chunk takes longer
// than its copies; a small tile's chunk does not, so four are in flight.

template <int WM, int WN, int NBM, int NBN, int NST>
struct Tile {
  static constexpr int NW = WM * WN, BM = WM * NBM * 16, BN = WN * NBN * 16;
  struct alignas(16) Stage {
    uint8_t a[BM][kChunk];
    uint8_t w[BN][kChunk];
  };
  struct Lds {
    Stage st[NST];
    alignas(16) float sal[2][BM][4];   // activation scales of 4 groups
  };
  // one 1 KB copy instruction moves 8 rows of 128 bytes; wave w takes every
  // NW-th, the last of them where there is one
  static constexpr int CA = BM / 8 / NW, CW = (BN / 8 + NW - 1) / NW;
  static_assert(CA * 8 * NW == BM && BN % 16 == 0, "whole copy instructions");
  static_assert(BM % 64 == 0 && BM / 64 <= NW, "one scale copy per wave at most");
};

template <int WM, int WN, int NBM, int NBN, int NST, int YT, bool GELU>
__global__ __launch_bounds__(64 * WM * WN) void gemm_fp8_tiles(const GemmArgs g, int tiles_m,
                                                               int tiles_n) {
  constexpr bool EXACT = YT == SVDQ_F32;
  using T = Tile<WM, WN, NBM, NBN, NST>;
  // one object: with two, the compiler tags copies and reads with the object
  // they belong to and makes every read wait for every copy in flight
  __shared__ typename T::Lds lds;
  auto& st = lds.st;
  auto& sal = lds.sal;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int wm = wave / WN, wn = wave % WN;
  const int rl = lane & 15, q = lane >> 4;

  const int tiles = tiles_m * tiles_n;
  const int slice = static_cast<int>(blockIdx.x) / tiles;
  int tm, tn;
  banded_tile(xcd_contiguous(static_cast<int>(blockIdx.x) % tiles, tiles), tiles_m, tiles_n, tm,
              tn);
  const int64_t m0 = static_cast<int64_t>(tm) * T::BM, n0 = static_cast<int64_t>(tn) * T::BN;
  const int C = static_cast<int>(g.Kp / kChunk);   // groups
  const int c0 = static_cast<int>(static_cast<int64_t>(C) * slice / g.slices);
  const int c1 = static_cast<int>(static_cast<int64_t>(C) * (slice + 1) / g.slices);

  // Rows past the end are clamped to the last one; their results are dropped.
  const int rows_a = static_cast<int>(g.M - m0 < T::BM ? g.M - m0 : T::BM);
  const int rows_w = static_cast<int>(g.N - n0 < T::BN ? g.N - n0 : T::BN);
  const __amdgpu_buffer_rsrc_t bs =
      make_buffer(g.sa + m0 * C, static_cast<uint32_t>(rows_a * C * 4));
  // position of row r's 16-byte unit u in LDS: u ^ ((r >> 1) & 7); an even and
  // an odd row lie in different halves of the 64 banks
  const int r8 = lane >> 3, unit = (lane & 7) ^ (4 * (wave & 1) + (r8 >> 1));
  static_assert(T::NW % 2 == 0, "a copy's rows start at 8 * wave, up to multiples of 16");
  uint32_t oa[T::CA], ow[T::CW];
#pragma unroll
  for (int i = 0; i < T::CA; ++i) {
    const int r = (T::NW * i + wave) * 8 + r8;
    oa[i] = static_cast<uint32_t>((r < rows_a ? r : rows_a - 1) * g.Kp + 16 * unit);
  }
#pragma unroll
  for (int i = 0; i < T::CW; ++i) {
    const int r = (T::NW * i + wave) * 8 + r8;
    ow[i] = static_cast<uint32_t>((r < rows_w ? r : rows_w - 1) * g.Kp + 16 * unit);
  }
  const int rs = 64 * wave + lane;
  const uint32_t os = static_cast<uint32_t>((rs < rows_a ? rs : rows_a - 1) * C * 4);

  // Copy `piece` of chunk c into stage s; a chunk past the end reads nothing (an
  // empty buffer), so that the pipeline below needs no branch.
  constexpr int kPieces = T::CA + T::CW;
  const uint32_t bytes_a = static_cast<uint32_t>(rows_a * g.Kp);
  const uint32_t bytes_w = static_cast<uint32_t>(rows_w * g.Kp);
  auto copy = [&](int s, int c, int piece) {
    const uint32_t at = static_cast<uint32_t>(c) * kChunk;
    if (piece < T::CA) {
      buffer_to_lds16(make_buffer(g.a + m0 * g.Kp, c < c1 ? bytes_a : 0),
                      &st[s].a[(T::NW * piece + wave) * 8][0], oa[piece < T::CA ? piece : 0], at);
    } else if (piece < kPieces) {
      const int i = piece - T::CA;
      if ((i + 1) * T::NW * 8 <= T::BN || (T::NW * i + wave) * 8 < T::BN)
        buffer_to_lds16(make_buffer(g.w + n0 * g.Kp, c < c1 ? bytes_w : 0),
                        &st[s].w[(T::NW * i + wave) * 8][0], ow[i], at);
    }
  };
  // The activation scales of chunk c and the next three, if c is the first of four.
  auto copy_scales = [&](int c) {
    if (c < c1 && ((c - c0) & 3) == 0 && wave < T::BM / 64)
      buffer_to_lds16(bs, &sal[((c - c0) >> 2) & 1][64 * wave][0], os, static_cast<uint32_t>(c) * 4);
  };

  // The wave's columns lie in one or two blocks of weight scales; the scales of
  // 64 groups at a time, one per lane.
  static_assert(NBN * 16 <= kFp8Block, "two blocks of weight scales at most");
  const int64_t nw0 = n0 + wn * NBN * 16, nb_last = (g.N - 1) / kFp8Block;
  const int64_t nb0 = nw0 / kFp8Block < nb_last ? nw0 / kFp8Block : nb_last;
  const int64_t nb1 = nb0 < nb_last ? nb0 + 1 : nb_last;
  const int split_j = static_cast<int>(((nb0 + 1) * kFp8Block - nw0) / 16);   // first of block 1
  float swv0 = 0.f, swv1 = 0.f;
  auto load_sw = [&](int c) {
    const bool in = c + lane < c1;
    swv0 = in ? g.sw[nb0 * C + c + lane] : 0.f;
    swv1 = in ? g.sw[nb1 * C + c + lane] : 0.f;
  };
  auto sw_of = [&](float v, int c) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), (c - c0) & 63));
  };

  v4f acc[NBM][NBN];
#pragma unroll
  for (int i = 0; i < NBM; ++i)
#pragma unroll
    for (int j = 0; j < NBN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  // A lane's 32 codes of a row are units q and q + 4 (the same K values on both
  // sides, which is all that matters). A 16-byte LDS read serves lanes 0-3,
  // 12-15 and 20-27 at once, then 4-11, 16-19 and 28-31: all 16 rows, with q
  // differing by 1 between two sets of 8, which lands them on different units.
  const int u0 = (q ^ (rl >> 1)) * 16, u1 = u0 ^ 64;
  auto frag = [&](const uint8_t (*rows)[kChunk], int block) {
    const uint8_t* p = rows[16 * block + rl];
    Frag<EXACT> f;
    f.set(*reinterpret_cast<const v4i*>(p + u0), *reinterpret_cast<const v4i*>(p + u1));
    return f;
  };
  auto scale_of = [&](int i, int c) {
    return sal[((c - c0) >> 2) & 1][(wm * NBM + i) * 16 + rl][(c - c0) & 3];
  };
  // this wave's copies but the newest n and all its LDS reads, then every wave's
  auto wait_but = [&](auto n) {
    __builtin_amdgcn_s_waitcnt(wait_copies(decltype(n)::value));
    __builtin_amdgcn_s_barrier();
  };

  // Software pipeline. The wave holds its activation blocks of a chunk and
  // streams its weight blocks, read D blocks ahead (the LDS answers later than
  // the NBM instructions of one block take). Product n = NBM * j + i goes out
  // with the four additions of product n - LAG behind it. A chunk's last D
  // blocks are read before the barrier in front of block NBN - D, so behind it
  // the stage is free: the copies of chunk c+NST go there, one every SP products
  // and on into chunk c+1 (issued together they hold up every wave at once),
  // and the blocks read ahead come from chunk c+1, whose copies the wait in
  // front of the barrier is for.
  constexpr int D = 2, LAG = NBM < 3 ? NBM : 3, TOT = NBM * NBN;
  constexpr int SP = kPieces * 2 - D * NBM <= (NBN - D) * NBM ? 2 : 1;
  constexpr int kEarly = (D * NBM + SP - 1) / SP;   // copies before the next chunk begins
  constexpr int kUniform = T::CA + T::BN / 8 / T::NW;   // copies per chunk of every wave
  static_assert(NBN % 2 == 0 && TOT % 4 == 0, "the four sets alternate across two chunks");
  static_assert(NST == 2 || NST == 4, "stages and operand sets are fixed in a run of NST chunks");
  static_assert(kPieces * SP - D * NBM <= (NBN - D) * NBM, "a chunk's copies precede its barrier");
  Frag<EXACT> fa[NBM], fw[4];
  v4f p[4];
  float sa[NBM], pend[NBM];            // activation scales; scales of products not yet added
  float sa_last[NBM], sw_last0 = 0.f, sw_last1 = 0.f;   // those of the chunk before
#pragma unroll
  for (int i = 0; i < NBM; ++i) sa[i] = sa_last[i] = pend[i] = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = v4f{0.f, 0.f, 0.f, 0.f};
  // acc += product set b, scaled, of row block i and weight block d
  auto add = [&](int i, int d, int b, float scale) {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][d][e] = __builtin_fmaf(p[b][e], scale, acc[i][d][e]);
    // the sums are made here: without this the compiler moves them past the
    // branches below and keeps every product of the chunk until then
    asm volatile("" : "+v"(acc[i][d]));
  };
  // chunk c in stage S, its first weight block in operand set P
  auto chunk = [&](int c, auto stage, auto first) {
    constexpr int S = decltype(stage)::value, P = decltype(first)::value;
    const float sw0 = sw_of(swv0, c), sw1 = sw_of(swv1, c);
#pragma unroll
    for (int j = 0; j < NBN; ++j) {
      if (j == NBN - D) {
        if (S == NST - 1 && ((c - c0) & 63) == 63) {
          load_sw(c + 1);
          __builtin_amdgcn_s_waitcnt(wait_vmem(0));
        }
        wait_but(std::integral_constant<int, (NST - 2) * kUniform>{});
        copy_scales(c + NST);
      }
      fw[(P + j + D) & 3] = j + D < NBN ? frag(st[S].w, wn * NBN + j + D)
                                        : frag(st[(S + 1) % NST].w, wn * NBN + j + D - NBN);
      float scale[NBM];
#pragma unroll
      for (int i = 0; i < NBM; ++i) scale[i] = sa[i] * (j < split_j ? sw0 : sw1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < NBM; ++i) {
        const int n = j * NBM + i;
        p[n & 3] = mfma_group(fw[(P + j) & 3], fa[i]);
        const int behind = n - (NBN - D) * NBM, cont = n + D * NBM;
        if (behind >= 0 && behind % SP == 0) copy(S, c + NST, behind / SP);
        if (cont < kPieces * SP && cont % SP == 0)
          copy((S + NST - 1) % NST, c + NST - 1, cont / SP);
        if (j + 1 == NBN) fa[i] = frag(st[(S + 1) % NST].a, wm * NBM + i);
        const int m = (n + TOT - LAG) % TOT, mi = m % NBM, mj = m / NBM;
        add(mi, mj, (n - LAG) & 3,
            n >= LAG ? pend[mi] : sa_last[mi] * (mj < split_j ? sw_last0 : sw_last1));
        pend[i] = scale[i];
        if (j + 1 == NBN) {
          sa_last[i] = sa[i];
          sa[i] = scale_of(i, c + 1);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    sw_last0 = sw0;
    sw_last1 = sw1;
  };
  load_sw(c0);
  __builtin_amdgcn_s_waitcnt(wait_vmem(0));
#pragma unroll
  for (int t = 0; t < NST; ++t) {
    copy_scales(c0 + t);
#pragma unroll
    for (int k = 0; k < (t + 1 < NST ? kPieces : kEarly); ++k) copy(t, c0 + t, k);
  }
  wait_but(std::integral_constant<int, (NST - 2) * kUniform>{});
#pragma unroll
  for (int j = 0; j < D; ++j) fw[j] = frag(st[0].w, wn * NBN + j);
#pragma unroll
  for (int i = 0; i < NBM; ++i) {
    fa[i] = frag(st[0].a, wm * NBM + i);
    sa[i] = scale_of(i, c0);
  }
  for (int c = c0; c < c1; c += NST) {
    static_for<NST>([&](auto t) {
      constexpr int S = decltype(t)::value;
      if (S == 0 || c + S < c1)
        chunk(c + S, t, std::integral_constant<int, (S * NBN) & 3>{});
    });
  }
#pragma unroll
  for (int m = TOT - LAG; m < TOT; ++m) {
    const int mi = m % NBM, mj = m / NBM;
    add(mi, mj, m & 3, sa_last[mi] * (mj < split_j ? sw_last0 : sw_last1));
  }
  wait_but(std::integral_constant<int, 0>{});   // the stages are free

  const int64_t mw = m0 + wm * NBM * 16, nw = nw0 + 4 * q;
  // A 16-bit Y goes out through the wave's share of LDS, from where a
  // lane stores 16 bytes and its neighbours the rest of the row's columns,
  // instead of 4 lanes a 32-byte piece of it, at any address (one that is not
  // aligned costs less than single elements: 8000 x 3001 x 128 28 us against 36).
  // Rows of 32 * NBN bytes, padded by 16 to spread the banks.
  constexpr int COLS = 16 * NBN, PITCH = COLS + 4;    // the fp32 rows further below
  constexpr int RB = 32 * NBN + 16, UN = 2 * NBN;     // bytes and 16-byte units of a row
  constexpr int SHARE = YT == SVDQ_F32 ? 16 * PITCH * 4 : NBM * 16 * RB;   // a wave's bytes
  static_assert(SHARE >= 16 * PITCH * 4 && sizeof(lds) >= static_cast<size_t>(T::NW) * SHARE,
                "a share holds what either way of storing puts there");
  uint8_t* share = reinterpret_cast<uint8_t*>(&lds) + wave * SHARE;
  if constexpr (YT != SVDQ_F32) {
    if (g.slices == 1 && nw0 + NBN * 16 <= g.N) {
#pragma unroll
      for (int j = 0; j < NBN; ++j) {
        const v4f b = bias4(g, nw + 16 * j);
#pragma unroll
        for (int i = 0; i < NBM; ++i)
          *reinterpret_cast<uint2*>(share + (16 * i + rl) * RB + 32 * j + 8 * q) =
              round4<YT, GELU>(acc[i][j], b);
      }
      uint16_t* y = static_cast<uint16_t*>(g.Y) + mw * g.ldy + nw0;
      const int rows = static_cast<int>(g.M - mw < NBM * 16 ? g.M - mw : NBM * 16);
#pragma unroll
      for (int t = 0; t < NBM * 16 * UN / 64; ++t) {
        const int at = 64 * t + lane, row = at / UN, col = at % UN;
        const v4i v = *reinterpret_cast<const v4i*>(share + row * RB + 16 * col);
        if (row < rows) *reinterpret_cast<v4i_any*>(y + row * g.ldy + 8 * col) = v;
      }
      return;
    }
  }
  constexpr int ES = YT == SVDQ_F32 ? 4 : 2;
  const bool vec = ((reinterpret_cast<uintptr_t>(g.Y) | (g.ldy * ES)) & (4 * ES - 1)) == 0;
  if (g.slices == 1 && vec) {
#pragma unroll
    for (int j = 0; j < NBN; ++j) {
      const v4f b = bias4(g, nw + 16 * j);
#pragma unroll
      for (int i = 0; i < NBM; ++i)
        finish4<YT, GELU>(g, acc[i][j], b, mw + 16 * i + rl, nw + 16 * j);
    }
  } else if (g.slices == 1) {
    // fp32 rows at any address, and 16-bit ones that end inside the wave's columns:
    // single elements, but in the order they lie in, 16 rows at a time through the
    // wave's share of LDS. From the accumulators each store would reach 16 rows
    // (fp32 2500 x 2501 x 2560: 57 us against 49).
    float* mem = reinterpret_cast<float*>(share);
    const int cols = static_cast<int>(g.N - nw0 < COLS ? g.N - nw0 : COLS);
#pragma unroll
    for (int i = 0; i < NBM; ++i) {
#pragma unroll
      for (int j = 0; j < NBN; ++j)
        *reinterpret_cast<v4f*>(mem + rl * PITCH + 16 * j + 4 * q) =
            acc[i][j] + bias4(g, nw + 16 * j);
#pragma unroll
      for (int t = 0; t < 4 * NBN; ++t) {
        const int at = 64 * t + lane, row = at / COLS, col = at % COLS;
        const int64_t m = mw + 16 * i + row;
        if (m < g.M && col < cols) {
          float x = mem[row * PITCH + col];
          if constexpr (GELU) x = gelu_tanh_f32(x);
          if constexpr (YT == SVDQ_F32) static_cast<float*>(g.Y)[m * g.ldy + nw0 + col] = x;
          else static_cast<uint16_t*>(g.Y)[m * g.ldy + nw0 + col] = bits16<YT>(x);
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NBM; ++i) {
      const int64_t m = mw + 16 * i + rl;
      if (m >= g.M) continue;
      float* out = g.part + (slice * g.M + m) * part_ld(g.N);
#pragma unroll
      for (int j = 0; j < NBN; ++j)
        if (nw + 16 * j < g.N) *reinterpret_cast<v4f*>(out + nw + 16 * j) = acc[i][j];
    }
  }
}

// Adds the slices' partial sums in slice order and finishes the outputs. Few
// outputs of many slices: what it takes is the loads' latency, so SLICES of them
// are in flight at once (slices past the last read its values and add nothing)
// and a workgroup is one wave, which spreads them over the most CUs.
template <int YT, bool GELU, int SLICES>
__global__ __launch_bounds__(64) void gemm_fp8_join(const GemmArgs g) {
  const int64_t per_row = part_ld(g.N) / 4;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
  if (t >= g.M * per_row) return;
  const int64_t m = t / per_row, n = (t - m * per_row) * 4;
  const v4f* p = reinterpret_cast<const v4f*>(g.part) + t;
  v4f x[SLICES];
#pragma unroll
  for (int s = 0; s < SLICES; ++s) x[s] = p[(s < g.slices ? s : 0) * g.M * per_row];
  const v4f b = bias4(g, n);
  v4f v = x[0];
#pragma unroll
  for (int s = 1; s < SLICES; ++s) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = s < g.slices ? v[e] + x[s][e] : v[e];
  }
  finish4<YT, GELU>(g, v, b, m, n);
}

template <int YT, bool GELU>
void launch_join(const GemmArgs& g, hipStream_t stream) {
  const unsigned wgs = static_cast<unsigned>((g.M * (part_ld(g.N) / 4) + 63) / 64);
  if (g.slices <= 4) hipLaunchKernelGGL((gemm_fp8_join<YT, GELU, 4>), dim3(wgs), dim3(64), 0, stream, g);
  else hipLaunchKernelGGL((gemm_fp8_join<YT, GELU, kMaxSlices>), dim3(wgs), dim3(64), 0, stream, g);
}

// ---------------------------------------------------------------------------
// Few rows

constexpr int kRowWaves = 8;

template <int YT, bool GELU>
__global__ __launch_bounds__(64 * kRowWaves) void gemm_fp8_rows(const GemmArgs g) {
  constexpr bool EXACT = YT == SVDQ_F32;
  __shared__ v4f sums[kRowWaves][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int rl = lane & 15, q = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int C = static_cast<int>(g.Kp / kChunk);
  const int64_t n = n0 + rl < g.N ? n0 + rl : g.N - 1;
  const int64_t m = rl < g.M ? rl : g.M - 1;
  const uint8_t* w = g.w + n * g.Kp + 32 * q;
  const uint8_t* a = g.a + m * g.Kp + 32 * q;
  const float* sa = g.sa + m * C;
  const float* sw = g.sw + (n0 / kFp8Block) * C;
  v4f acc = v4f{0.f, 0.f, 0.f, 0.f};
  for (int c = wave; c < C; c += kRowWaves) {
    const int64_t at = static_cast<int64_t>(c) * kChunk;
    const v4i* wp = reinterpret_cast<const v4i*>(w + at);
    const v4i* ap = reinterpret_cast<const v4i*>(a + at);
    Frag<EXACT> fw, fa;
    fw.set(wp[0], wp[1]);
    fa.set(ap[0], ap[1]);
    const float scale = sa[c] * sw[c];
    const v4f p = mfma_group(fw, fa);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(p[e], scale, acc[e]);
  }
  sums[wave][lane] = acc;
  __syncthreads();
  if (wave != 0) return;
  v4f v = sums[0][lane];
#pragma unroll
  for (int s = 1; s < kRowWaves; ++s) {
    const v4f o = sums[s][lane];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = v[e] + o[e];
  }
  finish4<YT, GELU>(g, v, bias4(g, n0 + 4 * q), rl, n0 + 4 * q);
}

constexpr int kFewRows = 16;

// The tile kernels' variants and their measured cost in microseconds: of a
// chunk when a workgroup has the chip almost to itself and when every slot is
// taken, and of a tile's start and end.
struct TileCost {
  int bm, bn, threads, per_cu;
  float alone, full, ends;
};
constexpr TileCost kTiles16[] = {{256, 256, 512, 1, 1.25f, 1.55f, 7.0f},
                                 {256, 192, 512, 1, 1.06f, 1.35f, 6.0f},
                                 {128, 128, 256, 2, 0.77f, 1.00f, 4.0f},
                                 {64, 128, 256, 3, 0.60f, 0.95f, 4.0f},
                                 {64, 64, 256, 2, 0.24f, 0.40f, 2.5f}};
constexpr TileCost kTiles32[] = {{256, 128, 512, 1, 1.60f, 2.10f, 6.0f},
                                 {64, 128, 256, 3, 0.90f, 1.65f, 4.0f},
                                 {64, 64, 256, 2, 0.50f, 0.72f, 2.5f}};

struct GemmPlan {
  int tile, slices;
};

// The variant and the split along K of least estimated time. A round of tiles
// that leaves slots empty runs its chunks the faster. A split costs a second
// launch and the partial tiles written and read, about 7 us and 2.5 TB/s.
template <int COUNT>
GemmPlan least(const TileCost (&tiles)[COUNT], int64_t M, int64_t N, int64_t Kp, bool split) {
  const int C = static_cast<int>(Kp / kChunk), cus = resident_slots() / 2;
  GemmPlan best{0, 1};
  float least = -1.f;
  for (int t = 0; t < COUNT; ++t) {
    const TileCost& k = tiles[t];
    const int64_t tiles_mn = ((M + k.bm - 1) / k.bm) * ((N + k.bn - 1) / k.bn);
    const int slots = cus * k.per_cu;
    for (int s = 1; s <= (split ? kMaxSlices : 1) && s * 2 <= C + 1; s *= 2) {
      const int64_t wgs = tiles_mn * s, rounds = wgs / slots;
      if (!grid_fits(wgs, k.threads)) break;
      const float chunks = static_cast<float>((C + s - 1) / s);
      const float part = static_cast<float>(wgs - rounds * slots) / static_cast<float>(slots);
      float us = static_cast<float>(rounds) * (chunks * k.full + k.ends);
      if (part > 0.f) us += chunks * (k.alone + part * (k.full - k.alone)) + k.ends;
      if (s > 1) us += 7.f + static_cast<float>(M) * static_cast<float>(N) * s * 8.f / 2.5e6f;
      if (least < 0.f || us < least) {
        least = us;
        best = GemmPlan{t, s};
      }
    }
  }
  return best;
}

GemmPlan gemm_plan(int64_t M, int64_t N, int64_t Kp, bool f32, bool split) {
  return f32 ? least(kTiles32, M, N, Kp, split) : least(kTiles16, M, N, Kp, split);
}

size_t split_bytes(int slices, int64_t M, int64_t N) {
  return slices > 1 ? static_cast<size_t>(slices) * M * part_ld(N) * 4 : 0;
}

template <int YT, bool GELU>
void launch_rows(const GemmArgs& g, hipStream_t stream) {
  hipLaunchKernelGGL((gemm_fp8_rows<YT, GELU>), dim3(static_cast<unsigned>((g.N + 15) / 16)),
                     dim3(64 * kRowWaves), 0, stream, g);
}

template <int WM, int WN, int NBM, int NBN, int NST, int YT, bool GELU>
void launch_tiles(const GemmArgs& g, hipStream_t stream) {
  using T = Tile<WM, WN, NBM, NBN, NST>;
  const int tiles_m = static_cast<int>((g.M + T::BM - 1) / T::BM);
  const int tiles_n = static_cast<int>((g.N + T::BN - 1) / T::BN);
  hipLaunchKernelGGL((gemm_fp8_tiles<WM, WN, NBM, NBN, NST, YT, GELU>),
                     dim3(static_cast<unsigned>(tiles_m * tiles_n * g.slices)), dim3(64 * T::NW),
                     0, stream, g, tiles_m, tiles_n);
}

template <int YT, bool GELU>
hipError_t launch_e(GemmArgs& g, size_t part_bytes, hipStream_t stream) {
  if (g.M <= kFewRows) {
    launch_rows<YT, GELU>(g, stream);
    return hipGetLastError();
  }
  GemmPlan p = gemm_plan(g.M, g.N, g.Kp, YT == SVDQ_F32, g.part != nullptr);
  if (part_bytes < split_bytes(p.slices, g.M, g.N)) p = gemm_plan(g.M, g.N, g.Kp, YT == SVDQ_F32, false);
  g.slices = p.slices;
  if constexpr (YT == SVDQ_F32) {
    // operands widened to fp16 take twice the registers
    if (p.tile == 0) launch_tiles<4, 2, 4, 4, 2, YT, GELU>(g, stream);
    else if (p.tile == 1) launch_tiles<2, 2, 2, 4, 2, YT, GELU>(g, stream);
    else launch_tiles<2, 2, 2, 2, 4, YT, GELU>(g, stream);
  } else {
    if (p.tile == 0) launch_tiles<4, 2, 4, 8, 2, YT, GELU>(g, stream);
    else if (p.tile == 1) launch_tiles<4, 2, 4, 6, 2, YT, GELU>(g, stream);
    else if (p.tile == 2) launch_tiles<2, 2, 4, 4, 2, YT, GELU>(g, stream);
    else if (p.tile == 3) launch_tiles<2, 2, 2, 4, 2, YT, GELU>(g, stream);
    else launch_tiles<2, 2, 2, 2, 4, YT, GELU>(g, stream);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || g.slices == 1) return e;
  launch_join<YT, GELU>(g, stream);
  return hipGetLastError();
}

}  // namespace

// Enough for either precision's plan: the output's type is not known here.
size_t gemm_fp8_split_bytes(int64_t M, int64_t N, int64_t Kp) {
  if (M <= kFewRows) return 0;
  const int s16 = gemm_plan(M, N, Kp, false, true).slices;
  const int s32 = gemm_plan(M, N, Kp, true, true).slices;
  return split_bytes(s16 > s32 ? s16 : s32, M, N);
}

bool gemm_fp8_fits(int64_t M, int64_t N, int y_dtype) {
  if (M <= kFewRows) return grid_fits((N + 15) / 16, 64 * kRowWaves);
  const TileCost& largest = y_dtype == SVDQ_F32 ? kTiles32[0] : kTiles16[0];
  return grid_fits(((M + largest.bm - 1) / largest.bm) * ((N + largest.bn - 1) / largest.bn),
                   largest.threads);
}

hipError_t launch_gemm_fp8(const uint8_t* a_codes, const float* a_scales, const uint8_t* w_codes,
                           const float* w_scales, const float* bias, void* Y, int y_dtype,
                           int64_t M, int64_t N, int64_t Kp, int64_t ldy, bool gelu, float* part,
                           size_t part_bytes, hipStream_t stream) {
  GemmArgs g{a_codes, w_codes, a_scales, w_scales, bias, Y, part, M, N, Kp, ldy, 1};
  if (y_dtype == SVDQ_F16)
    return gelu ? launch_e<SVDQ_F16, true>(g, part_bytes, stream)
                : launch_e<SVDQ_F16, false>(g, part_bytes, stream);
  if (y_dtype == SVDQ_BF16)
    return gelu ? launch_e<SVDQ_BF16, true>(g, part_bytes, stream)
                : launch_e<SVDQ_BF16, false>(g, part_bytes, stream);
  return gelu ? launch_e<SVDQ_F32, true>(g, part_bytes, stream)
                : launch_e<SVDQ_F32, false>(g, part_bytes, stream);
}

}  // namespace svdq
