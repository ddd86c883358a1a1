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
// instruction to the largest before they add them: 1e-5 to 5e-5 of |P_g| is
// lost (measured against fp64 on Gaussian and heavy-tailed groups; the
// accumulators across groups are fp32). That lies under an fp16 or bf16
// output's own rounding. An fp32 output takes the variant that widens the
// codes to fp16 (exact) and multiplies with v_mfma_f32_16x16x32_f16, whose
// sums are good to 1e-7, at half the matrix rate (EXACT below).
//
// Three kernels:
// - tiles: a workgroup computes BM x BN outputs, both operands copied from
//   global memory straight into LDS, one 128-byte row piece per row and chunk,
//   its 16-byte units XOR-swizzled by row % 8 so that the operand reads of 8
//   lanes cover all banks. Optionally split along K, each slice writing fp32
//   partial tiles, which a second kernel adds in slice order.
// - few rows (M <= 64): bound by reading the weights once. A workgroup owns 16
//   columns, its waves take the groups in turn, operands go straight to
//   registers, and the waves' accumulators are added through LDS in order.
#include <hip/hip_runtime.h>

#include "../../include/svdq.h"
#include "block_common.hpp"
#include "block_launch.hpp"
#include "k2_common.hpp"

namespace svdq {

namespace {

constexpr int kChunk = kFp8Block;   // K values per group and matrix instruction
constexpr int kWaitAll = 0x0070;    // vmcnt(0) expcnt(7) lgkmcnt(0)

struct GemmArgs {
  const uint8_t* a;
  const uint8_t* w;
  const float* sa;
  const float* sw;
  const float* bias;
  void* Y;
  float* part;                      // split along K: [slice][M][N] fp32
  int64_t M, N, Kp, ldy;
  int slices;
};

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

// The 4 bias values of columns n .. n+3 (0 without a bias and past the end).
__device__ __forceinline__ v4f bias4(const GemmArgs& g, int64_t n) {
  v4f b = v4f{0.f, 0.f, 0.f, 0.f};
  if (g.bias != nullptr) {
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = g.bias[n + e < g.N ? n + e : g.N - 1];
  }
  return b;
}

// The bias, the optional GELU and the one rounding to a 16-bit output.
template <int YT, bool GELU>
__device__ __forceinline__ uint2 round4(v4f v, v4f b) {
  uint32_t h[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float x = v[e] + b[e];
    if constexpr (GELU) x = gelu_tanh_f32(x);
    if constexpr (YT == SVDQ_F16) h[e] = f2h(x);
    else h[e] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
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
// Tiles

template <int WM, int WN, int NBM, int NBN>
struct Tile {
  static constexpr int BM = WM * NBM * 16, BN = WN * NBN * 16, NW = WM * WN;
  struct alignas(16) Stage {
    uint8_t a[BM][kChunk];
    uint8_t w[BN][kChunk];
  };
  struct Lds {
    Stage st[2];
    alignas(16) float sal[2][BM][4];   // activation scales of 4 groups
  };
  // one 1 KB copy instruction moves 8 rows of 128 bytes
  static constexpr int CA = BM / 8 / NW, CW = BN / 8 / NW;
  static_assert(CA * 8 * NW == BM && CW * 8 * NW == BN, "whole copy instructions per wave");
  static_assert(BM % 64 == 0 && BM / 64 <= NW, "one scale copy per wave at most");
};

template <int WM, int WN, int NBM, int NBN, int YT, bool GELU>
__global__ __launch_bounds__(64 * WM * WN) void gemm_fp8_tiles(const GemmArgs g, int tiles_m,
                                                               int tiles_n) {
  constexpr bool EXACT = YT == SVDQ_F32;
  using T = Tile<WM, WN, NBM, NBN>;
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
  const __amdgpu_buffer_rsrc_t ba = make_buffer(g.a + m0 * g.Kp, static_cast<uint32_t>(rows_a * g.Kp));
  const __amdgpu_buffer_rsrc_t bw = make_buffer(g.w + n0 * g.Kp, static_cast<uint32_t>(rows_w * g.Kp));
  const __amdgpu_buffer_rsrc_t bs = make_buffer(g.sa + m0 * C, static_cast<uint32_t>(rows_a * C * 4));
  const int r8 = lane >> 3, unit = (lane & 7) ^ r8;
  uint32_t oa[T::CA], ow[T::CW];
#pragma unroll
  for (int i = 0; i < T::CA; ++i) {
    const int r = (T::CA * wave + i) * 8 + r8;
    oa[i] = static_cast<uint32_t>((r < rows_a ? r : rows_a - 1) * g.Kp + 16 * unit);
  }
#pragma unroll
  for (int i = 0; i < T::CW; ++i) {
    const int r = (T::CW * wave + i) * 8 + r8;
    ow[i] = static_cast<uint32_t>((r < rows_w ? r : rows_w - 1) * g.Kp + 16 * unit);
  }
  const int rs = 64 * wave + lane;
  const uint32_t os = static_cast<uint32_t>((rs < rows_a ? rs : rows_a - 1) * C * 4);

  auto copy = [&](int s, int c) {
    const uint32_t at = static_cast<uint32_t>(c) * kChunk;
#pragma unroll
    for (int i = 0; i < T::CA; ++i)
      buffer_to_lds16(ba, &st[s].a[(T::CA * wave + i) * 8][0], oa[i], at);
#pragma unroll
    for (int i = 0; i < T::CW; ++i)
      buffer_to_lds16(bw, &st[s].w[(T::CW * wave + i) * 8][0], ow[i], at);
    // every fourth chunk: the scales of it and the next three
    if (((c - c0) & 3) == 0 && wave < T::BM / 64)
      buffer_to_lds16(bs, &sal[((c - c0) >> 2) & 1][64 * wave][0], os, static_cast<uint32_t>(c) * 4);
  };

  // the wave's weight scales, 64 groups at a time, one per lane
  const int64_t nb_last = (g.N - 1) / kFp8Block;
  const int64_t nb = (n0 + wn * NBN * 16) / kFp8Block;
  const float* swp = g.sw + (nb < nb_last ? nb : nb_last) * C;
  float swv = 0.f;

  v4f acc[NBM][NBN];
#pragma unroll
  for (int i = 0; i < NBM; ++i)
#pragma unroll
    for (int j = 0; j < NBN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  const int u0 = ((2 * q) ^ (lane & 7)) * 16, u1 = u0 ^ 16;
  auto frag = [&](const uint8_t (*rows)[kChunk], int block) {
    const uint8_t* p = rows[16 * block + rl];
    Frag<EXACT> f;
    f.set(*reinterpret_cast<const v4i*>(p + u0), *reinterpret_cast<const v4i*>(p + u1));
    return f;
  };

  // Software pipeline. While row block i's products go out, the products of
  // the block before it are added (two sets of partials), and block i+1 is read
  // (two sets of activation operands); each matrix instruction is followed by
  // the four additions of one issued NBN instructions earlier. The last block of
  // a chunk needs nothing more from its stage, so the barrier stands before it:
  // behind it go the copies of chunk c+2 into the stage just read, and the first
  // operands of chunk c+1, which the copies of the chunk before have brought.
  static_assert(NBM % 2 == 0, "the operand sets alternate across chunks too");
  Frag<EXACT> fw[NBN], fa[2];
  v4f p[2][NBN];
  float raw[2] = {0.f, 0.f}, sw = 0.f, sw_prev = 0.f;
#pragma unroll
  for (int j = 0; j < NBN; ++j) p[1][j] = v4f{0.f, 0.f, 0.f, 0.f};
  auto scale_of = [&](int i, int c) {
    return sal[((c - c0) >> 2) & 1][(wm * NBM + i) * 16 + rl][(c - c0) & 3];
  };
  auto wait_all = [&]() {              // this wave's copies and LDS reads, then every wave's
    __builtin_amdgcn_s_waitcnt(kWaitAll);
    __builtin_amdgcn_s_barrier();
  };
  swv = c0 + lane < c1 ? swp[c0 + lane] : 0.f;
  copy(0, c0);
  if (c0 + 1 < c1) copy(1, c0 + 1);
  wait_all();
  fa[0] = frag(st[0].a, wm * NBM);
  float next_raw = scale_of(0, c0);
#pragma unroll
  for (int j = 0; j < NBN; ++j) fw[j] = frag(st[0].w, wn * NBN + j);
  for (int c = c0; c < c1; ++c) {
    const int s = (c - c0) & 1;
    sw_prev = sw;
    sw = __builtin_bit_cast(
        float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, swv), (c - c0) & 63));
#pragma unroll
    for (int i = 0; i < NBM; ++i) {
      raw[i & 1] = next_raw;
      if (i + 1 < NBM) {
        fa[(i + 1) & 1] = frag(st[s].a, wm * NBM + i + 1);
        next_raw = scale_of(i + 1, c);
      } else {
        if (((c - c0) & 63) == 63) swv = c + 1 + lane < c1 ? swp[c + 1 + lane] : 0.f;
        wait_all();
        if (c + 2 < c1) copy(s, c + 2);
        fa[0] = frag(st[s ^ 1].a, wm * NBM);
        next_raw = scale_of(0, c + 1);
      }
      // the scale of the products added here: row block i-1 of this chunk, or
      // the last block of the chunk before
      const float scale = raw[(i + 1) & 1] * (i > 0 ? sw : sw_prev);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < NBN; ++j) {
        p[i & 1][j] = mfma_group(fw[j], fa[i & 1]);
        if (i + 1 == NBM) fw[j] = frag(st[s ^ 1].w, wn * NBN + j);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int d = (i + NBM - 1) % NBM;
          acc[d][j][e] = __builtin_fmaf(p[(i + 1) & 1][j][e], scale, acc[d][j][e]);
        }
        // the sums are made here: without this the compiler moves them past the
        // branches below and keeps every partial of the chunk until then
        asm volatile("" : "+v"(acc[(i + NBM - 1) % NBM][j]));
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  {
    const float scale = raw[1] * sw;
#pragma unroll
    for (int j = 0; j < NBN; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc[NBM - 1][j][e] = __builtin_fmaf(p[1][j][e], scale, acc[NBM - 1][j][e]);
  }

  const int64_t mw = m0 + wm * NBM * 16 + rl, nw = n0 + wn * NBN * 16 + 4 * q;
  // A 16-bit Y goes out through the wave's share of the stages, where a row's
  // 64 columns make one 128-byte line: 8 lanes store a whole line, instead of 4
  // lanes a 32-byte piece of it.
  if constexpr (YT != SVDQ_F32 && NBN == 4) {
    static_assert(sizeof(st) >= static_cast<size_t>(T::NW) * NBM * 16 * 128, "room for the tile");
    __syncthreads();                   // the last operands read ahead are not needed
    const int64_t n_wave = n0 + wn * 64;
    if (g.slices == 1 && n_wave + 64 <= g.N &&
        ((reinterpret_cast<uintptr_t>(g.Y) | (g.ldy * 2)) & 15) == 0) {
      uint8_t* mem = reinterpret_cast<uint8_t*>(&st) + wave * NBM * 16 * 128;
#pragma unroll
      for (int j = 0; j < NBN; ++j) {
        const v4f b = bias4(g, nw + 16 * j);
#pragma unroll
        for (int i = 0; i < NBM; ++i) {
          const int row = 16 * i + rl, u = (2 * j + (q >> 1)) ^ (row & 7);
          *reinterpret_cast<uint2*>(mem + row * 128 + u * 16 + (q & 1) * 8) =
              round4<YT, GELU>(acc[i][j], b);
        }
      }
      const int64_t m_wave = m0 + wm * NBM * 16;
      uint16_t* y = static_cast<uint16_t*>(g.Y) + n_wave + 8 * (lane & 7);
#pragma unroll
      for (int t = 0; t < 2 * NBM; ++t) {
        const int row = 8 * t + r8;
        const v4i v = *reinterpret_cast<const v4i*>(mem + row * 128 + (((lane & 7) ^ r8) << 4));
        if (m_wave + row < g.M) *reinterpret_cast<v4i*>(y + (m_wave + row) * g.ldy) = v;
      }
      return;
    }
  }
  if (g.slices == 1) {
#pragma unroll
    for (int j = 0; j < NBN; ++j) {
      const v4f b = bias4(g, nw + 16 * j);
#pragma unroll
      for (int i = 0; i < NBM; ++i) finish4<YT, GELU>(g, acc[i][j], b, mw + 16 * i, nw + 16 * j);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NBM; ++i) {
      if (mw + 16 * i >= g.M) continue;
      float* p = g.part + (slice * g.M + mw + 16 * i) * g.N;
#pragma unroll
      for (int j = 0; j < NBN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (nw + 16 * j + e < g.N) p[nw + 16 * j + e] = acc[i][j][e];
    }
  }
}

// Adds the slices' partial sums in slice order and finishes the outputs.
template <int YT, bool GELU>
__global__ __launch_bounds__(256) void gemm_fp8_join(const GemmArgs g) {
  const int64_t per_row = (g.N + 3) / 4;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t m = t / per_row, n = (t - m * per_row) * 4;
  if (m >= g.M) return;
  v4f v = v4f{0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < g.slices; ++s) {
    const float* p = g.part + (s * g.M + m) * g.N + n;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < g.N) v[e] = v[e] + p[e];
  }
  finish4<YT, GELU>(g, v, bias4(g, n), m, n);
}

// ---------------------------------------------------------------------------
// Few rows

constexpr int kRowWaves = 8;

template <int NBM, int YT, bool GELU>
__global__ __launch_bounds__(64 * kRowWaves) void gemm_fp8_rows(const GemmArgs g) {
  constexpr bool EXACT = YT == SVDQ_F32;
  __shared__ v4f sums[kRowWaves][NBM][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int rl = lane & 15, q = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int C = static_cast<int>(g.Kp / kChunk);
  const int64_t n = n0 + rl < g.N ? n0 + rl : g.N - 1;
  const uint8_t* w = g.w + n * g.Kp + 32 * q;
  const uint8_t* a[NBM];
  const float* sa[NBM];
#pragma unroll
  for (int i = 0; i < NBM; ++i) {
    const int64_t m = 16 * i + rl < g.M ? 16 * i + rl : g.M - 1;
    a[i] = g.a + m * g.Kp + 32 * q;
    sa[i] = g.sa + m * C;
  }
  const float* sw = g.sw + (n0 / kFp8Block) * C;
  v4f acc[NBM];
#pragma unroll
  for (int i = 0; i < NBM; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int c = wave; c < C; c += kRowWaves) {
    const int64_t at = static_cast<int64_t>(c) * kChunk;
    const v4i* wp = reinterpret_cast<const v4i*>(w + at);
    Frag<EXACT> fw;
    fw.set(wp[0], wp[1]);
#pragma unroll
    for (int i = 0; i < NBM; ++i) {
      const v4i* ap = reinterpret_cast<const v4i*>(a[i] + at);
      Frag<EXACT> fa;
      fa.set(ap[0], ap[1]);
      const float scale = sa[i][c] * sw[c];
      const v4f p = mfma_group(fw, fa);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = __builtin_fmaf(p[e], scale, acc[i][e]);
    }
  }
#pragma unroll
  for (int i = 0; i < NBM; ++i) sums[wave][i][lane] = acc[i];
  __syncthreads();
  for (int i = wave; i < NBM; i += kRowWaves) {
    v4f v = sums[0][i][lane];
#pragma unroll
    for (int s = 1; s < kRowWaves; ++s) {
      const v4f o = sums[s][i][lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = v[e] + o[e];
    }
    finish4<YT, GELU>(g, v, bias4(g, n0 + 4 * q), 16 * i + rl, n0 + 4 * q);
  }
}

constexpr int kFewRows = 64;

int split_slices(int64_t M, int64_t N, int64_t Kp) {
  if (M <= kFewRows) return 1;
  const int64_t tiles = ((M + 63) / 64) * ((N + 63) / 64);
  const int64_t C = Kp / kChunk;
  int64_t s = resident_slots() / tiles;
  if (s > C / 8) s = C / 8;
  return s < 2 ? 1 : static_cast<int>(s < 16 ? s : 16);
}

template <int YT, bool GELU>
void launch_rows(const GemmArgs& g, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((g.N + 15) / 16)), block(64 * kRowWaves);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, g); };
  if (g.M <= 16) go(gemm_fp8_rows<1, YT, GELU>);
  else if (g.M <= 32) go(gemm_fp8_rows<2, YT, GELU>);
  else go(gemm_fp8_rows<4, YT, GELU>);
}

template <int WM, int WN, int NBM, int NBN, int YT, bool GELU>
void launch_tiles(const GemmArgs& g, hipStream_t stream) {
  using T = Tile<WM, WN, NBM, NBN>;
  const int tiles_m = static_cast<int>((g.M + T::BM - 1) / T::BM);
  const int tiles_n = static_cast<int>((g.N + T::BN - 1) / T::BN);
  hipLaunchKernelGGL((gemm_fp8_tiles<WM, WN, NBM, NBN, YT, GELU>),
                     dim3(static_cast<unsigned>(tiles_m * tiles_n * g.slices)), dim3(64 * T::NW),
                     0, stream, g, tiles_m, tiles_n);
}

template <int YT, bool GELU>
hipError_t launch_e(GemmArgs& g, hipStream_t stream) {
  if (g.M <= kFewRows) {
    launch_rows<YT, GELU>(g, stream);
    return hipGetLastError();
  }
  const int64_t big = ((g.M + 255) / 256) * ((g.N + 255) / 256);
  if (big >= resident_slots() / 4) {
    g.slices = 1;
    // an fp32 output's operands take twice the registers
    launch_tiles<2, 4, YT == SVDQ_F32 ? 4 : 8, 4, YT, GELU>(g, stream);
    return hipGetLastError();
  }
  g.slices = g.part != nullptr ? split_slices(g.M, g.N, g.Kp) : 1;
  launch_tiles<2, 2, 2, 2, YT, GELU>(g, stream);
  if (g.slices > 1) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t threads = g.M * ((g.N + 3) / 4);
    hipLaunchKernelGGL((gemm_fp8_join<YT, GELU>), dim3(static_cast<unsigned>((threads + 255) / 256)),
                       dim3(256), 0, stream, g);
  }
  return hipGetLastError();
}

}  // namespace

size_t gemm_fp8_split_bytes(int64_t M, int64_t N, int64_t Kp) {
  const int s = split_slices(M, N, Kp);
  return s > 1 ? static_cast<size_t>(s) * M * N * 4 : 0;
}

hipError_t launch_gemm_fp8(const uint8_t* a_codes, const float* a_scales, const uint8_t* w_codes,
                           const float* w_scales, const float* bias, void* Y, int y_dtype,
                           int64_t M, int64_t N, int64_t Kp, int64_t ldy, bool gelu, float* part,
                           hipStream_t stream) {
  GemmArgs g{a_codes, w_codes, a_scales, w_scales, bias, Y, part, M, N, Kp, ldy, 1};
  if (y_dtype == SVDQ_F16)
    return gelu ? launch_e<SVDQ_F16, true>(g, stream) : launch_e<SVDQ_F16, false>(g, stream);
  if (y_dtype == SVDQ_BF16)
    return gelu ? launch_e<SVDQ_BF16, true>(g, stream) : launch_e<SVDQ_BF16, false>(g, stream);
  return gelu ? launch_e<SVDQ_F32, true>(g, stream) : launch_e<SVDQ_F32, false>(g, stream);
}

}  // namespace svdq
