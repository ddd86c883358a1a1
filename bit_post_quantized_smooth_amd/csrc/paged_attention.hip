// Attention over a paged cache: the launches, and the kernel that joins the parts of
// tiles that were split along their keys (gfx950).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../../include/svdq.h"
#include "block_common.hpp"
#include "device_launch.hpp"
#include "paged_attention.hpp"
#include "paged_line.hpp"

namespace svdq {

namespace {

constexpr float kNegInf = -__builtin_inff();

// Joins the parts of the tile that border w of the shares is the first to cut: 8 rows a
// workgroup, 32 lanes a row, 4 channels each, the parts in order.
constexpr int kJoinRows = 8;

template <class T>
__global__ __launch_bounds__(32 * kJoinRows) void paged_attention_join(const PagedArgs g, int wgs) {
  const int64_t per_head = head_work(g), work = per_head * g.Hkv;
  const int w = static_cast<int>(blockIdx.x) + 1;
  const int64_t each = share(g, work, wgs), c = w * each;
  if (c >= work) return;
  const Place p = place(g, per_head, c);
  const Sequence s = sequence(g, p.b);
  const int64_t cost = s.cost(p.r);
  if (left_whole(g, cost) || p.start >= c || p.start < c - each) return;
  const int tile_rows = s.few ? kFew : kMany;
  const int in_tile = static_cast<int>(blockIdx.y) * kJoinRows + static_cast<int>(threadIdx.x) / 32;
  const int r = p.r * tile_rows + in_tile, ch = 4 * (static_cast<int>(threadIdx.x) % 32);
  if (in_tile >= tile_rows || r >= s.n * g.G || ch >= g.D) return;
  const int parts = static_cast<int>((p.start + cost - 1) / each) - w + 2;    // from workgroup w - 1 on
  auto row_of = [&](int i) {
    return (static_cast<int64_t>(2 * (w - 1 + i)) + (i == 0 ? 1 : 0)) * g.part_rows + in_tile;
  };
  float top = kNegInf;
  for (int i = 0; i < parts; ++i) top = fmaxf(top, g.part_ml[2 * row_of(i)]);
  // 2^10 parts at most: the sum of their finite outputs is finite
  const float base = top == kNegInf ? 0.f : top + 10.f;
  v4f o = v4f{0.f, 0.f, 0.f, 0.f};
  float n = 0.f;
  for (int i = 0; i < parts; ++i) {
    const int64_t row = row_of(i);
    const float l = g.part_ml[2 * row + 1];
    if (l == 0.f) continue;              // nothing was written for it
    const float f = __builtin_amdgcn_exp2f(g.part_ml[2 * row] - base);
    n = __builtin_fmaf(l, f, n);
    const v4f x = *reinterpret_cast<const v4f*>(g.part_o + row * g.D + ch);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(x[e], f, o[e]);
  }
  const float inv = n == 0.f ? 0.f : 1.0f / n;
  const float vs = g.pages.v_scales != nullptr ? g.pages.v_scales[p.hk] : 1.f;
  T* op = static_cast<T*>(g.out) + (s.first + static_cast<int64_t>(r / g.G)) * g.o_t +
          (p.hk * g.G + r % g.G) * g.o_h + ch;
  typedef T vec4 __attribute__((ext_vector_type(4)));
  vec4 y;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = static_cast<T>(o[e] * inv * vs);
  *reinterpret_cast<vec4*>(op) = y;
}

// Workgroups: as many as are resident, fewer where the least share covers all the work
// that these sizes can hold.
int workgroups(int64_t T, int64_t B, int64_t capacity, int64_t Hkv, int64_t G) {
  const double tiles = static_cast<double>(T * G) / kMany + static_cast<double>(std::min(B, T));
  const double work = tiles * static_cast<double>(Hkv) * (kStart + 2.0 * static_cast<double>(capacity) + 2 * kMany);
  return static_cast<int>(std::min(static_cast<double>(resident_slots()), work / kLeast + 1));
}

template <class T>
hipError_t launch_t(const PagedArgs& g, hipStream_t stream) {
  const int wgs = workgroups(g.T, g.B, g.capacity, g.Hkv, g.G);
  g.D > 64 ? launch_paged_tiles<T, 128>(g, static_cast<unsigned>(wgs), stream)
           : launch_paged_tiles<T, 64>(g, static_cast<unsigned>(wgs), stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || g.part_rows == 0 || wgs < 2) return e;
  hipLaunchKernelGGL(paged_attention_join<T>, dim3(static_cast<unsigned>(wgs - 1), static_cast<unsigned>(g.part_rows / kJoinRows)),
                     dim3(32 * kJoinRows), 0, stream, g, wgs);
  return hipGetLastError();
}

}  // namespace

PartBytes paged_attention_parts(int64_t T, int64_t B, int64_t capacity, int64_t Hkv, int64_t G,
                                int64_t D) {
  // no tile is cut if the longest one is left whole
  if (T == 0 || B == 0 || kStart + (T * G <= kFew ? 1 : 2) * capacity <= kWhole) return {0, 0};
  const int wgs = workgroups(T, B, capacity, Hkv, G);
  if (wgs < 2) return {0, 0};
  const size_t rows = static_cast<size_t>(2 * wgs) * (T * G <= kFew ? kFew : kMany);
  return {(rows * 8 + 255) / 256 * 256, rows * static_cast<size_t>(D) * 4};
}

hipError_t launch_paged_attention(PagedArgs g, int dtype, hipStream_t stream) {
  return dtype == SVDQ_F16 ? launch_t<_Float16>(g, stream) : launch_t<__bf16>(g, stream);
}

}  // namespace svdq
