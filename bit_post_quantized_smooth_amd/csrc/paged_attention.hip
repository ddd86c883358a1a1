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

// Joins the parts of a tile that was cut. 32 lanes hold a row, 4 channels each, and a
// thread ROWS rows; the parts in order, AT_ONCE of each row on their way together, in one
// pass with the running maximum.
constexpr int kJoinRows = 8;             // rows of a workgroup at a time

template <class T, int ROWS, int AT_ONCE>
__device__ __forceinline__ void join(const PagedArgs& g, const Cut& cut, int first_slot, int first_row, int step) {
  const int ch = 4 * (static_cast<int>(threadIdx.x) % 32);
  v4f o[ROWS];
  float top[ROWS], n[ROWS];
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    o[k] = v4f{0.f, 0.f, 0.f, 0.f};
    top[k] = kNegInf;
    n[k] = 0.f;
  }
  for (int i0 = 0; i0 < cut.parts; i0 += AT_ONCE) {
    v4f x[ROWS][AT_ONCE];
    float m[ROWS][AT_ONCE], l[ROWS][AT_ONCE];
#pragma unroll
    for (int k = 0; k < ROWS; ++k)
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) {
        // behind the last part and row the last ones again
        const int part = min(i0 + i, cut.parts - 1), in_tile = min(first_row + k * step, cut.rows - 1);
        const int64_t row = static_cast<int64_t>(first_slot + 2 * part - (part == 0 ? 0 : 1)) * g.part_rows + in_tile;
        m[k][i] = g.part_ml[2 * row];
        l[k][i] = i0 + i < cut.parts ? g.part_ml[2 * row + 1] : 0.f;
        x[k][i] = *reinterpret_cast<const v4f*>(g.part_o + row * g.D + (ch < g.D ? ch : 0));
      }
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      float new_top = top[k];
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) new_top = l[k][i] != 0.f ? fmaxf(new_top, m[k][i]) : new_top;
      // 2^10 parts at most: with 2^-10 the sum of their finite outputs is finite
      const float base = new_top == kNegInf ? 0.f : new_top + 10.f;
      const float alpha = n[k] == 0.f ? 0.f : __builtin_amdgcn_exp2f(top[k] - new_top);
      n[k] *= alpha;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[k][e] *= alpha;
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) {
        if (l[k][i] == 0.f) continue;    // nothing was written for it
        const float f = __builtin_amdgcn_exp2f(m[k][i] - base);
        n[k] = __builtin_fmaf(l[k][i], f, n[k]);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[k][e] = __builtin_fmaf(x[k][i][e], f, o[k][e]);
      }
      top[k] = new_top;
    }
  }
  const float vs = g.pages.v_scales != nullptr ? g.pages.v_scales[cut.hk] : 1.f;
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    const int in_tile = first_row + k * step;
    if (in_tile >= cut.rows || ch >= g.D) continue;
    const float inv = n[k] == 0.f ? 0.f : 1.0f / n[k];
    const int r = cut.row + in_tile;
    T* op = static_cast<T*>(g.out) + (cut.first + static_cast<int64_t>(r / g.G)) * g.o_t +
            (cut.hk * g.G + r % g.G) * g.o_h + ch;
    typedef T vec4 __attribute__((ext_vector_type(4)));
    vec4 y;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = static_cast<T>(o[k][e] * inv * vs);
    *reinterpret_cast<vec4*>(op) = y;
  }
}

template <class T>
__global__ __launch_bounds__(32 * kJoinRows) void paged_attention_join(const PagedArgs g) {
  fetch_arguments(g);
  const int w = static_cast<int>(blockIdx.x);
  const Cut cut = g.cuts[w];
  if (cut.parts == 0) return;
  const int row = static_cast<int>(blockIdx.y) * kJoinRows + static_cast<int>(threadIdx.x) / 32;
  const int step = static_cast<int>(gridDim.y) * kJoinRows;
  if (cut.rows <= step) {
    if (row < cut.rows) join<T, 1, 8>(g, cut, 2 * w + 1, row, step);
  } else {
    for (int first = row; first < cut.rows; first += 4 * step) join<T, 4, 2>(g, cut, 2 * w + 1, first, step);
  }
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
  hipLaunchKernelGGL(paged_attention_join<T>, dim3(static_cast<unsigned>(wgs - 1), g.part_rows > kFew ? 4 : 1),
                     dim3(32 * kJoinRows), 0, stream, g);
  return hipGetLastError();
}

}  // namespace

PartBytes paged_attention_parts(int64_t T, int64_t B, int64_t capacity, int64_t Hkv, int64_t G,
                                int64_t D) {
  // no tile is cut if the longest one is left whole
  if (T == 0 || B == 0 ||
      (T * G <= kFew ? kStart + capacity <= kWholeFew : kStart + 2 * capacity <= kWholeMany))
    return {0, 0, 0};
  const int wgs = workgroups(T, B, capacity, Hkv, G);
  if (wgs < 2) return {0, 0, 0};
  const size_t rows = static_cast<size_t>(2 * wgs) * (T * G <= kFew ? kFew : kMany);
  return {static_cast<size_t>(wgs) * sizeof(Cut), rows * 8, rows * static_cast<size_t>(D) * 4};
}

hipError_t launch_paged_attention(PagedArgs g, int dtype, hipStream_t stream) {
  return dtype == SVDQ_F16 ? launch_t<_Float16>(g, stream) : launch_t<__bf16>(g, stream);
}

}  // namespace svdq
