// rotary.cu -- rotation of the heads of a step's rows by their positions.
//
//   out[r, h, pair] = pair turned by t = position[r] * frequency[pair]
//
// (rotary.cuh: the arithmetic, and why the angles hold at any position.)  Each
// value is read and written once; the angles of a row, the expensive part (some
// 60 instructions each), are made once for all of its heads, in shared memory.
#include <cuda_runtime.h>

#include <algorithm>

#include "dsa_internal.h"
#include "rotary.cuh"

namespace dsa {
namespace {

constexpr int kRotThreads = 256;

struct RotaryParams {
  const char *x;
  char *out;
  const int32_t *positions;
  const uint64_t *turns;
  int64_t items;                                      // (row, head) pairs
  int64_t x_stride, x_head, out_stride, out_head;     // bytes
  int32_t heads, width, offset, rot, layout, type, units, threads_a_head, items_a_cta;
  float amplitude;
  bool inverse, plan_rows, x_vec, out_vec;
};

// A CTA takes items_a_cta neighbouring (row, head) items; threads_a_head threads
// an item, each with the same units of every item that it meets.
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotaryParams p) {
  extern __shared__ float2 angles[];   // [rows of the CTA's items][rotary_pairs(rot)]
  grid_dependency();
  const int pairs = p.rot / 2, pitch = rotary_pairs(p.rot);
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * p.items_a_cta;
  const int n = static_cast<int>(min(static_cast<int64_t>(p.items_a_cta), p.items - i0));
  const int64_t row0 = i0 / p.heads;
  const uint32_t head0 = static_cast<uint32_t>(i0 - row0 * p.heads);
  const int rows = static_cast<int>((head0 + n - 1) / static_cast<uint32_t>(p.heads)) + 1;
  for (int k = threadIdx.x; k < rows * pairs; k += kRotThreads) {
    const int r = k / pairs, i = k - r * pairs;
    float2 w = rotary_angle(p.positions[row0 + r], p.turns[i], p.amplitude);
    if (p.inverse) w.y = -w.y;
    angles[r * pitch + i] = w;
  }
  __syncthreads();
  const int t = threadIdx.x % p.threads_a_head, per = kRotThreads / p.threads_a_head;
  const int first = threadIdx.x / p.threads_a_head;
  if (first >= per) return;   // (threads left over)
#pragma unroll 4
  for (int k = first; k < n; k += per) {
    const uint32_t at = head0 + k, r = at / static_cast<uint32_t>(p.heads), h = at - r * p.heads;
    const int64_t row = row0 + r;
    if (p.plan_rows && p.positions[row] < 0) continue;   // a capturable plan's padding
    const char *x = p.x + row * p.x_stride + h * p.x_head;
    char *out = p.out + row * p.out_stride + h * p.out_head;
    for (int u = t; u < p.units; u += p.threads_a_head)
      rotary_unit(u, p.rot, p.layout, p.offset, p.width, angles + r * pitch, x, p.type, p.x_vec, out, p.type, p.out_vec);
  }
}

// How a call's work is cut: threads an item, items a CTA, and the rows of which a CTA may hold angles.
struct Cut {
  int units, threads, items, rows;
  Cut(const dsa_rotary *table, const dsa_rotate_t &g, bool in_place) {
    // in place the columns beside the rotated ones are there already
    units = rotary_units(table->rot, g.layout) + (in_place ? 0 : rotary_copies(g.width, g.offset, table->rot));
    threads = std::min(units, kRotThreads);
    // four items a thread (twice eight columns a unit: two), while the rows' angles fit 48 KB
    const int64_t most = 48 * 1024 / (rotary_pairs(table->rot) * sizeof(float2));
    items = (g.layout == DSA_ROTARY_HALF ? 2 : 4) * (kRotThreads / threads);
    items = static_cast<int>(std::min<int64_t>(items, g.heads == 1 ? most : (most - 2) * g.heads + 1));
    rows = g.heads == 1 ? items : std::min(items, (items - 1) / g.heads + 2);
  }
};

}  // namespace

int64_t rotary_ctas(const dsa_rotary *table, const dsa_rotate_t &g, bool in_place) {
  const Cut cut(table, g, in_place);
  return (g.rows * g.heads + cut.items - 1) / cut.items;
}

cudaError_t launch_rotary(const dsa_rotary *table, const dsa_rotate_t &g, const void *x, const int32_t *positions,
                          bool plan_rows, void *out, cudaStream_t s, int32_t *launches) {
  const int size = g.type == DSA_BF16 ? 2 : 4;
  RotaryParams p{};
  p.x = static_cast<const char *>(x), p.out = static_cast<char *>(out);
  p.positions = positions, p.turns = table->turns;
  p.items = g.rows * g.heads;
  p.x_stride = g.x_stride * size, p.x_head = g.x_head * size, p.out_stride = g.out_stride * size, p.out_head = g.out_head * size;
  p.heads = g.heads, p.width = g.width, p.offset = g.offset, p.rot = table->rot, p.layout = g.layout, p.type = g.type;
  p.amplitude = table->amplitude, p.inverse = g.inverse != 0, p.plan_rows = plan_rows;
  const bool whole = rotary_whole(g.offset, p.rot, g.layout);
  auto vec = [&](const void *q, int64_t stride, int64_t head) {
    return whole && reinterpret_cast<uintptr_t>(q) % 16 == 0 && stride % 16 == 0 && head % 16 == 0;
  };
  p.x_vec = vec(x, p.x_stride, p.x_head), p.out_vec = vec(out, p.out_stride, p.out_head);
  const Cut cut(table, g, x == out);
  p.units = cut.units, p.threads_a_head = cut.threads, p.items_a_cta = cut.items;
  const int smem = cut.rows * rotary_pairs(p.rot) * static_cast<int>(sizeof(float2));
  *launches += 1;
  return launch_overlapped(rotary_kernel, dim3(static_cast<unsigned>(rotary_ctas(table, g, x == out))), kRotThreads, smem, 1, s, p);
}

}  // namespace dsa
