// rotary.cu -- rotation of the heads of a step's rows by their positions.
//
//   out[r, h, pair] = pair turned by t = position[r] * frequency[pair]
//
// (rotary.cuh: the arithmetic, and why the angles hold at any position.)  Each
// value is read and written once; the angles of a row, the expensive part (some
// 30 instructions each), are made once for all of its heads, in shared memory.
//
// Bound by HBM: 8192 rows x 128 heads of 64 columns out of rows of 192, bf16, 41.1 us
// (6.5 TB/s, 0.98 of a plain copy); 4096 x 64 x 128, 21.4 us (0.94); 1031 x 64 x 128 in
// fp32, 10.0 us (1.01).  One token of 128 heads: 1.9 us, a launch and one way to
// memory and back.  rotary_pieces_kernel takes what lies on 16 bytes; the
// general kernel, which asks every unit for its edges, is about twice as long where the
// source's row stride is odd (82, 54 and 18 us).
#include <cuda_runtime.h>

#include <algorithm>

#include "dsa_internal.h"
#include "rotary.cuh"

namespace dsa {
namespace {

constexpr int kRotThreads = 128;
constexpr int kRotItems = 2;   // (row, head) items a thread of rotary_pieces_kernel

struct RotaryParams {
  const char *x;
  char *out;
  const int32_t *positions;
  const uint64_t *turns;
  int64_t items;                                      // (row, head) pairs
  int64_t x_stride, x_head, out_stride, out_head;     // bytes
  int32_t heads, width, offset, rot, layout, type, units, threads_a_head, items_a_cta;
  float amplitude;
  bool inverse, plan_rows, x_vec, out_vec, in_place;
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

// The same where every piece of 16 bytes is whole and on 16 bytes: a unit is two pieces (a rotated pair of them where
// the layout is half), a thread's pieces are on their way while the angles are made, and stay packed.  (The general
// kernel took 70, 50 and 12.7 us for the three sizes above.  Small CTAs of short threads: 256 threads with four items
// each took 44.2, 23.5, 11.0 and, for one token, 2.3 us, 512 with four 63, 33, 16 and 2.8; one item a thread 48, 24, 11.5
// and 1.7.)
template <int kType>
__global__ void __launch_bounds__(kRotThreads) rotary_pieces_kernel(const RotaryParams p) {
  constexpr int N = kType == DSA_BF16 ? 8 : 4;   // columns a piece
  extern __shared__ float2 angles[];             // [rows of the CTA's items][rot / 2]
  grid_dependency();
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * p.items_a_cta;
  const int n = static_cast<int>(min(static_cast<int64_t>(p.items_a_cta), p.items - i0));
  const int64_t row0 = i0 / p.heads;
  const uint32_t head0 = static_cast<uint32_t>(i0 - row0 * p.heads);
  const int t = threadIdx.x % p.threads_a_head, per = kRotThreads / p.threads_a_head, first = threadIdx.x / p.threads_a_head;
  // this thread's two columns (-1: none), and the pair that each one's angles start with (-1: not rotated)
  int col[2], pair[2];
  const int half = p.rot / 2, end = p.offset + p.rot;
  if (p.layout == DSA_ROTARY_HALF) {
    const int rotated = half / N;
    if (t < rotated) {
      col[0] = p.offset + t * N, col[1] = col[0] + half;
      pair[0] = pair[1] = t * N;
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c = 2 * (t - rotated) + k, before = p.offset / N;
        col[k] = c < before ? c * N : end + (c - before) * N;
        if (col[k] >= p.width) col[k] = -1;
        pair[k] = -1;
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      col[k] = (2 * t + k) * N + (p.in_place ? p.offset : 0);
      pair[k] = col[k] >= p.offset && col[k] < end ? (col[k] - p.offset) / 2 : -1;
      if (col[k] >= (p.in_place ? end : p.width)) col[k] = -1;
    }
  }
  uint4 x[kRotItems][2];
  int local[kRotItems];      // each item's row of the CTA's, -1: none
  char *to[kRotItems];
#pragma unroll
  for (int i = 0; i < kRotItems; ++i) {
    const int k = first + i * per;
    const uint32_t at = head0 + k, r = at / static_cast<uint32_t>(p.heads), h = at - r * p.heads;
    local[i] = first < per && k < n && !(p.plan_rows && p.positions[row0 + r] < 0) ? static_cast<int>(r) : -1;
    to[i] = p.out + (row0 + r) * p.out_stride + h * p.out_head;
    const char *src = p.x + (row0 + r) * p.x_stride + h * p.x_head;
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (local[i] >= 0 && col[c] >= 0) x[i][c] = *reinterpret_cast<const uint4 *>(src + col[c] * (16 / N));
  }
  const int rows = static_cast<int>((head0 + n - 1) / static_cast<uint32_t>(p.heads)) + 1;
  for (int k = threadIdx.x; k < rows * half; k += kRotThreads) {
    const int r = k / half, i = k - r * half;
    float2 w = rotary_angle(p.positions[row0 + r], p.turns[i], p.amplitude);
    if (p.inverse) w.y = -w.y;
    angles[k] = w;
  }
  __syncthreads();
  auto unpack = [](float (&v)[N], const uint4 &u) {
    if constexpr (kType == DSA_BF16) unpack8(v, u);
    else v[0] = __uint_as_float(u.x), v[1] = __uint_as_float(u.y), v[2] = __uint_as_float(u.z), v[3] = __uint_as_float(u.w);
  };
  auto pack = [](const float (&v)[N]) {
    if constexpr (kType == DSA_BF16)
      return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    else return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  };
#pragma unroll
  for (int i = 0; i < kRotItems; ++i) {
    if (local[i] < 0) continue;
    const float2 *cs = angles + local[i] * half;
    float a[N], b[N];
    unpack(a, x[i][0]);
    unpack(b, x[i][1]);
    if (p.layout == DSA_ROTARY_HALF) {
      if (pair[0] >= 0) rotate_half(a, b, cs + pair[0]);
    } else {
      if (pair[0] >= 0) rotate_interleaved(a, cs + pair[0]);
      if (pair[1] >= 0) rotate_interleaved(b, cs + pair[1]);
    }
    if (col[0] >= 0) *reinterpret_cast<uint4 *>(to[i] + col[0] * (16 / N)) = pack(a);
    if (col[1] >= 0) *reinterpret_cast<uint4 *>(to[i] + col[1] * (16 / N)) = pack(b);
  }
}

// How a call's work is cut: threads an item, items a CTA, and the rows of which a CTA may hold angles.
struct Cut {
  bool pieces;      // rotary_pieces_kernel
  int units, threads, items, rows, pitch;
  Cut(const dsa_rotary *table, const dsa_rotate_t &g, const void *x, const void *out) {
    const int size = g.type == DSA_BF16 ? 2 : 4, rot = table->rot;
    const bool in_place = x == out, half = g.layout == DSA_ROTARY_HALF;
    auto on16 = [&](const void *q, int64_t stride, int64_t head) {
      return reinterpret_cast<uintptr_t>(q) % 16 == 0 && stride * size % 16 == 0 && head * size % 16 == 0;
    };
    pieces = rotary_whole(g.offset, rot, g.layout) && g.width % 8 == 0 && on16(x, g.x_stride, g.x_head) &&
             on16(out, g.out_stride, g.out_head);
    // in place the columns beside the rotated ones are there already
    if (pieces) {
      const int n = 16 / size, beside = in_place ? 0 : (g.width - rot) / n;
      units = half ? rot / 2 / n + (beside + 1) / 2 : (rot / n + beside + 1) / 2;
      pieces = units <= kRotThreads;
    }
    if (!pieces) units = rotary_units(rot, g.layout) + (in_place ? 0 : rotary_copies(g.width, g.offset, rot));
    threads = std::min(units, kRotThreads);
    pitch = pieces ? rot / 2 : rotary_pairs(rot);
    // kRotItems items a thread, in the general kernel four (two of twice eight columns), while the rows' angles fit 48 KB
    const int64_t most = 48 * 1024 / (pitch * sizeof(float2));
    items = (pieces ? kRotItems : half ? 2 : 4) * (kRotThreads / threads);
    items = static_cast<int>(std::min<int64_t>(items, g.heads == 1 ? most : (most - 2) * g.heads + 1));
    rows = g.heads == 1 ? items : std::min(items, (items - 1) / g.heads + 2);
  }
};

}  // namespace

int64_t rotary_ctas(const dsa_rotary *table, const dsa_rotate_t &g, const void *x, const void *out) {
  const Cut cut(table, g, x, out);
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
  p.amplitude = table->amplitude, p.inverse = g.inverse != 0, p.plan_rows = plan_rows, p.in_place = x == out;
  const bool whole = rotary_whole(g.offset, p.rot, g.layout);
  auto vec = [&](const void *q, int64_t stride, int64_t head) {
    return whole && reinterpret_cast<uintptr_t>(q) % 16 == 0 && stride % 16 == 0 && head % 16 == 0;
  };
  p.x_vec = vec(x, p.x_stride, p.x_head), p.out_vec = vec(out, p.out_stride, p.out_head);
  const Cut cut(table, g, x, out);
  p.units = cut.units, p.threads_a_head = cut.threads, p.items_a_cta = cut.items;
  const int smem = cut.rows * cut.pitch * static_cast<int>(sizeof(float2));
  const dim3 grid(static_cast<unsigned>((p.items + cut.items - 1) / cut.items));
  *launches += 1;
  if (!cut.pieces) return launch_overlapped(rotary_kernel, grid, kRotThreads, smem, 1, s, p);
  return g.type == DSA_BF16 ? launch_overlapped(rotary_pieces_kernel<DSA_BF16>, grid, kRotThreads, smem, 1, s, p)
                            : launch_overlapped(rotary_pieces_kernel<DSA_FP32>, grid, kRotThreads, smem, 1, s, p);
}

}  // namespace dsa
