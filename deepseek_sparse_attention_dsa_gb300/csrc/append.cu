// append.cu -- a step's rows into the paged caches, rotated by their positions
// on the way: latent rows [c | rotated k_pe] and index keys (bf16, or quantised
// to the 656- and 132-byte rows), or the keys and values of a GQA cache.
//
// Each value is read and written once.  Values to be quantised stay in fp32
// between rotation and code, so that they are rounded once.  append_runs_kernel takes
// sources and caches on 16 bytes in whole runs of 16 columns; append_kernel, a warp
// for each part of a row (its latent, its index key, its keys, its values), any
// others: with sources an element off 16 bytes 128 rows 3.9 us in place of 2.5, 8192
// rows into 8 bits 16.8 in place of 8.5, 8197 rows of keys and values from memory 21.0
// in place of 10.0 (fp32: 21.9 and 15.0).
#include <cuda_runtime.h>

#include <algorithm>

#include "dsa_internal.h"
#include "ptx.cuh"
#include "rotary.cuh"

namespace dsa {
namespace {

constexpr int kAppendWarps = 8;

enum Part { kPartLatent, kPartKey, kPartK, kPartV };

struct AppendParams {
  const int32_t *row_pos, *row_page_off, *row_npages, *row_page_start, *pages;
  const uint64_t *turns;
  int *err;
  int32_t T, P, num_pages, rot, parts, part[3];
  int32_t groups, side, deep;   // append_runs_kernel
  bool padded;                  // a capturable plan's rows
  float amplitude;
  // latents
  const char *c, *k_pe;
  char *latent;
  int64_t c_stride, k_pe_stride;   // bytes
  int32_t L, R, c_type, k_pe_type, layout, latent_row, rope_at;   // bytes of a cached row, and of its rope's start
  bool latent_fp8, c_vec, k_pe_vec, latent_vec, rope_vec;
  // index keys
  const char *keys;
  char *index;
  int64_t keys_stride;
  int32_t D, key_type, key_layout, key_offset;
  bool index_fp8, keys_vec, index_vec;
  // keys and values
  const char *k, *v;
  char *kv;
  int64_t k_stride, k_head, v_stride, v_head;
  int32_t heads, dim, kv_type, kv_layout, kv_offset;
  bool k_vec, v_vec, kv_vec;
};

// Eight columns from `col` on of a row of `width`, rounded to bf16.
__device__ __forceinline__ void copy8(const char *src, int type, bool src_vec, char *dst, bool dst_vec, int col, int width) {
  float v[8];
  load8(v, src, type, col, width, src_vec);
  store8(dst, DSA_BF16, col, width, dst_vec, v);
}

__global__ void __launch_bounds__(kAppendWarps * 32) append_kernel(const AppendParams p) {
  extern __shared__ float shared[];   // a warp: [rotary_pairs(rot)] angles, then [D] values of a key to be quantised
  grid_dependency();
  const int warp = threadIdx.x / 32, lane = lane_id();
  const int64_t task = static_cast<int64_t>(blockIdx.x) * kAppendWarps + warp;
  const int64_t row = task / p.parts;
  if (row >= p.T) return;
  const int part = p.part[task - row * p.parts];
  const int32_t pos = p.row_pos[row];
  if (pos < 0) return;   // padding of a capturable plan
  const int64_t slot = static_cast<int64_t>(p.row_page_start[row]) + pos, pi = slot / p.P;
  int page = -1;
  if (pi < p.row_npages[row]) page = p.pages[p.row_page_off[row] + pi];
  if (page < 0 || page >= p.num_pages) {
    if (lane == 0) atomicOr(p.err, kErrBounds);
    return;
  }
  const int in_page = static_cast<int>(slot - pi * p.P);
  const int64_t at = static_cast<int64_t>(page) * p.P + in_page;

  const int pitch = p.rot ? rotary_pairs(p.rot) : 0;
  float2 *cs = reinterpret_cast<float2 *>(shared) + warp * pitch;
  if (p.rot && part != kPartV) {
    for (int i = lane; i < p.rot / 2; i += 32) cs[i] = rotary_angle(pos, p.turns[i], p.amplitude);
    __syncwarp();
  }

  if (part == kPartLatent) {
    const char *c = p.c + row * p.c_stride, *k_pe = p.k_pe + row * p.k_pe_stride;
    char *out = p.latent + at * p.latent_row;
    if (p.latent_fp8) {
      for (int c0 = 0; c0 < p.L; c0 += 256) {   // (the whole warp: a group's maximum is over 16 lanes)
        const int col = c0 + lane * 8;
        float v[8];
        load8(v, c, p.c_type, col, p.L, p.c_vec);
        uint32_t m = amax_bits8(v);
#pragma unroll
        for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const GroupScale g(m);
        store_codes8(reinterpret_cast<uint8_t *>(out), col, p.L, p.latent_vec, codes8(v, g));
        if ((lane & 15) == 0 && col < p.L) reinterpret_cast<float *>(out + p.L)[col / 128] = g.scale;
      }
    } else {
      for (int col = lane * 8; col < p.L; col += 256) copy8(c, p.c_type, p.c_vec, out, p.latent_vec, col, p.L);
    }
    char *rope = out + p.rope_at;
    // (a table's rot is R, or R is 0 and it is the key's; without one the columns are copied)
    const int n = p.R == 0 ? 0 : p.rot ? rotary_units(p.rot, p.layout) : (p.R + 7) / 8;
    for (int u = lane; u < n; u += 32)
      rotary_unit(u, p.rot, p.layout, 0, p.R, cs, k_pe, p.k_pe_type, p.k_pe_vec, rope, DSA_BF16, p.rope_vec);
  } else if (part == kPartKey) {
    const char *key = p.keys + row * p.keys_stride;
    const int n = (p.rot ? rotary_units(p.rot, p.key_layout) : 0) + rotary_copies(p.D, p.key_offset, p.rot);
    if (p.index_fp8) {
      float *v = shared + kAppendWarps * pitch * 2 + warp * p.D;
      for (int u = lane; u < n; u += 32)
        rotary_unit(u, p.rot, p.key_layout, p.key_offset, p.D, cs, key, p.key_type, p.keys_vec, v, DSA_FP32, false);
      __syncwarp();
      // D is 128: one group, four columns a lane
      float x[4];
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(x[i] = v[lane * 4 + i]) & 0x7FFFFFFFu);
      const GroupScale g(__reduce_max_sync(0xffffffffu, m));
      char *base = p.index + static_cast<int64_t>(page) * p.P * (128 + 4);
      const uint32_t codes = g.scale < 0x1p-80f
                                 ? e4m3x4(x[0] / g.scale, x[1] / g.scale, x[2] / g.scale, x[3] / g.scale)
                                 : e4m3x4(g.quotient(x[0]), g.quotient(x[1]), g.quotient(x[2]), g.quotient(x[3]));
      reinterpret_cast<uint32_t *>(base + in_page * 128)[lane] = codes;
      if (lane == 0) *reinterpret_cast<float *>(base + static_cast<int64_t>(p.P) * 128 + in_page * 4) = g.scale;
    } else {
      char *out = p.index + at * p.D * 2;
      for (int u = lane; u < n; u += 32)
        rotary_unit(u, p.rot, p.key_layout, p.key_offset, p.D, cs, key, p.key_type, p.keys_vec, out, DSA_BF16, p.index_vec);
    }
  } else {
    const bool is_k = part == kPartK;
    char *out = p.kv + at * (4ll * p.heads * p.dim) + (is_k ? 0 : 2ll * p.heads * p.dim);
    const int rot = is_k ? p.rot : 0;
    const int n = (rot ? rotary_units(rot, p.kv_layout) : 0) + rotary_copies(p.dim, rot ? p.kv_offset : 0, rot);
    for (int i = lane; i < n * p.heads; i += 32) {
      const int h = i / n, u = i - h * n;
      const char *src = is_k ? p.k + row * p.k_stride + h * p.k_head : p.v + row * p.v_stride + h * p.v_head;
      rotary_unit(u, rot, p.kv_layout, rot ? p.kv_offset : 0, p.dim, cs, src, p.kv_type, is_k ? p.k_vec : p.v_vec,
                  out + 2ll * h * p.dim, DSA_BF16, p.kv_vec);
    }
  }
}

// The same where every row consists of whole runs of 16 columns on 16 bytes, in groups of eight lanes: 128 columns of a
// latent, its rope, an index key, a head of K or V.  A thread has one run of each of several rows: they are on their
// way, packed, while positions and pages are looked up and angles made, once for all of a row's groups.  The other
// column of a pair comes from a neighbouring lane, a group's maximum from its eight.  p.groups a row, p.side rows beside one
// another in a CTA and p.deep of them in a thread; neighbouring groups are the same part of neighbouring rows, so that a
// warp copies, turns or quantises and seldom does several of these (by rows: 9.3 us in place of 8.5).  kWide: some source
// is fp32.
// Bound by its instructions and by the way from one look-up to the next (launch, position, page, row: 2.5 us for 128 rows):
// 8192 rows into 8 bits take 8.5 us, 2.1 TB/s, with the sources in L2; 8197 rows of keys and values, 4 heads of 128 each,
// 8.6 us, 3.9 TB/s, and 10.0 from memory.  (With 8 columns a lane, twice the threads, 8192 rows took 2.4 us more; with 80
// registers and without the few spills that 64 cost, 8197 rows 0.7 to 1.4 us more.  A step of few rows has a kernel of
// its own, DEEP 1: 2.5 us for 128 rows in place of 2.9.)
constexpr int kAppendThreads = 256;
constexpr int kAppendRegisters = 64;   // a thread's, by the launch bounds
constexpr int kLaneCols = 16, kGroupLanes = 128 / kLaneCols;
template <bool kWide>
constexpr int kAppendDeep = kWide ? 2 : 4;
// Place of a row's angle q: lanes that read 8 or 16 of them from their own on meet no common bank.
__host__ __device__ constexpr int padded(int q) { return q + q / 16; }
constexpr int kAppendRows = kAppendThreads / kGroupLanes * 4;   // the most that a CTA has (one group a row)

template <bool kWide, int DEEP>
__global__ void __launch_bounds__(kAppendThreads, 4) append_runs_kernel(const AppendParams p) {
  constexpr int N = kLaneCols, W = kWide ? 4 : 2;
  extern __shared__ float2 angles[];   // [rows of the CTA][padded(rot / 2)]
  __shared__ int2 where[kAppendRows];  // of the CTA's rows: page (-1: nothing to write), slot in it
  grid_dependency();
  const int group = threadIdx.x / kGroupLanes, lane = threadIdx.x % kGroupLanes, local = group % p.side, rows = p.side * p.deep;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows;
  int gi = group / p.side, part = kPartLatent, base = 0;
  // the group's part of the row: latents (kv_lora_rank / 128 groups and the rope's), key, heads of K, heads of V
  int width = 0, type = DSA_BF16, rot = 0, layout = 0, offset = 0;
  int64_t stride = 0;
  const char *src = nullptr;
  bool rope = false;
  const int latent_groups = p.c ? (p.L + 127) / 128 + (p.R > 0 ? 1 : 0) : 0, key_groups = p.keys ? 1 : 0;
  if (gi < latent_groups) {
    rope = p.R > 0 && gi == latent_groups - 1;
    if (rope) src = p.k_pe, stride = p.k_pe_stride, width = p.R, type = p.k_pe_type, rot = p.rot, layout = p.layout;
    else src = p.c, stride = p.c_stride, width = p.L, type = p.c_type, base = gi * 128;
  } else if ((gi -= latent_groups) < key_groups) {
    part = kPartKey;
    src = p.keys, stride = p.keys_stride, width = p.D, type = p.key_type, rot = p.rot, layout = p.key_layout, offset = p.key_offset;
  } else {
    gi -= key_groups;
    part = gi < p.heads ? kPartK : kPartV;
    if (part == kPartV) gi -= p.heads;
    src = part == kPartK ? p.k + gi * p.k_head : p.v + gi * p.v_head;
    stride = part == kPartK ? p.k_stride : p.v_stride, width = p.dim, type = p.kv_type;
    if (part == kPartK) rot = p.rot, layout = p.kv_layout, offset = p.kv_offset;
  }
  const int col = base + lane * N;
  const bool mine = group < p.side * p.groups && col < width, is_bf16 = !kWide || type == DSA_BF16;
  const bool codes = (part == kPartLatent && !rope && p.latent_fp8) || (part == kPartKey && p.index_fp8);
  const bool turns = rot > 0 && mine && col >= offset && col < offset + rot, second = turns && col - offset >= rot / 2;
  const bool halves = __any_sync(0xffffffffu, rot > 0 && layout == DSA_ROTARY_HALF);     // (of the warp's groups)
  const bool any_codes = __any_sync(0xffffffffu, codes);
  // where this lane's run goes in a row of the cache, in bytes: row * row_bytes + at, or for index codes page by page
  int64_t row_bytes = 0, at_byte = 0;
  char *to = p.latent;
  if (part == kPartLatent) row_bytes = p.latent_row, at_byte = rope ? p.rope_at + 2 * col : p.latent_fp8 ? col : 2 * col;
  else if (part == kPartKey) to = p.index, row_bytes = p.index_fp8 ? 128 : 2 * p.D, at_byte = p.index_fp8 ? col : 2 * col;
  else to = p.kv, row_bytes = 4ll * p.heads * p.dim, at_byte = 2ll * ((part == kPartV ? p.heads : 0) + gi) * p.dim + 2 * col;
  to += at_byte;
  src += col * (is_bf16 ? 2 : 4);
  uint4 x[DEEP][W];
#pragma unroll
  for (int i = 0; i < DEEP; ++i) {
    const int64_t row = row0 + i * p.side + local;
    if (i < p.deep && mine && row < p.T && !(p.padded && p.row_pos[row] < 0)) {   // (padding is not read)
      const uint4 *from = reinterpret_cast<const uint4 *>(src + row * stride);
      x[i][0] = from[0], x[i][1] = from[1];
      if constexpr (kWide)
        if (!is_bf16) x[i][2] = from[2], x[i][3] = from[3];
    }
  }
  for (int r = threadIdx.x; r < rows; r += blockDim.x) {
    const int64_t row = row0 + r;
    int2 at = make_int2(-1, 0);
    if (row < p.T && p.row_pos[row] >= 0) {
      // (both are below 2^31)
      const uint32_t slot = static_cast<uint32_t>(p.row_page_start[row]) + static_cast<uint32_t>(p.row_pos[row]);
      const uint32_t pi = slot / static_cast<uint32_t>(p.P);
      if (pi < static_cast<uint32_t>(p.row_npages[row])) at = make_int2(p.pages[p.row_page_off[row] + pi], static_cast<int>(slot - pi * p.P));
      if (at.x < 0 || at.x >= p.num_pages) {
        atomicOr(p.err, kErrBounds);
        at.x = -1;
      }
    }
    where[r] = at;
  }
  if (p.rot) {
    const int half = p.rot / 2;
    // (from the last thread on: the first ones look the pages up)
    for (int k = blockDim.x - 1 - threadIdx.x; k < rows * half; k += blockDim.x) {
      const int r = k / half;
      if (row0 + r < p.T) angles[r * padded(half) + padded(k - r * half)] = rotary_angle(p.row_pos[row0 + r], p.turns[k - r * half], p.amplitude);
    }
  }
  __syncthreads();
  auto row_of = [&](const int2 place) {
    return part == kPartKey && p.index_fp8 ? to + static_cast<int64_t>(place.x) * p.P * (128 + 4) + place.y * 128
                                           : to + (static_cast<int64_t>(place.x) * p.P + place.y) * row_bytes;
  };
#pragma unroll
  for (int i = 0; i < DEEP; ++i) {
    if (i >= p.deep) break;      // uniform
    const int r = i * p.side + local;
    const int2 place = mine ? where[r] : make_int2(-1, 0);
    const bool in = place.x >= 0;
    if (!__any_sync(0xffffffffu, in && (turns || codes || !is_bf16))) {      // copied as it is
      if (in) {
        uint4 *out = reinterpret_cast<uint4 *>(row_of(place));
        out[0] = x[i][0], out[1] = x[i][1];
      }
      continue;
    }
    float v[N];
    if (!in) {
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = 0.f;
    } else if (is_bf16) {
      unpack8(*reinterpret_cast<float(*)[8]>(v), x[i][0]);
      unpack8(*reinterpret_cast<float(*)[8]>(v + 8), x[i][1]);
    } else if constexpr (kWide) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        v[4 * w] = __uint_as_float(x[i][w].x), v[4 * w + 1] = __uint_as_float(x[i][w].y);
        v[4 * w + 2] = __uint_as_float(x[i][w].z), v[4 * w + 3] = __uint_as_float(x[i][w].w);
      }
    }
    if (p.rot) {
      const int half = p.rot / 2, q = layout == DSA_ROTARY_HALF ? col - offset - (second ? half : 0) : (col - offset) / 2;
      const float2 *cs = angles + r * padded(half) + padded(q);
      if (turns && layout == DSA_ROTARY_INTERLEAVED) rotate_interleaved(v, cs);
      if (halves) {      // (all lanes of the warp take part in the exchange)
        const bool exchange = turns && layout == DSA_ROTARY_HALF;
        const int from = exchange ? lane + (second ? -1 : 1) * (half / N) : lane;
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const float other = __shfl_sync(0xffffffffu, v[k], from, kGroupLanes);
          if (exchange) v[k] = fmaf(v[k], cs[k].x, second ? other * cs[k].y : -other * cs[k].y);   // (as rotate_half, bit for bit)
        }
      }
    }
    uint32_t m = 0;
    if (any_codes) {
      m = max(amax_bits8(*reinterpret_cast<float(*)[8]>(v)), amax_bits8(*reinterpret_cast<float(*)[8]>(v + 8)));
#pragma unroll
      for (int o = kGroupLanes / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));   // the group's lanes
    }
    if (!in) continue;
    char *out = row_of(place);
    if (codes) {
      const GroupScale g(m);
      const uint2 a = codes8(*reinterpret_cast<float(*)[8]>(v), g), b = codes8(*reinterpret_cast<float(*)[8]>(v + 8), g);
      *reinterpret_cast<uint2 *>(out) = a;
      *reinterpret_cast<uint2 *>(out + 8) = b;
      if (lane == 0)
        *(part == kPartLatent ? reinterpret_cast<float *>(out - col + p.L) + base / 128
                              : reinterpret_cast<float *>(p.index + static_cast<int64_t>(place.x) * p.P * (128 + 4) +
                                                          static_cast<int64_t>(p.P) * 128) + place.y) = g.scale;
    } else {
      store8(out, DSA_BF16, 0, 8, true, *reinterpret_cast<float(*)[8]>(v));
      store8(out, DSA_BF16, 8, 16, true, *reinterpret_cast<float(*)[8]>(v + 8));
    }
  }
}

int bytes_of(int type) { return type == DSA_BF16 ? 2 : 4; }

bool on16(const void *p, int64_t stride_bytes, int64_t head_bytes = 0) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride_bytes % 16 == 0 && head_bytes % 16 == 0;
}

AppendParams append_base(const dsa_ctx *ctx, const dsa_plan_t *plan, const dsa_rotary *table) {
  AppendParams p{};
  p.row_pos = plan->row_pos, p.row_page_off = plan->row_page_off, p.row_npages = plan->row_npages;
  p.row_page_start = plan->row_page_start, p.pages = plan->pages, p.err = ctx->err;
  p.T = plan->T, p.P = ctx->cfg.page_size, p.num_pages = plan->cache_pages;
  p.padded = plan->capturable;
  if (table) p.turns = table->turns, p.rot = table->rot, p.amplitude = table->amplitude;
  return p;
}

void append_keys(const dsa_ctx *ctx, AppendParams &p, const dsa_append_t &a, const void *keys, void *index_cache) {
  const dsa_config_t &c = ctx->cfg;
  p.part[p.parts++] = kPartKey;
  p.keys = static_cast<const char *>(keys), p.index = static_cast<char *>(index_cache);
  p.key_type = a.key_type, p.keys_stride = a.keys_stride * bytes_of(a.key_type);
  p.D = c.index_dim, p.key_layout = a.key_layout, p.key_offset = p.rot ? a.key_offset : 0;
  p.index_fp8 = c.index_fmt == DSA_INDEX_FP8_132;
  const bool whole = rotary_whole(p.key_offset, p.rot, a.key_layout);
  p.keys_vec = whole && on16(keys, p.keys_stride);
  p.index_vec = whole && on16(index_cache, p.D * 2);
}

// Whether append_runs_kernel takes the call: whole runs of 16 columns, and pairs of them within a group of lanes.
bool whole_runs(const AppendParams &p) {
  auto turned = [&](int offset, int layout) {
    return offset % kLaneCols == 0 && p.rot % (layout == DSA_ROTARY_HALF ? 2 * kLaneCols : kLaneCols) == 0;
  };
  if (p.c && (!p.c_vec || p.L % kLaneCols || !p.latent_vec || p.R > 128 || p.R % kLaneCols ||
              (p.R > 0 && (!p.k_pe_vec || !p.rope_vec || !turned(0, p.layout)))))
    return false;
  if (p.keys && (!p.keys_vec || p.D > 128 || p.D % kLaneCols || !turned(p.key_offset, p.key_layout) ||
                 (p.index_fp8 ? reinterpret_cast<uintptr_t>(p.index) % 8 || p.P % 2 : !p.index_vec)))
    return false;
  if (p.k && (!p.k_vec || !p.v_vec || !p.kv_vec || p.dim > 128 || p.dim % kLaneCols || !turned(p.rot ? p.kv_offset : 0, p.kv_layout)))
    return false;
  return true;
}

cudaError_t launch_append(const dsa_ctx *ctx, AppendParams &p, cudaStream_t s, int32_t *launches) {
  *launches += 1;
  p.groups = (p.c ? (p.L + 127) / 128 + (p.R > 0 ? 1 : 0) : 0) + (p.keys ? 1 : 0) + (p.k ? 2 * p.heads : 0);
  if (whole_runs(p) && p.groups <= kAppendThreads / kGroupLanes) {
    const bool wide = (p.c && (p.c_type != DSA_BF16 || (p.R > 0 && p.k_pe_type != DSA_BF16))) || (p.keys && p.key_type != DSA_BF16) ||
                      (p.k && p.kv_type != DSA_BF16);
    // As many rows side by side as the threads hold, fewer where that leaves SMs without any; and a thread as deep as
    // takes least by waves of CTAs of some 2.5 us and 0.6 for each of its rows: one row for a decode step; for 8197
    // rows of K and V four, 8.6 us (three: 10.4, a second wave of few); for 8192 in 8 bits three, 8.5 us (four: 10.1).
    const int sms = std::max(1, ctx->num_sms);
    p.side = std::max(1, std::min(kAppendThreads / kGroupLanes / p.groups, p.T / sms));
    const int threads = (p.side * p.groups * kGroupLanes + 31) / 32 * 32, at_once = sms * (65536 / (kAppendRegisters * threads));
    // (whole_runs bounds rot by the 128 columns of what turns, so that one row a thread always fits)
    double least = 0.0;
    for (int deep = 1; deep <= (wide ? kAppendDeep<true> : kAppendDeep<false>); ++deep) {
      if (p.side * deep * padded(p.rot / 2) * sizeof(float2) > 46 * 1024) break;
      const int ctas = (p.T + p.side * deep - 1) / (p.side * deep);
      const double cost = ((ctas + at_once - 1) / at_once) * (2.5 + 0.6 * deep);
      if (deep == 1 || cost < least) least = cost, p.deep = deep;
    }
    const int rows = p.side * p.deep;
    auto kernel = wide ? p.deep == 1 ? append_runs_kernel<true, 1> : append_runs_kernel<true, kAppendDeep<true>>
                       : p.deep == 1 ? append_runs_kernel<false, 1> : append_runs_kernel<false, kAppendDeep<false>>;
    return launch_overlapped(kernel, dim3(static_cast<unsigned>((p.T + rows - 1) / rows)), threads,
                             rows * padded(p.rot / 2) * static_cast<int>(sizeof(float2)), 1, s, p);
  }
  int floats = p.rot ? rotary_pairs(p.rot) * 2 : 0;
  if (p.keys && p.index_fp8) floats += p.D;
  const int64_t tasks = static_cast<int64_t>(p.T) * p.parts;
  return launch_overlapped(append_kernel, dim3(static_cast<unsigned>((tasks + kAppendWarps - 1) / kAppendWarps)),
                           kAppendWarps * 32, floats * kAppendWarps * 4, 1, s, p);
}

}  // namespace

cudaError_t launch_append_latents(const dsa_ctx *ctx, const dsa_plan_t *plan, const dsa_rotary *table, const dsa_append_t &a,
                                  const void *c, const void *k_pe, void *latent_cache, const void *keys, void *index_cache,
                                  cudaStream_t s, int32_t *launches) {
  // (a rope of no columns: a table is the keys' alone, and without keys nothing turns, whatever its width)
  AppendParams p = append_base(ctx, plan, ctx->cfg.rope_dim > 0 || keys ? table : nullptr);
  if (c) {
    const dsa_config_t &g = ctx->cfg;
    p.part[p.parts++] = kPartLatent;
    p.c = static_cast<const char *>(c), p.k_pe = static_cast<const char *>(k_pe), p.latent = static_cast<char *>(latent_cache);
    p.L = g.kv_lora_rank, p.R = g.rope_dim, p.c_type = a.c_type, p.k_pe_type = a.k_pe_type, p.layout = a.layout;
    p.c_stride = a.c_stride * bytes_of(a.c_type), p.k_pe_stride = a.k_pe_stride * bytes_of(a.k_pe_type);
    p.latent_fp8 = g.latent_fmt == DSA_LATENT_FP8_656;
    p.rope_at = p.latent_fp8 ? p.L + 4 * (p.L / 128) : 2 * p.L;
    p.latent_row = p.rope_at + 2 * p.R;
    const bool whole = rotary_whole(0, p.rot, a.layout);
    p.c_vec = on16(c, p.c_stride), p.k_pe_vec = whole && on16(k_pe, p.k_pe_stride);
    p.latent_vec = on16(latent_cache, p.latent_row);
    p.rope_vec = whole && p.latent_vec && p.rope_at % 16 == 0;
  }
  if (keys) append_keys(ctx, p, a, keys, index_cache);
  return launch_append(ctx, p, s, launches);
}

cudaError_t launch_append_kv(const dsa_ctx *ctx, const dsa_plan_t *plan, const dsa_rotary *table, const dsa_append_t &a,
                             int32_t kv_heads, int32_t head_dim, const void *k, const void *v, void *kv_cache,
                             const void *keys, void *index_cache, cudaStream_t s, int32_t *launches) {
  AppendParams p = append_base(ctx, plan, table);
  p.part[p.parts++] = kPartK;
  p.part[p.parts++] = kPartV;
  p.k = static_cast<const char *>(k), p.v = static_cast<const char *>(v), p.kv = static_cast<char *>(kv_cache);
  p.heads = kv_heads, p.dim = head_dim, p.kv_type = a.kv_type, p.kv_layout = a.layout, p.kv_offset = a.kv_offset;
  const int size = bytes_of(a.kv_type);
  p.k_stride = a.k_stride * size, p.k_head = a.k_head * size, p.v_stride = a.v_stride * size, p.v_head = a.v_head * size;
  const bool whole = rotary_whole(p.rot ? p.kv_offset : 0, p.rot, a.layout);
  p.k_vec = whole && on16(k, p.k_stride, p.k_head), p.v_vec = on16(v, p.v_stride, p.v_head);
  p.kv_vec = whole && on16(kv_cache, 2ll * head_dim);
  if (keys) append_keys(ctx, p, a, keys, index_cache);
  return launch_append(ctx, p, s, launches);
}

}  // namespace dsa
