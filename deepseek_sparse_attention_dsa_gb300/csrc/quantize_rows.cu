// quantize_rows.cu -- bf16 or fp32 values to e4m3 codes with fp32 scales in the
// layouts of the 8-bit product (project.cu): rows with a scale per 128 columns
// (activations), matrices with a scale per 128 x 128 block (weights).  The rule
// is the one of quantize-on-store (fp8.cuh).  Bound by HBM: every value is read
// once and stays in registers between its group's maximum and its code (rows of
// 2048 x 65536 bf16: 63.3 us, 6.43 TB/s, 95% of the measured copy; blocks of 65536
// x 4096 bf16: 133 us, 6.06 TB/s; of 8192 x 4096: 19.9 us, and 16.6 where the codes
// of the last call are still in L2 to be written over).  With a division for each value the first took
// 149 us, bound by its instructions.  fp32 rows take 100.7 us (6.70 TB/s); rows off 16
// bytes a value a load, 144 us in bf16 and 138 in fp32 (blocks of 8192 x 4096 bf16: 37.7).
#include <cuda_runtime.h>

#include "dsa_internal.h"
#include "fp8.cuh"

namespace dsa {
namespace {

struct RowsParams {
  const char *x;
  uint8_t *codes;
  float *scales;
  const int32_t *count;
  int64_t rows, width;                               // values
  int64_t x_stride, codes_stride, scales_stride;     // bytes
  int64_t segments;                                  // warps a row
  int64_t per_row;
  int x_type;
  bool x_vec, codes_vec, dense;
};

// Pieces of eight columns a lane: a warp's segment of a row is kRowPieces * 256 columns.
constexpr int kRowPieces = 4;   // (four: the scales of a half warp's groups are shared out over four lanes)

// One warp a segment, 16 lanes a group.
__global__ void __launch_bounds__(256) quantize_rows_kernel(const RowsParams p) {
  grid_dependency();
  const int64_t task = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;
  const int64_t row = task / p.segments;
  if (row >= p.rows) return;
  int64_t width = p.width;
  if (p.count) {   // a dense matrix comes as one row, whose width is what the padding cuts
    const int64_t live = static_cast<int64_t>(*p.count) * p.per_row;
    if (p.dense) width = live < width ? live : width;
    else if (row >= live) return;
  }
  const int lane = threadIdx.x % 32;
  const int64_t col0 = (task % p.segments) * (kRowPieces * 256) + lane * 8;
  const char *x = p.x + row * p.x_stride;
  float v[kRowPieces][8];
#pragma unroll
  for (int c = 0; c < kRowPieces; ++c) load8(v[c], x, p.x_type, col0 + c * 256, width, p.x_vec);
#pragma unroll
  for (int c = 0; c < kRowPieces; ++c) {
    uint32_t m = amax_bits8(v[c]);
#pragma unroll
    for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const GroupScale g(m);
    const int64_t col = col0 + c * 256;
    store_codes8(p.codes + row * p.codes_stride, col, width, p.codes_vec, codes8(v[c], g));
    if ((lane & 15) == 0 && col < width)
      reinterpret_cast<float *>(reinterpret_cast<char *>(p.scales) + row * p.scales_stride)[col / 128] = g.scale;
  }
}

// The same for bf16 rows of whole 16-byte pieces on 16 bytes, codes on 8: the
// pieces wait in their packed form, half the registers.
__global__ void __launch_bounds__(256) quantize_rows_bf16_kernel(const RowsParams p) {
  grid_dependency();
  const uint32_t task = blockIdx.x * 8u + threadIdx.x / 32;   // (fewer than 2^32: the grid)
  const uint32_t segments = static_cast<uint32_t>(p.segments);
  const uint32_t row = segments >= task + 1 ? 0 : task / segments;
  if (row >= p.rows) return;
  int64_t width = p.width;
  if (p.count) {
    const int64_t live = static_cast<int64_t>(*p.count) * p.per_row;
    if (p.dense) width = live < width ? live : width;
    else if (row >= live) return;
  }
  const int lane = threadIdx.x % 32;
  const int64_t col0 = static_cast<int64_t>(task - row * segments) * (kRowPieces * 256) + lane * 8;
  const uint4 *x = reinterpret_cast<const uint4 *>(p.x + row * p.x_stride + col0 * 2);
  const int64_t left = width - col0;   // columns from this lane's first on
  uint4 u[kRowPieces];
#pragma unroll
  for (int c = 0; c < kRowPieces; ++c) u[c] = c * 256 < left ? __ldcs(x + c * 32) : make_uint4(0, 0, 0, 0);
  uint2 *codes = reinterpret_cast<uint2 *>(p.codes + row * p.codes_stride + col0);
  float *scales = reinterpret_cast<float *>(reinterpret_cast<char *>(p.scales) + row * p.scales_stride) + col0 / 128;
  // A half warp's four groups: their maxima, then both divisions of a group in
  // one lane of four (every lane would do them otherwise, half of the kernel's
  // instructions), then the scales back to the lanes
  uint32_t m[kRowPieces];
#pragma unroll
  for (int c = 0; c < kRowPieces; ++c) {
    m[c] = amax_bits8(u[c]);
#pragma unroll
    for (int o = 8; o; o >>= 1) m[c] = max(m[c], __shfl_xor_sync(0xffffffffu, m[c], o));
  }
  const float scale = group_scale(lane & 2 ? (lane & 1 ? m[3] : m[2]) : (lane & 1 ? m[1] : m[0]));
  const float r = 1.f / scale;
#pragma unroll
  for (int c = 0; c < kRowPieces; ++c) {
    const GroupScale g(__shfl_sync(0xffffffffu, scale, c, 16), __shfl_sync(0xffffffffu, r, c, 16));
    float v[8];
    unpack8(v, u[c]);
    const uint2 code = codes8(v, g);
    if (c * 256 < left) {
      codes[c * 32] = code;
      if ((lane & 15) == 0) scales[c * 2] = g.scale;
    }
  }
}

struct BlocksParams {
  const char *w;
  uint8_t *codes;
  float *scales;
  int64_t w_stride, w_batch, codes_stride, codes_batch, scales_stride, scales_batch;   // bytes
  int32_t n, k;
  int w_type;
  bool w_vec, codes_vec;
};

// One CTA a block of 128 x 128: 16 threads a row of it, 4 rows a thread.
// kPacked: bf16 in whole 16-byte pieces, which wait for the maximum in their
// packed form; many small CTAs keep enough of them in flight (8192 x 4096: 19.9 us;
// two CTAs an SM that walk blocks with the next one in flight 21.0, one CTA behind
// six stages of TMA loads 22.0, 256 threads a block 25).
template <bool kPacked>
__global__ void __launch_bounds__(512, kPacked ? 3 : 2) quantize_blocks_kernel(const BlocksParams p) {
  grid_dependency();
  const int64_t b = blockIdx.z;
  const int col = blockIdx.x * 128 + (threadIdx.x % 16) * 8;
  const int row0 = blockIdx.y * 128 + threadIdx.x / 16;
  const char *w = p.w + b * p.w_batch;
  uint4 u[kPacked ? 4 : 1];
  float v[kPacked ? 1 : 4][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = row0 + 32 * i;
    if (kPacked) {
      // (in bytes a column passes 32 bits)
      const char *at = w + row * p.w_stride + static_cast<int64_t>(col) * 2;
      u[kPacked ? i : 0] = row < p.n && col < p.k ? __ldcs(reinterpret_cast<const uint4 *>(at)) : make_uint4(0, 0, 0, 0);
    } else {
      if (row < p.n) {
        load8(v[kPacked ? 0 : i], w + row * p.w_stride, p.w_type, col, p.k, p.w_vec);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[kPacked ? 0 : i][j] = 0.f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, kPacked ? amax_bits8(u[kPacked ? i : 0]) : amax_bits8(v[kPacked ? 0 : i]));
  m = __reduce_max_sync(0xffffffffu, m);
  __shared__ uint32_t part[16];
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, part[i]);
  const GroupScale g(m);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = row0 + 32 * i;
    if (kPacked) unpack8(v[0], u[kPacked ? i : 0]);
    const uint2 c = codes8(v[kPacked ? 0 : i], g);
    if (row < p.n) store_codes8(p.codes + b * p.codes_batch + row * p.codes_stride, col, p.k, p.codes_vec, c);
  }
  if (threadIdx.x == 0)
    *reinterpret_cast<float *>(reinterpret_cast<char *>(p.scales) + b * p.scales_batch + blockIdx.y * p.scales_stride +
                               blockIdx.x * 4) = g.scale;
}

}  // namespace

cudaError_t launch_quantize_rows(const dsa_rows_t &r, const void *x, void *codes, float *scales, const int32_t *count,
                                 int32_t per_row, cudaStream_t s, int32_t *launches) {
  RowsParams p{};
  const int size = r.x_type == DSA_BF16 ? 2 : 4;
  p.x = static_cast<const char *>(x);
  p.codes = static_cast<uint8_t *>(codes);
  p.scales = scales;
  p.count = count;
  p.per_row = per_row;
  p.rows = r.rows;
  p.width = r.width;
  p.x_stride = r.x_stride * size;
  p.codes_stride = r.codes_stride;
  p.scales_stride = r.scales_stride * 4;
  p.x_type = r.x_type;
  // a dense matrix of whole groups is one long row: no lane idles on narrow rows
  if (r.width % 128 == 0 && r.x_stride == r.width && r.codes_stride == r.width && r.scales_stride == r.width / 128) {
    p.width = r.rows * r.width;
    p.rows = 1;
    p.per_row = static_cast<int64_t>(per_row) * r.width;
    p.dense = true;
  }
  const bool one = p.rows == 1;
  p.x_vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && (one || p.x_stride % 16 == 0);
  p.codes_vec = reinterpret_cast<uintptr_t>(codes) % 8 == 0 && (one || p.codes_stride % 8 == 0);
  p.segments = (p.width + kRowPieces * 256 - 1) / (kRowPieces * 256);
  const int64_t grid = (p.rows * p.segments + 7) / 8;
  const bool packed = p.x_type == DSA_BF16 && p.x_vec && p.codes_vec && p.width % 8 == 0 && grid < (int64_t(1) << 29);
  *launches += 1;
  return launch_overlapped(packed ? quantize_rows_bf16_kernel : quantize_rows_kernel, dim3(static_cast<unsigned>(grid)), 256,
                           0, 1, s, p);
}

cudaError_t launch_quantize_weight(const dsa_weight_t &w, const void *src, void *codes, float *scales, cudaStream_t s,
                                   int32_t *launches) {
  BlocksParams p{};
  const int size = w.w_type == DSA_BF16 ? 2 : 4;
  p.w = static_cast<const char *>(src);
  p.codes = static_cast<uint8_t *>(codes);
  p.scales = scales;
  p.w_stride = w.w_stride * size;
  p.w_batch = w.w_batch * size;
  p.codes_stride = w.codes_stride;
  p.codes_batch = w.codes_batch;
  p.scales_stride = w.scales_stride * 4;
  p.scales_batch = w.scales_batch * 4;
  p.n = w.n;
  p.k = w.k;
  p.w_type = w.w_type;
  p.w_vec = reinterpret_cast<uintptr_t>(src) % 16 == 0 && (w.n == 1 || p.w_stride % 16 == 0) &&
            (w.batch == 1 || p.w_batch % 16 == 0);
  p.codes_vec = reinterpret_cast<uintptr_t>(codes) % 8 == 0 && (w.n == 1 || p.codes_stride % 8 == 0) &&
                (w.batch == 1 || p.codes_batch % 8 == 0);
  const dim3 grid((w.k - 1) / 128 + 1, (w.n + 127) / 128, w.batch);
  const bool packed = w.w_type == DSA_BF16 && p.w_vec && w.k % 8 == 0;
  *launches += 1;
  return launch_overlapped(packed ? quantize_blocks_kernel<true> : quantize_blocks_kernel<false>, grid, 512, 0, 1, s, p);
}

}  // namespace dsa
