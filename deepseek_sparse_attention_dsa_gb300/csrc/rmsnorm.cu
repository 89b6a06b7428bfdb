// rmsnorm.cu -- root-mean-square norm of rows, with the residual's addition
// before it and an output in e4m3 codes with a scale per 128 columns.
//
//   h = x + residual          (fp32; residual_out is h rounded once)
//   y = h * weight / sqrt(mean(h^2) + eps)
//   out = y rounded once, or codes and scales of y's groups of 128 columns
//
// One pass: a row's values stay in the registers of the threads that read
// them between the sum of squares and the output, so x, residual and weight
// are each read once and every output written once.  Bound by HBM for many
// rows (8192 x 4096 with residual to codes: 36.9 us, 6.39 TB/s, 94% of the
// measured copy) and by one launch's latency for few (1 x 5120: 2.6 us).  fp32 or
// mixed types, and rows off 16 bytes, take rmsnorm_kernel, a row at a time: the same
// with x and residual in fp32 71.6 us (6.10 TB/s, 90%), bf16 with an fp32 residual 71.8
// (5.16 TB/s), bf16 rows at an odd stride 58.9 (4.0 TB/s).  A thread holds CH pieces of eight
// consecutive columns, piece c of thread t at column (c * THREADS + t) * 8, so
// 16 neighbouring lanes hold a group of 128 and its maximum is four shuffles.
#include <cuda_runtime.h>

#include <algorithm>

#include "dsa_internal.h"
#include "fp8.cuh"

namespace dsa {
namespace {

struct NormParams {
  const void *x, *weight, *residual;
  void *residual_out, *out;
  uint8_t *codes;
  float *scales;
  const int32_t *count;
  int64_t rows, x_stride, residual_stride, residual_out_stride, out_stride, codes_stride, scales_stride;  // bytes
  int32_t width, per_row;
  int x_type, weight_type, residual_type, out_type;
  bool x_vec, weight_vec, residual_vec, residual_out_vec, out_vec, codes_vec;
  float eps;
};

template <typename T>
__device__ __forceinline__ T *row_at(T *base, int64_t row, int64_t stride) {
  return reinterpret_cast<T *>(reinterpret_cast<uintptr_t>(base) + row * stride);
}

// TPR threads a row (32: a warp), ROWS rows a CTA.
template <int TPR, int ROWS, int CH>
__global__ void __launch_bounds__(TPR *ROWS) rmsnorm_kernel(const NormParams p) {
  grid_dependency();
  const int t = threadIdx.x % TPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / TPR;
  if (row >= live_rows(p.rows, p.count, p.per_row)) return;   // uniform over a row's threads
  const void *xr = row_at(static_cast<const char *>(p.x), row, p.x_stride);
  float h[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) load8(h[c], xr, p.x_type, (c * TPR + t) * 8, p.width, p.x_vec);
  if (p.residual) {
    const void *rr = row_at(static_cast<const char *>(p.residual), row, p.residual_stride);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float r[8];
      load8(r, rr, p.residual_type, (c * TPR + t) * 8, p.width, p.residual_vec);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] += r[i];
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(h[c][i], h[c][i], sum);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (TPR > 32) {
    __shared__ float part[TPR / 32];
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < TPR / 32; ++w) sum += part[w];
  }
  const float rstd = 1.f / sqrtf(sum / static_cast<float>(p.width) + p.eps);
  if (p.residual_out) {
    void *ro = row_at(static_cast<char *>(p.residual_out), row, p.residual_out_stride);
#pragma unroll
    for (int c = 0; c < CH; ++c) store8(ro, p.residual_type, (c * TPR + t) * 8, p.width, p.residual_out_vec, h[c]);
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * TPR + t) * 8;
    float w[8];
    if (p.weight) {
      load8(w, p.weight, p.weight_type, col, p.width, p.weight_vec);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 1.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) h[c][i] *= rstd * w[i];
    if (p.out) store8(row_at(static_cast<char *>(p.out), row, p.out_stride), p.out_type, col, p.width, p.out_vec, h[c]);
    if (p.codes) {
      uint32_t m = amax_bits8(h[c]);
#pragma unroll
      for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));   // the group's 16 lanes
      const GroupScale g(m);
      store_codes8(row_at(p.codes, row, p.codes_stride), col, p.width, p.codes_vec, codes8(h[c], g));
      if ((t & 15) == 0 && col < p.width) row_at(p.scales, row, p.scales_stride)[col / 128] = g.scale;
    }
  }
}

// The usual types, bf16 throughout in whole 16-byte pieces: a CTA (or a warp, TPR
// = 32) walks rows with the weights in its registers and the next row's pieces
// in flight while it norms this one.  1024 threads an SM; with a residual and
// rows of 1,032 to 4,096 columns 768, whose 85 registers a thread hold both
// streams without spills (8192 x 4096 to codes: 36.9 us against 39.7; without a
// residual it is 24.1 against 22.4, and wider rows leave one CTA an SM).
template <int TPR>
constexpr int kNormRows = TPR == 32 ? 8 : 1;   // rows a CTA
template <int TPR, bool kResidual>
constexpr int kNormCtas = (kResidual && (TPR == 128 || TPR == 256) ? 768 : 1024) / (TPR * kNormRows<TPR>);   // an SM

template <int TPR, int CH, bool kResidual>
__global__ void __launch_bounds__(TPR *kNormRows<TPR>, kNormCtas<TPR, kResidual>)
    rmsnorm_bf16_kernel(const NormParams p) {
  constexpr int ROWS = kNormRows<TPR>;
  __shared__ float part[2][TPR / 32];
  grid_dependency();
  const int t = threadIdx.x % TPR;
  const int64_t live = live_rows(p.rows, p.count, p.per_row);
  const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
  int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / TPR;
  if (row >= live) return;   // uniform over a row's threads
  const uint4 zero = make_uint4(0, 0, 0, 0);
  bool in[CH];
  uint4 w[CH], x[CH], r[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) in[c] = (c * TPR + t) * 8 < p.width;
  auto fetch = [&](int64_t at) {
    const uint4 *xr = reinterpret_cast<const uint4 *>(static_cast<const char *>(p.x) + at * p.x_stride) + t;
    const uint4 *rr = reinterpret_cast<const uint4 *>(static_cast<const char *>(p.residual) + at * p.residual_stride) + t;
#pragma unroll
    for (int c = 0; c < CH; ++c) x[c] = in[c] ? xr[c * TPR] : zero;
    if (kResidual)
#pragma unroll
      for (int c = 0; c < CH; ++c) r[c] = in[c] ? rr[c * TPR] : zero;
  };
  fetch(row);
#pragma unroll
  for (int c = 0; c < CH; ++c)
    w[c] = p.weight == nullptr ? make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u)
           : in[c]             ? static_cast<const uint4 *>(p.weight)[c * TPR + t]
                               : zero;
  for (int turn = 0;; turn ^= 1) {
    float h[CH][8], sum = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      unpack8(h[c], x[c]);
      if (kResidual) {
        float v[8];
        unpack8(v, r[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] += v[i];
      }
    }
    const int64_t next = row + step;
    if (next < live) fetch(next);
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(h[c][i], h[c][i], sum);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (TPR > 32) {
      // (two buffers: a warp that runs ahead writes the other one, and cannot
      // come back to this before every warp has passed the next barrier)
      if (threadIdx.x % 32 == 0) part[turn][threadIdx.x / 32] = sum;
      __syncthreads();
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < TPR / 32; ++i) sum += part[turn][i];
    }
    const float rstd = 1.f / sqrtf(sum / static_cast<float>(p.width) + p.eps);
    if (kResidual && p.residual_out) {
      void *ro = row_at(static_cast<char *>(p.residual_out), row, p.residual_out_stride);
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (in[c]) store8(ro, DSA_BF16, (c * TPR + t) * 8, p.width, true, h[c]);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * TPR + t) * 8;
      float wf[8];
      unpack8(wf, w[c]);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] *= rstd * wf[i];
      if (p.out && in[c]) store8(row_at(static_cast<char *>(p.out), row, p.out_stride), DSA_BF16, col, p.width, true, h[c]);
      if (p.codes) {
        uint32_t m = amax_bits8(h[c]);
#pragma unroll
        for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));   // the group's 16 lanes
        const GroupScale g(m);
        const uint2 code = codes8(h[c], g);
        if (in[c]) {
          *reinterpret_cast<uint2 *>(row_at(p.codes, row, p.codes_stride) + col) = code;
          if ((t & 15) == 0) row_at(p.scales, row, p.scales_stride)[col / 128] = g.scale;
        }
      }
    }
    if (next >= live) break;
    row = next;
  }
}

template <int TPR, int CH>
cudaError_t run_bf16(const NormParams &p, int num_sms, cudaStream_t s) {
  constexpr int ROWS = kNormRows<TPR>, THREADS = TPR * ROWS;
  const int64_t ctas = (p.rows + ROWS - 1) / ROWS;
  auto grid = [&](int per_sm) { return dim3(static_cast<unsigned>(std::min<int64_t>(ctas, static_cast<int64_t>(num_sms) * per_sm))); };
  if (p.residual)
    return launch_overlapped(rmsnorm_bf16_kernel<TPR, CH, true>, grid(kNormCtas<TPR, true>), THREADS, 0, 1, s, p);
  return launch_overlapped(rmsnorm_bf16_kernel<TPR, CH, false>, grid(kNormCtas<TPR, false>), THREADS, 0, 1, s, p);
}

bool aligned(const void *p, int64_t stride_bytes, int64_t rows, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (rows <= 1 || stride_bytes % bytes == 0);
}

template <int TPR, int ROWS, int CH>
cudaError_t run(const NormParams &p, cudaStream_t s) {
  return launch_overlapped(rmsnorm_kernel<TPR, ROWS, CH>, dim3(static_cast<unsigned>((p.rows + ROWS - 1) / ROWS)), TPR * ROWS,
                           0, 1, s, p);
}

}  // namespace

cudaError_t launch_rmsnorm(int num_sms, const dsa_norm_t &n, const void *x, const void *weight, const void *residual,
                           void *residual_out, void *out, void *codes, float *scales, const int32_t *count,
                           int32_t per_row, cudaStream_t s, int32_t *launches) {
  auto size = [](int type) { return type == DSA_BF16 ? 2 : 4; };
  NormParams p{};
  p.x = x;
  p.weight = weight;
  p.residual = residual;
  p.residual_out = residual_out;
  p.out = out;
  p.codes = static_cast<uint8_t *>(codes);
  p.scales = scales;
  p.count = count;
  p.per_row = per_row;
  p.rows = n.rows;
  p.width = n.width;
  p.x_type = n.x_type;
  p.weight_type = n.weight_type;
  p.residual_type = n.residual_type;
  p.out_type = n.out_type;
  p.eps = n.eps;
  p.x_stride = n.x_stride * size(n.x_type);
  p.residual_stride = n.residual_stride * size(n.residual_type);
  p.residual_out_stride = n.residual_out_stride * size(n.residual_type);
  p.out_stride = n.out_stride * size(n.out_type);
  p.codes_stride = n.codes_stride;
  p.scales_stride = n.scales_stride * 4;
  p.x_vec = aligned(x, p.x_stride, n.rows, 16);
  p.weight_vec = aligned(weight, 0, 1, 16);
  p.residual_vec = aligned(residual, p.residual_stride, n.rows, 16);
  p.residual_out_vec = aligned(residual_out, p.residual_out_stride, n.rows, 16);
  p.out_vec = aligned(out, p.out_stride, n.rows, 16);
  p.codes_vec = aligned(codes, p.codes_stride, n.rows, 8);
  const int pieces = (n.width + 7) / 8;
  if (n.width % 8 == 0 && pieces <= 2048 && n.x_type == DSA_BF16 && p.x_vec && (!weight || (n.weight_type == DSA_BF16 && p.weight_vec)) &&
      (!residual || (n.residual_type == DSA_BF16 && p.residual_vec)) && (!residual_out || p.residual_out_vec) &&
      (!out || (n.out_type == DSA_BF16 && p.out_vec)) && (!codes || p.codes_vec)) {
    *launches += 1;
    return pieces <= 32     ? run_bf16<32, 1>(p, num_sms, s)
           : pieces <= 64   ? run_bf16<32, 2>(p, num_sms, s)
           : pieces <= 128  ? run_bf16<64, 2>(p, num_sms, s)
           : pieces <= 256  ? run_bf16<128, 2>(p, num_sms, s)
           : pieces <= 512  ? run_bf16<256, 2>(p, num_sms, s)
           : pieces <= 1024 ? run_bf16<512, 2>(p, num_sms, s)
                            : run_bf16<1024, 2>(p, num_sms, s);
  }
  *launches += 1;
  return pieces <= 32     ? run<32, 8, 1>(p, s)
         : pieces <= 64   ? run<32, 8, 2>(p, s)
         : pieces <= 128  ? run<32, 8, 4>(p, s)
         : pieces <= 256  ? run<128, 1, 2>(p, s)
         : pieces <= 512  ? run<256, 1, 2>(p, s)
         : pieces <= 1024 ? run<512, 1, 2>(p, s)
         : pieces <= 2048 ? run<512, 1, 4>(p, s)
                          : run<1024, 1, 4>(p, s);   // up to DSA_NORM_MAX_WIDTH
}

}  // namespace dsa
