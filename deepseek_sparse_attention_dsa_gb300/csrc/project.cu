// project.cu -- matrix product of e4m3 codes with fp32 scales per block of 128:
//
//   out[m, b, n] = sum_kb a_scale[m, b, kb] * w_scale[b, n / 128, kb]
//                  * sum_{k in block kb} a[m, b, k] * w[b, n, k]
//
// for b = 0 .. batch-1 (the heads of an absorbed projection; 1 otherwise).
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "dsa_internal.h"
#include "fp8.cuh"

namespace dsa {
namespace {

struct ProjectParams {
  const uint8_t *a, *w;
  const float *a_scale, *w_scale;
  void *out;
  const int32_t *count;
  int64_t rows;
  int64_t a_stride, a_batch, w_stride, w_batch, as_stride, as_batch, ws_stride, ws_batch, out_stride, out_batch;
  int32_t n, k, per_row, out_type;
};

__device__ __forceinline__ float e4m3_value(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// CUDA-core form: 64 x 64 outputs a CTA, 4 x 4 a thread.
__global__ void __launch_bounds__(256) project_simt_kernel(const ProjectParams p) {
  __shared__ float as[32][65], ws[32][65];
  const int64_t live = live_rows(p.rows, p.count, p.per_row);
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * 64;
  if (m0 >= live) return;
  const int n0 = blockIdx.y * 64, b = blockIdx.z;
  const uint8_t *a = p.a + b * p.a_batch, *w = p.w + b * p.w_batch;
  const float *as_ = p.a_scale + b * p.as_batch, *ws_ = p.w_scale + b * p.ws_batch;
  const int tm = threadIdx.x / 16, tn = threadIdx.x % 16;
  float acc[4][4] = {};
  for (int kb = 0; kb * 128 < p.k; ++kb) {
    float part[4][4] = {};
    for (int k0 = kb * 128; k0 < min(p.k, kb * 128 + 128); k0 += 32) {
      __syncthreads();
      for (int i = threadIdx.x; i < 64 * 32; i += 256) {
        const int r = i / 32, c = i % 32;
        as[c][r] = m0 + r < live && k0 + c < p.k ? e4m3_value(a[(m0 + r) * p.a_stride + k0 + c]) : 0.f;
        ws[c][r] = n0 + r < p.n && k0 + c < p.k ? e4m3_value(w[(n0 + r) * p.w_stride + k0 + c]) : 0.f;
      }
      __syncthreads();
      for (int c = 0; c < 32; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[i][j] = fmaf(as[c][tm + 16 * i], ws[c][tn + 16 * j], part[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t m = m0 + tm + 16 * i;
      const float sa = m < live ? as_[m * p.as_stride + kb] : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tn + 16 * j;
        const float sw = n < p.n ? ws_[n / 128 * p.ws_stride + kb] : 0.f;
        acc[i][j] = fmaf(part[i][j], sa * sw, acc[i][j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + tm + 16 * i;
      const int n = n0 + tn + 16 * j;
      if (m >= live || n >= p.n) continue;
      const int64_t at = m * p.out_stride + b * p.out_batch + n;
      if (p.out_type == DSA_BF16) static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(acc[i][j]);
      else static_cast<float *>(p.out)[at] = acc[i][j];
    }
}

}  // namespace

bool project_tc_supported(const dsa_project_t &, const void *, const void *) { return false; }

cudaError_t launch_project_fp8(const dsa_ctx *, const dsa_project_t &g, const void *a, const float *a_scale,
                               const void *w, const float *w_scale, void *out, const int32_t *count, int32_t per_row,
                               cudaStream_t s, int32_t *launches) {
  ProjectParams p{};
  p.a = static_cast<const uint8_t *>(a);
  p.w = static_cast<const uint8_t *>(w);
  p.a_scale = a_scale;
  p.w_scale = w_scale;
  p.out = out;
  p.count = count;
  p.per_row = per_row;
  p.rows = g.rows;
  p.a_stride = g.a_stride, p.a_batch = g.a_batch;
  p.w_stride = g.w_stride, p.w_batch = g.w_batch;
  p.as_stride = g.a_scale_stride, p.as_batch = g.a_scale_batch;
  p.ws_stride = g.w_scale_stride, p.ws_batch = g.w_scale_batch;
  p.out_stride = g.out_stride, p.out_batch = g.out_batch;
  p.n = g.n, p.k = g.k;
  p.out_type = g.out_type;
  const dim3 grid(static_cast<unsigned>((g.rows + 63) / 64), (g.n + 63) / 64, g.batch);
  project_simt_kernel<<<grid, 256, 0, s>>>(p);
  *launches += 1;
  return cudaGetLastError();
}

}  // namespace dsa
