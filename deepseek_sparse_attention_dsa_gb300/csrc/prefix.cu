// prefix.cu -- dense causal GQA over the paged cache of msa.cu, for batches whose
// requests share their first pages (a system prompt, a document).
//
//   out[r, h] = sum_j p_j v_j / sum_j p_j,  p_j = 2^((q[r,h] . k_j) * sm_scale * log2 e - m),
//
// over the positions j = 0 .. pos(r) of row r's request, m the largest exponent.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "dsa_internal.h"
#include "fp8.cuh"
#include "ptx.cuh"

struct dsa_prefix_plan {
  const dsa_plan_t *plan = nullptr;
  dsa_msa_shape_t shape{};
  std::vector<dsa_prefix_t> prefixes;
  int64_t tokens_read = 0;
};

namespace dsa {
namespace {

constexpr float kPrefixLog2e = 1.4426950408889634f;
constexpr float kNoMax = -1.0e30f;   // the reference maximum of a row that has seen no key

__device__ __forceinline__ float exp2_approx(float x) {   // (relative error 2^-22; 0 for -inf)
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---------------------------------------------------------------------------
// any shape, on CUDA cores
// ---------------------------------------------------------------------------
struct PrefixSimpleParams {
  const __nv_bfloat16 *q, *kv;
  __nv_bfloat16 *out;
  const int32_t *row_pos, *row_page_off, *row_npages, *row_page_start, *pages;
  int *err;
  int32_t Hq, Hkv, D, P, num_pages;
  float scale_log2;
};

constexpr int kSimpleWarps = 8;
constexpr int kSimpleMaxDim = 512;

// A CTA a (row, query head): each warp takes every eighth key, lane l dims l, l + 32, ...
// with a softmax of its own, and the warps' sums are joined at the end.
__global__ void __launch_bounds__(kSimpleWarps * 32) prefix_simple_kernel(const PrefixSimpleParams p) {
  constexpr int N = kSimpleMaxDim / 32;
  __shared__ float part[kSimpleWarps][kSimpleMaxDim];
  __shared__ float max_of[kSimpleWarps], sum_of[kSimpleWarps];
  grid_dependency();
  const int64_t row = blockIdx.x / p.Hq;
  const int h = blockIdx.x - row * p.Hq, g = h / (p.Hq / p.Hkv);
  const int warp = threadIdx.x / 32, lane = lane_id();
  const int64_t pos = p.row_pos[row], start = p.row_page_start[row];
  const __nv_bfloat16 *q = p.q + (row * p.Hq + h) * p.D;
  float qv[N], o[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    qv[i] = lane + 32 * i < p.D ? __bfloat162float(q[lane + 32 * i]) * p.scale_log2 : 0.f;
    o[i] = 0.f;
  }
  float m = kNoMax, l = 0.f;
  for (int64_t j = warp; j <= pos; j += kSimpleWarps) {
    const int64_t slot = start + j, pi = slot / p.P;
    const int page = pi < p.row_npages[row] ? p.pages[p.row_page_off[row] + pi] : -1;
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) atomicOr(p.err, kErrBounds);
      continue;
    }
    const __nv_bfloat16 *k = p.kv + (static_cast<int64_t>(page) * p.P + slot % p.P) * 2 * p.Hkv * p.D + g * p.D;
    const __nv_bfloat16 *v = k + p.Hkv * p.D;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (lane + 32 * i < p.D) s = fmaf(qv[i], __bfloat162float(k[lane + 32 * i]), s);
#pragma unroll
    for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    const float top = fmaxf(m, s), keep = exp2_approx(m - top), e = exp2_approx(s - top);
    m = top;
    l = l * keep + e;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (lane + 32 * i < p.D) o[i] = fmaf(e, __bfloat162float(v[lane + 32 * i]), o[i] * keep);
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (lane + 32 * i < p.D) part[warp][lane + 32 * i] = o[i];
  if (lane == 0) max_of[warp] = m, sum_of[warp] = l;
  __syncthreads();
  float top = max_of[0], total = 0.f;
  for (int w = 1; w < kSimpleWarps; ++w) top = fmaxf(top, max_of[w]);
  for (int w = 0; w < kSimpleWarps; ++w) total += sum_of[w] * exp2_approx(max_of[w] - top);
  for (int d = threadIdx.x; d < p.D; d += kSimpleWarps * 32) {
    float sum = 0.f;
    for (int w = 0; w < kSimpleWarps; ++w) sum += part[w][d] * exp2_approx(max_of[w] - top);
    p.out[(row * p.Hq + h) * p.D + d] = __float2bfloat16_rn(sum / total);
  }
}

// ---------------------------------------------------------------------------
// plans
// ---------------------------------------------------------------------------
// Positions from the first on that spans a and b hold in the same slots of the same pages.
int64_t common_tokens(const dsa_plan_t &plan, const PlanSpan &a, const PlanSpan &b, int32_t page_size) {
  if (a.page_start != b.page_start) return 0;
  const int32_t *pa = plan.host_pages + a.page_off, *pb = plan.host_pages + b.page_off;
  int64_t n = std::min(a.num_pages, b.num_pages), i = 0;
  while (i < n && pa[i] == pb[i]) ++i;
  return std::min<int64_t>(std::max<int64_t>(i * page_size - a.page_start, 0), std::min(a.ctx_start, b.ctx_start));
}

constexpr int64_t kMinShared = 128;   // a found prefix has a tile of keys at least

// Runs of spans that start with the same pages: a run grows as long as that saves reads.
void find_prefixes(const dsa_plan_t &plan, int32_t page_size, std::vector<dsa_prefix_t> &out) {
  const int32_t n = static_cast<int32_t>(plan.spans.size());
  for (int32_t i = 0; i < n;) {
    int64_t tokens = INT32_MAX, saved = 0;
    int32_t j = i + 1;
    for (; j < n; ++j) {
      const int64_t t = std::min(tokens, common_tokens(plan, plan.spans[i], plan.spans[j], page_size));
      if (t < kMinShared || t * (j - i) <= saved) break;
      tokens = t, saved = t * (j - i);
    }
    if (j > i + 1) out.push_back(dsa_prefix_t{i, j - i, static_cast<int32_t>(tokens), 0});
    i = j;
  }
}

}  // namespace

dsa_status make_prefix_plan(const dsa_ctx *ctx, const dsa_plan_t *plan, const dsa_msa_shape_t &shape, const dsa_prefix_t *prefixes,
                            int32_t n, cudaStream_t, dsa_prefix_plan_t *pp) {
  const int32_t spans = static_cast<int32_t>(plan->spans.size()), P = ctx->cfg.page_size;
  pp->plan = plan, pp->shape = shape;
  if (n < 0) {
    find_prefixes(*plan, P, pp->prefixes);
  } else {
    int32_t next = 0;
    for (int32_t i = 0; i < n; ++i) {
      const dsa_prefix_t &x = prefixes[i];
      if (x.reserved != 0 || x.first_span < next || x.num_spans < 1 || x.num_spans > spans - x.first_span || x.tokens < 0)
        return DSA_ERR_INVALID_ARG;
      next = x.first_span + x.num_spans;
      const PlanSpan &a = plan->spans[x.first_span];
      for (int32_t j = x.first_span; j < next; ++j)
        if (common_tokens(*plan, a, plan->spans[j], P) < x.tokens) return DSA_ERR_INVALID_ARG;
      if (x.tokens > 0) pp->prefixes.push_back(x);
    }
  }
  for (const PlanSpan &s : plan->spans) pp->tokens_read += s.ctx_start + s.q_len;
  for (const dsa_prefix_t &x : pp->prefixes) pp->tokens_read -= static_cast<int64_t>(x.tokens) * (x.num_spans - 1);
  return DSA_OK;
}

cudaError_t launch_prefix_attend(const dsa_ctx *ctx, const dsa_prefix_plan_t *pp, const void *q, const void *kv, float sm_scale,
                                 void *out, cudaStream_t s, int32_t *launches) {
  const dsa_plan_t &plan = *pp->plan;
  PrefixSimpleParams p{};
  p.q = static_cast<const __nv_bfloat16 *>(q), p.kv = static_cast<const __nv_bfloat16 *>(kv);
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.row_pos = plan.row_pos, p.row_page_off = plan.row_page_off, p.row_npages = plan.row_npages;
  p.row_page_start = plan.row_page_start, p.pages = plan.pages, p.err = ctx->err;
  p.Hq = pp->shape.q_heads, p.Hkv = pp->shape.kv_heads, p.D = pp->shape.head_dim, p.P = ctx->cfg.page_size;
  p.num_pages = plan.cache_pages, p.scale_log2 = sm_scale * kPrefixLog2e;
  *launches += 1;
  return launch_overlapped(prefix_simple_kernel, dim3(static_cast<unsigned>(plan.T) * p.Hq), kSimpleWarps * 32, 0, 1, s, p);
}

}  // namespace dsa

using namespace dsa;

extern "C" {

dsa_status dsa_prefix_plan(dsa_ctx_t *ctx, const dsa_plan_t *plan, const dsa_msa_shape_t *shape, const dsa_prefix_t *prefixes,
                           int32_t num_prefixes, dsa_stream_t stream, dsa_prefix_plan_t **out) {
  if (!out) return DSA_ERR_INVALID_ARG;
  *out = nullptr;
  if (!ctx || !plan || plan->ctx != ctx || !shape || num_prefixes < -1 || (num_prefixes > 0 && !prefixes) || shape->reserved != 0 ||
      shape->kv_heads < 1 || shape->q_heads < 1 || shape->head_dim < 1 || shape->q_heads % shape->kv_heads != 0)
    return DSA_ERR_INVALID_ARG;
  if (plan->capturable || shape->head_dim > kSimpleMaxDim || shape->q_heads > 1024 ||
      static_cast<int64_t>(plan->T) * shape->q_heads > INT32_MAX)
    return DSA_ERR_UNSUPPORTED;
  dsa_prefix_plan_t *pp = new (std::nothrow) dsa_prefix_plan_t();
  if (!pp) return DSA_ERR_OOM;
  dsa_status st;
  try {
    st = make_prefix_plan(ctx, plan, *shape, prefixes, num_prefixes, reinterpret_cast<cudaStream_t>(stream), pp);
  } catch (...) {   // std::bad_alloc
    st = DSA_ERR_OOM;
  }
  if (st != DSA_OK) {
    dsa_prefix_plan_destroy(pp);
    return st;
  }
  *out = pp;
  return DSA_OK;
}

void dsa_prefix_plan_destroy(dsa_prefix_plan_t *pp) {
  if (!pp) return;
  delete pp;
}

dsa_status dsa_prefix_plan_get_info(const dsa_prefix_plan_t *pp, dsa_prefix_info_t *info) {
  if (!pp || !info) return DSA_ERR_INVALID_ARG;
  *info = dsa_prefix_info_t{};
  info->num_prefixes = static_cast<int32_t>(pp->prefixes.size());
  info->tokens_read = pp->tokens_read;
  return DSA_OK;
}

dsa_status dsa_prefix_attend(dsa_ctx_t *ctx, const dsa_prefix_plan_t *pp, const void *q, const void *kv_cache, float sm_scale,
                             void *out, dsa_stream_t stream) {
  if (!ctx || !pp || pp->plan->ctx != ctx || ctx->device < 0 || !(sm_scale >= 0.f) || !std::isfinite(sm_scale)) return DSA_ERR_INVALID_ARG;
  if (cudaSetDevice(ctx->device) != cudaSuccess) return DSA_ERR_CUDA;
  LaunchCount launched(ctx);
  if (pp->plan->T == 0) return DSA_OK;
  auto on16 = [](const void *p) { return p && reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  if (!on16(q) || !on16(kv_cache) || !on16(out)) return DSA_ERR_INVALID_ARG;
  return cuda_status(ctx, launch_prefix_attend(ctx, pp, q, kv_cache, sm_scale, out, reinterpret_cast<cudaStream_t>(stream),
                                               &launched.n));
}

}  // extern "C"
