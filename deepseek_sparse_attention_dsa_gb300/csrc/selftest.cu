// selftest.cu -- dsa_selftest_wait_timeout and dsa_selftest_warp_wait_timeout:
// the pipelines' bounded waits, made to run out on purpose.
//
// Every kernel of the library waits on mbarriers with mbar_wait, or a whole
// warp at a time with mbar_wait_warp and mbar_wait_warp_both (ptx.cuh), which
// give up after a time limit, set kErrTimeout in the context's error word and
// raise the CTA's abort flag so that every later wait of the CTA returns at
// once; the kernel then frees its tensor memory and exits, and the host reads
// DSA_ERR_TIMEOUT from dsa_get_error.  Nothing in a correct run reaches that
// path, so these entry points drive it directly: one CTA holds tensor memory,
// waits with a short limit on an mbarrier that nothing arrives on, waits on it
// again (which the raised abort flag must end at once), frees the tensor
// memory and exits.  No fault, trap or unbounded wait is involved.
#include <cuda_runtime.h>

#include "dsa_internal.h"
#include "ptx.cuh"

namespace dsa {
namespace {

__global__ void __launch_bounds__(64, 1) wait_timeout_kernel(int *err, uint64_t limit_ns, int64_t *result) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ int abort_flag;
  __shared__ uint32_t tmem_slot;
  const int warp = threadIdx.x / 32;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bar), 1);   // one arrival completes the phase; none comes
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&tmem_slot), 32);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  if (threadIdx.x == 32) {
    volatile int *flag = &abort_flag;
    const uint64_t t0 = globaltimer();
    const bool first = mbar_wait(smem_u32(&bar), 0, flag, err, limit_ns);
    const uint64_t t1 = globaltimer();
    const bool second = mbar_wait(smem_u32(&bar), 0, flag, err, limit_ns);
    const uint64_t t2 = globaltimer();
    result[0] = first ? 1 : 0;
    result[1] = static_cast<int64_t>(t1 - t0);
    result[2] = second ? 1 : 0;
    result[3] = static_cast<int64_t>(t2 - t1);
    result[4] = *flag;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem_base, 32);
}

// The same for the waits of a whole warp: each form runs out by itself on an
// abort flag of its own, and once more on the flag that it has raised.
__global__ void __launch_bounds__(64, 1) warp_wait_timeout_kernel(int *err, uint32_t limit_ns, int64_t *result) {
  __shared__ __align__(8) uint64_t never, done;
  __shared__ int abort_flag[4];
  __shared__ uint32_t tmem_slot;
  const int warp = threadIdx.x / 32;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&never), 1);   // one arrival completes the phase; none comes
    mbar_init(smem_u32(&done), 1);
    for (int i = 0; i < 4; ++i) abort_flag[i] = 0;
    fence_mbar_init();
    mbar_arrive(smem_u32(&done));
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&tmem_slot), 32);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  if (warp == 1) {
    const uint32_t n = smem_u32(&never), d = smem_u32(&done);
    auto wait = [&](int form, uint32_t flag) {
      switch (form) {
        case 0: return mbar_wait_warp(n, 0, flag, err, limit_ns);
        case 1: return mbar_wait_warp<true>(n, 0, flag, err, limit_ns);
        case 2: return mbar_wait_warp_both(n, 0, d, 0, flag, err, limit_ns);   // the first runs out, the second is complete
        default: return mbar_wait_warp_both(d, 0, n, 0, flag, err, limit_ns);
      }
    };
#pragma unroll 1
    for (int form = 0; form < 4; ++form) {
      const uint32_t flag = smem_u32(&abort_flag[form]);
      int64_t *r = result + 5 * form;
#pragma unroll 1
      for (int again = 0; again < 2; ++again) {
        __syncwarp();
        const uint64_t t0 = globaltimer();
        const uint32_t lanes = __ballot_sync(0xffffffffu, wait(form, flag));   // lanes that were told true: all or none
        const uint64_t t1 = globaltimer();
        if (lane_id() == 0) r[2 * again] = lanes, r[2 * again + 1] = static_cast<int64_t>(t1 - t0);
      }
      if (lane_id() == 0) r[4] = *reinterpret_cast<volatile int *>(&abort_flag[form]);
    }
    // a complete phase is one whatever the flag says
    const uint32_t flag = smem_u32(&abort_flag[0]);
    const uint32_t one = __ballot_sync(0xffffffffu, mbar_wait_warp(d, 0, flag, err, limit_ns));
    const uint32_t both = __ballot_sync(0xffffffffu, mbar_wait_warp_both(d, 0, d, 0, flag, err, limit_ns));
    if (lane_id() == 0) result[20] = one, result[21] = both;
    // what a CTA stays for once it gave up, and not otherwise (the last flag is down again)
    __syncwarp();
    if (lane_id() == 0) *reinterpret_cast<volatile int *>(&abort_flag[3]) = 0;
    __syncwarp();
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      const uint64_t t0 = globaltimer();
      linger_if_aborted(smem_u32(&abort_flag[3 * i]), limit_ns);
      __syncwarp();
      if (lane_id() == 0) result[22 + i] = static_cast<int64_t>(globaltimer() - t0);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem_base, 32);
}

// Checks the arguments, launches one CTA and reports.
template <typename Limit>
dsa_status run(void (*kern)(int *, Limit, int64_t *), dsa_ctx_t *ctx, uint64_t limit_ns, int64_t *result, dsa_stream_t stream) {
  if (!ctx || ctx->device < 0 || !result || limit_ns == 0 || limit_ns > kWaitLimitNs) return DSA_ERR_INVALID_ARG;
  if (cudaSetDevice(ctx->device) != cudaSuccess) return DSA_ERR_CUDA;
  kern<<<1, 64, 0, reinterpret_cast<cudaStream_t>(stream)>>>(ctx->err, static_cast<Limit>(limit_ns), result);
  ctx->last_launches = 1;
  return cuda_status(ctx, cudaGetLastError());
}

}  // namespace
}  // namespace dsa

extern "C" dsa_status dsa_selftest_wait_timeout(dsa_ctx_t *ctx, uint64_t limit_ns, int64_t *result,
                                                dsa_stream_t stream) {
  return dsa::run(dsa::wait_timeout_kernel, ctx, limit_ns, result, stream);
}

extern "C" dsa_status dsa_selftest_warp_wait_timeout(dsa_ctx_t *ctx, uint64_t limit_ns, int64_t *result,
                                                     dsa_stream_t stream) {
  return dsa::run(dsa::warp_wait_timeout_kernel, ctx, limit_ns, result, stream);
}
