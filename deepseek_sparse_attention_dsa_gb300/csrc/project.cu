// project.cu -- matrix product of e4m3 codes with fp32 scales per block of 128:
//
//   out[m, b, n] = sum_kb a_scale[m, b, kb] * w_scale[b, n / 128, kb]
//                  * sum_{k in block kb} a[m, b, k] * w[b, n, k]
//
// for b = 0 .. batch-1 (the heads of an absorbed projection; 1 otherwise).
//
// The scales change with every 128 of k, so the tensor core (tcgen05
// kind::f8f6f4) sums one block of 128 at a time into a tensor-memory buffer
// (four K = 32 steps) and the epilogue warps add the blocks up in registers:
// acc[col] += s * block[col], s = a_scale * w_scale.  Several buffers let the
// tensor core run ahead of that.  A block of 128 of every weight row has one
// scale for 128 rows, so a tile never needs more than one or two of them.
//
// project_tc_kernel, few rows: a tile is 128 weight rows (the MMA's 128 lanes) by
// NT = 16, 32 or 64 tokens (its columns); two helper warps put s for the tile's
// tokens into shared memory ahead of the epilogue.  Bound by the weights' bytes:
// 16 x 8192 x 8192 takes 12.9 us on one GB300 with the weights in DRAM, 67 MB at
// 5.2 TB/s, of which some 3 us are the first loads' latency and the last block's way
// out (8.2 us where they are in L2; 1 x 8192 x 2048: 5.4 and 3.9 us).
//
// project_rows_kernel, more rows: tokens are the lanes (see there).
//
// Few tiles: a cluster of S CTAs shares a tile, each taking a run of its k
// blocks.  The tile's tokens are dealt out to the ranks; every CTA sends its
// partial sums of a token to the token's owner (st.async, counted on the owner's
// mbarrier), which adds the S of them in rank order, so results do not depend on
// timing, and no CTA waits for another to finish (with the partial sums fetched
// from the other CTAs between two cluster barriers a call took 0.9 us longer).
//
// Warp roles: 0 TMA producer, 1 MMA issuer and tensor-memory owner, 2-3 scales,
// 4.. epilogue.  What their hand-overs cost decides the small tiles: a wait on a
// completed mbarrier is some 70 cycles, so the issuer tries both of its barriers
// in one go; arrivals that order nothing but completed reads are relaxed (with
// release semantics at cluster scope an arrival took 340 cycles, and over 1000
// beside TMA traffic: 770 us instead of 530 for 8192 x 8192 x 4096 at the time).
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "dsa_internal.h"
#include "fp8.cuh"
#include "ptx.cuh"

namespace dsa {
namespace {

struct ProjectParams {
  CUtensorMap tm_a;   // token codes as [rows][batch][k], box {128, 1, NT}, 128-byte swizzle
  CUtensorMap tm_w;   // weight codes as [batch][n][k], box {128, 128, 1}, 128-byte swizzle
  CUtensorMap tm_out; // out as [rows][batch][n], box {128 bytes, 1, 32}, 128-byte swizzle (where out_tma)
  const uint8_t *a, *w;
  const float *a_scale, *w_scale;
  void *out;
  const int32_t *count;
  int *err;
  int64_t rows;
  int64_t a_stride, a_batch, w_stride, w_batch, as_stride, as_batch, ws_stride, ws_batch, out_stride, out_batch;
  int32_t n, batch, per_row, out_type;
  int32_t k, kbs, split, split_log2;   // kbs: blocks of 128 of k; split: CTAs (pairs) of a cluster that share them
  bool out_vec;   // rows of out start on 16 bytes
  bool out_tma;   // TMA takes them: it stores whole boxes of live rows
};

__device__ __forceinline__ float4 ld_shared4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}

constexpr int kMaxSplit = 8;
// S partial sums of four values, `stride` bytes apart in this CTA's shared memory, in rank order.
__device__ __forceinline__ float4 sum_partials(uint32_t at, uint32_t stride, int split) {
  float4 v[kMaxSplit];
#pragma unroll
  for (int r = 0; r < kMaxSplit; ++r)
    if (r < split) v[r] = ld_shared4(at + r * stride);
  float4 sum = v[0];
#pragma unroll
  for (int r = 1; r < kMaxSplit; ++r)
    if (r < split) sum.x += v[r].x, sum.y += v[r].y, sum.z += v[r].z, sum.w += v[r].w;
  return sum;
}

template <int NT_>
struct ProjectTraits {
  static constexpr int NT = NT_;
  // A chunk is KC blocks of k: they arrive on one barrier, are multiplied into
  // neighbouring tensor-memory columns and handed over together, because each
  // hand-over costs the issuing warp some 400 cycles however small the block.
  static constexpr int KC = 2;
  static constexpr int EPI = NT == 64 ? 8 : 4;   // epilogue warps, a multiple of 4
  static constexpr int THREADS = 128 + 32 * EPI;
  static constexpr int COLS = NT / (EPI / 4);               // columns of an epilogue thread
  static constexpr int W_BYTES = 128 * 128, A_BYTES = NT * 128;
  static constexpr int BLOCK = W_BYTES + A_BYTES;           // one block of k of a stage: weights, tokens
  static constexpr int STAGE = KC * BLOCK;
  static constexpr int STAGES = NT == 64 ? 3 : 4;
  static constexpr int AB = 4;                              // tensor-memory buffers, each a chunk
  static constexpr int TMEM_COLS = AB * KC * NT;
  static constexpr int GK = 16, SG = 3;     // k blocks per scale slot (whole chunks), slots
  static constexpr int S_ROW = NT + 4;                      // floats of a k block's scales (+4: fewer bank conflicts)
  static constexpr int S_SLOT = GK * S_ROW * 4;
  static constexpr int S_VALS = NT * GK / 64;               // values a helper thread brings to a slot
  static constexpr uint32_t IDESC = mma_idesc(128, NT, 0u, false, false);   // kind::f8f6f4: format 0 = e4m3
  static constexpr int OFF_S = STAGES * STAGE;
  static constexpr int OFF_PART = OFF_S + SG * S_SLOT;      // partial sums (split): [rank][own token][weight row]
  static constexpr int OFF_BAR = OFF_PART + NT * 128 * 4;
  static constexpr int NBAR = 2 * STAGES + 2 * AB + 2 * SG + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(GK % KC == 0 && (TMEM_COLS & (TMEM_COLS - 1)) == 0 && TMEM_COLS <= 512, "chunks");
};

struct ProjectTile {
  int b, n0;
  int64_t m0;
};

// Tiles in order: tokens fastest, so that neighbouring CTAs share weights.
__device__ __forceinline__ ProjectTile tile_at(uint32_t t, uint32_t m_tiles, uint32_t n_tiles, int NT) {
  const uint32_t rest = m_tiles == 1 ? t : t / m_tiles, m = t - rest * m_tiles;
  const uint32_t b = rest < n_tiles ? 0 : rest / n_tiles;
  return {static_cast<int>(b), static_cast<int>(rest - b * n_tiles) * 128, static_cast<int64_t>(m) * NT};
}

__device__ __forceinline__ void store_out(const ProjectParams &p, int64_t m, int b, int n, float v) {
  const int64_t at = m * p.out_stride + b * p.out_batch + n;
  if (p.out_type == DSA_BF16) static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(v);
  else static_cast<float *>(p.out)[at] = v;
}

// Columns n .. n+3 of one row (n a multiple of 4).
__device__ __forceinline__ void store4(const ProjectParams &p, int64_t m, int b, int n, float4 v) {
  const int64_t at = m * p.out_stride + b * p.out_batch + n;
  if (p.out_vec && n + 4 <= p.n) {
    if (p.out_type == DSA_BF16)
      *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
    else
      *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = v;
    return;
  }
  const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < p.n) store_out(p, m, b, n + i, x[i]);
}

// The first of a rank's k blocks: they are dealt out evenly, the first kbs % split
// ranks having one more.  (A split is a power of two: a division at a kernel's
// start is on its way to the first load, and costs 0.1 us.)
__device__ __forceinline__ int first_block(const ProjectParams &p, int rank) {
  const int each = p.kbs >> p.split_log2;
  return each * rank + min(rank, p.kbs - (each << p.split_log2));
}

// Arrivals that barrier i takes, in the order of the kernels' barriers: one lane
// sets up each.  ctas: the CTAs whose epilogue warps hand buffers back.
template <typename C>
__device__ __forceinline__ uint32_t barrier_arrivals(int i, int ctas) {
  const int j = i - 2 * C::STAGES, k = j - 2 * C::AB;
  return j < C::AB ? 1 : k < 0 ? ctas * C::EPI : k < C::SG ? 64 : k < 2 * C::SG ? C::EPI : 1;
}

// How long a CTA that gave up stays.  The other CTAs that share its tile started
// with it and have as many blocks of k, none of 1 us, and then send their sums or
// give up themselves after one wait, a limit and its last tries.  (Pairs also
// meet at the end.)
__device__ __forceinline__ uint64_t stay_ns(int blocks) { return 2 * kWaitLimitNs + static_cast<uint64_t>(blocks) * 1000; }

template <int NT>
__global__ void __launch_bounds__(ProjectTraits<NT>::THREADS, 1) project_tc_kernel(const __grid_constant__ ProjectParams p) {
  using C = ProjectTraits<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (C::STAGES + s); };
  auto afull = [&](int b) { return bar0 + 8u * (2 * C::STAGES + b); };
  auto aempty = [&](int b) { return bar0 + 8u * (2 * C::STAGES + C::AB + b); };
  auto sfull = [&](int g) { return bar0 + 8u * (2 * C::STAGES + 2 * C::AB + g); };
  auto sempty = [&](int g) { return bar0 + 8u * (2 * C::STAGES + 2 * C::AB + C::SG + g); };
  const uint32_t partfull = bar0 + 8u * (2 * C::STAGES + 2 * C::AB + 2 * C::SG);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);
  const uint32_t aborted = sbase + C::OFF_MISC + 4;

  const int warp = threadIdx.x / 32;
  const int lane = lane_id();
  const int rank = p.split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int kb0 = first_block(p, rank), kb1 = first_block(p, rank + 1);

  launch_dependents();
  if (warp == 0) {
    if (lane < C::NBAR) mbar_init(bar0 + 8u * lane, barrier_arrivals<C>(lane, 1));
    if (lane == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  // the producer starts on the barriers that it has just made; the others wait
  // for them and for the tensor memory
  __syncwarp();
  if (warp == 0) {
    named_bar_arrive(1, C::THREADS);
  } else {
    tc_fence_before();
    named_bar_sync(1, C::THREADS);
    tc_fence_after();
  }
  if (p.split > 1) cluster_arrive_relaxed();   // (the barriers are fenced; nothing else is handed over)
  // (a row count in memory is an input; without one the first tile is known before the wait)
  if (p.count) grid_dependency_wait();
  const int64_t live = live_rows(p.rows, p.count, p.per_row);
  const uint32_t m_tiles = static_cast<uint32_t>((live + NT - 1) / NT);
  const uint32_t n_tiles = (p.n + 127) / 128;
  const uint32_t tiles = m_tiles * n_tiles * p.batch;
  const uint32_t t0 = blockIdx.x >> p.split_log2, t_step = gridDim.x >> p.split_log2;
  ProjectTile tile{};
  if (t0 < tiles) tile = tile_at(t0, m_tiles, n_tiles, NT);
  asm volatile("" ::"r"(tile.b), "r"(tile.n0), "l"(tile.m0));   // (not later)
  if (!p.count) grid_dependency_wait();
  const uint32_t tmem_base = warp == 0 ? 0 : *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    int st = 0;
    uint32_t ph = 0;
    bool ok = true;
    bool fresh = true;   // stages that have not been filled are not waited for
    for (uint32_t t = t0; t < tiles && ok; t += t_step) {
      if (t != t0) tile = tile_at(t, m_tiles, n_tiles, NT);
      for (int kb = kb0; kb < kb1; kb += C::KC) {
        if (!fresh && !(ok = mbar_wait_warp(empty(st), ph ^ 1, aborted, p.err))) break;
        if (elect_one()) {
          const int n = min(C::KC, kb1 - kb);
          mbar_arrive_expect_tx(full(st), n * C::BLOCK);
          uint32_t dst = sbase + st * C::STAGE;
          for (int j = 0; j < n; ++j, dst += C::BLOCK) {
            tma_load_3d(dst, &p.tm_w, (kb + j) * 128, tile.n0, tile.b, full(st));
            tma_load_3d(dst + C::W_BYTES, &p.tm_a, (kb + j) * 128, tile.b, static_cast<int32_t>(tile.m0), full(st));
          }
        }
        if (++st == C::STAGES) {
          st = 0;
          ph ^= 1;
          fresh = false;
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const uint64_t desc0 = smem_desc(sbase, 16, 1024, kSwizzle128);
    int st = 0;
    uint32_t ph = 0, i = 0;   // i: chunks so far
    bool ok = true;
    for (uint32_t t = t0; t < tiles && ok; t += t_step) {
      for (int kb = kb0; kb < kb1; kb += C::KC, ++i) {
        const uint32_t ab = i % C::AB;
        if (!(ok = mbar_wait_warp_both(full(st), ph, aempty(ab), (i / C::AB & 1) ^ 1, aborted, p.err))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t wd = desc0 + st * (C::STAGE >> 4);
          const uint32_t d = tmem_base + ab * (C::KC * NT);
#pragma unroll
          for (int j = 0; j < C::KC; ++j)
            if (kb + j < kb1) {
#pragma unroll
              for (int k = 0; k < 4; ++k)   // K = 32 codes (32 bytes) per step
                mma_f8<false>(d + j * NT, wd + j * (C::BLOCK >> 4) + 2 * k,
                              wd + j * (C::BLOCK >> 4) + (C::W_BYTES >> 4) + 2 * k, C::IDESC, k != 0 ? 1u : 0u);
            }
          mma_commit(empty(st));
          mma_commit(afull(ab));
        }
        if (++st == C::STAGES) {
          st = 0;
          ph ^= 1;
        }
      }
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ scales
    // thread: k block g of a slot and every (64 / GK)th token; the loads of
    // the next slot are in flight while this one waits for its turn.  (From L2:
    // the kernel may have been set up before its inputs were written, so none of
    // them is read-only for its whole life.)
    const int ht = threadIdx.x - 64;
    const int g = ht % C::GK, c0 = ht / C::GK;
    float sa[C::S_VALS], sw = 0.f;
    auto load = [&](const ProjectTile &tile, int kb) {
      const bool in = kb + g < kb1;
      sw = in ? __ldcg(p.w_scale + tile.b * p.ws_batch + tile.n0 / 128 * p.ws_stride + kb + g) : 0.f;
      const float *as = p.a_scale + tile.b * p.as_batch + kb + g;
#pragma unroll
      for (int j = 0; j < C::S_VALS; ++j) {
        const int64_t m = tile.m0 + c0 + j * (64 / C::GK);
        sa[j] = in && m < live ? __ldcg(as + m * p.as_stride) : 0.f;
      }
    };
    int sg = 0;
    uint32_t sph = 0;
    bool ok = true;
    if (t0 < tiles) load(tile, kb0);
    for (uint32_t t = t0; t < tiles && ok; t += t_step) {
      for (int kb = kb0; kb < kb1; kb += C::GK) {
        if (!(ok = mbar_wait_warp(sempty(sg), sph ^ 1, aborted, p.err))) break;
        float *slot = reinterpret_cast<float *>(smem + C::OFF_S + sg * C::S_SLOT) + g * C::S_ROW + c0;
#pragma unroll
        for (int j = 0; j < C::S_VALS; ++j) slot[j * (64 / C::GK)] = sa[j] * sw;
        mbar_arrive(sfull(sg));
        if (++sg == C::SG) {
          sg = 0;
          sph ^= 1;
        }
        if (kb + C::GK < kb1) load(tile, kb + C::GK);
        else if (t + t_step < tiles) load(tile = tile_at(t + t_step, m_tiles, n_tiles, NT), kb0);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3;
    const int col0 = (warp - 4) / 4 * C::COLS;
    const int nl = quad * 32 + lane;   // weight row within the tile
    if (p.split > 1) cluster_wait();   // the others are there (0.3 us, in the first loads' shade)
    int sg = 0;
    uint32_t sph = 0, i = 0;
    bool ok = true;
    for (uint32_t t = t0; t < tiles && ok; t += t_step) {
      float acc[C::COLS];
#pragma unroll
      for (int c = 0; c < C::COLS; ++c) acc[c] = 0.f;
      auto add = [&](const float *v, const float *srow) {
        const float4 *s4 = reinterpret_cast<const float4 *>(srow);
#pragma unroll
        for (int c = 0; c < C::COLS / 4; ++c) {
          const float4 sc = s4[c];
          acc[4 * c] = fmaf(v[4 * c], sc.x, acc[4 * c]);
          acc[4 * c + 1] = fmaf(v[4 * c + 1], sc.y, acc[4 * c + 1]);
          acc[4 * c + 2] = fmaf(v[4 * c + 2], sc.z, acc[4 * c + 2]);
          acc[4 * c + 3] = fmaf(v[4 * c + 3], sc.w, acc[4 * c + 3]);
        }
      };
      auto load = [&](uint32_t tb, float *v) {
        if (C::COLS == 16) tmem_ld16(tb, *reinterpret_cast<float(*)[16]>(v));
        else tmem_ld32(tb, *reinterpret_cast<float(*)[32]>(v));
      };
      for (int kb = kb0; kb < kb1 && ok; kb += C::GK) {
        if (!(ok = mbar_wait_warp(sfull(sg), sph, aborted, p.err))) break;
        const float *slot = reinterpret_cast<const float *>(smem + C::OFF_S + sg * C::S_SLOT) + col0;
        const int gn = min(C::GK, kb1 - kb);
        for (int g = 0; g < gn; g += C::KC, ++i) {
          const uint32_t ab = i % C::AB;
          if (!(ok = mbar_wait_warp(afull(ab), i / C::AB & 1, aborted, p.err))) break;
          tc_fence_after();
          const uint32_t tb = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + ab * (C::KC * NT) + col0;
          float v[C::KC][C::COLS];
#pragma unroll
          for (int j = 0; j < C::KC; ++j) load(tb + j * NT, v[j]);   // (past gn: old sums, not used)
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_relaxed(aempty(ab));   // everything is read: the buffer goes back
#pragma unroll
          for (int j = 0; j < C::KC; ++j)
            if (g + j < gn) add(v[j], slot + (g + j) * C::S_ROW);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sempty(sg));
        if (++sg == C::SG) {
          sg = 0;
          sph ^= 1;
        }
      }
      if (!ok) {
        if (p.split > 1) named_bar_arrive(2, 32 * C::EPI);   // the others may be on their way there
        break;
      }
      if (t != t0) tile = tile_at(t, m_tiles, n_tiles, NT);
      const int cols = static_cast<int>(min(live - tile.m0, static_cast<int64_t>(NT)));   // live tokens
      if (p.split == 1) {
        const int n = tile.n0 + nl;
        if (n < p.n) {
#pragma unroll
          for (int c = 0; c < C::COLS; ++c) {
            if (col0 + c >= cols) break;
            store_out(p, tile.m0 + col0 + c, tile.b, n, acc[c]);
          }
        }
        continue;
      }
      // token m of the tile belongs to rank m % split, as its token m / split
      const int split = p.split, sh = 31 - __clz(split), own = NT >> sh;   // (a power of two)
      const int mine = (cols - rank + split - 1) >> sh;
      if (warp == 4 && elect_one()) mbar_arrive_expect_tx(partfull, (split - 1) * max(mine, 0) * 512);
      const uint32_t part = sbase + C::OFF_PART + (rank * own * 128 + nl) * 4;
#pragma unroll
      for (int c = 0; c < C::COLS; ++c) {
        const int m = col0 + c;
        if (m >= cols) break;
        const uint32_t at = part + (m >> sh) * 512;
        const int to = m & (split - 1);
        if (to == rank) asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(acc[c]) : "memory");
        else st_async(map_to_cta(at, to), acc[c], map_to_cta(partfull, to));
      }
      named_bar_sync(2, 32 * C::EPI);
      if (!mbar_wait_warp<true>(partfull, 0, aborted, p.err)) break;   // the others' sums are there, and visible
      for (int i = threadIdx.x - 128; i < mine * 32; i += 32 * C::EPI) {   // a token, four weight rows
        const int m = i / 32, n4 = i % 32 * 4;
        const float4 sum = sum_partials(sbase + C::OFF_PART + (m * 128 + n4) * 4, own * 512, split);
        store4(p, tile.m0 + (m << sh) + rank, tile.b, tile.n0 + n4, sum);
      }
      break;   // one tile a cluster
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  linger_if_aborted(aborted, stay_ns(kb1 - kb0));
  if (warp == 1) tmem_dealloc(tmem_base, C::TMEM_COLS);
}

// ---------------------------------------------------------------------------
// More rows: tokens are the MMA's rows and lanes, weight rows its columns.  An
// epilogue thread then has one token and, its warp being on one weight block, s
// is one number per block of k; with weights on the lanes every column's s comes
// out of shared memory for every lane, which beyond 64 columns costs more of its
// bandwidth than the operands do (8192 x 8192 x 4096 on 128 x 128 tiles: 451 us
// with weights on the lanes, 257 with tokens).
//
//   kPair: a pair of CTAs (cta_group::2) on 256 tokens, 128 lanes in each, by N
//   weight rows; each CTA brings its tokens and half of the weights, so at N =
//   256 a block of k costs a CTA 32 KB for 128 x 256 x 128 products.
//   else: one CTA on 128 tokens by 128 weight rows.
//   SPLIT 2: two CTAs, or two pairs at N = 128, on the halves of a tile's k.  (Pairs
//   at N = 256 were slower split than whole: 512 x 4096 x 4096 14.4 us against 11.7
//   on smaller tiles; the partial sums of a CTA are then 64 KB.)
//
// Bounds, at 8192 x 8192 x 4096 (197 us, 2.79 PFLOP/s; 215 us when repeated, the
// card then at its power limit and 1.75 GHz): a block's 512 cycles of MMA, its
// way to the epilogue and back through two buffers, and 256 FMAs a scheduler;
// without the FMAs it took 169 us, without the loads too 142.  Tried and slower:
// packed FMAs (253 us), 16 epilogue warps (267 us: spills), the next block's
// first load before a block's last FMAs (loop-carried registers are copied).
// 128 x 128 tiles and N = 128 pairs are bound by operand reads from shared memory
// (540 and 410 cycles a block with neither loads nor FMAs, 64 bytes a cycle).
template <bool kPair_, int N_>
struct RowsTraits {
  static constexpr bool kPair = kPair_;
  static constexpr int N = N_, M = kPair ? 256 : 128;
  static constexpr int EPI = 8;                             // epilogue warps: 4 per half of the columns
  static constexpr int THREADS = 128 + 32 * EPI;
  static constexpr int COLS = N / 2;                        // columns of an epilogue thread
  static constexpr int W_ROWS = kPair ? N / 2 : N;
  static constexpr int A_BYTES = 128 * 128, W_BYTES = W_ROWS * 128;
  static constexpr int STAGE = A_BYTES + W_BYTES;
  static constexpr int STAGES = 4;                          // (powers of two, as AB: positions come out of one count)
  static constexpr int AB = 512 / N;                        // tensor-memory buffers, all its columns
  static constexpr int GK = 16, SG = 3;                     // k blocks per scale slot, slots
  static constexpr int S_ROW = 136;                         // floats of a k block's scales: 128 tokens, N / 128 weight blocks
  static constexpr int S_SLOT = GK * S_ROW * 4;
  static constexpr int TMEM_COLS = 512;
  static constexpr uint32_t IDESC = mma_idesc(M, N, 0u, false, false);
  static constexpr int OUT_WARP = 8192;                     // output staging of an epilogue warp: two boxes of 32 rows of 128 bytes
  static constexpr int OFF_OUT = STAGES * STAGE;
  static constexpr int OFF_S = OFF_OUT + EPI * OUT_WARP;
  static constexpr int OFF_BAR = OFF_S + SG * S_SLOT;
  static constexpr int NBAR = 2 * STAGES + 2 * AB + 2 * SG + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static_assert(SMEM <= 227 * 1024 && (COLS == 128 || 32 * COLS * 4 == OUT_WARP), "shared memory");
  // registers: 384 threads launch with 168 each (64,512); the split keeps that sum
  static constexpr int REGS_HELP = N == 256 ? 56 : 64, REGS_EPI = N == 256 ? 224 : 216;
  static_assert(128 * REGS_HELP + 32 * EPI * REGS_EPI <= 384 * 168, "registers");
};

__device__ __forceinline__ ProjectTile rows_tile_at(int t, int m_tiles, int n_tiles, int M, int N) {
  // groups of 8 token tiles, weights next, tokens within the group fastest:
  // the tiles that run together share both operands in L2
  // (divisions cost more than anything else between two tiles: one, where
  // there is one matrix and the group is whole)
  int b = 0;
  if (t >= m_tiles * n_tiles) {
    b = t / (m_tiles * n_tiles);
    t -= b * (m_tiles * n_tiles);
  }
  if (m_tiles == 1) return {b, t * N, 0};
  const int group = m_tiles <= 8 ? 0 : t / (8 * n_tiles);
  const int size = min(m_tiles - group * 8, 8);
  const int in_g = t - group * 8 * n_tiles;
  const int j = size == 8 ? in_g >> 3 : in_g / size;
  return {b, j * N, static_cast<int64_t>(group * 8 + in_g - j * size) * M};
}

// 32 rows of 128 bytes of columns from a swizzled box of shared memory to out, by one warp.
__device__ __noinline__ void write_box(const ProjectParams &p, const uint8_t *box, int lane, int es, int64_t m0,
                                       int64_t live, int b, int n0) {
  const int chunk = lane & 7, per = 16 / es, row0 = lane / 8;
  const int n = n0 + chunk * per;
  if (n >= p.n) return;
  uint4 u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = *reinterpret_cast<const uint4 *>(box + sw128_offset(row0 + 4 * i, chunk));
  uint8_t *out = static_cast<uint8_t *>(p.out) + ((m0 + row0) * p.out_stride + b * p.out_batch + n) * es;
  const int64_t step = 4 * p.out_stride * es;
  const bool whole = p.out_vec && n + per <= p.n;
#pragma unroll
  for (int i = 0; i < 8; ++i, out += step) {
    if (m0 + row0 + 4 * i >= live) return;
    if (whole) {
      *reinterpret_cast<uint4 *>(out) = u[i];
      continue;
    }
    const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (es == 4) {
        if (n + e < p.n) reinterpret_cast<uint32_t *>(out)[e] = w[e];
      } else {
        if (n + 2 * e < p.n) reinterpret_cast<uint16_t *>(out)[2 * e] = static_cast<uint16_t>(w[e]);
        if (n + 2 * e + 1 < p.n) reinterpret_cast<uint16_t *>(out)[2 * e + 1] = static_cast<uint16_t>(w[e] >> 16);
      }
    }
  }
}

template <bool kPair, int N, int SPLIT>
__global__ void __launch_bounds__(384, 1) project_rows_kernel(const __grid_constant__ ProjectParams p) {
  using C = RowsTraits<kPair, N>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (C::STAGES + s); };
  auto afull = [&](int b) { return bar0 + 8u * (2 * C::STAGES + b); };
  auto aempty = [&](int b) { return bar0 + 8u * (2 * C::STAGES + C::AB + b); };
  auto sfull = [&](int g) { return bar0 + 8u * (2 * C::STAGES + 2 * C::AB + g); };
  auto sempty = [&](int g) { return bar0 + 8u * (2 * C::STAGES + 2 * C::AB + C::SG + g); };
  const uint32_t partfull = bar0 + 8u * (2 * C::STAGES + 2 * C::AB + 2 * C::SG);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);
  const uint32_t aborted = sbase + C::OFF_MISC + 4;

  const int warp = threadIdx.x / 32;
  const int lane = lane_id();
  // the cluster: the CTAs, or pairs of neighbouring CTAs, that split a tile's k
  constexpr int CTAS = (kPair ? 2 : 1) * SPLIT, LOG2 = CTAS / 2;   // (1, 2 or 4)
  const int rank = CTAS > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int part = SPLIT > 1 ? (kPair ? rank / 2 : rank) : 0;      // of the k blocks
  const int lead = kPair && SPLIT > 1 ? rank & 2 : 0;              // the pair's first CTA
  const int half = kPair ? rank - lead : 0;                        // of the tile's tokens
  const int kb0 = SPLIT > 1 ? first_block(p, part) : 0, kb1 = SPLIT > 1 ? first_block(p, part + 1) : p.kbs;

  launch_dependents();
  if (warp == 0) {
    // (a pair's buffers: both CTAs' epilogue warps, on the first CTA's barrier)
    if (lane < C::NBAR) mbar_init(bar0 + 8u * lane, barrier_arrivals<C>(lane, kPair ? 2 : 1));
    if (lane == 0) *abort_flag = 0;
    fence_mbar_init();
    if (SPLIT > 1 && lane == C::NBAR - 1) mbar_arrive_expect_tx(partfull, C::EPI / 2 * C::OUT_WARP);
  }
  if (warp == 1) {
    if (kPair) {
      tmem_alloc_pair(smem_u32(tmem_slot), C::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
      tmem_relinquish();
    }
  }
  __syncwarp();
  if (kPair) {
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cluster_arrive_relaxed();   // (the barriers are fenced; nothing else is handed over)
  } else {
    // the producer starts on the barriers that it has just made; the others
    // wait for them and for the tensor memory
    if (warp == 0) {
      named_bar_arrive(1, C::THREADS);
    } else {
      tc_fence_before();
      named_bar_sync(1, C::THREADS);
      tc_fence_after();
    }
    if (SPLIT > 1) cluster_arrive_relaxed();
  }
  // (a row count in memory is an input; without one the first tile is known before the wait)
  if (p.count) grid_dependency_wait();
  const int64_t live = live_rows(p.rows, p.count, p.per_row);
  const int m_tiles = static_cast<int>((live + C::M - 1) / C::M);
  const int n_tiles = (p.n + N - 1) / N;
  const int tiles = m_tiles * n_tiles * p.batch;
  const int t0 = blockIdx.x >> LOG2;
  // (a cluster that splits k has one tile.  Said so to the compiler, pairs take
  // 9.4 us for 1031 x 704 x 5120, else 9.7; CTAs 10.2 and 9.9)
  auto next = [&](int t) { return SPLIT > 1 && kPair ? tiles : t + static_cast<int>(gridDim.x >> LOG2); };
  ProjectTile tile{};
  if (N == 128) {   // (at 256 columns there are no registers to keep it in)
    if (t0 < tiles) tile = rows_tile_at(t0, m_tiles, n_tiles, C::M, C::N);
    asm volatile("" ::"r"(tile.b), "r"(tile.n0), "l"(tile.m0));   // (not later)
  }
  if (kPair) cluster_wait();   // the others' barriers and tensor memory are ready
  if (!p.count) grid_dependency_wait();
  const uint32_t tmem_base = !kPair && warp == 0 ? 0 : *tmem_slot;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_HELP));
    if (warp == 0) {
      // ---------------------------------------------------------- producer (each CTA)
      int st = 0;
      uint32_t ph = 0;
      bool ok = true;
      bool fresh = true;   // stages that have not been filled are not waited for
      for (int t = t0; t < tiles && ok; t = next(t)) {
        if (N != 128 || t != t0) tile = rows_tile_at(t, m_tiles, n_tiles, C::M, C::N);
        const int m = static_cast<int>(tile.m0) + half * 128, n = tile.n0 + half * C::W_ROWS;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!fresh && !(ok = mbar_wait_warp(empty(st), ph ^ 1, aborted, p.err))) break;
          if (elect_one()) {
            const uint32_t dst = sbase + st * C::STAGE;
            if (kPair) {   // the first CTA's barrier counts both CTAs' bytes
              if (half == 0) mbar_arrive_expect_tx(full(st), 2 * C::STAGE);
              const uint32_t bar = map_to_cta(full(st), lead);
              tma_load_3d_pair(dst, &p.tm_a, kb * 128, tile.b, m, bar);
              tma_load_3d_pair(dst + C::A_BYTES, &p.tm_w, kb * 128, n, tile.b, bar);
            } else {
              mbar_arrive_expect_tx(full(st), C::STAGE);
              tma_load_3d(dst + C::A_BYTES, &p.tm_w, kb * 128, n, tile.b, full(st));
              tma_load_3d(dst, &p.tm_a, kb * 128, tile.b, m, full(st));
            }
          }
          __syncwarp();
          if (++st == C::STAGES) {
            st = 0;
            ph ^= 1;
            fresh = false;
          }
        }
      }
      // the last commits have arrived here before this CTA may leave
      for (int i = 0; kPair && i < C::STAGES && ok; ++i) {
        ok = mbar_wait_warp(empty(st), ph ^ 1, aborted, p.err);
        if (++st == C::STAGES) {
          st = 0;
          ph ^= 1;
        }
      }
    } else if (warp == 1 && half == 0) {
      // ---------------------------------------------------------- MMA issuer (a pair's first CTA)
      const uint64_t desc0 = smem_desc(sbase, 16, 1024, kSwizzle128);
      const uint32_t blocks = (t0 >= tiles ? 0u : 1u + (tiles - 1 - t0) / (gridDim.x >> LOG2)) * (kb1 - kb0);
#pragma unroll 1
      for (uint32_t i = 0; i < blocks; ++i) {   // the k blocks of all its tiles
        const uint32_t st = i % C::STAGES, ab = i % C::AB;
        if (!mbar_wait_warp_both(full(st), i / C::STAGES & 1, aempty(ab), (i / C::AB & 1) ^ 1, aborted, p.err)) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t ad = desc0 + st * (C::STAGE >> 4), wd = ad + (C::A_BYTES >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)   // K = 32 codes (32 bytes) per step
            mma_f8<kPair>(tmem_base + ab * N, ad + 2 * k, wd + 2 * k, C::IDESC, k != 0 ? 1u : 0u);
          if (kPair) {
            mma_commit_pair(empty(st), 3 << lead);
            mma_commit_pair(afull(ab), 3 << lead);
          } else {
            mma_commit(empty(st));
            mma_commit(afull(ab));
          }
        }
      }
    } else if (warp >= 2) {
      // ---------------------------------------------------------- scales (each CTA)
      // thread: k block g of a slot and every fourth token, copied without a
      // register in between; the weight blocks' scales go beside them
      const int ht = threadIdx.x - 64;
      const int g = ht % C::GK, c0 = ht / C::GK;
      int sg = 0;
      uint32_t sph = 0;
      bool ok = true;
      for (int t = t0; t < tiles && ok; t = next(t)) {
        if (N != 128 || t != t0) tile = rows_tile_at(t, m_tiles, n_tiles, C::M, C::N);
        const int m0 = static_cast<int>(tile.m0) + half * 128;
        for (int kb = kb0; kb < kb1; kb += C::GK) {
          if (!(ok = mbar_wait_warp(sempty(sg), sph ^ 1, aborted, p.err))) break;
          const uint32_t row = sbase + C::OFF_S + sg * C::S_SLOT + g * C::S_ROW * 4;
          if (kb + g < kb1) {
            const float *as = p.a_scale + tile.b * p.as_batch + kb + g;
#pragma unroll 4
            for (int c = c0; c < 128; c += 64 / C::GK)
              cp_async_4_zfill(row + c * 4, m0 + c < live ? as + (m0 + c) * p.as_stride : as, m0 + c < live ? 4 : 0);
            if (c0 < N / 128) {
              const int n = tile.n0 + c0 * 128;
              const float *ws = p.w_scale + tile.b * p.ws_batch + kb + g;
              cp_async_4_zfill(row + (128 + c0) * 4, n < p.n ? ws + n / 128 * p.ws_stride : ws, n < p.n ? 4 : 0);
            }
          }
          cp_async_mbar_arrive(sfull(sg));
          if (++sg == C::SG) {
            sg = 0;
            sph ^= 1;
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_EPI));
    const int quad = warp & 3;
    const int col0 = (warp - 4) / 4 * C::COLS;   // the warp's first column of the tile
    const uint32_t tb0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + col0;
    const int es = p.out_type == DSA_BF16 ? 2 : 4;
    uint8_t *stage_out = smem + C::OFF_OUT + (warp - 4) * C::OUT_WARP;
    int ab = 0, sg = 0;
    uint32_t aph = 0, sph = 0;
    bool ok = true;
    if (!kPair && SPLIT > 1) cluster_wait();   // the other CTA is there
    for (int t = t0; t < tiles && ok; t = next(t)) {
      float acc[C::COLS];
#pragma unroll
      for (int c = 0; c < C::COLS; ++c) acc[c] = 0.f;
      for (int kb = kb0; kb < kb1 && ok; kb += C::GK) {
        if (!(ok = mbar_wait_warp(sfull(sg), sph, aborted, p.err))) break;
        const float *slot = reinterpret_cast<const float *>(smem + C::OFF_S + sg * C::S_SLOT);
        const int gn = min(C::GK, kb1 - kb);
#pragma unroll 1
        for (int g = 0; g < gn; ++g) {
          if (!(ok = mbar_wait_warp(afull(ab), aph, aborted, p.err))) break;
          tc_fence_after();
          const uint32_t tb = tb0 + ab * N;
          const float sc = slot[g * C::S_ROW + quad * 32 + lane] * slot[g * C::S_ROW + 128 + col0 / 128];
          float v[2][32];
          tmem_ld32(tb, v[0]);
#pragma unroll
          for (int c = 0; c < C::COLS / 32; ++c) {
            tmem_ld_wait();
            if (c + 1 < C::COLS / 32) {
              tmem_ld32(tb + (c + 1) * 32, v[(c + 1) & 1]);
            } else {   // everything is read: the buffer goes back
              tc_fence_before();
              __syncwarp();
              if (lane == 0) {
                if (kPair) mbar_arrive_remote_relaxed(map_to_cta(aempty(ab), lead));
                else mbar_arrive_relaxed(aempty(ab));
              }
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[c * 32 + i] = fmaf(v[c & 1][i], sc, acc[c * 32 + i]);
          }
          if (++ab == C::AB) {
            ab = 0;
            aph ^= 1;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sempty(sg));
        if (++sg == C::SG) {
          sg = 0;
          sph ^= 1;
        }
      }
      if (!ok) break;
      tile = rows_tile_at(t, m_tiles, n_tiles, C::M, C::N);
      const int64_t mw = tile.m0 + half * 128 + quad * 32;   // the warp's first token
      const int nw = tile.n0 + col0;                         // and first column
      const uint32_t stage_addr = sbase + C::OFF_OUT + (warp - 4) * C::OUT_WARP;
      if (SPLIT > 1) {
        // two CTAs, or pairs, share the tile (one tile a cluster): part r finishes
        // what its CTAs hold of lanes 64 r .. 64 r + 63.  A warp of the other lanes
        // sends its sums into the staging of the same warp of the other part, four
        // columns of its 32 rows at a time.
        const uint32_t at = stage_addr + lane * 16;
        if (quad / 2 != part) {
          const int other = rank ^ (kPair ? 2 : 1);
          const uint32_t to = map_to_cta(at, other), bar = map_to_cta(partfull, other);
#pragma unroll
          for (int c = 0; c < C::COLS; c += 4) st_async4(to + c * 128, acc + c, bar);
          break;
        }
        if (!mbar_wait_warp<true>(partfull, 0, aborted, p.err)) break;
#pragma unroll
        for (int c = 0; c < C::COLS; c += 4) {
          const float4 v = ld_shared4(at + c * 128);
          acc[c] += v.x, acc[c + 1] += v.y, acc[c + 2] += v.z, acc[c + 3] += v.w;
        }
        __syncwarp();   // the staging is read before it is filled again
      }
      // out, through shared memory: boxes of 32 rows by 128 bytes of columns,
      // at most two at a time.  A TMA store takes them while the next tile is
      // under way; rows that TMA cannot take are written here, four to an
      // instruction.
      if (lane == 0) bulk_wait_read_all();     // the last tile's stores have read the boxes
      __syncwarp();
#pragma unroll
      for (int c0 = 0; c0 < C::COLS; c0 += 32) {   // half a box of bf16, a box of fp32
        uint8_t *dst = stage_out + (es == 2 ? c0 / 64 : c0 / 32 % 2) * 4096;
#pragma unroll
        for (int q = 0; q < 8; q += 2) {       // eight columns
          const float *x = acc + c0 + 4 * q;
          if (es == 2) {
            *reinterpret_cast<uint4 *>(dst + sw128_offset(lane, c0 % 64 / 8 + q / 2)) =
                make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
          } else {
            *reinterpret_cast<float4 *>(dst + sw128_offset(lane, q)) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4 *>(dst + sw128_offset(lane, q + 1)) = make_float4(x[4], x[5], x[6], x[7]);
          }
        }
        if (es == 2 ? c0 + 32 < C::COLS : c0 % 64 == 0) continue;
        const int n = es == 2 ? nw : nw + c0 - 32, per = 128 / es;   // the first box's first column, a box's columns
        const bool two = es == 4 || C::COLS == 128;
        // (what is past p.rows TMA drops, what is past the live rows it would write;
        // the vote makes the branch uniform for the compiler too)
        if (__all_sync(0xffffffffu, p.out_tma && (p.count == nullptr || mw + 32 <= live))) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && mw < live) {
            if (n < p.n) tma_store_3d(&p.tm_out, stage_addr, n, tile.b, static_cast<int32_t>(mw));
            if (two && n + per < p.n) tma_store_3d(&p.tm_out, stage_addr + 4096, n + per, tile.b, static_cast<int32_t>(mw));
            bulk_commit();
            if (c0 + 32 < C::COLS) bulk_wait_read_all();   // the boxes are filled once more
          }
          __syncwarp();
        } else {
          __syncwarp();
          write_box(p, stage_out, lane, es, mw, live, tile.b, n);
          if (two) write_box(p, stage_out + 4096, lane, es, mw, live, tile.b, n + per);
          __syncwarp();
        }
      }
    }
    if (lane == 0) bulk_wait_read_all();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  linger_if_aborted(aborted, stay_ns(kb1 - kb0));
  if (kPair) {
    cluster_arrive_relaxed();
    cluster_wait();   // no CTA leaves while another may signal it or read its operands
  }
  if (warp == 1) {
    if (kPair) tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    else tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

__device__ __forceinline__ float e4m3_value(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// CUDA-core form, for codes that are not on 16 bytes (or have a stride of 0): 64 x 64
// outputs a CTA, 4 x 4 a thread.  Right, and slow: a byte of codes a load, products on
// the FMA pipe, nothing of the next block in flight (8192 x 8192, k 4100: 22.2 ms where
// k 4096 takes 0.2 and 32-bit products of a library 8.6; 128 x 8192, k 4100: 436 us
// against 10; 1 x 8192, k 2052: 210 us against 5).
__global__ void __launch_bounds__(256) project_simt_kernel(const ProjectParams p) {
  __shared__ float as[32][65], ws[32][65];
  grid_dependency();
  const int64_t live = live_rows(p.rows, p.count, p.per_row);
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * 64;
  if (m0 >= live) return;
  const int n0 = blockIdx.y * 64, b = blockIdx.z;
  const uint8_t *a = p.a + b * p.a_batch, *w = p.w + b * p.w_batch;
  const float *as_ = p.a_scale + b * p.as_batch, *ws_ = p.w_scale + b * p.ws_batch;
  const int tm = threadIdx.x / 16, tn = threadIdx.x % 16;
  float acc[4][4] = {};
  for (int kb = 0; kb < p.kbs; ++kb) {
    float part[4][4] = {};
    const int width = min(p.k - kb * 128, 128);
    for (int j0 = 0; j0 < width; j0 += 32) {
      const int k0 = kb * 128 + j0;
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

// Tensor maps of both operands, box_a tokens and box_w weight rows a box.
bool encode_operands(const dsa_project_t &g, ProjectParams &p, uint32_t box_a, uint32_t box_w) {
  // a dimension of one element takes any stride
  auto stride = [](int64_t st, int64_t count) { return static_cast<uint64_t>(count > 1 ? st : 16); };
  const uint64_t a_dims[3] = {static_cast<uint64_t>(g.k), static_cast<uint64_t>(g.batch), static_cast<uint64_t>(g.rows)};
  const uint64_t a_strides[2] = {stride(g.a_batch, g.batch), stride(g.a_stride, g.rows)};
  const uint32_t a_box[3] = {128, 1, box_a};
  const uint64_t w_dims[3] = {static_cast<uint64_t>(g.k), static_cast<uint64_t>(g.n), static_cast<uint64_t>(g.batch)};
  const uint64_t w_strides[2] = {stride(g.w_stride, g.n), stride(g.w_batch, g.batch)};
  const uint32_t w_box[3] = {128, box_w, 1};
  return encode_tiled_3d(&p.tm_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<uint8_t *>(p.a), a_dims, a_strides, a_box,
                         CU_TENSOR_MAP_SWIZZLE_128B) &&
         encode_tiled_3d(&p.tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<uint8_t *>(p.w), w_dims, w_strides, w_box,
                         CU_TENSOR_MAP_SWIZZLE_128B);
}

cudaError_t launch(const dsa_ctx *ctx, void (*kern)(ProjectParams), int threads, int smem, int64_t grid, int cluster,
                   std::atomic<uint64_t> &smem_limit_set, const ProjectParams &p, cudaStream_t s) {
  if (cudaError_t e = ensure_smem_limit(kern, smem, ctx->device, smem_limit_set); e != cudaSuccess) return e;
  return launch_overlapped(kern, dim3(static_cast<unsigned>(grid)), threads, smem, cluster, s, p);
}

// Tiles of M tokens by N weight rows.
int64_t tiles_of(const dsa_project_t &g, int M, int N) {
  return (g.rows + M - 1) / M * ((static_cast<int64_t>(g.n) + N - 1) / N) * g.batch;
}

template <bool kPair, int N, int SPLIT>
cudaError_t run_rows(const dsa_ctx *ctx, const dsa_project_t &g, ProjectParams &p, cudaStream_t s) {
  using C = RowsTraits<kPair, N>;
  if (!encode_operands(g, p, 128, C::W_ROWS)) return cudaErrorInvalidValue;
  p.split = SPLIT, p.split_log2 = SPLIT / 2;
  if (p.out_vec) {
    const bool bf16 = g.out_type == DSA_BF16;
    const int64_t es = bf16 ? 2 : 4;
    const uint64_t dims[3] = {static_cast<uint64_t>(g.n), static_cast<uint64_t>(g.batch), static_cast<uint64_t>(g.rows)};
    const uint64_t strides[2] = {static_cast<uint64_t>(g.batch > 1 ? g.out_batch * es : 16),
                                 static_cast<uint64_t>(g.rows > 1 ? g.out_stride * es : 16)};
    const uint32_t box[3] = {static_cast<uint32_t>(128 / es), 1, 32};
    p.out_tma = encode_tiled_3d(&p.tm_out, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                                p.out, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  const int64_t tiles = tiles_of(g, C::M, N);
  const int cluster = (kPair ? 2 : 1) * SPLIT;
  const int64_t grid = SPLIT > 1 ? tiles * cluster : cluster * std::min<int64_t>(tiles, ctx->num_sms / cluster);
  static std::atomic<uint64_t> smem_limit_set{0};
  return launch(ctx, project_rows_kernel<kPair, N, SPLIT>, C::THREADS, C::SMEM, grid, cluster, smem_limit_set, p, s);
}

template <int NT>
cudaError_t run_tc(const dsa_ctx *ctx, const dsa_project_t &g, ProjectParams &p, int split, cudaStream_t s) {
  using C = ProjectTraits<NT>;
  if (!encode_operands(g, p, NT, 128)) return cudaErrorInvalidValue;
  p.split = split, p.split_log2 = split == 8 ? 3 : split / 2;
  const int64_t tiles = tiles_of(g, NT, 128);
  const int64_t grid = split > 1 ? tiles * split : std::min<int64_t>(tiles, ctx->num_sms);
  static std::atomic<uint64_t> smem_limit_set{0};
  return launch(ctx, project_tc_kernel<NT>, C::THREADS, C::SMEM, grid, split, smem_limit_set, p, s);
}

// Clusters of `ctas` CTAs, one to an SM, that the device holds at once: less than
// its SMs allow, as a cluster lies within a group of them (a GB300 with 152 SMs
// holds 36 of four and 15 of eight; 48 x 2048 x 8192 on 16 clusters of eight took
// 11.1 us, on as many of four 7.4).  Asked of the driver once a device, for
// project_tc_kernel<64>, and used for every form: all of them take more than half of
// an SM's shared memory, which makes it one CTA an SM whichever it is.
int clusters_at_once(const dsa_ctx *ctx, int ctas) {
  if (ctas <= 2) return ctx->num_sms / ctas;
  static std::atomic<int> known[64][2];
  const int dev = ctx->device < 64 ? ctx->device : 63, slot = ctas == 4 ? 0 : 1;
  int n = ctx->device < 64 ? known[dev][slot].load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  using C = ProjectTraits<64>;
  static std::atomic<uint64_t> smem_limit_set{0};
  if (ensure_smem_limit(project_tc_kernel<64>, C::SMEM, ctx->device, smem_limit_set) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas * ctx->num_sms);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, project_tc_kernel<64>, &cfg) != cudaSuccess) return 0;
  if (ctx->device < 64) known[dev][slot].store(n, std::memory_order_relaxed);
  return n;
}

// The kernel (tokens a tile: 16, 32, 64 with weights on the lanes; 128 on one
// CTA and 256 on a pair with tokens on the lanes, 257 the pair with 256 columns)
// and the CTAs, or pairs, that split a tile's k: the least of what a time for a block
// of k, one for a tile's end, one for a pair's start and one for a split (us) make of
// the blocks that the busiest CTA gets.  The times are a fit, by random search, to
// what every form took at 35 sizes with the weights partly in L2; at those the choice
// is within 1.5% of the best form.  At 30 sizes that had no part in it, drawn over
// the logarithms of 1-4000 rows, 256-24576 columns and k of 256-16384, it was within 4%
// at 28 and 19 and 21% slower at two, where more than two tiles of some forms fall to a
// CTA (2643 x 1984 x 608: {257} 10.0 us, {256} 8.4; 1829 x 5864 x 6192: {256} 82 us, {257}
// 68).  Measured on either side of its choices (us a call): 128 x 8192 x 4096 9.5 with
// {128, 2 CTAs}, 11.4 with {64}, 12.5 with {128};
// 200 x 4096 x 4096 8.2 with {256, 2 pairs}, 8.8 with {128, 2 CTAs}, 10.4 with {64};
// 256 x 8192 x 4096 13.0 with {256}, 13.1 with {128}, 16.6 with {257}; 1024 x 4096 x
// 4096 18.0 with {257}, 21.7 with {128}; 16 x 8192 x 2048 4.5 with {16, 2}, 5.0 with
// {16}.
void choose(const dsa_ctx *ctx, const dsa_project_t &g, int *nt, int *split) {
  struct Form {
    int nt, m, n, ctas, max_split;
    float block, tile, start;
  };
  static const Form forms[] = {{16, 16, 128, 1, 8, 0.17f, 0.18f, 0.f},    {32, 32, 128, 1, 8, 0.18f, 0.52f, 0.f},
                               {64, 64, 128, 1, 8, 0.26f, 0.91f, 0.f},    {128, 128, 128, 1, 2, 0.31f, 0.52f, 0.f},
                               {256, 256, 128, 2, 2, 0.27f, 0.52f, 0.16f}, {257, 256, 256, 2, 1, 0.46f, 0.50f, 0.15f}};
  const int kbs = (g.k - 1) / 128 + 1;
  float best = 0.f;
  *nt = 0;
  for (const Form &f : forms) {
    if (f.m < 64 && g.rows > 4 * f.m) continue;
    const int64_t tiles = tiles_of(g, f.m, f.n), cap = ctx->num_sms / f.ctas;
    if (f.m >= 128 && tiles >= INT32_MAX / 8) continue;   // (32-bit tile counts)
    for (int s = 1; s <= f.max_split; s *= 2) {
      if (s > 1 && (kbs < 2 * s || tiles > clusters_at_once(ctx, s * f.ctas))) break;
      const int64_t per_cta = s > 1 ? 1 : (tiles + cap - 1) / cap;
      const float t = static_cast<float>(per_cta) * (((kbs + s - 1) / s) * f.block + f.tile) + f.start + (s > 1 ? 0.64f : 0.f);
      if (*nt == 0 || t < best) best = t, *nt = f.nt, *split = s;
    }
  }
}

}  // namespace

bool project_tc_supported(const dsa_project_t &g, const void *a, const void *w) {
  auto on16 = [](int64_t stride, int64_t count) {
    return count <= 1 || (stride >= 16 && stride % 16 == 0 && stride < (int64_t(1) << 40));
  };
  return reinterpret_cast<uintptr_t>(a) % 16 == 0 && reinterpret_cast<uintptr_t>(w) % 16 == 0 &&
         on16(g.a_stride, g.rows) && on16(g.a_batch, g.batch) && on16(g.w_stride, g.n) && on16(g.w_batch, g.batch);
}

cudaError_t launch_project_fp8(const dsa_ctx *ctx, const dsa_project_t &g, const void *a, const float *a_scale,
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
  p.n = g.n, p.k = g.k, p.kbs = (g.k - 1) / 128 + 1;
  p.split = 1;
  p.batch = g.batch;
  p.out_type = g.out_type;
  p.err = ctx->err;
  const int64_t es = g.out_type == DSA_BF16 ? 2 : 4;
  p.out_vec = reinterpret_cast<uintptr_t>(out) % 16 == 0 && (g.rows == 1 || g.out_stride * es % 16 == 0) &&
              (g.batch == 1 || g.out_batch * es % 16 == 0);
  if (project_tc_supported(g, a, w)) {
    int nt, split;
    choose(ctx, g, &nt, &split);
    *launches += 1;
    switch (nt) {
      case 16: return run_tc<16>(ctx, g, p, split, s);
      case 32: return run_tc<32>(ctx, g, p, split, s);
      case 64: return run_tc<64>(ctx, g, p, split, s);
      case 128: return split > 1 ? run_rows<false, 128, 2>(ctx, g, p, s) : run_rows<false, 128, 1>(ctx, g, p, s);
      case 256: return split > 1 ? run_rows<true, 128, 2>(ctx, g, p, s) : run_rows<true, 128, 1>(ctx, g, p, s);
      default: return run_rows<true, 256, 1>(ctx, g, p, s);
    }
  }
  const dim3 grid(static_cast<unsigned>((g.rows + 63) / 64), (g.n + 63) / 64, g.batch);
  *launches += 1;
  return launch_overlapped(project_simt_kernel, grid, 256, 0, 1, s, p);
}

}  // namespace dsa
