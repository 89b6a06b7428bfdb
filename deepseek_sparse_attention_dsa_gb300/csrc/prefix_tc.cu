// prefix_tc.cu -- the attention over a shared prefix on the tensor cores.
//
// For a tile of 128 lanes (rows x heads of one kv head, so that the rows of many
// requests meet the same keys in one product) and tiles of 128 keys:
//     S = Q . K^T      (M = lanes, N = keys; both from shared memory)
//     P = 2^(S * sm_scale * log2 e - m)  in bf16, over S in tensor memory
//     O += P . V       (M = lanes, N = dims; A = P from tensor memory)
// with a reference maximum m per lane that moves only when a logit is more than
// 2^8 above it (O is rescaled then, in tensor memory).  A thread is a lane: its
// maximum and sum need no exchange.
//
// A CTA has two streams of steps, each with its S and O (all 512 columns): while one
// is in its softmax the tensor core works for the other.  Two tiles of queries over
// the same keys are the two streams of a pair (each key tile is loaded once for
// both); a lone tile's keys are given to the streams of many CTAs instead, each
// with keys of its own.  Warps 0-3 and 4-7: a stream's softmax; warps 8 and 10 load, by
// TMA into a ring of half-tiles (K or V of 128 keys); warp 9 issues the products.  A
// chain that more than one stream worked on leaves partial results, which
// prefix_join_kernel adds up in a fixed order.
//
// P is rounded to bf16 (half a step, 2^-8 of a weight; the sum l takes it unrounded), S, m,
// l and O are fp32.  Measured, 64 query heads over 4 of 128, bf16:
//   16 x 128 rows behind 16384 shared tokens   674 us, 1,657 TFLOP/s, 0.86 of a library product's burst and 0.95 of its
//                                              sustained rate
//   8192 rows of one sequence                  683 us, 1,609 TFLOP/s
//   256 rows on two documents of 32768         247 us (148 at the burst rate, 107 at a copy's)
//   32 rows behind 8192                        20.2 us (8.1 at a copy's rate; 22.1 with three sets of inputs in turn)
//   8 rows of 100000 tokens each alone         233 us, 7.0 TB/s
//   4 rows behind 1024                         7.2 us
// A pair's tile takes some 2,700 cycles, 2,048 of them the tensor core's; the others go
// between a step's last product and the next one's first, and to the softmax, whose
// way from S to the first weights (800 cycles) is about as long as the other
// stream's products.  Lone tiles wait for memory (5.9 TB/s over 256 x 1100 tokens); few rows
// for the first load (2 us), the partial results (2 us) and the join (3 to 4 us).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "fp8.cuh"
#include "prefix.h"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescale = 8.0f;        // log2 units that a logit may be above the reference maximum
constexpr float kNoMax = -3.0e38f;      // the reference maximum of a lane that has seen no key (finite: less -inf it is no NaN)
constexpr int kThreads = 352;
constexpr int kKeyWarp = 8, kMmaWarp = 9, kValueWarp = 10;

__device__ __forceinline__ float exp2_approx(float x) {   // (relative error 2^-22; 0 for -inf)
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void st_global8(void *p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// Four lanes' 128 bytes each, from a row a lane to the same quarter of four rows: b[i] is then this lane's 32 bytes
// of the i-th lane's row, so that a store of them fills whole lines.  (A lane a row, each store of a warp touched 32
// lines, and a pair's 128 KB of partial results took some 3 us in place of 2.)
__device__ __forceinline__ void across_quad(uint32_t (&b)[4][8]) {
#pragma unroll
  for (int d = 1; d <= 2; d <<= 1) {
    const bool upper = lane_id() & d;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & d) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? b[i][k] : b[i | d][k], d);
        (upper ? b[i][k] : b[i | d][k]) = got;
      }
    }
  }
}

struct PrefixParams {
  CUtensorMap tm_kv;   // cache as [pages * P, 2 * Hkv * D], box {64, BH}
  CUtensorMap tm_q;    // q as [T, Hq, D], box {64, group, rows_a_tile}
  CUtensorMap tm_q_small;   // the same, box {64, group, 64 / group}
  const PrefixSeg *segs;
  const PrefixCta *ctas;
  const int32_t *pages;
  __nv_bfloat16 *out;
  float *part_o;
  float2 *part_ml;
  int *err;
  int32_t Hq, Hkv, group, P, BH, q_bytes, q_small_bytes;
  float scale_log2;
};

template <int D>
struct Cfg {
  static constexpr int CH = D / 64;                     // 64-column chunks of a row
  static constexpr int CHUNK = kPrefixTile * 128;       // bytes: 128 rows of 64 columns
  static constexpr int HALF = CH * CHUNK;               // K or V of a tile
  static constexpr int NS = D == 128 ? 5 : 8;           // half-tiles in the ring
  static constexpr int SMALL = kPrefixTile / 2 * 128;   // second of two buffers of 64 lanes: into each chunk of a stream's Q
  // (queries first: a product over the second buffer reads 64 lanes past it, which are dead)
  static constexpr int OFF_RING = 2 * HALF;
  static constexpr int OFF_BAR = OFF_RING + NS * HALF;
  static constexpr int BARS = 2 * NS + 16;
  static constexpr int OFF_MISC = OFF_BAR + BARS * 8;
  static constexpr int BYTES = OFF_MISC + 16 + 1024;    // + alignment slack
  static constexpr uint32_t S_COL = 0, O_COL = 256;     // stream w's S at S_COL + 128 w, O at O_COL + 128 w
  static constexpr uint32_t IDESC_QK = mma_idesc(128, kPrefixTile, 1u, false, false);
  static constexpr uint32_t IDESC_PV = mma_idesc(128, D, 1u, false, true);
};

// Order of the ring's half-tiles.  A pair's key tile i: K, V at 2 i, 2 i + 1 of the phase.  The lone streams'
// steps t (stream t & 1): K(0), K(1), V(0), K(2), V(1), ... K(n - 1), V(n - 2), V(n - 1), the order of their use.
__device__ __forceinline__ int lone_k(int t) { return t > 0 ? 2 * t - 1 : 0; }
__device__ __forceinline__ int lone_v(int t, int n) { return t < n - 1 ? 2 * t + 2 : 2 * n - 1; }

// A place in the ring: its slot, and the parity of that slot's use.
template <int NS>
struct Ring {
  int st;
  uint32_t phase;
  __device__ __forceinline__ explicit Ring(int i) : st(i % NS), phase(static_cast<uint32_t>(i / NS) & 1u) {}
  __device__ __forceinline__ void skip(int n) {
    st += n;
    if (st >= NS) st -= NS, phase ^= 1u;
  }
};

// A walk over the tiles of a list of segments.  The next one's length is loaded a segment ahead: at its end it has
// looked at the two behind its list (two more lie behind the last of all lists).
struct Walk {
  const PrefixSeg *seg;
  int j, n, n_next;   // tile of the segment, its tiles, the next one's
  __device__ __forceinline__ void start(const PrefixSeg *s) { seg = s, j = 0, n = s->ntiles, n_next = s[1].ntiles; }
  __device__ __forceinline__ void next() {
    if (++j == n) seg += 1, j = 0, n = n_next, n_next = seg[1].ntiles;
  }
};
__device__ __forceinline__ void prefetch_seg(const PrefixSeg *s) {
  asm volatile("prefetch.global.L1 [%0];" ::"l"(s));
  asm volatile("prefetch.global.L1 [%0];" ::"l"(reinterpret_cast<const char *>(s) + sizeof(PrefixSeg) - 4));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prefix_tc_kernel(const __grid_constant__ PrefixParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem), bar0 = sbase + C::OFF_BAR;
  auto full = [&](int r) { return bar0 + 8u * (r % C::NS); };
  auto empty = [&](int r) { return bar0 + 8u * (C::NS + r % C::NS); };
  auto phase = [&](int r) { return static_cast<uint32_t>(r / C::NS) & 1u; };
  auto qfull = [&](int w, int b) { return bar0 + 8u * (2 * C::NS + 2 * w + b); };
  auto qempty = [&](int w, int b) { return bar0 + 8u * (2 * C::NS + 4 + 2 * w + b); };
  auto sfull = [&](int w) { return bar0 + 8u * (2 * C::NS + 8 + w); };
  auto pfull = [&](int w, int h) { return bar0 + 8u * (2 * C::NS + 10 + 2 * w + h); };   // h: the first 64 keys, the others
  auto ofull = [&](int w) { return bar0 + 8u * (2 * C::NS + 14 + w); };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);
  const uint32_t abort_addr = sbase + C::OFF_MISC + 4;
  const int warp = threadIdx.x / 32, lane = lane_id();

  if (threadIdx.x == 0) {
    for (int r = 0; r < C::NS; ++r) {
      mbar_init(full(r), 1);
      mbar_init(empty(r), 1);
    }
    for (int w = 0; w < 2; ++w) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(qfull(w, b), 1);
        mbar_init(qempty(w, b), 1);
      }
      mbar_init(sfull(w), 1);
      mbar_init(pfull(w, 0), 4);   // one arrival a warp
      mbar_init(pfull(w, 1), 4);
      mbar_init(ofull(w), 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_kv);
    tma_prefetch_desc(&p.tm_q);
    tma_prefetch_desc(&p.tm_q_small);
  }
  // (No kernel before, launched early as this one is, can still have to take its own tensor memory on this SM: those
  // that use it leave too little shared memory for this CTA.)
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  launch_dependents();
  const PrefixCta cta = p.ctas[blockIdx.x];   // (the plan's: nothing of this launch's stream writes it)
  const int na = cta.tiles_a, nb = cta.tiles_b;
  const bool small = cta.small != 0;

  if (warp == kKeyWarp || warp == kValueWarp) {
    // ------------------------------------------------------------ loads
    // A warp for the keys (and the queries) and one for the values, each with the ring's places of its own: a half-tile
    // takes some 1000 cycles of waits, look-ups and issue, and the products of lone tiles are done with two in less.
    // (Each waits for its slots in the ring's order and less than a round of it apart, which a parity tells.)
    const bool values = warp == kValueWarp;
    // A lane's box: box lane / CH of the tile, chunk lane % CH; its cache row, or -1
    const int box = lane / C::CH, chunk = lane % C::CH, boxes = kPrefixTile / p.BH;
    // (The page is looked at when the tile is loaded, a step later: the table's latency would hold up every load.  It is
    // one of the plan's, which were checked against the cache's size when it was made.)
    struct Box {
      int page, slot;
      __device__ __forceinline__ int row(int P) const { return page < 0 ? -1 : page * P + slot; }
    };
    auto lookup = [&](const Walk &k) {
      const PrefixSeg &s = *k.seg;
      const int q0 = s.slot0 + k.j * kPrefixTile + box * p.BH;
      Box x{-1, 0};
      if (box < boxes && q0 + p.BH > s.lo && q0 < s.hi) {
        const uint32_t pi = static_cast<uint32_t>(q0) / static_cast<uint32_t>(p.P);
        x.slot = q0 - static_cast<int>(pi) * p.P;
        x.page = p.pages[s.page_off + pi];
      }
      return x;
    };
    bool waited = false;      // for the kernels before: the plan's tables are read ahead of that, nothing else
    int last = -1;            // this warp's last place in the ring
    uint32_t q_loaded = 0, q_odd = 0;      // bit 2 w + b: stream w's buffer b has been loaded; an odd number of times
    bool ok = true;
    auto load = [&](int r, int x0, int row) {   // the ring's half-tile r, columns x0 ..
      if (!waited) grid_dependency_wait();
      waited = true;
      ok = ok && mbar_wait_warp(empty(r), phase(r) ^ 1u, abort_addr, p.err);
      if (!ok) return;
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, row >= 0)) * p.BH * 128;
      if (lane == 0) {
        if (bytes) mbar_arrive_expect_tx(full(r), bytes);
        else mbar_arrive(full(r));
      }
      __syncwarp();
      if (row >= 0) tma_load_2d(sbase + C::OFF_RING + (r % C::NS) * C::HALF + chunk * C::CHUNK + box * p.BH * 128, &p.tm_kv, x0 + chunk * 64, row, full(r));
      last = r;
    };
    // Stream w's queries: of a pair or a large tile into the whole of its buffer, of tiles of up to 64 lanes (`small`)
    // into one half and the other by turns, so that the next ones are there when the last ones are done with.
    auto load_q = [&](int w, const PrefixSeg *s, int tile, bool small, int b) {
      const uint32_t bit = 1u << (2 * w + b), busy = q_loaded & (small ? bit : 3u << (2 * w));
      for (int o = 0; o < 2; ++o)
        if (busy >> (2 * w + o) & 1) ok = ok && mbar_wait_warp(qempty(w, o), (q_odd >> (2 * w + o) & 1) ^ 1, abort_addr, p.err);
      if (!ok) return;
      if (lane == 0) {
        mbar_arrive_expect_tx(qfull(w, b), small ? p.q_small_bytes : p.q_bytes);
        for (int c = 0; c < C::CH; ++c)
          tma_load_3d(sbase + w * C::HALF + c * C::CHUNK + b * C::SMALL, small ? &p.tm_q_small : &p.tm_q, c * 64, s->g * p.group,
                      s->row[tile], qfull(w, b));
      }
      __syncwarp();
      q_loaded |= bit, q_odd ^= bit;
    };
    // (a tile's pages are looked up one tile ahead)
    if (na > 0) {
      Walk k;
      k.start(p.segs + cta.a0);
      Box ahead = lookup(k);
      for (int i = 0; i < na && ok; ++i) {
        const int row = ahead.row(p.P);
        const PrefixSeg *s = k.seg;
        const bool first = k.j == 0;
        k.next();
        if (i + 1 < na) ahead = lookup(k);
        load(2 * i + values, (values ? p.Hkv + s->g : s->g) * D, row);
        if (first && !values) {
          load_q(0, s, 0, false, 0);
          load_q(1, s, 1, false, 0);
        }
      }
    }
    if (nb > 0 && ok) {
      Walk k[2];
      int left[2] = {(nb + 1) / 2, nb / 2};
      Box ahead[2];
      uint32_t turn = 0;      // bit w: the buffer of stream w's next queries
      for (int w = 0; w < 2; ++w)
        if (left[w] > 0) {
          k[w].start(p.segs + cta.b0[w]);
          ahead[w] = lookup(k[w]);
        }
#pragma unroll 1
      for (int t0 = 0; t0 < nb && ok; t0 += 2) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int t = t0 + w;
          if (t >= nb) break;
          const PrefixSeg *s = k[w].seg;
          const bool first = k[w].j == 0;
          const int row = ahead[w].row(p.P);
          --left[w];
          k[w].next();
          if (left[w] > 0) ahead[w] = lookup(k[w]);
          load(2 * na + (values ? lone_v(t, nb) : lone_k(t)), (values ? p.Hkv + s->g : s->g) * D, row);
          if (first && !values) {
            prefetch_seg(s + 1);
            load_q(w, s, 0, small, turn >> w & 1);
            if (small) turn ^= 1u << w;
          }
        }
      }
    }
    // nothing of ours may still be landing when the CTA leaves (an abort apart, all of it has been used)
    if (lane == 0 && !ok) {
      volatile int no_abort = 0;
      for (int r = max(0, last - C::NS + 1); r <= last; ++r) {
        const int i = r - 2 * na;
        const bool value = i < 0 ? (r & 1) != 0 : i == 2 * nb - 1 || (i > 0 && i % 2 == 0);   // (of pairs, of lone_v)
        if (value == values) mbar_wait(full(r), phase(r), &no_abort, p.err);
      }
      for (int w = 0; w < 2; ++w)
        for (int b = 0; b < 2; ++b)
          if (q_loaded >> (2 * w + b) & 1) mbar_wait(qfull(w, b), (q_odd >> (2 * w + b) & 1) ^ 1, &no_abort, p.err);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    // One warp for both streams, so that half-tiles are awaited in the order in which they were asked for (a parity
    // says nothing of a fill two uses away).  The whole warp walks and waits, one elected thread issues: its operands
    // stay in uniform registers.  (Issued by a lane that a branch picked, each of the 16 instructions of a step took
    // some 80 cycles.)  The tensor core holds no more than a few products, so that the issue keeps its pace, and whatever
    // the warp does between two of them idles it: what the next step needs is looked at, and the walk goes on, ahead of a
    // step's last products (`peek`); what a step begins with is tried together.
    const uint64_t desc_q0 = smem_desc(sbase, 16, 1024, kSwizzle128), desc_k0 = smem_desc(sbase + C::OFF_RING, 16, 1024, kSwizzle128),
                   desc_v0 = smem_desc(sbase + C::OFF_RING, C::CHUNK, 1024, kSwizzle128);
    auto slot_full = [&](const Ring<C::NS> &r) { return bar0 + 8u * r.st; };
    auto slot_empty = [&](const Ring<C::NS> &r) { return bar0 + 8u * (C::NS + r.st); };
    grid_dependency_wait();      // (a barrier's time limit is for this kernel's own work, not for that of the kernels before)
    uint32_t q_phase = 0, p_phase = 0;      // bit 2 w + b: stream w's buffer b; bit w: stream w's
    uint32_t turn = 0;                      // bit w: the buffer of stream w's queries
    bool ok = true, met = false;            // met: what the next step begins with is there
    auto nothing = [] {};
    auto qk = [&](int w, const Ring<C::NS> r, bool first, bool last, bool release, bool halves, auto walk, auto peek) {
      const uint32_t b = (turn >> w) & 1;
      if (first) {
        ok = ok && mbar_wait_warp(qfull(w, b), (q_phase >> (2 * w + b)) & 1, abort_addr, p.err);
        q_phase ^= 1u << (2 * w + b);
        tc_fence_after();
      }
      if (last && halves) turn ^= 1u << w;
      if (!ok) return;
      const uint64_t q = desc_q0 + (w * C::HALF >> 4) + b * (C::SMALL >> 4), k = desc_k0 + r.st * (C::HALF >> 4);
      auto product = [&](int n) {
        const int at = (n >> 2) * (C::CHUNK >> 4) + 2 * (n & 3);
        mma_f16_ss(tmem + C::S_COL + w * 128, q + at, k + at, C::IDESC_QK, n > 0 ? 1u : 0u);
      };
      constexpr int N = 4 * C::CH, WALK = N / 2 - 1, PEEK = N - 2;
      if (elect_one()) {
#pragma unroll
        for (int n = 0; n < WALK; ++n) product(n);
      }
      __syncwarp();
      walk();
      if (elect_one()) {
#pragma unroll
        for (int n = WALK; n < PEEK; ++n) product(n);
      }
      __syncwarp();
      peek();
      if (elect_one()) {
#pragma unroll
        for (int n = PEEK; n < N; ++n) product(n);
        mma_commit(sfull(w));
        if (release) mma_commit(slot_empty(r));
        if (last) mma_commit(qempty(w, b));
      }
      __syncwarp();
    };
    // Whether the values, weights and (more) keys that stream w's step begins with are there.
    auto there = [&](int w, const Ring<C::NS> &v, const Ring<C::NS> &k, bool more) {
      const uint32_t ph = (p_phase >> w) & 1;
      return more ? mbar_test_warp_three(slot_full(v), v.phase, slot_full(k), k.phase, pfull(w, 0), ph)
                  : mbar_test_warp_both(slot_full(v), v.phase, pfull(w, 0), ph);
    };
    // Stream w's step: O += P V, and behind it (they run in order, and S's columns hold P) the next S of the stream.
    // walk: goes on to the next step; peek: looks at what it begins with.
    auto step = [&](int w, const Ring<C::NS> v, const Walk &kp, const Ring<C::NS> k, const Walk &kq, bool more, bool release,
                    bool halves, auto walk, auto peek) {
      const uint32_t ph = (p_phase >> w) & 1;
      if (!met) {
        if (more) ok = ok && mbar_wait_warp_three(slot_full(v), v.phase, slot_full(k), k.phase, pfull(w, 0), ph, abort_addr, p.err);
        else ok = ok && mbar_wait_warp_both(slot_full(v), v.phase, pfull(w, 0), ph, abort_addr, p.err);
      }
      p_phase ^= 1u << w;
      met = false;
      if (!ok) return;
      tc_fence_after();
      const uint64_t vd = desc_v0 + v.st * (C::HALF >> 4);
      const bool last = kp.j + 1 == kp.n, first = kp.j == 0, q_first = kq.j == 0, q_last = kq.j + 1 == kq.n;
      if (elect_one()) {
#pragma unroll
        for (int i = 0; i < 4; ++i)   // A: 16 keys are 8 columns; B read MN-major: 64-dim chunks CHUNK apart
          mma_f16_ts(tmem + C::O_COL + w * 128, tmem + C::S_COL + w * 128 + i * 8, vd + i * (16 * 128 >> 4), C::IDESC_PV,
                     (!first || i > 0) ? 1u : 0u);
      }
      __syncwarp();
      ok = mbar_wait_warp(pfull(w, 1), ph, abort_addr, p.err);
      if (!ok) return;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int i = 4; i < 8; ++i)
          mma_f16_ts(tmem + C::O_COL + w * 128, tmem + C::S_COL + w * 128 + i * 8, vd + i * (16 * 128 >> 4), C::IDESC_PV, 1u);
        if (release) mma_commit(slot_empty(v));
        if (last) mma_commit(ofull(w));
      }
      __syncwarp();
      if (more) {
        qk(w, k, q_first, q_last, release, halves, walk, peek);
      } else {
        walk();
        peek();
      }
    };
    if (na > 0) {
      Walk kq, kp;
      kq.start(p.segs + cta.a0);
      kp = kq;
      Ring<C::NS> rk(0), rv(1);
      ok = mbar_wait_warp(slot_full(rk), rk.phase, abort_addr, p.err);
      tc_fence_after();
      qk(0, rk, true, kq.n == 1, false, false, nothing, nothing);
      qk(1, rk, true, kq.n == 1, true, false, nothing, nothing);
      kq.next();
      rk.skip(2);
#pragma unroll 1
      for (int i = 0; i < na && ok; ++i) {
        const bool more = i + 1 < na;
        step(0, rv, kp, rk, kq, more, false, false, nothing, [&] { met = there(1, rv, rk, more); });
        step(
            1, rv, kp, rk, kq, more, true, false,
            [&] {
              rv.skip(2);
              kp.next();
              if (more) {
                kq.next();
                rk.skip(2);
              }
            },
            [&] { met = more && there(0, rv, rk, i + 2 < na); });
      }
      met = false;
    }
    if (nb > 0 && ok) {
      Walk kq[2], kp[2];
      Ring<C::NS> rk(2 * na), rv(2 * na + lone_v(0, nb));
#pragma unroll
      for (int w = 0; w < 2; ++w)
        if (w < nb) {
          kq[w].start(p.segs + cta.b0[w]);
          kp[w] = kq[w];
          ok = ok && mbar_wait_warp(slot_full(rk), rk.phase, abort_addr, p.err);
          tc_fence_after();
          qk(w, rk, true, kq[w].n == 1, true, small, nothing, nothing);
          kq[w].next();
          rk.skip(w + 1);      // K(0), K(1), then every other half-tile
        }
#pragma unroll 1
      for (int t = 0; t < nb && ok; t += 2) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int u = t + w;
          if (u < nb) {
            const bool more = u + 2 < nb;
            step(
                w, rv, kp[w], rk, kq[w], more, true, small,
                [&] {
                  kp[w].next();
                  rv.skip(more ? 2 : 1);
                  if (more) {
                    kq[w].next();
                    rk.skip(2);
                  }
                },
                [&] { met = u + 1 < nb && there(w ^ 1, rv, rk, u + 3 < nb); });
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int w = warp >> 2;
    const int i = (warp & 3) * 32 + lane;   // lane of the tile
    const uint32_t t_lane = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t t_s = t_lane + C::S_COL + w * 128, t_o = t_lane + C::O_COL + w * 128;
    const int own_row = i / p.group, own_head = i - own_row * p.group;
    int s_waits = 0, o_waits = 0;
    bool ok = true;
    grid_dependency_wait();      // (before the first store)
    // The pairs' segments, then this stream's own (in one loop: the code is large enough to miss the instruction
    // cache).
    const int n_a = cta.a1 - cta.a0, n_b = cta.b1[w] - cta.b0[w];
    auto seg_at = [&](int k) { return p.segs + (k < n_a ? cta.a0 + k : cta.b0[w] + k - n_a); };
    int done = 0;      // key tiles of the part before this segment
#pragma unroll 1
    for (int n_seg = 0; n_seg < n_a + n_b; ++n_seg) {
      const bool lone = n_seg >= n_a;
      if (n_seg == n_a) done = 0;
      const PrefixSeg &s = *seg_at(n_seg);
      const int tile = lone ? 0 : w;
      const bool zero = lone || w == 0;      // whether this stream clears values that no lane sees
      const int limit = s.causal ? s.limit[tile] + own_row : s.hi;
      const int least = s.causal ? s.limit[tile] : s.hi;   // every lane sees the slots below
      const int n = s.ntiles, lo = s.lo, hi = s.hi, slot0 = s.slot0, part = s.part[tile], lanes = s.lanes[tile];
      const int out_row = (s.row[tile] + own_row) * p.Hq + s.g * p.group + own_head;   // (rows x heads are below 2^31)
      if (n_seg + 1 < n_a + n_b) prefetch_seg(seg_at(n_seg + 1));
      // a warp without live lanes leaves P as it is (what comes of it stays in dead lanes of O) and only keeps step
      const bool dead = (warp & 3) * 32 >= lanes;
      float m = kNoMax, l = 0.f;
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        const int t0 = slot0 + j * kPrefixTile;
        ok = mbar_wait_warp(sfull(w), s_waits & 1, abort_addr, p.err);
        ++s_waits;
        if (!ok) break;
        tc_fence_after();
        // values of slots that no lane sees are cleared once they are there (a zero weight must not meet what
        // they hold, or what an unloaded box left)
        if (zero && (t0 < lo || t0 + kPrefixTile > hi)) {
          const int r = lone ? 2 * na + lone_v(2 * (done + j) + w, nb) : 2 * (done + j) + 1;
          ok = mbar_wait_warp(full(r), phase(r), abort_addr, p.err);
          if (!ok) break;
          const int before = max(lo - t0, 0), from = min(hi - t0, kPrefixTile);   // rows [0, before) and [from, 128)
          const uint32_t v = sbase + C::OFF_RING + (r % C::NS) * C::HALF;
#pragma unroll 1
          for (int k = i; k < (before + kPrefixTile - from) * 8; k += 128) {
            const uint32_t at = v + (k + (k >> 3 >= before ? (from - before) * 8 : 0)) * 16;
#pragma unroll
            for (int c = 0; c < C::CH; ++c) st_shared_v4(at + c * C::CHUNK, make_uint4(0u, 0u, 0u, 0u));
          }
          fence_proxy_async_smem();
        }
        if (dead) {
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(pfull(w, 0));
            mbar_arrive(pfull(w, 1));
          }
          continue;
        }
        if (t0 < lo || t0 + kPrefixTile > least) {
          // slots that the lane does not see, in tensor memory: kept out of the unrolled code below
#pragma unroll 1
          for (int c0 = 0; c0 < kPrefixTile; c0 += 16) {
            const int s0 = t0 + c0;
            if (s0 >= lo && s0 + 16 <= least) continue;
            float v[16];
            if (s0 + 16 > lo && s0 < hi) {
              tmem_ld16(t_s + c0, v);
              tmem_ld_wait();
            }
#pragma unroll
            for (int c = 0; c < 16; ++c)
              if (s0 + c < lo || s0 + c >= min(limit, hi)) v[c] = -INFINITY;
            tmem_st16(t_s + c0, v);
          }
          tmem_st_wait();
        }
        // Half of S at a time in registers (all of it, 128, leaves too few for the rest and spills): the maximum of the
        // upper half, then of the lower one, whose weights are made from the same registers while the upper half
        // comes again.
        float x[64], mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int h = 1; h >= 0; --h) {
          tmem_ld32(t_s + h * 64, *reinterpret_cast<float(*)[32]>(x));
          tmem_ld32(t_s + h * 64 + 32, *reinterpret_cast<float(*)[32]>(x + 32));
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 64; c += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = fmaxf(fmaxf(mx[k], x[c + k]), x[c + 4 + k]);
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
        const bool move = top > m + kRescale;
        if (__any_sync(0xffffffffu, move)) {
          const float keep = move ? exp2_approx(m - top) : 1.f;
          m = move ? top : m;
          l *= keep;
          // (every earlier product into O is complete: this S was issued after it)
          if (j > 0) {
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float o[16];
              tmem_ld16(t_o + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] *= keep;
              tmem_st16(t_o + c, o);
            }
          }
        }
        // the weights, 64 keys at a time: the product starts on the first of them
        const uint64_t scale2 = f2_pack(p.scale_log2, p.scale_log2), minus2 = f2_pack(-m, -m);
        uint64_t sum[2] = {f2_pack(l, 0.f), f2_pack(0.f, 0.f)};
        auto weights = [&](int q, const float *v) {      // of 32 keys; they lie over columns of S that have been read
          uint32_t packed[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            float a, b;
            f2_unpack(f2_fma(f2_pack(v[2 * c], v[2 * c + 1]), scale2, minus2), a, b);
            a = exp2_approx(a), b = exp2_approx(b);
            sum[c & 1] = f2_add(sum[c & 1], f2_pack(a, b));
            packed[c] = pack_bf16(a, b);
          }
          tmem_st16(t_s + q * 16, packed);
        };
        auto hand_over = [&](int h) {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(pfull(w, h));
        };
        float y[32];
        tmem_ld32(t_s + 64, y);
        weights(0, x);
        weights(1, x + 32);
        hand_over(0);
        tmem_ld_wait();
        tmem_ld32(t_s + 96, *reinterpret_cast<float(*)[32]>(x));
        weights(2, y);
        tmem_ld_wait();
        weights(3, x);
        hand_over(1);
        float a, b;
        f2_unpack(f2_add(sum[0], sum[1]), a, b);
        l = a + b;
      }
      ok = ok && mbar_wait_warp(ofull(w), o_waits & 1, abort_addr, p.err);
      ++o_waits;
      if (!ok) break;
      done += n;
      tc_fence_after();
      // Many rows: whole lines, for some 300 shuffles (8192 rows of one sequence 732 us against 785); few: a row a lane,
      // which is over sooner (4 rows behind 1024 tokens 7.3 us against 8.0).
      if (lanes > kPrefixTile / 2) {
        if (!dead) {
          const float scale = part < 0 ? 1.f / l : 1.f;
          const int quad = i & ~3, quarter = lane & 3;
#pragma unroll 1
          for (int c = 0; c < D; c += 64) {
            float o[64];
            tmem_ld32(t_o + c, *reinterpret_cast<float(*)[32]>(o));
            tmem_ld32(t_o + c + 32, *reinterpret_cast<float(*)[32]>(o + 32));
            tmem_ld_wait();
            uint32_t b[4][8];
            if (part < 0) {
#pragma unroll
              for (int k = 0; k < 32; ++k) b[k / 8][k % 8] = pack_bf16(o[2 * k] * scale, o[2 * k + 1] * scale);
              across_quad(b);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const int to = __shfl_sync(0xffffffffu, out_row, (lane & ~3) + r);
                if (quad + r < lanes) {      // (the output is on 16 bytes)
                  uint4 *at = reinterpret_cast<uint4 *>(p.out + static_cast<int64_t>(to) * D + c + quarter * 16);
                  at[0] = make_uint4(b[r][0], b[r][1], b[r][2], b[r][3]);
                  at[1] = make_uint4(b[r][4], b[r][5], b[r][6], b[r][7]);
                }
              }
            } else {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int k = 0; k < 32; ++k) b[k / 8][k % 8] = __float_as_uint(o[h * 32 + k]);
                across_quad(b);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                  if (quad + r < lanes) st_global8(p.part_o + (static_cast<int64_t>(part) + quad + r) * D + c + h * 32 + quarter * 8, b[r]);
              }
            }
          }
        }
      } else if (!dead) {
        const float scale = part < 0 ? 1.f / l : 1.f;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld32(t_o + c, o);
          tmem_ld_wait();
          if (i < lanes && part < 0) {
#pragma unroll
            for (int k = 0; k < 32; k += 8)
              *reinterpret_cast<uint4 *>(p.out + static_cast<int64_t>(out_row) * D + c + k) =
                  make_uint4(pack_bf16(o[k] * scale, o[k + 1] * scale), pack_bf16(o[k + 2] * scale, o[k + 3] * scale),
                             pack_bf16(o[k + 4] * scale, o[k + 5] * scale), pack_bf16(o[k + 6] * scale, o[k + 7] * scale));
          } else if (i < lanes) {
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
              uint32_t b[8];
#pragma unroll
              for (int u = 0; u < 8; ++u) b[u] = __float_as_uint(o[k + u]);
              st_global8(p.part_o + (static_cast<int64_t>(part) + i) * D + c + k, b);
            }
          }
          __syncwarp();
        }
      }
      if (!dead && part >= 0 && i < lanes) p.part_ml[part + i] = make_float2(m, l);
      tc_fence_before();   // (O is read: the stream's next products into it follow its next arrival)
    }
  }
  __syncthreads();
  linger_if_aborted(abort_addr, 1000 * 1000);   // (products in flight end in microseconds)
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

struct JoinParams {
  const PrefixJoin *join;
  const float *part_o;
  const float2 *part_ml;
  __nv_bfloat16 *out;
  int64_t items;
  int32_t Hq, group;
};

// A warp a (row, query head): its partial results, the own keys' first, in their order.  A lane holds D / 32 dims, and
// of 32 parts at a time the weight of one; a dozen parts are loaded at once, ahead of their weights.  Four warps and
// few registers, so that a CTA is set up beside the CTA of the attention that it waits for.
constexpr int kJoinWarps = 4;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) prefix_join_kernel(const JoinParams p) {
  constexpr int N = D / 32, kAtOnce = 12;
  launch_dependents();
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kJoinWarps + threadIdx.x / 32;
  const int lane = lane_id();
  PrefixJoin at{};
  int hl = 0;
  if (item < p.items) {   // (the table is the plan's: nothing of this launch's stream writes it)
    const int64_t entry = item / p.group;
    hl = static_cast<int>(item - entry * p.group);
    at = p.join[entry];
  }
  grid_dependency_wait();
  const int n = at.count[0] + at.count[1];
  if (n == 0) return;   // past the end
  auto lane_of = [&](int k) {
    const bool own = k < at.count[0];
    const int i = own ? k : k - at.count[0];
    return static_cast<int64_t>(own ? at.first[0] : at.first[1]) + static_cast<int64_t>(i) * (own ? at.stride[0] : at.stride[1]) + hl;
  };
  float top = kNoMax, sum = 0.f, o[N];
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = 0.f;
  for (int k0 = 0; k0 < n; k0 += 32) {
    float2 ml = make_float2(kNoMax, 0.f);
    if (k0 + lane < n) ml = p.part_ml[lane_of(k0 + lane)];
    float weight = 0.f;
    const int parts = min(n - k0, 32);
    for (int k = 0; k < parts; k += kAtOnce) {
      float v[kAtOnce][N];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        if (k + u >= parts) break;
        const float *src = p.part_o + lane_of(k0 + k + u) * D + lane * N;
        if constexpr (N == 4) *reinterpret_cast<float4 *>(v[u]) = *reinterpret_cast<const float4 *>(src);
        else *reinterpret_cast<float2 *>(v[u]) = *reinterpret_cast<const float2 *>(src);
      }
      if (k == 0) {
        float most = fmaxf(top, ml.x);
#pragma unroll
        for (int w = 16; w; w >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, w));
        const float keep = exp2_approx(top - most);
        weight = exp2_approx(ml.x - most);
        top = most;
        sum *= keep;
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] *= keep;
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        if (k + u >= parts) break;
        const float x = __shfl_sync(0xffffffffu, weight, k + u), y = __shfl_sync(0xffffffffu, ml.y, k + u);
        sum = fmaf(x, y, sum);
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = fmaf(x, v[u][i], o[i]);
      }
    }
  }
  const float scale = 1.f / sum;
  __nv_bfloat16 *out = p.out + (static_cast<int64_t>(at.row) * p.Hq + at.g * p.group + hl) * D + lane * N;
#pragma unroll
  for (int i = 0; i < N; i += 2) *reinterpret_cast<uint32_t *>(out + i) = pack_bf16(o[i] * scale, o[i + 1] * scale);
}

template <int D>
cudaError_t run(const dsa_ctx *ctx, const dsa_prefix_plan_t *pp, const void *q, const void *kv, float sm_scale, void *out,
                cudaStream_t s, int32_t *launches) {
  const dsa_plan_t &plan = *pp->plan;
  const dsa_msa_shape_t &ms = pp->shape;
  PrefixParams p{};
  p.P = ctx->cfg.page_size, p.BH = plan.box_rows;
  p.Hq = ms.q_heads, p.Hkv = ms.kv_heads, p.group = ms.q_heads / ms.kv_heads;
  const uint64_t cols = 2ull * ms.kv_heads * D;
  const uint64_t dims[3] = {D, static_cast<uint64_t>(ms.q_heads), static_cast<uint64_t>(plan.T)};
  const uint64_t strides[2] = {D * 2, static_cast<uint64_t>(ms.q_heads) * D * 2};
  const uint32_t box[3] = {64, static_cast<uint32_t>(p.group), static_cast<uint32_t>(pp->rows_a_tile)};
  const uint32_t small_rows = std::max(1, kPrefixTile / 2 / p.group);   // (a group above 64: no tile is small)
  const uint32_t small_box[3] = {64, static_cast<uint32_t>(p.group), small_rows};
  if (!encode_tiled_2d(&p.tm_kv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, const_cast<void *>(kv), cols,
                       static_cast<uint64_t>(plan.cache_pages) * p.P, cols * 2, 64, p.BH, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tiled_3d(&p.tm_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, const_cast<void *>(q), dims, strides, box,
                       CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tiled_3d(&p.tm_q_small, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, const_cast<void *>(q), dims, strides, small_box,
                       CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  p.segs = pp->segs, p.ctas = pp->ctas, p.pages = plan.pages;
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.part_o = pp->part_o, p.part_ml = pp->part_ml, p.err = ctx->err;
  p.q_bytes = pp->rows_a_tile * p.group * D * 2;
  p.q_small_bytes = static_cast<int32_t>(small_rows) * p.group * D * 2;
  p.scale_log2 = sm_scale * kLog2e;
  static std::atomic<uint64_t> smem_limit_set{0};
  cudaError_t e = ensure_smem_limit(prefix_tc_kernel<D>, Cfg<D>::BYTES, ctx->device, smem_limit_set);
  if (e != cudaSuccess) return e;
  *launches += 1;
  e = launch_overlapped(prefix_tc_kernel<D>, dim3(pp->n_ctas), kThreads, Cfg<D>::BYTES, pp->paired ? 2 : 1, s, p);
  if (e != cudaSuccess || pp->n_join == 0) return e;
  JoinParams j{pp->join, pp->part_o, pp->part_ml, p.out, static_cast<int64_t>(pp->n_join) * p.group, p.Hq, p.group};
  *launches += 1;
  return launch_overlapped(prefix_join_kernel<D>, dim3(static_cast<unsigned>((j.items + kJoinWarps - 1) / kJoinWarps)),
                           kJoinWarps * 32, 0, 1, s, j);
}

}  // namespace

bool prefix_tc_supported(const dsa_config_t &c, const dsa_msa_shape_t &s) {
  return (s.head_dim == 128 || s.head_dim == 64) && s.q_heads / s.kv_heads <= kPrefixTile && c.page_size % 8 == 0;
}

cudaError_t launch_prefix_tc(const dsa_ctx *ctx, const dsa_prefix_plan_t *pp, const void *q, const void *kv, float sm_scale,
                             void *out, cudaStream_t s, int32_t *launches) {
  return pp->shape.head_dim == 128 ? run<128>(ctx, pp, q, kv, sm_scale, out, s, launches)
                                   : run<64>(ctx, pp, q, kv, sm_scale, out, s, launches);
}

}  // namespace dsa
