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

#include "fp8.cuh"
#include "prefix.h"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr float kPrefixLog2e = 1.4426950408889634f;
constexpr float kNoMax = -3.0e38f;   // the reference maximum of a row that has seen no key

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
  int32_t head_warps, blocks;   // warps side by side over heads (the others over keys), CTAs a (row, kv head)
  float scale_log2;
};

constexpr int kSimpleWarps = 8;
constexpr int kSimpleMaxDim = 512;
constexpr int kSimpleSmem = 200 * 1024;

// 32-bit words of a staged row: odd, so that lanes that read one word of neighbouring rows meet no common bank.
__host__ __device__ constexpr int simple_pitch(int dim) { return ((dim + 1) / 2) | 1; }
// Shared memory of a CTA: K and V of 32 keys for each warp over keys, later the warps' sums; behind it the queries.
__host__ __device__ constexpr int simple_smem(int dim, int heads, int key_warps) {
  const int tiles = 2 * 32 * key_warps * simple_pitch(dim), sums = kSimpleWarps * heads * dim;
  return ((tiles > sums ? tiles : sums) + kSimpleWarps * heads * (dim + 1)) * 4;
}

// A CTA a (row, some heads of a kv head): a warp takes HEADS of them and every key_warps-th 32 keys of a tile, a lane a
// key of S and two dims in 64 of O, with a softmax of its own; the warps over the same heads are joined at the end, in
// their order.  K and V go through shared memory once for all of the CTA's heads; nothing is loaded while a tile is
// worked on.  32 rows behind 8192 tokens, 64 heads over 4 of 96: 0.93 ms, 6.9 TFLOP/s (a warp a key at a time, its dims
// over the lanes: 8.2); 1024 rows of one sequence 1.2 ms (15.8).  With head_dim 128 and pages of 63 these take 1.0 and 1.3
// ms, where the tensor cores' kernel takes 0.02 and 0.03 with pages of 64.
template <int HEADS>
__global__ void __launch_bounds__(kSimpleWarps * 32) prefix_simple_kernel(const PrefixSimpleParams p) {
  constexpr int N = kSimpleMaxDim / 64;
  extern __shared__ uint32_t simple_shared[];
  __shared__ float max_of[kSimpleWarps][HEADS], sum_of[kSimpleWarps][HEADS];
  grid_dependency();
  const int block = blockIdx.x % p.blocks, g = blockIdx.x / p.blocks % p.Hkv;
  const int64_t row = blockIdx.x / p.blocks / p.Hkv;
  const int warp = threadIdx.x / 32, lane = lane_id(), group = p.Hq / p.Hkv;
  const int key_warps = kSimpleWarps / p.head_warps, head_warp = warp % p.head_warps, key_warp = warp / p.head_warps;
  const int head0 = (block * p.head_warps + head_warp) * HEADS;   // of the group; those from `group` on are not there
  const int words = (p.D + 1) / 2, pitch = simple_pitch(p.D), keys = 32 * key_warps;
  const int tiles = 2 * keys * pitch, sums = kSimpleWarps * HEADS * p.D;
  uint32_t *k_tile = simple_shared, *v_tile = k_tile + keys * pitch;
  float *q = reinterpret_cast<float *>(simple_shared + max(tiles, sums)) + warp * HEADS * (p.D + 1);
  const int64_t pos = p.row_pos[row], start = p.row_page_start[row];
  for (int d = lane; d < HEADS * (p.D + 1); d += 32) {
    const int h = d / (p.D + 1), c = d - h * (p.D + 1);
    q[d] = c < p.D && head0 + h < group ? __bfloat162float(p.q[(row * p.Hq + g * group + head0 + h) * p.D + c]) * p.scale_log2 : 0.f;
  }
  __syncwarp();
  float m[HEADS], l[HEADS], o[HEADS][2 * N];
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    m[h] = kNoMax, l[h] = 0.f;
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) o[h][i] = 0.f;
  }
  for (int64_t j0 = 0; j0 <= pos; j0 += keys) {
    const int n = static_cast<int>(min(static_cast<int64_t>(keys), pos + 1 - j0));
    __syncthreads();
    // The warp's keys (warp, warp + 8, ...): a lane looks one of them up, then four rows are on their way at once.
    int64_t place = -1;      // element of the cache where the key's row begins (-1: past the end, zeros)
    if (const int k = lane * kSimpleWarps + warp; k < n) {
      const int64_t slot = start + j0 + k, pi = slot / p.P;
      const int page = pi < p.row_npages[row] ? p.pages[p.row_page_off[row] + pi] : -1;
      if (page >= 0 && page < p.num_pages)
        place = (static_cast<int64_t>(page) * p.P + (slot - pi * p.P)) * 2 * p.Hkv * p.D + static_cast<int64_t>(g) * p.D;
      else
        atomicOr(p.err, kErrBounds);
    }
    const int64_t to_v = static_cast<int64_t>(p.Hkv) * p.D;
    for (int k0 = 0; k0 < keys / kSimpleWarps; k0 += 4) {      // (a multiple of 4)
      int64_t from[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) from[u] = __shfl_sync(0xffffffffu, place, k0 + u);
      for (int i = lane; i < words; i += 32) {
        uint32_t a[4], b[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          a[u] = b[u] = 0;
          if (from[u] < 0) continue;
          const __nv_bfloat16 *x = p.kv + from[u] + 2 * i;
          if (p.D % 2 == 0) {
            a[u] = *reinterpret_cast<const uint32_t *>(x), b[u] = *reinterpret_cast<const uint32_t *>(x + to_v);
          } else {
            a[u] = __bfloat16_as_ushort(x[0]), b[u] = __bfloat16_as_ushort(x[to_v]);
            if (2 * i + 1 < p.D)
              a[u] |= static_cast<uint32_t>(__bfloat16_as_ushort(x[1])) << 16,
                  b[u] |= static_cast<uint32_t>(__bfloat16_as_ushort(x[to_v + 1])) << 16;
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int at = ((k0 + u) * kSimpleWarps + warp) * pitch + i;
          k_tile[at] = a[u], v_tile[at] = b[u];
        }
      }
    }
    __syncthreads();
    auto low = [](uint32_t w) { return __uint_as_float(w << 16); };
    auto high = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
    const int key = key_warp * 32 + lane;
    float e[HEADS];
#pragma unroll
    for (int h = 0; h < HEADS; ++h) e[h] = 0.f;
#pragma unroll 4
    for (int i = 0; i < words; ++i) {      // (an odd head_dim: the last pair's second query is 0)
      const uint32_t w = k_tile[key * pitch + i];
#pragma unroll
      for (int h = 0; h < HEADS; ++h)
        e[h] = fmaf(q[h * (p.D + 1) + 2 * i], low(w), fmaf(q[h * (p.D + 1) + 2 * i + 1], high(w), e[h]));
    }
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
      const float s = key < n ? e[h] : -INFINITY;
      float top = s;
#pragma unroll
      for (int w = 16; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
      top = fmaxf(top, m[h]);
      const float keep = exp2_approx(m[h] - top);
      e[h] = exp2_approx(s - top);
      m[h] = top;
      l[h] = l[h] * keep + e[h];      // (the lane's share)
#pragma unroll
      for (int i = 0; i < 2 * N; ++i) o[h][i] *= keep;
    }
#pragma unroll 4
    for (int k = 0; k < 32; ++k) {
      const uint32_t *v = v_tile + (key_warp * 32 + k) * pitch;
      float x[HEADS];
#pragma unroll
      for (int h = 0; h < HEADS; ++h) x[h] = __shfl_sync(0xffffffffu, e[h], k);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (i * 32 >= words) break;      // uniform
        const uint32_t w = lane + 32 * i < words ? v[lane + 32 * i] : 0u;
#pragma unroll
        for (int h = 0; h < HEADS; ++h) {
          o[h][2 * i] = fmaf(x[h], low(w), o[h][2 * i]);
          o[h][2 * i + 1] = fmaf(x[h], high(w), o[h][2 * i + 1]);
        }
      }
    }
  }
  __syncthreads();
  float *part = reinterpret_cast<float *>(simple_shared);   // [warp][head][D]
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
#pragma unroll
    for (int w = 16; w; w >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], w);
    if (lane == 0) max_of[warp][h] = m[h], sum_of[warp][h] = l[h];
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) {
      const int d = 2 * (lane + 32 * (i / 2)) + i % 2;
      if (d < p.D) part[(warp * HEADS + h) * p.D + d] = o[h][i];
    }
  }
  __syncthreads();
  for (int x = threadIdx.x; x < p.head_warps * HEADS * p.D; x += kSimpleWarps * 32) {
    const int at = x / p.D, d = x - at * p.D, w0 = at / HEADS, h = at - w0 * HEADS, head = block * p.head_warps * HEADS + at;
    if (head >= group) break;
    float top = max_of[w0][h], total = 0.f, sum = 0.f;
    for (int k = 1; k < key_warps; ++k) top = fmaxf(top, max_of[w0 + k * p.head_warps][h]);
    for (int k = 0; k < key_warps; ++k) {
      const int w = w0 + k * p.head_warps;
      const float keep = exp2_approx(max_of[w][h] - top);
      total = fmaf(sum_of[w][h], keep, total);
      sum = fmaf(part[(w * HEADS + h) * p.D + d], keep, sum);
    }
    p.out[(row * p.Hq + g * group + head) * p.D + d] = __float2bfloat16_rn(sum / total);
  }
}

template <int HEADS>
cudaError_t run_simple(const dsa_ctx *ctx, PrefixSimpleParams &p, int32_t T, cudaStream_t s) {
  const int group = p.Hq / p.Hkv;
  // as many heads a CTA as there are (their keys are staged once), fewer where that leaves SMs idle or its sums no room
  p.head_warps = 1;
  while (p.head_warps < kSimpleWarps && p.head_warps * HEADS < group) p.head_warps *= 2;
  auto ctas = [&] { return static_cast<int64_t>(T) * p.Hkv * ((group + p.head_warps * HEADS - 1) / (p.head_warps * HEADS)); };
  auto smem = [&](int head_warps) { return simple_smem(p.D, HEADS, kSimpleWarps / head_warps); };
  while (p.head_warps > 1 && ctas() < 2 * ctx->num_sms && smem(p.head_warps / 2) <= kSimpleSmem) p.head_warps /= 2;
  while (smem(p.head_warps) > kSimpleSmem) p.head_warps *= 2;
  p.blocks = (group + p.head_warps * HEADS - 1) / (p.head_warps * HEADS);
  static std::atomic<uint64_t> smem_limit_set{0};
  cudaError_t e = ensure_smem_limit(prefix_simple_kernel<HEADS>, kSimpleSmem, ctx->device, smem_limit_set);
  if (e != cudaSuccess) return e;
  return launch_overlapped(prefix_simple_kernel<HEADS>, dim3(static_cast<unsigned>(ctas())), kSimpleWarps * 32, smem(p.head_warps), 1, s, p);
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

// ---- the tensor cores' work
struct Chain {
  int32_t tile[2];              // tiles of queries (-1: one only)
  int32_t span, causal;
  int32_t g, slot0, ntiles, lo, hi;
};
struct QueryTile {
  int32_t row, rows;
};
// Tiles [t0, t1) of a chain.
struct Piece {
  int32_t chain, t0, t1;
};

// What a CTA spends on a piece, in us: a key tile, and beside its tiles the queries' load, the first product's latency
// and the output, which for a lone tile goes by its lanes.  Measured on 152 SMs: a pair's tile 1.4 in a long chain and
// up to 2 in one of seven, its partial results 2 to 3; lone tiles two streams at a time, 1.05 out of L2.  (Over 29
// batches 1.7 for a pair's tile, 2.5 to 4 for its start, 0.9 to 1.1 and 0.7 to 1.4 for a lone tile took up to 1 % more,
// two of them at once up to 3 %.)
struct Cost {
  double tile, start;
};
constexpr Cost kPairCost{1.5, 3.0}, kLoneCost{1.0, 1.0};
constexpr double kLoneLane = 0.0125;
constexpr double kLeast = 2.5;      // fewer CTAs rather than less than this for each

// A line of pieces in runs of at most `most` each: a piece that does not fit is cut, unless that would leave a sliver
// of it in a run that has something already (a cut costs a start).  Returns how many; `out`, where given, gets them.
template <typename CostOf>
int cut_line(const std::vector<Piece> &line, double most, CostOf cost_of, std::vector<std::vector<Piece>> *out = nullptr) {
  int runs = 1;
  double room = most;
  bool empty = true;
  if (out) out->assign(1, {});
  auto put = [&](const Piece &x) {
    empty = false;
    if (out) out->back().push_back(x);
  };
  for (Piece x : line)
    for (;;) {
      const Cost c = cost_of(x);
      const int32_t n = x.t1 - x.t0;
      if (n * c.tile + c.start <= room || (empty && n == 1)) {
        put(x);
        room -= n * c.tile + c.start;
        break;
      }
      int32_t here = static_cast<int32_t>(std::max(0.0, (room - c.start) / c.tile));
      here = std::min(empty ? std::max(here, 1) : here * c.tile < 0.1 * most ? 0 : here, n - 1);
      if (here > 0) put(Piece{x.chain, x.t0, x.t0 + here});
      x.t0 += here;
      ++runs;
      room = most, empty = true;
      if (out) out->emplace_back();
    }
  return runs;
}

// Partial results of a tile of queries and a kv head: `count` of them from `first` on (0: its only segment writes
// the output).
struct Parts {
  int32_t first, count;
};
// A row's tile over its own keys and its tile over the shared ones (-1: none), and its first lane in each.
struct RowTiles {
  int32_t own, own_lane, shared, shared_lane;
};

struct Work {
  std::vector<QueryTile> tiles;
  std::vector<Chain> chains;
  std::vector<PrefixSeg> segs;
  std::vector<PrefixCta> ctas;
  std::vector<PrefixJoin> join;
};

void lay_out(const dsa_ctx *ctx, dsa_prefix_plan_t *pp, Work &w) {
  const dsa_plan_t &plan = *pp->plan;
  const int32_t Hkv = pp->shape.kv_heads, group = pp->shape.q_heads / Hkv, per = kPrefixTile / group, BH = plan.box_rows;
  pp->rows_a_tile = per;
  std::vector<RowTiles> rows(plan.T, RowTiles{-1, 0, -1, 0});
  // Rows [r0, r1) against slots lo .. hi - 1 (causal: row r sees those below limit0 + r - r0 + 1 - ...).
  auto add = [&](int32_t r0, int32_t r1, int32_t span, int64_t lo, int64_t hi, bool causal, bool shared) {
    const PlanSpan &sp = plan.spans[span];
    const int32_t first = static_cast<int32_t>(w.tiles.size());
    for (int32_t r = r0; r < r1; r += per) {
      const int32_t n = std::min(per, r1 - r), id = static_cast<int32_t>(w.tiles.size());
      w.tiles.push_back(QueryTile{r, n});
      for (int32_t k = 0; k < n; ++k) {
        RowTiles &x = rows[r + k];
        (shared ? x.shared : x.own) = id;
        (shared ? x.shared_lane : x.own_lane) = k * group;
      }
    }
    const int32_t count = static_cast<int32_t>(w.tiles.size()) - first;
    const int32_t slot0 = static_cast<int32_t>(lo / BH * BH);
    for (int32_t g = 0; g < Hkv; ++g)
      for (int32_t t = 0; t < count; t += 2) {
        const bool pair = t + 1 < count;
        const QueryTile &last = w.tiles[first + t + pair];
        // a causal chain ends behind its last row's own key
        const int64_t end = causal ? static_cast<int64_t>(sp.page_start) + sp.ctx_start + (last.row + last.rows - sp.q_start) : hi;
        w.chains.push_back(Chain{{first + t, pair ? first + t + 1 : -1}, span, causal, g, slot0,
                                 static_cast<int32_t>((end - slot0 + kPrefixTile - 1) / kPrefixTile), static_cast<int32_t>(lo),
                                 static_cast<int32_t>(end)});
      }
  };
  size_t next = 0;
  const int32_t spans = static_cast<int32_t>(plan.spans.size());
  for (int32_t i = 0; i < spans;) {
    const dsa_prefix_t *x = next < pp->prefixes.size() && pp->prefixes[next].first_span == i ? &pp->prefixes[next++] : nullptr;
    const int32_t end = x ? x->first_span + x->num_spans : i + 1;
    for (int32_t j = i; j < end;) {
      // A span that fills tiles by itself takes the shared keys with its own in one chain: its rows need no joining, and
      // the pages are in L2 for the next span.  The others' rows are put together, in runs of neighbours.
      auto fills = [&](int32_t k) { return !x || plan.spans[k].q_len >= 4 * per; };
      const PlanSpan &s = plan.spans[j];
      const int64_t start = s.page_start;
      int32_t k = j;
      while (k < end && !fills(k)) ++k;
      if (k > j) {
        const PlanSpan &l = plan.spans[k - 1];
        add(s.q_start, l.q_start + l.q_len, j, start, start + x->tokens, false, true);
        for (int32_t m = j; m < k; ++m) {
          const PlanSpan &o = plan.spans[m];
          add(o.q_start, o.q_start + o.q_len, m, start + x->tokens, 0, true, false);
        }
      }
      if (k < end) {
        const PlanSpan &o = plan.spans[k];
        add(o.q_start, o.q_start + o.q_len, k, o.page_start, 0, true, false);
        ++k;
      }
      j = k;
    }
    i = end;
  }
  // One line, the pairs' chains, then the lone tiles', cut evenly over the CTAs.  Chains of pairs over the same keys
  // that are longer than a CTA's share go in blocks of about that, all pairs' first block first, so that CTAs that
  // run together read the same keys.
  auto cost_of_chain = [&](const Chain &c) {
    return c.tile[1] >= 0 ? kPairCost : Cost{kLoneCost.tile, kLoneCost.start + kLoneLane * w.tiles[c.tile[0]].rows * group};
  };
  auto cost_of = [&](const Piece &x) { return cost_of_chain(w.chains[x.chain]); };
  const int n = std::max(2, ctx->num_sms / 2 * 2);
  double cost = 0.0;
  for (const Chain &c : w.chains) {
    const Cost x = cost_of_chain(c);
    cost += c.ntiles * x.tile + x.start;
  }
  const double share = std::max(4.0, (cost / n - kPairCost.start) / kPairCost.tile);
  std::vector<Piece> lone;
  for (size_t c = 0; c < w.chains.size(); ++c)
    if (w.chains[c].tile[1] < 0) lone.push_back(Piece{static_cast<int32_t>(c), 0, w.chains[c].ntiles});
  auto line_of = [&](double block) {
    std::vector<Piece> line;
    std::vector<int32_t> done;      // tiles of a chain of the group that are in the line
    for (size_t c = 0; c < w.chains.size();) {
      const Chain &x = w.chains[c];
      size_t e = c + 1;
      while (e < w.chains.size() && w.chains[e].span == x.span && w.chains[e].g == x.g && w.chains[e].slot0 == x.slot0 &&
             w.chains[e].causal == x.causal)
        ++e;
      int32_t most = 0;
      for (size_t k = c; k < e; ++k)
        if (w.chains[k].tile[1] >= 0) most = std::max(most, w.chains[k].ntiles);
      const int32_t blocks = std::max(1, static_cast<int32_t>(most / block + 0.5));
      done.assign(e - c, 0);
      for (int32_t i = 1; i <= blocks; ++i) {
        const int32_t end = static_cast<int32_t>(static_cast<int64_t>(most) * i / blocks);
        for (size_t k = c; k < e; ++k) {
          const int32_t tiles = w.chains[k].ntiles, t = done[k - c];
          if (w.chains[k].tile[1] < 0 || t >= tiles || t >= end) continue;
          done[k - c] = tiles - end < block / 3 ? tiles : end;      // (no sliver behind it)
          line.push_back(Piece{static_cast<int32_t>(k), t, done[k - c]});
        }
      }
      c = e;
    }
    line.insert(line.end(), lone.begin(), lone.end());
    return line;
  };
  // The least that a CTA can be given so that n of them do, with the blocks that leave the least: a block that does not
  // fit a whole number of times ends in a rest, which costs a start of its own (32 rows behind 8192 tokens took 26 us
  // with blocks of the share alone and 20.5 with these; over 29 batches one size took 5 % longer than the best of five,
  // three 1.6 %).
  std::vector<Piece> line;
  double high = 0.0;
  for (const double f : {1.0, 0.85, 1.2, 0.7, 1.45}) {
    std::vector<Piece> tried = line_of(share * f);
    double low = std::max(cost / n, kLeast), top = low;
    if (cut_line(tried, low, cost_of) > n) {
      while (cut_line(tried, top, cost_of) > n) top *= 1.25;
      for (int i = 0; i < 8; ++i) {
        const double mid = 0.5 * (low + top);
        (cut_line(tried, mid, cost_of) <= n ? top : low) = mid;
      }
    }
    if (line.empty() || top < high) high = top, line.swap(tried);
  }
  std::vector<std::vector<Piece>> runs;
  cut_line(line, high, cost_of, &runs);
  // neighbours share a TPC where there are more of them than TPCs (launched as clusters of two): lone tiles beside
  // pairs, both wait longer for their loads
  pp->paired = static_cast<int>(runs.size()) > n / 2;
  if (pp->paired && runs.size() % 2) runs.emplace_back();
  w.ctas.assign(runs.size(), PrefixCta{});
  std::vector<int32_t> pieces_of(w.tiles.size() * Hkv, 0);
  auto put = [&](const Piece &x) {
    const Chain &c = w.chains[x.chain];
    PrefixSeg s{};
    for (int m = 0; m < 2; ++m) {
      if (c.tile[m] < 0) continue;
      const QueryTile &t = w.tiles[c.tile[m]];
      const PlanSpan &sp = plan.spans[c.span];
      s.row[m] = t.row, s.lanes[m] = t.rows * group;
      s.limit[m] = c.causal ? sp.page_start + sp.ctx_start + (t.row - sp.q_start) + 1 : c.hi;
      s.part[m] = pieces_of[static_cast<size_t>(c.tile[m]) * Hkv + c.g]++;   // (its number, for now)
    }
    s.causal = c.causal, s.g = c.g;
    s.page_off = plan.spans[c.span].page_off;
    s.slot0 = c.slot0 + x.t0 * kPrefixTile, s.ntiles = x.t1 - x.t0;
    s.lo = c.lo, s.hi = c.hi;
    w.segs.push_back(s);
    return static_cast<size_t>(x.chain);
  };
  std::vector<size_t> chain_of;
  for (size_t i = 0; i < w.ctas.size(); ++i) {
    PrefixCta &cta = w.ctas[i];
    cta.a0 = static_cast<int32_t>(w.segs.size());
    size_t at = 0;                          // (the pairs come first)
    for (; at < runs[i].size() && w.chains[runs[i][at].chain].tile[1] >= 0; ++at) {
      chain_of.push_back(put(runs[i][at]));
      cta.tiles_a += runs[i][at].t1 - runs[i][at].t0;
    }
    cta.a1 = static_cast<int32_t>(w.segs.size());
    for (size_t k = at; k < runs[i].size(); ++k) cta.tiles_b += runs[i][k].t1 - runs[i][k].t0;
    int32_t left = (cta.tiles_b + 1) / 2;   // the first stream's tiles
    int32_t from = 0;                       // tiles of piece `at` that are laid out
    for (int m = 0; m < 2; ++m) {
      cta.b0[m] = static_cast<int32_t>(w.segs.size());
      if (m == 1) left = cta.tiles_b / 2;
      while (left > 0) {
        const Piece &x = runs[i][at];
        const int32_t k = std::min(left, x.t1 - x.t0 - from);
        chain_of.push_back(put(Piece{x.chain, x.t0 + from, x.t0 + from + k}));
        left -= k, from += k;
        if (from == x.t1 - x.t0) ++at, from = 0;
      }
      cta.b1[m] = static_cast<int32_t>(w.segs.size());
    }
    cta.small = 1;
    for (int32_t k = cta.a1; k < static_cast<int32_t>(w.segs.size()); ++k)
      if (w.segs[k].lanes[0] > kPrefixTile / 2) cta.small = 0;
  }
  // partial results: none where a tile's only result is its own keys' only segment
  std::vector<char> has_shared(w.tiles.size(), 0);
  for (const RowTiles &r : rows)
    if (r.shared >= 0) has_shared[r.own] = has_shared[r.shared] = 1;
  std::vector<Parts> parts(w.tiles.size() * Hkv);
  int64_t lanes = 0;
  for (size_t t = 0; t < w.tiles.size(); ++t)
    for (int32_t g = 0; g < Hkv; ++g) {
      Parts &x = parts[t * Hkv + g];
      const int32_t count = pieces_of[t * Hkv + g];
      if (count == 1 && !has_shared[t]) continue;   // (count stays 0)
      x = Parts{static_cast<int32_t>(lanes), count};
      lanes += static_cast<int64_t>(count) * w.tiles[t].rows * group;
    }
  for (int32_t r = 0; r < plan.T; ++r)
    for (int32_t g = 0; g < Hkv; ++g) {
      PrefixJoin x{r, g, {0, 0}, {0, 0}, {0, 0}};
      const int32_t tile[2] = {rows[r].own, rows[r].shared}, lane[2] = {rows[r].own_lane, rows[r].shared_lane};
      for (int k = 0; k < 2; ++k) {
        if (tile[k] < 0) continue;
        const Parts &y = parts[static_cast<size_t>(tile[k]) * Hkv + g];
        x.first[k] = y.first + lane[k], x.count[k] = y.count, x.stride[k] = w.tiles[tile[k]].rows * group;
      }
      if (x.count[0] > 0) w.join.push_back(x);
    }
  pp->n_join = static_cast<int32_t>(w.join.size());
  pp->part_lanes = lanes;
  for (size_t i = 0; i < w.segs.size(); ++i)
    for (int m = 0; m < 2; ++m) {
      const int32_t t = w.chains[chain_of[i]].tile[m];
      if (t < 0) continue;
      const Parts &x = parts[static_cast<size_t>(t) * Hkv + w.segs[i].g];
      w.segs[i].part[m] = x.count ? x.first + w.segs[i].part[m] * w.segs[i].lanes[m] : -1;
    }
  w.segs.resize(w.segs.size() + 2);   // (a walk that ends looks at two behind its last, and uses neither)
  pp->n_ctas = static_cast<int32_t>(w.ctas.size());
}

// The tables and the partial results' space on the device, in order on `stream`.
dsa_status upload(const dsa_ctx *ctx, dsa_prefix_plan_t *pp, const Work &w) {
  auto round = [](size_t n) { return (n + 255) / 256 * 256; };
  const size_t o_seg = 0, o_cta = o_seg + round(w.segs.size() * sizeof(PrefixSeg)),
               o_join = o_cta + round(w.ctas.size() * sizeof(PrefixCta)), tables = o_join + round(w.join.size() * sizeof(PrefixJoin)),
               o_ml = tables + round(static_cast<size_t>(pp->part_lanes) * pp->shape.head_dim * sizeof(float)),
               bytes = o_ml + round(static_cast<size_t>(pp->part_lanes) * sizeof(float2)) + 256;
  pp->host.assign(tables, 0);
  std::memcpy(pp->host.data() + o_seg, w.segs.data(), w.segs.size() * sizeof(PrefixSeg));
  std::memcpy(pp->host.data() + o_cta, w.ctas.data(), w.ctas.size() * sizeof(PrefixCta));
  std::memcpy(pp->host.data() + o_join, w.join.data(), w.join.size() * sizeof(PrefixJoin));
  if (ctx->device < 0) return DSA_OK;
  if (cudaSetDevice(ctx->device) != cudaSuccess) return DSA_ERR_CUDA;
  if (cudaMallocAsync(reinterpret_cast<void **>(&pp->dev), bytes, pp->stream) != cudaSuccess) {
    cudaGetLastError();
    pp->dev = nullptr;
    return DSA_ERR_OOM;
  }
  if (cudaMemcpyAsync(pp->dev, pp->host.data(), tables, cudaMemcpyHostToDevice, pp->stream) != cudaSuccess) return DSA_ERR_CUDA;
  pp->segs = reinterpret_cast<PrefixSeg *>(pp->dev + o_seg), pp->ctas = reinterpret_cast<PrefixCta *>(pp->dev + o_cta);
  pp->join = reinterpret_cast<PrefixJoin *>(pp->dev + o_join);
  pp->part_o = reinterpret_cast<float *>(pp->dev + tables), pp->part_ml = reinterpret_cast<float2 *>(pp->dev + o_ml);
  return DSA_OK;
}

}  // namespace

dsa_status make_prefix_plan(const dsa_ctx *ctx, const dsa_plan_t *plan, const dsa_msa_shape_t &shape, const dsa_prefix_t *prefixes,
                            int32_t n, cudaStream_t stream, dsa_prefix_plan_t *pp) {
  const int32_t spans = static_cast<int32_t>(plan->spans.size()), P = ctx->cfg.page_size;
  pp->plan = plan, pp->shape = shape, pp->stream = stream, pp->device = ctx->device;
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
  // (TMA takes 32-bit cache rows, the tables 32-bit slots)
  int64_t end = static_cast<int64_t>(plan->cache_pages) * P;
  for (const PlanSpan &s : plan->spans) end = std::max(end, static_cast<int64_t>(s.page_start) + s.ctx_start + s.q_len + 2 * kPrefixTile);
  pp->tc = prefix_tc_supported(ctx->cfg, shape) && end <= INT32_MAX;
  if (!pp->tc || plan->T == 0) return DSA_OK;
  Work w;
  lay_out(ctx, pp, w);
  if (pp->part_lanes > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  return upload(ctx, pp, w);
}

cudaError_t launch_prefix_attend(const dsa_ctx *ctx, const dsa_prefix_plan_t *pp, const void *q, const void *kv, float sm_scale,
                                 void *out, cudaStream_t s, int32_t *launches) {
  if (pp->tc) return launch_prefix_tc(ctx, pp, q, kv, sm_scale, out, s, launches);
  const dsa_plan_t &plan = *pp->plan;
  PrefixSimpleParams p{};
  p.q = static_cast<const __nv_bfloat16 *>(q), p.kv = static_cast<const __nv_bfloat16 *>(kv);
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.row_pos = plan.row_pos, p.row_page_off = plan.row_page_off, p.row_npages = plan.row_npages;
  p.row_page_start = plan.row_page_start, p.pages = plan.pages, p.err = ctx->err;
  p.Hq = pp->shape.q_heads, p.Hkv = pp->shape.kv_heads, p.D = pp->shape.head_dim, p.P = ctx->cfg.page_size;
  p.num_pages = plan.cache_pages, p.scale_log2 = sm_scale * kPrefixLog2e;
  *launches += 1;
  return p.Hq > p.Hkv ? run_simple<2>(ctx, p, plan.T, s) : run_simple<1>(ctx, p, plan.T, s);
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
  if (pp->dev) {
    cudaSetDevice(pp->device);
    cudaFreeAsync(pp->dev, pp->stream);
  }
  delete pp;
}

dsa_status dsa_prefix_plan_get_info(const dsa_prefix_plan_t *pp, dsa_prefix_info_t *info) {
  if (!pp || !info) return DSA_ERR_INVALID_ARG;
  *info = dsa_prefix_info_t{};
  info->num_prefixes = static_cast<int32_t>(pp->prefixes.size());
  info->on_tensor_cores = pp->tc ? 1 : 0;
  info->tokens_read = pp->tokens_read;
  return DSA_OK;
}

dsa_status dsa_prefix_attend(dsa_ctx_t *ctx, const dsa_prefix_plan_t *pp, const void *q, const void *kv_cache, float sm_scale,
                             void *out, dsa_stream_t stream) {
  if (!ctx || !pp || pp->plan->ctx != ctx || ctx->device < 0 || !(sm_scale > 0.f) || !std::isfinite(sm_scale)) return DSA_ERR_INVALID_ARG;
  if (cudaSetDevice(ctx->device) != cudaSuccess) return DSA_ERR_CUDA;
  LaunchCount launched(ctx);
  if (pp->plan->T == 0) return DSA_OK;
  auto on16 = [](const void *p) { return p && reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  if (!on16(q) || !on16(kv_cache) || !on16(out)) return DSA_ERR_INVALID_ARG;
  const uintptr_t from = reinterpret_cast<uintptr_t>(q), to = reinterpret_cast<uintptr_t>(out),
                  bytes = static_cast<uintptr_t>(pp->plan->T) * pp->shape.q_heads * pp->shape.head_dim * 2;
  if (from < to + bytes && to < from + bytes) return DSA_ERR_INVALID_ARG;   // a row's queries may be read after another's output
  return cuda_status(ctx, launch_prefix_attend(ctx, pp, q, kv_cache, sm_scale, out, reinterpret_cast<cudaStream_t>(stream),
                                               &launched.n));
}

}  // extern "C"
