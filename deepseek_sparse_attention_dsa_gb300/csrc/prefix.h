// prefix.h -- the work of the attention over a shared prefix, as its planner
// (prefix.cu) lays it out and its tensor-core kernels (prefix_tc.cu) take it.
//
// Rows of the matrix products are (row, query head of one kv head) pairs: a tile of
// queries is rows_a_tile rows x group heads, at most 128 lanes.  A chain is a tile,
// or two neighbouring ones, against a run of keys in tiles of 128; a segment is what
// one CTA does of a chain.  Keys are counted in slots (page_start + position).
#pragma once
#include <vector>

#include "dsa_internal.h"

namespace dsa {

constexpr int kPrefixTile = 128;   // keys a tile, and lanes a tile of queries

struct alignas(16) PrefixSeg {   // (64 bytes)
  int32_t row[2], lanes[2];     // first row and live lanes of each tile of queries (one: lanes[1] = 0)
  int32_t part[2];              // where lane 0's partial result goes, in lanes; -1: lanes are written to the output
  int32_t limit[2];             // causal: lane l sees slots below limit + l / group
  int32_t causal;
  int32_t g;                    // kv head
  int32_t page_off;
  int32_t slot0, ntiles;        // first tile's first slot (a multiple of the box height), key tiles
  int32_t lo, hi;               // slots that some lane sees: lo .. hi - 1; not causal: every lane
};

// A CTA's segments: pairs [a0, a1) with key tiles `tiles_a` in all, then one list for each of its two
// streams, [b0[w], b1[w]), with tiles_b in both (the first stream's are half of them, rounded up).
struct PrefixCta {
  int32_t a0, a1, tiles_a;
  int32_t b0[2], b1[2], tiles_b;
  int32_t small;           // no tile of the streams' own lists has more than 64 lanes
};

// A row's partial results for the heads of kv head g: over its own keys, then over the shared ones; part k of each
// lies `stride` lanes behind the one before, from `first` (the group's first head) on.  Only rows that have such.
struct PrefixJoin {
  int32_t row, g;
  int32_t first[2], count[2], stride[2];
};

}  // namespace dsa

struct dsa_prefix_plan {
  const dsa_plan_t *plan = nullptr;
  dsa_msa_shape_t shape{};
  std::vector<dsa_prefix_t> prefixes;
  int64_t tokens_read = 0;
  // tensor cores
  bool tc = false;
  bool paired = false;                   // neighbouring CTAs on one TPC
  cudaStream_t stream = nullptr;
  int device = -1;
  int32_t rows_a_tile = 0, n_ctas = 0, n_join = 0;
  int64_t part_lanes = 0;
  std::vector<char> host;                // staging copy of the tables
  char *dev = nullptr;
  dsa::PrefixSeg *segs = nullptr;        // device, and two more behind the last
  dsa::PrefixCta *ctas = nullptr;
  dsa::PrefixJoin *join = nullptr;       // [n_join]
  float *part_o = nullptr;               // [lane][head_dim]
  float2 *part_ml = nullptr;             // [lane]: reference maximum (log2 units), sum
};

namespace dsa {
bool prefix_tc_supported(const dsa_config_t &c, const dsa_msa_shape_t &s);
cudaError_t launch_prefix_tc(const dsa_ctx *ctx, const dsa_prefix_plan_t *pp, const void *q, const void *kv, float sm_scale,
                             void *out, cudaStream_t s, int32_t *launches);
}  // namespace dsa
