// What the tree-attention kernels share: the work's layout over CTAs.
//
// A unit is the work of one key/value head on one block of query rows of one
// request (row = node * G + head of the group), over the request's tokens on
// all ranks (fused call) or on one rank (partials).  Its tokens are counted in
// tiles; a tile never crosses a rank.  All units' tiles in a row are cut into
// equal runs, one per CTA, so a CTA holds the end of one unit, some whole
// units and the start of another.  A unit inside one run is finished by its
// CTA; one that is cut leaves a partial per run, which the merge joins.
// Partial slots: a run has at most two cut pieces, its first (slot 2 run) and
// its last (2 run + 1).
#pragma once

#include "dcp_common.cuh"

namespace dcp {

constexpr int kTreeMaxNodes = 64;      // bits of a node's mask

struct TreeArgs {
  const void* q;          // [N][Hq][d]
  const int32_t* q_start; // [B + 1]
  const int32_t* ctx;     // [B]
  const uint64_t* mask;   // [N]
  int N, B, Hq, Hkv, G, d, max_tree;
  Layout L;
  int per_rank;           // 0: a unit spans the ranks; 1: units per rank
  int rows;               // query rows of a block
  int tile;               // tokens of a tile
  int parts;              // most runs
  float sl2;              // scale * log2(e)
  dcp_rank_ptrs_t k, v;
  const int32_t* bt;
  int max_vb;
  int64_t stride;
  int64_t nb;
  const float* sink;
  void* out;              // fused: [N][Hq][d] of out_dtype; partials: float [dcp][N][Hq][d]
  int out_dtype;
  float* lse;             // fused: [N][Hq] or NULL; partials: [dcp][N][Hq]
  int32_t* err;
  // workspace
  int64_t* first_tile;    // [E + 1] first tile of entry e's units, E = B or B * dcp
  int32_t* first_unit;    // [E + 1]
  int32_t* nodes;         // [B] nodes of a request (0: none, or refused)
  int32_t* hdr;           // runs in use, error word
  float* part_o;          // [2 parts][rows][d], normalised
  float* part_lse;        // [2 parts][rows], in log2 units
};

// Tokens of [0, len) on rank r.
__host__ __device__ __forceinline__ int tree_local(int64_t len, int r, const Layout& L) {
  const int64_t vbs = (int64_t)L.bs * L.dcp;
  const int rem = (int)(len % vbs), turn = L.I * L.dcp;
  int p = rem % turn - r * L.I;
  p = p < 0 ? 0 : (p > L.I ? L.I : p);
  return (int)(len / vbs * L.bs) + rem / turn * L.I + p;
}

// Global position of rank r's local position p.
__device__ __forceinline__ int64_t tree_global(int p, int r, const Layout& L) {
  const int vb = p / L.bs, loc = p - vb * L.bs;
  const int run = loc / L.I;
  return (int64_t)vb * L.bs * L.dcp + ((int64_t)run * L.dcp + r) * L.I + (loc - run * L.I);
}

// Run k of the tiles [0, total) over `parts`.
__device__ __forceinline__ int64_t tree_run(int64_t total, int parts, int k) {
  return total * k / parts;
}
__device__ __forceinline__ int tree_run_of(int64_t total, int parts, int64_t tile) {
  return (int)(((tile + 1) * parts - 1) / total);
}

// A piece: tiles [t0, t0 + n) of one unit.
struct TreePiece {
  int e, b, r0, r1;     // entry, request, ranks
  int g, rb;            // key/value head, row block
  int t0, n;            // first tile (within the unit) and count
  int slot;             // partial slot, -1: the whole unit
};

// The piece at tile `t` of run `run`, [begin, end); e: an entry at or before it.
__device__ __forceinline__ TreePiece tree_piece(const TreeArgs& A, int& e, int64_t t,
                                                int64_t begin, int64_t end, int run) {
  while (__ldcg(A.first_tile + e + 1) <= t) ++e;
  const int64_t base = __ldcg(A.first_tile + e);
  const int u0 = __ldcg(A.first_unit + e);
  const int units = __ldcg(A.first_unit + e + 1) - u0;
  const int per = (int)((__ldcg(A.first_tile + e + 1) - base) / units);
  const int ui = (int)((t - base) / per);
  TreePiece p;
  p.e = e;
  p.b = A.per_rank ? e / A.L.dcp : e;
  p.r0 = A.per_rank ? e % A.L.dcp : 0;
  p.r1 = A.per_rank ? p.r0 + 1 : A.L.dcp;
  const int blocks = units / A.Hkv;
  p.g = ui / blocks;
  p.rb = ui - p.g * blocks;
  p.t0 = (int)((t - base) - (int64_t)ui * per);
  const int64_t left = end - t;
  p.n = per - p.t0 < left ? per - p.t0 : (int)left;
  p.slot = p.t0 == 0 && p.n == per ? -1 : 2 * run + (t == begin ? 0 : 1);
  return p;
}

// Entry that holds tile t (first_tile[e] <= t < first_tile[e + 1]).
__device__ __forceinline__ int tree_entry(const TreeArgs& A, int E, int64_t t) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldcg(A.first_tile + mid) <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// Token row of an output row: request row `row` (node * G + head of the group).
__device__ __forceinline__ int64_t tree_out_row(const TreeArgs& A, const TreePiece& p, int row) {
  const int64_t tok = __ldcg(A.q_start + p.b) + row / A.G;
  return ((int64_t)(A.per_rank ? p.r0 : 0) * A.N + tok) * A.Hq + p.g * A.G + row % A.G;
}

// The tensor-core kernel (dcp_tree_tc.cu): bf16, head_dim 64 or 128, pages of a
// multiple of 16 tokens.  Blocks of 128 or 256 rows, tiles of 128 tokens.
bool tree_tc_shape(int d, dcp_dtype_t dtype, int block_size);
bool tree_tc_supported(const dcp_layout_t& layout, int d, dcp_dtype_t dtype,
                       const dcp_paged_kv_t& kv, int Hkv);
int launch_tree_tc(const TreeArgs& A, cudaStream_t s);

}  // namespace dcp
