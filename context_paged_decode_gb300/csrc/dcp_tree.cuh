// What the tree-attention kernels share: the work's layout over CTAs.
//
// A unit is the work of one key/value head on one block of query rows of one
// request (row = node * G + head of the group), over the request's tokens on
// all ranks (fused call) or on one rank (partials).  Each rank's tokens are cut
// into chunks, and the chunks of a unit, rank after rank, into tiles.  What a unit costs beside them (loading
// queries, writing rows) counts as `extra` empty tiles behind its own.  All
// units' tiles in a row are cut into equal runs, one per CTA, so a CTA holds the end of one unit, some whole
// units and the start of another.  A unit inside one run is finished by its
// CTA; one that is cut leaves a partial per run, and the partials are joined in
// the order of the runs (by the last CTA that comes to them, or by a merge).
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
  int rows;               // query rows of a block: whole nodes
  int chunk, tile;        // tokens of a chunk and of a tile
  int parts;              // most runs
  int extra;              // most tiles that a unit counts for beside its own
  int join;               // the last CTA to come joins a cut unit, not the merge
  int self;               // the kernel's CTAs plan for themselves (few entries)
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
  struct TreeEntry* entry;   // [E], E = B or B * dcp
  int32_t* run_entry;        // [parts] entry of each run's first tile
  int32_t* hdr;              // runs in use, error word, tiles (64 bits), extra in use
  float* part_o;             // [2 parts][rows][d], normalised
  float* part_lse;           // [2 parts][rows], in log2 units
  int32_t* arrived;          // [parts] partials there of the unit whose first run it is
};

// One request's units (on one rank, for partials), in two 16-byte reads: a
// workspace is aligned to 16 bytes and no more, and so is a plan in shared memory.
struct __align__(16) TreeEntry {
  int64_t tile0;   // first tile of its units
  int32_t units;   // 0: none (refused, no nodes, or nothing on the rank)
  int32_t per;     // tiles of a unit
  int32_t nodes;
  int32_t ctx;
  int32_t q0;      // first token
  int32_t pad;
};
static_assert(sizeof(TreeEntry) == 32 && alignof(TreeEntry) == 16, "two 16-byte pieces");

__device__ __forceinline__ TreeEntry tree_load(const TreeArgs& A, int e) {
  const int4* p = reinterpret_cast<const int4*>(A.entry + e);
  const int4 x = __ldcg(p), y = __ldcg(p + 1);
  TreeEntry n;
  n.tile0 = (int64_t)(uint32_t)x.x | (int64_t)x.y << 32;
  n.units = x.z;
  n.per = x.w;
  n.nodes = y.x;
  n.ctx = y.y;
  n.q0 = y.z;
  n.pad = 0;
  return n;
}

// Tokens of [0, len) on rank r are base + clamp(rest - r * I, 0, I): whole
// turns round the ranks, and what the last one leaves.
struct TreeLen {
  int base, rest;
  __host__ __device__ __forceinline__ TreeLen(int len, const Layout& L) {
    const uint32_t vbs = (uint32_t)(L.bs * L.dcp), turn = (uint32_t)(L.I * L.dcp);
    const uint32_t full = (uint32_t)len / vbs, rem = (uint32_t)len - full * vbs;
    const uint32_t q = rem / turn;
    base = (int)(full * L.bs + q * L.I);
    rest = (int)(rem - q * turn);
  }
  __host__ __device__ __forceinline__ int on(int r, const Layout& L) const {
    const int p = rest - r * L.I;
    return base + (p < 0 ? 0 : (p > L.I ? L.I : p));
  }
};

// Global position of rank r's local position p.
__device__ __forceinline__ int tree_global(int p, int r, const Layout& L) {
  const int vb = p / L.bs, loc = p - vb * L.bs;
  const int run = loc / L.I;
  return vb * L.bs * L.dcp + (run * L.dcp + r) * L.I + (loc - run * L.I);
}

// Run k of the tiles [0, total) over `parts` begins at total * k / parts, and
// tile t is in run ((t + 1) * parts - 1) / total; in 32 bits where they hold it
// (a 64-bit division is some 150 instructions, and the merge takes three a row).
__device__ __forceinline__ int64_t tree_run(int64_t total, int parts, int k) {
  const int64_t x = total * k;
  return (uint64_t)x >> 32 ? x / parts : (int64_t)((uint32_t)x / (uint32_t)parts);
}
__device__ __forceinline__ int tree_run_of(int64_t total, int parts, int64_t tile) {
  const int64_t x = (tile + 1) * parts - 1;
  return (uint64_t)x >> 32 ? (int)(x / total) : (int)((uint32_t)x / (uint32_t)total);
}

// A piece: tiles [t0, t0 + n) of one unit.
struct TreePiece {
  int b, r0, r1;        // request, ranks
  int T, ctx, q0;       // its nodes, cached tokens and first token
  int g, rb;            // key/value head, row block
  int t0, n;            // first tile (within the unit) and count
  int slot;             // partial slot, -1: the whole unit
  int64_t u0;           // the unit's first tile, among all
  int per;              // its tiles
};

// Entry e as its request asks for it (tile0 is left to the plan); a request
// that cannot be is refused, and counted if `count`.
__device__ __forceinline__ TreeEntry tree_request(const TreeArgs& A, int e, bool count) {
  TreeEntry n;
  n.tile0 = 0;
  n.units = n.per = n.nodes = n.ctx = n.q0 = n.pad = 0;
  const int b = A.per_rank ? e / A.L.dcp : e, r = A.per_rank ? e % A.L.dcp : 0;
  const int q0 = __ldcg(A.q_start + b), q1 = __ldcg(A.q_start + b + 1);
  const int64_t ctx = __ldcg(A.ctx + b);
  const int T = q1 - q0;
  if (q0 < 0 || q1 < q0 || q1 > A.N || T > A.max_tree || ctx < 0 ||
      ctx + T > (int64_t)A.max_vb * A.L.bs * A.L.dcp) {
    if (count && r == 0) count_error(A.err);
    return n;
  }
  if (T == 0) return n;
  const int r1 = A.per_rank ? r + 1 : A.L.dcp;
  const TreeLen len((int)ctx + T, A.L);
  for (int x = r; x < r1; ++x) n.per += (len.on(x, A.L) + A.chunk - 1) / A.chunk;
  n.per = (n.per + A.tile / A.chunk - 1) / (A.tile / A.chunk);
  if (n.per > 0) n.units = A.Hkv * ((T * A.G + A.rows - 1) / A.rows);
  n.nodes = T;
  n.ctx = (int)ctx;
  n.q0 = q0;
  return n;
}

// Tiles that a unit counts for beside its own: no more than a run would have,
// so small calls spread their tiles over all CTAs.
__device__ __forceinline__ int64_t tree_extra(const TreeArgs& A, int64_t tiles) {
  const int64_t run = tiles / A.parts;
  return run < A.extra ? run : A.extra;
}

// The plan of a call with few entries, made by a warp of each CTA for itself:
// a kernel and a wait less than a plan of its own.  With 1, 4, 8 and 16 requests
// of 8 nodes over up to 1500 tokens 15.9, 20.7, 22.4 and 28.9 us against 18.4,
// 23.0, 24.6 and 30.7; 16 x 5 nodes on one key head 20.0 against 22.1, fp32 22.7
// against 25.6.  It gains as much at the last of these as at the first: what ends
// it is the room that shared memory has beside the tiles, 16 entries (17 at most).
// CTA 0 leaves it for the merge.
constexpr int kTreeSelf = 16;
struct TreeSelf {
  TreeEntry entry[kTreeSelf];
  int64_t end[kTreeSelf];   // tiles up to and with each entry
  int64_t total;
  int parts, extra;
};

__device__ __forceinline__ void tree_self_plan(const TreeArgs& A, TreeSelf* S) {
  const int lane = threadIdx.x & 31, E = A.per_rank ? A.B * A.L.dcp : A.B;
  TreeEntry n;
  n.tile0 = 0;
  n.units = n.per = n.nodes = n.ctx = n.q0 = n.pad = 0;
  if (lane < E) n = tree_request(A, lane, blockIdx.x == 0);
  int64_t t = (int64_t)n.units * n.per, u = n.units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t pt = __shfl_up_sync(0xffffffffu, t, o);
    const int64_t pu = __shfl_up_sync(0xffffffffu, u, o);
    if (lane >= o) {
      t += pt;
      u += pu;
    }
  }
  const int64_t tiles = __shfl_sync(0xffffffffu, t, 31), units = __shfl_sync(0xffffffffu, u, 31);
  const int64_t extra = tree_extra(A, tiles), total = tiles + extra * units;
  n.tile0 = t + extra * u - n.units * (n.per + extra);
  const int parts = total < A.parts ? (int)total : A.parts;
  if (lane < E) {
    S->entry[lane] = n;
    S->end[lane] = t + extra * u;
    if (blockIdx.x == 0) A.entry[lane] = n;
  }
  if (lane == 0) {
    S->total = total;
    S->parts = parts;
    S->extra = (int)extra;
    if (blockIdx.x == 0) {
      A.hdr[0] = parts;
      A.hdr[1] = 0;
      *reinterpret_cast<int64_t*>(A.hdr + 2) = total;
      A.hdr[4] = (int)extra;
    }
  }
}

// A run's pieces in order.
struct TreeWalk {
  int64_t t, begin, end, total;
  int run, e, extra, parts;
  TreeEntry n;
  const TreeSelf* self;   // the CTA's own plan, or NULL
  __device__ __forceinline__ void load(const TreeArgs& A) {
    n = self ? self->entry[e] : tree_load(A, e);
  }
};

__device__ __forceinline__ TreeWalk tree_walk(const TreeArgs& A, int run, const TreeSelf* self) {
  TreeWalk w;
  w.self = self;
  w.parts = self ? self->parts : __ldcg(A.hdr);
  w.total = self ? self->total : __ldcg(reinterpret_cast<const int64_t*>(A.hdr + 2));
  w.extra = self ? self->extra : __ldcg(A.hdr + 4);
  w.run = run;
  w.e = 0;
  w.t = w.begin = w.end = 0;
  if (run < w.parts) {
    w.t = w.begin = tree_run(w.total, w.parts, run);
    w.end = tree_run(w.total, w.parts, run + 1);
    if (self) {   // the first entry that ends behind the run's start (whole warps come here)
      const int lane = threadIdx.x & 31, E = A.per_rank ? A.B * A.L.dcp : A.B;
      const bool behind = lane < E && self->end[lane] > w.begin;
      w.e = __ffs(__ballot_sync(0xffffffffu, behind)) - 1;
    } else {
      w.e = __ldcg(A.run_entry + run);
    }
    w.load(A);
  }
  return w;
}

// The next piece of the walk, if one is left.
__device__ __forceinline__ bool tree_next(const TreeArgs& A, TreeWalk& w, TreePiece& p) {
  while (w.t < w.end) {
    const int unit = w.n.per + w.extra;
    if (w.t >= w.n.tile0 + (int64_t)w.n.units * unit) {
      ++w.e;
      w.load(A);
      continue;
    }
    const int64_t in = w.t - w.n.tile0;
    const int ui = (int)(in / unit), blocks = w.n.units / A.Hkv;
    p.t0 = (int)(in - (int64_t)ui * unit);
    const int64_t left = w.end - w.t;
    const int take = unit - p.t0 < left ? unit - p.t0 : (int)left;   // with empty ones
    p.n = min(p.t0 + take, w.n.per) - p.t0;
    p.slot = p.t0 == 0 && p.n == w.n.per ? -1 : 2 * w.run + (w.t == w.begin ? 0 : 1);
    w.t += take;
    if (p.n <= 0) continue;
    p.u0 = w.n.tile0 + (int64_t)ui * unit;
    p.per = w.n.per;
    p.b = A.per_rank ? w.e / A.L.dcp : w.e;
    p.r0 = A.per_rank ? w.e % A.L.dcp : 0;
    p.r1 = A.per_rank ? p.r0 + 1 : A.L.dcp;
    p.T = w.n.nodes;
    p.ctx = w.n.ctx;
    p.q0 = w.n.q0;
    p.g = ui / blocks;
    p.rb = ui - p.g * blocks;
    return true;
  }
  return false;
}

// Token row of an output row: request row `row` (node * G + head of the group).
__device__ __forceinline__ int64_t tree_out_row(const TreeArgs& A, const TreePiece& p, int row) {
  const int64_t tok = p.q0 + row / A.G;
  return ((int64_t)(A.per_rank ? p.r0 : 0) * A.N + tok) * A.Hq + p.g * A.G + row % A.G;
}

// The tensor-core kernel (dcp_tree_tc.cu): bf16, head_dim 64 or 128, pages of a
// multiple of 16 tokens.  Blocks of 128 or 256 rows, tiles of 128 tokens.
bool tree_tc_shape(int d, dcp_dtype_t dtype, int block_size);
bool tree_tc_supported(const dcp_layout_t& layout, int d, dcp_dtype_t dtype,
                       const dcp_paged_kv_t& kv, int Hkv);
int launch_tree_tc(const TreeArgs& A, cudaStream_t s);

}  // namespace dcp
