// The life of a cache's pages: who holds which, and how many hold one.
//
// State (dcp_pages_t): a block table per rank (or one that all ranks share),
// each request's length, a reference count for each page, and a bitmap of the
// free pages (bit set <=> count 0).  Two operations change it:
//   resize  listed requests to new lengths: pages behind the new length are
//           released, missing ones allocated, and the open page that a cut
//           leaves (partly filled, written next) is replaced by the request's
//           own if others hold it too;
//   fork    children take over their parents' pages: full ones are shared
//           (count + 1), the open one gets a page of the child's own.
// Releases come before allocations, and allocation takes the lowest free page
// for the first need, needs in the order of the list: the result depends on
// nothing but the arguments.  Atomics add to counts and set bits, so their
// order does not matter; two that a request's release and another's share one
// page are both counted before any page is taken.
//
// One cluster of eight CTAs runs each table from end to end; its phases are
// separated by cluster barriers, so a call is one launch (and a small one that
// stores the lengths, which every table reads).  What bounds it: latency, a
// dozen dependent loads and barriers; the entries themselves move at 4096
// threads a table.
#include "dcp_common.cuh"
#include "dcp_ptx.cuh"

namespace dcp {

constexpr int kPgCluster = 8;
constexpr int kPgThreads = 512;
constexpr int kPgAll = kPgCluster * kPgThreads;   // threads of a table

struct PagesArgs {
  Layout L;
  int32_t* bt;
  int64_t stride;      // entries between tables
  int B, max_vb;
  int64_t nb;
  int words;           // of the bitmap
  int shared;          // one table for every rank
  int32_t* seq;
  int32_t* ref;
  uint32_t* bits;
  const int32_t* up;   // fork: parent rows
  const int32_t* row;  // requests that change
  const int32_t* len;  // resize: their new lengths
  int N;
  int32_t* src;        // [tables][N]
  int32_t* dst;
  char* ws;
  size_t ws_table;     // workspace bytes of a table
  int32_t* err;
};

// Workspace of one table: claim[B] (which list entry owns a request),
// need[N] (pages << 1 | replaces the open page), first[N + 1] (needs before
// n), old[N] (page to release after the allocation), sums[kPgCluster].
struct PagesWs {
  int32_t *claim, *need, *first, *old, *sums;
};

__host__ __device__ inline size_t pages_ws_table(int64_t B, int64_t N) {
  return ((size_t)(B + 3 * N + 1 + kPgCluster) * sizeof(int32_t) + 255) / 256 * 256;
}

__device__ __forceinline__ PagesWs pages_ws(const PagesArgs& A, int table) {
  PagesWs w;
  w.claim = (int32_t*)(A.ws + A.ws_table * table);
  w.need = w.claim + A.B;
  w.first = w.need + A.N;
  w.old = w.first + A.N + 1;
  w.sums = w.old + A.N;
  return w;
}

// Tokens of the open page of a length on rank r (0 .. bs; a shared table's
// page stands for the whole virtual block).
__device__ __forceinline__ int open_tokens(const PagesArgs& A, int64_t len, int r) {
  const int vbs = A.L.bs * A.L.dcp, turn = A.L.I * A.L.dcp;
  const int rem = (int)(len % vbs);
  if (A.shared) return rem;
  return rem / turn * A.L.I + min(max(rem % turn - r * A.L.I, 0), A.L.I);
}

// State is read past the SM's L1 (__ldcg) throughout: other CTAs write it in
// this call, and the kernels of the call before may still run when this one is
// launched.
struct PagesReq {
  bool ok;
  int c;          // row that changes
  int p;          // fork: parent
  int64_t old, len;
  int ov, nv;     // virtual blocks held before and after
};

// One entry of the list, checked.  Reads claim, so only after its barrier.
template <bool kFork>
__device__ __forceinline__ PagesReq pages_req(const PagesArgs& A, const PagesWs& w, int n) {
  PagesReq q;
  const int64_t vbs = (int64_t)A.L.bs * A.L.dcp;
  q.ok = false;
  q.c = __ldcg(A.row + n);
  q.p = kFork ? __ldcg(A.up + n) : -1;
  q.old = q.len = 0;
  q.ov = q.nv = 0;
  if (q.c < 0 || q.c >= A.B || __ldcg(w.claim + q.c) != n) return q;
  if (kFork) {
    // a parent that the same call overwrites has no defined pages
    if (q.p < 0 || q.p >= A.B || __ldcg(w.claim + q.p) != 0x7fffffff) return q;
    q.len = __ldcg(A.seq + q.p);
  } else {
    q.len = __ldcg(A.len + n);
  }
  q.old = max(__ldcg(A.seq + q.c), 0);
  if (q.len < 0 || (q.len + vbs - 1) / vbs > A.max_vb) return q;
  q.nv = (int)((q.len + vbs - 1) / vbs);
  q.ov = (int)min((q.old + vbs - 1) / vbs, (int64_t)A.max_vb);
  q.ok = true;
  return q;
}

__device__ __forceinline__ void release_page(const PagesArgs& A, int32_t* ref, uint32_t* bits,
                                             int id) {
  if (id < 0 || id >= A.nb) {
    count_error(A.err);
    return;
  }
  const int was = atomicSub(ref + id, 1);
  if (was == 1) atomicOr(bits + (id >> 5), 1u << (id & 31));
  if (was <= 0) {   // nobody held it: put the count back
    atomicAdd(ref + id, 1);
    count_error(A.err);
  }
}

// Exclusive scan over the CTA; *total gets the sum.
__device__ __forceinline__ int pg_scan(int v, int* sh, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) sh[w] = x;
  __syncthreads();
  int before = 0, sum = 0;
  for (int i = 0; i < kPgThreads / 32; ++i) {
    if (i < w) before += sh[i];
    sum += sh[i];
  }
  *total = sum;
  return before + x - v;
}

template <bool kFork>
__global__ void __cluster_dims__(kPgCluster, 1, 1) __launch_bounds__(kPgThreads)
pages_kernel(const __grid_constant__ PagesArgs A) {
  __shared__ int sh[kPgThreads / 32];
  griddep_launch_dependents();   // the next call's first kernel may start its launch
  griddep_wait();                // launched chained: the preceding kernel completed
  const int table = blockIdx.x / kPgCluster;
  const int cta = (int)cluster_ctarank();
  const int tid = threadIdx.x, lane = tid & 31;
  const int gid = cta * kPgThreads + tid;
  const PagesWs w = pages_ws(A, table);
  int32_t* bt = A.bt + table * A.stride;
  int32_t* ref = A.ref + (int64_t)table * A.nb;
  uint32_t* bits = A.bits + (int64_t)table * A.words;
  int32_t* src = A.src + (int64_t)table * A.N;
  int32_t* dst = A.dst + (int64_t)table * A.N;
  const int full = A.shared ? A.L.bs * A.L.dcp : A.L.bs;   // tokens that fill an open page

  // who changes which request: the first entry that names it
  for (int i = gid; i < A.B; i += kPgAll) w.claim[i] = 0x7fffffff;
  cluster_sync();
  for (int n = gid; n < A.N; n += kPgAll) {
    const int c = __ldcg(A.row + n);
    if (c >= 0 && c < A.B) atomicMin(w.claim + c, n);
  }
  cluster_sync();

  // releases.  `share` warps take turns on one entry where there are few.
  const int nwarps = kPgAll / 32, gw = gid >> 5;
  const int share = A.N < nwarps ? nwarps / max(A.N, 1) : 1;
  for (int n = gw / share; n < A.N; n += nwarps / share) {
    const PagesReq q = pages_req<kFork>(A, w, n);
    if (!q.ok) continue;
    int32_t* row = bt + (int64_t)q.c * A.max_vb;
    const int v0 = kFork ? 0 : q.nv;
    const int step = 32 * share;
    for (int v = v0 + (gw % share) * 32 + lane; v < q.ov; v += 4 * step) {
      int id[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) id[j] = v + j * step < q.ov ? __ldcg(row + v + j * step) : 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (v + j * step < q.ov) {
          release_page(A, ref, bits, id[j]);
          row[v + j * step] = -1;
        }
    }
  }
  cluster_sync();

  // needs of each entry, and the free pages of each CTA's part of the bitmap
  for (int n = gid; n < A.N; n += kPgAll) {
    const PagesReq q = pages_req<kFork>(A, w, n);
    int need = 0, again = 0;
    src[n] = dst[n] = -1;
    w.old[n] = -1;
    if (!q.ok) {
      if (table == 0) count_error(A.err);
    } else {
      const int64_t cut = kFork ? q.len : min(q.old, q.len);
      const int64_t vbs = (int64_t)A.L.bs * A.L.dcp;
      const int cv = (int)(cut / vbs);
      if (cut % vbs != 0 && open_tokens(A, cut, table) < full) {
        if (kFork) {
          again = 1;
        } else {
          const int id = __ldcg(bt + (int64_t)q.c * A.max_vb + cv);
          again = id >= 0 && id < A.nb && __ldcg(ref + id) > 1;
        }
      }
      need = again + (kFork ? 0 : max(q.nv - q.ov, 0));
    }
    w.need[n] = need << 1 | again;
  }
  const int per = (A.words + kPgAll - 1) / kPgAll;
  const int w0 = min(gid * per, A.words), w1 = min(w0 + per, A.words);
  int mine = 0, sum;
  for (int i = w0; i < w1; ++i) mine += __popc(__ldcg(bits + i));
  int base = pg_scan(mine, sh, &sum);
  if (tid == 0) w.sums[cta] = sum;
  cluster_sync();

  // CTA 0 counts the needs before each entry
  if (cta == 0) {
    int run = 0;
    for (int n0 = 0; n0 < A.N; n0 += kPgThreads) {
      const int n = n0 + tid;
      const int v = n < A.N ? __ldcg(w.need + n) >> 1 : 0;
      const int at = pg_scan(v, sh, &sum);
      if (n < A.N) w.first[n] = run + at;
      run += sum;
    }
    if (tid == 0) w.first[A.N] = run;
  }
  cluster_sync();

  // page k of the free ones, in increasing order, goes to need k
  const int W = __ldcg(w.first + A.N);
  int have = 0;
  for (int i = 0; i < kPgCluster; ++i) {
    const int s = __ldcg(w.sums + i);
    if (i < cta) base += s;
    have += s;
  }
  auto give = [&](int k, int id) {
    int lo = 0, hi = A.N;   // first[lo] <= k < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldcg(w.first + mid) <= k) lo = mid; else hi = mid;
    }
    const PagesReq q = pages_req<kFork>(A, w, lo);
    int j = k - __ldcg(w.first + lo);
    int32_t* row = bt + (int64_t)q.c * A.max_vb;
    if (__ldcg(w.need + lo) & 1) {
      if (j == 0) {   // the open page
        const int64_t cut = kFork ? q.len : min(q.old, q.len);
        const int cv = (int)(cut / ((int64_t)A.L.bs * A.L.dcp));
        const int from = __ldcg(kFork ? bt + (int64_t)q.p * A.max_vb + cv : row + cv);
        if (!kFork) w.old[lo] = from;
        if (open_tokens(A, cut, table) > 0) {
          if (from < 0 || from >= A.nb) {
            count_error(A.err);
          } else if (id >= 0) {
            src[lo] = from;
            dst[lo] = id;
          }
        }
        row[cv] = id;
        return;
      }
      --j;
    }
    row[q.ov + j] = id;
  };
  if (mine > 0 && base < W) {
    int k = base;
    for (int i = w0; i < w1 && k < W; ++i) {
      uint32_t word = __ldcg(bits + i), taken = 0;
      while (word && k < W) {
        const int bit = __ffs(word) - 1;
        word &= word - 1;
        taken |= 1u << bit;
        const int id = i * 32 + bit;
        ref[id] = 1;
        give(k++, id);
      }
      if (taken) atomicAnd(bits + i, ~taken);
    }
  }
  for (int k = have + gid; k < W; k += kPgAll) {   // no page left
    count_error(A.err);
    give(k, -1);
  }
  cluster_sync();

  if (kFork) {
    // the parents' other pages, one holder more
    for (int n = gw / share; n < A.N; n += nwarps / share) {
      const PagesReq q = pages_req<true>(A, w, n);
      if (!q.ok) continue;
      const int32_t* from = bt + (int64_t)q.p * A.max_vb;
      int32_t* row = bt + (int64_t)q.c * A.max_vb;
      const int nv = q.nv - (__ldcg(w.need + n) & 1);   // the open page has been given
      const int step = 32 * share;
      for (int v = (gw % share) * 32 + lane; v < nv; v += 4 * step) {
        int id[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) id[j] = v + j * step < nv ? __ldcg(from + v + j * step) : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (v + j * step >= nv) continue;
          if (id[j] < 0 || id[j] >= A.nb) {
            count_error(A.err);
            id[j] = -1;
          } else {
            atomicAdd(ref + id[j], 1);
          }
          row[v + j * step] = id[j];
        }
      }
    }
  } else {
    // the shared open pages that were replaced, one holder less
    for (int n = gid; n < A.N; n += kPgAll) {
      const int id = __ldcg(w.old + n);
      if (id >= 0) release_page(A, ref, bits, id);
    }
  }
}

// The lengths, once every table has read the old ones (table 0's claims).
template <bool kFork>
__global__ void pages_lens_kernel(const __grid_constant__ PagesArgs A) {
  griddep_launch_dependents();
  griddep_wait();
  const PagesWs w = pages_ws(A, 0);
  for (int n = blockIdx.x * blockDim.x + threadIdx.x; n < A.N; n += gridDim.x * blockDim.x) {
    const PagesReq q = pages_req<kFork>(A, w, n);
    if (q.ok) A.seq[q.c] = (int32_t)q.len;
  }
}

__global__ void pages_init_kernel(int32_t* bt, int64_t entries, int32_t* seq, int B, int32_t* ref,
                                  int64_t pages, uint32_t* bits, int64_t words, int wpt,
                                  int64_t nb) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  const int64_t i0 = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  for (int64_t i = i0; i < entries; i += step) bt[i] = -1;
  for (int64_t i = i0; i < B; i += step) seq[i] = 0;
  for (int64_t i = i0; i < pages; i += step) ref[i] = 0;
  for (int64_t i = i0; i < words; i += step) {
    const int64_t left = nb - (i % wpt) * 32;
    bits[i] = left >= 32 ? 0xffffffffu : (left > 0 ? (1u << left) - 1u : 0u);
  }
}

static int pages_tables(const dcp_layout_t& L, const dcp_pages_t& p) {
  return p.bt_rank_stride == 0 ? 1 : L.dcp_size;
}

static int pages_ok(const dcp_layout_t& L, const dcp_pages_t& p) {
  if (!layout_ok(L) || p.num_reqs < 0 || p.max_vblocks < 0 || p.num_blocks < 0 ||
      p.bt_rank_stride < 0 ||
      (p.bt_rank_stride != 0 && p.bt_rank_stride < (int64_t)p.num_reqs * p.max_vblocks))
    return DCP_EINVAL;
  if (p.num_blocks >= (int64_t(1) << 31) - 32 ||
      (int64_t)p.max_vblocks * L.block_size * L.dcp_size >= (int64_t(1) << 31))
    return DCP_EUNSUPPORTED;
  if ((p.num_reqs > 0 && (!p.seq_lens || (p.max_vblocks > 0 && !p.block_table))) ||
      (p.num_blocks > 0 && (!p.ref_count || !p.free_bits)))
    return DCP_EINVAL;
  return DCP_OK;
}

template <bool kFork>
static int launch_pages(const dcp_layout_t& L, const dcp_pages_t& p, const int32_t* up,
                        const int32_t* row, const int32_t* len, int N, int32_t* src, int32_t* dst,
                        void* ws, size_t ws_bytes, int32_t* err, cudaStream_t s) {
  const int rc = pages_ok(L, p);
  if (rc != DCP_OK) return rc;
  if (N < 0) return DCP_EINVAL;
  if (N == 0) return DCP_OK;
  if (!row || (kFork ? !up : !len) || !src || !dst) return DCP_EINVAL;
  if ((int64_t)N * p.max_vblocks >= (int64_t(1) << 30)) return DCP_EUNSUPPORTED;
  const int tables = pages_tables(L, p);
  PagesArgs A;
  A.L = Layout{L.dcp_size, L.block_size, L.interleave};
  A.bt = p.block_table;
  A.stride = p.bt_rank_stride;
  A.B = p.num_reqs;
  A.max_vb = p.max_vblocks;
  A.nb = p.num_blocks;
  A.words = (int)((p.num_blocks + 31) / 32);
  A.shared = p.bt_rank_stride == 0 ? 1 : 0;
  A.seq = p.seq_lens;
  A.ref = p.ref_count;
  A.bits = p.free_bits;
  A.up = up;
  A.row = row;
  A.len = len;
  A.N = N;
  A.src = src;
  A.dst = dst;
  A.ws = (char*)ws;
  A.ws_table = pages_ws_table(p.num_reqs, N);
  A.err = err;
  if (!ws || ws_bytes < A.ws_table * tables) return DCP_EWORKSPACE;
  cudaError_t e = launch_chained(pages_kernel<kFork>, (unsigned)(tables * kPgCluster), kPgThreads,
                                 0, s, A);
  if (e != cudaSuccess) return launch_status_report(e);
  const unsigned grid = (unsigned)((N + 255) / 256 < 64 ? (N + 255) / 256 : 64);
  e = launch_chained(pages_lens_kernel<kFork>, grid, 256, 0, s, A);
  if (e != cudaSuccess) return launch_status_report(e);
  return launch_status();
}

}  // namespace dcp

using namespace dcp;

extern "C" {

int dcp_pages_init(dcp_layout_t layout, dcp_pages_t pages, dcp_stream_t stream) {
  dcp::NvtxRange nvtx_range("dcp_pages_init");
  const int rc = pages_ok(layout, pages);
  if (rc != DCP_OK) return rc;
  const int tables = pages_tables(layout, pages);
  const int wpt = (int)((pages.num_blocks + 31) / 32);
  // tables lie bt_rank_stride apart; what lies between them is not written
  const int64_t per = (int64_t)pages.num_reqs * pages.max_vblocks;
  for (int t = 0; t < tables; ++t) {
    const cudaError_t e = launch_chained(
        pages_init_kernel, (unsigned)(2 * num_sms()), 256, 0, (cudaStream_t)stream,
        pages.block_table + t * pages.bt_rank_stride, per, pages.seq_lens,
        t == 0 ? (int)pages.num_reqs : 0, pages.ref_count + t * pages.num_blocks, pages.num_blocks,
        pages.free_bits + (int64_t)t * wpt, (int64_t)wpt, wpt > 0 ? wpt : 1, pages.num_blocks);
    if (e != cudaSuccess) return launch_status_report(e);
  }
  return launch_status();
}

int dcp_pages_workspace_size(dcp_layout_t layout, dcp_pages_t pages, int32_t num, size_t* bytes) {
  const int rc = pages_ok(layout, pages);
  if (rc != DCP_OK) return rc;
  if (!bytes || num < 0) return DCP_EINVAL;
  *bytes = pages_ws_table(pages.num_reqs, num) * pages_tables(layout, pages);
  return DCP_OK;
}

int dcp_pages_resize(dcp_layout_t layout, dcp_pages_t pages, const int32_t* req,
                     const int32_t* new_lens, int32_t num, int32_t* copy_src, int32_t* copy_dst,
                     void* workspace, size_t workspace_bytes, int32_t* err_count,
                     dcp_stream_t stream) {
  dcp::NvtxRange nvtx_range("dcp_pages_resize");
  return launch_pages<false>(layout, pages, nullptr, req, new_lens, num, copy_src, copy_dst,
                             workspace, workspace_bytes, err_count, (cudaStream_t)stream);
}

int dcp_pages_fork(dcp_layout_t layout, dcp_pages_t pages, const int32_t* parent,
                   const int32_t* child, int32_t num, int32_t* copy_src, int32_t* copy_dst,
                   void* workspace, size_t workspace_bytes, int32_t* err_count,
                   dcp_stream_t stream) {
  dcp::NvtxRange nvtx_range("dcp_pages_fork");
  return launch_pages<true>(layout, pages, parent, child, nullptr, num, copy_src, copy_dst,
                            workspace, workspace_bytes, err_count, (cudaStream_t)stream);
}

}  // extern "C"
