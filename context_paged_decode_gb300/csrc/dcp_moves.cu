// Moves of cached bytes: whole pages, and single tokens inside a request.
//
// dcp_pages_copy carries out the copies that a fork or a cut asks for (the
// open page of each, per rank), dcp_cache_compact moves the accepted drafted
// tokens together behind the context:
//     row(ctx + path[i]) -> row(ctx + i),  path strictly increasing.
// Both take every pool of a model (keys and values of all layers) in one
// launch, through a device array of pool pointers.  Both are bound by bytes
// read and written once, and by latency when there are few.
#include "dcp_common.cuh"
#include "dcp_ptx.cuh"

namespace dcp {

struct PoolSet {
  const uint64_t* ptr;   // [num_pools][dcp]
  int num_pools, H, n16; // heads, 16-byte chunks of a row
  int64_t nb;
};

// A usable pool pointer, or NULL.
__device__ __forceinline__ uint4* pool_at(const PoolSet& P, int pool, int dcp, int r) {
  const uint64_t p = __ldcg(P.ptr + (int64_t)pool * dcp + r);
  return (p & 15) ? nullptr : reinterpret_cast<uint4*>(p);
}

constexpr int kCopyThreads = 256;
constexpr int kCopyDepth = 8;     // 16-byte loads in flight per thread
constexpr int kCopyList = 2048;   // most entries of a list that is kept in shared memory
constexpr int kCopyBits = 1 << 15;   // of each set of pages, by the low bits of their numbers
constexpr int kCopySmall = 1024;  // most 16-byte pieces of a small page

// A CTA takes `each` copies of one rank and pool: a page is H * bs rows in one
// piece.  128 open pages of 32 KB on 8 ranks in 2 pools (134 MB) take 23 us from
// HBM, and four of them 2.7 us, bound by two dependent loads.
//
// Copies that touch the same page (one writes what another reads or writes) have
// to keep the order of the list.  CTAs cannot wait for one another, so the first
// of them does all such copies of its rank and pool, where each thread moves the
// same 16 bytes of every page and needs no barrier.  Whether there are any is
// found from the whole list, which the CTA has in shared memory, while the first
// rows of the page are on their way.  Small pages of a long list are shared out to
// few CTAs, where sets of the pages that are read and written say first that there
// are none: with 2048 copies on 8 ranks in 2 pools pages of 2, 4, 8 and 16 KB take
// 60, 62, 90 and 178 us, and 83, 90, 107 and 167 by one CTA a copy that looks for
// no others (looking through the list for each one makes the first 231 us).  Pages
// of 32 KB take 322 us, and 318 so; 344 in few CTAs.
__global__ void __launch_bounds__(kCopyThreads)
pages_copy_kernel(PoolSet P, int dcp, int tables, const int32_t* src,
                  const int32_t* dst, int n, int each, int groups, bool sets, int64_t page16, int32_t* err) {
  extern __shared__ __align__(16) uint32_t s_mem[];
  const bool kept = n > 1 && n <= kCopyList;
  // the sets (pages read, written, written twice), if there are any, and the list
  uint32_t(*const s_set)[kCopyBits / 32] = reinterpret_cast<uint32_t(*)[kCopyBits / 32]>(s_mem);
  int* const s_src = reinterpret_cast<int*>(s_mem) + (sets ? 3 * kCopyBits / 32 : 0);
  int* const s_dst = s_src + n;
  griddep_launch_dependents();   // the next call's first kernel may start its launch
  griddep_wait();                // launched chained: the preceding kernel completed
  const int tid = threadIdx.x;
  const int g = blockIdx.x % groups, pool = blockIdx.x / groups % P.num_pools;
  const int r = blockIdx.x / groups / P.num_pools;
  const int32_t* from = src + (int64_t)(tables == 1 ? 0 : r) * n;
  const int32_t* to = dst + (int64_t)(tables == 1 ? 0 : r) * n;
  uint4* const base = pool_at(P, pool, dcp, r);
  auto moves = [&](int p, int q) {   // can be made, and has work
    return p >= 0 && p < P.nb && q >= 0 && q < P.nb && p != q;
  };
  if (sets) {
    for (int j = tid; j < 3 * kCopyBits / 128; j += kCopyThreads)
      reinterpret_cast<uint4*>(s_mem)[j] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
  }
  if (n > 1) {
#pragma unroll 4
    for (int j = tid; j < n; j += kCopyThreads) {
      const int p = __ldcg(from + j), q = __ldcg(to + j);
      if (kept) {
        s_src[j] = p;
        s_dst[j] = q;
      }
      if (sets && moves(p, q)) {
        const int w = q % kCopyBits / 32;
        const uint32_t bit = 1u << (q & 31);
        atomicOr(&s_set[0][p % kCopyBits / 32], 1u << (p & 31));
        if (atomicOr(&s_set[1][w], bit) & bit) atomicOr(&s_set[2][w], bit);
      }
    }
    __syncthreads();
  }
  auto has = [&](int set, int p) { return (s_set[set][p % kCopyBits / 32] >> (p & 31)) & 1; };
  auto entry = [&](int j, int& p, int& q) {
    p = kept ? s_src[j] : __ldcg(from + j);
    q = kept ? s_dst[j] : __ldcg(to + j);
  };
  // does another copy touch a page of copy k, p -> q? (all threads ask)
  auto shared = [&](int p, int q, int k) {
    if (sets && !has(1, p) && !has(0, q) && !has(2, q)) return false;
    bool hit = false;
    for (int j = tid; j < n; j += kCopyThreads) {
      int x, y;
      entry(j, x, y);
      hit |= j != k && (y == p || x == q || y == q) && moves(x, y);
    }
    return __syncthreads_or(hit) != 0;
  };
  uint4 x[kCopyDepth];
  auto load = [&](int p, int64_t c) {
#pragma unroll
    for (int j = 0; j < kCopyDepth; ++j)
      if (c + j * kCopyThreads < page16) x[j] = __ldcg(base + p * page16 + c + j * kCopyThreads);
  };
  auto store = [&](int q, int64_t c) {
#pragma unroll
    for (int j = 0; j < kCopyDepth; ++j)
      if (c + j * kCopyThreads < page16) base[q * page16 + c + j * kCopyThreads] = x[j];
  };
  const int i1 = min((int64_t)n, ((int64_t)g + 1) * each);
  for (int i = g * each; i < i1; ++i) {
    int a, b;
    entry(i, a, b);
    if (a == -1 && b == -1) continue;
    if (a < 0 || a >= P.nb || b < 0 || b >= P.nb || !base) {
      if (tid == 0) count_error(err);
      continue;
    }
    if (a == b) continue;
    load(a, tid);
    if (n > 1 && shared(a, b, i)) {
      int k = 0, p, q;
      for (; k < i; ++k) {           // an earlier one does them all
        entry(k, p, q);
        if (moves(p, q) && shared(p, q, k)) break;
      }
      if (k < i) continue;
      for (; k < n; ++k) {
        entry(k, p, q);
        if (!moves(p, q) || !shared(p, q, k)) continue;
        for (int64_t c = tid; c < page16; c += kCopyThreads * kCopyDepth) {
          load(p, c);
          store(q, c);
        }
      }
      continue;
    }
    store(b, tid);
    for (int64_t c = tid + kCopyThreads * kCopyDepth; c < page16; c += kCopyThreads * kCopyDepth) {
      load(a, c);
      store(b, c);
    }
  }
}

struct CompactTokArgs {
  Layout L;
  PoolSet P;
  const int32_t* bt;
  int max_vb;
  int64_t stride;
  const int32_t* ctx;
  const int32_t* path;   // [B][max_path]
  const int32_t* n;      // [B]
  int max_path;
  int32_t* new_lens;     // [B] or NULL
  int32_t* err;
};

constexpr int kMoveThreads = 256;
constexpr int kMoveChunk = 128;   // moves resolved at a time
constexpr int kMoveDepth = 8;
constexpr int kMovePtrs = 1024;   // pool addresses kept in shared memory

// blockIdx.x = request, blockIdx.y = share of its columns.  A thread owns a
// 16-byte column of a (pool, head) and moves its rows in order.  Row i goes to
// place i and comes from path[i] >= i, and every later row comes from behind
// place i, so a row is read before anything is written over it, by the thread
// that writes it.  A step's few tokens are bound by the loads that hang on one
// another, so lengths, paths and pool addresses come in one go, then the table
// entries, then the rows (32 requests of 5 tokens, 8 pools: 5.0 us, 6.6 when each
// is loaded where it is needed).
__global__ void __launch_bounds__(kMoveThreads) cache_compact_kernel(const __grid_constant__ CompactTokArgs A) {
  __shared__ int s_sr[kMoveChunk], s_dr[kMoveChunk];          // ranks
  __shared__ int64_t s_src[kMoveChunk], s_dst[kMoveChunk];    // row of head 0 in the rank's pool
  __shared__ uint64_t s_ptr[kMovePtrs];
  __shared__ int s_good;
  griddep_launch_dependents();   // the next call's first kernel may start its launch
  griddep_wait();                // launched chained: the preceding kernel completed
  const int b = blockIdx.x, tid = threadIdx.x;
  const int32_t* path = A.path + (int64_t)b * A.max_path;
  const int dcp = A.L.dcp;
  int node = 0, before = -1;         // this thread's entry of the path, and the one before
  auto entry = [&](int i) {
    if (tid >= kMoveChunk || i >= A.max_path) return;
    node = __ldcg(path + i);
    if (i > 0) before = __ldcg(path + i - 1);
  };
  entry(tid);
  const int ptrs = A.P.num_pools <= kMovePtrs / dcp ? A.P.num_pools * dcp : 0;
  for (int i = tid; i < ptrs; i += kMoveThreads) s_ptr[i] = __ldcg(A.P.ptr + i);
  auto pool_of = [&](int pool, int r) {
    if (ptrs == 0) return pool_at(A.P, pool, dcp, r);
    const uint64_t p = s_ptr[pool * dcp + r];
    return (p & 15) ? nullptr : reinterpret_cast<uint4*>(p);
  };
  const int64_t ctx = __ldcg(A.ctx + b);
  const int n = __ldcg(A.n + b);
  if (ctx < 0 || n < 0 || n > A.max_path) {
    if (blockIdx.y == 0 && tid == 0) {
      count_error(A.err);
      if (A.new_lens) A.new_lens[b] = (int32_t)max(ctx, (int64_t)0);
    }
    return;
  }
  const int64_t cols = (int64_t)A.P.num_pools * A.P.H * A.P.n16;
  int kept = 0;
  for (int i0 = 0; i0 < n; i0 += kMoveChunk) {
    const int m = min(kMoveChunk, n - i0);
    __syncthreads();   // the last chunk's moves are done with the arrays
    if (tid == 0) s_good = m;
    __syncthreads();
    if (tid < m) {
      const int i = i0 + tid;
      if (i0 > 0) entry(i);
      const int64_t p = node;
      bool ok = p >= i && p > before;
      auto place = [&](int64_t x, int& r, int64_t& row) {
        int64_t vb;
        int loc;
        place_token(x, A.L, r, vb, loc);
        const int64_t phys =
            vb < A.max_vb ? (int64_t)__ldcg(A.bt + r * A.stride + (int64_t)b * A.max_vb + vb) : -1;
        if (phys < 0 || phys >= A.P.nb) return false;
        row = phys * A.P.H * A.L.bs + loc;
        return true;
      };
      int sr = 0, dr = 0;
      int64_t src = 0, dst = 0;
      if (ok) ok = place(ctx + p, sr, src) && place(ctx + i, dr, dst);
      s_sr[tid] = sr;
      s_dr[tid] = dr;
      s_src[tid] = src;
      s_dst[tid] = dst;
      if (!ok) atomicMin(&s_good, tid);
    }
    __syncthreads();
    const int good = s_good;
    kept += good;
    // a prefix that stays where it is needs no move
    int first = 0;
    while (first < good && s_src[first] == s_dst[first] && s_sr[first] == s_dr[first]) ++first;
    if (first < good)
      for (int64_t c = blockIdx.y * (int64_t)kMoveThreads + tid; c < cols;
           c += (int64_t)gridDim.y * kMoveThreads) {
        const int chunk = (int)(c % A.P.n16);
        const int h = (int)(c / A.P.n16 % A.P.H);
        const int pool = (int)(c / A.P.n16 / A.P.H);
        const int64_t head = (int64_t)h * A.L.bs;
        for (int j0 = first; j0 < good; j0 += kMoveDepth) {
          uint4 x[kMoveDepth];
#pragma unroll
          for (int j = 0; j < kMoveDepth; ++j)
            if (j0 + j < good) {
              const uint4* p = pool_of(pool, s_sr[j0 + j]);
              if (p) x[j] = __ldcg(p + (s_src[j0 + j] + head) * A.P.n16 + chunk);
            }
#pragma unroll
          for (int j = 0; j < kMoveDepth; ++j)
            if (j0 + j < good) {
              uint4* p = pool_of(pool, s_dr[j0 + j]);
              const bool from = pool_of(pool, s_sr[j0 + j]) != nullptr;
              if (p && from)
                p[(s_dst[j0 + j] + head) * A.P.n16 + chunk] = x[j];
              else if (h == 0 && chunk == 0)
                count_error(A.err);
            }
        }
      }
    if (good < m) {   // nothing behind a bad entry is moved
      if (blockIdx.y == 0 && tid == 0) count_error(A.err);
      break;
    }
  }
  if (A.new_lens && blockIdx.y == 0 && tid == 0) A.new_lens[b] = (int32_t)(ctx + kept);
}

static bool pool_set_ok(const dcp_pool_set_t& p) {
  return p.num_pools >= 0 && p.num_heads >= 1 && p.row_bytes >= 1 && p.num_blocks >= 0;
}

}  // namespace dcp

using namespace dcp;

extern "C" {

int dcp_pages_copy(dcp_layout_t layout, dcp_pool_set_t pools, const int32_t* copy_src,
                   const int32_t* copy_dst, int32_t num_tables, int32_t num, int32_t* err_count,
                   dcp_stream_t stream) {
  dcp::NvtxRange nvtx_range("dcp_pages_copy");
  if (!layout_ok(layout) || !pool_set_ok(pools) || num < 0 ||
      (num_tables != 1 && num_tables != layout.dcp_size))
    return DCP_EINVAL;
  if (pools.row_bytes % 16 != 0) return DCP_EUNSUPPORTED;
  if (num == 0 || pools.num_pools == 0) return DCP_OK;
  if (!pools.ptr || !copy_src || !copy_dst || copy_src == copy_dst) return DCP_EINVAL;
  const PoolSet P{pools.ptr, pools.num_pools, pools.num_heads, pools.row_bytes / 16,
                  pools.num_blocks};
  const int64_t page16 = (int64_t)pools.num_heads * layout.block_size * (pools.row_bytes / 16);
  const int64_t sets = (int64_t)layout.dcp_size * pools.num_pools;
  if (sets >= (int64_t(1) << 30)) return DCP_EUNSUPPORTED;
  const bool small = page16 <= kCopySmall;
  // copies of a CTA: one, unless that would be too many CTAs
  const int64_t most = (int64_t)(small ? 4 : 32) * num_sms();
  const int64_t each = ((int64_t)num * sets + most - 1) / most;
  const int take = (int)(each < num ? each : num), groups = (num - 1) / take + 1;
  const bool filter = small && take >= 4 && num > kCopyThreads;
  const size_t smem = (filter ? 3 * kCopyBits / 8 : 0) +
                      (num > 1 && num <= kCopyList ? 2 * sizeof(int32_t) * num : 0);
  const cudaError_t e = launch_chained(
      pages_copy_kernel, (unsigned)(groups * sets), kCopyThreads, smem, (cudaStream_t)stream, P,
      (int)layout.dcp_size, (int)num_tables, copy_src, copy_dst, (int)num, take, groups, filter,
      page16, err_count);
  if (e != cudaSuccess) return launch_status_report(e);
  return launch_status();
}

int dcp_cache_compact(dcp_layout_t layout, dcp_pool_set_t pools, const int32_t* block_table,
                      int32_t num_reqs, int32_t max_vblocks, int64_t bt_rank_stride,
                      const int32_t* ctx_lens, const int32_t* path, const int32_t* path_len,
                      int32_t max_path, int32_t* new_lens, int32_t* err_count,
                      dcp_stream_t stream) {
  dcp::NvtxRange nvtx_range("dcp_cache_compact");
  if (!layout_ok(layout) || !pool_set_ok(pools) || num_reqs < 0 || max_vblocks < 0 ||
      bt_rank_stride < 0 || max_path < 0)
    return DCP_EINVAL;
  if (pools.row_bytes % 16 != 0 ||
      (int64_t)layout.block_size * layout.dcp_size >= (int64_t(1) << 31))
    return DCP_EUNSUPPORTED;
  if (num_reqs == 0) return DCP_OK;
  if ((pools.num_pools > 0 && !pools.ptr) || !block_table || !ctx_lens || !path_len ||
      (max_path > 0 && !path))
    return DCP_EINVAL;
  // every CTA of a request reads its length, its path and its table, and one stores the new length
  const int64_t each = (int64_t)num_reqs * 4;
  if (!apart({{new_lens, each}},
             {{ctx_lens, each}, {path_len, each}, {path, each * max_path},
              {block_table, (layout.dcp_size - 1) * bt_rank_stride * 4 + each * max_vblocks},
              {pools.ptr, (int64_t)pools.num_pools * layout.dcp_size * 8}}))
    return DCP_EINVAL;
  CompactTokArgs A;
  A.L = Layout{layout.dcp_size, layout.block_size, layout.interleave};
  A.P = PoolSet{pools.ptr, pools.num_pools, pools.num_heads, pools.row_bytes / 16,
                pools.num_blocks};
  A.bt = block_table;
  A.max_vb = max_vblocks;
  A.stride = bt_rank_stride;
  A.ctx = ctx_lens;
  A.path = path;
  A.n = path_len;
  A.max_path = max_path;
  A.new_lens = new_lens;
  A.err = err_count;
  // one column per thread where the card can hold them all (eight CTAs an SM)
  const int64_t cols = (int64_t)pools.num_pools * pools.num_heads * A.P.n16;
  int64_t y = (cols + kMoveThreads - 1) / kMoveThreads;
  const int64_t most = ((int64_t)8 * num_sms() + num_reqs - 1) / num_reqs;
  if (y > most) y = most;
  if (y < 1) y = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)num_reqs, (unsigned)y);
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, cache_compact_kernel, A);
  if (e != cudaSuccess) return launch_status_report(e);
  return launch_status();
}

}  // extern "C"
