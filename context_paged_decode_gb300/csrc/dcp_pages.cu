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
// Clusters of eight CTAs run the tables from end to end, with two or three
// cluster barriers: one for all tables if the work is small, whose CTAs are
// divided among them, else one for each.  One cluster stores the lengths,
// which every table reads, itself, after its first barrier; several leave that
// to a small second launch.  What bounds it: latency.  So each CTA checks the whole
// list for itself in shared memory (a hash of the requests finds names that
// come twice, and children that are parents) rather than ask the others, and
// pages are handed out 32 at a time, a lane per bit of the bitmap.  (With the
// claims and prefix sums in global memory and a thread per bitmap word, 128
// forks of 250 pages on 8 ranks took 41 us, and 128 requests of a few new
// pages 28; they take 16 and 14 now, 2 us of launch in each.)
#include "dcp_common.cuh"
#include "dcp_ptx.cuh"

namespace dcp {

constexpr int kPgCluster = 8;
constexpr int kPgThreads = 512;
constexpr int kPgMaxList = 2048;
// Most table columns (and 32 for each list entry) of a CTA for one cluster to do
// all tables.  Free, fork, copy and grow of 4 requests of 33 columns on 2 ranks
// take 25.3 us so and 28.9 us with a cluster for each, 16 requests of 252
// columns on 8 ranks (4544 to a CTA) 33.1 and 36.0; but 32 such requests (9088)
// 48.6 and 41.8, 128 of 33 columns (8320) 63.0 and 46.2.
constexpr int64_t kPgSmall = 5120;
// And most of them for a CTA alone to do a table, whose threads then meet in
// the CTA: those 4 requests 20.9 us, 23.0 with four CTAs a table; 12 of them
// (780) 21.5 and 23.8, but 32 (2080) 27.1 and 26.6.
constexpr int64_t kPgOne = 1024;

struct PagesArgs {
  Layout L;
  int32_t* bt;
  int64_t stride;      // entries between tables
  int B, max_vb;
  int64_t nb;
  int words;           // of the bitmap
  int shared;          // one table for every rank
  int tables, per;     // CTAs of each: kPgCluster, or a power of two below
  int alone;           // one cluster does everything
  int32_t* seq;
  int32_t* ref;
  uint32_t* bits;
  const int32_t* up;   // fork: parent rows
  const int32_t* row;  // requests that change
  const int32_t* len;  // resize: their new lengths
  int N, hash;         // list entries, slots of the hash (a power of two)
  int32_t* src;        // [tables][N]
  int32_t* dst;
  int32_t* sums;       // workspace: free pages of each CTA's words [tables][kPgCluster]
  int32_t* new_len;    // workspace: [N] what the lengths become (-1: entry skipped)
  int32_t* err;
};

// Shared memory of a CTA, in ints: the list and what was found about it.  The
// hash is done with when needs are counted, and lies over the arrays for that.
struct PagesList {
  int *c, *p, *old, *len;          // request (-1: skipped), parent, old and new length
  int *first, *need, *page;        // needs before n [N + 1], needs << 1 | open page again, page
  int *key, *val;
  __device__ __forceinline__ PagesList(int* sm, int N, int hash) {
    c = sm;
    p = c + N;
    old = p + N;
    len = old + N;
    first = len + N;
    need = first + N + 1;
    page = need + N;
    key = first;
    val = key + hash;
  }
};

static size_t pages_smem(int N, int hash) {
  const size_t over = (size_t)2 * hash > (size_t)3 * N + 1 ? (size_t)2 * hash : (size_t)3 * N + 1;
  return ((size_t)4 * N + over) * sizeof(int32_t);
}

// Tokens of the open page of a length on rank r (0 .. bs; a shared table's
// page stands for the whole virtual block).
__device__ __forceinline__ int open_tokens(const PagesArgs& A, int len, int r) {
  const int vbs = A.L.bs * A.L.dcp, turn = A.L.I * A.L.dcp;
  const int rem = len % vbs;
  if (A.shared) return rem;
  return rem / turn * A.L.I + min(max(rem % turn - r * A.L.I, 0), A.L.I);
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

// State is read past the SM's L1 (__ldcg) throughout: other CTAs write it in
// this call, and the kernels of the call before may still run when this one is
// launched.
template <bool kFork>
__global__ void __cluster_dims__(kPgCluster, 1, 1) __launch_bounds__(kPgThreads)
pages_kernel(const __grid_constant__ PagesArgs A) {
  extern __shared__ int sm[];
  __shared__ int sh[kPgThreads / 32];
  __shared__ int s_any, s_needs;
  griddep_launch_dependents();   // the next call's first kernel may start its launch
  griddep_wait();                // launched chained: the preceding kernel completed
  const int table = blockIdx.x / A.per, cta = blockIdx.x % A.per;
  const int tid = threadIdx.x, lane = tid & 31;
  const int gw = cta * (kPgThreads / 32) + (tid >> 5);   // warp of the table
  const int warps = A.per * (kPgThreads / 32);           // and how many it has
  const int N = A.N, vbs = A.L.bs * A.L.dcp;
  // a CTA too many checks the list and keeps step, and has no work
  const bool spare = table >= A.tables;
  const int mine_n = spare ? 0 : N, words = spare ? 0 : A.words;
  int32_t* bt = A.bt + table * A.stride;
  int32_t* ref = A.ref + (int64_t)table * A.nb;
  uint32_t* bits = A.bits + (int64_t)table * A.words;
  int32_t* src = A.src + (int64_t)table * N;
  int32_t* dst = A.dst + (int64_t)table * N;
  const int full = A.shared ? vbs : A.L.bs;   // tokens that fill an open page
  auto table_sync = [&]() {                   // of a table's CTAs, and whoever shares their cluster
    if (A.per == 1) __syncthreads(); else cluster_sync();
  };
  auto blocks = [&](int len) { return (int)(((int64_t)len + vbs - 1) / vbs); };

  // the list, and the first entry that names each request
  PagesList S(sm, N, A.hash);
  if (tid == 0) s_any = s_needs = 0;
  for (int n = tid; n < N; n += kPgThreads) {
    S.c[n] = __ldcg(A.row + n);
    S.p[n] = kFork ? __ldcg(A.up + n) : __ldcg(A.len + n);
  }
  for (int i = tid; i < A.hash; i += kPgThreads) {
    S.key[i] = -1;
    S.val[i] = 0x7fffffff;
  }
  __syncthreads();
  auto slot = [&](int c) { return (int)((uint32_t)c * 2654435761u >> 7) & (A.hash - 1); };
  for (int n = tid; n < N; n += kPgThreads) {
    const int c = S.c[n];
    if (c < 0 || c >= A.B) continue;
    int h = slot(c);
    for (;;) {   // ends: the hash has at least twice as many slots as entries
      const int k = atomicCAS(S.key + h, -1, c);
      if (k == -1 || k == c) break;
      h = (h + 1) & (A.hash - 1);
    }
    atomicMin(S.val + h, n);
  }
  __syncthreads();
  auto named = [&](int c) {   // first entry that names c, or none
    int h = slot(c);
    while (S.key[h] != c && S.key[h] != -1) h = (h + 1) & (A.hash - 1);
    return S.key[h] == c ? S.val[h] : 0x7fffffff;
  };
  for (int n = tid; n < N; n += kPgThreads) {
    const int c = S.c[n], x = S.p[n];
    bool ok = c >= 0 && c < A.B && named(c) == n;
    int old = 0, len = x;
    // a parent that the same call overwrites has no defined pages
    if (ok && kFork) ok = x >= 0 && x < A.B && named(x) == 0x7fffffff;
    if (ok) {
      old = max(__ldcg(A.seq + c), 0);
      if (kFork) len = __ldcg(A.seq + x);
      ok = len >= 0 && blocks(len) <= A.max_vb;
    }
    S.old[n] = min(blocks(old), A.max_vb) == blocks(old) ? old : A.max_vb * vbs;
    S.len[n] = ok ? len : -1;
    if (!kFork && ok && (blocks(len) > blocks(S.old[n]) || min(S.old[n], len) % vbs != 0))
      s_needs = 1;
    if (table == 0 && cta == 0) {
      if (!ok) count_error(A.err);
      if (!A.alone) A.new_len[n] = ok ? len : -1;
    }
  }
  __syncthreads();   // (the hash is read for the last time above)

  // Releases, and for a fork the pages that the child shares with its parent.
  // The parent holds those throughout, so no release can free one.  `share`
  // warps take turns on an entry where there are few.
  const int share = N < warps ? warps / N : 1;
  for (int n = gw / share; n < mine_n; n += warps / share) {
    const int len = S.len[n];
    if (len < 0) continue;
    int32_t* row = bt + (int64_t)S.c[n] * A.max_vb;
    const int32_t* from = bt + (int64_t)(kFork ? S.p[n] : 0) * A.max_vb;
    const int ov = blocks(S.old[n]), nv = blocks(len);
    // a fork's last page is not shared if it is open
    const int kept = kFork ? nv - (len % vbs != 0 && open_tokens(A, len, table) < full) : 0;
    const int v0 = kFork ? 0 : nv, v1 = max(ov, kept), step = 32 * share;
    for (int v = v0 + (gw % share) * 32 + lane; v < v1; v += 4 * step) {
      int gone[4], take[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int u = v + j * step;
        gone[j] = u < ov ? __ldcg(row + u) : -1;
        take[j] = u < kept ? __ldcg(from + u) : -1;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int u = v + j * step;
        if (u >= v1) continue;
        if (u < ov) release_page(A, ref, bits, gone[j]);
        int id = -1;
        if (u < kept) {
          if (take[j] >= 0 && take[j] < A.nb) {
            id = take[j];
            atomicAdd(ref + id, 1);
          } else {
            count_error(A.err);
          }
        }
        row[u] = id;
      }
    }
  }
  if (A.tables == 1) table_sync(); else cluster_sync();
  if (A.alone && blockIdx.x == 0)   // every table has read the old lengths
    for (int n = tid; n < N; n += kPgThreads)
      if (S.len[n] >= 0) A.seq[S.c[n]] = S.len[n];

  // Nothing to take when the lengths alone say so, as in every table: requests
  // that are freed, or cut at the end of a page.
  if (!kFork && !s_needs) {
    for (int n = cta * kPgThreads + tid; n < mine_n; n += warps * 32) src[n] = dst[n] = -1;
    return;
  }

  // what each entry needs, summed up by every CTA for itself
  int W = 0;
  for (int n0 = 0; n0 < mine_n; n0 += kPgThreads) {
    const int n = n0 + tid;
    int need = 0, again = 0, page = -1;
    if (n < N && S.len[n] >= 0) {
      const int old = S.old[n], len = S.len[n], cut = kFork ? len : min(old, len);
      const int cv = cut / vbs;
      if (cut % vbs != 0 && open_tokens(A, cut, table) < full) {
        page = __ldcg(bt + (int64_t)(kFork ? S.p[n] : S.c[n]) * A.max_vb + cv);
        again = kFork || (page >= 0 && page < A.nb && __ldcg(ref + page) > 1);
      }
      need = again + (kFork ? 0 : max(blocks(len) - blocks(old), 0));
    }
    int sum;
    const int at = pg_scan(need, sh, &sum);
    if (n < N) {
      S.first[n] = W + at;
      S.need[n] = need << 1 | again;
      S.page[n] = page;
      if (again) s_any = 1;
      if (n / kPgThreads % A.per == cta) src[n] = dst[n] = -1;
    }
    W += sum;
  }
  if (tid == 0) S.first[N] = W;
  // free pages of this warp's words
  const int each = (words + warps - 1) / warps;
  const int w0 = min(gw * each, words), w1 = min(w0 + each, words);
  int mine = 0, sum;
  for (int i = w0 + lane; i < w1; i += 32) mine += __popc(__ldcg(bits + i));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  int base = pg_scan(lane == 0 ? mine : 0, sh, &sum);
  base = __shfl_sync(0xffffffffu, base, 0);
  if (tid == 0 && A.per > 1) A.sums[blockIdx.x] = sum;
  table_sync();

  int have = A.per == 1 ? sum : 0;
  for (int i = 0; i < A.per && A.per > 1; ++i) {
    const int s = __ldcg(A.sums + table * A.per + i);
    if (i < cta) base += s;
    have += s;
  }
  // page k of the free ones, in increasing order, goes to need k
  auto give = [&](int k, int id) {
    int lo = 0, hi = N;   // first[lo] <= k < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (S.first[mid] <= k) lo = mid; else hi = mid;
    }
    int j = k - S.first[lo];
    int32_t* row = bt + (int64_t)S.c[lo] * A.max_vb;
    if (S.need[lo] & 1) {
      if (j == 0) {   // the open page
        const int cut = kFork ? S.len[lo] : min(S.old[lo], S.len[lo]);
        const int from = S.page[lo];
        if (open_tokens(A, cut, table) > 0) {
          if (from < 0 || from >= A.nb) {
            count_error(A.err);
          } else if (id >= 0) {
            src[lo] = from;
            dst[lo] = id;
          }
        }
        row[cut / vbs] = id;
        return;
      }
      --j;
    }
    row[blocks(S.old[lo]) + j] = id;
  };
  for (int i0 = w0; i0 < w1 && base < W; i0 += 32) {
    const uint32_t mine_w = i0 + lane < w1 ? __ldcg(bits + i0 + lane) : 0u;
    for (int i = i0; i < min(i0 + 32, w1) && base < W; ++i) {
      const uint32_t word = __shfl_sync(0xffffffffu, mine_w, i - i0);
      const int k = base + __popc(word & ((1u << lane) - 1u));
      const bool take = ((word >> lane) & 1) && k < W;
      if (take) {
        const int id = i * 32 + lane;
        ref[id] = 1;
        give(k, id);
      }
      const uint32_t taken = __ballot_sync(0xffffffffu, take);
      if (lane == 0 && taken) bits[i] = word & ~taken;
      base += __popc(word);
    }
  }
  for (int k = have + cta * kPgThreads + tid; k < W; k += warps * 32) {   // no page left
    count_error(A.err);
    give(k, -1);
  }
  if (!kFork && (s_any || A.per < kPgCluster)) {   // (the same in a table's CTAs)
    // the shared open pages that were replaced, one holder less
    table_sync();
    for (int n = cta * kPgThreads + tid; n < mine_n; n += warps * 32)
      if (S.need[n] & 1) release_page(A, ref, bits, S.page[n]);
  }
}

// The lengths, once every table has read the old ones.
__global__ void pages_lens_kernel(const __grid_constant__ PagesArgs A) {
  griddep_launch_dependents();
  griddep_wait();
  for (int n = blockIdx.x * blockDim.x + threadIdx.x; n < A.N; n += gridDim.x * blockDim.x) {
    const int len = __ldcg(A.new_len + n);
    if (len >= 0) A.seq[__ldcg(A.row + n)] = len;
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

static size_t pages_ws_bytes(int N) {
  return (size_t)(DCP_MAX_RANKS * kPgCluster + N) * sizeof(int32_t);
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
      (int64_t)L.block_size * L.dcp_size >= (int64_t(1) << 31) ||
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
  if (N > kPgMaxList || (int64_t)N * p.max_vblocks >= (int64_t(1) << 30)) return DCP_EUNSUPPORTED;
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
  A.tables = tables;
  A.per = kPgCluster;
  while (A.per > 0 && A.per * tables > kPgCluster) A.per /= 2;
  A.alone = tables == 1 || (int64_t)N * (p.max_vblocks + 32) <= kPgSmall * A.per;
  if (!A.alone) A.per = kPgCluster;
  if (A.alone && (int64_t)N * (p.max_vblocks + 32) <= kPgOne) A.per = 1;
  A.N = N;
  A.hash = 64;
  while (A.hash < 2 * N) A.hash *= 2;
  A.src = src;
  A.dst = dst;
  A.sums = (int32_t*)ws;
  A.new_len = A.sums + DCP_MAX_RANKS * kPgCluster;
  A.err = err;
  if (!ws || ws_bytes < pages_ws_bytes(N) || ((uintptr_t)ws & 3)) return DCP_EWORKSPACE;
  // Other CTAs still read the list while these are written, and the lengths are
  // stored by its requests at the end: a list that changes meanwhile would name
  // requests that were never checked.  (New lengths are read before any are
  // stored, so the state's own may be the list.)
  const int64_t list = (int64_t)N * 4, T = tables;
  const Bytes state[4] = {
      {p.block_table, ((T - 1) * p.bt_rank_stride + (int64_t)p.num_reqs * p.max_vblocks) * 4},
      {p.ref_count, T * p.num_blocks * 4},
      {p.free_bits, T * A.words * 4},
      {p.seq_lens, (int64_t)p.num_reqs * 4}};
  const Bytes which{row, list}, other{kFork ? up : len, list};
  if (!apart({{src, T * list}, {dst, T * list}, {ws, (int64_t)pages_ws_bytes(N)}},
             {which, other, state[0], state[1], state[2], state[3]}) ||
      !apart({state[0], state[1], state[2], state[3]}, {which}) ||
      !apart({state[0], state[1], state[2]}, {other}))
    return DCP_EINVAL;
  const size_t smem = pages_smem(N, A.hash);
  if (!allow_smem<pages_kernel<kFork>>()) return DCP_ECUDA;
  const unsigned ctas = A.alone ? kPgCluster : (unsigned)(tables * kPgCluster);
  cudaError_t e = launch_chained(pages_kernel<kFork>, ctas, kPgThreads, smem, s, A);
  if (e != cudaSuccess) return launch_status_report(e);
  if (A.alone) return launch_status();
  const unsigned grid = (unsigned)((N + 255) / 256 < 64 ? (N + 255) / 256 : 64);
  e = launch_chained(pages_lens_kernel, grid, 256, 0, s, A);
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
  if (num > kPgMaxList) return DCP_EUNSUPPORTED;
  *bytes = pages_ws_bytes(num);
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
