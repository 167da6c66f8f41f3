// Shared by the 8-bit cache (dcp_q8_cache.cu) and scored decode attention
// (dcp_scored.cu, dcp_scored_mma.cu): the sharded layout without divisions,
// the tokens that a request sees, how they are cut over the CTAs, and how a
// score is formed.
#pragma once

#include "dcp_common.cuh"
#include "dcp_ptx.cuh"

namespace dcp {

// n / d for 0 <= n < 2^31 by a multiplication (round-up method: with
// l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1 the quotient is
// (hi(n m) + n) >> l; the sum fits, as both terms are below 2^31).
struct FastDiv {
  uint32_t m, d;
  int l;
  FastDiv() = default;
  explicit FastDiv(uint32_t div) : d(div) {
    l = 0;
    while (l < 31 && (1u << l) < div) ++l;
    m = (uint32_t)(((uint64_t(1) << 32) * ((uint64_t(1) << l) - div)) / div + 1);
  }
  __device__ __forceinline__ int div(int n) const {
    return (int)((__umulhi((uint32_t)n, m) + (uint32_t)n) >> l);
  }
};

// The interleaved layout: page of `bs` tokens per rank in each virtual block
// of bs * dcp tokens, runs of I tokens going round the ranks.
struct Shards {
  int dcp, bs, I, vbs, turn;
  FastDiv by_vbs, by_turn, by_I, by_bs;
  Shards() = default;
  explicit Shards(const dcp_layout_t& L)
      : dcp(L.dcp_size), bs(L.block_size), I(L.interleave), vbs(L.block_size * L.dcp_size),
        turn(L.interleave * L.dcp_size), by_vbs(vbs), by_turn(turn), by_I(I), by_bs(bs) {}

  __device__ __forceinline__ void place(int x, int& rank, int& vb, int& loc) const {
    vb = by_vbs.div(x);
    const int off = x - vb * vbs, q = by_turn.div(off), in = off - q * turn;
    rank = by_I.div(in);
    loc = q * I + in - rank * I;
  }
  // Position of place `loc` of rank's page of virtual block vb.
  __device__ __forceinline__ int position(int vb, int rank, int loc) const {
    const int q = by_I.div(loc);
    return vb * vbs + q * turn + rank * I + loc - q * I;
  }
};

// Tokens of [0, x) on each rank: what is the same for all ranks is worked out once.
struct Below {
  int base = 0, in = 0;   // whole runs, and what is left of the last turn
  Below() = default;
  __device__ __forceinline__ Below(const Shards& S, int x) {
    const int full = S.by_vbs.div(x), rem = x - full * S.vbs, q = S.by_turn.div(rem);
    base = full * S.bs + q * S.I;
    in = rem - q * S.turn;
  }
  __device__ __forceinline__ int on(const Shards& S, int r) const {
    return base + min(max(in - r * S.I, 0), S.I);
  }
};

inline bool shards_ok(const dcp_layout_t& L) {
  return layout_ok(L) && (int64_t)L.block_size * L.dcp_size < (int64_t(1) << 30);
}

// ---------------------------------------------------------------------------
// scored decode attention
// ---------------------------------------------------------------------------

constexpr int kRows = 16;          // tokens of a tile: places [16 t, 16 t + 16) of a rank's tokens
constexpr int kScoredWarps = 4;    // of a CTA

struct ScoredArgs {
  Shards S;
  int B, Hq, Hkv, G, d;
  int apart;                 // per-rank outputs: an entry is a rank of a request
  const void* q;             // [B][Hq][d]
  float scale, cap, inv_cap;
  int window, prefix;
  const float* slopes;       // [Hq] or NULL
  const int32_t* first;      // [B] or NULL
  const int32_t* lens;       // [B]
  const float* sink;         // [Hq] or NULL
  const int32_t* bt;
  int max_vb;
  int64_t bt_stride, nb;
  dcp_rank_ptrs_t k, v, sc;
  void* out;                 // [entries][Hq][d]
  int out_dtype;
  float* out_lse;            // [entries][Hq] or NULL
  int32_t* err;
  // workspace
  int32_t* before;           // [entries + 1] tiles of a head in front of an entry, then a chunk's
  float* part_lse;           // [chunks + units][G]
  float* part_o;             // [chunks + units][G][d]
  int ctas, least;           // chunks at most (the grid), and the fewest tiles of one
  int unit_ctas;             // CTAs of a unit (a cluster) where units are not cut elsewhere, or 0
  __device__ __forceinline__ int entries() const { return apart ? B * S.dcp : B; }
};

// What a request sees of a rank, as two runs of the rank's tokens (the first,
// kept tokens of the document, and the window), and their tiles.
struct RankTokens {
  int a0, a1, b0, b1;
  __device__ __forceinline__ int a_tiles() const { return a1 > a0 ? (a1 + 15) / 16 - a0 / 16 : 0; }
  __device__ __forceinline__ int b_tiles() const { return b1 > b0 ? (b1 + 15) / 16 - b0 / 16 : 0; }
};

struct Seen {
  Below lo, p, w, n;
  bool kept;   // there is a run of kept tokens apart from the window
  __device__ __forceinline__ Seen(const ScoredArgs& A, int lo_, int p_, int w_, int n_)
      : n(A.S, n_), kept(p_ > lo_) {
    if (w_ > 0) w = Below(A.S, w_);
    if (kept) {
      lo = Below(A.S, lo_);
      p = Below(A.S, p_);
    }
  }
  __device__ __forceinline__ RankTokens on(const Shards& S, int r) const {
    RankTokens t;
    t.b0 = w.on(S, r);
    t.b1 = n.on(S, r);
    t.a0 = t.a1 = 0;
    if (kept) {
      t.a0 = lo.on(S, r);
      t.a1 = p.on(S, r);
    }
    return t;
  }
  __device__ __forceinline__ int tiles(const Shards& S, int r) const {
    const RankTokens t = on(S, r);
    return t.a_tiles() + t.b_tiles();
  }
};

// Length n of the request, and with lo the document's start: tokens x of
// [lo, n) with x >= w = max(lo, n - window) or x < p = lo + prefix.  Tokens
// beyond the block table are not there.  Negative lengths count as 0.
__device__ __forceinline__ Seen seen_of(const ScoredArgs& A, int b, bool count) {
  const int len = __ldg(A.lens + b), lo0 = A.first ? __ldg(A.first + b) : 0;
  const int64_t room = (int64_t)A.max_vb * A.S.vbs;
  if (count && (len < 0 || len > room)) count_error(A.err);
  const int there = (int)min((int64_t)max(len, 0), room);
  const int lo = min(max(lo0, 0), there);
  int w = A.window > 0 ? max(lo, len - A.window) : lo;   // len >= 0 or there = 0
  w = min(w, there);
  const int p = (int)min((int64_t)lo + A.prefix, (int64_t)w);
  // kept tokens that reach the window are one run with it
  if (p >= w) return Seen(A, 0, 0, lo, there);
  return Seen(A, lo, p, w, there);
}

// Entry e is request e % B, on rank e / B where ranks are apart.
__device__ __forceinline__ int entry_tiles(const ScoredArgs& A, int e, bool count) {
  const int b = A.apart ? e % A.B : e;
  const Seen s = seen_of(A, b, count && e < A.B);
  if (A.apart) return s.tiles(A.S, e / A.B);
  int n = 0;
  for (int r = 0; r < A.S.dcp; ++r) n += s.tiles(A.S, r);
  return n;
}

// The same by a warp, a rank in each lane.
__device__ __forceinline__ int entry_tiles_by_warp(const ScoredArgs& A, int e, bool count) {
  const int lane = threadIdx.x & 31, R = A.apart ? 1 : A.S.dcp;
  const Seen s = seen_of(A, A.apart ? e % A.B : e, count && lane == 0 && e < A.B);
  const int r = (A.apart ? e / A.B : 0) + min(lane, R - 1);
  return __reduce_add_sync(0xffffffffu, lane < R ? s.tiles(A.S, r) : 0);
}

// A unit is a key/value head of an entry, its tiles those of the ranks in
// order.  All units' tiles, end to end (entry by entry, head by head), are a line
// that is cut into chunks of `each` tiles.  The piece of unit u in chunk i has its
// partial result at i + u: along the line either the unit or the chunk goes up by
// one from piece to piece, or both, so no two pieces share one.  The host sees
// to it that the line has fewer than 2^30 tiles.
struct Line {
  int all, each;   // tiles, and those of a chunk
  int per;         // entries that a thread has counted
};

// Every thread of the CTA calls it; all get the same, and s_before[i] is what
// lies in front of thread i's entries, in tiles of a head.  The lengths are read
// by every CTA: a plan of one CTA in front would cost a launch, of the 12 to 16
// us that the shortest calls take that are cut by the line.
template <int kThreads>
__device__ __forceinline__ Line plan_line(const ScoredArgs& A, int chunk, int* s_before) {
  __shared__ int s_sum[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int E = A.entries();
  Line line;
  line.per = (E + kThreads - 1) / kThreads;
  const int e0 = min(tid * line.per, E), e1 = min(e0 + line.per, E);
  int sum = 0;
  for (int e = e0; e < e1; ++e) sum += entry_tiles(A, e, chunk == 0);   // counts bad lengths
  int upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) s_sum[warp] = upto;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) upto += s_sum[w];
    total += s_sum[w];
  }
  s_before[tid] = upto - sum;
  line.all = total * A.Hkv;
  line.each = max(A.least, (line.all + A.ctas - 1) / A.ctas);
  __syncthreads();
  return line;
}

// For the merge (the CTA of chunk 0 calls it): what lies in front of each entry,
// and the chunks' size.
template <int kThreads>
__device__ __forceinline__ void keep_line(const ScoredArgs& A, const Line& line,
                                          const int* s_before) {
  const int E = A.entries(), tid = threadIdx.x;
  const int e0 = min(tid * line.per, E), e1 = min(e0 + line.per, E);
  int before = s_before[tid];
  for (int e = e0; e < e1; ++e) {
    A.before[e] = before;
    if (e + 1 < e1) before += entry_tiles(A, e, false);
  }
  if (tid == 0) {
    A.before[E] = line.all / A.Hkv;
    A.before[E + 1] = line.each;
  }
}

// The entries in front of which tile t of the line does not lie: the first of
// those that one thread has counted.  The whole warp asks for one t.
template <int kThreads>
__device__ __forceinline__ void seek_entry(const ScoredArgs& A, const Line& line,
                                           const int* s_before, int t, int& e, int& start) {
  const int lane = threadIdx.x & 31;
  int n = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i)
    n += __popc(__ballot_sync(0xffffffffu, s_before[i * 32 + lane] * A.Hkv <= t));
  e = min((n - 1) * line.per, A.entries() - 1);
  start = s_before[n - 1] * A.Hkv;
}

// A chunk's part of a unit: tiles [k0, k1) of the n of head g of entry e.
struct Piece {
  int e, g, k0, k1, n;
  int start, t;   // first tile of the entry, and the line's tile behind the piece
};

// The piece that begins with tile t, in a chunk that ends with t1, of entry e
// with n tiles a head.
__device__ __forceinline__ Piece piece_of(const ScoredArgs& A, int t, int t1, int e, int start,
                                          int n) {
  Piece p;
  p.e = e, p.n = n, p.start = start;
  p.g = (int)((uint32_t)(t - start) / (uint32_t)max(n, 1));
  p.k0 = t - start - p.g * n;
  p.k1 = min(n, p.k0 + (t1 - t));
  p.t = t + (p.k1 - p.k0);
  return p;
}

// The same with an entry at or in front of it.
__device__ __forceinline__ Piece piece_at(const ScoredArgs& A, int t, int t1, int e, int start) {
  int n = entry_tiles(A, e, false);
  while (t - start >= n * A.Hkv && e + 1 < A.entries()) {
    start += n * A.Hkv;
    n = entry_tiles(A, ++e, false);
  }
  return piece_of(A, t, t1, e, start, n);
}

// A score is compared with its head's reference only to see whether it passes it
// by more than 2^4; while none of a warp's does (one vote), nothing is rescaled.
constexpr float kSlack = 4.f;
constexpr float kNone = -3e38f;  // a reference before there is a score

// tanh as one quotient, off by 2^-21 of it at most.  Below 7/8 it is the continued fraction
// y / (1 + z / (3 + z / (5 + z / (7 + z / 9)))), z = y^2, off by 2^-25.7 there; above,
// (1 - e) / (1 + e) with e = e^-2|y|, whose error of 2^-22 counts less than half.  What is left
// are the rounding of its parts and the reciprocal's 2^-23.
__device__ __forceinline__ float tanh_of(float y) {
  const float e = ex2_ftz(fabsf(y) * (-2.f * kLog2e)), z = y * y;
  const bool near = fabsf(y) < 0.875f;
  const float num = near ? y * fmaf(z, z + 105.f, 945.f) : copysignf(1.f - e, y);
  const float den = near ? fmaf(z, fmaf(z, 15.f, 420.f), 945.f) : 1.f + e;
  float inv;   // den is at least 1, and below 1279
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(den));
  return num * inv;
}

// A scaled score in base 2: capped, and less the distance's share.
__device__ __forceinline__ float formed(const ScoredArgs& A, float t, float slope, float far) {
  if (A.cap > 0.f) t = A.cap * tanh_of(t * A.inv_cap);
  if (A.slopes) t -= slope * far;
  return t * kLog2e;
}

// Result of head `hh` of unit (e, g): the output itself if the piece is the
// whole unit (with the sink), else the partial result in `slot`.
struct PieceOut {
  bool whole;
  int64_t slot, row;   // row: e * Hq + g * G
};

// Four values from column 4 i on, counted over the unit's heads.
__device__ __forceinline__ void put_four(const ScoredArgs& A, const PieceOut& P, int i, float4 y) {
  if (!P.whole)
    reinterpret_cast<float4*>(A.part_o + P.slot * A.G * A.d)[i] = y;
  else if (A.out_dtype == DCP_F32)
    reinterpret_cast<float4*>((float*)A.out + P.row * A.d)[i] = y;
  else
    reinterpret_cast<uint2*>((__nv_bfloat16*)A.out + P.row * A.d)[i] =
        make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
}

// Natural LSE with the sink's, and the weight that the values keep beside it.
__device__ __forceinline__ float with_sink(const float* sink, int h, float lse, float& weight) {
  weight = 1.f;
  if (!sink) return lse;
  const float s = __ldg(sink + h), m = fmaxf(s, lse);
  if (m == -INFINITY) return lse;
  const float all = m + logf(expf(s - m) + expf(lse - m));
  weight = lse == -INFINITY ? 0.f : expf(lse - all);
  return all;
}

__device__ __forceinline__ void put_lse(const ScoredArgs& A, const PieceOut& P, int hh, float lse) {
  if (!P.whole)
    A.part_lse[P.slot * A.G + hh] = lse;
  else if (A.out_lse)
    A.out_lse[P.row + hh] = lse;
}

__device__ __forceinline__ float remote_f32(uint32_t cluster_addr) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(cluster_addr) : "memory");
  return x;
}
__device__ __forceinline__ float4 remote_f32x4(uint32_t cluster_addr) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "r"(cluster_addr)
               : "memory");
  return x;
}

// A unit that a cluster has whole: each CTA, the lines of CTA `rank` of C, has a part
// of its tiles and in shared memory that part's result for heads [h0, h0 + heads): their
// LSE at lse[h * lse_step] and `quads` times four values at o[h * o_step].  Between two
// cluster barriers the cluster's first kScoredWarps warps call this: as many lanes a
// column as there are CTAs, each with one CTA's part, a CTA every C-th column.
__device__ __forceinline__ void join_cluster(const ScoredArgs& A, int e, int g, int h0, int heads,
                                             int quads, const float* lse, int lse_step,
                                             const float4* o, int o_step) {
  const int C = A.unit_ctas, rank = blockIdx.x % C, columns = heads * quads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane & (C - 1);
  PieceOut P;
  P.whole = true;
  P.slot = 0;
  P.row = (int64_t)e * A.Hq + g * A.G;
  for (int first = warp * 32; first < columns; first += kScoredWarps * 32) {
    const int own = first + (lane & ~(C - 1)) + rank;
    const int i = own < columns ? own : 0, h = i / quads;
    const float l = remote_f32(mapa_shared(smem_u32(lse + h * lse_step), c));
    const float4 y = remote_f32x4(mapa_shared(smem_u32(o + h * o_step + (i - h * quads)), c));
    const bool any = l != -INFINITY;   // else it has seen nothing
    float M = l;
    for (int x = 1; x < C; x *= 2) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
    float sum = any ? expf(l - M) : 0.f;
    for (int x = 1; x < C; x *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    float weight, mine = sum == 0.f ? -INFINITY : M + logf(sum);
    const float all = with_sink(A.sink, g * A.G + h0 + h, mine, weight);
    const float w = any ? expf(l - mine) * weight : 0.f;
    float4 z = any ? make_float4(w * y.x, w * y.y, w * y.z, w * y.w)
                   : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x = 1; x < C; x *= 2) {
      z.x += __shfl_xor_sync(0xffffffffu, z.x, x);
      z.y += __shfl_xor_sync(0xffffffffu, z.y, x);
      z.z += __shfl_xor_sync(0xffffffffu, z.z, x);
      z.w += __shfl_xor_sync(0xffffffffu, z.w, x);
    }
    if (own >= columns || c != 0) continue;
    put_four(A, P, h0 * quads + i, z);
    if (i % quads == 0) put_lse(A, P, h0 + h, all);
  }
}

constexpr int kUnitCtas = 16;   // of a unit's cluster at most

// Clusters beyond the eight CTAs that every device has: allowed once per device.
template <auto kKernel>
inline cudaError_t allow_clusters(int ctas) {
  if (ctas <= 8) return cudaSuccess;
  static bool allowed[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool kept = dev >= 0 && dev < 64;
  if (kept && allowed[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && kept) allowed[dev] = true;
  return e;
}

inline cudaLaunchAttribute cluster_of(int ctas) {
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = (unsigned)ctas;
  a.val.clusterDim.y = a.val.clusterDim.z = 1;
  return a;
}

// Clusters of 1, 2, 4, 8 or 16 CTAs of a kernel that run at once on the current device (the
// larger ones leave gaps, how many depends on the kernel's registers and shared memory), and 0
// if that cannot be told.  Asked once for each size and number of heads, on which `smem` depends.
template <auto kKernel>
inline int clusters_at_once(int ctas, int heads, unsigned block, size_t smem) {
  static int known[64][kUnitCtas + 1][17] = {};   // and 1
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const bool kept = dev >= 0 && dev < 64;
  if (kept && known[dev][ctas][heads]) return known[dev][ctas][heads] - 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr = cluster_of(ctas);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (allow_clusters<kKernel>(ctas) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kKernel, &cfg) != cudaSuccess) {
    cudaGetLastError();   // left for no other call to read
    n = 0;
  }
  if (kept) known[dev][ctas][heads] = n + 1;
  return n;
}

// As launch_chained, the grid in clusters of a unit's CTAs.
template <auto kKernel, class... Args>
inline cudaError_t launch_scored(const ScoredArgs& A, unsigned block, size_t smem, cudaStream_t s,
                                 const Args&... args) {
  const cudaError_t e = allow_clusters<kKernel>(A.unit_ctas);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)A.ctas);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1] = cluster_of(A.unit_ctas);
  cfg.attrs = attr;
  cfg.numAttrs = A.unit_ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kKernel, args...);
}

// Which kernel a cache takes: the tensor-core kernel (dcp_scored_mma.cu) or
// the one for any type and shape (dcp_scored.cu).
enum CacheKind { kCacheF32, kCacheBf16, kCacheE4m3 };
bool scored_mma_ok(const ScoredArgs& A, CacheKind kind, bool q_bf16);
int scored_mma_wave(int d, int G, CacheKind kind);   // CTAs that run at once
int scored_mma_clusters(const ScoredArgs& A, CacheKind kind, int ctas);   // that run at once
int launch_scored_mma(const ScoredArgs& A, CacheKind kind, cudaStream_t s);

}  // namespace dcp
