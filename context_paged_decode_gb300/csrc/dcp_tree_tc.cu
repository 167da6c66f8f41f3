// tcgen05 kernel of the drafted-tree attention: bf16, head_dim 64 or 128.
//
// The query heads of a group and the drafted nodes share each key/value row,
// so a unit's scores S = Q K^T (rows = node * G + head) and O = P V are dense
// products over its tokens with up to 256 rows; the masks touch only the few
// tiles that hold drafted nodes.  Bytes bound it up to about 128 rows: a
// 128-token tile of keys and values (64 KB at head_dim 128) takes an SM 1.5 us
// of its share of the measured bandwidth, its two products 0.5 us for 128
// rows, its softmax 0.5 us of the exponential unit.  Measured (GPU time of the
// whole call): 32 requests x 16 nodes, 32 query over 8 key heads of 128, 8
// ranks, up to 65536 tokens (3.05 GB): 452-466 us, 6.5-6.7 TB/s, 0.97-0.99 of
// the copy bandwidth.  8 requests x 64 nodes (256 rows) over up to 65536 tokens
// (655 MB, 149 GFLOP): 152-160 us, 4.2 TB/s and 0.95 PFLOP/s; there a tile's chain
// of scores, softmax and products is what the two streams cannot fill (copies of
// the kernel without the products, or without the exponentials, took 0.93 and
// 0.97 of its time), and short contexts are bound by what a unit costs beside
// its tiles, some 8 to 10 of them.
//
// One CTA per SM works through its run of tiles (see dcp_tree.cuh).  Two
// softmax warpgroups, a tensor-memory score buffer and an output accumulator
// each:
//  * up to 128 rows (kTwo false) they take the tiles in turn, with the same
//    queries, and join their sums at the end of a unit: one computes its
//    softmax while the tensor core works for the other;
//  * up to 256 rows (kTwo true) each has half of the rows and both go through
//    every tile, which is read once.
// Warps: 0 and 2 load keys and values by TMA (chunks of 16 rows, a page or part
// of one, a lane each), into a ring of their own; 3 loads the queries,
// whose rows (node, head of the group) are one box of the query tensor, and
// goes over the values; 1 issues the products; 4-7 and 8-11 are the softmax, one row per thread, its
// 128 scores in registers (which the other warps give up for it).  P goes back
// to tensor memory over the scores it came from (bf16, half the columns) and
// is the A operand of P V.  The score product of a stream's next tile is issued
// after P V of its last, so a score barrier also says that the accumulator is
// at rest, and the rare rescale (only when the maximum grows by more than 2^8)
// needs no wait of its own.
//
// Masked tokens have P = 0, but 0 * x is not 0 for infinities and NaN.  Rows of
// V past the end or of unusable pages are zeroed in shared memory, and so are
// non-finite values of drafted nodes; the rows that do see such a node get its
// values added afterwards, one by one (tree_fix).  A warp of its own does that
// as the values arrive: by the softmax warps, on the way from the scores to P,
// 8 x 64 nodes over up to 65536 tokens took 165 us (153 now), over up to 5000
// tokens 53 (47).
//
// Roundings: P is rounded to bf16 for the product (2^-8 of each weight, whose
// errors average out; the sums of P are taken before it, in 32 bits), and the
// output once when it is stored.  Scores, maxima, sums and partials have 32 bits.
//
// Every wait is bounded; a timed-out role stops waiting and working but keeps
// step at the named barriers, so the kernel always ends.
#include <mutex>
#include <string.h>

#include "dcp_ptx.cuh"
#include "dcp_tree.cuh"

namespace dcp {

struct TreeTcArgs {
  CUtensorMap kmap[DCP_MAX_RANKS];   // [num_blocks * Hkv * bs rows][d], box 64 x 16
  CUtensorMap vmap[DCP_MAX_RANKS];
  CUtensorMap qmap;                  // [N][Hq][d], box 64 x G x `nodes`
  TreeArgs t;
  int nodes;                         // of a query tile: 128 / G
};

constexpr int kTtTile = 128;
constexpr int kTtChunk = 16;                 // tokens of one box: a page or part of one
constexpr int kTtChunks = kTtTile / kTtChunk;
constexpr int kTtThreads = 384;
constexpr int kHalfBytes = kTtTile * 128;    // 64 columns of a tile or of a query block
constexpr float kTtGrow = 8.f;               // log2 units
constexpr int kTtStuck = 1 << 20;
// Places of the flag that says that a unit's values were cleaned, one unit after
// another.  The value warp comes to unit i + 2 when the scores of unit i + 1 are
// done, which the row writes of unit i may not be (with a tile or two a unit no
// wait for them lies between), so two places are too few.  It comes to unit
// i + 3 after the scores of i + 2, which are issued behind the wait for unit i.
constexpr int kTtFlags = 3;

template <int D, bool kTwo>
struct TreeTc {
  static constexpr int kSlot = kTtTile * D * 2;
  static constexpr int kQ = (kTwo ? 2 : 1) * kSlot;
  // 224 KB of tiles; 3 KB stay for the rest
  static constexpr int kKSlots = (224 * 1024 - kQ) / kSlot / 2;
  static constexpr int kVSlots = (224 * 1024 - kQ) / kSlot - kKSlots;
  static constexpr int kVOff = kKSlots * kSlot;
  static constexpr int kQOff = kVOff + kVSlots * kSlot;
  static constexpr int kMlOff = kQOff + kQ;                 // float2 [2 stream][128]
  static constexpr int kFlagOff = kMlOff + 2 * 128 * 8;     // int [kTtFlags], joins
  static constexpr int kPlanOff = kFlagOff + 4 * (kTtFlags + 1);   // TreeSelf
  static constexpr int kBarOff = kPlanOff + (int)sizeof(TreeSelf);
  static constexpr int kBars = 2 * kKSlots + 3 * kVSlots + 8;
  static constexpr int kSmem = kBarOff + 8 * kBars + 8;
  static_assert(kSmem <= 227 * 1024 && kBarOff % 8 == 0 && kPlanOff % alignof(TreeSelf) == 0,
                "shared memory");
  static constexpr uint32_t kColS = 0, kColO = 256;         // two of each, 128 and D apart
};

// A lane's chunk of a tile (lanes 0 .. 7 have one), tile after tile.  Chunks of
// several ranks share a tile: with a tile per rank's end, short contexts over
// many ranks spent most of their tiles on a few tokens each.
struct ChunkIt {
  TreeLen len, old;       // with and without the nodes
  int r, x;               // rank, chunk on it
  int n, c, lc;           // the rank's tokens, chunks and context tokens
  __device__ __forceinline__ void at(const TreeArgs& A, int rank) {
    r = rank;
    n = len.on(r, A.L);
    c = (n + kTtChunk - 1) / kTtChunk;
    lc = old.on(r, A.L);
  }
  __device__ __forceinline__ ChunkIt(const TreeArgs& A, const TreePiece& p, int tile, int lane)
      : len(p.ctx + p.T, A.L), old(p.ctx, A.L) {
    at(A, p.r0);
    x = (p.t0 + tile) * kTtChunks + lane;
    settle(A, p);
  }
  __device__ __forceinline__ void settle(const TreeArgs& A, const TreePiece& p) {
    while (x >= c && r + 1 < p.r1) {
      x -= c;
      at(A, r + 1);
    }
  }
  __device__ __forceinline__ void step(const TreeArgs& A, const TreePiece& p, int tiles) {
    x += tiles * kTtChunks;
    settle(A, p);
  }
  __device__ __forceinline__ bool has(int lane) const { return lane < kTtChunks && x < c; }
};

// The chunks of a tile as bits of tokens: the low half those that all rows see,
// the high half those that are there.  The table entry is loaded a tile ahead.
struct ChunkBits {
  ChunkIt it;
  int raw;
  __device__ __forceinline__ ChunkBits(const TreeArgs& A, const TreePiece& p, int tile, int lane)
      : it(A, p, tile, lane) {
    fetch(A, p, lane);
  }
  __device__ __forceinline__ void fetch(const TreeArgs& A, const TreePiece& p, int lane) {
    raw = -1;
    const int j = it.x * kTtChunk / A.L.bs;
    if (it.has(lane) && j < A.max_vb)
      raw = __ldcg(A.bt + it.r * A.stride + (int64_t)p.b * A.max_vb + j);
  }
  __device__ __forceinline__ void next(const TreeArgs& A, const TreePiece& p, int tiles, int lane) {
    it.step(A, p, tiles);
    fetch(A, p, lane);
  }
  __device__ __forceinline__ uint32_t bits(const TreeArgs& A, int lane) const {
    if (!it.has(lane) || raw < 0 || (int64_t)raw >= A.nb) return 0u;
    const int at = it.x * kTtChunk, there = min(it.n - at, kTtChunk);
    const int old = min(max(it.lc - at, 0), there);
    return ((1u << old) - 1u) | ((1u << there) - 1u) << 16;
  }
};

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Of each eight lanes, lane i's piece j (four registers) goes to lane j's piece i.
__device__ __forceinline__ void transpose8(uint32_t (&x)[32], int lane) {
#pragma unroll
  for (int b = 1; b < 8; b <<= 1) {
    const bool up = lane & b;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (!(j & b)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t &lo = x[4 * j + i], &hi = x[4 * (j | b) + i];
          const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, b);
          if (up) lo = got; else hi = got;
        }
      }
  }
}

__device__ __forceinline__ bool bf16_odd(uint32_t h) { return (h & 0x7F80u) == 0x7F80u; }

// Adds to output row `row` (columns [c0, c1)) what it sees of non-finite values
// of drafted nodes, which the product took as zero.  Rare and slow.
template <int D>
__device__ __noinline__ void tree_fix(const TreeArgs& A, const TreePiece& p, int row, int c0,
                                      int c1, float M, float f, void* dst, bool f32) {
  const int T = p.T;
  const int64_t ctx = p.ctx, tok = p.q0 + row / A.G;
  const uint64_t mask = __ldcg((const unsigned long long*)A.mask + tok);
  const __nv_bfloat16* q =
      (const __nv_bfloat16*)A.q + (tok * A.Hq + p.g * A.G + row % A.G) * (int64_t)D;
  for (int j = 0; j < T; ++j) {
    if (!((mask >> j) & 1)) continue;
    int r, loc;
    int64_t vb;
    place_token(ctx + j, A.L, r, vb, loc);
    if (r < p.r0 || r >= p.r1) continue;
    int x = (int)((vb * A.L.bs + loc) / kTtChunk);       // chunk of the unit
    const TreeLen len(p.ctx + T, A.L);
    for (int y = p.r0; y < r; ++y) x += (len.on(y, A.L) + kTtChunk - 1) / kTtChunk;
    if (x / kTtChunks < p.t0 || x / kTtChunks >= p.t0 + p.n) continue;
    const int64_t phys =
        vb < A.max_vb ? (int64_t)__ldcg(A.bt + r * A.stride + (int64_t)p.b * A.max_vb + vb) : -1;
    if (phys < 0 || phys >= A.nb) continue;
    const int64_t kv = ((phys * A.Hkv + p.g) * A.L.bs + loc) * D;
    const __nv_bfloat16* k = (const __nv_bfloat16*)A.k.ptr[r] + kv;
    const __nv_bfloat16* v = (const __nv_bfloat16*)A.v.ptr[r] + kv;
    float w = -1.f;
    for (int c = c0; c < c1; ++c) {
      const float x = __bfloat162float(__ldcg(v + c));
      if (isfinite(x)) continue;
      if (w < 0.f) {
        float s = 0.f;
        for (int i = 0; i < D; ++i)
          s = fmaf(__bfloat162float(__ldcg(q + i)), __bfloat162float(__ldcg(k + i)), s);
        w = exp2f(s * A.sl2 - M) * f;
      }
      if (f32)
        ((float*)dst)[c] += w * x;
      else
        ((__nv_bfloat16*)dst)[c] =
            __float2bfloat16_rn(__bfloat162float(((__nv_bfloat16*)dst)[c]) + w * x);
    }
  }
}

// Joins the partials of a unit that was cut (runs k0 .. k1), in the order of the
// runs, whoever does it: a warp takes four rows at a time, a lane a part's LSE
// of each and D / 32 columns, four parts' values in flight.
template <int D>
__device__ __forceinline__ void tree_join(const TreeArgs& A, const TreePiece& p, int k0, int k1,
                                          bool late, int nrows, int warp) {
  constexpr int kV = D / 32, kR = 4, kP = 4;
  const int lane = threadIdx.x & 31;
  auto slot = [&](int k) { return (int64_t)(2 * k + (k == k0 && late)) * A.rows; };
  const bool sunk = A.sink != nullptr;
#pragma unroll 1
  for (int r0 = warp * kR; r0 < nrows; r0 += 8 * kR) {
    float v[kR][kP][kV];
    auto fetch = [&](int k) {
#pragma unroll
      for (int x = 0; x < kR; ++x)
#pragma unroll
        for (int y = 0; y < kP; ++y)
#pragma unroll
          for (int z = 0; z < kV; ++z) v[x][y][z] = 0.f;
#pragma unroll
      for (int x = 0; x < kR; ++x)
#pragma unroll
        for (int y = 0; y < kP; ++y)
          if (r0 + x < nrows && k + y <= k1) {
            const float* src = A.part_o + (slot(k + y) + r0 + x) * D + lane * kV;
            if (kV == 4) {
              const float4 q = __ldcg((const float4*)src);
              v[x][y][0] = q.x;
              v[x][y][1] = q.y;
              v[x][y][2 % kV] = q.z;
              v[x][y][3 % kV] = q.w;
            } else {
              const float2 q = __ldcg((const float2*)src);
              v[x][y][0] = q.x;
              v[x][y][1] = q.y;
            }
          }
    };
    fetch(k0);
    float M[kR], L[kR], s2[kR], acc[kR][kV];
#pragma unroll
    for (int x = 0; x < kR; ++x) {
      const int h = p.g * A.G + (p.rb * A.rows + r0 + x) % A.G;
      M[x] = s2[x] = sunk ? __ldcg(A.sink + h) * kLog2e : -INFINITY;
#pragma unroll
      for (int z = 0; z < kV; ++z) acc[x][z] = 0.f;
    }
#pragma unroll 1
    for (int k = k0; k <= k1; k += 32)
#pragma unroll
      for (int x = 0; x < kR; ++x)
        M[x] = fmaxf(M[x], warp_max(r0 + x < nrows && k + lane <= k1
                                        ? __ldcg(A.part_lse + slot(k + lane) + r0 + x)
                                        : -INFINITY));
#pragma unroll
    for (int x = 0; x < kR; ++x) {
      if (M[x] == -INFINITY) M[x] = 0.f;
      L[x] = sunk ? exp2f(s2[x] - M[x]) : 0.f;
    }
#pragma unroll 1
    for (int k = k0; k <= k1; k += 32) {
      float part[kR];
#pragma unroll
      for (int x = 0; x < kR; ++x) {
        const float lse = r0 + x < nrows && k + lane <= k1
                              ? __ldcg(A.part_lse + slot(k + lane) + r0 + x)
                              : -INFINITY;
        // a part that saw nothing does not count, whatever its values are
        part[x] = lse == -INFINITY ? 0.f : exp2f(lse - M[x]);
        L[x] += warp_sum(part[x]);
      }
#pragma unroll 1
      for (int y0 = 0; y0 < 32 && k + y0 <= k1; y0 += kP) {
        if (k + y0 > k0) fetch(k + y0);
#pragma unroll
        for (int x = 0; x < kR; ++x)
#pragma unroll
          for (int y = 0; y < kP; ++y) {
            const float w = __shfl_sync(0xffffffffu, part[x], (y0 + y) & 31);
            if (w != 0.f) {
#pragma unroll
              for (int z = 0; z < kV; ++z) acc[x][z] = fmaf(w, v[x][y][z], acc[x][z]);
            }
          }
      }
    }
#pragma unroll
    for (int x = 0; x < kR; ++x) {
      if (r0 + x >= nrows) continue;
      const float inv = L[x] == 0.f ? 0.f : 1.f / L[x];
      const int64_t orow = tree_out_row(A, p, p.rb * A.rows + r0 + x);
      if (A.out_dtype == DCP_F32) {
        float* dst = (float*)A.out + orow * D + lane * kV;
#pragma unroll
        for (int z = 0; z < kV; z += 2)
          *(float2*)(dst + z) = make_float2(acc[x][z] * inv, acc[x][z + 1] * inv);
      } else {
        uint32_t* dst = (uint32_t*)((__nv_bfloat16*)A.out + orow * D + lane * kV);
#pragma unroll
        for (int z = 0; z < kV; z += 2) dst[z / 2] = pack_bf16(acc[x][z] * inv, acc[x][z + 1] * inv);
      }
      if (lane == 0 && A.lse) A.lse[orow] = L[x] == 0.f ? -INFINITY : (M[x] + log2f(L[x])) * kLn2;
    }
  }
}

template <int D, bool kTwo>
__global__ void __launch_bounds__(kTtThreads, 1)
tree_tc_kernel(const __grid_constant__ TreeTcArgs X) {
  using C = TreeTc<D, kTwo>;
  const TreeArgs& A = X.t;
  extern __shared__ __align__(1024) uint8_t smem[];   // no room is left to round up in
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bars = sbase + C::kBarOff;
  const uint32_t b_k = bars, b_kfree = b_k + 8 * C::kKSlots;        // keys: there, read
  const uint32_t b_v = b_kfree + 8 * C::kKSlots, b_vfree = b_v + 8 * C::kVSlots;
  const uint32_t b_vok = b_vfree + 8 * C::kVSlots;   // values may be read by the product
  const uint32_t b_s = b_vok + 8 * C::kVSlots;    // +stream: scores are there
  const uint32_t b_p = b_s + 16;                  // +stream: P is there
  const uint32_t b_o = b_p + 16, b_ofree = b_o + 8, b_q = b_o + 16, b_qfree = b_o + 24;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kBarOff + 8 * C::kBars);
  volatile int* flag = reinterpret_cast<int*>(smem + C::kFlagOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  griddep_launch_dependents();
  if (sbase & 1023) {   // the swizzle's atoms need it
    if (threadIdx.x == 0 && A.err) atomicAdd(A.err, kTtStuck);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kKSlots; ++i) {
      mbar_init(b_k + 8 * i, 1);
      mbar_init(b_kfree + 8 * i, 1);
    }
    for (int i = 0; i < C::kVSlots; ++i) {
      mbar_init(b_v + 8 * i, 1);
      mbar_init(b_vfree + 8 * i, 1);
      mbar_init(b_vok + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_s + 8 * i, 1);
      mbar_init(b_p + 8 * i, 4);
    }
    mbar_init(b_o, 1);
    mbar_init(b_ofree, 8);
    mbar_init(b_q, 1);
    mbar_init(b_qfree, 1);
    fence_mbar_init();
    for (int i = 0; i < kTtFlags; ++i) flag[i] = 0;
    prefetch_tmap(&X.qmap);
    for (int r = 0; r < A.L.dcp; ++r) {
      prefetch_tmap(&X.kmap[r]);
      prefetch_tmap(&X.vmap[r]);
    }
  }
  if (warp == 1) {
    tc_alloc(smem_u32(tmem_slot), 512);
    tc_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();   // the plan, and what the calls before wrote

  TreeSelf* own_plan = reinterpret_cast<TreeSelf*>(smem + C::kPlanOff);
  if (A.self) {
    if (warp == 0) tree_self_plan(A, own_plan);
    __syncthreads();
  }
  int32_t* errp = A.err ? A.err : A.hdr + 1;
  TreeWalk walk = tree_walk(A, blockIdx.x, A.self ? own_plan : nullptr);
  const int srows = X.nodes * A.G;   // rows of a stream's query tile
  auto block_rows = [&](const TreePiece& p) { return min(A.rows, p.T * A.G - p.rb * A.rows); };

  if (warp < 4) {
    // 128 x 88 + 256 x 208 registers are the 384 x 168 of the launch
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0 || warp == 2) {
      // ---------------- keys (0) and values (2) ----------------
      const bool val = warp == 2;
      const uint64_t pol = policy_evict_first();
      const int slots = val ? C::kVSlots : C::kKSlots;
      const uint32_t full = val ? b_v : b_k, free = val ? b_vfree : b_kfree;
      const uint32_t ring = sbase + (val ? C::kVOff : 0) + lane * kTtChunk * 128;
      const CUtensorMap* maps = val ? X.vmap : X.kmap;
      uint32_t slot = 0, par = 1, loaded = 0;
      bool dead = false;
      TreePiece p;
      while (!dead && tree_next(A, walk, p)) {
        const int32_t* bt = A.bt + (int64_t)p.b * A.max_vb;
        // This lane's part of a tile: table entry (-1: beyond the table), its
        // row in the page, and whether it has tokens.  The entry is loaded
        // two tiles ahead and first looked at when its turn comes.
        struct Part {
          int raw, off, r;
          bool has;
        };
        ChunkIt it(A, p, 0, lane);
        int fetched = 0;
        auto fetch = [&]() {
          Part x;
          x.raw = -1;
          x.off = 0;
          x.r = it.r;
          x.has = false;
          if (fetched < p.n) {
            x.has = it.has(lane);
            const int pos = it.x * kTtChunk, j = pos / A.L.bs;
            x.off = pos - j * A.L.bs;
            if (x.has && j < A.max_vb) x.raw = __ldcg(bt + it.r * A.stride + j);
            ++fetched;
            if (fetched < p.n) it.step(A, p, 1);
          }
          return x;
        };
        Part a = fetch(), b = fetch();
        for (int k = 0; k < p.n; ++k) {
          const Part c = a;
          a = b;
          b = fetch();
          const bool ok = c.has && c.raw >= 0 && (int64_t)c.raw < A.nb;
          const uint32_t m = __ballot_sync(0xffffffffu, ok);
          if (c.has && !ok && !val) count_error(A.err);
          if (!__all_sync(0xffffffffu, mbar_wait(free + 8 * slot, par))) {
            dead = true;
            break;
          }
          const uint32_t bar = full + 8 * slot;
          if (lane == 0) {
            if (m)
              mbar_arrive_expect_tx(bar, __popc(m) * kTtChunk * D * 2);
            else
              mbar_arrive(bar);
          }
          __syncwarp();
          if (ok) {
            const int row = (int)(((int64_t)c.raw * A.Hkv + p.g) * A.L.bs + c.off);
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tma_load_2d_hint(ring + slot * C::kSlot + h * kHalfBytes, &maps[c.r], 64 * h, row,
                               bar, pol);
          }
          __syncwarp();
          if (++slot == (uint32_t)slots) {
            slot = 0;
            par ^= 1;
          }
          ++loaded;
        }
      }
      // nothing may still be on its way when the CTA ends, whoever gave up
      for (uint32_t t = loaded < (uint32_t)slots ? 0 : loaded - slots; t < loaded; ++t)
        mbar_wait(full + 8 * (t % slots), (t / slots) & 1);
      if (dead && lane == 0) atomicAdd(errp, kTtStuck);
    } else if (warp == 3) {
      // ---------------- queries, and values that must not count ----------------
      uint32_t item = 0, vs = 0, vp = 0;
      bool dead = false;
      auto wait = [&](uint32_t bar, uint32_t par) {
        if (!dead && !__all_sync(0xffffffffu, mbar_wait(bar, par))) dead = true;
      };
      TreePiece p;
      while (!dead && tree_next(A, walk, p)) {
        if (item > 0) wait(b_qfree, (item - 1) & 1);
        if (dead) break;
        if (lane == 0) {
          const bool two = kTwo && block_rows(p) > srows;
          mbar_arrive_expect_tx(b_q, (two ? 2 : 1) * srows * D * 2);
          const int node = p.q0 + p.rb * (A.rows / A.G);
          for (int s = 0; s < (two ? 2 : 1); ++s)
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tma_load_3d(sbase + C::kQOff + s * C::kSlot + h * kHalfBytes, &X.qmap, 64 * h,
                          p.g * A.G, node + s * X.nodes, b_q);
        }
        __syncwarp();
        ChunkBits it(A, p, 0, lane);
        for (int k = 0; k < p.n && !dead; ++k) {
          const uint32_t bits = it.bits(A, lane);
          if (k + 1 < p.n) it.next(A, p, 1, lane);
          wait(b_v + 8 * vs, vp);
          if (dead) break;
          uint32_t odd_chunks = __ballot_sync(0xffffffffu, bits != ~0u) & 0xFFu;
          if (odd_chunks) {
            // rows of V that nobody sees become zero, and so do odd values of
            // nodes; a row is kRow lanes of 16 bytes
            const uint32_t v = sbase + C::kVOff + vs * C::kSlot;
            constexpr int kRow = D / 8, kAtOnce = 32 / kRow;
            const int ch = lane % kRow;
            do {
              const int c = __ffs(odd_chunks) - 1;
              odd_chunks &= odd_chunks - 1;
              const uint32_t mine = __shfl_sync(0xffffffffu, bits, c);
              uint32_t rows = ~mine & 0xFFFFu;            // not seen by all
              for (; rows; rows &= rows - 1) {
                // the next kAtOnce such rows, one for each kRow lanes
                uint32_t rest = rows;
#pragma unroll
                for (int i = 1; i < kAtOnce; ++i)
                  if (lane / kRow >= i) rest &= rest - 1;
                if (rest) {
                  const int o = __ffs(rest) - 1, tok = c * kTtChunk + o;
                  const uint32_t at =
                      v + (ch >> 3) * kHalfBytes + tok * 128 + (((ch & 7) ^ (tok & 7)) << 4);
                  uint32_t w[4] = {0u, 0u, 0u, 0u};
                  bool odd = !((mine >> (16 + o)) & 1);
                  if (!odd) {
                    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                 : "r"(at));
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                      if (bf16_odd(w[x])) {
                        w[x] &= 0xFFFF0000u;
                        odd = true;
                      }
                      if (bf16_odd(w[x] >> 16)) {
                        w[x] &= 0xFFFFu;
                        odd = true;
                      }
                    }
                    if (odd) flag[item % kTtFlags] = (int)item + 1;
                  }
                  if (odd)
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(w[0]),
                                 "r"(w[1]), "r"(w[2]), "r"(w[3])
                                 : "memory");
                }
#pragma unroll
                for (int i = 1; i < kAtOnce; ++i) rows &= rows - 1;
              }
            } while (odd_chunks);
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(b_vok + 8 * vs);
          if (++vs == C::kVSlots) {
            vs = 0;
            vp ^= 1;
          }
        }
        ++item;
      }
      if (item > 0) mbar_wait(b_q, (item - 1) & 1);
      if (dead && lane == 0) atomicAdd(errp, kTtStuck);
    } else {
      // ---------------- products ----------------
      // The whole warp runs this, with values that all lanes share (what is
      // read from memory is broadcast so that the compiler knows it), and one
      // lane is elected per instruction.  From a single-lane branch, beside
      // two softmax warps, a product took twice its 64 cycles to issue.
      constexpr uint32_t kIdQK = idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t kIdPV = idesc_bf16_f32(128, D, false, true);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      uint32_t ks = 0, kp = 0, vs = 0, vp = 0;   // ring places and parities
      uint32_t item = 0, np0 = 0, np1 = 0;
      bool dead = false;
      auto wait = [&](uint32_t bar, uint32_t par) {
        if (dead) return false;
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, par))) return true;
        if (!__all_sync(0xffffffffu, mbar_wait(bar, par))) dead = true;
        return !dead;
      };
      // A wait for what is there already still takes this warp 150 to 250
      // cycles beside the softmax, so a tile's keys and values are waited for
      // before P is, on which the softmax of the next tile hangs (64 nodes over
      // 65536 tokens: 75.5 us, 77.0 the other way round), and a wait tries once
      // before it loops (73.4).
      auto have_k = [&]() { wait(b_k + 8 * ks, kp); };
      auto have_v = [&]() { wait(b_vok + 8 * vs, vp); };
      // scores of the ring's next tile into stream s; `last`: its last reader
      auto qk = [&](int s, bool last) {
        if (dead) return;
        tc_fence_after();
        const uint64_t a = sdesc_sw128(sbase + C::kQOff + (kTwo ? s * C::kSlot : 0), 0, 1024);
        const uint64_t b = sdesc_sw128(sbase + ks * C::kSlot, 0, 1024);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint64_t off = (uint64_t)(((i >> 2) * kHalfBytes + (i & 3) * 32) >> 4);
          tc_mma_ss_elect(tm + C::kColS + s * 128, a + off, b + off, kIdQK, i);
        }
        tc_commit_elect(b_s + 8 * s);
        if (last) {
          tc_commit_elect(b_kfree + 8 * ks);
          if (++ks == C::kKSlots) {
            ks = 0;
            kp ^= 1;
          }
        }
      };
      auto pv = [&](int s, bool first, bool last) {
        if (!wait(b_p + 8 * s, (s ? np1 : np0) & 1)) return;
        if (s) ++np1; else ++np0;
        tc_fence_after();
        const uint64_t v = sdesc_sw128(sbase + C::kVOff + vs * C::kSlot, kHalfBytes, 1024);
#pragma unroll
        for (int i = 0; i < kTtTile / 16; ++i)
          tc_mma_ts_elect(tm + C::kColO + s * D, tm + C::kColS + s * 128 + i * 8,
                          v + (uint64_t)((i * 16 * 128) >> 4), kIdPV, (!first || i > 0) ? 1u : 0u);
        if (last) {
          tc_commit_elect(b_vfree + 8 * vs);
          if (++vs == C::kVSlots) {
            vs = 0;
            vp ^= 1;
          }
        }
      };
      TreePiece p;
      for (; !dead && tree_next(A, walk, p); ++item) {
        const int n = __shfl_sync(0xffffffffu, p.n, 0);
        wait(b_q, item & 1);
        if (!kTwo) {
#pragma unroll 1
          for (int k = 0; k <= n && !dead; ++k) {
            if (k < n) {
              have_k();
              qk(k & 1, true);
              if (k == n - 1) tc_commit_elect(b_qfree);
            }
            if (k == 1) wait(b_ofree, (item & 1) ^ 1);
            if (k > 0) {
              have_v();
              pv((k - 1) & 1, k <= 2, true);
            }
          }
        } else {
          const int streams = __shfl_sync(0xffffffffu, block_rows(p) > srows ? 2 : 1, 0);
#pragma unroll 1
          for (int k = 0; k <= n && !dead; ++k) {
            if (k == 1) wait(b_ofree, (item & 1) ^ 1);
            if (k > 0) have_v();
            if (k < n) have_k();
#pragma unroll 1
            for (int s = 0; s < streams; ++s) {
              if (k > 0) pv(s, k == 1, s + 1 == streams);
              if (k < n) qk(s, s + 1 == streams);
            }
            if (k == n - 1) tc_commit_elect(b_qfree);
          }
        }
        if (!dead) tc_commit_elect(b_o);
      }
      if (dead) {   // the products issued so far come to an end first
        tc_commit_elect(b_o);
        mbar_wait(b_o, (item - 1) & 1);
        __syncwarp();
      }
      if (dead && lane == 0) atomicAdd(errp, kTtStuck);
    }
  } else {
    // ---------------- softmax: a row per thread ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int s = (warp - 4) >> 2;                 // stream
    const int quarter = warp & 3;                  // tensor-memory lanes 32 quarter ..
    const int row = quarter * 32 + lane;           // row of the stream's query tile
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t ts = tmem + lane_off + C::kColS + s * 128;
    const uint32_t to = tmem + lane_off + C::kColO + s * D;
    float2* ml = reinterpret_cast<float2*>(smem + C::kMlOff);
    const int step = kTwo ? 1 : 2;
    uint32_t item = 0, ns = 0;
    bool dead = false;
    auto wait = [&](uint32_t bar, uint32_t par) {
      if (!dead && !__all_sync(0xffffffffu, mbar_wait(bar, par))) dead = true;
    };
    TreePiece p;
    for (; tree_next(A, walk, p); ++item) {
      const int nrows = block_rows(p);
      const int srow0 = kTwo ? s * srows : 0;            // the stream's first row of the block
      const int brow = srow0 + row;                      // row of the block
      const int have = min(srows, nrows - srow0);        // rows of the stream
      const bool real = row < have;
      const bool mine = quarter * 32 < have;             // warp has rows
      const bool takes = have > 0;                       // stream has work
      const int urow = p.rb * A.rows + brow;             // row of the request
      const uint64_t mask =
          real ? __ldcg((const unsigned long long*)A.mask + p.q0 + urow / A.G) : 0ull;
      float m = -INFINITY, l = 0.f;
      bool filled = false;                               // the accumulator holds earlier tiles
      if (takes) {
        ChunkBits it(A, p, !kTwo && p.n > s ? s : 0, lane);
        for (int k = kTwo ? 0 : s; k < p.n; k += step) {
          // this lane's chunk: first position and rank, and its tokens
          const int c_pos = it.it.x * kTtChunk, c_rank = it.it.r;
          const uint32_t bits = it.bits(A, lane);
          const uint32_t plain = __ballot_sync(0xffffffffu, bits == ~0u);
          if (k + step < p.n) it.next(A, p, step, lane);
          // a tile whose tokens all rows see takes no masks
          const bool special = (plain & 0xFFu) != 0xFFu;
          uint32_t vis[4] = {~0u, ~0u, ~0u, ~0u};
          uint32_t masked = 0;                // groups that some row sees in part
          if (special) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const uint32_t lo = __shfl_sync(0xffffffffu, bits, 2 * g);
              const uint32_t hi = __shfl_sync(0xffffffffu, bits, 2 * g + 1);
              vis[g] = __byte_perm(lo, hi, 0x5410);
              uint32_t nodes = __byte_perm(lo, hi, 0x7632) & ~vis[g];
              if (vis[g] != ~0u) masked |= 1u << g;
              if (nodes) {   // by this row's mask
                const int from = 2 * g + (lane >> 4);
                const int pos = __shfl_sync(0xffffffffu, c_pos, from) + (lane & 15);
                const int rank = __shfl_sync(0xffffffffu, c_rank, from);
                const int node = (tree_global(pos, rank, A.L) - p.ctx) & 63;
                do {
                  const int o = __ffs(nodes) - 1;
                  nodes &= nodes - 1;
                  const int j = __shfl_sync(0xffffffffu, node, o);
                  vis[g] |= ((uint32_t)(mask >> j) & 1u) << o;
                } while (nodes);
              }
            }
          }
          wait(b_s + 8 * s, ns & 1);
          ++ns;
          if (!dead && mine) {
            tc_fence_after();
            uint32_t x[4][32];
            auto load = [&]() {
#pragma unroll
              for (int g = 0; g < 4; ++g) tc_ld32(ts + g * 32, x[g]);
#pragma unroll
              for (int g = 0; g < 4; ++g) tc_wait_ld(x[g]);
              if (special) {
#pragma unroll
                for (int g = 0; g < 4; ++g)
                  if ((masked >> g) & 1) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                      if (!((vis[g] >> i) & 1)) x[g][i] = 0xff800000u;   // -inf
                  }
              }
            };
            load();
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = -INFINITY;
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
              for (int i = 0; i < 32; ++i) y[i & 7] = fmaxf(y[i & 7], __uint_as_float(x[g][i]));
#pragma unroll
            for (int w = 4; w > 0; w >>= 1)
#pragma unroll
              for (int i = 0; i < w; ++i) y[i] = fmaxf(y[i], y[i + w]);
            const float mx = y[0] * A.sl2;
            float f = 1.f;                  // for what the accumulator holds
            if (mx > m + kTtGrow || m == -INFINITY) {
              if (m != -INFINITY) {
                f = ex2_ftz(m - mx);
                l *= f;
              }
              m = mx;
            }
            if (filled && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
              for (int g = 0; g < D / 32; ++g) {
                tc_ld32(to + g * 32, x[0]);
                tc_wait_ld(x[0]);
#pragma unroll
                for (int i = 0; i < 32; ++i) x[0][i] = __float_as_uint(__uint_as_float(x[0][i]) * f);
                tc_st32(to + g * 32, x[0]);
              }
              tc_wait_st();
              load();   // the registers held the accumulator meanwhile
            }
            const float mb = m == -INFINITY ? 0.f : m;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              uint32_t pk[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float a = ex2_ftz(fmaf(__uint_as_float(x[g][2 * i]), A.sl2, -mb));
                const float b = ex2_ftz(fmaf(__uint_as_float(x[g][2 * i + 1]), A.sl2, -mb));
                sum[i & 3] += a + b;
                pk[i] = pack_bf16(a, b);
              }
              tc_st16(ts + g * 16, pk);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            filled = true;
            tc_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(b_p + 8 * s);
        }
      }
      // ---------------- the unit's (or piece's) rows ----------------
      wait(b_o, item & 1);
      tc_fence_after();
      // (written again only when the next unit's products are done, which wait
      // for every warp to have left this one)
      ml[s * 128 + row] = make_float2(m, l);
      bar_sync(3, 256);
      const bool odd = flag[item % kTtFlags] == (int)item + 1;
      if (!dead && mine && takes) {
        const float mb = m == -INFINITY ? 0.f : m;
        float M = mb, L = l, a0 = 1.f, a1 = 0.f;
        if (!kTwo) {
          const float2 o = ml[(s ^ 1) * 128 + row];
          const float ob = o.x == -INFINITY ? 0.f : o.x;
          // sums that are zero do not count, whatever their maximum
          M = l == 0.f ? ob : (o.y == 0.f ? mb : fmaxf(mb, ob));
          const float am = l == 0.f ? 0.f : ex2_ftz(mb - M);
          const float ao = o.y == 0.f ? 0.f : ex2_ftz(ob - M);
          L = s == 0 ? l * am + o.y * ao : o.y * ao + l * am;
          a0 = s == 0 ? am : ao;
          a1 = s == 0 ? ao : am;
        }
        const bool direct = p.slot < 0;
        const bool sunk = direct && A.sink != nullptr;
        float lse2 = -INFINITY, f = 0.f;
        const int h = p.g * A.G + urow % A.G;
        if (sunk) {
          const float s2 = __ldcg(A.sink + h) * kLog2e;
          const float top = L == 0.f ? s2 : fmaxf(M, s2);
          if (top > -INFINITY) {
            const float aa = L == 0.f ? 0.f : exp2f(M - top);
            const float tot = L * aa + exp2f(s2 - top);
            lse2 = top + log2f(tot);
            f = L == 0.f ? 0.f : aa / tot;
          } else if (L != 0.f) {
            lse2 = M + log2f(L);
            f = 1.f / L;
          }
        } else if (L != 0.f) {
          lse2 = M + log2f(L);
          f = 1.f / L;
        }
        const int64_t orow = direct && real ? tree_out_row(A, p, urow) : 0;
        const bool f32 = !direct || A.out_dtype == DCP_F32;
        void* dst = direct ? (f32 ? (void*)((float*)A.out + orow * D)
                                  : (void*)((__nv_bfloat16*)A.out + orow * D))
                           : (void*)(A.part_o + ((int64_t)p.slot * A.rows + brow) * D);
        const bool other = !kTwo && p.n > 1;      // the second stream had tiles
        const int c0 = kTwo ? 0 : s * (D / 2), c1 = kTwo ? D : c0 + D / 2;
        const uint32_t o0 = tmem + lane_off + C::kColO + (kTwo ? s * D : 0);
#pragma unroll 1
        for (int c = c0; c < c1; c += 32) {
          uint32_t x[32], y[32];
          tc_ld32(o0 + c, x);
          tc_wait_ld(x);
          const float fa = a0 * f, fb = a1 * f;
          if (other) {
            tc_ld32(o0 + D + c, y);
            tc_wait_ld(y);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float v = L == 0.f ? 0.f : __uint_as_float(x[i]) * fa;
            if (other && fb != 0.f) v = fmaf(__uint_as_float(y[i]), fb, v);
            x[i] = __float_as_uint(v);
          }
          if (kTwo && !direct) {
            // eight lanes exchange pieces so that they write 128 bytes of a row
            // at a time: 64 nodes over 65536 tokens 71.2 us, 73.4 when each lane
            // writes its own row.  With half of the rows the exchange's cold
            // instructions cost as much (8 nodes over 1500 tokens 16.0 and 15.3).
            transpose8(x, lane);
            float* part = A.part_o + ((int64_t)p.slot * A.rows + srow0) * D + c + 4 * (lane & 7);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int to_row = quarter * 32 + (lane & 24) + i;
              if (to_row < have)
                *reinterpret_cast<uint4*>(part + to_row * D) =
                    make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
            }
          } else if (real) {
            if (f32) {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<uint4*>((float*)dst + c + i) =
                    make_uint4(x[i], x[i + 1], x[i + 2], x[i + 3]);
            } else {
#pragma unroll
              for (int i = 0; i < 32; i += 8) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  w[j] = pack_bf16(__uint_as_float(x[i + 2 * j]), __uint_as_float(x[i + 2 * j + 1]));
                *reinterpret_cast<uint4*>((__nv_bfloat16*)dst + c + i) =
                    make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
        }
        if (kTwo && odd) __syncwarp();
        if (real) {
          if (odd) tree_fix<D>(A, p, urow, c0, c1, M, f, dst, f32);
          if (kTwo || s == 0) {
            if (!direct)
              A.part_lse[(int64_t)p.slot * A.rows + brow] = lse2;
            else if (A.lse)
              A.lse[orow] = lse2 * kLn2;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_ofree);
      if (p.slot >= 0 && A.join) {
        // the last run to bring its part joins them all
        const int k0 = tree_run_of(walk.total, walk.parts, p.u0);
        const int k1 = tree_run_of(walk.total, walk.parts, p.u0 + p.per - 1);
        __threadfence();
        bar_sync(3, 256);
        if (threadIdx.x == 128) {
          const int before = atomicAdd(A.arrived + k0, 1);
          flag[kTtFlags] = before == k1 - k0;
          __threadfence();
        }
        bar_sync(3, 256);
        if (flag[kTtFlags])
          tree_join<D>(A, p, k0, k1, tree_run(walk.total, walk.parts, k0) != p.u0, nrows, warp - 4);
      }
    }
    if (dead && lane == 0) atomicAdd(errp, kTtStuck);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tc_dealloc(tmem, 512);
  }
}

// [N][Hq][d] as boxes of 64 columns, G heads and `nodes` tokens.
static bool encode_q(CUtensorMap* map, const TreeArgs& A, int nodes) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)A.d, (cuuint64_t)A.Hq, (cuuint64_t)A.N};
  cuuint64_t strides[2] = {(cuuint64_t)A.d * 2, (cuuint64_t)A.Hq * A.d * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)A.G, (cuuint32_t)nodes};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(A.q), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool tree_tc_shape(int d, dcp_dtype_t dtype, int block_size) {
  return dtype == DCP_BF16 && (d == 64 || d == 128) && block_size % 16 == 0;
}

bool tree_tc_supported(const dcp_layout_t& layout, int d, dcp_dtype_t dtype,
                       const dcp_paged_kv_t& kv, int Hkv) {
  return tree_tc_shape(d, dtype, layout.block_size) &&
         (int64_t)kv.num_blocks * Hkv * layout.block_size < (int64_t(1) << 31) &&
         tensor_map_encoder() != nullptr;
}

template <int D, bool kTwo>
static int go(const TreeTcArgs& X, cudaStream_t s) {
  const int smem = TreeTc<D, kTwo>::kSmem;
  static_assert(TreeTc<D, kTwo>::kSmem <= 227 * 1024, "shared memory");
  if (!allow_smem<tree_tc_kernel<D, kTwo>>()) return DCP_ECUDA;
  const cudaError_t e = launch_chained(tree_tc_kernel<D, kTwo>, (unsigned)X.t.parts, kTtThreads,
                                       smem, s, X);
  return e == cudaSuccess ? launch_status() : launch_status_report(e);
}

int launch_tree_tc(const TreeArgs& A, cudaStream_t s) {
  TreeTcArgs X;
  memset(&X, 0, sizeof(X));
  X.t = A;
  X.nodes = 128 / A.G;
  if (!encode_q(&X.qmap, A, X.nodes)) return DCP_ECUDA;
  const uint64_t rows = (uint64_t)A.nb * A.Hkv * A.L.bs;
  for (int r = 0; r < A.L.dcp; ++r)
    if (!encode_2d_bf16_sw128(&X.kmap[r], A.k.ptr[r], A.d, rows > 0 ? rows : 1, A.d * 2, 64,
                              kTtChunk) ||
        !encode_2d_bf16_sw128(&X.vmap[r], A.v.ptr[r], A.d, rows > 0 ? rows : 1, A.d * 2, 64, kTtChunk))
      return DCP_ECUDA;
  const bool two = A.rows > X.nodes * A.G;
  if (A.d == 64) return two ? go<64, true>(X, s) : go<64, false>(X, s);
  return two ? go<128, true>(X, s) : go<128, false>(X, s);
}

}  // namespace dcp
