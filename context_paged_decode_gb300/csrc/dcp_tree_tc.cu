// tcgen05 kernel of the drafted-tree attention: bf16, head_dim 64 or 128.
//
// The query heads of a group and the drafted nodes share each key/value row,
// so a unit's scores S = Q K^T (rows = node * G + head) and O = P V are dense
// products over its tokens with up to 256 rows; the masks touch only the few
// tiles that hold drafted nodes.  Bytes bound it up to about 128 rows: a
// 128-token tile of keys and values (64 KB at head_dim 128) takes an SM 1.5 us
// of its share of the measured bandwidth, its two products 0.7 us for 128
// rows, its softmax 0.5 us of the exponential unit.
//
// One CTA per SM works through its run of tiles (see dcp_tree.cuh).  Two
// softmax warpgroups, a tensor-memory score buffer and an output accumulator
// each:
//  * up to 128 rows (kTwo false) they take the tiles in turn, with the same
//    queries, and join their sums at the end of a unit: one computes its
//    softmax while the tensor core works for the other;
//  * up to 256 rows (kTwo true) each has 128 of the rows and both go through
//    every tile, which is read once.
// Warps: 0 loads keys and values by TMA (boxes of 16 to 128 rows, a page or part
// of one, a lane each) into a ring of slots that alternate K and V; 1 issues the products; 2 and 3 load queries; 4-7 and 8-11
// are the softmax, one row per thread.  P goes back to tensor memory over the
// scores it came from (bf16, half the columns) and is the A operand of P V.
// The score product of a stream's next tile is issued after P V of its last,
// so a score barrier also says that the accumulator is at rest, and the rare
// rescale (only when the maximum grows by more than 2^8) needs no wait of its
// own.
//
// Masked tokens have P = 0, but 0 * x is not 0 for infinities and NaN.  Rows of
// V past the end or of unusable pages are zeroed in shared memory, and so are
// non-finite values of drafted nodes; the rows that do see such a node get its
// values added afterwards, one by one (tree_fix).
//
// Every wait is bounded; a timed-out role stops waiting and working but keeps
// step at the named barriers, so the kernel always ends.
#include <mutex>
#include <string.h>

#include "dcp_ptx.cuh"
#include "dcp_tree.cuh"

namespace dcp {

struct TreeTcArgs {
  CUtensorMap kmap[DCP_MAX_RANKS];   // [num_blocks * Hkv * bs rows][d], box 64 x `box`
  CUtensorMap vmap[DCP_MAX_RANKS];
  TreeArgs t;
  int box;                           // rows of a box: a power of two that divides bs, 16 .. 128
};

constexpr int kTtTile = 128;
constexpr int kTtThreads = 384;
constexpr int kHalfBytes = kTtTile * 128;    // 64 columns of a tile or of a query block
constexpr float kTtGrow = 8.f;               // log2 units
constexpr int kTtStuck = 1 << 20;

template <int D, bool kTwo>
struct TreeTc {
  static constexpr int kSlot = kTtTile * D * 2;
  static constexpr int kQ = (kTwo ? 2 : 1) * kSlot;
  static constexpr int kSlots = (224 * 1024 - kQ) / kSlot;  // 3 KB stay for the rest
  static constexpr int kQOff = kSlots * kSlot;
  static constexpr int kMlOff = kQOff + kQ;                 // float2 [2 stream][128]
  static constexpr int kCodeOff = kMlOff + 2 * 128 * 8;     // uint8 [2 stream][128]
  static constexpr int kFlagOff = kCodeOff + 2 * 128;       // int [2 parity]
  static constexpr int kBarOff = kFlagOff + 16;
  static constexpr int kBars = 2 * kSlots + 8;
  static constexpr int kSmem = kBarOff + 8 * kBars + 16;
  static constexpr uint32_t kColS = 0, kColO = 256;         // two of each, 128 and D apart
};

// Tiles of a unit in order: rank by rank.
struct TileIt {
  int r, tr, n, nt, lc;   // rank, tile on it, its tokens, tiles and context tokens
  __device__ __forceinline__ void at(const TreeArgs& A, int rank, int64_t len, int64_t ctx) {
    r = rank;
    n = tree_local(len, r, A.L);
    nt = (n + kTtTile - 1) / kTtTile;
    lc = tree_local(ctx, r, A.L);
  }
  __device__ __forceinline__ void seek(const TreeArgs& A, const TreePiece& p, int64_t len,
                                       int64_t ctx) {
    at(A, p.r0, len, ctx);
    tr = p.t0;
    settle(A, p, len, ctx);
  }
  __device__ __forceinline__ void settle(const TreeArgs& A, const TreePiece& p, int64_t len,
                                         int64_t ctx) {
    while (tr >= nt && r + 1 < p.r1) {
      tr -= nt;
      at(A, r + 1, len, ctx);
    }
  }
  __device__ __forceinline__ void step(const TreeArgs& A, const TreePiece& p, int64_t len,
                                       int64_t ctx, int k) {
    tr += k;
    settle(A, p, len, ctx);
  }
};

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ bool bf16_odd(uint32_t h) { return (h & 0x7F80u) == 0x7F80u; }

// Adds to output row `row` (columns [c0, c1)) what it sees of non-finite values
// of drafted nodes, which the product took as zero.  Rare and slow.
template <int D>
__device__ __noinline__ void tree_fix(const TreeArgs& A, const TreePiece& p, int T, int64_t ctx,
                                      int row, int c0, int c1, float M, float f, void* dst,
                                      bool f32) {
  const int64_t tok = __ldcg(A.q_start + p.b) + row / A.G;
  const uint64_t mask = __ldcg((const unsigned long long*)A.mask + tok);
  const __nv_bfloat16* q =
      (const __nv_bfloat16*)A.q + (tok * A.Hq + p.g * A.G + row % A.G) * (int64_t)D;
  for (int j = 0; j < T; ++j) {
    if (!((mask >> j) & 1)) continue;
    int r, loc;
    int64_t vb;
    place_token(ctx + j, A.L, r, vb, loc);
    if (r < p.r0 || r >= p.r1) continue;
    int t = (int)((vb * A.L.bs + loc) / kTtTile);        // tile of the unit
    for (int x = p.r0; x < r; ++x)
      t += (tree_local(ctx + T, x, A.L) + kTtTile - 1) / kTtTile;
    if (t < p.t0 || t >= p.t0 + p.n) continue;
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

template <int D, bool kTwo>
__global__ void __launch_bounds__(kTtThreads, 1)
tree_tc_kernel(const __grid_constant__ TreeTcArgs X) {
  using C = TreeTc<D, kTwo>;
  const TreeArgs& A = X.t;
  extern __shared__ __align__(1024) uint8_t smem[];   // no room is left to round up in
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bars = sbase + C::kBarOff;
  const uint32_t b_full = bars, b_empty = bars + 8 * C::kSlots;
  const uint32_t b_s = b_empty + 8 * C::kSlots;   // +stream: scores are there
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
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(b_full + 8 * i, 1);
      mbar_init(b_empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_s + 8 * i, 1);
      mbar_init(b_p + 8 * i, 4);
    }
    mbar_init(b_o, 1);
    mbar_init(b_ofree, 8);
    mbar_init(b_q, 2);
    mbar_init(b_qfree, 1);
    fence_mbar_init();
    flag[0] = flag[1] = 0;
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

  const int E = A.per_rank ? A.B * A.L.dcp : A.B;
  const int64_t total = __ldcg(A.first_tile + E);
  const int parts = __ldcg(A.hdr);
  const int run = blockIdx.x;
  int32_t* errp = A.err ? A.err : A.hdr + 1;
  const int64_t begin = run < parts ? tree_run(total, parts, run) : 0;
  const int64_t end = run < parts ? tree_run(total, parts, run + 1) : 0;
  int e = begin < end ? tree_entry(A, E, begin) : 0;

  auto block_rows = [&](const TreePiece& p, int T) {
    return min(A.rows, T * A.G - p.rb * A.rows);
  };

  if (warp == 0) {
    // ---------------- keys and values ----------------
    const uint64_t pol = policy_evict_first();
    const int box = X.box, nu = kTtTile / box;
    uint32_t seq = 0;
    bool dead = false;
    for (int64_t t = begin; t < end && !dead;) {
      const TreePiece p = tree_piece(A, e, t, begin, end, run);
      t += p.n;
      const int64_t ctx = __ldcg(A.ctx + p.b), len = ctx + __ldcg(A.nodes + p.b);
      const int32_t* bt = A.bt + (int64_t)p.b * A.max_vb;
      TileIt it;
      it.seek(A, p, len, ctx);
      // row of this lane's part of the tile, -1: nothing there, -2: unusable page
      auto part = [&](const TileIt& i) -> int64_t {
        const int pos = i.tr * kTtTile + lane * box;
        if (lane >= nu || pos >= i.n) return -1;
        const int j = pos / A.L.bs;
        const int64_t phys = j < A.max_vb ? (int64_t)__ldcg(bt + i.r * A.stride + j) : -1;
        if (phys < 0 || phys >= A.nb) return -2;
        return (phys * A.Hkv + p.g) * A.L.bs + (pos - j * A.L.bs);
      };
      int64_t row = part(it);
      for (int k = 0; k < p.n && !dead; ++k) {
        const int64_t mine = row;
        const int r = it.r;
        if (k + 1 < p.n) {
          it.step(A, p, len, ctx, 1);
          row = part(it);
        }
        const uint32_t m = __ballot_sync(0xffffffffu, mine >= 0);
        if (mine == -2) count_error(A.err);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++seq) {
          const uint32_t slot = seq % C::kSlots, u = seq / C::kSlots;
          if (!__all_sync(0xffffffffu, mbar_wait(b_empty + 8 * slot, (u & 1) ^ 1))) {
            dead = true;
            break;
          }
          const uint32_t bar = b_full + 8 * slot;
          if (lane == 0) {
            if (m)
              mbar_arrive_expect_tx(bar, __popc(m) * box * D * 2);
            else
              mbar_arrive(bar);
          }
          __syncwarp();
          if (mine >= 0) {
            const void* map = kv ? &X.vmap[r] : &X.kmap[r];
            const uint32_t dst = sbase + slot * C::kSlot + lane * box * 128;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              tma_load_2d_hint(dst + c * kHalfBytes, map, 64 * c, (int)mine, bar, pol);
          }
          __syncwarp();
        }
      }
    }
    if (dead && lane == 0) atomicAdd(errp, kTtStuck);
  } else if (warp == 1) {
    // ---------------- products ----------------
    if (lane == 0) {
      constexpr uint32_t kIdQK = idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t kIdPV = idesc_bf16_f32(128, D, false, true);
      uint32_t seq = 0, item = 0, np[2] = {0, 0};
      bool dead = false;
      auto wait = [&](uint32_t bar, uint32_t par) {
        if (!dead && !mbar_wait(bar, par)) dead = true;
        return !dead;
      };
      // scores of tile `tile` (counted over the run) into stream s
      auto qk = [&](int s, uint32_t tile, bool last) {
        const uint32_t i = 2 * tile, slot = i % C::kSlots;
        if (!wait(b_full + 8 * slot, (i / C::kSlots) & 1)) return;
        tc_fence_after();
        const uint64_t a = sdesc_sw128(sbase + C::kQOff + (kTwo ? s * C::kSlot : 0), 0, 1024);
        const uint64_t b = sdesc_sw128(sbase + slot * C::kSlot, 0, 1024);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t off = (uint64_t)((c * kHalfBytes + kk * 32) >> 4);
            tc_mma_ss(tmem + C::kColS + s * 128, a + off, b + off, kIdQK, (c | kk) != 0);
          }
        tc_commit(b_s + 8 * s);
        if (last) tc_commit(b_empty + 8 * slot);
      };
      auto pv = [&](int s, uint32_t tile, bool first, bool last) {
        const uint32_t i = 2 * tile + 1, slot = i % C::kSlots;
        if (!wait(b_p + 8 * s, np[s] & 1) || !wait(b_full + 8 * slot, (i / C::kSlots) & 1)) return;
        ++np[s];
        tc_fence_after();
        const uint32_t v = sbase + slot * C::kSlot;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          tc_mma_ts(tmem + C::kColO + s * D, tmem + C::kColS + s * 128 + kk * 8,
                    sdesc_sw128(v + kk * 16 * 128, kHalfBytes, 1024), kIdPV,
                    (!first || kk > 0) ? 1u : 0u);
        if (last) tc_commit(b_empty + 8 * slot);
      };
      for (int64_t t = begin; t < end && !dead; ++item) {
        const TreePiece p = tree_piece(A, e, t, begin, end, run);
        t += p.n;
        const bool two = kTwo && block_rows(p, __ldcg(A.nodes + p.b)) > 128;
        wait(b_q, item & 1);
        if (!kTwo) {
          for (int k = 0; k <= p.n && !dead; ++k) {
            if (k < p.n) {
              qk(k & 1, seq + k, true);
              if (k == p.n - 1) tc_commit(b_qfree);
            }
            if (k == 1) wait(b_ofree, (item & 1) ^ 1);
            if (k > 0) pv((k - 1) & 1, seq + k - 1, k <= 2, true);
          }
        } else {
          qk(0, seq, !two);
          if (two) qk(1, seq, true);
          if (p.n == 1) tc_commit(b_qfree);
          wait(b_ofree, (item & 1) ^ 1);
          for (int k = 0; k < p.n && !dead; ++k) {
            pv(0, seq + k, k == 0, !two);
            if (k + 1 < p.n) qk(0, seq + k + 1, !two);
            if (two) {
              pv(1, seq + k, k == 0, true);
              if (k + 1 < p.n) qk(1, seq + k + 1, true);
            }
            if (k + 2 == p.n) tc_commit(b_qfree);
          }
        }
        seq += p.n;
        if (!dead) tc_commit(b_o);
      }
      if (dead) atomicAdd(errp, kTtStuck);
    }
  } else if (warp < 4) {
    // ---------------- queries ----------------
    const int tid = threadIdx.x - 64;
    uint32_t item = 0;
    bool dead = false;
    for (int64_t t = begin; t < end && !dead; ++item) {
      const TreePiece p = tree_piece(A, e, t, begin, end, run);
      t += p.n;
      const int T = __ldcg(A.nodes + p.b), nrows = block_rows(p, T);
      const int64_t tok0 = __ldcg(A.q_start + p.b);
      constexpr int cpr = D / 8;
      if (item > 0 && !__all_sync(0xffffffffu, mbar_wait(b_qfree, (item - 1) & 1))) {
        dead = true;
        break;
      }
      for (int i0 = tid; i0 < nrows * cpr; i0 += 64 * 8) {
        uint4 x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = i0 + 64 * j;
          if (i < nrows * cpr) {
            const int rr = p.rb * A.rows + i / cpr;
            const int node = rr / A.G;
            x[j] = __ldcg((const uint4*)A.q +
                          ((tok0 + node) * A.Hq + p.g * A.G + (rr - node * A.G)) * cpr + i % cpr);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = i0 + 64 * j;
          if (i < nrows * cpr) {
            const int row = i / cpr, c = i % cpr;
            const uint32_t dst = sbase + C::kQOff + (row >> 7) * C::kSlot + (c >> 3) * kHalfBytes +
                                 (row & 127) * 128 + (((c & 7) ^ (row & 7)) << 4);
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(x[j].x),
                         "r"(x[j].y), "r"(x[j].z), "r"(x[j].w)
                         : "memory");
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_q);
    }
    if (dead && lane == 0) atomicAdd(errp, kTtStuck);
  } else {
    // ---------------- softmax: a row per thread ----------------
    const int s = (warp - 4) >> 2;                 // stream
    const int quarter = warp & 3;                  // tensor-memory lanes 32 quarter ..
    const int row = quarter * 32 + lane;           // row of the stream's 128
    const int wtid = threadIdx.x - 128 - s * 128;  // thread of the warpgroup
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t ts = tmem + lane_off + C::kColS + s * 128;
    const uint32_t to = tmem + lane_off + C::kColO + s * D;
    uint8_t* code = smem + C::kCodeOff + s * 128;
    float2* ml = reinterpret_cast<float2*>(smem + C::kMlOff);
    const int step = kTwo ? 1 : 2;
    uint32_t seq = 0, item = 0, ns = 0;
    bool dead = false;
    auto wait = [&](uint32_t bar, uint32_t par) {
      if (!dead && !__all_sync(0xffffffffu, mbar_wait(bar, par))) dead = true;
    };
    for (int64_t t = begin; t < end; ++item) {
      const TreePiece p = tree_piece(A, e, t, begin, end, run);
      t += p.n;
      const int T = __ldcg(A.nodes + p.b);
      const int64_t ctx = __ldcg(A.ctx + p.b), len = ctx + T;
      const int nrows = block_rows(p, T);
      const int brow = kTwo ? s * 128 + row : row;       // row of the block
      const bool mine = (kTwo ? s * 128 : 0) + quarter * 32 < nrows;   // warp has rows
      const bool takes = !kTwo || s == 0 || nrows > 128;               // stream has work
      const int urow = p.rb * A.rows + brow;             // row of the request
      const uint64_t mask =
          brow < nrows
              ? __ldcg((const unsigned long long*)A.mask + __ldcg(A.q_start + p.b) + urow / A.G)
              : 0ull;
      float m = -INFINITY, l = 0.f;
      bool filled = false;                               // the accumulator holds earlier tiles
      if (takes) {
        TileIt it;
        it.seek(A, p, len, ctx);
        if (!kTwo && s == 1) it.step(A, p, len, ctx, 1);
        for (int k = kTwo ? 0 : s; k < p.n; k += step) {
          const int p0 = it.tr * kTtTile, nv = min(kTtTile, it.n - p0);
          // usable pages of the tile, 16 tokens a bit
          bool good = true;
          if (lane < 8 && lane * 16 < nv) {
            const int j = (p0 + lane * 16) / A.L.bs;
            const int64_t phys =
                j < A.max_vb
                    ? (int64_t)__ldcg(A.bt + it.r * A.stride + (int64_t)p.b * A.max_vb + j)
                    : -1;
            good = phys >= 0 && phys < A.nb;
          }
          const uint32_t pages = __ballot_sync(0xffffffffu, good);
          const bool special = nv < kTtTile || p0 + nv > it.lc || (pages & 0xFFu) != 0xFFu;
          const uint32_t vi = 2 * (seq + k) + 1;          // the tile's V slot
          uint32_t vis[4] = {~0u, ~0u, ~0u, ~0u};
          if (special) {
            // who sees token wtid: 64 everyone, 255 nobody, else node's bit
            const int pos = p0 + wtid;
            int c = 255;
            if (wtid < nv && ((pages >> (wtid >> 4)) & 1))
              c = pos < it.lc ? 64 : (int)(tree_global(pos, it.r, A.L) - ctx);
            code[wtid] = (uint8_t)c;
            bar_sync(1 + s, 128);
            wait(b_full + 8 * (vi % C::kSlots), (vi / C::kSlots) & 1);
            const uint32_t v = sbase + (vi % C::kSlots) * C::kSlot;
            if (!dead) {
              // V rows nobody sees become zero, as do odd values of nodes
              for (int i = wtid; i < kTtTile * (D / 8); i += 128) {
                const int tok = i / (D / 8), ch = i % (D / 8), cd = code[tok];
                if (cd == 64) continue;
                const uint32_t at = v + (ch >> 3) * kHalfBytes + tok * 128 +
                                    (((ch & 7) ^ (tok & 7)) << 4);
                uint32_t w[4] = {0u, 0u, 0u, 0u};
                bool odd = cd == 255;
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
                  if (odd) flag[item & 1] = (int)item + 1;
                }
                if (odd)
                  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(w[0]),
                               "r"(w[1]), "r"(w[2]), "r"(w[3])
                               : "memory");
              }
              fence_proxy_async_smem();
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              uint32_t bits = 0;
              for (int i = 0; i < 32; ++i) {
                const int cd = code[g * 32 + i];
                const uint32_t on = cd == 64 ? 1u : cd < 64 ? (uint32_t)(mask >> cd) & 1u : 0u;
                bits |= on << i;
              }
              vis[g] = bits;
            }
            bar_sync(1 + s, 128);   // the codes may be written again
          }
          wait(b_s + 8 * s, ns & 1);
          ++ns;
          if (!dead && mine) {
            tc_fence_after();
            float mx = -INFINITY;
            uint32_t x[32];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              tc_ld32(ts + g * 32, x);
              tc_wait_ld(x);
              if (special) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  mx = fmaxf(mx, (vis[g] >> i) & 1 ? __uint_as_float(x[i]) : -INFINITY);
              } else {
                float y[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < 32; ++i) y[i & 3] = fmaxf(y[i & 3], __uint_as_float(x[i]));
                mx = fmaxf(mx, fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])));
              }
            }
            mx *= A.sl2;
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
                tc_ld32(to + g * 32, x);
                tc_wait_ld(x);
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
                tc_st32(to + g * 32, x);
              }
            }
            const float mb = m == -INFINITY ? 0.f : m;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              tc_ld32(ts + g * 32, x);
              tc_wait_ld(x);
              uint32_t pk[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float a = ex2_ftz(fmaf(__uint_as_float(x[2 * i]), A.sl2, -mb));
                float b = ex2_ftz(fmaf(__uint_as_float(x[2 * i + 1]), A.sl2, -mb));
                if (special) {
                  a = (vis[g] >> (2 * i)) & 1 ? a : 0.f;
                  b = (vis[g] >> (2 * i + 1)) & 1 ? b : 0.f;
                }
                sum[i & 3] += a + b;
                pk[i] = pack_bf16(a, b);
              }
              tc_st16(ts + g * 16, pk);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            filled = true;
            tc_wait_st();
            tc_fence_before();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(b_p + 8 * s);
          if (k + step < p.n) it.step(A, p, len, ctx, step);
        }
      }
      // ---------------- the unit's (or piece's) rows ----------------
      wait(b_o, item & 1);
      tc_fence_after();
      // (written again only when the next unit's products are done, which wait
      // for every warp to have left this one)
      ml[s * 128 + row] = make_float2(m, l);
      bar_sync(3, 256);
      const bool odd = flag[item & 1] == (int)item + 1;
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
        float M2 = M;
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
        const bool real = brow < nrows;
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
          if (real) {
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
        if (real) {
          if (odd) tree_fix<D>(A, p, T, ctx, urow, c0, c1, M2, f, dst, f32);
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
      seq += p.n;
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

static int tree_box(int bs) {
  int b = 16;
  while (b < 128 && bs % (2 * b) == 0) b *= 2;
  return b;
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
  if (cudaFuncSetAttribute(tree_tc_kernel<D, kTwo>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           smem) != cudaSuccess) {
    cudaGetLastError();
    return DCP_ECUDA;
  }
  const cudaError_t e = launch_chained(tree_tc_kernel<D, kTwo>, (unsigned)X.t.parts, kTtThreads,
                                       smem, s, X);
  return e == cudaSuccess ? launch_status() : launch_status_report(e);
}

int launch_tree_tc(const TreeArgs& A, cudaStream_t s) {
  TreeTcArgs X;
  memset(&X, 0, sizeof(X));
  X.t = A;
  X.box = tree_box(A.L.bs);
  const uint64_t rows = (uint64_t)A.nb * A.Hkv * A.L.bs;
  for (int r = 0; r < A.L.dcp; ++r)
    if (!encode_2d_bf16_sw128(&X.kmap[r], A.k.ptr[r], A.d, rows > 0 ? rows : 1, A.d * 2, 64,
                              X.box) ||
        !encode_2d_bf16_sw128(&X.vmap[r], A.v.ptr[r], A.d, rows > 0 ? rows : 1, A.d * 2, 64, X.box))
      return DCP_ECUDA;
  if (A.d == 64) return A.rows > 128 ? go<64, true>(X, s) : go<64, false>(X, s);
  return A.rows > 128 ? go<128, true>(X, s) : go<128, false>(X, s);
}

}  // namespace dcp
