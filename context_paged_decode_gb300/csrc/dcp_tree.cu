// Attention of drafted token trees over the sharded paged cache: plan, the
// CUDA-core kernel for any supported shape, merge, and the entry points.
//
// Request b has ctx_b cached tokens and T_b drafted nodes stored behind them,
// node j at position ctx_b + j.  Every node sees the whole context and those
// nodes whose bits its mask has (its ancestors and itself).  Ranks attend
// their own shards and the parts are joined by log-sum-exp, page "Decode
// Context Parallel (DCP)", section "Decode"; with one node and its own bit
// set this is the ordinary decode step.
#include "dcp_ptx.cuh"
#include "dcp_tree.cuh"

namespace dcp {

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------

// Every kernel here may be launched, as a programmatic dependent, while the
// kernels before it still run, so what those write (and the plan, which the
// next call writes to the same workspace) is read past the SM's L1 (__ldcg):
// a read-only load may find a line that an earlier grid left there.
constexpr int kTreePlanThreads = 256;

// One CTA: checks the requests, counts each entry's tiles and units, sums them
// up, and finds each run's first entry.
__global__ void __launch_bounds__(kTreePlanThreads) tree_plan_kernel(const __grid_constant__ TreeArgs A) {
  __shared__ int64_t sh_t[kTreePlanThreads / 32], sh_u[kTreePlanThreads / 32];
  __shared__ int64_t s_end[kTreePlanThreads];   // tiles up to each entry of the block
  griddep_launch_dependents();   // the next call's first kernel may start its launch
  griddep_wait();                // launched chained: the preceding kernel completed
  const int E = A.per_rank ? A.B * A.L.dcp : A.B;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const bool single = E <= kTreePlanThreads;
  int64_t tiles = 0, units = 0, extra = 0, total = 0;
  for (int k = tid; k < A.parts; k += kTreePlanThreads) A.arrived[k] = 0;
  // more entries than threads: a first round only for the sums
  for (int round = single ? 1 : 0; round < 2; ++round) {
    const int64_t all_t = tiles, all_u = units;
    tiles = units = 0;
    for (int e0 = 0; e0 < E; e0 += kTreePlanThreads) {
      const int e = e0 + tid;
      TreeEntry n;
      n.units = n.per = n.nodes = n.ctx = n.q0 = n.pad = 0;
      if (e < E) n = tree_request(A, e, round == 1);
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
      __syncthreads();
      if (lane == 31) {
        sh_t[w] = t;
        sh_u[w] = u;
      }
      __syncthreads();
      const int64_t block_t = tiles, block_u = units;
      t += tiles;
      u += units;   // with this entry's own
      for (int i = 0; i < kTreePlanThreads / 32; ++i) {
        if (i < w) {
          t += sh_t[i];
          u += sh_u[i];
        }
        tiles += sh_t[i];
        units += sh_u[i];
      }
      if (round == 0) continue;
      const int64_t sum_t = single ? tiles : all_t, sum_u = single ? units : all_u;
      extra = tree_extra(A, sum_t);
      total = sum_t + extra * sum_u;
      const int64_t end = t + extra * u;
      n.tile0 = end - n.units * (n.per + extra);
      if (e < E) A.entry[e] = n;
      // the runs that begin in this block's entries
      s_end[tid] = end;
      __syncthreads();
      const int64_t first = block_t + extra * block_u, last = tiles + extra * units;
      const int parts = (int)(total < A.parts ? total : A.parts);
      for (int k = tid; k < parts; k += kTreePlanThreads) {
        const int64_t at = tree_run(total, parts, k);
        if (at < first || at >= last) continue;
        int lo = 0, hi = kTreePlanThreads - 1;   // first entry that ends behind `at`
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (s_end[mid] > at) hi = mid; else lo = mid + 1;
        }
        A.run_entry[k] = e0 + lo;
      }
    }
  }
  if (tid == 0) {
    A.hdr[0] = total < A.parts ? (int)total : A.parts;
    A.hdr[1] = 0;
    *reinterpret_cast<int64_t*>(A.hdr + 2) = total;
    A.hdr[4] = (int)extra;
  }
}

// ---------------------------------------------------------------------------
// writing a row
// ---------------------------------------------------------------------------

// Factor for an unnormalised row (maximum m in log2 units, sum l) with an
// optional sink, and its LSE in log2 units (-inf: nothing was seen).
__device__ __forceinline__ float tree_close(float m, float l, bool has_sink, float sink,
                                            float& lse2) {
  if (has_sink) {
    const float s2 = sink * kLog2e, M = fmaxf(m, s2);
    if (M > -INFINITY) {
      const float a = m == -INFINITY ? 0.f : exp2f(m - M);
      const float L = l * a + exp2f(s2 - M);
      lse2 = M + log2f(L);
      return a / L;
    }
  }
  if (l == 0.f) {
    lse2 = -INFINITY;
    return 0.f;
  }
  lse2 = m + log2f(l);
  return 1.f / l;
}

// ---------------------------------------------------------------------------
// CUDA-core kernel
// ---------------------------------------------------------------------------

constexpr int kTgTile = 64;     // tokens of a tile, two per lane
constexpr int kTgWarps = 8;
constexpr int kTgPad = 16;      // bytes: a lane's 16-byte reads of its own K row hit 32 banks

template <typename T>
struct Chunk;                   // 16 bytes of T as floats
template <>
struct Chunk<float> {
  static constexpr int n = 4;
  static __device__ __forceinline__ void to(const uint4& x, float* f) {
    f[0] = __uint_as_float(x.x);
    f[1] = __uint_as_float(x.y);
    f[2] = __uint_as_float(x.z);
    f[3] = __uint_as_float(x.w);
  }
};
template <>
struct Chunk<__nv_bfloat16> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void to(const uint4& x, float* f) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(w[i]);
      f[2 * i + 1] = bf16_hi(w[i]);
    }
  }
};

// Columns of a lane: consecutive ones, so that a row of V is read in one piece
// per lane (two columns of up to 64, four of each 128).
template <int DPL>
__device__ __forceinline__ int tg_col(int lane, int i) {
  return DPL == 2 ? lane * 2 + i : (i >> 2) * 128 + lane * 4 + (i & 3);
}

// A lane's columns of a row, zeros beyond its end.
template <int DPL>
__device__ __forceinline__ void tg_row(const float* row, int d, int lane, float* v) {
#pragma unroll
  for (int i = 0; i < DPL; i += 4) {
    const int c = tg_col<DPL>(lane, i);
    if (DPL == 2) {
      const float2 x = c < d ? *(const float2*)(row + c) : make_float2(0.f, 0.f);
      v[0] = x.x;
      v[1] = x.y;
    } else {
      const float4 x = c < d ? *(const float4*)(row + c) : make_float4(0.f, 0.f, 0.f, 0.f);
      v[i] = x.x;
      v[i + 1] = x.y;
      v[(i + 2) % DPL] = x.z;
      v[(i + 3) % DPL] = x.w;
    }
  }
}
template <int DPL>
__device__ __forceinline__ void tg_row(const __nv_bfloat16* row, int d, int lane, float* v) {
#pragma unroll
  for (int i = 0; i < DPL; i += 4) {
    const int c = tg_col<DPL>(lane, i);
    uint2 x = make_uint2(0u, 0u);
    if (DPL == 2) {
      if (c < d) x.x = *(const uint32_t*)(row + c);
    } else if (c < d) {
      x = *(const uint2*)(row + c);
    }
    v[i] = bf16_lo(x.x);
    v[i + 1] = bf16_hi(x.x);
    if (DPL > 2) {
      v[(i + 2) % DPL] = bf16_lo(x.y);
      v[(i + 3) % DPL] = bf16_hi(x.y);
    }
  }
}

// 16 bytes to shared memory, past the L1; zeros if `there` is false.
__device__ __forceinline__ void tg_copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void tg_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// All groups but the newest one have landed.
__device__ __forceinline__ void tg_wait() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

// Scores on the lanes (a lane has tokens lane and lane + 32 of the tile, whose
// K rows it reads from shared memory), output on the lanes as well, the
// probabilities between them through shared memory.  A warp carries RW query
// rows, so each K and V value read serves RW products.  Eight rows would halve
// the shared-memory reads, but leave registers for one CTA an SM, whose eight
// warps cannot hide each other's latency (4 requests x 16 nodes, d 128, 8192
// tokens: 140 us against 69).  Keys of the next tile are on their way while the
// values of this one are used, and its values while the next scores are made,
// so one buffer of each does.  With d 256, where an SM holds one CTA, that took
// 4 requests x 4 nodes over up to 8192 tokens (8 heads, bf16) from 219 us to
// 135; with two CTAs it changes nothing (d 128 as above: 66 and 67).  Masked
// tokens have probability zero, and values that nobody sees are zeros in shared
// memory; if a drafted node's value is not finite, the tile's products skip
// unseen nodes one by one.  What bounds it: the products on the CUDA cores and
// the shared-memory reads that feed them (those 66 us are 17 TFLOP/s; a tile's
// products would take 43% of its cycles, its reads 60%), and on short contexts
// latency: 2 x 11 nodes over up to 3001 tokens of 2 heads of 64 in fp32 (4.3
// MB) take 22.6 to 23.5 us, the merge 5 of them.
template <typename T, int DPL, int RW>
__global__ void __launch_bounds__(kTgWarps * 32)
tree_generic_kernel(const __grid_constant__ TreeArgs A) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t s_row[2][kTgTile];   // K/V row of a token, -1: not there
  __shared__ int s_code[2][kTgTile];      // node, 64: seen by all, 255: by none
  __shared__ TreeSelf s_plan;
  constexpr int kRows = kTgWarps * RW, CN = Chunk<T>::n;
  const int d = A.d, d4 = d >> 2;
  const int row_bytes = d * (int)sizeof(T), pitch = row_bytes + kTgPad;
  float* sq = reinterpret_cast<float*>(smem);                  // [rows][d]
  float* sp = sq + kRows * d;                                  // [warps][tile][RW]
  uint8_t* sv = reinterpret_cast<uint8_t*>(sp + kTgTile * kRows);   // [tile][d]
  uint8_t* sk = sv + kTgTile * row_bytes;                      // [tile][d + pad]
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float* pw = sp + warp * kTgTile * RW;
  const int cpr = d / CN;          // 16-byte pieces of a row
  const int lpr = cpr <= 8 ? 8 : (cpr <= 16 ? 16 : 32);   // lanes that copy one
  if (A.self) {
    if (warp == 0) tree_self_plan(A, &s_plan);
    __syncthreads();
  }
  for (int run = blockIdx.x; run < A.parts; run += gridDim.x) {
    TreeWalk walk = tree_walk(A, run, A.self ? &s_plan : nullptr);
    TreePiece p;
    while (tree_next(A, walk, p)) {
      const int ctx = p.ctx;
      const TreeLen len(ctx + p.T, A.L);
      const int row0 = p.rb * A.rows, nrows = min(A.rows, p.T * A.G - row0);
      // rank and tile within the rank of the next tile to be loaded
      int r = p.r0, tr = p.t0, n_r = len.on(r, A.L);
      auto settle = [&]() {
        while (tr >= (n_r + kTgTile - 1) / kTgTile) {
          tr -= (n_r + kTgTile - 1) / kTgTile;
          n_r = len.on(++r, A.L);
        }
      };
      // its token `tid`: the row, and who sees it
      int64_t t_row = -1;
      int t_code = 255;
      auto look = [&]() {
        t_row = -1;
        t_code = 255;
        const int pos = tr * kTgTile + tid;
        if (tid >= kTgTile || pos >= n_r) return;
        const int j = pos / A.L.bs;
        const int64_t phys =
            j < A.max_vb ? (int64_t)__ldcg(A.bt + r * A.stride + (int64_t)p.b * A.max_vb + j) : -1;
        if (phys >= 0 && phys < A.nb) {
          t_row = (phys * A.Hkv + p.g) * A.L.bs + (pos - j * A.L.bs);
          const int x = tree_global(pos, r, A.L) - ctx;
          t_code = x < 0 ? 64 : x;
        } else {
          count_error(A.err);
        }
      };
      auto keep = [&](int buf) {
        if (tid < kTgTile) {
          s_row[buf][tid] = t_row;
          s_code[buf][tid] = t_code;
        }
      };
      auto bring = [&](uint8_t* to, int to_pitch, const void* pool, int buf) {
        for (int j = (warp * 32 + lane) / lpr; j < kTgTile; j += kTgWarps * 32 / lpr) {
          const int64_t row = s_row[buf][j];
          const uint8_t* from = (const uint8_t*)pool + (row < 0 ? 0 : row) * row_bytes;
          for (int c = lane % lpr; c < cpr; c += lpr)
            tg_copy16(smem_u32(to + j * to_pitch + c * 16), from + c * 16, row >= 0);
        }
        tg_commit();
      };
      settle();
      look();
      __syncthreads();                 // the last piece is done with all of it
      keep(0);
      for (int i = tid; i < nrows * cpr; i += kTgWarps * 32) {
        const int row = i / cpr, c = (i - row * cpr) * CN, rr = row0 + row;
        const int64_t tok = p.q0 + rr / A.G;
        float f[CN];
        Chunk<T>::to(__ldcg((const uint4*)((const T*)A.q +
                                           (tok * A.Hq + p.g * A.G + rr % A.G) * d + c)),
                     f);
#pragma unroll
        for (int x = 0; x < CN; x += 4)
          *(float4*)(sq + row * d + c + x) = make_float4(f[x], f[x + 1], f[x + 2], f[x + 3]);
      }
      uint64_t mask[RW];
      float m[RW], l[RW], o[RW][DPL];
#pragma unroll
      for (int x = 0; x < RW; ++x) {
        const int row = warp * RW + x;
        mask[x] = row < nrows ? __ldcg((const unsigned long long*)A.mask + p.q0 +
                                       (row0 + row) / A.G)
                              : 0ull;
        m[x] = -INFINITY;
        l[x] = 0.f;
#pragma unroll
        for (int i = 0; i < DPL; ++i) o[x][i] = 0.f;
      }
      const bool idle = warp * RW >= nrows;   // no rows here (uniform in the warp)
      __syncthreads();
      bring(sk, pitch, A.k.ptr[r], 0);
      bring(sv, row_bytes, A.v.ptr[r], 0);
      for (int step = 0; step < p.n; ++step) {
        const int buf = step & 1;
        const bool more = step + 1 < p.n;
        if (more) {   // the next tile's table entries come during the scores
          ++tr;
          settle();
          look();
        }
        tg_wait();
        __syncthreads();               // the keys are there
        float s[2][RW];
#pragma unroll
        for (int x = 0; x < RW; ++x) s[0][x] = s[1][x] = 0.f;
        const uint4* k0 = (const uint4*)(sk + lane * pitch);
        const uint4* k1 = (const uint4*)(sk + (lane + 32) * pitch);
        const float4* qr = (const float4*)(sq + warp * RW * d);
#pragma unroll 2
        for (int c = 0; c < (idle ? 0 : cpr); ++c) {
          float a[CN], e[CN];
          Chunk<T>::to(k0[c], a);
          Chunk<T>::to(k1[c], e);
#pragma unroll
          for (int y = 0; y < CN; y += 4)
#pragma unroll
            for (int x = 0; x < RW; ++x) {
              const float4 b = qr[x * d4 + c * (CN / 4) + y / 4];
              s[0][x] = fmaf(a[y], b.x,
                             fmaf(a[y + 1], b.y, fmaf(a[y + 2], b.z, fmaf(a[y + 3], b.w, s[0][x]))));
              s[1][x] = fmaf(e[y], b.x,
                             fmaf(e[y + 1], b.y, fmaf(e[y + 2], b.z, fmaf(e[y + 3], b.w, s[1][x]))));
            }
        }
        if (more) keep(buf ^ 1);
        __syncthreads();               // the keys are done with
        if (more)
          bring(sk, pitch, A.k.ptr[r], buf ^ 1);
        else
          tg_commit();
        uint32_t vis[2][RW];
        if (!idle) {
          const int code0 = s_code[buf][lane], code1 = s_code[buf][lane + 32];
#pragma unroll
          for (int x = 0; x < RW; ++x) {
            const bool on0 = code0 == 64 || (code0 < 64 && ((mask[x] >> code0) & 1));
            const bool on1 = code1 == 64 || (code1 < 64 && ((mask[x] >> code1) & 1));
            vis[0][x] = __ballot_sync(0xffffffffu, on0);
            vis[1][x] = __ballot_sync(0xffffffffu, on1);
            const float s0 = on0 ? s[0][x] * A.sl2 : -INFINITY;
            const float s1 = on1 ? s[1][x] * A.sl2 : -INFINITY;
            const float mn = fmaxf(m[x], warp_max(fmaxf(s0, s1)));
            const float mb = mn == -INFINITY ? 0.f : mn;
            const float al = exp2f(m[x] - mb);
            const float p0 = on0 ? exp2f(s0 - mb) : 0.f, p1 = on1 ? exp2f(s1 - mb) : 0.f;
            l[x] = l[x] * al + (p0 + p1);      // this lane's tokens
            m[x] = mn;
#pragma unroll
            for (int i = 0; i < DPL; ++i) o[x][i] *= al;
            pw[lane * RW + x] = p0;
            pw[(lane + 32) * RW + x] = p1;
          }
        }
        tg_wait();
        // the values are there, and if nodes are among them some may not be finite
        bool odd = __syncthreads_or(tid < kTgTile && s_code[buf][tid] < 64);
        if (odd) {
          bool bad = false;
          for (int j = (warp * 32 + lane) / lpr; j < kTgTile; j += kTgWarps * 32 / lpr)
            if (s_code[buf][j] < 64)
              for (int c = lane % lpr; c < cpr; c += lpr) {
                float f[CN];
                Chunk<T>::to(*(const uint4*)(sv + j * row_bytes + c * 16), f);
#pragma unroll
                for (int x = 0; x < CN; ++x) bad |= !isfinite(f[x]);
              }
          odd = __syncthreads_or(bad);
        }
        if (!idle) {
          const T* vt = reinterpret_cast<const T*>(sv);
          if (!odd) {
#pragma unroll 4
            for (int j = 0; j < kTgTile; ++j) {
              float pj[RW], v[DPL];
              if (RW == 4) {
                const float4 q = *(const float4*)(pw + j * RW);
                pj[0] = q.x;
                pj[1] = q.y;
                pj[2 % RW] = q.z;
                pj[3 % RW] = q.w;
              } else {
                const float2 q = *(const float2*)(pw + j * RW);
                pj[0] = q.x;
                pj[1] = q.y;
              }
              tg_row<DPL>(vt + j * d, d, lane, v);
#pragma unroll
              for (int i = 0; i < DPL; ++i)
#pragma unroll
                for (int x = 0; x < RW; ++x) o[x][i] = fmaf(pj[x], v[i], o[x][i]);
            }
          } else {
#pragma unroll 1
            for (int j = 0; j < kTgTile; ++j) {
              float v[DPL];
              tg_row<DPL>(vt + j * d, d, lane, v);
#pragma unroll
              for (int x = 0; x < RW; ++x) {
                if (!(((j < 32 ? vis[0][x] : vis[1][x]) >> (j & 31)) & 1)) continue;
                const float pj = pw[j * RW + x];
#pragma unroll
                for (int i = 0; i < DPL; ++i) o[x][i] = fmaf(pj, v[i], o[x][i]);
              }
            }
          }
        }
        if (more) {
          __syncthreads();             // the values are done with
          bring(sv, row_bytes, A.v.ptr[r], buf ^ 1);
        }
      }
#pragma unroll
      for (int x = 0; x < RW; ++x) {
        const int row = warp * RW + x;
        if (row >= nrows) continue;
        const float lt = warp_sum(l[x]);
        const bool whole = p.slot < 0, sunk = whole && A.sink != nullptr;
        const int h = p.g * A.G + (row0 + row) % A.G;
        float lse2;
        const float f = tree_close(m[x], lt, sunk, sunk ? __ldcg(A.sink + h) : 0.f, lse2);
        const int64_t at = whole ? tree_out_row(A, p, row0 + row) : (int64_t)p.slot * A.rows + row;
        float* of = (whole ? (float*)A.out : A.part_o) + at * d;
        __nv_bfloat16* ob = (__nv_bfloat16*)A.out + at * d;
        const bool wide = !whole || A.out_dtype == DCP_F32;
#pragma unroll
        for (int i = 0; i < DPL; i += 2) {
          const int c = tg_col<DPL>(lane, i);
          if (c >= d) continue;
          const float a = lt == 0.f ? 0.f : o[x][i] * f, b = lt == 0.f ? 0.f : o[x][i + 1] * f;
          if (wide)
            *(float2*)(of + c) = make_float2(a, b);
          else
            *(uint32_t*)(ob + c) = pack_bf16(a, b);
        }
        if (lane == 0) {
          if (!whole)
            A.part_lse[at] = lse2;
          else if (A.lse)
            A.lse[at] = lse2 * kLn2;
        }
      }
    }
  }
}

template <typename T, int DPL, int RW>
static int launch_tree_cores(const TreeArgs& A, cudaStream_t s) {
  constexpr int kRows = kTgWarps * RW;
  const size_t row = (size_t)A.d * sizeof(T);
  const size_t smem = sizeof(float) * kRows * ((size_t)A.d + kTgTile) +
                      kTgTile * (2 * row + kTgPad);
  if (!allow_smem<tree_generic_kernel<T, DPL, RW>>()) return DCP_ECUDA;
  const cudaError_t e = launch_chained(tree_generic_kernel<T, DPL, RW>, (unsigned)A.parts,
                                       kTgWarps * 32, smem, s, A);
  return e == cudaSuccess ? launch_status() : launch_status_report(e);
}

template <typename T, int DPL>
static int launch_tree_rows(const TreeArgs& A, cudaStream_t s) {
  return A.rows <= 16 ? launch_tree_cores<T, DPL, 2>(A, s) : launch_tree_cores<T, DPL, 4>(A, s);
}

template <typename T>
static int launch_tree_generic(const TreeArgs& A, cudaStream_t s) {
  if (A.d <= 64) return launch_tree_rows<T, 2>(A, s);
  if (A.d <= 128) return launch_tree_rows<T, 4>(A, s);
  return launch_tree_rows<T, 8>(A, s);
}

// ---------------------------------------------------------------------------
// merge of cut units, and of ranks that hold nothing
// ---------------------------------------------------------------------------

// W warps per output row (each takes every W-th part).  Rows whose unit lay in
// one run were written by its CTA; rows of refused requests and outside every
// request stay as they were.  Latency bounds it: a row waits for its entry, then
// for its parts, and a kernel this short also for its instructions, so there is
// one loop with a running maximum.  Few rows have many parts, which two warps
// fetch at once, eight at a time: a call of 8 nodes over 1500 tokens takes 15.9
// us, 16.1 with four warps, 16.5 with eight, 18.3 with one; 16 x 5 nodes on one
// key head 19.9, 20.4, 22.7 and 22.4 us, 64 nodes over 65536 tokens 71.5, 73.7,
// 80.3 and 72.2 (fp32, 2 x 11 nodes, 22.6, 21.5, 20.3 and 30.3).  Many rows get a
// warp each, which keeps more of them in flight: with 8 requests of 64 nodes
// (16384 rows) the call takes 153 us, 165 with two warps, 189 with four.  `joined`: the parts are joined already, only ranks that
// hold nothing are left.  A lane has DPL columns: consecutive ones where a row is
// 32 DPL wide (kWide), else every 32nd.
constexpr int64_t kTreeSplitRows = 2048;   // most rows that get two warps each

template <int DPL, bool kWide, int W>
__global__ void __launch_bounds__(256)
tree_merge_kernel(const __grid_constant__ TreeArgs A, bool joined) {
  constexpr int kFly = W > 1 ? 8 : 4;    // parts of a warp in flight at once
  constexpr int kRows = 8 / W;           // rows of a block
  __shared__ float s_acc[W > 1 ? 8 : 1][W > 1 ? 32 * DPL : 1], s_m[8], s_l[8];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int parts = __ldcg(A.hdr), extra = __ldcg(A.hdr + 4);
  const int64_t total = __ldcg(reinterpret_cast<const int64_t*>(A.hdr + 2));
  // blockIdx.x: (rank,) request; rows of it (node, head) by warps
  const int r = A.per_rank ? blockIdx.x / A.B : 0, b = blockIdx.x - r * A.B;
  const TreeEntry n = tree_load(A, A.per_rank ? b * A.L.dcp + r : b);
  const int mine = n.nodes * A.Hq;
  for (int i0 = blockIdx.y * kRows; i0 < mine; i0 += gridDim.y * kRows) {
    const int i = i0 + warp / W;
    const bool real = i < mine;
    const int j = i / A.Hq, h = i - j * A.Hq;
    const int64_t row = ((int64_t)r * A.N + n.q0 + j) * A.Hq + h;
    float* of = (float*)A.out + row * A.d;
    __nv_bfloat16* ob = (__nv_bfloat16*)A.out + row * A.d;
    if (n.units == 0) {   // a rank without tokens of this request
      if (real && warp % W == 0) {
        for (int c = lane; c < A.d; c += 32) of[c] = 0.f;
        if (lane == 0) A.lse[row] = -INFINITY;
      }
      continue;
    }
    if (joined) return;
    const int g = h / A.G, ur = j * A.G + h % A.G;   // row of the unit's request
    const int rb = ur / A.rows, rr = ur - rb * A.rows;
    const int64_t t0 = n.tile0 + (int64_t)(g * (n.units / A.Hkv) + rb) * (n.per + extra);
    int k0 = 0, k1 = 0;
    bool late = false;
    if (real) {
      k0 = tree_run_of(total, parts, t0);
      k1 = tree_run_of(total, parts, t0 + n.per - 1);
      late = tree_run(total, parts, k0) != t0;   // run k0 began before this unit
    }
    const bool cut = k0 != k1;
    const bool sunk = A.sink != nullptr && warp % W == 0;   // the sink counts once
    float M = sunk && cut ? __ldcg(A.sink + h) * kLog2e : -INFINITY;
    float L = M == -INFINITY ? 0.f : 1.f, acc[DPL];
#pragma unroll
    for (int y = 0; y < DPL; ++y) acc[y] = 0.f;
#pragma unroll 1
    for (int k = k0 + warp % W; cut && k <= k1; k += kFly * W) {
      float e[kFly], v[kFly][DPL];
#pragma unroll
      for (int x = 0; x < kFly; ++x) {
        e[x] = -INFINITY;
#pragma unroll
        for (int y = 0; y < DPL; ++y) v[x][y] = 0.f;
        const int kx = k + x * W;
        if (kx > k1) continue;
        const int64_t at = (int64_t)(2 * kx + (kx == k0 && late)) * A.rows + rr;
        e[x] = __ldcg(A.part_lse + at);
        const float* src = A.part_o + at * A.d;
        if (!kWide) {
#pragma unroll
          for (int y = 0; y < DPL; ++y)
            if (y * 32 < A.d) v[x][y] = __ldcg(src + y * 32 + lane);
        } else if (DPL == 2) {
          const float2 q = __ldcg((const float2*)(src + lane * 2));
          v[x][0] = q.x;
          v[x][1] = q.y;
        } else {
#pragma unroll
          for (int y = 0; y < DPL; y += 4) {
            const float4 q = __ldcg((const float4*)(src + lane * DPL + y));
            v[x][y] = q.x;
            v[x][y + 1] = q.y;
            v[x][(y + 2) % DPL] = q.z;
            v[x][(y + 3) % DPL] = q.w;
          }
        }
      }
      float top = M;
#pragma unroll
      for (int x = 0; x < kFly; ++x) top = fmaxf(top, e[x]);
      // the maximum stays -inf while no part saw anything: 0 would bury parts far below it
      const float base = top == -INFINITY ? 0.f : top;
      const float f = L == 0.f ? 0.f : exp2f(M - base);
      M = top;
      L *= f;
#pragma unroll
      for (int y = 0; y < DPL; ++y) acc[y] *= f;
#pragma unroll
      for (int x = 0; x < kFly; ++x) {
        // a part that saw nothing does not count, whatever its values are
        const float w = e[x] == -INFINITY ? 0.f : exp2f(e[x] - base);
        L += w;
        if (w != 0.f) {
#pragma unroll
          for (int y = 0; y < DPL; ++y) acc[y] = fmaf(w, v[x][y], acc[y]);
        }
      }
    }
    if (W > 1) {
      // the row's first warp joins what the others found, in their order
      __syncthreads();
      if (warp % W != 0) {
#pragma unroll
        for (int y = 0; y < DPL; ++y) s_acc[warp][y * 32 + lane] = acc[y];
        if (lane == 0) {
          s_m[warp] = M;
          s_l[warp] = L;
        }
      }
      __syncthreads();
      if (warp % W != 0) continue;
#pragma unroll
      for (int x = 1; x < W; ++x) {
        const float m2 = s_m[warp + x], l2 = s_l[warp + x];
        if (l2 == 0.f) continue;
        const float base = L == 0.f ? m2 : fmaxf(M, m2);
        const float f = L == 0.f ? 0.f : exp2f(M - base), w = exp2f(m2 - base);
        M = base;
        L = L * f + l2 * w;
#pragma unroll
        for (int y = 0; y < DPL; ++y) acc[y] = acc[y] * f + s_acc[warp + x][y * 32 + lane] * w;
      }
    }
    if (!cut) continue;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    if (kWide) {
#pragma unroll
      for (int y = 0; y < DPL; y += 2) {
        const int c = lane * DPL + y;
        if (A.out_dtype == DCP_F32)
          *(float2*)(of + c) = make_float2(acc[y] * inv, acc[y + 1] * inv);
        else
          *(uint32_t*)(ob + c) = pack_bf16(acc[y] * inv, acc[y + 1] * inv);
      }
    } else {
#pragma unroll
      for (int y = 0; y < DPL; ++y)
        if (y * 32 < A.d) {
          if (A.out_dtype == DCP_F32)
            of[y * 32 + lane] = acc[y] * inv;
          else
            ob[y * 32 + lane] = __float2bfloat16_rn(acc[y] * inv);
        }
    }
    if (lane == 0 && A.lse) A.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
  }
}

template <int DPL, bool kWide>
static cudaError_t launch_tree_merge(const TreeArgs& A, cudaStream_t s) {
  const int64_t rows = (int64_t)A.max_tree * A.Hq;       // of a request
  const unsigned x = (unsigned)A.B * (A.per_rank ? A.L.dcp : 1);
  const bool split = rows * x <= kTreeSplitRows;
  const int64_t y = (rows + (split ? 3 : 7)) / (split ? 4 : 8);
  const dim3 grid(x, (unsigned)(y < 8192 ? y : 8192));
  return split ? launch_chained(tree_merge_kernel<DPL, kWide, 2>, grid, 256, 0, s, A, A.join != 0)
               : launch_chained(tree_merge_kernel<DPL, kWide, 1>, grid, 256, 0, s, A, A.join != 0);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

// Query rows of a block (whole nodes), tokens of a tile and runs of the kernel
// for a call.  The tensor-core kernel takes one 128-row tile of queries where
// all nodes of a request fit it, else two.
struct TreeShape {
  int rows, chunk, tile, parts, extra;
};

static TreeShape tree_shape(bool tc, int G, int max_tree, int ranks) {
  if (!tc) {
    // blocks of 16 rows where they hold a request's, else of 32
    const int rows = max_tree * G <= 16 ? 16 : 32;
    return TreeShape{rows / G * G, kTgTile, kTgTile, 2 * num_sms(), 0};
  }
  const int nodes = 128 / G;
  // what a unit costs beside its tiles: a start and an end, and at each rank's
  // end a tile that is masked (32 requests x 16 nodes on 8 ranks over up to 65536
  // tokens: 488 us with 2 more, 467 with 10)
  return TreeShape{(max_tree <= nodes ? 1 : 2) * nodes * G, 16, 128, num_sms(), 2 + ranks};
}

static size_t tree_carve(TreeArgs* A, void* ws, int B, int dcp, int parts, int rows, int d) {
  const size_t E = (size_t)B * dcp;   // enough for both kinds of entries
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = (char*)ws + at;
    at += align_up(bytes, 256);
    return p;
  };
  char* hdr = take(32);
  char* en = take(sizeof(TreeEntry) * E);
  char* re = take(sizeof(int32_t) * (size_t)parts);
  char* ar = take(sizeof(int32_t) * (size_t)parts);
  char* pl = take(sizeof(float) * 2 * (size_t)parts * rows);
  char* po = take(sizeof(float) * 2 * (size_t)parts * rows * d);
  if (A) {
    A->hdr = (int32_t*)hdr;
    A->entry = (TreeEntry*)en;
    A->run_entry = (int32_t*)re;
    A->arrived = (int32_t*)ar;
    A->part_lse = (float*)pl;
    A->part_o = (float*)po;
  }
  return at;
}

static bool tree_shape_ok(const dcp_layout_t& L, int B, int max_tree, int Hq, int Hkv, int d,
                          dcp_dtype_t dtype) {
  return layout_ok(L) && B >= 0 && max_tree >= 1 && max_tree <= kTreeMaxNodes && Hq >= 1 &&
         Hkv >= 1 && Hq % Hkv == 0 && Hq / Hkv <= 16 && d >= 32 && d % 32 == 0 && d <= 256 &&
         (dtype == DCP_F32 || dtype == DCP_BF16);
}

static int tree_call(const dcp_layout_t& layout, const void* q, const int32_t* q_start, int N,
                     int B, int max_tree, int Hq, int Hkv, int d, float scale, dcp_dtype_t dtype,
                     const dcp_paged_kv_t& kv, const int32_t* ctx, const uint64_t* mask,
                     const float* sink, void* out, dcp_dtype_t out_dtype, float* lse,
                     bool per_rank, void* ws, size_t ws_bytes, int32_t* err, cudaStream_t s) {
  if (!tree_shape_ok(layout, B, max_tree, Hq, Hkv, d, dtype) || N < 0 || kv.num_blocks < 0 ||
      kv.max_vblocks < 0 || kv.bt_rank_stride < 0 || !(scale > 0.f) ||
      (out_dtype != DCP_F32 && out_dtype != DCP_BF16))
    return DCP_EINVAL;
  if (N == 0 || B == 0) return DCP_OK;
  if (!q || !q_start || !ctx || !mask || !out || (per_rank && !lse) || !kv.block_table ||
      !ranks_ok(kv.k, layout.dcp_size) || !ranks_ok(kv.v, layout.dcp_size))
    return DCP_EINVAL;
  if ((int64_t)B * layout.dcp_size * Hkv * 64 >= (int64_t(1) << 30) ||
      (int64_t)layout.block_size * layout.dcp_size >= (int64_t(1) << 31) ||
      (int64_t)kv.max_vblocks * layout.block_size * layout.dcp_size >= (int64_t(1) << 31) ||
      ((uintptr_t)q & 15) || ((uintptr_t)out & 15))
    return DCP_EUNSUPPORTED;
  for (int r = 0; r < layout.dcp_size; ++r)
    if (((uintptr_t)kv.k.ptr[r] & 15) || ((uintptr_t)kv.v.ptr[r] & 15)) return DCP_EUNSUPPORTED;
  const bool tc = tree_tc_supported(layout, d, dtype, kv, Hkv);
  const TreeShape S = tree_shape(tc, Hq / Hkv, max_tree, per_rank ? 1 : layout.dcp_size);
  TreeArgs A;
  A.q = q;
  A.q_start = q_start;
  A.ctx = ctx;
  A.mask = mask;
  A.N = N;
  A.B = B;
  A.Hq = Hq;
  A.Hkv = Hkv;
  A.G = Hq / Hkv;
  A.d = d;
  A.max_tree = max_tree;
  A.L = Layout{layout.dcp_size, layout.block_size, layout.interleave};
  A.per_rank = per_rank ? 1 : 0;
  A.rows = S.rows;
  A.chunk = S.chunk;
  A.tile = S.tile;
  A.parts = S.parts;
  A.extra = S.extra;
  // With at least as many units as runs a unit is cut into two or three parts,
  // which the last CTA to come joins in passing; with fewer it is cut into many,
  // and the merge's warps join them faster than one CTA would (GPU time, 32 x 16
  // nodes over up to 4096 tokens: 77 us against 79 and a launch less; 16 x 5
  // nodes on one key head: 45 us against 20).
  A.self = (per_rank ? (int64_t)B * layout.dcp_size : (int64_t)B) <= kTreeSelf ? 1 : 0;
  A.join = tc && !A.self && (int64_t)B * Hkv * (per_rank ? layout.dcp_size : 1) >= S.parts ? 1 : 0;
  A.sl2 = scale * kLog2e;
  A.k = kv.k;
  A.v = kv.v;
  A.bt = kv.block_table;
  A.max_vb = kv.max_vblocks;
  A.stride = kv.bt_rank_stride;
  A.nb = kv.num_blocks;
  A.sink = sink;
  A.out = out;
  A.out_dtype = out_dtype;
  A.lse = lse;
  A.err = err;
  const size_t need = tree_carve(&A, ws, B, layout.dcp_size, S.parts, S.rows, d);
  if (!ws || ws_bytes < need || ((uintptr_t)ws & 15)) return DCP_EWORKSPACE;
  // other CTAs read the queries, lists and masks until the end
  const int64_t rows = (per_rank ? layout.dcp_size : 1) * (int64_t)N * Hq;
  if (!apart({{out, rows * d * (out_dtype == DCP_F32 ? 4 : 2)}, {lse, rows * 4}, {ws, (int64_t)need}},
             {{q, (int64_t)N * Hq * d * (dtype == DCP_F32 ? 4 : 2)},
              {q_start, (int64_t)(B + 1) * 4},
              {ctx, (int64_t)B * 4},
              {mask, (int64_t)N * 8},
              {sink, (int64_t)Hq * 4},
              {kv.block_table,
               ((layout.dcp_size - 1) * kv.bt_rank_stride + (int64_t)B * kv.max_vblocks) * 4}}))
    return DCP_EINVAL;
  cudaError_t e = cudaSuccess;
  if (!A.self) e = launch_chained(tree_plan_kernel, 1, kTreePlanThreads, 0, s, A);
  if (e != cudaSuccess) return launch_status_report(e);
  const int rc = tc                 ? launch_tree_tc(A, s)
                 : dtype == DCP_F32 ? launch_tree_generic<float>(A, s)
                                    : launch_tree_generic<__nv_bfloat16>(A, s);
  if (rc != DCP_OK) return rc;
  if (A.join && !per_rank) return launch_status();   // nothing is left to merge
  if (d <= 64)
    e = d == 64 ? launch_tree_merge<2, true>(A, s) : launch_tree_merge<2, false>(A, s);
  else if (d <= 128)
    e = d == 128 ? launch_tree_merge<4, true>(A, s) : launch_tree_merge<4, false>(A, s);
  else
    e = d == 256 ? launch_tree_merge<8, true>(A, s) : launch_tree_merge<8, false>(A, s);
  if (e != cudaSuccess) return launch_status_report(e);
  return launch_status();
}

}  // namespace dcp

using namespace dcp;

extern "C" {

int dcp_tree_workspace_size(dcp_layout_t layout, int32_t num_reqs, int32_t max_tree,
                            int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                            dcp_dtype_t dtype, size_t* bytes) {
  if (!bytes || !tree_shape_ok(layout, num_reqs, max_tree, num_q_heads, num_kv_heads, head_dim,
                               dtype))
    return DCP_EINVAL;
  // a call on a cache too large for 32-bit rows takes the other kernel
  *bytes = 0;
  for (int tc = 0; tc <= (tree_tc_shape(head_dim, dtype, layout.block_size) ? 1 : 0); ++tc) {
    const TreeShape S = tree_shape(tc != 0, num_q_heads / num_kv_heads, max_tree, 1);
    const size_t n =
        tree_carve(nullptr, nullptr, num_reqs, layout.dcp_size, S.parts, S.rows, head_dim);
    if (n > *bytes) *bytes = n;
  }
  return DCP_OK;
}

int dcp_tree_partial_gqa(dcp_layout_t layout, const void* q, const int32_t* q_start,
                         int32_t num_tokens, int32_t num_reqs, int32_t max_tree,
                         int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, float scale,
                         dcp_dtype_t dtype, dcp_paged_kv_t kv, const int32_t* ctx_lens,
                         const uint64_t* tree_mask, float* part_o, float* part_lse,
                         void* workspace, size_t workspace_bytes, int32_t* err_count,
                         dcp_stream_t stream) {
  dcp::NvtxRange nvtx_range("dcp_tree_partial_gqa");
  return tree_call(layout, q, q_start, num_tokens, num_reqs, max_tree, num_q_heads, num_kv_heads,
                   head_dim, scale, dtype, kv, ctx_lens, tree_mask, nullptr, part_o, DCP_F32,
                   part_lse, true, workspace, workspace_bytes, err_count, (cudaStream_t)stream);
}

int dcp_tree_decode_gqa(dcp_layout_t layout, const void* q, const int32_t* q_start,
                        int32_t num_tokens, int32_t num_reqs, int32_t max_tree,
                        int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, float scale,
                        dcp_dtype_t dtype, dcp_paged_kv_t kv, const int32_t* ctx_lens,
                        const uint64_t* tree_mask, const float* sink, void* out,
                        dcp_dtype_t out_dtype, float* out_lse, void* workspace,
                        size_t workspace_bytes, int32_t* err_count, dcp_stream_t stream) {
  dcp::NvtxRange nvtx_range("dcp_tree_decode_gqa");
  return tree_call(layout, q, q_start, num_tokens, num_reqs, max_tree, num_q_heads, num_kv_heads,
                   head_dim, scale, dtype, kv, ctx_lens, tree_mask, sink, out, out_dtype, out_lse,
                   false, workspace, workspace_bytes, err_count, (cudaStream_t)stream);
}

}  // extern "C"
