// Scored decode attention: one query per request over the sharded paged cache
// in 16, 32 or 8 bits, with scores that may be capped, biased by distance, or
// limited to a window, the document's first tokens and the document.  This
// file has the kernel for any type and shape, the choice between units whole in a
// cluster and units cut anywhere, the merge of the latter, and the entry points; dcp_scored_mma.cu has the tensor-core kernel.
//
// With L tokens, the query at position L - 1, and x the position of a key:
//     t = scale q.k;  t = cap tanh(t / cap);  t = t - slope[h] (L - 1 - x)
//     lse = ln( sum_seen e^t + e^sink ),  o = sum_seen e^(t - lse) v.
#include <math.h>
#include <algorithm>

#include "dcp_q8.cuh"
#include "dcp_scored.cuh"

namespace dcp {

// ---------------------------------------------------------------------------
// any type and shape
// ---------------------------------------------------------------------------

// Four values of a cache row in 32 bits.
template <int kKind>
struct Four;
template <>
struct Four<kCacheF32> {
  using Raw = float4;
  static constexpr int kBytes = 16;
  static __device__ __forceinline__ float4 of(Raw x) { return x; }
};
template <>
struct Four<kCacheBf16> {
  using Raw = uint2;
  static constexpr int kBytes = 8;
  static __device__ __forceinline__ float4 of(Raw x) {
    return make_float4(bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y));
  }
};
template <>
struct Four<kCacheE4m3> {
  using Raw = uint32_t;
  static constexpr int kBytes = 4;
  static __device__ __forceinline__ float4 of(Raw x) { return e4m3x4_f32(x); }
};

// CTAs that run at once, by their registers (the kernel's launch bounds).
constexpr int generic_per_sm(int di) { return di == 8 ? 2 : di == 4 ? 3 : 4; }

// Eight lanes take a token, so a warp takes four at a time; HP heads of the unit
// in one pass over the tokens.  The products run in fp32 on the CUDA cores.  The
// heads' sums over the lanes are exchanged so that each lane gets one head's
// score, which it forms alone, and the weights go round again: with every score
// formed by all eight lanes two requests of up to 2048 tokens, 32/8 heads of 128 in
// fp32, took 40 us, not 26 (by the line both; in clusters 22).  Bound by its instructions and few warps an SM.
template <int kKind, int DI, int HP>
__global__ void __launch_bounds__(kScoredWarps * 32, generic_per_sm(DI))
scored_generic_kernel(const __grid_constant__ ScoredArgs A, bool q_bf16) {
  using F = Four<kKind>;
  using Raw = typename F::Raw;
  __shared__ __align__(16) float s_q[HP][DI * 32];
  constexpr int kParts = kScoredWarps * 4;   // sums of their own: four tokens of each warp
  __shared__ __align__(16) float4 s_o[kParts][HP][DI * 8];
  __shared__ float s_m[kParts][HP], s_l[kParts][HP];
  __shared__ float s_unit[kParts];   // what a part's values are held in units of
  griddep_wait();                // launched chained: the preceding kernel completed
  __shared__ int s_before[kScoredWarps * 32];
  __shared__ float s_lse[HP];
  const int chunk = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sub = lane & 7, grp = lane >> 3;
  const int di = A.d / 32;
  Piece at;
  int t1 = 0;
  if (A.unit_ctas) {   // a part of one unit, perhaps an empty one
    const int u = chunk / A.unit_ctas, rank = chunk % A.unit_ctas;
    at.e = u / A.Hkv, at.g = u % A.Hkv;
    at.n = entry_tiles_by_warp(A, at.e, rank == 0 && at.g == 0 && warp == 0);
    at.k0 = (int)((int64_t)at.n * rank / A.unit_ctas);
    at.k1 = (int)((int64_t)at.n * (rank + 1) / A.unit_ctas);
    at.t = 0;
  } else {
    const Line line = plan_line<kScoredWarps * 32>(A, chunk, s_before);
    if (chunk == 0) keep_line<kScoredWarps * 32>(A, line, s_before);
    at.t = (int)min((int64_t)line.each * chunk, (int64_t)line.all);
    t1 = (int)min((int64_t)at.t + line.each, (int64_t)line.all);
    seek_entry<kScoredWarps * 32>(A, line, s_before, at.t, at.e, at.start);
  }
  for (bool more = A.unit_ctas || at.t < t1; more; more = at.t < t1) {
    if (!A.unit_ctas) at = piece_at(A, at.t, t1, at.e, at.start);
    const int e = at.e, g = at.g, k0 = at.k0, k1 = at.k1, n = at.n;
    const int b = A.apart ? e % A.B : e, r0 = A.apart ? e / A.B : 0;
    const int r1 = A.apart ? r0 + 1 : A.S.dcp;
    const Seen seen = seen_of(A, b, false);
    const int last = __ldg(A.lens + b) - 1;
    PieceOut P;
    P.whole = A.unit_ctas ? A.unit_ctas == 1 : k0 == 0 && k1 == n;
    P.slot = chunk + (int64_t)e * A.Hkv + g;
    P.row = (int64_t)e * A.Hq + g * A.G;
    for (int h0 = 0; h0 < A.G; h0 += HP) {
      __syncthreads();
      for (int i = tid; i < HP * A.d; i += kScoredWarps * 32) {
        const int hh = i / A.d, c = i - hh * A.d;
        const int64_t at = ((int64_t)b * A.Hq + g * A.G + h0 + hh) * A.d + c;
        s_q[hh][c] = h0 + hh >= A.G ? 0.f
                     : q_bf16 ? __bfloat162float(((const __nv_bfloat16*)A.q)[at])
                              : ((const float*)A.q)[at];
      }
      __syncthreads();
      const int own = sub & (HP - 1);   // this lane's head
      const float slope =
          A.slopes && h0 + own < A.G ? __ldg(A.slopes + g * A.G + h0 + own) : 0.f;
      float m = kNone, l = 0.f;
      // 8-bit values are summed in units of the largest power of two of a scale so far: a sum of
      // values near the largest numbers would leave 32 bits, and so would small ones' weights
      float unit = 0x1p-126f, per_unit = 0x1p126f;
      float4 o[HP][DI];
#pragma unroll
      for (int h = 0; h < HP; ++h)
#pragma unroll
        for (int i = 0; i < DI; ++i) o[h][i] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = k0 + warp; k < k1; k += kScoredWarps) {
        // the k-th tile: rank by rank, first the kept tokens and then the window
        int r = r0, left = k, p0 = 0, lo = 0, hi = 0;
        for (; r < r1; ++r) {
          const RankTokens T = seen.on(A.S, r);
          const int na = T.a_tiles(), nb = T.b_tiles();
          if (left < na) {
            p0 = (T.a0 / kRows + left) * kRows, lo = T.a0, hi = T.a1;
            break;
          }
          left -= na;
          if (left < nb) {
            p0 = (T.b0 / kRows + left) * kRows, lo = T.b0, hi = T.b1;
            break;
          }
          left -= nb;
        }
        // a token's page in each lane (twice); then the tokens four at a time, each asked for
        // before the one in front of it is used
        const int mine = p0 + (lane & (kRows - 1));
        const int my_vb = A.S.by_bs.div(mine), my_loc = mine - my_vb * A.S.bs;
        int64_t my_ph = -1;
        float2 my_sc = make_float2(1.f, 1.f);
        if (mine >= lo && mine < hi) {
          if (my_vb < A.max_vb)
            my_ph = __ldg(A.bt + r * A.bt_stride + (int64_t)b * A.max_vb + my_vb);
          if (my_ph < 0 || my_ph >= A.nb) {
            my_ph = -1;
            if (lane < kRows && h0 == 0) count_error(A.err);
          } else {
            my_ph = my_ph * A.Hkv + g;
            if (kKind == kCacheE4m3)
              my_sc = __ldg(reinterpret_cast<const float2*>(A.sc.ptr[r]) + my_ph * 2);
          }
        }
        const float my_far = (float)(last - A.S.position(my_vb, r, my_loc));
        Raw kn[DI], vn[DI];
        bool ok_next = false;
        auto ask = [&](int i) {
          const int64_t ph = __shfl_sync(0xffffffffu, my_ph, i + grp);
          const int loc = __shfl_sync(0xffffffffu, my_loc, i + grp);
          const int64_t at = (ph * A.S.bs + loc) * A.d;
          const Raw* kr = (const Raw*)((const char*)A.k.ptr[r] + at / 4 * F::kBytes) + sub;
          const Raw* vr = (const Raw*)((const char*)A.v.ptr[r] + at / 4 * F::kBytes) + sub;
          ok_next = ph >= 0;
#pragma unroll
          for (int j = 0; j < DI; ++j) {
            if (ok_next && j < di) {
              kn[j] = __ldg(kr + 8 * j);
              vn[j] = __ldg(vr + 8 * j);
            }
          }
        };
        ask(0);
#pragma unroll 1
        for (int i0 = 0; i0 < kRows; i0 += 4) {
          const bool ok = ok_next;
          const float ks = __shfl_sync(0xffffffffu, my_sc.x, i0 + grp);
          const float vs = __shfl_sync(0xffffffffu, my_sc.y, i0 + grp);
          const float far = __shfl_sync(0xffffffffu, my_far, i0 + grp);
          float4 kk[DI], vv[DI];
#pragma unroll
          for (int i = 0; i < DI; ++i) {
            kk[i] = vv[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (ok && i < di) {
              kk[i] = F::of(kn[i]);
              vv[i] = F::of(vn[i]);
            }
          }
          if (i0 + 4 < kRows) ask(i0 + 4);
          float dot[HP];
#pragma unroll
          for (int h = 0; h < HP; ++h) {
            dot[h] = 0.f;
#pragma unroll
            for (int i = 0; i < DI; ++i) {
              if (i < di) {
                const float4 q4 = *reinterpret_cast<const float4*>(&s_q[h][(sub + 8 * i) * 4]);
                dot[h] = fmaf(q4.x, kk[i].x, dot[h]);
                dot[h] = fmaf(q4.y, kk[i].y, dot[h]);
                dot[h] = fmaf(q4.z, kk[i].z, dot[h]);
                dot[h] = fmaf(q4.w, kk[i].w, dot[h]);
              }
            }
          }
          // the sum over the eight lanes of head `own`: two neighbours share out the heads by
          // pairs, then pairs of lanes by twos
#pragma unroll
          for (int step = 1; step < HP; step *= 2) {
            const bool up = sub & step;
#pragma unroll
            for (int h = 0; h < HP / (2 * step); ++h) {
              const float give = up ? dot[2 * h] : dot[2 * h + 1];
              dot[h] = (up ? dot[2 * h + 1] : dot[2 * h]) + __shfl_xor_sync(0xffffffffu, give, step);
            }
          }
#pragma unroll
          for (int step = HP; step < 8; step *= 2) dot[0] += __shfl_xor_sync(0xffffffffu, dot[0], step);
          const float x = ok ? formed(A, dot[0] * ks * A.scale, slope, far) : -INFINITY;
          const bool over = x - m > kSlack;
          const bool larger = kKind == kCacheE4m3 && ok && vs >= 2.f * unit;
          if (__any_sync(0xffffffffu, over || larger)) {
            float down = over ? exp2f(m - x) : 1.f;
            if (over) m = x;
            l *= down;
            if (larger) {
              const int e = __float_as_int(vs) & 0x7f800000;   // its power of two
              per_unit = __int_as_float(e == 0x7f000000 ? 0x00400000 : 0x7f000000 - e);
              down *= unit * per_unit;
              unit = __int_as_float(e);
            }
#pragma unroll
            for (int h = 0; h < HP; ++h) {
              const float d = __shfl_sync(0xffffffffu, down, (lane & 24) | h);
#pragma unroll
              for (int i = 0; i < DI; ++i) {
                o[h][i].x *= d;
                o[h][i].y *= d;
                o[h][i].z *= d;
                o[h][i].w *= d;
              }
            }
          }
          const float w = exp2f(x - m);
          l += w;
          const float wv = kKind == kCacheE4m3 ? w * (vs * per_unit) : w;
#pragma unroll
          for (int h = 0; h < HP; ++h) {
            const float wh = __shfl_sync(0xffffffffu, wv, (lane & 24) | h);
#pragma unroll
            for (int i = 0; i < DI; ++i) {
              o[h][i].x = fmaf(wh, vv[i].x, o[h][i].x);
              o[h][i].y = fmaf(wh, vv[i].y, o[h][i].y);
              o[h][i].z = fmaf(wh, vv[i].z, o[h][i].z);
              o[h][i].w = fmaf(wh, vv[i].w, o[h][i].w);
            }
          }
        }
      }
      // the sums against a common reference
      const int part = warp * 4 + grp;
#pragma unroll
      for (int h = 0; h < HP; ++h)
#pragma unroll
        for (int i = 0; i < DI; ++i)
          if (i < di) s_o[part][h][sub + 8 * i] = o[h][i];
      if (sub == 0) s_unit[part] = kKind == kCacheE4m3 ? unit : 1.f;
      if (sub < HP) {
        s_m[part][sub] = m;
        s_l[part][sub] = l;
      }
      __syncthreads();
      if (tid < HP && h0 + tid < A.G) {   // a head's sums become the parts' factors
        float M = kNone, Ls = 0.f;
        for (int p = 0; p < kParts; ++p) M = fmaxf(M, s_m[p][tid]);
        for (int p = 0; p < kParts; ++p)   // nothing seen: no part (a sum that is NaN has one)
          if (s_l[p][tid] != 0.f) Ls = fmaf(s_l[p][tid], exp2f(s_m[p][tid] - M), Ls);
        const bool any = Ls != 0.f;
        float weight = 1.f, lse = any ? (M + log2f(Ls)) * kLn2 : -INFINITY;
        if (P.whole) lse = with_sink(A.sink, g * A.G + h0 + tid, lse, weight);
        if (A.unit_ctas > 1)
          s_lse[tid] = lse;   // for the cluster
        else
          put_lse(A, P, h0 + tid, lse);
        for (int p = 0; p < kParts; ++p)
          s_l[p][tid] = any && s_l[p][tid] != 0.f ? exp2f(s_m[p][tid] - M) / Ls * weight : 0.f;
      }
      __syncthreads();
      const int quads = A.d / 4;
      for (int i = tid; i < HP * quads; i += kScoredWarps * 32) {
        const int hh = i / quads, c = i - hh * quads;
        if (h0 + hh >= A.G) break;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int p = 0; p < kParts; ++p) {
          const float f = s_l[p][hh], unit_p = s_unit[p];
          const float4 v4 = s_o[p][hh][c];
          y.x = fmaf(f * v4.x, unit_p, y.x);
          y.y = fmaf(f * v4.y, unit_p, y.y);
          y.z = fmaf(f * v4.z, unit_p, y.z);
          y.w = fmaf(f * v4.w, unit_p, y.w);
        }
        if (A.unit_ctas > 1)
          s_o[0][hh][c] = y;   // for the cluster, over what only it has read
        else
          put_four(A, P, (h0 + hh) * quads + c, y);
      }
      if (A.unit_ctas > 1) {
        __syncwarp();
        cluster_sync();
        join_cluster(A, e, g, h0, min(HP, A.G - h0), quads, s_lse, 1, &s_o[0][0][0], DI * 8);
        __syncwarp();
        cluster_sync();   // all have read what is in this CTA
      }
    }
  }
}

// ---------------------------------------------------------------------------
// merge
// ---------------------------------------------------------------------------

constexpr int kMergeThreads = 512;
constexpr int kMergeAhead = 4;     // rows a thread asks for at a time
constexpr int kMergeKept = 64;     // parts whose weights are kept

// A CTA joins the parts of one unit, in the order of its tiles: the heads' LSE
// and the parts' weights first, a head a warp, while the first rows are on their
// way; then each thread four values of a head, the parts shared out to groups of
// threads that are summed in their order.  Units that one CTA of the main kernel
// had whole are done already; units without a tile get zeros here.  Bound by two
// dependent loads and the launch: 3 us for 12 parts of 4 heads of 128.
__global__ void __launch_bounds__(kMergeThreads)
scored_merge_kernel(const __grid_constant__ ScoredArgs A) {
  __shared__ float s_lse[16], s_keep[16], s_weight[16][kMergeKept];
  __shared__ __align__(16) float4 s_acc[kMergeThreads];
  griddep_wait();
  griddep_launch_dependents();   // the next call's first kernel may start its launch
  const int u = blockIdx.x, e = u / A.Hkv, g = u - e * A.Hkv, tid = threadIdx.x;
  const int before = A.before[e], n = A.before[e + 1] - before;
  const uint32_t each = A.before[A.entries() + 1];
  const uint32_t t0 = before * A.Hkv + g * n, i0 = t0 / each;
  const int parts = n ? (int)((t0 + n - 1) / each - i0) + 1 : 0;
  if (parts == 1) return;
  const int64_t slot = (int64_t)i0 + u;
  const int lane = tid & 31, warp = tid >> 5;
  const int quads = A.d / 4, cols = A.G * quads;
  const int groups = max(kMergeThreads / cols, 1);
  const int grp = min(tid / cols, groups);   // the last threads may have no group
  const int c_first = tid - grp * cols;
  const float4* const po = reinterpret_cast<const float4*>(A.part_o + slot * A.G * A.d);
  float4 y[kMergeAhead];
  auto ask = [&](int i, int c) {
#pragma unroll
    for (int j = 0; j < kMergeAhead; ++j)
      if (i + j * groups < parts) y[j] = po[(int64_t)(i + j * groups) * cols + c];
  };
  if (grp < groups && c_first < cols) ask(grp, c_first);
  for (int hh = warp; hh < A.G; hh += kMergeThreads / 32) {
    const float* pl = A.part_lse + slot * A.G + hh;
    const float x0 = lane < parts ? pl[(int64_t)lane * A.G] : -INFINITY;
    const float x1 = lane + 32 < parts ? pl[(int64_t)(lane + 32) * A.G] : -INFINITY;
    float m = fmaxf(x0, x1);
    for (int i = lane + 64; i < parts; i += 32) m = fmaxf(m, pl[(int64_t)i * A.G]);
    m = warp_max(m);
    auto weigh = [&](float x, float ref) { return x == -INFINITY ? 0.f : expf(x - ref); };
    float s = weigh(x0, m) + weigh(x1, m);
    for (int i = lane + 64; i < parts; i += 32) s += weigh(pl[(int64_t)i * A.G], m);
    s = warp_sum(s);
    float keep, lse = s == 0.f ? -INFINITY : m + logf(s);
    const float all = with_sink(A.sink, g * A.G + hh, lse, keep);
    s_weight[hh][lane] = weigh(x0, lse) * keep;
    s_weight[hh][lane + 32] = weigh(x1, lse) * keep;
    if (lane == 0) {
      s_lse[hh] = lse;
      s_keep[hh] = keep;
      if (A.out_lse) A.out_lse[(int64_t)e * A.Hq + g * A.G + hh] = all;
    }
  }
  __syncthreads();
  for (int c0 = 0; c0 < cols; c0 += kMergeThreads) {
    const int c = c0 + c_first;
    const bool mine = grp < groups && c < cols;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const int hh = mine ? c / quads : 0;
    if (mine) {
      for (int i = grp; i < parts; i += kMergeAhead * groups) {
        if (c0 > 0 || i > grp) ask(i, c);
#pragma unroll
        for (int j = 0; j < kMergeAhead; ++j) {
          const int p = i + j * groups;
          if (p >= parts) continue;
          float w;
          if (p < kMergeKept) {
            w = s_weight[hh][p];
          } else {
            const float x = A.part_lse[(slot + p) * A.G + hh];
            w = x == -INFINITY ? 0.f : expf(x - s_lse[hh]) * s_keep[hh];
          }
          if (w == 0.f) continue;   // a part that saw nothing
          acc.x = fmaf(w, y[j].x, acc.x);
          acc.y = fmaf(w, y[j].y, acc.y);
          acc.z = fmaf(w, y[j].z, acc.z);
          acc.w = fmaf(w, y[j].w, acc.w);
        }
      }
    }
    if (groups > 1) {
      s_acc[tid] = acc;
      __syncthreads();
      if (tid < cols)
        for (int j = 1; j < groups; ++j) {
          const float4 z = s_acc[tid + j * cols];
          acc.x += z.x, acc.y += z.y, acc.z += z.z, acc.w += z.w;
        }
    }
    if (mine && grp == 0) {
      const int64_t at = (int64_t)e * A.Hq * quads + (int64_t)g * cols + c;
      if (A.out_dtype == DCP_F32)
        reinterpret_cast<float4*>(A.out)[at] = acc;
      else
        reinterpret_cast<uint2*>(A.out)[at] =
            make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
    }
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

static int generic_ctas(int d) { return num_sms() * generic_per_sm(d <= 64 ? 2 : d <= 128 ? 4 : 8); }

// Heads of a pass over the tokens: 8 values a lane of 2 heads fit into registers.
constexpr int heads_a_pass(int d, int G) { return G == 1 ? 1 : d <= 128 ? 4 : 2; }

// The kernel's variants, each with what the host asks of it.
template <int kKind, int DI, int HP>
struct Generic {
  static constexpr auto kKernel = scored_generic_kernel<kKind, DI, HP>;
  static constexpr unsigned kBlock = kScoredWarps * 32;

  static int clusters(int ctas) { return clusters_at_once<kKernel>(ctas, 0, kBlock, 0); }

  static int launch(const ScoredArgs& A, bool q_bf16, cudaStream_t s) {
    const cudaError_t e = launch_scored<kKernel>(A, kBlock, 0, s, A, q_bf16);
    return e == cudaSuccess ? launch_status() : launch_status_report(e);
  }
};

// `use` of the variant that a call takes.
template <int kKind, class Use>
static int with_generic(const ScoredArgs& A, Use&& use) {
  if (A.d <= 64)
    return A.G == 1 ? use(Generic<kKind, 2, 1>()) : use(Generic<kKind, 2, heads_a_pass(64, 2)>());
  if (A.d <= 128)
    return A.G == 1 ? use(Generic<kKind, 4, 1>()) : use(Generic<kKind, 4, heads_a_pass(128, 2)>());
  return A.G == 1 ? use(Generic<kKind, 8, 1>()) : use(Generic<kKind, 8, heads_a_pass(256, 2)>());
}
template <class Use>
static int with_generic(const ScoredArgs& A, CacheKind kind, Use&& use) {
  return kind == kCacheF32    ? with_generic<kCacheF32>(A, use)
         : kind == kCacheBf16 ? with_generic<kCacheBf16>(A, use)
                              : with_generic<kCacheE4m3>(A, use);
}

static bool shape_ok(const dcp_layout_t& L, int B, int Hq, int Hkv, int d) {
  return shards_ok(L) && B >= 0 && Hq >= 1 && Hkv >= 1 && Hq % Hkv == 0 && Hq / Hkv <= 16 &&
         d >= 32 && d % 32 == 0 && d <= 256;
}

static size_t before_bytes(int64_t entries) { return align_up((size_t)(entries + 2) * 4, 256); }

// CTAs of a unit where that is better than cutting the line, else 0.  A unit whole in a
// cluster needs no plan and no second kernel; its warps go through more rounds of tiles (one
// tile a warp) than those of an even cut of the line.  How long requests are is not known here:
// the table is a bound, the line evens out requests of unlike lengths, and a cluster waits for
// the longest.  So the line is counted as if all requests but one filled half of the table, and
// with a round more where chunks may end a unit and begin the next.  What its plan, second launch
// and merge are worth in rounds is by sweeps of both ways over 3208 calls with full tables or
// with mixed lengths (all caches, 1 to 16 heads a unit, heads of 64 to 256, 1 to 32 requests of 64
// to 48000 tokens) and 1860 with tables that are full, half full, full to a quarter or to a
// sixteenth: on the tensor cores 10, and one for each round of the merge's loads, as few units
// leave it many parts; on CUDA cores 3 of 64 dims in one pass of heads.  Where the table is full
// less would be better, where it is nearly empty more:
//   8 bits, two requests, 16/1 heads of 128, table for 24000: of 24000 tokens 28.9 us in clusters
//     and 38.0 by the line, of 1500 11.6 and 16.3;
//   bf16, 16 requests, 16/1 heads of 64, table for 9000: of 9000 19.8 and 18.2, of 4500 13.5 and 16.7;
//   8 bits, one, 32/8 heads: of 24000 in a table for as many 27.3 and 20.1 (the line is taken);
//   fp32, two, 8/2 heads of 64, table for 3000: of 3000 13.4 and 12.9, of 1500 11.3 and 16.5.
// Of the cluster sizes that run at once the smallest that leaves a warp 3 tiles at most (CUDA
// cores 1.5), else the largest: of 8 bits, 32/8 heads, 400 tokens take 6.9 us in eight CTAs and 7.6
// in sixteen, 3000 tokens 10.1 and 9.2.
// `wave` CTAs run at once; `tiles` are the most of a unit.
template <class AtOnce>
static int unit_ctas_of(const ScoredArgs& A, bool mma, int64_t wave, int64_t units, int64_t tiles,
                        AtOnce&& at_once) {
  auto rounds = [](int64_t n, int64_t at_a_time) { return (n + at_a_time - 1) / at_a_time; };
  int c = kUnitCtas;
  while (c > 1 && (2 * tiles <= (mma ? 6 : 3) * kScoredWarps * (c / 2) || at_once(c) < units)) c /= 2;
  if (at_once(c) < units) return 0;
  // tiles of a chunk of the line
  int64_t each = rounds(rounds(tiles * units * (A.B + 1), 2 * (int64_t)A.B), wave);
  if (each < A.least) each = A.least;
  const int64_t more =
      rounds(tiles, (int64_t)kScoredWarps * c) - rounds(each, kScoredWarps) - (units > 1);
  if (!mma) {
    const int hp = heads_a_pass(A.d, A.G), passes = (A.G + hp - 1) / hp;
    return more * passes * A.d <= 3 * 64 ? c : 0;
  }
  // the merge: parts of a unit, of which `groups` times kMergeAhead come at a time
  const int cols = A.G * A.d / 4, groups = cols < kMergeThreads ? kMergeThreads / cols : 1;
  const double loads = (double)rounds(tiles, each) / (groups * kMergeAhead);
  return more <= 10. + loads ? c : 0;
}

// Chunks of a call at most: one for each CTA that runs at once.
static int most_chunks(int d, int G) {
  int most = generic_ctas(d);
  for (CacheKind kind : {kCacheBf16, kCacheE4m3}) {
    const int n = scored_mma_wave(d, G, kind);
    if (n > most) most = n;
  }
  return most;
}

static size_t workspace_bytes_of(int64_t entries, int Hq, int Hkv, int d) {
  const int G = Hq / Hkv;
  const size_t rows = (size_t)(most_chunks(d, G) + entries * Hkv) * G;
  return before_bytes(entries) + align_up(rows * 4, 256) + rows * d * 4;
}

struct Cache {
  dcp_rank_ptrs_t k, v, sc;
  int64_t nb;
  const int32_t* bt;
  int32_t max_vb;
  int64_t bt_stride;
  CacheKind kind;
};

static bool aligned16(const dcp_rank_ptrs_t& p, int dcp) {
  for (int r = 0; r < dcp; ++r)
    if ((uintptr_t)p.ptr[r] & 15) return false;
  return true;
}

static int scored_call(const dcp_layout_t& layout, const void* q, int B, int Hq, int Hkv, int d,
                       float scale, dcp_dtype_t dtype, const Cache& kv, const int32_t* seq_lens,
                       const dcp_scores_t& f, const float* sink, bool apart_, void* out,
                       dcp_dtype_t out_dtype, float* out_lse, void* ws, size_t ws_bytes,
                       int32_t* err, cudaStream_t s) {
  if (!shape_ok(layout, B, Hq, Hkv, d) || (dtype != DCP_F32 && dtype != DCP_BF16) ||
      (out_dtype != DCP_F32 && out_dtype != DCP_BF16) || kv.nb < 0 || kv.max_vb < 0 ||
      kv.bt_stride < 0 || !isfinite(scale) || !(f.cap == 0.f || isnormal(f.cap)) ||
      f.cap < 0.f || f.window < 0 || f.prefix < 0)
    return DCP_EINVAL;
  if (B == 0) return DCP_OK;
  const int dcp = layout.dcp_size;
  const bool scaled = kv.kind == kCacheE4m3;
  if (!q || !seq_lens || !out || (apart_ && !out_lse) || !kv.bt || !ranks_ok(kv.k, dcp) ||
      !ranks_ok(kv.v, dcp) || (scaled && !ranks_ok(kv.sc, dcp)))
    return DCP_EINVAL;
  const int64_t entries = apart_ ? (int64_t)B * dcp : B;
  if (entries * Hkv >= (int64_t(1) << 30) ||
      (uintptr_t)q % 16 || (uintptr_t)out % 16 || (uintptr_t)ws % 16 || !aligned16(kv.k, dcp) ||
      !aligned16(kv.v, dcp) || (scaled && !aligned16(kv.sc, dcp)))
    return DCP_EUNSUPPORTED;
  // the most tiles a full table can have: a rank's first and last of each of two runs may be part
  const int64_t room = (int64_t)kv.max_vb * layout.block_size * dcp;
  const int64_t tiles = (room / kRows + 4 * dcp) * B * Hkv;
  // a rank's tokens and a tile's rest fit in 31 bits (and `tiles`, then, in 64)
  if (room > INT32_MAX - 256 || tiles >= (int64_t(1) << 30)) return DCP_EUNSUPPORTED;
  const size_t need = workspace_bytes_of(entries, Hq, Hkv, d);
  if (!ws || ws_bytes < need) return DCP_EWORKSPACE;
  const int64_t es = dtype == DCP_F32 ? 4 : 2, os = out_dtype == DCP_F32 ? 4 : 2;
  const Bytes reads[] = {{q, (int64_t)B * Hq * d * es},
                         {seq_lens, (int64_t)B * 4},
                         {f.slopes, (int64_t)Hq * 4},
                         {f.first, (int64_t)B * 4},
                         {sink, (int64_t)Hq * 4},
                         {kv.bt, ((kv.bt_stride ? dcp - 1 : 0) * kv.bt_stride +
                                  (int64_t)B * kv.max_vb) * 4}};
  const Bytes writes[] = {{out, entries * Hq * d * os},
                          {out_lse, entries * Hq * 4},
                          {ws, (int64_t)need},
                          {err, 4}};
  const int64_t unit = scaled ? 1 : es, pool = kv.nb * Hkv * layout.block_size * d * unit;
  for (const Bytes& w : writes) {
    for (const Bytes& r : reads)
      if (overlap(w, r)) return DCP_EINVAL;
    for (const Bytes& x : writes)
      if (&x != &w && overlap(w, x)) return DCP_EINVAL;
    for (int r = 0; r < dcp; ++r)
      if (overlap(w, {kv.k.ptr[r], pool}) || overlap(w, {kv.v.ptr[r], pool}) ||
          (scaled && overlap(w, {kv.sc.ptr[r], kv.nb * Hkv * 16})))
        return DCP_EINVAL;
  }
  ScoredArgs A;
  memset((void*)&A, 0, sizeof(A));
  A.S = Shards(layout);
  A.B = B, A.Hq = Hq, A.Hkv = Hkv, A.G = Hq / Hkv, A.d = d;
  A.apart = apart_;
  A.q = q;
  A.scale = scale;
  A.cap = f.cap;
  A.inv_cap = f.cap > 0.f ? 1.f / f.cap : 0.f;
  A.window = f.window, A.prefix = f.prefix, A.slopes = f.slopes, A.first = f.first;
  A.lens = seq_lens;
  A.sink = sink;
  A.bt = kv.bt, A.max_vb = kv.max_vb, A.bt_stride = kv.bt_stride, A.nb = kv.nb;
  A.k = kv.k, A.v = kv.v, A.sc = kv.sc;
  A.out = out, A.out_dtype = out_dtype, A.out_lse = out_lse, A.err = err;
  char* w = (char*)ws;
  A.before = (int32_t*)w;
  w += before_bytes(entries);
  const bool mma = scored_mma_ok(A, kv.kind, dtype == DCP_BF16);
  A.least = (mma ? 2 : 1) * kScoredWarps;
  // no more chunks than a full table has
  const int64_t useful = (tiles + A.least - 1) / A.least;
  const int wave = mma ? scored_mma_wave(d, A.G, kv.kind) : generic_ctas(d);
  A.ctas = (int64_t)wave > useful ? (useful > 0 ? (int)useful : 1) : wave;
  // the most tiles of a unit, by the table and by the window: a rank's last may be part, of a
  // window its first too, and both of kept tokens.  (Where documents start is not known here: a
  // call is cut as if they started at 0.)
  const int64_t kept = f.window > 0 ? (int64_t)f.window + f.prefix : room;
  const int64_t tokens = kept < room ? kept : room;
  const int ends = f.window <= 0 ? 1 : f.prefix > 0 ? 4 : 2;
  const int64_t per_rank = (tokens / dcp + 2 * layout.interleave) / kRows + ends;
  // a rank's part of the table, and a tile for each token, bound them too
  const int64_t held = ((int64_t)kv.max_vb * layout.block_size + kRows - 1) / kRows;
  int64_t most = apart_ ? per_rank : tokens / kRows + ends * dcp;
  most = std::min({most, apart_ ? held : held * dcp, tokens});
  A.unit_ctas = unit_ctas_of(A, mma, wave, entries * Hkv, most, [&](int ctas) {
    return mma ? scored_mma_clusters(A, kv.kind, ctas)
               : with_generic(A, kv.kind, [&](auto v) { return v.clusters(ctas); });
  });
  if (A.unit_ctas) A.ctas = (int)(entries * Hkv) * A.unit_ctas;
  A.part_lse = (float*)w;
  w += align_up((size_t)(A.ctas + entries * Hkv) * A.G * 4, 256);
  A.part_o = (float*)w;
  int rc = DCP_OK;
  if (mma) {
    rc = launch_scored_mma(A, kv.kind, s);
  } else {
    rc = with_generic(A, kv.kind, [&](auto v) { return v.launch(A, dtype == DCP_BF16, s); });
  }
  if (rc) return rc;
  if (A.unit_ctas) return launch_status();
  const cudaError_t e = launch_chained(scored_merge_kernel, (unsigned)(entries * Hkv),
                                       kMergeThreads, 0, s, A);
  if (e != cudaSuccess) return launch_status_report(e);
  return launch_status();
}

static Cache cache_of(const dcp_paged_kv_t& kv, dcp_dtype_t dtype) {
  Cache c = {kv.k, kv.v, {}, kv.num_blocks, kv.block_table, kv.max_vblocks, kv.bt_rank_stride,
             dtype == DCP_F32 ? kCacheF32 : kCacheBf16};
  return c;
}

static Cache cache_of(const dcp_paged_kv8_t& kv) {
  Cache c = {kv.k, kv.v, kv.scale, kv.num_blocks, kv.block_table, kv.max_vblocks,
             kv.bt_rank_stride, kCacheE4m3};
  return c;
}

}  // namespace dcp

using namespace dcp;

extern "C" {

int dcp_scored_workspace_size(dcp_layout_t layout, int32_t num_reqs, int32_t num_q_heads,
                              int32_t num_kv_heads, int32_t head_dim, int32_t per_rank,
                              size_t* bytes) {
  if (!bytes || !shape_ok(layout, num_reqs, num_q_heads, num_kv_heads, head_dim))
    return DCP_EINVAL;
  *bytes = workspace_bytes_of(per_rank ? (int64_t)num_reqs * layout.dcp_size : num_reqs,
                              num_q_heads, num_kv_heads, head_dim);
  return DCP_OK;
}

int dcp_scored_decode_gqa(dcp_layout_t layout, const void* q, int32_t num_reqs,
                          int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, float scale,
                          dcp_dtype_t dtype, dcp_paged_kv_t kv, const int32_t* seq_lens,
                          dcp_scores_t scores, const float* sink, void* out, dcp_dtype_t out_dtype,
                          float* out_lse, void* workspace, size_t workspace_bytes,
                          int32_t* err_count, dcp_stream_t stream) {
  dcp::NvtxRange nvtx_range("dcp_scored_decode_gqa");
  return scored_call(layout, q, num_reqs, num_q_heads, num_kv_heads, head_dim, scale, dtype,
                     cache_of(kv, dtype), seq_lens, scores, sink, false, out, out_dtype, out_lse,
                     workspace, workspace_bytes, err_count, (cudaStream_t)stream);
}

int dcp_scored_partial_gqa(dcp_layout_t layout, const void* q, int32_t num_reqs,
                           int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, float scale,
                           dcp_dtype_t dtype, dcp_paged_kv_t kv, const int32_t* seq_lens,
                           dcp_scores_t scores, float* part_o, float* part_lse, void* workspace,
                           size_t workspace_bytes, int32_t* err_count, dcp_stream_t stream) {
  dcp::NvtxRange nvtx_range("dcp_scored_partial_gqa");
  return scored_call(layout, q, num_reqs, num_q_heads, num_kv_heads, head_dim, scale, dtype,
                     cache_of(kv, dtype), seq_lens, scores, nullptr, true, part_o, DCP_F32,
                     part_lse, workspace, workspace_bytes, err_count, (cudaStream_t)stream);
}

int dcp_q8_decode_gqa(dcp_layout_t layout, const void* q, int32_t num_reqs, int32_t num_q_heads,
                      int32_t num_kv_heads, int32_t head_dim, float scale, dcp_dtype_t dtype,
                      dcp_paged_kv8_t kv, const int32_t* seq_lens, dcp_scores_t scores,
                      const float* sink, void* out, dcp_dtype_t out_dtype, float* out_lse,
                      void* workspace, size_t workspace_bytes, int32_t* err_count,
                      dcp_stream_t stream) {
  dcp::NvtxRange nvtx_range("dcp_q8_decode_gqa");
  return scored_call(layout, q, num_reqs, num_q_heads, num_kv_heads, head_dim, scale, dtype,
                     cache_of(kv), seq_lens, scores, sink, false, out, out_dtype, out_lse,
                     workspace, workspace_bytes, err_count, (cudaStream_t)stream);
}

int dcp_q8_partial_gqa(dcp_layout_t layout, const void* q, int32_t num_reqs, int32_t num_q_heads,
                       int32_t num_kv_heads, int32_t head_dim, float scale, dcp_dtype_t dtype,
                       dcp_paged_kv8_t kv, const int32_t* seq_lens, dcp_scores_t scores,
                       float* part_o, float* part_lse, void* workspace, size_t workspace_bytes,
                       int32_t* err_count, dcp_stream_t stream) {
  dcp::NvtxRange nvtx_range("dcp_q8_partial_gqa");
  return scored_call(layout, q, num_reqs, num_q_heads, num_kv_heads, head_dim, scale, dtype,
                     cache_of(kv), seq_lens, scores, nullptr, true, part_o, DCP_F32, part_lse,
                     workspace, workspace_bytes, err_count, (cudaStream_t)stream);
}

}  // extern "C"
