// Scored decode attention on the tensor cores, over bf16 and e4m3 caches.
//
// A unit has up to 16 query heads and any number of tokens, so a product's
// 16-row side is the tokens and its 8-column side the heads (mma.sync
// m16n8k16; one or two column tiles of heads):
//     S^T [16 tokens x 8 heads] = K Q^T,   O^T [16 dims x 8 heads] += V^T P^T.
// With tcgen05 the heads would fill a fraction of its smallest tile, and e4m3
// operands would need the other one in 8 bits too.  The calls are bound by the
// bytes of the cache; what has to stay below that is the instructions a byte.
//
// e4m3 numbers become fp16, which holds them exactly.  The query is fp16 too,
// scaled by a power of two for each head so that its largest entry is near 2^14:
// bf16's eight bits fit down to 2^-31 of the largest; smaller entries lose bits
// of theirs (fp16's last step is 2^-24 of one, 2^-38 of the largest), and what is
// below half of that step becomes 0.
// The page's scale of the keys goes to the score, that of the values to the
// weight (below).  Products accumulate in fp32; scores, their maxima and sums
// are fp32.
#include <string.h>

#include "dcp_q8.cuh"
#include "dcp_scored.cuh"

namespace dcp {

struct ScoredMaps {
  CUtensorMap k[DCP_MAX_RANKS], v[DCP_MAX_RANKS];
};

__device__ __forceinline__ void mma_f16_16816(float* c, const uint32_t* a, uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An 8 x 8 tile of 16-bit numbers, transposed across the warp.
__device__ __forceinline__ uint32_t transposed8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool E8>
__device__ __forceinline__ void mma_16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if (E8)
    mma_f16_16816(c, a, b0, b1);
  else
    mma_bf16_16816(c, a, b0, b1);
}

// Sizes of a variant: D dims, e4m3 or bf16, NT tiles of eight heads.
template <int D, bool E8, int NT>
struct Shape {
  static constexpr int kRowBytes = D * (E8 ? 1 : 2);
  static constexpr int kTileBytes = kRows * kRowBytes;       // of keys, and of values
  static constexpr int kBoxBytes = kRowBytes < 128 ? kRowBytes : 128;
  static constexpr int kBoxes = kRowBytes / kBoxBytes;
  // 16 KB a warp on their way: with 12 or 8 KB 524288 tokens in 8 bits take 193 or 201 us, not 190
  static constexpr int kStages = 16384 / (2 * kTileBytes);
  static constexpr int kPerSm = NT == 1 ? 3 : 2;
  static constexpr int kRing = kScoredWarps * kStages * 2 * kTileBytes;
  static constexpr int kMeta = kScoredWarps * kStages * (16 + 16 + 8 + 8);
  static __host__ __device__ constexpr int smem(int G) {
    return 1024 + kRing + kMeta + kScoredWarps * G * (D + 4) * 4;
  }
  // Byte of 16-byte chunk c of a row, as the copies' swizzle lays it.
  static __device__ __forceinline__ uint32_t at(int row, int c) {
    if (kBoxBytes == 64) return row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
    return (c >> 3) * (kRows * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
  }
  // The same for chunk 2 i + c from that of chunk c < 2.
  static __device__ __forceinline__ uint32_t on(uint32_t first, int i) {
    return (first ^ ((2 * i & 7) << 4)) + (2 * i >> 3) * (kRows * 128);
  }
};

constexpr float kLift = 11.f;    // fp16 weights are held times 2^11: up to 2^15 with the slack, and
                                 // in full precision down to 2^-25
constexpr int kScoredStuck = 1 << 20;   // err_count increment for a wait that timed out

// Four warps a CTA use tiles, each every fourth one of the CTA's chunk from a ring
// of its own; a fifth looks the tiles up, 32 at a time and one in each lane, and
// fills the rings by TMA, a lane for each, over the ends of pieces.  (Each warp
// filling its own ring had a quarter of its instructions for that, and what
// bounded the kernel was the length of a warp's chain of instructions.)
constexpr int kScoredThreads = (kScoredWarps + 1) * 32;

__device__ __forceinline__ void sync_users() {   // the warps that use tiles
  asm volatile("bar.sync 1, %0;" ::"n"(kScoredWarps * 32) : "memory");
}

template <int D, bool E8, int NT, bool kFormed>
__global__ void __launch_bounds__(kScoredThreads, Shape<D, E8, NT>::kPerSm)
scored_mma_kernel(const __grid_constant__ ScoredArgs A, const __grid_constant__ ScoredMaps maps) {
  using Z = Shape<D, E8, NT>;
  constexpr int ST = Z::kStages, TB = Z::kTileBytes, KS = D / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int NS = kScoredWarps * ST;   // stages: tile k of the chunk has stage k % NS
  const uint32_t ring = smem_u32(smem);
  float* const s_scale = reinterpret_cast<float*>(smem + Z::kRing);
  int4* const s_desc = reinterpret_cast<int4*>(smem + Z::kRing + NS * 16);
  const uint32_t full = smem_u32(smem + Z::kRing + NS * 32), empty = full + NS * 8;
  float* const s_ml = reinterpret_cast<float*>(smem + Z::kRing + Z::kMeta);   // [G][warps][4]
  float* const s_o = s_ml + kScoredWarps * A.G * 4;                          // [warps][G][D]
  __shared__ int s_before[kScoredThreads];
  if (tid < NS) {
    mbar_init(full + 8 * tid, 1);
    mbar_init(empty + 8 * tid, 1);
    fence_mbar_init();
  }
  if (tid < A.S.dcp) {
    prefetch_tmap(&maps.k[tid]);
    prefetch_tmap(&maps.v[tid]);
  }
  __syncthreads();
  griddep_wait();                // launched chained: the preceding kernel completed
  const int chunk = blockIdx.x;
  int t0, t1, e0, start0, n0 = 0;
  const int rank = A.unit_ctas ? chunk % A.unit_ctas : 0;
  if (A.unit_ctas) {   // a part of one unit, on a line of this entry alone
    const int u = chunk / A.unit_ctas, g = u % A.Hkv;
    e0 = u / A.Hkv;
    n0 = entry_tiles_by_warp(A, e0, rank == 0 && g == 0 && warp == 0);
    t0 = g * n0 + (int)((int64_t)n0 * rank / A.unit_ctas);
    t1 = g * n0 + (int)((int64_t)n0 * (rank + 1) / A.unit_ctas);
    start0 = 0;
  } else {
    const Line line = plan_line<kScoredThreads>(A, chunk, s_before);
    t0 = (int)min((int64_t)line.each * chunk, (int64_t)line.all);
    t1 = (int)min((int64_t)t0 + line.each, (int64_t)line.all);
    if (chunk == 0) keep_line<kScoredThreads>(A, line, s_before);
    seek_entry<kScoredThreads>(A, line, s_before, t0, e0, start0);
  }

  if (warp == kScoredWarps) {
    // --- the warp that fills the rings ---
    const uint64_t pol = policy_evict_first();
    int we = e0, wstart = start0;
    int d_row, d_ph, d_info, d_p0;   // this lane's tile
    auto look_up = [&](int t) {
      bool todo = t < t1;
      d_row = -1, d_ph = d_info = d_p0 = 0;
      const int R = A.apart ? 1 : A.S.dcp;
      for (;;) {   // entry by entry, a rank's tokens in each lane
        const int b = A.apart ? we % A.B : we, r0 = A.apart ? we / A.B : 0;
        RankTokens T = seen_of(A, b, false).on(A.S, r0 + min(lane, R - 1));
        const int na = T.a_tiles();
        int upto = lane < R ? na + T.b_tiles() : 0;
#pragma unroll
        for (int o = 1; o < DCP_MAX_RANKS; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += x;
        }
        const int n = __shfl_sync(0xffffffffu, upto, R - 1);
        const bool here = todo && t - wstart < n * A.Hkv;
        int g = 0, left = 0;
        if (here) {
          g = (int)((uint32_t)(t - wstart) / (uint32_t)n);
          left = t - wstart - g * n;
        }
        int r = 0;
        for (int x = 0; x < R - 1; ++x) r += left >= __shfl_sync(0xffffffffu, upto, x);
        const int up_r = __shfl_sync(0xffffffffu, upto, r), na_r = __shfl_sync(0xffffffffu, na, r);
        const int a0 = __shfl_sync(0xffffffffu, T.a0, r), a1 = __shfl_sync(0xffffffffu, T.a1, r);
        const int b0 = __shfl_sync(0xffffffffu, T.b0, r), b1 = __shfl_sync(0xffffffffu, T.b1, r);
        if (here) {   // first the kept tokens, then the window
          const int nb_r = (b1 + kRows - 1) / kRows - b0 / kRows;
          const int k = left - (up_r - na_r - (b1 > b0 ? nb_r : 0));
          const bool kept = k < na_r;
          const int lo = kept ? a0 : b0, hi = kept ? a1 : b1;
          d_p0 = ((lo / kRows) + k - (kept ? 0 : na_r)) * kRows;
          const int vb = A.S.by_bs.div(d_p0);
          r += r0;
          int64_t page = -1;
          if (vb < A.max_vb)
            page = __ldg(A.bt + r * A.bt_stride + (int64_t)b * A.max_vb + vb);
          d_info = max(lo - d_p0, 0) | min(hi - d_p0, kRows) << 8 | r << 16;
          if (page >= 0 && page < A.nb) {
            d_ph = (int)(page * A.Hkv + g);
            d_row = d_ph * A.S.bs + (d_p0 - vb * A.S.bs);
          }
          todo = false;
        }
        if (!__any_sync(0xffffffffu, todo) || we + 1 >= A.entries()) break;
        wstart += n * A.Hkv;
        ++we;
      }
    };
    int st = lane & 3, turn = 0;   // this lane's next stage, and how often it was filled
    bool dead = false;             // a wait timed out: fill no more
    for (int k0 = t0; k0 < t1; k0 += 32) {
      look_up(k0 + lane);
      for (int i = 0; i < 32 && k0 + i < t1; i += kScoredWarps) {
        const int from = i + (lane & 3);
        const int row = __shfl_sync(0xffffffffu, d_row, from);
        const int ph = __shfl_sync(0xffffffffu, d_ph, from);
        const int info = __shfl_sync(0xffffffffu, d_info, from);
        const int p0 = __shfl_sync(0xffffffffu, d_p0, from);
        if (lane < kScoredWarps && k0 + from < t1 && !dead) {
          const uint32_t bar = full + 8 * st, dst = ring + st * 2 * TB;
          const int r = info >> 16;
          dead = turn > 0 && !mbar_wait(empty + 8 * st, (turn - 1) & 1);
          if (!dead) {
            s_desc[st] = make_int4(row, info, p0, 0);
            if (row >= 0) {
              mbar_arrive_expect_tx(bar, 2 * TB + (E8 ? 16 : 0));
#pragma unroll
              for (int x = 0; x < Z::kBoxes; ++x) {
                tma_load_2d_hint(dst + x * kRows * 128, &maps.k[r], x * 128, row, bar, pol);
                tma_load_2d_hint(dst + TB + x * kRows * 128, &maps.v[r], x * 128, row, bar, pol);
              }
              if (E8)
                bulk_load(smem_u32(s_scale + st * 4), (const char*)A.sc.ptr[r] + (int64_t)ph * 16,
                          16, bar);
            } else {
              count_error(A.err);
              mbar_arrive(bar);
            }
          } else if (A.err) {
            atomicAdd(A.err, kScoredStuck);
          }
          st += kScoredWarps;
          if (st >= NS) {
            st -= NS;
            ++turn;
          }
        }
        __syncwarp();
      }
    }
    if (A.unit_ctas > 1) {   // as the others
      cluster_sync();
      cluster_sync();
    }
    griddep_launch_dependents();   // as below
    return;
  }

  // --- the warps that use them ---
  const int gq = lane >> 2, tq = lane & 3;
  // what this lane gives ldmatrix of a tile's keys and of its values: the rows of the four
  // 8 x 8 tiles are tokens 0-7 and 8-15 of one chunk and of the next
  const int mi = lane >> 3;
  const uint32_t k_at = Z::at((mi & 1) * 8 + (lane & 7), mi >> 1);
  const uint32_t v_at = E8 ? k_at : Z::at((mi >> 1) * 8 + (lane & 7), mi & 1);
  bool dead = false;   // a wait timed out: wait no more
  // queries as the B operand: what they are in memory, asked for ahead, of head gq (+ 8);
  // in 8 bits in the order of a row of keys in its fragments, dims 4 tq .. 4 tq + 3 of each 16
  uint32_t qb[NT][KS][2];
  auto ask_queries = [&](const Piece& p) {
    const int b = A.apart ? p.e % A.B : p.e;
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      const bool there = gq + 8 * x < A.G;
      const __nv_bfloat16* qh =
          (const __nv_bfloat16*)A.q + ((int64_t)b * A.Hq + p.g * A.G + gq + 8 * x) * D;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        if (E8) {
          const uint2 w = there ? __ldg(reinterpret_cast<const uint2*>(qh + ks * 16 + tq * 4))
                                : make_uint2(0u, 0u);
          qb[x][ks][0] = w.x;
          qb[x][ks][1] = w.y;
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qb[x][ks][i] =
                there ? __ldg(reinterpret_cast<const uint32_t*>(qh + ks * 16 + i * 8 + tq * 2)) : 0u;
        }
      }
    }
  };
  int st = warp, phase = 0;
  Piece at;
  if (t0 < t1) {
    at = A.unit_ctas ? piece_of(A, t0, t1, e0, start0, n0) : piece_at(A, t0, t1, e0, start0);
    ask_queries(at);
  }
  int used = t0 + warp;   // this warp's next tile
  for (bool more = t0 < t1; more;) {
    const int e = at.e, g = at.g, k0 = at.k0, k1 = at.k1, n = at.n;
    const int upto = at.t;
    int last = 0;
    if (kFormed) last = __ldg(A.lens + (A.apart ? e % A.B : e)) - 1;

    // of heads 2 tq, 2 tq + 1 (+ 8) what a product is to be multiplied by
    float mul[NT][2], slope[NT][2];
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      float up = 1.f;
      if (E8) {
        float top = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
          top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16_lo(qb[x][ks][0])), fabsf(bf16_hi(qb[x][ks][0]))),
                                 fmaxf(fabsf(bf16_lo(qb[x][ks][1])), fabsf(bf16_hi(qb[x][ks][1])))));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^(14 - exponent of the largest); beside an infinity the others stay finite; all 0 or NaN: 1
        const int ex = (__float_as_int(top) >> 23) - 127;
        if (top > 0.f) up = __int_as_float((min(14 - ex, 126) + 127) << 23);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qb[x][ks][i] = pack_f16(bf16_lo(qb[x][ks][i]) * up, bf16_hi(qb[x][ks][i]) * up);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int h = 2 * tq + i + 8 * x;
        mul[x][i] = kFormed ? A.scale : A.scale * kLog2e;
        if (E8) mul[x][i] /= __shfl_sync(0xffffffffu, up, (2 * tq + i) * 4);
        slope[x][i] = kFormed && A.slopes && h < A.G ? __ldg(A.slopes + g * A.G + h) : 0.f;
      }
    }
    // references: of the scores (ref) and, in 8 bits, of scores and the values' scales together
    // (the score vref and the scale 2^vlift, apart: their sum would lose the scale beside a
    // score beyond 2^24)
    float o[NT][KS][4], l[NT][2], ref[NT][2], vref[NT][2], vlift[NT][2];
#pragma unroll
    for (int x = 0; x < NT; ++x) {
#pragma unroll
      for (int i = 0; i < KS; ++i) o[x][i][0] = o[x][i][1] = o[x][i][2] = o[x][i][3] = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[x][i] = vlift[x][i] = 0.f;
        ref[x][i] = vref[x][i] = kNone;
      }
    }

    for (; used < upto; used += kScoredWarps) {
      if (!dead && !mbar_wait(full + 8 * st, phase)) {
        dead = true;
        if (lane == 0 && A.err) atomicAdd(A.err, kScoredStuck);
      }
      dead = __any_sync(0xffffffffu, dead);
      const int4 desc = s_desc[st];
      if (!dead && desc.x >= 0) {
        const uint32_t kb = ring + st * 2 * TB, vb = kb + TB;
        const int lo = desc.y & 255, hi = (desc.y >> 8) & 255;
        float ks_ = 1.f, vlog = 0.f;   // the keys' scale, and log2 of the values'
        if (E8) {
          const float2 both = *reinterpret_cast<const float2*>(s_scale + st * 4);
          ks_ = both.x;
          const int bits = __float_as_int(both.y), mant = bits & 0x7fffff;
          vlog = (float)((bits >> 23) - 127);     // exact for a power of two
          if ((uint32_t)bits - 0x00800000u >= 0x7f000000u)   // below 2^-126 (of 0 -inf, a weight of
            vlog = log2f(both.y * 0x1p24f) - 24.f;           // nothing), or no scale: NaN or inf
          else if (mant)
            vlog += log2f(__int_as_float(mant | 0x3f800000));
        }
        const bool edge = lo > 0 || hi < kRows;
        if (edge) {   // values that do not count are zeros, so 0 * NaN is not met
          for (int i = lane; i < kRows * (Z::kRowBytes / 16); i += 32) {
            const int row = i / (Z::kRowBytes / 16), c = i % (Z::kRowBytes / 16);
            if (row < lo || row >= hi)
              asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(vb + Z::at(row, c)), "r"(0u)
                           : "memory");
          }
          fence_proxy_async_smem();   // before the next tile is copied over them
          __syncwarp();
        }
        // S^T = K Q^T, in two chains of products
        float s[NT][4], s2[NT][4];
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[x][i] = s2[x][i] = 0.f;
        {
          if (E8) {
#pragma unroll
            for (int i = 0; i < KS / 2; ++i) {
              uint32_t r[4];
              ldsm_x4(Z::on(kb + k_at, i), r[0], r[1], r[2], r[3]);
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                uint32_t a[4];
                e4m3x4_f16(r[2 * c], a[0], a[2]);
                e4m3x4_f16(r[2 * c + 1], a[1], a[3]);
#pragma unroll
                for (int x = 0; x < NT; ++x)
                  mma_16816<E8>(c ? s2[x] : s[x], a, qb[x][2 * i + c][0], qb[x][2 * i + c][1]);
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < KS; ++i) {
              uint32_t a[4];
              ldsm_x4(Z::on(kb + k_at, i), a[0], a[1], a[2], a[3]);
#pragma unroll
              for (int x = 0; x < NT; ++x)
                mma_16816<E8>(i & 1 ? s2[x] : s[x], a, qb[x][i][0], qb[x][i][1]);
            }
          }
        }
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[x][i] += s2[x][i];
        // scores in base 2, of tokens gq (two heads) and gq + 8
        if (kFormed) {
          float far[2] = {0.f, 0.f};
          if (A.slopes) {
            const int r = desc.y >> 16, p = desc.z + gq, page = A.S.by_bs.div(p);
            far[0] = (float)(last - A.S.position(page, r, p - page * A.S.bs));
            far[1] = (float)(last - A.S.position(page, r, p + 8 - page * A.S.bs));
          }
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              s[x][i] = formed(A, s[x][i] * (mul[x][i & 1] * ks_), slope[x][i & 1], far[i >> 1]);
        } else {
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[x][i] *= mul[x][i & 1] * ks_;
        }
        if (edge) {
          const bool in[2] = {gq >= lo && gq < hi, gq + 8 >= lo && gq + 8 < hi};
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[x][i] = in[i >> 1] ? s[x][i] : -INFINITY;
        }
        bool over = false;
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float m = fmaxf(s[x][h], s[x][h + 2]);
            over |= m - ref[x][h] > kSlack;
            if (E8) over |= m - vref[x][h] > kSlack - vlog + vlift[x][h];
          }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float m = fmaxf(s[x][h], s[x][h + 2]);
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
              float down = 1.f;
              if (m - ref[x][h] > kSlack) {   // never for a tile that sees nothing
                down = ex2_ftz(ref[x][h] - m);
                l[x][h] *= down;
                ref[x][h] = m;
              }
              if (E8) {
                down = 1.f;
                if (m - vref[x][h] > kSlack - vlog + vlift[x][h]) {
                  down = ex2_ftz((vref[x][h] - m) + (vlift[x][h] - vlog));
                  vref[x][h] = m;
                  vlift[x][h] = vlog;
                }
              }
#pragma unroll
              for (int i = 0; i < KS; ++i) {
                o[x][i][h] *= down;
                o[x][i][h + 2] *= down;
              }
            }
        }
        // weights, and as the B operand of P V: of 8 bits in fp16, which is off by 2^-11 of each
        // at most, an eighth of an output's rounding to bf16 (two terms would cost 1.5%: 32
        // requests of up to 65536 tokens 194.9 us, not 192).  In bf16 they would be off by 2^-8, as
        // much as the output, so there they are the sum of two numbers, to 2^-15: the upper half
        // of the 32 bits, and the rest rounded.  The rest is made larger by 2^-24 of the weight,
        // so that it is not 0, which beside a value of infinity would give NaN.  A second product
        // a tile costs nothing beside the bytes (a window of 4096 tokens, 32 requests, 90.2 us
        // with either, bias over whole contexts 74.0).
        uint32_t pb[NT][2], pl[NT][2];
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          float p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int h = i & 1;
            p[i] = ex2_ftz(s[x][i] - ref[x][h]);
            l[x][h] += p[i];
            if (E8) p[i] = ex2_ftz((s[x][i] - vref[x][h]) + (vlog - vlift[x][h] + kLift));
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float p0 = p[2 * i], p1 = p[2 * i + 1];
            if (E8) {
              pb[x][i] = transposed8(pack_f16(p0, p1));
            } else {
              const uint32_t hi = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
              pb[x][i] = transposed8(hi);
              pl[x][i] = transposed8(pack_bf16(fmaf(p0, 0x1p-24f, p0 - bf16_lo(hi)),
                                               fmaf(p1, 0x1p-24f, p1 - bf16_hi(hi))));
            }
          }
        }
        // O^T += V^T P^T.  In 8 bits row j of a tile of 16 dims is dim 2 j, row 8 + j dim 2 j + 1.
        if (E8) {
#pragma unroll
          for (int i = 0; i < KS / 2; ++i) {
            uint32_t r[4];
            ldsm_x4_t(Z::on(vb + v_at, i), r[0], r[1], r[2], r[3]);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              // bytes (token, dim) 00 01 10 11 -> 00 10 01 11
              uint32_t a[4];
              e4m3x4_f16(__byte_perm(r[2 * c], 0, 0x3120), a[0], a[1]);
              e4m3x4_f16(__byte_perm(r[2 * c + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
              for (int x = 0; x < NT; ++x) mma_16816<E8>(o[x][2 * i + c], a, pb[x][0], pb[x][1]);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            uint32_t a[4];
            ldsm_x4_t(Z::on(vb + v_at, i), a[0], a[1], a[2], a[3]);
#pragma unroll
            for (int x = 0; x < NT; ++x) {
              mma_16816<E8>(o[x][i], a, pb[x][0], pb[x][1]);
              mma_16816<E8>(o[x][i], a, pl[x][0], pl[x][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8 * st);
      st += kScoredWarps;
      if (st >= NS) {
        st -= NS;
        phase ^= 1;
      }
    }

    // the next piece, and its queries on their way
    PieceOut P;
    P.whole = A.unit_ctas ? A.unit_ctas == 1 : k0 == 0 && k1 == n;
    P.slot = chunk + (int64_t)e * A.Hkv + g;
    P.row = (int64_t)e * A.Hq + g * A.G;
    more = at.t < t1;
    if (more) {
      at = piece_at(A, at.t, t1, e, at.start);
      ask_queries(at);
    }

    // --- the piece's result: the warps' sums against a common reference ---
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float sum = l[x][h];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int hh = 2 * tq + h + 8 * x;
        if (hh >= A.G) continue;
        if (gq == 0)
          *reinterpret_cast<float4*>(s_ml + (hh * kScoredWarps + warp) * 4) =
              E8 ? make_float4(ref[x][h], sum, vref[x][h], vlift[x][h])
                 : make_float4(ref[x][h], sum, ref[x][h], 0.f);
        float* os = s_o + (warp * A.G + hh) * D;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          if (E8) {
            *reinterpret_cast<float2*>(os + i * 16 + 2 * gq) = make_float2(o[x][i][h], o[x][i][h + 2]);
          } else {
            os[i * 16 + gq] = o[x][i][h];
            os[i * 16 + gq + 8] = o[x][i][h + 2];
          }
        }
      }
    sync_users();
    // a head's four numbers of each warp become its four factors, and one for all that is
    // multiplied first: in one product the lift and a long request's sum would take a values'
    // scale of 2^-110 out of 32 bits.  The factors are held times 2^-kSlack, as a score may
    // pass its reference by that beside a scale of 2^127.
    if (tid < A.G) {
      float4* const ml = reinterpret_cast<float4*>(s_ml) + tid * kScoredWarps;
      float M = kNone, Ls = 0.f;
      float4 w[kScoredWarps];
#pragma unroll
      for (int i = 0; i < kScoredWarps; ++i) {
        w[i] = ml[i];
        M = fmaxf(M, w[i].x);
      }
#pragma unroll
      for (int i = 0; i < kScoredWarps; ++i)   // nothing seen: no part (a sum that is NaN has one)
        if (w[i].y != 0.f) Ls = fmaf(w[i].y, ex2_ftz(w[i].x - M), Ls);
      const bool any = Ls != 0.f;
      float weight = 1.f, lse = any ? (M + log2f(Ls)) * kLn2 : -INFINITY;
      if (P.whole) lse = with_sink(A.sink, g * A.G + tid, lse, weight);
      if (A.unit_ctas > 1)
        s_ml[tid * kScoredWarps * 4 + kScoredWarps] = lse;   // for the cluster
      else
        put_lse(A, P, tid, lse);
      float* const to = reinterpret_cast<float*>(ml);
#pragma unroll
      for (int i = 0; i < kScoredWarps; ++i)
        to[i] = any && w[i].y != 0.f ? exp2f((w[i].z - M) + (w[i].w - kSlack)) : 0.f;
      to[kScoredWarps + 1] = any ? exp2f(kSlack - (E8 ? kLift : 0.f)) / Ls * weight : 0.f;
    }
    sync_users();
    for (int i = tid; i < A.G * (D / 4); i += kScoredWarps * 32) {
      const float* const of_head = s_ml + i / (D / 4) * kScoredWarps * 4;
      const float4 f = *reinterpret_cast<const float4*>(of_head);
      const float all = of_head[kScoredWarps + 1];
      const float4* os = reinterpret_cast<const float4*>(s_o) + i;
      const float fs[4] = {f.x, f.y, f.z, f.w};
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kScoredWarps; ++w) {
        const float4 x = os[w * A.G * (D / 4)];
        y.x = fmaf(x.x * all, fs[w], y.x);
        y.y = fmaf(x.y * all, fs[w], y.y);
        y.z = fmaf(x.z * all, fs[w], y.z);
        y.w = fmaf(x.w * all, fs[w], y.w);
      }
      if (A.unit_ctas > 1)
        reinterpret_cast<float4*>(s_o)[i] = y;   // for the cluster, over what only it has read
      else
        put_four(A, P, i, y);
    }
    sync_users();
  }
  if (A.unit_ctas > 1) {
    // --- the cluster's results joined, each CTA a share of the columns ---
    const int g = chunk / A.unit_ctas % A.Hkv;
    if (t0 == t1 && tid < A.G) s_ml[tid * kScoredWarps * 4 + kScoredWarps] = -INFINITY;
    __syncwarp();
    cluster_sync();
    join_cluster(A, e0, g, 0, A.G, D / 4, s_ml + kScoredWarps, kScoredWarps * 4,
                 reinterpret_cast<const float4*>(s_o), D / 4);
    __syncwarp();
    cluster_sync();   // all have read what is in this CTA
  } else if (A.unit_ctas == 1 && t0 == t1) {   // nothing is seen
    PieceOut P;
    P.whole = true;
    P.slot = 0;
    const int g = chunk % A.Hkv;
    P.row = (int64_t)e0 * A.Hq + g * A.G;
    for (int i = tid; i < A.G * (D / 4); i += kScoredWarps * 32)
      put_four(A, P, i, make_float4(0.f, 0.f, 0.f, 0.f));
    float weight;
    if (tid < A.G) put_lse(A, P, tid, with_sink(A.sink, g * A.G + tid, -INFINITY, weight));
  }
  // Only now may the merge start its launch, and only after its wait the next
  // call: 32 requests called in a row take 204 us each so, 315 where both kernels
  // say so at their start (the next call's CTAs come in beside the merge's).
  griddep_launch_dependents();
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

// bf16 queries, heads of 64 or 128, pages of whole tiles, and rows that a
// tensor map's coordinate can name; anything else runs on the CUDA cores.
bool scored_mma_ok(const ScoredArgs& A, CacheKind kind, bool q_bf16) {
  return kind != kCacheF32 && q_bf16 && (A.d == 64 || A.d == 128) && A.S.bs % kRows == 0 &&
         A.nb * A.Hkv * A.S.bs < (int64_t(1) << 31) && tensor_map_encoder() != nullptr;
}

// Bytes of rows of `row` bytes, in boxes of 16 rows of up to 128 bytes.
static bool encode_rows(CUtensorMap* map, const void* base, uint64_t row, uint64_t rows) {
  cuuint64_t dims[2] = {row, rows > 0 ? rows : 1};
  cuuint64_t strides[1] = {row};
  cuuint32_t box[2] = {(cuuint32_t)(row < 128 ? row : 128), kRows};
  cuuint32_t estr[2] = {1, 1};
  return tensor_map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims,
                              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              row < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The kernel's variants, each with what the host asks of it.
template <int D, bool E8, int NT, bool kFormed>
struct Variant {
  using Z = Shape<D, E8, NT>;
  static constexpr auto kKernel = scored_mma_kernel<D, E8, NT, kFormed>;

  static int clusters(const ScoredArgs& A, int ctas) {
    return allow_smem<kKernel>() ? clusters_at_once<kKernel>(ctas, A.G, kScoredThreads, Z::smem(A.G))
                                 : 0;
  }

  static int launch(const ScoredArgs& A, cudaStream_t s) {
    if (!allow_smem<kKernel>()) return DCP_ECUDA;
    ScoredMaps maps;
    memset((void*)&maps, 0, sizeof(maps));
    const uint64_t rows = (uint64_t)A.nb * A.Hkv * A.S.bs;
    for (int r = 0; r < A.S.dcp; ++r)
      if (!encode_rows(&maps.k[r], A.k.ptr[r], Z::kRowBytes, rows) ||
          !encode_rows(&maps.v[r], A.v.ptr[r], Z::kRowBytes, rows))
        return DCP_ECUDA;
    const cudaError_t e = launch_scored<kKernel>(A, kScoredThreads, Z::smem(A.G), s, A, maps);
    return e == cudaSuccess ? launch_status() : launch_status_report(e);
  }
};

// `use` of the variant that a call takes.
template <int D, bool E8, class Use>
static int with_variant(const ScoredArgs& A, Use&& use) {
  if (A.cap > 0.f || A.slopes)
    return A.G <= 8 ? use(Variant<D, E8, 1, true>()) : use(Variant<D, E8, 2, true>());
  return A.G <= 8 ? use(Variant<D, E8, 1, false>()) : use(Variant<D, E8, 2, false>());
}
template <class Use>
static int with_variant(const ScoredArgs& A, CacheKind kind, Use&& use) {
  if (A.d == 64)
    return kind == kCacheE4m3 ? with_variant<64, true>(A, use) : with_variant<64, false>(A, use);
  return kind == kCacheE4m3 ? with_variant<128, true>(A, use) : with_variant<128, false>(A, use);
}

int scored_mma_clusters(const ScoredArgs& A, CacheKind kind, int ctas) {
  return with_variant(A, kind, [&](auto v) { return v.clusters(A, ctas); });
}

int launch_scored_mma(const ScoredArgs& A, CacheKind kind, cudaStream_t s) {
  return with_variant(A, kind, [&](auto v) { return v.launch(A, s); });
}

template <int D, bool E8, int NT>
static int one_wave(int G) {
  using Z = Shape<D, E8, NT>;
  const int fit = 228 * 1024 / (Z::smem(G) + 2048);
  return num_sms() * (fit < Z::kPerSm ? fit : Z::kPerSm);
}

int scored_mma_wave(int d, int G, CacheKind kind) {
  const bool e8 = kind == kCacheE4m3;
  if (d == 64)
    return G <= 8 ? (e8 ? one_wave<64, true, 1>(G) : one_wave<64, false, 1>(G))
                  : (e8 ? one_wave<64, true, 2>(G) : one_wave<64, false, 2>(G));
  return G <= 8 ? (e8 ? one_wave<128, true, 1>(G) : one_wave<128, false, 1>(G))
                : (e8 ? one_wave<128, true, 2>(G) : one_wave<128, false, 2>(G));
}

}  // namespace dcp
