// Rotary positions with one or several axes, fused with the owner-masked
// write of keys and values into the per-rank paged pools.
//
// Pair i of a token's rotated entries turns by
//     angle = positions[axis[i]][t] * inv_freq[i],
//     (a, b) -> (a cos - b sin, b cos + a sin),   cos, sin times `scaling`.
// Images and video give each token a time, a height and a width, and `axis`
// says which of them a pair follows; text has one axis.
//
// The angle is needed only modulo one turn.  inv_freq / 2pi is held as a
// 64-bit fraction of a turn (from two doubles, so that all 64 bits count), and
// position * fraction in wrapping 64-bit integers is the angle's fraction; its
// error is the position times 2^-64 of a turn.  A 32-bit float product loses
// it (a position of 10^6 at frequency 1 is off by 0.03 rad).  The top 32 bits
// of the fraction count.  A float of them would keep 24, so the nearest quarter
// turn is taken off them first, the rest goes to sincospif, and what the float
// of the rest leaves turns its result by the first order.
//
// What bounds it: reading q, k, v and writing them once.  The heads of a token
// are rows of one size; up to 16 KB of them (all of a token's, or a part) are
// brought into a ring of shared memory by bulk copies, rotated in place, and
// sent by bulk copies to q_out, k_out and each rank's pool, so no thread waits
// for global memory and values and unrotated rows pass through no register.
// The token's cosines and sines are computed meanwhile, once for its heads.
// Measured: 8192 tokens of 32 + 8 + 8 heads of 128 in bf16, three axes (202 MB)
// 36.6-36.9 us, 5.5 TB/s or 0.81 of the copy bandwidth; 1025 tokens of 128 + 1
// latent rows of 576 (305 MB) 52 us, 0.87; 256 tokens of a decode step 4.7 us.
// (With plain loads and stores by a CTA per token the first two took 54 and 75.)
// In place (q_out is q) only the rotated entries of q move: that is a kernel
// with a CTA per token and plain loads.
#include "dcp_common.cuh"
#include "dcp_ptx.cuh"

namespace dcp {

struct RopeArgs {
  const uint4* q;
  const uint4* k;
  const uint4* v;
  uint4* q_out;
  uint4* k_out;
  int64_t q_stride, k_stride, v_stride;  // 16-byte chunks between tokens
  const int64_t* pos;                    // [axes][T]
  const float* inv_freq;                 // [half]
  const int32_t* axis;                   // [half] or NULL
  const int64_t* slot;                   // [dcp][T]
  int64_t T, num_slots;
  int Hq, Hk, Hv;                        // heads of q, of k, of v (0: no v)
  int n16;                               // chunks of a head row
  int ru, off16;                         // rotated units of a row; first rotated chunk
  int uq, uk, uv;                        // units of a q, k and v row (a q row in place: only the
                                         // rotated ones)
  uint32_t mq, mk, mv;                   // ceil(2^32 / units), for the division
  int half, axes, bs, dcp;
  float scaling;
  dcp_rank_ptrs_t kp, vp;
  int32_t* err;
};

// n / d for n * d < 2^32 with m = ceil(2^32 / d)
__device__ __forceinline__ int fast_div(uint32_t n, uint32_t m, int d) {
  return d == 1 ? (int)n : (int)__umulhi(n, m);
}

// The rotation of one unit: its kN pairs are u * kN + i.  The table holds pair
// p's (cos, sin) at (p % kN) * ru + p / kN, so that a warp's units, which
// follow one another, read neighbouring entries.
template <bool kF32, bool kHalves>
__device__ __forceinline__ void rotate_unit(uint4& x, uint4& y, int u, int ru, const float2* cs) {
  constexpr int kN = kF32 ? 4 : 8;     // elements of a chunk
  float a[kN], b[kN];
  const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kF32) {
      a[i] = __uint_as_float(xs[i]);
      b[i] = __uint_as_float(ys[i]);
    } else {
      a[2 * i] = bf16_lo(xs[i]);
      a[2 * i + 1] = bf16_hi(xs[i]);
      b[2 * i] = bf16_lo(ys[i]);
      b[2 * i + 1] = bf16_hi(ys[i]);
    }
  }
  if (kHalves) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float2 t = cs[i * ru + u];
      const float p = a[i], q = b[i];
      a[i] = p * t.x - q * t.y;
      b[i] = q * t.x + p * t.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) {
      const float2 t = cs[i * ru + u], s = cs[(i + kN / 2) * ru + u];
      const float p = a[2 * i], q = a[2 * i + 1], r = b[2 * i], w = b[2 * i + 1];
      a[2 * i] = p * t.x - q * t.y;
      a[2 * i + 1] = q * t.x + p * t.y;
      b[2 * i] = r * s.x - w * s.y;
      b[2 * i + 1] = w * s.x + r * s.y;
    }
  }
  if (kF32) {
    x = make_uint4(__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(a[2]),
                   __float_as_uint(a[3]));
    y = make_uint4(__float_as_uint(b[0]), __float_as_uint(b[1]), __float_as_uint(b[2]),
                   __float_as_uint(b[3]));
  } else {
    x = make_uint4(pack_bf16(a[0], a[1]), pack_bf16(a[2 % kN], a[3 % kN]),
                   pack_bf16(a[4 % kN], a[5 % kN]), pack_bf16(a[6 % kN], a[7 % kN]));
    y = make_uint4(pack_bf16(b[0], b[1]), pack_bf16(b[2 % kN], b[3 % kN]),
                   pack_bf16(b[4 % kN], b[5 % kN]), pack_bf16(b[6 % kN], b[7 % kN]));
  }
}

constexpr double kInv2Pi = 0.15915494309189535;          // 1 / (2 pi), rounded
constexpr double kInv2PiLow = -9.839338337591243e-18;     // what the rounding left

// Turns per position as a 64-bit fraction: inv_freq / (2 pi) in two doubles.
__device__ __forceinline__ uint64_t turns_of(float inv_freq) {
  const double f = (double)inv_freq;
  const double hi = f * kInv2Pi;
  const double lo = fma(f, kInv2Pi, -hi) + f * kInv2PiLow;
  return (uint64_t)rint((hi - floor(hi)) * 18446744073709551616.0) +
         (uint64_t)(int64_t)rint(lo * 18446744073709551616.0);
}

// (cos, sin) of a 64-bit fraction of a turn.  The fraction is rounded to 32 bits
// (2^-33 of a turn); the float of at most 2^29 leaves at most 2^4 of them, a
// turn of 2.4e-8 rad, whose second order is far below the results' bits.
__device__ __forceinline__ float2 turned(uint64_t frac) {
  const uint32_t top = (uint32_t)((frac + 0x80000000ull) >> 32);
  const uint32_t quarter = (top + 0x20000000u) >> 30;
  const int32_t rest = (int32_t)(top - (quarter << 30));       // an eighth of a turn at most
  const float x = (float)rest;
  const float left = (float)(rest - (int32_t)x) * 1.4629180792671596e-9f;   // pi 2^-31: in rad
  float s, c;
  sincospif(x * 4.656612873077393e-10f, &s, &c);               // 2^-31: in half turns
  const float s1 = fmaf(c, left, s), c1 = fmaf(-s, left, c);
  const float a = quarter & 1 ? s1 : c1, b = quarter & 1 ? c1 : s1;
  // quarters 0 .. 3: (c, s), (-s, c), (-c, -s), (s, -c)
  return make_float2((quarter + 1) & 2 ? -a : a, quarter & 2 ? -b : b);
}

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 4;        // units in flight per thread
constexpr int kMaxHalf = 512;

struct RopeUnit {
  int kind;                // 0 q, 1 k, 2 v
  int h, u;                // head, unit of the row; u < ru: rotated
  int c0, c1;              // chunks of the row (c1 < 0: one chunk)
};

template <bool kHalves>
__device__ __forceinline__ RopeUnit rope_unit(const RopeArgs& A, int i) {
  RopeUnit U;
  int nq = A.Hq * A.uq, nk = A.Hk * A.uk;
  int rel;
  if (i < nq) {
    U.kind = 0;
    U.h = fast_div(i, A.mq, A.uq);
    U.u = i - U.h * A.uq;
  } else if (i < nq + nk) {
    U.kind = 1;
    U.h = fast_div(i - nq, A.mk, A.uk);
    U.u = i - nq - U.h * A.uk;
  } else {
    U.kind = 2;
    U.h = fast_div(i - nq - nk, A.mv, A.uv);
    U.u = i - nq - nk - U.h * A.uv;
  }
  const int ru = U.kind == 2 ? 0 : A.ru;
  if (U.u < ru) {
    U.c0 = A.off16 + (kHalves ? U.u : 2 * U.u);
    U.c1 = U.c0 + (kHalves ? A.ru : 1);
  } else {
    rel = 2 * (U.u - ru);
    const int rest = A.n16 - 2 * ru;
    U.c0 = ru > 0 && rel >= A.off16 ? rel + 2 * ru : rel;
    ++rel;
    U.c1 = rel >= rest ? -1 : (ru > 0 && rel >= A.off16 ? rel + 2 * ru : rel);
    U.u = -1;
  }
  return U;
}

template <bool kF32, bool kHalves>
__global__ void __launch_bounds__(kRopeThreads) rope_write_kernel(const __grid_constant__ RopeArgs A) {
  __shared__ float2 cs[kMaxHalf];
  __shared__ int s_dst[DCP_MAX_RANKS];
  __shared__ int64_t s_row[DCP_MAX_RANKS];
  __shared__ int s_n;
  griddep_launch_dependents();   // the next call's first kernel may start its launch
  griddep_wait();                // launched chained: the preceding kernel completed
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x;
  const int total = A.Hq * A.uq + A.Hk * A.uk + A.Hv * A.uv;
  const uint4* src[3] = {A.q + t * A.q_stride, A.k + t * A.k_stride, A.v + t * A.v_stride};

  auto load = [&](int i, RopeUnit& U, uint4& x, uint4& y) {
    U = rope_unit<kHalves>(A, i);
    const uint4* p = (U.kind == 0 ? src[0] : U.kind == 1 ? src[1] : src[2]) + (int64_t)U.h * A.n16;
    x = __ldcg(p + U.c0);
    y = U.c1 >= 0 ? __ldcg(p + U.c1) : make_uint4(0u, 0u, 0u, 0u);
  };
  auto finish = [&](const RopeUnit& U, uint4 x, uint4 y) {
    if (U.u >= 0) rotate_unit<kF32, kHalves>(x, y, U.u, A.ru, cs);
    if (U.kind == 0) {
      uint4* p = A.q_out + (t * A.Hq + U.h) * A.n16;
      p[U.c0] = x;
      if (U.c1 >= 0) p[U.c1] = y;
      return;
    }
    if (U.kind == 1 && A.k_out) {
      uint4* p = A.k_out + (t * A.Hk + U.h) * A.n16;
      p[U.c0] = x;
      if (U.c1 >= 0) p[U.c1] = y;
    }
    for (int j = 0; j < s_n; ++j) {
      const int r = s_dst[j];
      uint4* p = (uint4*)(U.kind == 1 ? A.kp.ptr[r] : A.vp.ptr[r]) +
                 (s_row[j] + (int64_t)U.h * A.bs) * A.n16;
      p[U.c0] = x;
      if (U.c1 >= 0) p[U.c1] = y;
    }
  };

  RopeUnit U[kRopeBatch];
  uint4 x[kRopeBatch], y[kRopeBatch];
#pragma unroll
  for (int j = 0; j < kRopeBatch; ++j)
    if (tid + j * kRopeThreads < total) load(tid + j * kRopeThreads, U[j], x[j], y[j]);

  // the ranks that store this token (warp 7, the last to have trigonometry)
  if (tid >= kRopeThreads - 32) {
    const int r = tid - (kRopeThreads - 32);
    const int64_t s = r < A.dcp ? __ldcg(A.slot + (int64_t)r * A.T + t) : -1;
    const bool ok = s >= 0 && s < A.num_slots;
    if (!ok && s != -1) count_error(A.err);
    const uint32_t m = __ballot_sync(0xffffffffu, ok);
    if (ok) {
      const int at = __popc(m & ((1u << r) - 1u));
      const int64_t blk = s / A.bs;
      s_dst[at] = r;
      s_row[at] = blk * A.Hk * A.bs + (s - blk * A.bs);
    }
    if (r == 0) s_n = __popc(m);
  }
  for (int i = tid; i < A.half; i += kRopeThreads) {
    int ax = A.axis ? __ldcg(A.axis + i) : 0;
    if (ax < 0 || ax >= A.axes) {
      if (t == 0) count_error(A.err);
      ax = 0;
    }
    const uint64_t p = (uint64_t)__ldcg(A.pos + (int64_t)ax * A.T + t);
    const float2 t1 = turned(p * turns_of(__ldcg(A.inv_freq + i)));
    constexpr int kN = kF32 ? 4 : 8;
    cs[(i % kN) * A.ru + i / kN] = make_float2(t1.x * A.scaling, t1.y * A.scaling);
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kRopeBatch; ++j)
    if (tid + j * kRopeThreads < total) finish(U[j], x[j], y[j]);
  for (int i0 = tid + kRopeBatch * kRopeThreads; i0 < total; i0 += kRopeBatch * kRopeThreads) {
#pragma unroll
    for (int j = 0; j < kRopeBatch; ++j)
      if (i0 + j * kRopeThreads < total) load(i0 + j * kRopeThreads, U[j], x[j], y[j]);
#pragma unroll
    for (int j = 0; j < kRopeBatch; ++j)
      if (i0 + j * kRopeThreads < total) finish(U[j], x[j], y[j]);
  }
}

constexpr int kRbThreads = 128;
constexpr int kRbStages = 2;
constexpr int kRbPerSm = 8;           // CTAs of an SM, as far as shared memory goes
constexpr int kRbItem = 16 * 1024;    // most bytes of an item, unless a row is longer
constexpr int kRbPairs = kMaxHalf / kRbThreads;

struct RopeBulk {
  int rows, parts;       // rows of an item, items of a token
  uint32_t mr;           // for i / ru
  int items;
  int stage;             // bytes of a stage
};

// Two stages and eight CTAs an SM: three to five stages, items of 8 or 32 KB, 96
// or 256 threads and 6 or 12 CTAs were within 1% or slower (8192 tokens).  Eight
// CTAs need the bound on registers: at 72 of them seven fit, and the last wave
// took the call from 36 us to 47.
template <bool kF32, bool kHalves>
__global__ void __launch_bounds__(kRbThreads, kRbPerSm)
rope_bulk_kernel(const __grid_constant__ RopeArgs A, const RopeBulk B) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kRbStages];
  constexpr int kN = kF32 ? 4 : 8;
  const int tid = threadIdx.x, lane = tid & 31;
  const uint32_t base = smem_u32(smem);
  const int row_bytes = A.n16 * 16, R = A.Hq + A.Hk + A.Hv;
  float2* const cs = reinterpret_cast<float2*>(smem + kRbStages * B.stage);   // [2][half]
  griddep_launch_dependents();   // the next call's first kernel may start its launch
  if (tid == 0) {
    for (int i = 0; i < kRbStages; ++i) mbar_init(smem_u32(full + i), 1);
    fence_mbar_init();
  }
  __syncthreads();
  griddep_wait();                // launched chained: the preceding kernel completed

  // rows [r0, r1) of an item's token, by whose they are
  auto load = [&](int item, int stage) {   // thread 0
    const int64_t t = item / B.parts;
    const int r0 = (item - (int)t * B.parts) * B.rows, r1 = min(r0 + B.rows, R);
    const uint32_t bar = smem_u32(full + stage), dst = base + stage * B.stage;
    mbar_arrive_expect_tx(bar, (r1 - r0) * row_bytes);
    auto part = [&](const uint4* src, int64_t stride, int lo, int hi) {
      const int a = max(r0, lo), b = min(r1, hi);
      if (a < b)
        bulk_load(dst + (a - r0) * row_bytes, src + t * stride + (int64_t)(a - lo) * A.n16,
                  (b - a) * row_bytes, bar);
    };
    part(A.q, A.q_stride, 0, A.Hq);
    part(A.k, A.k_stride, A.Hq, A.Hq + A.Hk);
    part(A.v, A.v_stride, A.Hq + A.Hk, R);
  };
  if (tid == 0)
    for (int k = 0; k < kRbStages - 1; ++k) {
      const int64_t item = blockIdx.x + (int64_t)k * gridDim.x;
      if (item < B.items) load((int)item, k);
    }
  // this thread's pairs: turns per position as a 64-bit fraction
  uint64_t per[kRbPairs];
  int ax[kRbPairs];
#pragma unroll
  for (int j = 0; j < kRbPairs; ++j) {
    const int i = tid + j * kRbThreads;
    per[j] = 0;
    ax[j] = 0;
    if (i >= A.half) continue;
    per[j] = turns_of(__ldcg(A.inv_freq + i));
    ax[j] = A.axis ? __ldcg(A.axis + i) : 0;
    if (ax[j] < 0 || ax[j] >= A.axes) {
      if (blockIdx.x == 0) count_error(A.err);
      ax[j] = 0;
    }
  }
  auto position = [&](int item, int j) -> uint64_t {
    return tid + j * kRbThreads < A.half && item < B.items
               ? (uint64_t)__ldcg(A.pos + (int64_t)ax[j] * A.T + item / B.parts)
               : 0ull;
  };
  uint64_t pos[kRbPairs];
#pragma unroll
  for (int j = 0; j < kRbPairs; ++j) pos[j] = position(blockIdx.x, j);

  uint32_t dead = 0;             // 1 + the round whose load did not come
  uint32_t k = 0;
  for (int64_t it = blockIdx.x; it < B.items; it += gridDim.x, ++k) {
    const int item = (int)it, stage = k % kRbStages;
    const int64_t t = item / B.parts;
    const int r0 = (item - (int)t * B.parts) * B.rows, r1 = min(r0 + B.rows, R);
    const int64_t nxt = it + gridDim.x;
    const bool writes = r1 > A.Hq;            // keys or values among the rows
    // the token's slot on rank `lane` (warp 0, which issues the stores)
    int64_t slot = -1;
    if (tid < 32 && writes && lane < A.dcp) slot = __ldcg(A.slot + (int64_t)lane * A.T + t);
    float2* tab = cs + (k & 1) * A.half;
#pragma unroll
    for (int j = 0; j < kRbPairs; ++j) {
      const int i = tid + j * kRbThreads;
      if (j * kRbThreads < A.half && i < A.half) {
        const float2 t1 = turned(pos[j] * per[j]);
        tab[(i % kN) * A.ru + i / kN] = make_float2(t1.x * A.scaling, t1.y * A.scaling);
      }
      pos[j] = position(nxt < B.items ? (int)nxt : B.items, j);
    }
    if (!dead && !mbar_wait(smem_u32(full + stage), (k / kRbStages) & 1)) dead = k + 1;
    __syncthreads();
    uint4* rows = reinterpret_cast<uint4*>(smem + stage * B.stage);
    const int turn = max(min(r1, A.Hq + A.Hk) - r0, 0) * A.ru;
    for (int i = tid; i < turn; i += kRbThreads) {
      const int row = fast_div(i, B.mr, A.ru), u = i - row * A.ru;
      uint4* p = rows + row * A.n16 + A.off16 + (kHalves ? u : 2 * u);
      uint4* q = p + (kHalves ? A.ru : 1);
      uint4 x = *p, y = *q;
      rotate_unit<kF32, kHalves>(x, y, u, A.ru, tab);
      *p = x;
      *q = y;
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (tid < 32) {
      const uint32_t src = base + stage * B.stage;
      if (!__any_sync(0xffffffffu, dead != 0)) {
        if (lane == 0) {
          const int b = min(r1, A.Hq);
          if (r0 < b)
            bulk_store(A.q_out + (t * A.Hq + r0) * A.n16, src, (b - r0) * row_bytes);
          const int c0 = max(r0, A.Hq), c1 = min(r1, A.Hq + A.Hk);
          if (A.k_out && c0 < c1)
            bulk_store(A.k_out + (t * A.Hk + c0 - A.Hq) * A.n16, src + (c0 - r0) * row_bytes,
                       (c1 - c0) * row_bytes);
        }
        if (writes) {
          const bool ok = slot >= 0 && slot < A.num_slots;
          if (!ok && slot != -1 && r0 <= A.Hq) count_error(A.err);
          uint32_t m = __ballot_sync(0xffffffffu, ok);
          while (m) {
            const int r = __ffs(m) - 1;
            m &= m - 1;
            const int64_t s = __shfl_sync(0xffffffffu, slot, r), blk = s / A.bs;
            for (int row = max(r0, A.Hq) + lane; row < r1; row += 32) {
              const bool val = row >= A.Hq + A.Hk;
              const int h = row - A.Hq - (val ? A.Hk : 0);
              bulk_store((uint4*)(val ? A.vp.ptr[r] : A.kp.ptr[r]) +
                             ((blk * A.Hk + h) * A.bs + (s - blk * A.bs)) * A.n16,
                         src + (row - r0) * row_bytes, row_bytes);
            }
          }
        }
      }
      bulk_commit();
      bulk_wait_read<1>();     // the stage before this one has been read
      __syncwarp();
      const int64_t ahead = it + (int64_t)(kRbStages - 1) * gridDim.x;
      if (lane == 0 && !dead && ahead < B.items) load((int)ahead, (k + kRbStages - 1) % kRbStages);
    }
  }
  if (tid < 32) bulk_wait_read<0>();   // shared memory is left only when it has been read
  if (dead && tid == 0) {   // the load that did not come, for a last time
    mbar_wait(smem_u32(full + (dead - 1) % kRbStages), ((dead - 1) / kRbStages) & 1);
    if (A.err) atomicAdd(A.err, 1 << 20);
  }
}

static uint32_t div_magic(int d) {
  return d <= 1 ? 0u : (uint32_t)(((uint64_t(1) << 32) + (uint64_t)d - 1) / (uint64_t)d);
}

template <bool kF32, bool kHalves>
static cudaError_t launch_bulk(const RopeArgs& A, const RopeBulk& B, unsigned grid, int smem,
                               cudaStream_t s) {
  if (!allow_smem<rope_bulk_kernel<kF32, kHalves>>()) return cudaErrorInvalidValue;
  return launch_chained(rope_bulk_kernel<kF32, kHalves>, grid, kRbThreads, smem, s, A, B);
}

static int launch_rope(RopeArgs& A, int rot, int rot_at, int d, int es, bool interleaved,
                       cudaStream_t s) {
  A.n16 = d * es / 16;
  A.ru = rot * es / 32;
  A.off16 = rot_at * es / 16;
  A.half = rot / 2;
  const int rest = A.n16 - 2 * A.ru;
  A.uk = A.ru + (rest + 1) / 2;
  A.uv = (A.n16 + 1) / 2;
  // in place, the unrotated chunks of q stay where they are
  A.uq = A.q_out == A.q && A.q_stride == (int64_t)A.Hq * A.n16 ? A.ru : A.uk;
  A.mq = div_magic(A.uq);
  A.mk = div_magic(A.uk);
  A.mv = div_magic(A.uv);
  cudaError_t e;
  const int R = A.Hq + A.Hk + A.Hv, row_bytes = A.n16 * 16;
  RopeBulk B;
  B.parts = 1;
  if (row_bytes * R > kRbItem) {
    B.rows = kRbItem / row_bytes > 0 ? kRbItem / row_bytes : 1;
    B.parts = (R + B.rows - 1) / B.rows;
  }
  B.rows = (R + B.parts - 1) / B.parts;
  B.parts = (R + B.rows - 1) / B.rows;
  B.mr = div_magic(A.ru);
  B.stage = (B.rows * row_bytes + 127) / 128 * 128;
  const bool in_place = A.Hq > 0 && A.uq != A.uk;
  if (!in_place && A.T * B.parts < (int64_t(1) << 31)) {
    B.items = (int)(A.T * B.parts);
    const int smem = kRbStages * B.stage + 2 * A.half * (int)sizeof(float2);
    const int fit = 224 * 1024 / (smem + 1024 + 64);
    const int per_sm = fit < 1 ? 1 : (fit < kRbPerSm ? fit : kRbPerSm);
    const int64_t most = (int64_t)per_sm * num_sms();
    const unsigned grid = (unsigned)(B.items < most ? B.items : most);
    if (es == 4)
      e = interleaved ? launch_bulk<true, false>(A, B, grid, smem, s)
                      : launch_bulk<true, true>(A, B, grid, smem, s);
    else
      e = interleaved ? launch_bulk<false, false>(A, B, grid, smem, s)
                      : launch_bulk<false, true>(A, B, grid, smem, s);
    if (e != cudaSuccess) return launch_status_report(e);
    return launch_status();
  }
  const unsigned grid = (unsigned)A.T;
  if (es == 4)
    e = interleaved ? launch_chained(rope_write_kernel<true, false>, grid, kRopeThreads, 0, s, A)
                    : launch_chained(rope_write_kernel<true, true>, grid, kRopeThreads, 0, s, A);
  else
    e = interleaved ? launch_chained(rope_write_kernel<false, false>, grid, kRopeThreads, 0, s, A)
                    : launch_chained(rope_write_kernel<false, true>, grid, kRopeThreads, 0, s, A);
  if (e != cudaSuccess) return launch_status_report(e);
  return launch_status();
}

static inline int elem_bytes(dcp_dtype_t d) { return d == DCP_F32 ? 4 : (d == DCP_BF16 ? 2 : 0); }
static inline bool al16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// Rows of `row` bytes, one for each token, `stride` bytes apart.
struct TokenRows {
  const void* p;
  int64_t stride, row;
};

// Whether the packed rows of an output lie over rows of an input: CTAs read and
// write different tokens at the same time, so that is refused, but for an output
// that is the input itself, token by token (`same`: where the rows hold the same heads).
static bool rows_clash(const void* out, int64_t row, const TokenRows& in, int64_t T, bool same) {
  if (!out || !in.p || row <= 0 || in.row <= 0) return false;
  const int64_t off = (int64_t)((uintptr_t)out - (uintptr_t)in.p);
  if (same && off == 0 && (T == 1 || in.stride == row)) return false;
  // the first token whose row ends behind the output's start
  const int64_t i = off < in.row ? 0 : (off - in.row) / in.stride + 1;
  return i < T && i * in.stride < off + T * row;
}

// Checks shared by both entry points; DCP_OK when the shape can run.
static int rope_shape(const dcp_layout_t& L, int64_t T, int Hq, int Hk, int d, int es, int rot,
                      int axes, int64_t num_blocks) {
  if (!layout_ok(L) || es == 0 || T < 0 || Hq < 0 || Hk < 1 || d < 1 || rot < 2 || rot > d ||
      axes < 1 || num_blocks < 0)
    return DCP_EINVAL;
  // the division by units a row takes under 2^20 units a token and 4096 a row
  if (T >= (int64_t(1) << 31) || d > 8192 || (d * es) % 16 != 0 || rot % 16 != 0 ||
      rot / 2 > kMaxHalf ||
      ((int64_t)Hq + 2 * (int64_t)Hk) * (d * es / 16) >= (int64_t(1) << 20))
    return DCP_EUNSUPPORTED;
  return DCP_OK;
}

}  // namespace dcp

using namespace dcp;

extern "C" {

int dcp_rope_write_gqa(dcp_layout_t layout, const void* q, int64_t q_stride, const void* k,
                       int64_t k_stride, const void* v, int64_t v_stride, int64_t num_tokens,
                       int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                       dcp_dtype_t dtype, const int64_t* positions, int32_t num_axes,
                       const float* inv_freq, const int32_t* axis, int32_t rot_dim,
                       int32_t interleaved, float scaling, const int64_t* slot,
                       int64_t num_blocks, dcp_rank_ptrs_t k_cache, dcp_rank_ptrs_t v_cache,
                       void* q_out, void* k_out, int32_t* err_count, dcp_stream_t stream) {
  dcp::NvtxRange nvtx_range("dcp_rope_write_gqa");
  const int es = elem_bytes(dtype);
  const int rc = rope_shape(layout, num_tokens, num_q_heads, num_kv_heads, head_dim, es, rot_dim,
                            num_axes, num_blocks);
  if (rc != DCP_OK) return rc;
  if (num_tokens == 0) return DCP_OK;
  if ((num_q_heads > 0 && (!q || !q_out)) || !k || !v || !positions || !inv_freq || !slot ||
      !ranks_ok(k_cache, layout.dcp_size) || !ranks_ok(v_cache, layout.dcp_size))
    return DCP_EINVAL;
  if (q_stride < (int64_t)num_q_heads * head_dim || k_stride < (int64_t)num_kv_heads * head_dim ||
      v_stride < (int64_t)num_kv_heads * head_dim)
    return DCP_EINVAL;
  if (!al16(q) || !al16(k) || !al16(v) || !al16(q_out) || !al16(k_out) || (q_stride * es) % 16 ||
      (k_stride * es) % 16 || (v_stride * es) % 16)
    return DCP_EUNSUPPORTED;
  for (int r = 0; r < layout.dcp_size; ++r)
    if (!al16(k_cache.ptr[r]) || !al16(v_cache.ptr[r])) return DCP_EUNSUPPORTED;
  const int64_t T = num_tokens, half = rot_dim / 2, qr = (int64_t)num_q_heads * head_dim * es,
                kr = (int64_t)num_kv_heads * head_dim * es;
  const TokenRows tq{num_q_heads > 0 ? q : nullptr, q_stride * es, qr}, tk{k, k_stride * es, kr},
      tv{v, v_stride * es, kr};
  if (num_q_heads == 0) q_out = nullptr;
  if (rows_clash(q_out, qr, tq, T, true) || rows_clash(q_out, qr, tk, T, false) ||
      rows_clash(q_out, qr, tv, T, false) || rows_clash(k_out, kr, tk, T, true) ||
      rows_clash(k_out, kr, tq, T, false) || rows_clash(k_out, kr, tv, T, false) ||
      !apart({{q_out, T * qr}, {k_out, T * kr}},
             {{positions, num_axes * T * 8}, {inv_freq, half * 4}, {axis, half * 4},
              {slot, layout.dcp_size * T * 8}}))
    return DCP_EINVAL;
  RopeArgs A;
  A.q = (const uint4*)q;
  A.k = (const uint4*)k;
  A.v = (const uint4*)v;
  A.q_out = (uint4*)q_out;
  A.k_out = (uint4*)k_out;
  A.q_stride = q_stride * es / 16;
  A.k_stride = k_stride * es / 16;
  A.v_stride = v_stride * es / 16;
  A.pos = positions;
  A.inv_freq = inv_freq;
  A.axis = axis;
  A.slot = slot;
  A.T = num_tokens;
  A.num_slots = num_blocks * layout.block_size;
  A.Hq = num_q_heads;
  A.Hk = A.Hv = num_kv_heads;
  A.axes = num_axes;
  A.bs = layout.block_size;
  A.dcp = layout.dcp_size;
  A.scaling = scaling;
  A.kp = k_cache;
  A.vp = v_cache;
  A.err = err_count;
  return launch_rope(A, rot_dim, 0, head_dim, es, interleaved != 0, (cudaStream_t)stream);
}

int dcp_rope_write_mla(dcp_layout_t layout, const void* q, int64_t q_stride, const void* kv,
                       int64_t kv_stride, int64_t num_tokens, int32_t num_q_heads, int32_t kv_dim,
                       dcp_dtype_t dtype, const int64_t* positions, int32_t num_axes,
                       const float* inv_freq, const int32_t* axis, int32_t rot_dim,
                       int32_t interleaved, float scaling, const int64_t* slot,
                       int64_t num_blocks, dcp_rank_ptrs_t cache, void* q_out,
                       int32_t* err_count, dcp_stream_t stream) {
  dcp::NvtxRange nvtx_range("dcp_rope_write_mla");
  const int es = elem_bytes(dtype);
  const int rc = rope_shape(layout, num_tokens, num_q_heads, 1, kv_dim, es, rot_dim, num_axes,
                            num_blocks);
  if (rc != DCP_OK) return rc;
  if (num_tokens == 0) return DCP_OK;
  if ((num_q_heads > 0 && (!q || !q_out)) || !kv || !positions || !inv_freq || !slot ||
      !ranks_ok(cache, layout.dcp_size))
    return DCP_EINVAL;
  if (q_stride < (int64_t)num_q_heads * kv_dim || kv_stride < kv_dim) return DCP_EINVAL;
  if (!al16(q) || !al16(kv) || !al16(q_out) || (q_stride * es) % 16 || (kv_stride * es) % 16)
    return DCP_EUNSUPPORTED;
  for (int r = 0; r < layout.dcp_size; ++r)
    if (!al16(cache.ptr[r])) return DCP_EUNSUPPORTED;
  const int64_t T = num_tokens, half = rot_dim / 2, qr = (int64_t)num_q_heads * kv_dim * es;
  if (num_q_heads == 0) q_out = nullptr;
  if (rows_clash(q_out, qr, {q, q_stride * es, qr}, T, true) ||
      rows_clash(q_out, qr, {kv, kv_stride * es, (int64_t)kv_dim * es}, T, false) ||
      !apart({{q_out, T * qr}}, {{positions, num_axes * T * 8}, {inv_freq, half * 4},
                                 {axis, half * 4}, {slot, layout.dcp_size * T * 8}}))
    return DCP_EINVAL;
  RopeArgs A;
  A.q = (const uint4*)q;
  A.k = (const uint4*)kv;
  A.v = nullptr;
  A.q_out = (uint4*)q_out;
  A.k_out = nullptr;
  A.q_stride = q_stride * es / 16;
  A.k_stride = kv_stride * es / 16;
  A.v_stride = 0;
  A.pos = positions;
  A.inv_freq = inv_freq;
  A.axis = axis;
  A.slot = slot;
  A.T = num_tokens;
  A.num_slots = num_blocks * layout.block_size;
  A.Hq = num_q_heads;
  A.Hk = 1;
  A.Hv = 0;
  A.axes = num_axes;
  A.bs = layout.block_size;
  A.dcp = layout.dcp_size;
  A.scaling = scaling;
  A.kp = A.vp = cache;
  A.err = err_count;
  return launch_rope(A, rot_dim, kv_dim - rot_dim, kv_dim, es, interleaved != 0,
                     (cudaStream_t)stream);
}

}  // extern "C"
