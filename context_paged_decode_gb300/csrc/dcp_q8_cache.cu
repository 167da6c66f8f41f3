// The 8-bit cache: keys and values quantised as they are written, and read
// back.  A page and head has one scale for its keys and one for its values, a
// power of two s; a number x is held as the e4m3 number nearest to x / s.
#include <type_traits>

#include "dcp_q8.cuh"
#include "dcp_scored.cuh"

namespace dcp {

struct AppendArgs {
  Shards S;
  const void* src[2];        // keys, values: [N][Hkv][d], `stride` bytes between tokens
  int64_t stride[2];
  dcp_rank_ptrs_t pool[2], sc;
  const int32_t* start;      // [B + 1]
  const int32_t* ctx;        // [B]
  int N, B, Hkv, d;
  const int32_t* bt;
  int max_vb;
  int64_t bt_stride, nb;
  int per_warp;              // tokens that a warp looks at
  int32_t* err;
};

// Numbers 4 i .. 4 i + 3 of 16 bytes.
template <typename T>
__device__ __forceinline__ float4 quad(const uint4& x, int i);
template <>
__device__ __forceinline__ float4 quad<float>(const uint4& x, int) {
  return make_float4(__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z),
                     __uint_as_float(x.w));
}
template <>
__device__ __forceinline__ float4 quad<__nv_bfloat16>(const uint4& x, int i) {
  const uint32_t a = i ? x.z : x.x, b = i ? x.w : x.y;
  return make_float4(bf16_lo(a), bf16_hi(a), bf16_lo(b), bf16_hi(b));
}

// 16 bytes of numbers times a power of two (bf16: two at a time, exact but for
// results below 2^-126, which are 0 in e4m3).
template <typename T>
__device__ __forceinline__ uint4 times(const uint4& x, float by);
template <>
__device__ __forceinline__ uint4 times<float>(const uint4& x, float by) {
  return make_uint4(__float_as_uint(__uint_as_float(x.x) * by),
                    __float_as_uint(__uint_as_float(x.y) * by),
                    __float_as_uint(__uint_as_float(x.z) * by),
                    __float_as_uint(__uint_as_float(x.w) * by));
}
template <>
__device__ __forceinline__ uint4 times<__nv_bfloat16>(const uint4& x, float by) {
  const __nv_bfloat162 b = __float2bfloat162_rn(by);
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), b);
    w[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// |x| of a finite number, 0 of others.
__device__ __forceinline__ float size_of(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}

// The larger of top and the sizes of 16 bytes of numbers; NaN does not count.
template <typename T>
__device__ __forceinline__ void raise(uint32_t& top, const uint4& x);
template <>
__device__ __forceinline__ void raise<float>(uint32_t& top, const uint4& x) {
  const float a = fmaxf(fabsf(__uint_as_float(x.x)), fabsf(__uint_as_float(x.y)));
  const float b = fmaxf(fabsf(__uint_as_float(x.z)), fabsf(__uint_as_float(x.w)));
  top = __float_as_uint(fmaxf(__uint_as_float(top), fmaxf(a, b)));
}
template <>
__device__ __forceinline__ void raise<__nv_bfloat16>(uint32_t& top, const uint4& x) {   // two at a time
  __nv_bfloat162 m = *reinterpret_cast<__nv_bfloat162*>(&top);
  const uint32_t w[4] = {x.x & 0x7fff7fffu, x.y & 0x7fff7fffu, x.z & 0x7fff7fffu, x.w & 0x7fff7fffu};
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&w[i]));
  top = *reinterpret_cast<uint32_t*>(&m);
}
template <typename T>
__device__ __forceinline__ float raised(uint32_t top) {
  return sizeof(T) == 4 ? __uint_as_float(top) : fmaxf(bf16_lo(top), bf16_hi(top));
}

constexpr int kAppendDepth = 8;    // 16-byte loads in flight per thread

// The tokens that a call writes to one page, for one head and one of K and V,
// are one warp's: it reads them, finds their size and the page's scale, and
// writes them, and if the scale grows also the page's other places.  Which
// tokens those are follows from the request's run of positions, so there is no
// sorting, nothing to clear and no atomic.  A warp looks at a few tokens in a
// row and takes the pages whose turn is one of them: of a page's new tokens the
// (rank * bs / dcp)-th, so that the pages of one virtual block, whose first
// tokens lie side by side, go to different warps; a CTA's warps share out what
// they have found (the few tokens of a first or last page lie side by side all
// the same: 16.0 us for the prompts of 8192 tokens where each keeps its own, 11.5
// with four warps, 10.7 with eight).
template <typename T, int kAppendWarps>
__global__ void __launch_bounds__(kAppendWarps * 32, kAppendWarps == 4 ? 6 : 3)
q8_append_kernel(const __grid_constant__ AppendArgs A) {
  __shared__ int s_found[kAppendWarps];
  __shared__ int4 s_page[kAppendWarps * 16], s_req[kAppendWarps * 16];
  griddep_launch_dependents();   // the next call's first kernel may start its launch
  griddep_wait();                // launched chained: the preceding kernel completed
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.y, which = blockIdx.z;
  const int64_t room = min((int64_t)A.max_vb * A.S.vbs, (int64_t)INT32_MAX);
  auto usable = [&](int c, int q0, int q1) {
    return c >= 0 && q0 >= 0 && q1 >= q0 && q1 <= A.N && (int64_t)c + (q1 - q0) <= room;
  };
  if (blockIdx.x == 0 && h == 0 && which == 0 && A.err)
    for (int b = threadIdx.x; b < A.B; b += kAppendWarps * 32)
      if (!usable(__ldg(A.ctx + b), __ldg(A.start + b), __ldg(A.start + b + 1))) count_error(A.err);
  const int64_t first = ((int64_t)blockIdx.x * kAppendWarps + warp) * A.per_warp;
  // this lane's token and its request, the last whose start lies at or before it
  const int t = (int)first + lane;
  int b, c = 0, q0 = 0, q1 = 0;
  auto starts_upto = [&](int s) {   // of 32 starts in order, one a lane: those <= t
    int n = 0;
#pragma unroll
    for (int step = 16; step > 0; step >>= 1) {
      const int x = __shfl_sync(0xffffffffu, s, n + step - 1);
      if (x <= t) n += step;
    }
    const int x = __shfl_sync(0xffffffffu, s, n & 31);
    return n + (n < 32 && x <= t);
  };
  if (A.B < 32) {   // all that is to be known of the requests in one load
    const int s = lane <= A.B ? __ldg(A.start + lane) : INT32_MAX;
    const int ctx = lane < A.B ? __ldg(A.ctx + lane) : 0;
    b = starts_upto(s) - 1;
    c = __shfl_sync(0xffffffffu, ctx, b & 31);
    q0 = __shfl_sync(0xffffffffu, s, b & 31);
    q1 = __shfl_sync(0xffffffffu, s, (b + 1) & 31);
  } else {
    int at = 0;
#pragma unroll 4
    for (int i = lane; i <= A.B; i += 32) at += __ldg(A.start + i) <= first;
    b = __reduce_add_sync(0xffffffffu, at) - 1;
    for (int base = b + 1;; base += 32) {
      const int n = starts_upto(base + lane <= A.B ? __ldg(A.start + base + lane) : INT32_MAX);
      b += n;
      if (!__any_sync(0xffffffffu, n == 32)) break;
    }
    if (b >= 0 && b < A.B) {
      c = __ldg(A.ctx + b);
      q0 = __ldg(A.start + b);
      q1 = __ldg(A.start + b + 1);
    }
  }
  // is the token the one that stands for its page?
  bool mine = false;
  int rank = 0, vb = 0, loc0 = 0, n = 0;
  if (lane < A.per_warp && t < A.N && b >= 0 && b < A.B && usable(c, q0, q1) && t >= q0 && t < q1) {
    int loc;
    A.S.place(c + t - q0, rank, vb, loc);
    const int page0 = vb * A.S.bs;
    loc0 = max(Below(A.S, c).on(A.S, rank) - page0, 0);
    n = min(Below(A.S, c + q1 - q0).on(A.S, rank) - page0, A.S.bs) - loc0;
    mine = loc == loc0 + rank * A.S.bs / A.S.dcp % n;
  }
  // a lane takes what becomes 16 bytes of a row, of several rows
  constexpr int kLoads = sizeof(T), kEach = kAppendDepth / kLoads;
  const int chunks = A.d / 16, rows = 32 / chunks, batch = rows * kEach;
  const int row = lane / chunks, chunk = lane - row * chunks;
  const bool busy = row < rows;
  const uint32_t found = __ballot_sync(0xffffffffu, mine);
  if (lane == 0) s_found[warp] = __popc(found);
  __syncthreads();
  int total = 0, at = 0;
#pragma unroll
  for (int w = 0; w < kAppendWarps; ++w) {
    if (w == warp) at = total;
    total += s_found[w];
  }
  if (mine) {
    at += __popc(found & ((1u << lane) - 1));
    s_page[at] = make_int4(rank, vb, loc0, n);
    s_req[at] = make_int4(b, c, q0, 0);
  }
  __syncthreads();
  for (int turn = warp; turn < total; turn += kAppendWarps) {
    const int4 of_page = s_page[turn], of_req = s_req[turn];
    const int pr = of_page.x, pv = of_page.y, pl = of_page.z, pn = of_page.w;
    const int pb = of_req.x, pc = of_req.y, pq = of_req.z;
    // the first rows are on their way before the table's answer
    const char* src = (const char*)A.src[which] + (int64_t)h * A.d * sizeof(T);
    const int64_t stride = A.stride[which];
    const int64_t page =
        __ldg(A.bt + pr * A.bt_stride + (int64_t)pb * A.max_vb + pv);
    uint4 x[kEach][kLoads];
    auto each_row = [&](bool reload, auto&& use) {   // use(16 numbers of a row, its number)
      for (int i0 = row; i0 < pn + row; i0 += batch) {
        if (reload) {
#pragma unroll
          for (int j = 0; j < kEach; ++j) {
            const int i = i0 + j * rows;
            const bool have = busy && i < pn;
            const int64_t tok = have ? pq + (A.S.position(pv, pr, pl + i) - pc) : 0;
            const uint4* from = reinterpret_cast<const uint4*>(src + tok * stride) + chunk * kLoads;
#pragma unroll
            for (int k = 0; k < kLoads; ++k) x[j][k] = have ? __ldg(from + k) : make_uint4(0u, 0u, 0u, 0u);
          }
        }
#pragma unroll
        for (int j = 0; j < kEach; ++j)
          if (busy && i0 + j * rows < pn) use(x[j], i0 + j * rows);
      }
    };
    uint32_t most = 0;
    each_row(true, [&](const uint4(&y)[kLoads], int) {
#pragma unroll
      for (int k = 0; k < kLoads; ++k) raise<T>(most, y[k]);
    });
    float top = raised<T>(most);
    if (page < 0 || page >= A.nb) {
      if (lane == 0 && h == 0 && which == 0) count_error(A.err);
      continue;
    }
    uint8_t* dst = (uint8_t*)A.pool[which].ptr[pr] + (page * A.Hkv + h) * A.S.bs * A.d;
    float* scale = (float*)A.sc.ptr[pr] + (page * A.Hkv + h) * kScaleFloats + which;
    const float held = pl > 0 ? __ldcg(scale) : 0.f;
    top = warp_max(top);
    if (top > 3.402823466e38f) {   // infinities do not count
      top = 0.f;
      each_row(true, [&](const uint4(&y)[kLoads], int) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 z = quad<T>(y[k * kLoads / 4], k * kLoads % 4 ? 1 : 0);
          top = fmaxf(top, fmaxf(fmaxf(size_of(z.x), size_of(z.y)),
                                 fmaxf(size_of(z.z), size_of(z.w))));
        }
      });
      top = warp_max(top);
    }
    // a page that begins, or whose scale is none, keeps nothing
    const float old = held > 0.f && held <= 3.402823466e38f ? held : 0.f;
    const float now = fmaxf(old, scale_for(top));
    const bool grows = old > 0.f && now > old;
    const bool once = pn <= batch;   // still in registers
    const float inv = 1.f / now;     // exact for a power of two; others divide
    uint8_t* const to = dst + (int64_t)pl * A.d + chunk * 16;
    if ((__float_as_uint(now) & 0x7fffffu) == 0)
      each_row(!once, [&](const uint4(&y)[kLoads], int i) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[k] = f32x4_e4m3(quad<T>(times<T>(y[k * kLoads / 4], inv), k * kLoads % 4 ? 1 : 0));
        *reinterpret_cast<uint4*>(to + (int64_t)i * A.d) = make_uint4(w[0], w[1], w[2], w[3]);
      });
    else
      each_row(true, [&](const uint4(&y)[kLoads], int i) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 z = quad<T>(y[k * kLoads / 4], k * kLoads % 4 ? 1 : 0);
          w[k] = f32x4_e4m3(make_float4(z.x / now, z.y / now, z.z / now, z.w / now));
        }
        *reinterpret_cast<uint4*>(to + (int64_t)i * A.d) = make_uint4(w[0], w[1], w[2], w[3]);
      });
    if (grows) {   // the page's other places
      const float by = old / now;
      for (int l = row; busy && l < A.S.bs; l += rows) {
        if (l >= pl && l < pl + pn) continue;
        uint4* const at = reinterpret_cast<uint4*>(dst + (int64_t)l * A.d) + chunk;
        const uint4 held4 = *at;
        uint32_t w[4] = {held4.x, held4.y, held4.z, held4.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 y = e4m3x4_f32(w[k]);
          w[k] = f32x4_e4m3(make_float4(y.x * by, y.y * by, y.z * by, y.w * by));
        }
        *at = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    __syncwarp();
    if (lane == 0) *scale = now;
  }
}

template <typename T, int kWarps>
static cudaError_t launch_append(const AppendArgs& A, cudaStream_t s) {
  const int64_t warps = ((int64_t)A.N + A.per_warp - 1) / A.per_warp;
  const dim3 grid((unsigned)((warps + kWarps - 1) / kWarps), (unsigned)A.Hkv, 2);
  return launch_chained(q8_append_kernel<T, kWarps>, grid, kWarps * 32, 0, s, A);
}

struct GatherArgs {
  Shards S;
  dcp_rank_ptrs_t pool[2], sc;
  const int32_t* bt;
  int B, Hkv, d, max_vb;
  int64_t bt_stride, nb;
  const int32_t* req;
  const int64_t* pos;
  int64_t N;
  int per_cta;      // tokens of a CTA
  void* out[2];
  int32_t* err;
};

constexpr int kGatherThreads = 256;
constexpr int kGatherTokens = 16;  // of a CTA at most; a power of two, as CTAs take 1, 2, 4 ...
static_assert((kGatherTokens & (kGatherTokens - 1)) == 0, "CTAs take 1, 2, 4 ... tokens");
constexpr int kGatherDepth = 8;    // loads in flight per thread

// A CTA looks up a few tokens' rows; a thread then reads what becomes 16 bytes,
// so that a warp writes 512 bytes in one piece (16 numbers a thread, written in
// two or four pieces, took 71 us for 65536 tokens of 8 heads of 128, not 66), at
// the same place of every row that it has a part of: what hangs on the place is
// worked out once (a division for each piece: 66 us, not 64).
template <typename T>
__global__ void __launch_bounds__(kGatherThreads)
q8_gather_kernel(const __grid_constant__ GatherArgs A) {
  using Raw = typename std::conditional<sizeof(T) == 4, uint32_t, uint2>::type;
  constexpr int kVals = 16 / sizeof(T);
  __shared__ const uint8_t* s_row[2][kGatherTokens];   // a token's first head, NULL: missing
  __shared__ const float* s_scale[kGatherTokens];
  griddep_launch_dependents();   // the next call's first kernel may start its launch
  griddep_wait();                // launched chained: the preceding kernel completed
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * A.per_cta;
  const int tokens = (int)min((int64_t)A.per_cta, A.N - t0);
  if (tid < tokens) {
    const int b = __ldg(A.req + t0 + tid);
    const int64_t x = __ldg(A.pos + t0 + tid);
    int rank = 0, vb = 0, loc = 0;
    int64_t page = -1;
    if (b >= 0 && b < A.B && x >= 0 && x < (int64_t)A.max_vb * A.S.vbs && x < INT32_MAX) {
      A.S.place((int)x, rank, vb, loc);
      page = __ldg(A.bt + rank * A.bt_stride + (int64_t)b * A.max_vb + vb);
    }
    const bool there = page >= 0 && page < A.nb;
    if (!there) count_error(A.err);
    const int64_t at = (page * A.Hkv * A.S.bs + loc) * A.d;
    s_row[0][tid] = there ? (const uint8_t*)A.pool[0].ptr[rank] + at : nullptr;
    s_row[1][tid] = there ? (const uint8_t*)A.pool[1].ptr[rank] + at : nullptr;
    s_scale[tid] = there ? (const float*)A.sc.ptr[rank] + page * A.Hkv * kScaleFloats : nullptr;
  }
  __syncthreads();
  const int per_row = A.Hkv * A.d / kVals, per_head = A.d / kVals;   // pieces of 16 bytes
  // threads side by side on one row, as many rows at a time as there are threads for
  const int side = min(per_row, kGatherThreads), rows = kGatherThreads / side;
  const int first = tid / side;
  if (first >= rows) return;
  for (int piece = tid - first * side; piece < per_row; piece += side) {
    const int h = piece / per_head;
    const int64_t at = (int64_t)h * A.S.bs * A.d + (piece - h * per_head) * kVals;
    for (int r0 = first; r0 < 2 * tokens; r0 += rows * kGatherDepth) {   // keys, then values
      Raw x[kGatherDepth];
      float s[kGatherDepth];
#pragma unroll
      for (int j = 0; j < kGatherDepth; ++j) {
        const int r = r0 + j * rows;
        if (r >= 2 * tokens) break;
        const int which = r >= tokens, t = r - which * tokens;
        const uint8_t* row = s_row[which][t];
        x[j] = Raw{};
        s[j] = 0.f;
        if (row) {   // a missing token is zeros
          x[j] = __ldg(reinterpret_cast<const Raw*>(row + at));
          s[j] = __ldg(s_scale[t] + h * kScaleFloats + which);
        }
      }
#pragma unroll
      for (int j = 0; j < kGatherDepth; ++j) {
        const int r = r0 + j * rows;
        if (r >= 2 * tokens) break;
        const int which = r >= tokens, t = r - which * tokens;
        uint4* out = reinterpret_cast<uint4*>(A.out[which]) + (t0 + t) * per_row + piece;
        float4 y[kVals / 4];
#pragma unroll
        for (int k = 0; k < kVals / 4; ++k) {
          y[k] = e4m3x4_f32(reinterpret_cast<const uint32_t*>(&x[j])[k]);
          y[k] = make_float4(y[k].x * s[j], y[k].y * s[j], y[k].z * s[j], y[k].w * s[j]);
        }
        if (kVals == 4)
          *reinterpret_cast<float4*>(out) = y[0];
        else
          *out = make_uint4(pack_bf16(y[0].x, y[0].y), pack_bf16(y[0].z, y[0].w),
                            pack_bf16(y[kVals / 4 - 1].x, y[kVals / 4 - 1].y),
                            pack_bf16(y[kVals / 4 - 1].z, y[kVals / 4 - 1].w));
      }
    }
  }
}

static bool kv8_ok(const dcp_layout_t& L, const dcp_paged_kv8_t& kv) {
  return kv.num_blocks >= 0 && kv.max_vblocks >= 0 && kv.bt_rank_stride >= 0 && kv.block_table &&
         ranks_ok(kv.k, L.dcp_size) && ranks_ok(kv.v, L.dcp_size) && ranks_ok(kv.scale, L.dcp_size);
}

static bool kv8_aligned(const dcp_layout_t& L, const dcp_paged_kv8_t& kv) {
  for (int r = 0; r < L.dcp_size; ++r)
    if (((uintptr_t)kv.k.ptr[r] | (uintptr_t)kv.v.ptr[r] | (uintptr_t)kv.scale.ptr[r]) & 15)
      return false;
  return true;
}

// Whether a span lies over the pools or the scales.
static bool over_cache(const dcp_layout_t& L, const dcp_paged_kv8_t& kv, int Hkv, int d,
                       const Bytes& x) {
  const int64_t ph = kv.num_blocks * Hkv, pool = ph * L.block_size * d;
  for (int r = 0; r < L.dcp_size; ++r)
    if (overlap(x, {kv.k.ptr[r], pool}) || overlap(x, {kv.v.ptr[r], pool}) ||
        overlap(x, {kv.scale.ptr[r], ph * kScaleFloats * 4}))
      return true;
  return false;
}

static bool head_ok(int Hkv, int d) {
  return Hkv >= 1 && d >= 32 && d % 32 == 0 && d <= 256;
}

}  // namespace dcp

using namespace dcp;

extern "C" {

int dcp_q8_append_gqa(dcp_layout_t layout, const void* k, int64_t k_stride, const void* v,
                      int64_t v_stride, int32_t num_tokens, const int32_t* q_start,
                      const int32_t* ctx_lens, int32_t num_reqs, int32_t num_kv_heads,
                      int32_t head_dim, dcp_dtype_t dtype, dcp_paged_kv8_t kv, int32_t* err_count,
                      dcp_stream_t stream) {
  dcp::NvtxRange nvtx_range("dcp_q8_append_gqa");
  if (!shards_ok(layout) || !head_ok(num_kv_heads, head_dim) || num_tokens < 0 || num_reqs < 0 ||
      (dtype != DCP_F32 && dtype != DCP_BF16))
    return DCP_EINVAL;
  const int64_t row = (int64_t)num_kv_heads * head_dim, es = dtype == DCP_F32 ? 4 : 2;
  if (k_stride < row || v_stride < row) return DCP_EINVAL;
  if (num_tokens == 0 || num_reqs == 0) return DCP_OK;
  if (!k || !v || !q_start || !ctx_lens || !kv8_ok(layout, kv)) return DCP_EINVAL;
  if ((uintptr_t)k % 16 || (uintptr_t)v % 16 || k_stride * es % 16 || v_stride * es % 16 ||
      !kv8_aligned(layout, kv) || num_kv_heads > 65535)
    return DCP_EUNSUPPORTED;
  const Bytes reads[] = {{k, ((num_tokens - 1) * k_stride + row) * es},
                         {v, ((num_tokens - 1) * v_stride + row) * es},
                         {q_start, ((int64_t)num_reqs + 1) * 4},
                         {ctx_lens, (int64_t)num_reqs * 4}};
  for (const Bytes& x : reads)
    if (over_cache(layout, kv, num_kv_heads, head_dim, x)) return DCP_EINVAL;
  AppendArgs A;
  A.S = Shards(layout);
  A.src[0] = k, A.src[1] = v;
  A.stride[0] = k_stride * es, A.stride[1] = v_stride * es;
  A.pool[0] = kv.k, A.pool[1] = kv.v, A.sc = kv.scale;
  A.start = q_start, A.ctx = ctx_lens;
  A.N = num_tokens, A.B = num_reqs, A.Hkv = num_kv_heads, A.d = head_dim;
  A.bt = kv.block_table, A.max_vb = kv.max_vblocks, A.bt_stride = kv.bt_rank_stride;
  A.nb = kv.num_blocks;
  A.err = err_count;
  // one token a warp while that fills the GPU once over, then up to 16
  const int64_t fill = (int64_t)num_sms() * 64;
  A.per_warp = 1;
  while (A.per_warp < 16 &&
         ((int64_t)num_tokens + A.per_warp - 1) / A.per_warp * num_kv_heads * 2 > fill)
    A.per_warp *= 2;
  // a token a warp: CTAs of four warps (32 tokens 3.4 us, of eight 3.7); else of eight
  const cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e =
      A.per_warp == 1
          ? (dtype == DCP_F32 ? launch_append<float, 4>(A, st) : launch_append<__nv_bfloat16, 4>(A, st))
          : (dtype == DCP_F32 ? launch_append<float, 8>(A, st)
                              : launch_append<__nv_bfloat16, 8>(A, st));
  if (e != cudaSuccess) return launch_status_report(e);
  return launch_status();
}

int dcp_q8_gather_gqa(dcp_layout_t layout, dcp_paged_kv8_t kv, int32_t num_reqs,
                      int32_t num_kv_heads, int32_t head_dim, const int32_t* req_idx,
                      const int64_t* positions, int64_t num_tokens, void* k_out, void* v_out,
                      dcp_dtype_t dtype, int32_t* err_count, dcp_stream_t stream) {
  dcp::NvtxRange nvtx_range("dcp_q8_gather_gqa");
  if (!shards_ok(layout) || !head_ok(num_kv_heads, head_dim) || num_tokens < 0 || num_reqs < 0 ||
      (dtype != DCP_F32 && dtype != DCP_BF16))
    return DCP_EINVAL;
  if (num_tokens == 0) return DCP_OK;
  if (!req_idx || !positions || !k_out || !v_out || !kv8_ok(layout, kv)) return DCP_EINVAL;
  const int64_t row = (int64_t)num_kv_heads * head_dim, es = dtype == DCP_F32 ? 4 : 2;
  if ((uintptr_t)k_out % 16 || (uintptr_t)v_out % 16 || !kv8_aligned(layout, kv) ||
      num_tokens >= (int64_t(1) << 31) || row > (1 << 20))
    return DCP_EUNSUPPORTED;
  const Bytes ko = {k_out, num_tokens * row * es}, vo = {v_out, num_tokens * row * es};
  if (!apart({ko, vo}, {{req_idx, num_tokens * 4}, {positions, num_tokens * 8}}) ||
      over_cache(layout, kv, num_kv_heads, head_dim, ko) ||
      over_cache(layout, kv, num_kv_heads, head_dim, vo))
    return DCP_EINVAL;
  GatherArgs A;
  A.S = Shards(layout);
  A.pool[0] = kv.k, A.pool[1] = kv.v, A.sc = kv.scale;
  A.bt = kv.block_table, A.max_vb = kv.max_vblocks, A.bt_stride = kv.bt_rank_stride;
  A.nb = kv.num_blocks;
  A.B = num_reqs, A.Hkv = num_kv_heads, A.d = head_dim;
  A.req = req_idx, A.pos = positions, A.N = num_tokens;
  A.out[0] = k_out, A.out[1] = v_out;
  A.err = err_count;
  // a token a CTA while they all run at once, then up to sixteen (65536 tokens of 8 heads of 128
  // take 64 us, with 8 or 32 a CTA 69 or 66)
  const int64_t fill = (int64_t)num_sms() * 16;
  A.per_cta = 1;
  while (A.per_cta < kGatherTokens && (num_tokens + A.per_cta - 1) / A.per_cta > fill) A.per_cta *= 2;
  const unsigned grid = (unsigned)((num_tokens + A.per_cta - 1) / A.per_cta);
  const cudaError_t e =
      dtype == DCP_F32
          ? launch_chained(q8_gather_kernel<float>, grid, kGatherThreads, 0, (cudaStream_t)stream, A)
          : launch_chained(q8_gather_kernel<__nv_bfloat16>, grid, kGatherThreads, 0,
                           (cudaStream_t)stream, A);
  if (e != cudaSuccess) return launch_status_report(e);
  return launch_status();
}

}  // extern "C"
