// The 8-bit cache: keys and values quantised as they are written, and read
// back.  A page and head has one scale for its keys and one for its values, a
// power of two s; a number x is held as the e4m3 number nearest to x / s.
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

template <typename T>
__device__ __forceinline__ float4 quad(const uint4& x, int i);   // numbers 4 i .. 4 i + 3 of 16 bytes
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

// |x| of a finite number, 0 of others.
__device__ __forceinline__ float size_of(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}

constexpr int kAppendWarps = 8;
constexpr int kAppendDepth = 8;    // 16-byte loads in flight per thread

// The tokens that a call writes to one page, for one head and one of K and V,
// are one warp's: it reads them, finds their size and the page's scale, and
// writes them, and if the scale grows also the page's other places.  Which
// tokens those are follows from the request's run of positions, so there is no
// sorting, nothing to clear and no atomic.  A warp looks at a few tokens in a
// row and takes the pages whose turn is one of them: of a page's new tokens the
// (rank * bs / dcp)-th, so that the pages of one virtual block, whose first
// tokens lie side by side, go to different warps.
template <typename T>
__global__ void __launch_bounds__(kAppendWarps * 32)
q8_append_kernel(const __grid_constant__ AppendArgs A) {
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
  if (first >= A.N) return;
  // the request of the first token: starts that lie at or before it
  int at = 0;
#pragma unroll 4
  for (int i = lane; i <= A.B; i += 32) at += __ldg(A.start + i) <= first;
  at = __reduce_add_sync(0xffffffffu, at) - 1;
  // the request of this lane's token, from the starts behind it in order
  const int t = (int)first + lane;
  int b = at;
  for (int base = at + 1;; base += 32) {
    const int s = base + lane <= A.B ? __ldg(A.start + base + lane) : INT32_MAX;
    int n = 0;   // starts <= t, by halves
#pragma unroll
    for (int step = 16; step > 0; step >>= 1) {
      const int x = __shfl_sync(0xffffffffu, s, n + step - 1);
      if (x <= t) n += step;
    }
    n += __shfl_sync(0xffffffffu, s, n & 31) <= t && n < 32;
    b += n;
    if (!__any_sync(0xffffffffu, n == 32)) break;
  }
  // is the token the one that stands for its page?
  bool mine = false;
  int rank = 0, vb = 0, loc0 = 0, n = 0, c = 0, q0 = 0;
  if (lane < A.per_warp && t < A.N && b >= 0 && b < A.B) {
    c = __ldg(A.ctx + b);
    q0 = __ldg(A.start + b);
    const int q1 = __ldg(A.start + b + 1);
    if (usable(c, q0, q1) && t >= q0 && t < q1) {
      int loc;
      A.S.place(c + t - q0, rank, vb, loc);
      const int page0 = vb * A.S.bs;
      loc0 = max(Below(A.S, c).on(A.S, rank) - page0, 0);
      n = min(Below(A.S, c + q1 - q0).on(A.S, rank) - page0, A.S.bs) - loc0;
      mine = loc == loc0 + rank * A.S.bs / A.S.dcp % n;
    }
  }
  const int chunks = A.d * (int)sizeof(T) / 16, rows = max(32 / chunks, 1);
  const int row = lane / chunks, chunk = lane - row * chunks;   // with chunks > 32: row 0
  const bool busy = row < rows;
  constexpr int kOut = 16 / sizeof(T);   // bytes that 16 bytes become
  for (uint32_t todo = __ballot_sync(0xffffffffu, mine); todo; todo &= todo - 1) {
    const int who = __ffs(todo) - 1;
    const int pr = __shfl_sync(0xffffffffu, rank, who), pv = __shfl_sync(0xffffffffu, vb, who);
    const int pl = __shfl_sync(0xffffffffu, loc0, who), pn = __shfl_sync(0xffffffffu, n, who);
    const int pc = __shfl_sync(0xffffffffu, c, who), pq = __shfl_sync(0xffffffffu, q0, who);
    const int pb = __shfl_sync(0xffffffffu, b, who);
    const int64_t page =
        __ldg(A.bt + pr * A.bt_stride + (int64_t)pb * A.max_vb + pv);
    if (page < 0 || page >= A.nb) {
      if (lane == 0 && h == 0 && which == 0) count_error(A.err);
      continue;
    }
    const char* src = (const char*)A.src[which] + (int64_t)h * A.d * sizeof(T);
    const int64_t stride = A.stride[which];
    uint8_t* dst = (uint8_t*)A.pool[which].ptr[pr] + (page * A.Hkv + h) * A.S.bs * A.d;
    float* scale = (float*)A.sc.ptr[pr] + (page * A.Hkv + h) * kScaleFloats + which;
    const float held = pl > 0 ? __ldcg(scale) : 0.f;
    auto load = [&](int i, int ch) {   // place pl + i
      const int64_t tok = pq + (A.S.position(pv, pr, pl + i) - pc);
      return __ldg(reinterpret_cast<const uint4*>(src + tok * stride) + ch);
    };
    uint4 x[kAppendDepth];
    float top = 0.f;
    for (int ch = chunk; ch < chunks; ch += 32) {
      for (int i0 = 0; i0 < pn; i0 += rows * kAppendDepth) {
#pragma unroll
        for (int j = 0; j < kAppendDepth; ++j) {
          const int i = i0 + j * rows + row;
          x[j] = busy && i < pn ? load(i, ch) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int j = 0; j < kAppendDepth; ++j)
#pragma unroll
          for (int k = 0; k < kOut / 4; ++k) {
            const float4 y = quad<T>(x[j], k);
            top = fmaxf(top, fmaxf(fmaxf(size_of(y.x), size_of(y.y)),
                                   fmaxf(size_of(y.z), size_of(y.w))));
          }
      }
    }
    top = warp_max(top);
    // a page that begins, or whose scale is none, keeps nothing
    const float old = held > 0.f && held <= 3.402823466e38f ? held : 0.f;
    const float now = fmaxf(old, scale_for(top));
    const bool grows = old > 0.f && now > old;
    const bool power = (__float_as_uint(now) & 0x7fffffu) == 0;
    const float inv = 1.f / now;     // exact for a power of two; others divide
    auto scaled = [&](float4 y) {
      return power ? make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv)
                   : make_float4(y.x / now, y.y / now, y.z / now, y.w / now);
    };
    const bool once = pn <= rows * kAppendDepth && chunks <= 32;   // still in registers
    for (int ch = chunk; ch < chunks; ch += 32) {
      for (int i0 = 0; i0 < pn; i0 += rows * kAppendDepth) {
        if (!once) {
#pragma unroll
          for (int j = 0; j < kAppendDepth; ++j) {
            const int i = i0 + j * rows + row;
            if (busy && i < pn) x[j] = load(i, ch);
          }
        }
#pragma unroll
        for (int j = 0; j < kAppendDepth; ++j) {
          const int i = i0 + j * rows + row;
          if (!busy || i >= pn) continue;
          uint8_t* to = dst + (int64_t)(pl + i) * A.d + ch * kOut;
          const uint32_t lo = f32x4_e4m3(scaled(quad<T>(x[j], 0)));
          if (kOut == 4)
            *reinterpret_cast<uint32_t*>(to) = lo;
          else
            *reinterpret_cast<uint2*>(to) =
                make_uint2(lo, f32x4_e4m3(scaled(quad<T>(x[j], 1))));
        }
      }
    }
    if (grows) {   // the page's other places, 4 numbers a lane
      const float by = old / now;
      const int quads = A.d / 4;
      for (int i = lane; i < A.S.bs * quads; i += 32) {
        const int l = i / quads;
        if (l >= pl && l < pl + pn) continue;
        uint32_t* to = reinterpret_cast<uint32_t*>(dst) + i;
        const float4 y = e4m3x4_f32(*to);
        *to = f32x4_e4m3(make_float4(y.x * by, y.y * by, y.z * by, y.w * by));
      }
    }
    __syncwarp();
    if (lane == 0) *scale = now;
  }
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
  int per_cta;      // tokens of a CTA, at most 32
  void* out[2];
  int32_t* err;
};

constexpr int kGatherThreads = 256;

// A CTA looks up a few tokens' rows, then its threads take 16 numbers each of a
// token's heads, first the keys and then the values.
template <typename T>
__global__ void __launch_bounds__(kGatherThreads)
q8_gather_kernel(const __grid_constant__ GatherArgs A) {
  __shared__ int s_rank[32], s_loc[32];
  __shared__ int64_t s_page[32];
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
    if (page < 0 || page >= A.nb) {
      page = -1;
      count_error(A.err);
    }
    s_rank[tid] = rank;
    s_loc[tid] = loc;
    s_page[tid] = page;
  }
  __syncthreads();
  const int chunks = A.d / 16, each = A.Hkv * chunks, all = tokens * each * 2;
  for (int i = tid; i < all; i += kGatherThreads) {
    const int tw = i / each, rem = i - tw * each, t = tw >> 1, which = tw & 1;
    const int h = rem / chunks, ch = rem - h * chunks;
    const int64_t page = s_page[t];
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    float s = 0.f;
    if (page >= 0) {
      const int64_t ph = page * A.Hkv + h;
      const int r = s_rank[t];
      x = __ldg(reinterpret_cast<const uint4*>((const uint8_t*)A.pool[which].ptr[r] +
                                               (ph * A.S.bs + s_loc[t]) * A.d) + ch);
      s = __ldg((const float*)A.sc.ptr[r] + ph * kScaleFloats + which);
    }
    // a missing token is zeros
    const uint32_t in[4] = {x.x, x.y, x.z, x.w};
    float4 y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[j] = e4m3x4_f32(in[j]);
      y[j] = page >= 0 ? make_float4(y[j].x * s, y[j].y * s, y[j].z * s, y[j].w * s)
                       : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int64_t at = (((t0 + t) * A.Hkv + h) * A.d + ch * 16) * (int64_t)sizeof(T);
    uint4* to = reinterpret_cast<uint4*>((char*)A.out[which] + at);
    if (sizeof(T) == 4) {
#pragma unroll
      for (int j = 0; j < 4; ++j) reinterpret_cast<float4*>(to)[j] = y[j];
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        to[j] = make_uint4(pack_bf16(y[2 * j].x, y[2 * j].y), pack_bf16(y[2 * j].z, y[2 * j].w),
                           pack_bf16(y[2 * j + 1].x, y[2 * j + 1].y),
                           pack_bf16(y[2 * j + 1].z, y[2 * j + 1].w));
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
  const int64_t warps = ((int64_t)num_tokens + A.per_warp - 1) / A.per_warp;
  const dim3 grid((unsigned)((warps + kAppendWarps - 1) / kAppendWarps), (unsigned)num_kv_heads, 2);
  const cudaError_t e =
      dtype == DCP_F32
          ? launch_chained(q8_append_kernel<float>, grid, kAppendWarps * 32, 0,
                           (cudaStream_t)stream, A)
          : launch_chained(q8_append_kernel<__nv_bfloat16>, grid, kAppendWarps * 32, 0,
                           (cudaStream_t)stream, A);
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
  const int64_t fill = (int64_t)num_sms() * 16;
  A.per_cta = 1;
  while (A.per_cta < 32 && (num_tokens + A.per_cta - 1) / A.per_cta > fill) A.per_cta *= 2;
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
