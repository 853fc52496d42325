// ts_kv_page_bounds: the bounds of each page's keys, kept beside the pages for
// ts_select_pages.
//
// Of a page and kv head, over the page's tokens that the sequence holds:
//   M[d] = max_t K[t, d],  m[d] = min_t K[t, d],  s = max(max |M|, max |m|, 1e-10) / 127,
// kept as 8-bit codes ceil(M / s) and floor(m / s) and the float32 scale s.
// Rounding outward keeps them bounds of the keys.
//
// A new token changes its own page alone, so a call takes the pages that hold a
// row of the batch: row r is a page's first of the batch if it is its sequence's
// first, or the first of the page. Pages are computed anew from their K rows, so
// a call may be repeated, and a page given to another sequence needs no reset.
//
// HBM bounds a prompt step, latency a decode step: 15,000 rows of 8 x 128 in bf16 7.3
// us (38 MB, 5.1 TB/s; from a cold L2 14 us under a profiler), in float32 9.4 us (74 MB,
// 7.8 TB/s out of L2; cold 20 us), one new row of each of 64 sequences 2.6 us (float32
// 2.9), of which three dependent lookups and the launch are most.
// Extremes stay packed, two bf16 an instruction that keeps a NaN; with widened values
// and a division each, 15,000 rows took 18 us.
#include "ts_ragged.cuh"

namespace ts {
namespace {

constexpr int kWarps = 8;  // per CTA, one kv head each

struct BoundsParams {
  int8_t* bounds;
  float* scale;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* q_indptr;
  int32_t bt_stride, T, B, H_kv, num_pages, span;
  PageSize page_size;
};

// Running maxima and minima of 16 bytes of K a row; NaN once there is one.
template <typename T>
struct Extremes;
template <>
struct Extremes<__nv_bfloat16> {
  __nv_bfloat162 top[4], low[4];
  __device__ __forceinline__ Extremes() {
#pragma unroll
    for (int i = 0; i < 4; ++i) set(top[i], 0xff80ff80u), set(low[i], 0x7f807f80u);  // -inf, +inf
  }
  __device__ __forceinline__ static void set(__nv_bfloat162& x, uint32_t w) {
    x = *reinterpret_cast<__nv_bfloat162*>(&w);
  }
  __device__ __forceinline__ void add(const uint4& w) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 x;
      set(x, u[i]);
      top[i] = __hmax2_nan(top[i], x);
      low[i] = __hmin2_nan(low[i], x);
    }
  }
  __device__ __forceinline__ void join(int o) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      top[i] = __hmax2_nan(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
      low[i] = __hmin2_nan(low[i], __shfl_xor_sync(0xffffffffu, low[i], o));
    }
  }
  __device__ __forceinline__ void get(float (&x)[8], bool upper) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(upper ? top[i] : low[i]);
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
};
template <>
struct Extremes<float> {
  float top[4], low[4];
  __device__ __forceinline__ Extremes() {
#pragma unroll
    for (int i = 0; i < 4; ++i) top[i] = -INFINITY, low[i] = INFINITY;
  }
  __device__ __forceinline__ static void max_of(float& x, float y) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(y));
  }
  __device__ __forceinline__ static void min_of(float& x, float y) {
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(y));
  }
  __device__ __forceinline__ void add(const uint4& w) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) max_of(top[i], __uint_as_float(u[i])), min_of(low[i], __uint_as_float(u[i]));
  }
  __device__ __forceinline__ void join(int o) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      max_of(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
      min_of(low[i], __shfl_xor_sync(0xffffffffu, low[i], o));
    }
  }
  __device__ __forceinline__ void get(float (&x)[4], bool upper) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = upper ? top[i] : low[i];
  }
};

// Codes of n bounds, outward: ceil (upper) or floor of x / scale, within +-127; 0 where the scale is not
// finite. `exact`: by a division each, for quotients that quotients() may not round as one.
template <int N>
__device__ __forceinline__ void store_codes(int8_t* to, const float (&x)[N], float scale, bool upper, bool exact) {
  uint32_t byte[N];
  const float inv = reciprocal(scale), sign = upper ? 1.f : -1.f;  // floor(y) = -ceil(-y)
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    float2 y = quotients(make_float2(x[i], x[i + 1]), make_float2(-scale, -scale), make_float2(inv, inv));
    if (exact) y = make_float2(__fdiv_rn(x[i], scale), __fdiv_rn(x[i + 1], scale));
    // 1.5 * 2^23 more: the whole number is in the last bits
    byte[i] = __float_as_uint(fmaf(sign, fminf(ceilf(y.x * sign), 127.f), 12582912.f));
    byte[i + 1] = __float_as_uint(fmaf(sign, fminf(ceilf(y.y * sign), 127.f), 12582912.f));
  }
  uint32_t w[N / 4];
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    w[i] = scale < INFINITY ? __byte_perm(__byte_perm(byte[4 * i], byte[4 * i + 1], 0x0040),
                                          __byte_perm(byte[4 * i + 2], byte[4 * i + 3], 0x0040), 0x5410)
                            : 0u;
  if constexpr (N == 8)
    *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(to) = w[0];
}

// A warp takes `span` rows of the batch and one kv head; a row of D values is
// held by kLanes lanes of 16 bytes, kRows rows at a time.
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32, 4) page_bounds_kernel(const T* k_pool, const BoundsParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  constexpr int kLanes = D * static_cast<int>(sizeof(T)) / 16, kRows = 32 / kLanes, kEach = 16 / sizeof(T);
  constexpr int kAhead = 16 / kRows;  // loads in flight: sixteen rows
  const int lane = threadIdx.x & 31;
  const int h = blockIdx.y * kWarps + (threadIdx.x >> 5);
  if (h >= p.H_kv) return;
  const int ps = p.page_size.rows;
  // lane i looks at row i of the span: is it the first of its page in this batch?
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * p.span, r = r0 + lane;
  const int base = max(0, ragged_floor(p.q_indptr, p.B, static_cast<int>(r0), lane));
  int b = base;
  if (p.span > 1) {  // sequences that begin inside the span
    const int at = base + 1 + lane;
    const int begins = at < p.B ? p.q_indptr[at] : 0x7fffffff;
    const int inside = __popc(__ballot_sync(0xffffffffu, begins < r0 + 32));
    for (int k = 0; k < inside; ++k) b += __shfl_sync(0xffffffffu, begins, k) <= r;
    if (inside == 32) {  // (many empty ones: search on)
      int hi = p.B;
      while (hi - b > 1) {
        const int mid = (b + hi) >> 1;
        if (p.q_indptr[mid] <= r)
          b = mid;
        else
          hi = mid;
      }
    }
  }
  int page = -1, count = 0;
  if (lane < p.span && r < p.T) {
    const int first = p.q_indptr[b], end = p.q_indptr[b + 1];
    if (first <= r && r < end) {
      const int L = p.seq_lens[b], pos = L - (end - static_cast<int>(r));
      const int slot = p.page_size.shift >= 0 ? pos >> p.page_size.shift : pos / ps;
      const int at = pos - slot * ps;
      if (pos >= 0 && (r == first || at == 0) && slot < p.bt_stride) {
        page = p.block_table[static_cast<int64_t>(b) * p.bt_stride + slot];
        if (page >= p.num_pages) page = -1;
        count = min(ps, L - slot * ps);
      }
    }
  }
  unsigned todo = __ballot_sync(0xffffffffu, page >= 0);
  const int l = lane % kLanes, sub = lane / kLanes;
  while (todo) {
    const int from = __ffs(todo) - 1;
    todo &= todo - 1;
    const int64_t pg = __shfl_sync(0xffffffffu, page, from);
    const int n = __shfl_sync(0xffffffffu, count, from);
    const uint4* k = reinterpret_cast<const uint4*>(k_pool + (pg * ps * p.H_kv + h) * D) + l;
    const int64_t step = static_cast<int64_t>(p.H_kv) * D * sizeof(T) / 16;
    Extremes<T> e;
    for (int t0 = sub; t0 < n; t0 += kAhead * kRows) {
      uint4 w[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) w[u] = k[min(t0 + u * kRows, n - 1) * step];  // (a row again changes nothing)
#pragma unroll
      for (int u = 0; u < kAhead; ++u) e.add(w[u]);
    }
#pragma unroll
    for (int o = 16; o >= kLanes; o >>= 1) e.join(o);
    float top[kEach], low[kEach];
    e.get(top, true);
    e.get(low, false);
    uint32_t largest = 0u, least = 0xffffffffu;  // magnitudes order as their bits do, NaN above all
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const uint32_t a = __float_as_uint(top[i]) & 0x7fffffffu, c = __float_as_uint(low[i]) & 0x7fffffffu;
      largest = max(largest, max(a, c));
      least = min(least, min(a - 1u, c - 1u));  // (zeros last)
    }
    largest = __reduce_max_sync(0xffffffffu, largest);
    const float scale = largest >= 0x7f800000u ? INFINITY : fmaxf(__uint_as_float(largest), 1e-10f) * (1.f / 127.f);
    // quotients below 2^-11, and scales whose reciprocal may not be the rounded one: see quotient()
    const bool exact = __any_sync(0xffffffffu, least != 0xffffffffu && __uint_as_float(least) < scale * 0x1p-11f) ||
                       all_ones(scale);
    int8_t* to = p.bounds + (pg * p.H_kv + h) * 2 * D + l * kEach;
    if (kRows == 1) {
      store_codes(to, top, scale, true, exact);
      store_codes(to + D, low, scale, false, exact);
    } else if (sub < 2) {  // a half each
      const bool upper = sub == 0;
      float x[kEach];
#pragma unroll
      for (int i = 0; i < kEach; ++i) x[i] = upper ? top[i] : low[i];
      store_codes(to + sub * D, x, scale, upper, exact);
    }
    if (lane == 0) p.scale[pg * p.H_kv + h] = scale;
  }
}

template <typename T>
ts_status launch(int D, const void* k_pool, const BoundsParams& p, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.T - 1) / p.span + 1), static_cast<unsigned>((p.H_kv - 1) / kWarps + 1));
  cfg.blockDim = dim3(32 * (p.H_kv < kWarps ? p.H_kv : kWarps));
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kern = D == 64 ? page_bounds_kernel<T, 64> : page_bounds_kernel<T, 128>;
  LaunchTrace trace("page_bounds_kernel", stream);
  return cuda_check(cudaLaunchKernelEx(&cfg, kern, static_cast<const T*>(k_pool), p), "ts_kv_page_bounds: launch");
}

}  // namespace
}  // namespace ts

extern "C" ts_status ts_kv_page_bounds(const void* k_pool, int8_t* bounds, float* bound_scale,
                                       const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens,
                                       const int32_t* q_indptr, int32_t T, int32_t B, int32_t H_kv, int32_t D,
                                       int32_t page_size, int32_t num_pages, ts_dtype dtype, void* stream) {
  using namespace ts;
  const char* who = "ts_kv_page_bounds";
  if (T < 0 || B < 0 || H_kv <= 0 || D <= 0 || page_size <= 0 || num_pages <= 0 || bt_stride <= 0)
    return fail(TS_ERR_INVALID_ARG, "%s: bad sizes (T=%d B=%d H_kv=%d D=%d ps=%d P=%d bt=%d)", who, T, B, H_kv, D,
                page_size, num_pages, bt_stride);
  if (dtype != TS_F32 && dtype != TS_BF16)
    return fail(TS_ERR_INVALID_ARG, "%s: bad dtype %d", who, static_cast<int>(dtype));
  if (D != 64 && D != 128) return fail(TS_ERR_UNSUPPORTED, "%s: D=%d (supported 64, 128)", who, D);
  if (H_kv > 4096) return fail(TS_ERR_UNSUPPORTED, "%s: more than 4096 heads", who);
  if (T == 0 || B == 0) return TS_OK;
  if (!k_pool || !bounds || !bound_scale || !block_table || !seq_lens || !q_indptr)
    return fail(TS_ERR_INVALID_ARG, "%s: null pointer", who);
  for (const void* x : {k_pool, static_cast<const void*>(bounds)})
    if (reinterpret_cast<uintptr_t>(x) % 16 != 0)
      return fail(TS_ERR_INVALID_ARG, "%s: pool and bounds must be 16-byte aligned", who);
  if (reinterpret_cast<uintptr_t>(bound_scale) % 4 != 0)
    return fail(TS_ERR_INVALID_ARG, "%s: scales must be 4-byte aligned", who);
  // Few rows: a warp each, so that the pages of a decode step are taken at once (64 rows: 2.6 us); many: a warp
  // looks 16 over for the first of each page (15,000 rows: 7.3 us, with 8 8.9, with 32 10.6, a warp each 27).
  const int span = T <= 2048 ? 1 : 16;
  const BoundsParams p{bounds, bound_scale, block_table, seq_lens, q_indptr, bt_stride, T,
                       B,      H_kv,        num_pages,   span,     PageSize(page_size)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == TS_BF16 ? launch<__nv_bfloat16>(D, k_pool, p, s) : launch<float>(D, k_pool, p, s);
}
