// ts_paged_decode_sparse_attn: decode attention over chosen pages, a list for
// every query row and kv head (ts_select_pages makes them).
//
// Of a query row at position p, over the tokens t <= p of the listed pages:
//   s_t = scale * <q, K_t>,  O = sum_t softmax(s)_t V_t,  LSE = log sum_t exp(s_t).
//
// A work item is a query row and kv head; its list is cut into `parts` equal
// ranges, one CTA each, so that few rows fill the device. The warps of a CTA take
// the listed pages in turn, a page's rows kRows at a time: 16 bytes of a row per
// lane, the g query heads in registers, a running maximum and sum per group of
// lanes. States are joined over lanes, then warps, then (parts > 1) by a second
// kernel from float32 states in the workspace.
#include "ts_common.cuh"

#include <cmath>

namespace ts {
namespace {

constexpr int kWarps = 4;
constexpr float kLog2eS = 1.4426950408889634f;
constexpr float kLn2S = 0.6931471805599453f;

struct SparseParams {
  const void* q;
  const void* k_pool;
  const void* v_pool;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* page_idx;
  void* out;
  float* lse;
  float* part_o;    // [parts, rows, H_q, D]
  float* part_lse;  // [parts, rows, H_q], base 2
  uint32_t* err_word;
  int32_t bt_stride, rows, q_len, H_kv, page_size, num_pages, pages, parts;
  float scale_log2;
};

template <typename T>
__device__ __forceinline__ void widen(const uint4& w, float (&x)[16 / sizeof(T)]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      const float2 f = bf16x2_to_float2(u[i]);
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    } else {
      x[i] = __uint_as_float(u[i]);
    }
  }
}

template <typename T>
__device__ __forceinline__ void store4(T* to, float4 v) {
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint2*>(to) = make_uint2(float2_to_bf16x2(v.x, v.y), float2_to_bf16x2(v.z, v.w));
  else
    *reinterpret_cast<float4*>(to) = v;
}

// A listed page: its pool page and how many of its tokens the row sees (0: none).
struct Listed {
  int32_t page, tokens;
};
__device__ __forceinline__ Listed listed_page(const SparseParams& p, int idx, int b, int pos) {
  Listed e{0, 0};
  if (idx < 0 || static_cast<int64_t>(idx) * p.page_size > pos) return e;
  const int page = idx < p.bt_stride ? p.block_table[static_cast<int64_t>(b) * p.bt_stride + idx] : -1;
  if (page < 0 || page >= p.num_pages) {
    set_device_error(p.err_word, TS_DEVERR_PAGE_RANGE);
    return e;
  }
  e.page = page;
  e.tokens = min(p.page_size, pos - idx * p.page_size + 1);
  return e;
}

template <typename T, int D, int G>
__global__ void __launch_bounds__(kWarps * 32) sparse_decode_kernel(const SparseParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  constexpr int kEach = 16 / static_cast<int>(sizeof(T)), kLanes = D / kEach, kRows = 32 / kLanes, kAhead = 4;
  __shared__ float sh_m[kWarps][G], sh_l[kWarps][G];
  __shared__ __align__(16) float sh_o[kWarps][G][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % kLanes, sub = lane / kLanes;
  const int64_t item = blockIdx.x / static_cast<unsigned>(p.parts);
  const int part = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.parts));
  const int row = static_cast<int>(item / p.H_kv), h = static_cast<int>(item % p.H_kv);
  const int b = row / p.q_len, pos = p.seq_lens[b] - p.q_len + (row - b * p.q_len);
  const int H_q = p.H_kv * G;

  float q[G][kEach], acc[G][kEach], m[G], sum[G];
  const T* qsrc = static_cast<const T*>(p.q) + (static_cast<int64_t>(row) * H_q + h * G) * D + l * kEach;
#pragma unroll
  for (int i = 0; i < G; ++i) {
    widen<T>(*reinterpret_cast<const uint4*>(qsrc + i * D), q[i]);
    m[i] = -INFINITY;
    sum[i] = 0.f;
#pragma unroll
    for (int d = 0; d < kEach; ++d) acc[i][d] = 0.f, q[i][d] *= p.scale_log2;
  }
  const int32_t* list = p.page_idx + item * p.pages;
  const int i0 = static_cast<int>(static_cast<int64_t>(p.pages) * part / p.parts);
  const int i1 = static_cast<int>(static_cast<int64_t>(p.pages) * (part + 1) / p.parts);
  const int64_t step = static_cast<int64_t>(p.H_kv) * D;  // elements between rows
  for (int c0 = i0 + warp; c0 < i1; c0 += 32 * kWarps) {
    // lane i looks up the i-th of this warp's next 32 entries
    const int mine = c0 + lane * kWarps;
    const Listed e = mine < i1 ? listed_page(p, list[mine], b, pos) : Listed{0, 0};
    for (unsigned todo = __ballot_sync(0xffffffffu, e.tokens > 0); todo; todo &= todo - 1) {
      const int from = __ffs(todo) - 1;
      const int64_t page = __shfl_sync(0xffffffffu, e.page, from);
      const int n = __shfl_sync(0xffffffffu, e.tokens, from);
      const int64_t base = (page * p.page_size * p.H_kv + h) * D + l * kEach;
      const T* kp = static_cast<const T*>(p.k_pool) + base;
      const T* vp = static_cast<const T*>(p.v_pool) + base;
      for (int t0 = sub; t0 - sub < n; t0 += kAhead * kRows) {
        uint4 kw[kAhead], vw[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int64_t at = min(t0 + u * kRows, n - 1) * step;
          kw[u] = *reinterpret_cast<const uint4*>(kp + at);
          vw[u] = *reinterpret_cast<const uint4*>(vp + at);
        }
        float s[kAhead][G];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          float x[kEach];
          widen<T>(kw[u], x);
#pragma unroll
          for (int i = 0; i < G; ++i) {
            float d = q[i][0] * x[0];
#pragma unroll
            for (int j = 1; j < kEach; ++j) d = fmaf(q[i][j], x[j], d);
            s[u][i] = d;
          }
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < G; ++i) s[u][i] += __shfl_xor_sync(0xffffffffu, s[u][i], o);
          if (t0 + u * kRows >= n) {
#pragma unroll
            for (int i = 0; i < G; ++i) s[u][i] = -INFINITY;
          }
        }
#pragma unroll
        for (int i = 0; i < G; ++i) {
          float top = m[i];
#pragma unroll
          for (int u = 0; u < kAhead; ++u) top = fmaxf(top, s[u][i]);
          const float ref = top == -INFINITY ? 0.f : top;
          const float scale = fast_exp2(m[i] - ref);
          m[i] = top;
          sum[i] *= scale;
#pragma unroll
          for (int j = 0; j < kEach; ++j) acc[i][j] *= scale;
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            s[u][i] = fast_exp2(s[u][i] - ref);
            sum[i] += s[u][i];
          }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if (t0 + u * kRows >= n) continue;  // (what such rows hold must not count, not even NaN)
          float x[kEach];
          widen<T>(vw[u], x);
#pragma unroll
          for (int i = 0; i < G; ++i)
#pragma unroll
            for (int j = 0; j < kEach; ++j) acc[i][j] = fmaf(s[u][i], x[j], acc[i][j]);
        }
      }
    }
  }
  // joined over the groups of lanes
#pragma unroll
  for (int o = 16; o >= kLanes; o >>= 1) {
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m[i], o), top = fmaxf(m[i], m2);
      const float ref = top == -INFINITY ? 0.f : top;
      const float a = fast_exp2(m[i] - ref), c = fast_exp2(m2 - ref);
      m[i] = top;
      sum[i] = a * sum[i] + c * __shfl_xor_sync(0xffffffffu, sum[i], o);
#pragma unroll
      for (int j = 0; j < kEach; ++j) acc[i][j] = a * acc[i][j] + c * __shfl_xor_sync(0xffffffffu, acc[i][j], o);
    }
  }
  if (sub == 0) {
#pragma unroll
    for (int i = 0; i < G; ++i) {
      if (l == 0) sh_m[warp][i] = m[i], sh_l[warp][i] = sum[i];
#pragma unroll
      for (int j = 0; j < kEach; ++j) sh_o[warp][i][l * kEach + j] = acc[i][j];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < G * D / 4; e += kWarps * 32) {
    const int i = e / (D / 4), d = e % (D / 4) * 4;
    float top = sh_m[0][i];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sh_m[w][i]);
    const float ref = top == -INFINITY ? 0.f : top;
    float total = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float a = fast_exp2(sh_m[w][i] - ref);
      const float4 x = *reinterpret_cast<const float4*>(&sh_o[w][i][d]);
      total = fmaf(a, sh_l[w][i], total);
      o = make_float4(fmaf(a, x.x, o.x), fmaf(a, x.y, o.y), fmaf(a, x.z, o.z), fmaf(a, x.w, o.w));
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;  // (NaN stays NaN)
    o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    const float lse2 = total == 0.f ? -INFINITY : ref + log2f(total);
    const int64_t at = static_cast<int64_t>(row) * H_q + h * G + i;
    if (p.parts == 1) {
      store4(static_cast<T*>(p.out) + at * D + d, o);
      if (d == 0 && p.lse != nullptr) p.lse[at] = lse2 * kLn2S;
    } else {
      const int64_t to = static_cast<int64_t>(part) * p.rows * H_q + at;
      *reinterpret_cast<float4*>(p.part_o + to * D + d) = o;
      if (d == 0) p.part_lse[to] = lse2;
    }
  }
}

// Joins the parts of a query head: D / 4 threads each.
template <typename T, int D>
__global__ void __launch_bounds__(128) sparse_merge_kernel(const SparseParams p, int32_t heads) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int64_t e = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
  const int64_t at = e / (D / 4), total_heads = static_cast<int64_t>(p.rows) * heads;
  const int d = static_cast<int>(e % (D / 4)) * 4;
  if (at >= total_heads) return;
  float top = -INFINITY;
  for (int i = 0; i < p.parts; ++i) top = fmaxf(top, p.part_lse[i * total_heads + at]);
  const float ref = top == -INFINITY ? 0.f : top;
  float total = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < p.parts; ++i) {
    const float a = fast_exp2(p.part_lse[i * total_heads + at] - ref);
    const float4 x = *reinterpret_cast<const float4*>(p.part_o + (i * total_heads + at) * D + d);
    total += a;
    o = make_float4(fmaf(a, x.x, o.x), fmaf(a, x.y, o.y), fmaf(a, x.z, o.z), fmaf(a, x.w, o.w));
  }
  const float inv = total == 0.f ? 0.f : 1.f / total;
  store4(static_cast<T*>(p.out) + at * D + d, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
  if (d == 0 && p.lse != nullptr) p.lse[at] = total == 0.f ? -INFINITY : (ref + log2f(total)) * kLn2S;
}

// Parts of each list: so many CTAs that the device is filled, each with a page
// per warp at least.
int sparse_parts(int64_t items, int pages) {
  const int64_t want = (static_cast<int64_t>(paged_decode_ctas()) * 4 + items - 1) / (items > 0 ? items : 1);
  const int64_t most = (pages + kWarps - 1) / kWarps;
  return static_cast<int>(want < 1 ? 1 : want > most ? most : want);
}

size_t sparse_bytes(int64_t rows, int H_q, int D, int parts) {
  const size_t states = parts > 1 ? static_cast<size_t>(parts) * rows * H_q * (D + 1) * sizeof(float) : 0;
  return align_up(kWorkspaceAlign + states, kWorkspaceAlign);
}

template <typename K, typename... A>
cudaError_t launch_pdl(K kern, unsigned grid, int threads, cudaStream_t stream, A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename T, int D>
ts_status launch(int g, const SparseParams& p, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(p.rows) * p.H_kv * p.parts);
  {
    LaunchTrace trace("sparse_decode_kernel", s);
    const auto kern = g == 1   ? sparse_decode_kernel<T, D, 1>
                      : g == 2 ? sparse_decode_kernel<T, D, 2>
                      : g == 4 ? sparse_decode_kernel<T, D, 4>
                               : sparse_decode_kernel<T, D, 8>;
    const ts_status st = cuda_check(launch_pdl(kern, grid, kWarps * 32, s, p), "ts_paged_decode_sparse_attn: launch");
    if (st != TS_OK || p.parts == 1) return st;
  }
  const int64_t threads = static_cast<int64_t>(p.rows) * p.H_kv * g * (D / 4);
  LaunchTrace trace("sparse_merge_kernel", s);
  return cuda_check(launch_pdl(sparse_merge_kernel<T, D>, static_cast<unsigned>((threads - 1) / 128 + 1), 128, s, p,
                               p.H_kv * g),
                    "ts_paged_decode_sparse_attn: merge launch");
}

bool supported(int H_q, int H_kv, int D, int page_size) {
  const int g = H_kv > 0 && H_q % H_kv == 0 ? H_q / H_kv : 0;
  return (D == 64 || D == 128) && (g == 1 || g == 2 || g == 4 || g == 8) &&
         (H_kv == 1 || H_kv == 2 || H_kv == 4 || H_kv == 8) &&
         (page_size == 8 || page_size == 16 || page_size == 32);
}

}  // namespace
}  // namespace ts

extern "C" size_t ts_paged_decode_sparse_workspace_size(int32_t B, int32_t q_len, int32_t H_q, int32_t H_kv,
                                                        int32_t D, int32_t page_size, int32_t pages) {
  using namespace ts;
  const int64_t rows = static_cast<int64_t>(B) * q_len;
  if (B < 0 || q_len <= 0 || pages <= 0 || rows > (1 << 24) || !supported(H_q, H_kv, D, page_size)) return 0;
  return sparse_bytes(rows, H_q, D, sparse_parts(rows * H_kv, pages));
}

extern "C" ts_status ts_paged_decode_sparse_attn(const void* q, const void* k_pool, const void* v_pool,
                                                 const int32_t* block_table, int32_t bt_stride,
                                                 const int32_t* seq_lens, const int32_t* page_idx, int32_t pages,
                                                 int32_t B, int32_t q_len, int32_t H_q, int32_t H_kv, int32_t D,
                                                 int32_t page_size, int32_t num_pages, float scale, ts_dtype dtype,
                                                 void* out, float* lse, void* workspace, size_t workspace_bytes,
                                                 void* stream) {
  using namespace ts;
  const char* who = "ts_paged_decode_sparse_attn";
  if (B < 0 || q_len <= 0 || H_q <= 0 || H_kv <= 0 || D <= 0 || page_size <= 0 || num_pages <= 0 ||
      bt_stride <= 0 || pages <= 0)
    return fail(TS_ERR_INVALID_ARG, "%s: bad sizes (B=%d q_len=%d H_q=%d H_kv=%d D=%d ps=%d P=%d bt=%d pages=%d)",
                who, B, q_len, H_q, H_kv, D, page_size, num_pages, bt_stride, pages);
  if (H_q % H_kv != 0) return fail(TS_ERR_INVALID_ARG, "%s: H_q=%d not a multiple of H_kv=%d", who, H_q, H_kv);
  if (static_cast<int64_t>(num_pages) * page_size >= (1ll << 31))
    return fail(TS_ERR_INVALID_ARG, "%s: num_pages * page_size must stay below 2^31", who);
  if (dtype != TS_F32 && dtype != TS_BF16)
    return fail(TS_ERR_INVALID_ARG, "%s: bad dtype %d", who, static_cast<int>(dtype));
  if (!std::isfinite(scale)) return fail(TS_ERR_INVALID_ARG, "%s: scale is not finite", who);
  if (!supported(H_q, H_kv, D, page_size))
    return fail(TS_ERR_UNSUPPORTED,
                "%s: H_q=%d H_kv=%d D=%d page_size=%d (H_q / H_kv and H_kv in {1, 2, 4, 8}, D in {64, 128}, "
                "page_size in {8, 16, 32})", who, H_q, H_kv, D, page_size);
  const int64_t rows = static_cast<int64_t>(B) * q_len;
  if (rows > (1 << 24)) return fail(TS_ERR_UNSUPPORTED, "%s: more than 2^24 query rows", who);
  if (B == 0) return TS_OK;
  if (!q || !k_pool || !v_pool || !block_table || !seq_lens || !page_idx || !out)
    return fail(TS_ERR_INVALID_ARG, "%s: null pointer", who);
  for (const void* x : {q, k_pool, v_pool, static_cast<const void*>(out)})
    if (reinterpret_cast<uintptr_t>(x) % 16 != 0)
      return fail(TS_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", who);
  const int parts = sparse_parts(rows * H_kv, pages);
  const size_t bytes = sparse_bytes(rows, H_q, D, parts);
  if (!workspace || workspace_bytes < bytes || reinterpret_cast<uintptr_t>(workspace) % kWorkspaceAlign != 0)
    return fail(TS_ERR_WORKSPACE, "%s: workspace %zu B < %zu B needed or misaligned", who, workspace_bytes, bytes);
  float* part_o = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + kWorkspaceAlign);
  const SparseParams p{q, k_pool, v_pool, block_table, seq_lens, page_idx, out, lse, part_o,
                       part_o + static_cast<size_t>(parts) * rows * H_q * D, static_cast<uint32_t*>(workspace),
                       bt_stride, static_cast<int32_t>(rows), q_len, H_kv, page_size, num_pages, pages, parts,
                       scale * kLog2eS};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int g = H_q / H_kv;
  if (dtype == TS_BF16)
    return D == 64 ? launch<__nv_bfloat16, 64>(g, p, s) : launch<__nv_bfloat16, 128>(g, p, s);
  return D == 64 ? launch<float, 64>(g, p, s) : launch<float, 128>(g, p, s);
}
