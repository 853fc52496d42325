// ts_select_pages: the pages of a sequence whose bounds (ts_kv_page_bounds)
// promise most for a query, for ts_paged_decode_sparse_attn.
//
// Of a query head's row q, with qs = max(max |q|, 1e-10) / 127 and the codes
// c = round(q / qs); of a page's codes M', m' and scale s:
//   dot = sum_d max(c[d] M'[d], c[d] m'[d]),   score = max over the g heads of (dot * qs) * s,
// the bound of the products of the quantized query with any of the page's keys.
// dot is a whole number below 2^24 and the two products are float32, each rounded
// once, so that the scores and with them the choice are the same on every run and
// device. A term is c M' where c > 0 and c m' where c < 0: the row [max(c, 0),
// min(c, 0)] times the row [M', m'], four 8-bit products an instruction.
//
// page_score_kernel: HBM bounds it (2 D + 4 bytes a page and head). A warp keeps
// the codes of the g query heads of one kv head in registers; 2 D / 16 lanes take
// a page's bounds, 16 bytes each.
// page_pick_kernel: a CTA per query row and kv head finds the threshold by
// counting in bins that halve no range but cut the remaining one in 2048, then
// lists the pages above it in order; equal scores go to the lowest pages.
#include "ts_common.cuh"

#include <cmath>

namespace ts {
namespace {

constexpr int kWarps = 8, kPickThreads = 512, kPickBins = 2048, kPickSmemKeys = 8192;
constexpr int kSlots = 64;  // pages per scoring CTA

struct SelectParams {
  const int8_t* bounds;
  const float* bound_scale;
  const int32_t* block_table;
  const int32_t* seq_lens;
  uint32_t* keys;  // [rows, H_kv, bt_stride]
  int32_t* page_idx;
  uint32_t* err_word;
  int32_t bt_stride, q_len, H_kv, page_size, num_pages, pages, first, last;
};

// Pages of the query at the row's position, as far as the table has slots; < 0 position: none.
__device__ __forceinline__ int pages_of(const SelectParams& p, int row, bool* past) {
  const int b = row / p.q_len;
  const int pos = p.seq_lens[b] - p.q_len + (row - b * p.q_len);
  if (pos < 0) return 0;
  const int have = pos / p.page_size + 1;
  *past = have > p.bt_stride;
  return min(have, p.bt_stride);
}

// Scores as whole numbers of their order: NaN above all, 0 is no score's.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 becomes 0: they are equal
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <typename T, int D, int G>
__global__ void __launch_bounds__(kWarps * 32) page_score_kernel(const T* __restrict__ q, const SelectParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  constexpr int kL = 2 * D / 16, kU = 32 / kL;  // lanes of a page's bounds, pages at a time
  __shared__ __align__(16) int8_t code[8 * G][2 * D];
  __shared__ float q_scale[8 * G];
  __shared__ int32_t page[kSlots];
  const int row = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = row / p.q_len, i0 = blockIdx.x * kSlots;
  bool past = false;
  const int have = pages_of(p, row, &past);
  if (have <= p.pages || i0 >= have) {
    if (past && blockIdx.x == 0 && threadIdx.x == 0) set_device_error(p.err_word, TS_DEVERR_PAGE_RANGE);
    return;
  }
  if (past && threadIdx.x == 0) set_device_error(p.err_word, TS_DEVERR_PAGE_RANGE);
  for (int i = threadIdx.x; i < kSlots; i += kWarps * 32) {
    int pg = -1;
    if (i0 + i < have) {
      pg = p.block_table[static_cast<int64_t>(b) * p.bt_stride + i0 + i];
      if (pg < 0 || pg >= p.num_pages) {
        set_device_error(p.err_word, TS_DEVERR_PAGE_RANGE);
        pg = -1;
      }
    }
    page[i] = pg;
  }
  const int H_q = p.H_kv * G;
  for (int h = warp; h < H_q; h += kWarps) {
    const T* src = q + (static_cast<int64_t>(row) * H_q + h) * D;
    float x[D / 32];
    uint32_t largest = 0u;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      x[i] = static_cast<float>(src[lane + 32 * i]);
      largest = max(largest, __float_as_uint(x[i]) & 0x7fffffffu);
    }
    largest = __reduce_max_sync(0xffffffffu, largest);
    const bool odd = largest >= 0x7f800000u;
    const float top = __uint_as_float(largest);  // (a NaN stays one)
    const float scale = odd ? top : fmaxf(top, 1e-10f) * (1.f / 127.f);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int c = odd ? 0 : static_cast<int>(fminf(fmaxf(rintf(__fdiv_rn(x[i], scale)), -127.f), 127.f));
      code[h][lane + 32 * i] = static_cast<int8_t>(max(c, 0));
      code[h][D + lane + 32 * i] = static_cast<int8_t>(min(c, 0));
    }
    if (lane == 0) q_scale[h] = scale;
  }
  __syncthreads();

  const int h = warp % p.H_kv, share = warp / p.H_kv, shares = kWarps / p.H_kv;
  const int l = lane % kL, sub = lane / kL;
  uint4 c[G];
#pragma unroll
  for (int i = 0; i < G; ++i) c[i] = *reinterpret_cast<const uint4*>(&code[h * G + i][16 * l]);
  // after the sums a lane holds those of one head: its index follows from the lane
  int mine = 0;
#pragma unroll
  for (int n = G / 2, o = kL / 2; n > 0; n >>= 1, o >>= 1) mine += (l & o) ? n : 0;
  const float qs = q_scale[h * G + mine];
  uint32_t* keys = p.keys + (static_cast<int64_t>(row) * p.H_kv + h) * p.bt_stride;

  constexpr int kAhead = 4;
  const int step = shares * kU;
  for (int j0 = share * kU + sub; j0 - sub < kSlots; j0 += kAhead * step) {
    uint4 w[kAhead];
    float s[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = j0 + u * step;
      const int pg = j < kSlots ? page[j] : -1;
      const int64_t at = static_cast<int64_t>(max(pg, 0)) * p.H_kv + h;
      w[u] = *reinterpret_cast<const uint4*>(p.bounds + at * 2 * D + 16 * l);
      s[u] = p.bound_scale[at];
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = j0 + u * step;
      int v[G];
#pragma unroll
      for (int i = 0; i < G; ++i) {
        v[i] = __dp4a(static_cast<int>(c[i].x), static_cast<int>(w[u].x), 0);
        v[i] = __dp4a(static_cast<int>(c[i].y), static_cast<int>(w[u].y), v[i]);
        v[i] = __dp4a(static_cast<int>(c[i].z), static_cast<int>(w[u].z), v[i]);
        v[i] = __dp4a(static_cast<int>(c[i].w), static_cast<int>(w[u].w), v[i]);
      }
      int o = kL / 2;
#pragma unroll
      for (int n = G / 2; n > 0; n >>= 1, o >>= 1) {
        const bool upper = (l & o) != 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
          const int send = upper ? v[i] : v[i + n];
          v[i] = (upper ? v[i + n] : v[i]) + __shfl_xor_sync(0xffffffffu, send, o);
        }
      }
#pragma unroll
      for (; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
      uint32_t key = order_key(static_cast<float>(v[0]) * qs * s[u]);
      o = kL / 2;
#pragma unroll
      for (int n = G / 2; n > 0; n >>= 1, o >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
      if (l == 0 && j < kSlots && i0 + j < have) keys[i0 + j] = page[j] >= 0 ? key : 0u;
    }
  }
}

__global__ void __launch_bounds__(kPickThreads) page_pick_kernel(const SelectParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  __shared__ uint32_t bins[kPickBins];
  __shared__ uint32_t kept[kPickSmemKeys];
  __shared__ uint32_t warp_a[kPickThreads / 32], warp_b[kPickThreads / 32];
  __shared__ uint32_t shared_lo, shared_hi, shared_need, shared_bin;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t item = blockIdx.x;  // (row, kv head)
  const int row = static_cast<int>(item / p.H_kv);
  bool past = false;
  const int have = pages_of(p, row, &past);
  int32_t* out = p.page_idx + item * p.pages;
  if (have <= p.pages) {
    if (past && tid == 0) set_device_error(p.err_word, TS_DEVERR_PAGE_RANGE);
    for (int i = tid; i < p.pages; i += kPickThreads) out[i] = i < have ? i : -1;
    return;
  }
  const int n = have - p.first - p.last, need0 = p.pages - p.first - p.last;  // n > need0
  for (int i = tid; i < p.first; i += kPickThreads) out[i] = i;
  for (int i = tid; i < p.last; i += kPickThreads) out[p.pages - p.last + i] = have - p.last + i;
  if (need0 == 0) return;
  const uint32_t* keys = p.keys + item * p.bt_stride + p.first;
  if (n <= kPickSmemKeys) {
    for (int i = tid; i < n; i += kPickThreads) kept[i] = keys[i];
    keys = kept;
  }
  if (tid == 0) shared_lo = 0xffffffffu, shared_hi = 0u, shared_need = static_cast<uint32_t>(need0);
  __syncthreads();
  {
    uint32_t lo = 0xffffffffu, hi = 0u;
    for (int i = tid; i < n; i += kPickThreads) lo = min(lo, keys[i]), hi = max(hi, keys[i]);
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) atomicMin(&shared_lo, lo), atomicMax(&shared_hi, hi);
  }
  __syncthreads();
  // [lo, hi] holds the need-th largest key; cut it in bins until it is one value
  uint32_t lo = shared_lo, hi = shared_hi, need = shared_need;
  while (lo < hi) {
    const int shift = max(0, 32 - __clz(static_cast<int>(hi - lo)) - 11);
    for (int i = tid; i < kPickBins; i += kPickThreads) bins[i] = 0u;
    __syncthreads();
    for (int i = tid; i < n; i += kPickThreads) {
      const uint32_t k = keys[i];
      if (k >= lo && k <= hi) atomicAdd(&bins[(k - lo) >> shift], 1u);
    }
    __syncthreads();
    // counts from the highest bin down; four bins a thread
    constexpr int kEach = kPickBins / kPickThreads;
    uint32_t sum = 0u;
#pragma unroll
    for (int i = 0; i < kEach; ++i) sum += bins[kPickBins - 1 - (tid * kEach + i)];
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_a[warp] = incl;
    __syncthreads();
    uint32_t before = 0u;
    for (int i = 0; i < warp; ++i) before += warp_a[i];
    uint32_t above = before + incl - sum;  // keys in higher bins than this thread's
    if (above < need && above + sum >= need) {
      for (int i = 0; i < kEach; ++i) {
        const int bin = kPickBins - 1 - (tid * kEach + i);
        if (above + bins[bin] >= need) {
          shared_bin = static_cast<uint32_t>(bin);
          shared_need = need - above;
          break;
        }
        above += bins[bin];
      }
    }
    __syncthreads();
    need = shared_need;
    lo += shared_bin << shift;
    hi = lo + min(hi - lo, (1u << shift) - 1u);
    __syncthreads();
  }
  // keys above lo, and the first `need` equal to it, in order of their pages
  const int each = (n + kPickThreads - 1) / kPickThreads, a0 = min(n, tid * each), a1 = min(n, a0 + each);
  uint32_t more = 0u, same = 0u;
  for (int i = a0; i < a1; ++i) more += keys[i] > lo, same += keys[i] == lo;
  uint32_t more_incl = more, same_incl = same;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, more_incl, o), z = __shfl_up_sync(0xffffffffu, same_incl, o);
    if (lane >= o) more_incl += y, same_incl += z;
  }
  if (lane == 31) warp_a[warp] = more_incl, warp_b[warp] = same_incl;
  __syncthreads();
  uint32_t more_at = more_incl - more, same_at = same_incl - same;
  for (int i = 0; i < warp; ++i) more_at += warp_a[i], same_at += warp_b[i];
  for (int i = a0; i < a1; ++i) {
    const uint32_t k = keys[i];
    const bool equal = k == lo;
    if (k > lo || (equal && same_at < need)) out[p.first + more_at + min(same_at, need)] = p.first + i;
    more_at += k > lo;
    same_at += equal;
  }
}

template <typename K, typename... A>
cudaError_t launch_pdl(K kern, dim3 grid, int threads, cudaStream_t stream, A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename T, int D>
cudaError_t launch_score(int g, dim3 grid, cudaStream_t stream, const void* q, const SelectParams& p) {
  const T* src = static_cast<const T*>(q);
  switch (g) {
    case 1: return launch_pdl(page_score_kernel<T, D, 1>, grid, kWarps * 32, stream, src, p);
    case 2: return launch_pdl(page_score_kernel<T, D, 2>, grid, kWarps * 32, stream, src, p);
    case 4: return launch_pdl(page_score_kernel<T, D, 4>, grid, kWarps * 32, stream, src, p);
    default: return launch_pdl(page_score_kernel<T, D, 8>, grid, kWarps * 32, stream, src, p);
  }
}

size_t select_bytes(int64_t rows, int H_kv, int bt_stride) {
  return align_up(kWorkspaceAlign + static_cast<size_t>(rows) * H_kv * bt_stride * sizeof(uint32_t), kWorkspaceAlign);
}

}  // namespace
}  // namespace ts

extern "C" size_t ts_select_pages_workspace_size(int32_t B, int32_t q_len, int32_t H_kv, int32_t bt_stride) {
  if (B < 0 || q_len <= 0 || H_kv <= 0 || H_kv > 8 || bt_stride <= 0 || static_cast<int64_t>(B) * q_len > 0x7fffffff)
    return 0;
  return ts::select_bytes(static_cast<int64_t>(B) * q_len, H_kv, bt_stride);
}

extern "C" ts_status ts_select_pages(const void* q, const int8_t* bounds, const float* bound_scale,
                                     const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens,
                                     int32_t B, int32_t q_len, int32_t H_q, int32_t H_kv, int32_t D,
                                     int32_t page_size, int32_t num_pages, int32_t pages, int32_t first,
                                     int32_t last, ts_dtype dtype, int32_t* page_idx, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  using namespace ts;
  const char* who = "ts_select_pages";
  if (B < 0 || q_len <= 0 || H_q <= 0 || H_kv <= 0 || D <= 0 || page_size <= 0 || num_pages <= 0 || bt_stride <= 0)
    return fail(TS_ERR_INVALID_ARG, "%s: bad sizes (B=%d q_len=%d H_q=%d H_kv=%d D=%d ps=%d P=%d bt=%d)", who, B,
                q_len, H_q, H_kv, D, page_size, num_pages, bt_stride);
  if (H_q % H_kv != 0) return fail(TS_ERR_INVALID_ARG, "%s: H_q=%d not a multiple of H_kv=%d", who, H_q, H_kv);
  if (dtype != TS_F32 && dtype != TS_BF16)
    return fail(TS_ERR_INVALID_ARG, "%s: bad dtype %d", who, static_cast<int>(dtype));
  if (pages <= 0 || first < 0 || last < 1 || static_cast<int64_t>(first) + last > pages)
    return fail(TS_ERR_INVALID_ARG, "%s: pages=%d first=%d last=%d (first >= 0, last >= 1, first + last <= pages)",
                who, pages, first, last);
  const int g = H_q / H_kv;
  if ((D != 64 && D != 128) || (g != 1 && g != 2 && g != 4 && g != 8) ||
      (H_kv != 1 && H_kv != 2 && H_kv != 4 && H_kv != 8))
    return fail(TS_ERR_UNSUPPORTED, "%s: H_q=%d H_kv=%d D=%d (H_q / H_kv and H_kv in {1, 2, 4, 8}, D in {64, 128})",
                who, H_q, H_kv, D);
  const int64_t rows = static_cast<int64_t>(B) * q_len;
  if (rows > 65535) return fail(TS_ERR_UNSUPPORTED, "%s: more than 65535 query rows", who);
  if (B == 0) return TS_OK;
  if (!q || !bounds || !bound_scale || !block_table || !seq_lens || !page_idx)
    return fail(TS_ERR_INVALID_ARG, "%s: null pointer", who);
  for (const void* x : {q, static_cast<const void*>(bounds)})
    if (reinterpret_cast<uintptr_t>(x) % 16 != 0)
      return fail(TS_ERR_INVALID_ARG, "%s: queries and bounds must be 16-byte aligned", who);
  const size_t bytes = select_bytes(rows, H_kv, bt_stride);
  if (!workspace || workspace_bytes < bytes || reinterpret_cast<uintptr_t>(workspace) % kWorkspaceAlign != 0)
    return fail(TS_ERR_WORKSPACE, "%s: workspace %zu B < %zu B needed or misaligned", who, workspace_bytes, bytes);
  const SelectParams p{bounds,    bound_scale, block_table, seq_lens,
                       reinterpret_cast<uint32_t*>(static_cast<unsigned char*>(workspace) + kWorkspaceAlign),
                       page_idx,  static_cast<uint32_t*>(workspace), bt_stride, q_len, H_kv, page_size, num_pages,
                       pages, first, last};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (bt_stride > pages && pages > first + last) {  // else nothing is ranked
    const dim3 grid(static_cast<unsigned>((bt_stride - 1) / kSlots + 1), static_cast<unsigned>(rows));
    LaunchTrace trace("page_score_kernel", s);
    const cudaError_t e =
        dtype == TS_BF16 ? (D == 64 ? launch_score<__nv_bfloat16, 64>(g, grid, s, q, p)
                                    : launch_score<__nv_bfloat16, 128>(g, grid, s, q, p))
                         : (D == 64 ? launch_score<float, 64>(g, grid, s, q, p)
                                    : launch_score<float, 128>(g, grid, s, q, p));
    const ts_status st = cuda_check(e, "ts_select_pages: launch");
    if (st != TS_OK) return st;
  }
  LaunchTrace trace("page_pick_kernel", s);
  return cuda_check(launch_pdl(page_pick_kernel, dim3(static_cast<unsigned>(rows * H_kv)), kPickThreads, s, p),
                    "ts_select_pages: launch");
}
