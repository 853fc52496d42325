// ts_paged_prefill_attn, float32: on the CUDA cores, with float32 products and
// sums throughout. (The tensor pipe has no float32 product; products of bf16
// terms that add up to float32 values are not built here.)
//
// A CTA takes 128 query rows (128 / g tokens times the g heads of one kv head)
// and walks the keys that some of them sees in tiles of 64. Thread (y, x) of
// 16 x 16 holds an 8 x 4 patch of the scores and 8 rows x D / 16 columns of O
// in registers, as pairs for the packed multiply-add; K and V tiles are
// gathered page by page into shared memory, rows padded by 16 bytes so that
// 16-byte reads of different keys fall into different banks. Running maximum
// and sum per row, in float32.
//
// What bounds it: the issue of packed multiply-adds and of the shared reads that
// feed them, 12 of 16 bytes for 64 packed multiply-adds of the scores (1024
// tokens over 8192, 32 / 8 heads of 128: 3.8 ms, 38 TFLOP/s, about half of the
// multiply-adds' own rate; with a 4 x 4 patch 5.3 ms).
//
// Few rows over a long context leave most SMs idle, so each CTA's keys are
// split over as many CTAs as the device has room for twice over; the parts are
// joined by LSE (16 tokens over 28,000: 0.43 ms, with one part 5.5 ms). The
// number of parts is one for the whole batch, from its counts of rows and
// sequences: a long context among many short chunks is not split further (16
// tokens over 28,000 beside 63 chunks of one token: 7.0 ms).
#include <algorithm>
#include <cmath>

#include "ts_ragged.cuh"

namespace ts {
namespace {

constexpr int kRows = 128, kKeys = 64, kThreads = 256;
constexpr float kLog2eC = 1.4426950408889634f;
constexpr float kLn2C = 0.6931471805599453f;

struct F32Params {
  const float* q;
  const float* k_pool;
  const float* v_pool;
  float* out;
  float* lse;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* q_indptr;
  int64_t q_stride;
  int32_t T, B, bt_stride, H_q, H_kv, g, page_size, num_pages, window, sinks, tile_tokens;
  int32_t parts;    // CTAs that share a block's keys
  float* part_o;    // [parts, T, H_q, D], used from two parts on
  float* part_lse;  // [parts, T, H_q]
  float scale_log2;
  uint32_t* err_word;
};

template <int D>
struct Smem {
  static constexpr int kStep = D + 4;  // floats between rows of Q, K and V
  float q[kRows * kStep];
  float k[kKeys * kStep];
  float v[kKeys * kStep];
  float p[kKeys * (kRows + 4)];  // weights, key-major
  int row[kKeys];                // pool row of each key, -1: not seen by any row, or no such page
  int seq, block;
};

__device__ __forceinline__ int tiles_of(int keys) { return keys > 0 ? (keys - 1) / kKeys + 1 : 0; }

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prefill_f32_kernel(const F32Params p) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(smem_raw);
  constexpr int kStep = Smem<D>::kStep, kCols = D / 16, kPStep = kRows + 4;
  const int tid = threadIdx.x, lane = tid & 31;
  pdl_wait_primary();
  pdl_launch_dependents();
  // block index -> (sequence, token block): prefix sums of the block counts
  if (tid < 32) {
    int found = -1, block = 0, before = 0;
    for (int b0 = 0; b0 < p.B && found < 0; b0 += 32) {
      const int b = b0 + lane;
      int n = 0;
      if (b < p.B) {
        const int r0 = p.q_indptr[b], r1 = p.q_indptr[b + 1];
        n = (r0 >= 0 && r0 <= r1 && r1 <= p.T) ? r1 - r0 : 0;  // rows outside the batch: none
      }
      const int mine = (n + p.tile_tokens - 1) / p.tile_tokens;
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const int at = static_cast<int>(blockIdx.x) - before - (incl - mine);
      const unsigned hit = __ballot_sync(0xffffffffu, at >= 0 && at < mine);
      if (hit) {
        found = b0 + __ffs(hit) - 1;
        block = __shfl_sync(0xffffffffu, at, __ffs(hit) - 1);
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      sm.seq = found;
      sm.block = block;
    }
  }
  __syncthreads();
  const int b = sm.seq, h = blockIdx.y, part = blockIdx.z;
  if (b < 0) return;
  const int row0 = p.q_indptr[b], n = p.q_indptr[b + 1] - row0, L = max(p.seq_lens[b], 0);
  const int j0 = sm.block * p.tile_tokens, tokens = min(n - j0, p.tile_tokens);
  const int p0 = L - n + j0;
  const long long cap = min(static_cast<long long>(p.bt_stride) * p.page_size, 1ll << 30);
  const int khi = static_cast<int>(min(static_cast<long long>(max(p0 + tokens, 0)), cap));
  int klo = (p.window > 0 && p0 >= p.window) ? p0 - p.window + 1 : 0;
  if (klo <= p.sinks) klo = 0;
  const int w0 = klo / kKeys;
  const int ns = klo > 0 ? min(tiles_of(p.sinks), w0) : 0;
  const int nt = ns + max(0, tiles_of(khi) - w0);
  if (tid == 0 && part == 0 && p0 + tokens > khi && p0 + tokens > 0)
    set_device_error(p.err_word, TS_DEVERR_PAGE_RANGE);
  const int i0 = static_cast<int>(static_cast<long long>(nt) * part / p.parts);
  const int i1 = static_cast<int>(static_cast<long long>(nt) * (part + 1) / p.parts);

  const int rows = tokens * p.g;
  for (int i = tid; i < kRows * (D / 4); i += kThreads) {
    const int r = i / (D / 4), c = i % (D / 4) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows) {
      const int64_t t = row0 + j0 + r / p.g;
      v = *reinterpret_cast<const float4*>(p.q + t * p.q_stride + (h * p.g + r % p.g) * D + c);
    }
    *reinterpret_cast<float4*>(sm.q + r * kStep + c) = v;
  }
  const int x = tid & 15, y = tid >> 4;
  float m[8], l[8];
  float2 o[8][kCols / 2];
  int pos[8];
#pragma unroll
  for (int a = 0; a < 8; ++a) {
    m[a] = -INFINITY;
    l[a] = 0.f;
    pos[a] = p0 + (y * 8 + a) / p.g;
#pragma unroll
    for (int c = 0; c < kCols / 2; ++c) o[a][c] = make_float2(0.f, 0.f);
  }
  for (int i = i0; i < i1; ++i) {
    const int k0 = (i < ns ? i : w0 + i - ns) * kKeys;
    __syncthreads();  // the previous tile's reads are done
    if (tid < kKeys) {
      const int t = k0 + tid;
      int row = -1;
      if (t < khi && (t >= klo || t < p.sinks)) {
        const int page = p.block_table[static_cast<int64_t>(b) * p.bt_stride + t / p.page_size];
        if (page >= 0 && page < p.num_pages)
          row = page * p.page_size + t % p.page_size;
        else
          set_device_error(p.err_word, TS_DEVERR_PAGE_RANGE);
      }
      sm.row[tid] = row;
    }
    __syncthreads();
    // four rows' loads in flight per thread
    constexpr int kVecs = kKeys * (D / 4);
#pragma unroll
    for (int e0 = 0; e0 < kVecs; e0 += 4 * kThreads) {
      float4 kv[4], vv[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int e = e0 + u * kThreads + tid, key = e / (D / 4), c = e % (D / 4) * 4;
        const int row = sm.row[key];
        kv[u] = vv[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row >= 0) {
          const int64_t at = (static_cast<int64_t>(row) * p.H_kv + h) * D + c;
          kv[u] = *reinterpret_cast<const float4*>(p.k_pool + at);
          vv[u] = *reinterpret_cast<const float4*>(p.v_pool + at);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int e = e0 + u * kThreads + tid, key = e / (D / 4), c = e % (D / 4) * 4;
        *reinterpret_cast<float4*>(sm.k + key * kStep + c) = kv[u];
        *reinterpret_cast<float4*>(sm.v + key * kStep + c) = vv[u];
      }
    }
    __syncthreads();
    float2 s2[8][4];  // sums over even and over odd columns
#pragma unroll
    for (int a = 0; a < 8; ++a)
#pragma unroll
      for (int c = 0; c < 4; ++c) s2[a][c] = make_float2(0.f, 0.f);
#pragma unroll 2
    for (int d = 0; d < D; d += 4) {
      float4 kb[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) kb[c] = *reinterpret_cast<const float4*>(sm.k + (x + 16 * c) * kStep + d);
#pragma unroll
      for (int a = 0; a < 8; ++a) {
        const float4 qa = *reinterpret_cast<const float4*>(sm.q + (y * 8 + a) * kStep + d);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          s2[a][c] = __ffma2_rn(make_float2(qa.x, qa.y), make_float2(kb[c].x, kb[c].y), s2[a][c]);
          s2[a][c] = __ffma2_rn(make_float2(qa.z, qa.w), make_float2(kb[c].z, kb[c].w), s2[a][c]);
        }
      }
    }
    float e[8][4];
#pragma unroll
    for (int a = 0; a < 8; ++a) {
      const int first = (p.window > 0 && pos[a] >= p.window) ? pos[a] - p.window + 1 : 0;
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int key = x + 16 * c, t = k0 + key;
        const bool vis = sm.row[key] >= 0 && t <= pos[a] && (t >= first || t < p.sinks);
        e[a][c] = vis ? (s2[a][c].x + s2[a][c].y) * p.scale_log2 : -INFINITY;
        mx = fmaxf(mx, e[a][c]);
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mnew = fmaxf(m[a], mx);
      const float ms = mnew == -INFINITY ? 0.f : mnew;
      const float alpha = m[a] == -INFINITY ? 0.f : exp2f(m[a] - ms);
      m[a] = mnew;
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        e[a][c] = exp2f(e[a][c] - ms);
        sum += e[a][c];
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      l[a] = l[a] * alpha + sum;
      const float2 al = make_float2(alpha, alpha);
#pragma unroll
      for (int c = 0; c < kCols / 2; ++c) o[a][c] = __fmul2_rn(o[a][c], al);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float4* to = reinterpret_cast<float4*>(sm.p + (x + 16 * c) * kPStep + y * 8);
      to[0] = make_float4(e[0][c], e[1][c], e[2][c], e[3][c]);
      to[1] = make_float4(e[4][c], e[5][c], e[6][c], e[7][c]);
    }
    __syncwarp();  // a row's weights are written and read by one half warp
#pragma unroll 2
    for (int key = 0; key < kKeys; ++key) {
      const float4 wa = *reinterpret_cast<const float4*>(sm.p + key * kPStep + y * 8);
      const float4 wb = *reinterpret_cast<const float4*>(sm.p + key * kPStep + y * 8 + 4);
      const float w[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
#pragma unroll
      for (int c = 0; c < kCols; c += 4) {
        const float4 v = *reinterpret_cast<const float4*>(sm.v + key * kStep + c * 16 + x * 4);
#pragma unroll
        for (int a = 0; a < 8; ++a) {
          const float2 w2 = make_float2(w[a], w[a]);
          o[a][c / 2] = __ffma2_rn(w2, make_float2(v.x, v.y), o[a][c / 2]);
          o[a][c / 2 + 1] = __ffma2_rn(w2, make_float2(v.z, v.w), o[a][c / 2 + 1]);
        }
      }
    }
  }
  const bool whole = p.parts == 1;
  const int64_t all = static_cast<int64_t>(p.T) * p.H_q * part;
#pragma unroll
  for (int a = 0; a < 8; ++a) {
    const int r = y * 8 + a;
    if (r >= rows) continue;
    const int64_t row = static_cast<int64_t>(row0 + j0 + r / p.g) * p.H_q + h * p.g + r % p.g;
    const float inv = l[a] == 0.f ? 0.f : 1.f / l[a];  // no key: O = 0, LSE = -inf; a NaN sum stays NaN
    float* to = whole ? p.out + row * D : p.part_o + (all + row) * D;
#pragma unroll
    for (int c = 0; c < kCols; c += 4)
      *reinterpret_cast<float4*>(to + c * 16 + x * 4) =
          make_float4(o[a][c / 2].x * inv, o[a][c / 2].y * inv, o[a][c / 2 + 1].x * inv, o[a][c / 2 + 1].y * inv);
    if (x == 0) {
      const float lse = l[a] == 0.f ? -INFINITY : (m[a] + log2f(l[a])) * kLn2C;
      if (!whole)
        p.part_lse[all + row] = lse;
      else if (p.lse)
        p.lse[row] = lse;
    }
  }
}

// Joins the parts of every row: a warp per (token, head).
template <int D>
__global__ void __launch_bounds__(256) prefill_f32_merge_kernel(const F32Params p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t rows = static_cast<int64_t>(p.T) * p.H_q;
  if (row >= rows) return;
  const int b = ragged_sequence(p.q_indptr, p.B, static_cast<int>(row / p.H_q), lane);
  if (b < 0 || p.q_indptr[b] < 0 || p.q_indptr[b + 1] > p.T) return;  // no sequence's row, no parts
  float mx = -INFINITY;
  for (int i = lane; i < p.parts; i += 32) mx = fmaxf(mx, p.part_lse[i * rows + row]);
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
  const float ms = mx == -INFINITY ? 0.f : mx;
  constexpr int kV = D / 32;  // values per lane
  float a[kV], sum = 0.f;
#pragma unroll
  for (int c = 0; c < kV; ++c) a[c] = 0.f;
#pragma unroll 4
  for (int i = 0; i < p.parts; ++i) {
    const float w = expf(p.part_lse[i * rows + row] - ms);
    sum += w;
#pragma unroll
    for (int c = 0; c < kV; ++c) a[c] = fmaf(w, p.part_o[(i * rows + row) * D + c * 32 + lane], a[c]);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int c = 0; c < kV; ++c) p.out[row * D + c * 32 + lane] = a[c] * inv;
  if (lane == 0 && p.lse) p.lse[row] = sum == 0.f ? -INFINITY : ms + logf(sum);
}

template <int D>
ts_status launch(const F32Params& prm, int blocks, cudaStream_t s) {
  ts_status st = prepare_once(reinterpret_cast<const void*>(prefill_f32_kernel<D>), [](const void* f) {
    return cuda_check(cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Smem<D>)),
                      "float32 prefill smem attribute");
  });
  if (st != TS_OK) return st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(prm.H_kv), static_cast<unsigned>(prm.parts));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Smem<D>);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  {
    LaunchTrace trace("prefill_f32_kernel", s);
    st = cuda_check(cudaLaunchKernelEx(&cfg, prefill_f32_kernel<D>, prm), "float32 prefill launch");
  }
  if (st != TS_OK || prm.parts == 1) return st;
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(prm.T) * prm.H_q + 7) / 8));
  cfg.dynamicSmemBytes = 0;
  LaunchTrace trace("prefill_f32_merge_kernel", s);
  return cuda_check(cudaLaunchKernelEx(&cfg, prefill_f32_merge_kernel<D>, prm), "float32 prefill merge launch");
}

}  // namespace

// part_o and part_lse have room for 2 * ctas blocks of 128 rows.
ts_status launch_prefill_f32(const float* q, int64_t q_stride, const float* k_pool, const float* v_pool,
                             const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens,
                             const int32_t* q_indptr, int32_t T, int32_t B, int32_t H_q, int32_t H_kv, int32_t D,
                             int32_t page_size, int32_t num_pages, int32_t window, int32_t sinks, float scale,
                             float* out, float* lse, uint32_t* err_word, float* part_o, float* part_lse, int32_t ctas,
                             cudaStream_t stream) {
  F32Params prm;
  prm.q = q;
  prm.k_pool = k_pool;
  prm.v_pool = v_pool;
  prm.out = out;
  prm.lse = lse;
  prm.block_table = block_table;
  prm.seq_lens = seq_lens;
  prm.q_indptr = q_indptr;
  prm.q_stride = q_stride;
  prm.T = T;
  prm.B = B;
  prm.bt_stride = bt_stride;
  prm.H_q = H_q;
  prm.H_kv = H_kv;
  prm.g = H_q / H_kv;
  prm.page_size = page_size;
  prm.num_pages = num_pages;
  prm.window = window;
  prm.sinks = sinks;
  prm.tile_tokens = kRows / prm.g;
  prm.part_o = part_o;
  prm.part_lse = part_lse;
  prm.scale_log2 = scale * kLog2eC;
  prm.err_word = err_word;
  // one block per token block and kv head; a sequence's last may be partial.
  // They hold T * H_q rows in blocks * H_kv * 128 places, so that as many parts
  // as keep 2 * ctas blocks fit the places for parts.
  const long long blocks = T / prm.tile_tokens + static_cast<long long>(B < T ? B : T);
  if (blocks > INT32_MAX) return fail(TS_ERR_UNSUPPORTED, "ts_paged_prefill_attn: T=%d, B=%d", T, B);
  prm.parts = static_cast<int32_t>(std::max(1ll, std::min(256ll, 2ll * ctas / (blocks * H_kv))));
  return D == 64 ? launch<64>(prm, static_cast<int>(blocks), stream) : launch<128>(prm, static_cast<int>(blocks), stream);
}

}  // namespace ts
