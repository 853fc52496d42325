// ts_paged_prefill_attn, float32: the tensor pipe has no float32 product, so
// this path runs on the CUDA cores and keeps float32 accuracy.
//
// A CTA takes 64 query rows (64 / g tokens times the g heads of one kv head)
// and walks the keys that some of them sees in tiles of 64. Thread (y, x) of
// 16 x 16 holds a 4 x 4 patch of the scores and 4 rows x D / 16 columns of O
// in registers; K and V tiles are gathered page by page into shared memory,
// padded so that 16-byte reads of different keys fall into different banks.
// Running maximum and sum per row, in float32. What bounds it: the packed
// float32 FMA rate and the shared-memory reads that feed it.
#include <cmath>

#include "ts_common.cuh"

namespace ts {
namespace {

constexpr int kRows = 64, kKeys = 64, kThreads = 256;
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

template <int D>
__global__ void __launch_bounds__(kThreads) prefill_f32_kernel(const F32Params p) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(smem_raw);
  constexpr int kStep = Smem<D>::kStep, kCols = D / 16;
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
  const int b = sm.seq, h = blockIdx.y;
  if (b < 0) return;
  const int row0 = p.q_indptr[b], n = p.q_indptr[b + 1] - row0, L = max(p.seq_lens[b], 0);
  const int j0 = sm.block * p.tile_tokens, tokens = min(n - j0, p.tile_tokens);
  const int p0 = L - n + j0;
  const long long cap = static_cast<long long>(p.bt_stride) * p.page_size;
  const int khi = static_cast<int>(min(static_cast<long long>(max(p0 + tokens, 0)), cap));
  int klo = (p.window > 0 && p0 >= p.window) ? p0 - p.window + 1 : 0;
  if (klo <= p.sinks) klo = 0;
  const int w0 = klo / kKeys;
  const int ns = klo > 0 ? min((p.sinks + kKeys - 1) / kKeys, w0) : 0;
  const int nt = ns + max(0, (khi + kKeys - 1) / kKeys - w0);
  if (tid == 0 && p0 + tokens > khi && p0 + tokens > 0) set_device_error(p.err_word, TS_DEVERR_PAGE_RANGE);

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
  float m[4], l[4], o[4][kCols];
  int pos[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    m[a] = -INFINITY;
    l[a] = 0.f;
    pos[a] = p0 + (y * 4 + a) / p.g;
#pragma unroll
    for (int c = 0; c < kCols; ++c) o[a][c] = 0.f;
  }
  for (int i = 0; i < nt; ++i) {
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
    for (int e = tid; e < kKeys * (D / 4); e += kThreads) {
      const int key = e / (D / 4), c = e % (D / 4) * 4;
      const int row = sm.row[key];
      float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
      if (row >= 0) {
        const int64_t at = (static_cast<int64_t>(row) * p.H_kv + h) * D + c;
        kv = *reinterpret_cast<const float4*>(p.k_pool + at);
        vv = *reinterpret_cast<const float4*>(p.v_pool + at);
      }
      *reinterpret_cast<float4*>(sm.k + key * kStep + c) = kv;
      *reinterpret_cast<float4*>(sm.v + key * kStep + c) = vv;
    }
    __syncthreads();
    float s[4][4] = {};
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      float4 qa[4], kb[4];
#pragma unroll
      for (int a = 0; a < 4; ++a) qa[a] = *reinterpret_cast<const float4*>(sm.q + (y * 4 + a) * kStep + d);
#pragma unroll
      for (int c = 0; c < 4; ++c) kb[c] = *reinterpret_cast<const float4*>(sm.k + (x + 16 * c) * kStep + d);
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          s[a][c] = fmaf(qa[a].x, kb[c].x, s[a][c]);
          s[a][c] = fmaf(qa[a].y, kb[c].y, s[a][c]);
          s[a][c] = fmaf(qa[a].z, kb[c].z, s[a][c]);
          s[a][c] = fmaf(qa[a].w, kb[c].w, s[a][c]);
        }
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int first = (p.window > 0 && pos[a] >= p.window) ? pos[a] - p.window + 1 : 0;
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int key = x + 16 * c, t = k0 + key;
        const bool vis = sm.row[key] >= 0 && t <= pos[a] && (t >= first || t < p.sinks);
        s[a][c] = vis ? s[a][c] * p.scale_log2 : -INFINITY;
        mx = fmaxf(mx, s[a][c]);
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
        const float e = exp2f(s[a][c] - ms);
        sm.p[(x + 16 * c) * (kRows + 4) + y * 4 + a] = e;
        sum += e;
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      l[a] = l[a] * alpha + sum;
#pragma unroll
      for (int c = 0; c < kCols; ++c) o[a][c] *= alpha;
    }
    __syncwarp();  // a row's weights are written and read by one half warp
#pragma unroll 4
    for (int key = 0; key < kKeys; ++key) {
      const float4 w = *reinterpret_cast<const float4*>(sm.p + key * (kRows + 4) + y * 4);
      const float wa[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int c = 0; c < kCols; c += 4) {
        const float4 v = *reinterpret_cast<const float4*>(sm.v + key * kStep + c * 16 + x * 4);
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          o[a][c] = fmaf(wa[a], v.x, o[a][c]);
          o[a][c + 1] = fmaf(wa[a], v.y, o[a][c + 1]);
          o[a][c + 2] = fmaf(wa[a], v.z, o[a][c + 2]);
          o[a][c + 3] = fmaf(wa[a], v.w, o[a][c + 3]);
        }
      }
    }
  }
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int r = y * 4 + a;
    if (r >= rows) continue;
    const int64_t row = static_cast<int64_t>(row0 + j0 + r / p.g) * p.H_q + h * p.g + r % p.g;
    const float inv = l[a] > 0.f ? 1.f / l[a] : 0.f;
#pragma unroll
    for (int c = 0; c < kCols; c += 4)
      *reinterpret_cast<float4*>(p.out + row * D + c * 16 + x * 4) =
          make_float4(o[a][c] * inv, o[a][c + 1] * inv, o[a][c + 2] * inv, o[a][c + 3] * inv);
    if (x == 0 && p.lse) p.lse[row] = l[a] > 0.f ? (m[a] + log2f(l[a])) * kLn2C : -INFINITY;
  }
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
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(prm.H_kv));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Smem<D>);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  LaunchTrace trace("prefill_f32_kernel", s);
  return cuda_check(cudaLaunchKernelEx(&cfg, prefill_f32_kernel<D>, prm), "float32 prefill launch");
}

}  // namespace

ts_status launch_prefill_f32(const float* q, int64_t q_stride, const float* k_pool, const float* v_pool,
                             const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens,
                             const int32_t* q_indptr, int32_t T, int32_t B, int32_t H_q, int32_t H_kv, int32_t D,
                             int32_t page_size, int32_t num_pages, int32_t window, int32_t sinks, float scale,
                             float* out, float* lse, uint32_t* err_word, cudaStream_t stream) {
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
  prm.scale_log2 = scale * kLog2eC;
  prm.err_word = err_word;
  // one block per token block and kv head; a sequence's last may be partial
  const long long blocks = T / prm.tile_tokens + static_cast<long long>(B < T ? B : T);
  if (blocks > INT32_MAX) return fail(TS_ERR_UNSUPPORTED, "ts_paged_prefill_attn: T=%d, B=%d", T, B);
  return D == 64 ? launch<64>(prm, static_cast<int>(blocks), stream) : launch<128>(prm, static_cast<int>(blocks), stream);
}

}  // namespace ts
