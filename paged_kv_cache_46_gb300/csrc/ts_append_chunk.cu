// ts_kv_append_chunk and ts_kv_append_chunk_fp8: write the K and V rows of a
// ragged batch of prompt chunks into their pages, as they are or quantized to
// e4m3 codes.
//
// Row r of the batch belongs to the sequence b with q_indptr[b] <= r <
// q_indptr[b + 1]; as its token j = r - q_indptr[b] of n, it sits at position
// seq_lens[b] - n + j, in page block_table[b][pos / page_size] at row pos %
// page_size (SwiftLLM page, section 3.1).
//
// Both kernels take one warp per row, K and V: the row's sequence is found by
// a 32-way search over q_indptr, so no plan is made on the host and none has
// to be kept, and a short chunk spreads over as many SMs as it has rows / 8.
// Both are bound by HBM: each value is read once and written once.
#include <cuda_fp8.h>

#include "ts_ragged.cuh"

namespace ts {
namespace {

constexpr int kWarps = 8;  // rows per CTA
constexpr float kE4M3Max = 448.0f;

struct ChunkRows {
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* q_indptr;
  int32_t bt_stride, T, B, H_kv, page_size, num_pages;
};

// Pool row of batch row r, or -1 if it has none (no sequence, a position in
// front of the first token, a slot or page out of range).
__device__ __forceinline__ int64_t chunk_pool_row(const ChunkRows& c, int r, int lane) {
  const int b = ragged_sequence(c.q_indptr, c.B, r, lane);
  if (b < 0) return -1;
  return pool_row(c.block_table, c.bt_stride, b, c.seq_lens[b] - (c.q_indptr[b + 1] - r), c.page_size, c.num_pages);
}

// row_vecs: 16-byte vectors of one row; src_vecs: of the step between rows.
__global__ void __launch_bounds__(kWarps * 32) kv_append_chunk_kernel(const uint4* __restrict__ k_new,
                                                                      const uint4* __restrict__ v_new,
                                                                      uint4* __restrict__ k_pool,
                                                                      uint4* __restrict__ v_pool, ChunkRows c,
                                                                      int32_t row_vecs, int64_t src_vecs) {
  // Programmatic dependent launch as in ts_kv_append.
  pdl_wait_primary();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (r >= c.T) return;
  const uint4* ks = k_new + r * src_vecs;
  const uint4* vs = v_new + r * src_vecs;
  const int64_t row = chunk_pool_row(c, r, lane);
  if (row < 0) return;
  uint4* kd = k_pool + row * row_vecs;
  uint4* vd = v_pool + row * row_vecs;
  // four vectors of K and of V per lane in flight
  for (int i0 = lane; i0 < row_vecs; i0 += 128) {
    uint4 k[4], v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + 32 * u;
      if (i < row_vecs) {
        k[u] = ks[i];
        v[u] = vs[i];
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + 32 * u;
      if (i < row_vecs) {
        kd[i] = k[u];
        vd[i] = v[u];
      }
    }
  }
}

// Eight values of a lane, widened.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = bf16x2_to_float2(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  } else {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
}

// Quantization as ts_kv_append_fp8, bit for bit: a group is the D values of
// one (token, kv head); scale = max(max |x|, 1e-10) / 448, code =
// e4m3(clamp(x / scale, -448, 448)), in float32 rounded to nearest even.
// D / 8 lanes hold a group, eight values each, so that a warp quantizes two
// (D = 128) or four (D = 64) groups at a time and stores 8 bytes of codes per
// lane. src_step: elements between rows of k_new (and of v_new).
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) kv_append_chunk_fp8_kernel(
    const T* __restrict__ k_new, const T* __restrict__ v_new, uint8_t* __restrict__ k_pool,
    uint8_t* __restrict__ v_pool, float* __restrict__ k_scale, float* __restrict__ v_scale, ChunkRows c,
    int64_t src_step) {
  pdl_wait_primary();
  pdl_launch_dependents();
  constexpr int kLanes = D / 8, kPerStep = 32 / kLanes;
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (r >= c.T) return;
  const int64_t row = chunk_pool_row(c, r, lane);
  if (row < 0) return;
  const int at = (lane % kLanes) * 8;
  // groups 0 .. H_kv - 1 are K's heads, the others V's
  for (int g0 = 0; g0 < 2 * c.H_kv; g0 += kPerStep) {
    const int gi = g0 + lane / kLanes;
    const bool real = gi < 2 * c.H_kv;
    const bool is_v = gi >= c.H_kv;
    const int h = is_v ? gi - c.H_kv : gi;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (real) load8((is_v ? v_new : k_new) + r * src_step + h * D + at, x);
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float scale = __fdiv_rn(fmaxf(amax, 1e-10f), kE4M3Max);
    uint32_t code[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = fminf(fmaxf(__fdiv_rn(x[i], scale), -kE4M3Max), kE4M3Max);
      code[i / 4] |= static_cast<uint32_t>(__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3)) << (8 * (i % 4));
    }
    if (real) {
      const int64_t cell = row * c.H_kv + h;
      *reinterpret_cast<uint2*>((is_v ? v_pool : k_pool) + cell * D + at) = make_uint2(code[0], code[1]);
      if (at == 0) (is_v ? v_scale : k_scale)[cell] = scale;
    }
  }
}

// Argument checks that both calls share; TS_OK with *enqueue = false where
// there is nothing to write.
ts_status check(const char* who, const void* k_new, const void* v_new, const void* k_pool, const void* v_pool,
                const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens, const int32_t* q_indptr,
                int64_t new_stride, int32_t T, int32_t B, int32_t H_kv, int32_t D, int32_t page_size,
                int32_t num_pages, ts_dtype dtype, bool* enqueue) {
  *enqueue = false;
  if (T < 0 || B < 0 || H_kv <= 0 || D <= 0 || page_size <= 0 || num_pages <= 0 || bt_stride <= 0)
    return fail(TS_ERR_INVALID_ARG, "%s: bad sizes (T=%d B=%d H_kv=%d D=%d ps=%d P=%d bt=%d)", who, T, B, H_kv, D,
                page_size, num_pages, bt_stride);
  if (dtype != TS_F32 && dtype != TS_BF16)
    return fail(TS_ERR_INVALID_ARG, "%s: bad dtype %d", who, static_cast<int>(dtype));
  const int64_t width = static_cast<int64_t>(H_kv) * D, es = dtype == TS_F32 ? 4 : 2;
  if (width * es > (1 << 20))
    return fail(TS_ERR_UNSUPPORTED, "%s: a row of H_kv=%d x D=%d exceeds 1 MiB", who, H_kv, D);
  if (new_stride < width)
    return fail(TS_ERR_INVALID_ARG, "%s: rows %lld elements apart are narrower than H_kv*D=%lld", who,
                static_cast<long long>(new_stride), static_cast<long long>(width));
  if (T == 0 || B == 0) return TS_OK;
  if (!k_new || !v_new || !k_pool || !v_pool || !block_table || !seq_lens || !q_indptr)
    return fail(TS_ERR_INVALID_ARG, "%s: null pointer", who);
  if (width * es % 16 != 0 || new_stride * es % 16 != 0)
    return fail(TS_ERR_UNSUPPORTED, "%s: rows of %lld B, %lld B apart, are not multiples of 16 B", who,
                static_cast<long long>(width * es), static_cast<long long>(new_stride * es));
  for (const void* p : {k_new, v_new, k_pool, v_pool})
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0)
      return fail(TS_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", who);
  *enqueue = true;
  return TS_OK;
}

struct RowLaunch {
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = {};
  RowLaunch(int32_t rows, cudaStream_t stream) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>((rows - 1) / kWarps + 1));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
};

template <typename T>
ts_status launch_fp8(int D, const void* k_new, const void* v_new, void* k_pool, void* v_pool, float* k_scale,
                     float* v_scale, const ChunkRows& c, int64_t new_stride, cudaStream_t stream) {
  RowLaunch l(c.T, stream);
  auto kern = D == 64 ? kv_append_chunk_fp8_kernel<T, 64> : kv_append_chunk_fp8_kernel<T, 128>;
  LaunchTrace trace("kv_append_chunk_fp8_kernel", stream);
  return cuda_check(cudaLaunchKernelEx(&l.cfg, kern, static_cast<const T*>(k_new), static_cast<const T*>(v_new),
                                       static_cast<uint8_t*>(k_pool), static_cast<uint8_t*>(v_pool), k_scale,
                                       v_scale, c, new_stride),
                    "ts_kv_append_chunk_fp8: launch");
}

}  // namespace
}  // namespace ts

extern "C" ts_status ts_kv_append_chunk(const void* k_new, const void* v_new, void* k_pool, void* v_pool,
                                        const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens,
                                        const int32_t* q_indptr, int64_t new_stride, int32_t T, int32_t B,
                                        int32_t H_kv, int32_t D, int32_t page_size, int32_t num_pages,
                                        ts_dtype dtype, void* stream) {
  using namespace ts;
  bool enqueue;
  const ts_status st = check("ts_kv_append_chunk", k_new, v_new, k_pool, v_pool, block_table, bt_stride, seq_lens,
                             q_indptr, new_stride, T, B, H_kv, D, page_size, num_pages, dtype, &enqueue);
  if (st != TS_OK || !enqueue) return st;
  const int64_t es = dtype == TS_F32 ? 4 : 2;
  const ChunkRows c{block_table, seq_lens, q_indptr, bt_stride, T, B, H_kv, page_size, num_pages};
  RowLaunch l(T, static_cast<cudaStream_t>(stream));
  LaunchTrace trace("kv_append_chunk_kernel", l.cfg.stream);
  return cuda_check(cudaLaunchKernelEx(&l.cfg, kv_append_chunk_kernel, static_cast<const uint4*>(k_new),
                                       static_cast<const uint4*>(v_new), static_cast<uint4*>(k_pool),
                                       static_cast<uint4*>(v_pool), c,
                                       static_cast<int32_t>(H_kv * D * es / 16), new_stride * es / 16),
                    "ts_kv_append_chunk: launch");
}

extern "C" ts_status ts_kv_append_chunk_fp8(const void* k_new, const void* v_new, void* k_pool, void* v_pool,
                                            float* k_scale, float* v_scale, const int32_t* block_table,
                                            int32_t bt_stride, const int32_t* seq_lens, const int32_t* q_indptr,
                                            int64_t new_stride, int32_t T, int32_t B, int32_t H_kv, int32_t D,
                                            int32_t page_size, int32_t num_pages, ts_dtype dtype, void* stream) {
  using namespace ts;
  const char* who = "ts_kv_append_chunk_fp8";
  bool enqueue;
  const ts_status st = check(who, k_new, v_new, k_pool, v_pool, block_table, bt_stride, seq_lens, q_indptr,
                             new_stride, T, B, H_kv, D, page_size, num_pages, dtype, &enqueue);
  if (st != TS_OK) return st;
  if (D != 64 && D != 128) return fail(TS_ERR_UNSUPPORTED, "%s: D=%d (supported 64, 128)", who, D);
  if (!enqueue) return TS_OK;
  if (!k_scale || !v_scale) return fail(TS_ERR_INVALID_ARG, "%s: null scale array", who);
  for (const void* p : {k_scale, v_scale})
    if (reinterpret_cast<uintptr_t>(p) % 4 != 0)
      return fail(TS_ERR_INVALID_ARG, "%s: scale arrays must be 4-byte aligned", who);
  const ChunkRows c{block_table, seq_lens, q_indptr, bt_stride, T, B, H_kv, page_size, num_pages};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == TS_BF16)
    return launch_fp8<__nv_bfloat16>(D, k_new, v_new, k_pool, v_pool, k_scale, v_scale, c, new_stride, s);
  return launch_fp8<float>(D, k_new, v_new, k_pool, v_pool, k_scale, v_scale, c, new_stride, s);
}
