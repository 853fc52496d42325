// ts_kv_append_chunk and ts_kv_append_chunk_fp8: write the K and V rows of a
// ragged batch of prompt chunks into their pages, as they are or quantized to
// e4m3 codes.
//
// Row r of the batch belongs to the sequence b with q_indptr[b] <= r <
// q_indptr[b + 1]; as its token j = r - q_indptr[b] of n, it sits at position
// seq_lens[b] - n + j, in page block_table[b][pos / page_size] at row pos %
// page_size (SwiftLLM page, section 3.1).
//
// A warp takes a row (K and V, or one of them where they are quantized) and
// finds the row's sequence by a 32-way search over q_indptr: no plan is made on
// the host and none has to be kept. Each value is read once and written once, and
// HBM bounds the copy. 15,000 bf16 rows of 8 x 128 (a part of a fused
// projection's rows): the copy 20.7 us, 123 MB at 5.9 TB/s; the quantizing one
// 21.4 us for 16,000 rows, 99 MB at 4.6 TB/s: its issue slots are active 63 % of
// the time and HBM at 68 % of its rate, neither exhausted.
// 33 rows: 2.4 and 2.6 us, of which the launch and two dependent loads are most.
#include <cuda_fp8.h>

#include "ts_ragged.cuh"

namespace ts {
namespace {

constexpr int kWarps = 8;  // per CTA

struct ChunkRows {
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* q_indptr;
  int32_t bt_stride, T, B, H_kv, num_pages;
  PageSize page_size;
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

// Eight values of a lane as they are stored: four or eight words.
template <typename T>
struct Eight {
  uint32_t w[2 * sizeof(T)];
  __device__ __forceinline__ void load(const T* p) {
    const uint4* v = reinterpret_cast<const uint4*>(p);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
      const uint4 a = v[i];
      w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
    }
  }
  __device__ __forceinline__ float2 pair(int i) const {
    if constexpr (sizeof(T) == 2)
      return bf16x2_to_float2(w[i]);
    else
      return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  }
  // The sign bits of values 4 i .. 4 i + 3, as those of four codes.
  __device__ __forceinline__ uint32_t signs(int i) const {
    if constexpr (sizeof(T) == 2)
      return __byte_perm(w[2 * i], w[2 * i + 1], 0x7531) & 0x80808080u;
    else
      return __byte_perm(__byte_perm(w[4 * i], w[4 * i + 1], 0x0073), __byte_perm(w[4 * i + 2], w[4 * i + 3], 0x0073),
                         0x5410) & 0x80808080u;
  }
  // The largest magnitude's float32 bits. Magnitudes order as their bits do,
  // with infinities and NaN above all others.
  __device__ __forceinline__ uint32_t largest() const {
    if constexpr (sizeof(T) == 2) {
      const uint32_t m = 0x7fff7fffu;
      const uint32_t a = __vmaxu2(__vmaxu2(w[0] & m, w[1] & m), __vmaxu2(w[2] & m, w[3] & m));
      return max(a << 16, a & 0xffff0000u);
    } else {
      uint32_t a = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) a = max(a, w[i] & 0x7fffffffu);
      return a;
    }
  }
};

// The codes of a lane's eight values by the definition: one quotient each.
template <typename T>
__device__ __forceinline__ uint2 codes_by_definition(const Eight<T>& x, float scale) {
  uint32_t code[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = x.pair(i / 2);
    const float y = __fdiv_rn(i % 2 ? f.y : f.x, scale);
    // the saturating cast is the clamp, and keeps a NaN
    code[i / 4] |= static_cast<uint32_t>(__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3)) << (8 * (i % 4));
  }
  return make_uint2(code[0], code[1]);
}

// Quantization as ts_kv_append_fp8, bit for bit: a group is the D values of
// one (token, kv head); scale = max(max |x|, 1e-10) / 448, code =
// e4m3(clamp(x / scale, -448, 448)), in float32 rounded to nearest even. A NaN
// makes its group's scale and codes NaN, an infinity the scale infinite.
//
// One warp per row of K, of V or of both. D / 8 lanes hold a group, eight values each,
// so that a warp takes two (D = 128) or four (D = 64) groups at a time, and
// loads kBatch times that before the first of it is quantized. A group shares
// one divisor, so its quotients take a reciprocal and five multiply-adds each
// instead of a division each. Groups that hold an infinity or NaN, or whose
// scale's reciprocal may not be the rounded one, take the definition's divisions.
// src_step: elements between rows of k_new (and of v_new).
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32, sizeof(T) == 2 ? 5 : 4) kv_append_chunk_fp8_kernel(
    const T* __restrict__ k_new, const T* __restrict__ v_new, uint8_t* __restrict__ k_pool,
    uint8_t* __restrict__ v_pool, float* __restrict__ k_scale, float* __restrict__ v_scale, ChunkRows c,
    int64_t src_step, int32_t both) {
  pdl_wait_primary();
  pdl_launch_dependents();
  constexpr int kLanes = D / 8, kPerStep = 32 / kLanes, kBatch = 4;
  const int lane = threadIdx.x & 31;
  const int w = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int r = both ? w : w >> 1;
  if (r >= c.T) return;
  bool is_v = !both && (w & 1) != 0;
  const int at = (lane % kLanes) * 8;
  const T* src = (is_v ? v_new : k_new) + r * src_step + at;
  Eight<T> x[kBatch];
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int h = h0 + u * kPerStep + lane / kLanes;
      if (h < c.H_kv) {
        x[u].load(src + h * D);
      } else {
#pragma unroll
        for (uint32_t& w : x[u].w) w = 0u;
      }
    }
  };
  load(0);  // the values do not wait for the row's place
  const int64_t row = chunk_pool_row(c, r, lane);
  if (row < 0) return;
  uint8_t* pool = (is_v ? v_pool : k_pool) + row * c.H_kv * D + at;
  float* scales = (is_v ? v_scale : k_scale) + row * c.H_kv;
  for (int h0 = 0;;) {
    uint32_t top[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) top[u] = x[u].largest();
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
      for (int u = 0; u < kBatch; ++u) top[u] = max(top[u], __shfl_xor_sync(0xffffffffu, top[u], o));
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int h = h0 + u * kPerStep + lane / kLanes;
      float scale = quotient(fmaxf(__uint_as_float(top[u]), 1e-10f), kE4M3Max, 1.f / kE4M3Max);
      const float inv = reciprocal(scale);
      uint32_t two[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        two[i] = __nv_cvt_float2_to_fp8x2(
            quotients(x[u].pair(i), make_float2(-scale, -scale), make_float2(inv, inv)), __NV_SATFINITE, __NV_E4M3);
      // (the steps above lose the sign of a zero)
      uint2 code = make_uint2(two[0] | two[1] << 16 | x[u].signs(0), two[2] | two[3] << 16 | x[u].signs(1));
      if (__any_sync(0xffffffffu, top[u] >= 0x7f800000u || all_ones(scale))) {
        scale = e4m3_group_scale(top[u]);  // of finite groups: the same again
        code = codes_by_definition(x[u], scale);
      }
      if (h < c.H_kv) {
        *reinterpret_cast<uint2*>(pool + h * D) = code;
        if (at == 0) scales[h] = scale;
      }
    }
    h0 += kBatch * kPerStep;
    if (h0 >= c.H_kv) {
      if (!both || is_v) return;
      is_v = true;
      h0 = 0;
      src = v_new + r * src_step + at;
      pool = v_pool + row * c.H_kv * D + at;
      scales = v_scale + row * c.H_kv;
    }
    load(h0);
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
  RowLaunch(int32_t rows, int per_cta, cudaStream_t stream) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>((rows - 1) / per_cta + 1));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
};

template <typename T>
ts_status launch_fp8(int D, const void* k_new, const void* v_new, void* k_pool, void* v_pool, float* k_scale,
                     float* v_scale, const ChunkRows& c, int64_t new_stride, cudaStream_t stream) {
  // A warp takes a row's K and V where that alone fills the device twice over
  // (half as many searches: 19.9 us against 20.6 for 15,000 rows of 8 x 128, 34.9
  // against 37.2 for 30,000), one of them below (33 rows: 2.4 us against 3.5;
  // 6,000: 9.97 against 10.0).
  const int both = c.T >= 2 * 40 * device_sm_count() ? 1 : 0;
  RowLaunch l(c.T, both ? kWarps : kWarps / 2, stream);
  auto kern = D == 64 ? kv_append_chunk_fp8_kernel<T, 64> : kv_append_chunk_fp8_kernel<T, 128>;
  LaunchTrace trace("kv_append_chunk_fp8_kernel", stream);
  return cuda_check(cudaLaunchKernelEx(&l.cfg, kern, static_cast<const T*>(k_new), static_cast<const T*>(v_new),
                                       static_cast<uint8_t*>(k_pool), static_cast<uint8_t*>(v_pool), k_scale,
                                       v_scale, c, new_stride, both),
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
  const ChunkRows c{block_table, seq_lens, q_indptr, bt_stride, T, B, H_kv, num_pages, PageSize(page_size)};
  RowLaunch l(T, kWarps, static_cast<cudaStream_t>(stream));
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
  const ChunkRows c{block_table, seq_lens, q_indptr, bt_stride, T, B, H_kv, num_pages, PageSize(page_size)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == TS_BF16)
    return launch_fp8<__nv_bfloat16>(D, k_new, v_new, k_pool, v_pool, k_scale, v_scale, c, new_stride, s);
  return launch_fp8<float>(D, k_new, v_new, k_pool, v_pool, k_scale, v_scale, c, new_stride, s);
}
