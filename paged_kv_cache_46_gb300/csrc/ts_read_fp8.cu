// ts_kv_read_fp8: read an fp8 (e4m3fn) paged cache back into rows.
//
// Row r of the result belongs to the sequence b with kv_indptr[b] <= r <
// kv_indptr[b + 1] and holds its token t = r - kv_indptr[b], where t <
// seq_lens[b]: K[t] = code * k_scale[t], the same for V (token-group scales:
// tokenspeed 딥다이브, fiv.co.kr, section 6-4; placement: SwiftLLM page,
// section 3.1). Other rows are left as they were.
//
// One warp per row, K and V. A lane takes eight codes at a time (an 8-byte
// load, one 16-byte store in bf16). The codes widen exactly, the product with
// the scale is rounded to float32 and then to the result's type.
// Bound by HBM: a byte of code in, two or four bytes out. 157,000 rows of 8 x
// 128 to bf16: 145 us, 974 MB at 6.7 TB/s (99 % of the device's copy rate); 999
// rows: 3.0 us.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ts_ragged.cuh"

namespace ts {
namespace {

constexpr int kWarps = 8;   // rows per CTA
constexpr int kUnroll = 4;  // loads of a lane in flight

__device__ __forceinline__ float2 widen2(uint32_t pair) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(pair), __NV_E4M3);
  return __half22float2(__half2(h));
}

template <typename T>
__device__ __forceinline__ void store8(T* p, uint2 code, float scale) {
  float2 f[4] = {widen2(code.x & 0xffffu), widen2(code.x >> 16), widen2(code.y & 0xffffu), widen2(code.y >> 16)};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = make_float2(f[i].x * scale, f[i].y * scale);
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) = make_uint4(float2_to_bf16x2(f[0].x, f[0].y), float2_to_bf16x2(f[1].x, f[1].y),
                                              float2_to_bf16x2(f[2].x, f[2].y), float2_to_bf16x2(f[3].x, f[3].y));
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) kv_read_fp8_kernel(
    const uint8_t* __restrict__ k_pool, const uint8_t* __restrict__ v_pool, const float* __restrict__ k_scale,
    const float* __restrict__ v_scale, const int32_t* __restrict__ block_table, int32_t bt_stride,
    const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ kv_indptr, int32_t rows, int32_t B,
    int32_t H_kv, PageSize page_size, int32_t num_pages, T* __restrict__ k_out, T* __restrict__ v_out) {
  // Programmatic dependent launch as in ts_kv_append.
  pdl_wait_primary();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (r >= rows) return;
  const int b = ragged_sequence(kv_indptr, B, r, lane);
  if (b < 0) return;
  const int t = r - kv_indptr[b];
  if (t >= seq_lens[b]) return;
  const int64_t row = pool_row(block_table, bt_stride, b, t, page_size, num_pages);
  if (row < 0) return;
  const int vecs = H_kv * (D / 8);  // of 8 codes, in K's row; V's follow
  const int64_t src = row * vecs, dst = static_cast<int64_t>(r) * vecs;
  const uint2* kc = reinterpret_cast<const uint2*>(k_pool) + src;
  const uint2* vc = reinterpret_cast<const uint2*>(v_pool) + src;
  const float* ks = k_scale + row * H_kv;
  const float* vs = v_scale + row * H_kv;
  for (int i0 = lane; i0 < 2 * vecs; i0 += 32 * kUnroll) {
    uint2 code[kUnroll];
    float scale[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + 32 * u;
      if (i < 2 * vecs) {
        const bool is_v = i >= vecs;
        const int at = is_v ? i - vecs : i;
        code[u] = (is_v ? vc : kc)[at];
        scale[u] = (is_v ? vs : ks)[at / (D / 8)];
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + 32 * u;
      if (i < 2 * vecs) {
        const bool is_v = i >= vecs;
        const int at = is_v ? i - vecs : i;
        store8((is_v ? v_out : k_out) + (dst + at) * 8, code[u], scale[u]);
      }
    }
  }
}

template <typename T>
ts_status launch(int D, const void* k_pool, const void* v_pool, const float* k_scale, const float* v_scale,
                 const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens, const int32_t* kv_indptr,
                 int32_t rows, int32_t B, int32_t H_kv, int32_t page_size, int32_t num_pages, void* k_out,
                 void* v_out, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((rows - 1) / kWarps + 1));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kern = D == 64 ? kv_read_fp8_kernel<T, 64> : kv_read_fp8_kernel<T, 128>;
  LaunchTrace trace("kv_read_fp8_kernel", stream);
  return cuda_check(cudaLaunchKernelEx(&cfg, kern, static_cast<const uint8_t*>(k_pool),
                                       static_cast<const uint8_t*>(v_pool), k_scale, v_scale, block_table, bt_stride,
                                       seq_lens, kv_indptr, rows, B, H_kv, PageSize(page_size), num_pages,
                                       static_cast<T*>(k_out), static_cast<T*>(v_out)),
                    "ts_kv_read_fp8: launch");
}

}  // namespace
}  // namespace ts

extern "C" ts_status ts_kv_read_fp8(const void* k_pool, const void* v_pool, const float* k_scale,
                                    const float* v_scale, const int32_t* block_table, int32_t bt_stride,
                                    const int32_t* seq_lens, const int32_t* kv_indptr, int32_t rows, int32_t B,
                                    int32_t H_kv, int32_t D, int32_t page_size, int32_t num_pages, ts_dtype dtype,
                                    void* k_out, void* v_out, void* stream) {
  using namespace ts;
  const char* who = "ts_kv_read_fp8";
  if (rows < 0 || B < 0 || H_kv <= 0 || D <= 0 || page_size <= 0 || num_pages <= 0 || bt_stride <= 0)
    return fail(TS_ERR_INVALID_ARG, "%s: bad sizes (rows=%d B=%d H_kv=%d D=%d ps=%d P=%d bt=%d)", who, rows, B, H_kv,
                D, page_size, num_pages, bt_stride);
  if (dtype != TS_F32 && dtype != TS_BF16)
    return fail(TS_ERR_INVALID_ARG, "%s: bad dtype %d", who, static_cast<int>(dtype));
  if (D != 64 && D != 128) return fail(TS_ERR_UNSUPPORTED, "%s: D=%d (supported 64, 128)", who, D);
  if (static_cast<int64_t>(H_kv) * D > (1 << 20))
    return fail(TS_ERR_UNSUPPORTED, "%s: H_kv=%d: a row of codes exceeds 1 MiB", who, H_kv);
  if (rows == 0 || B == 0) return TS_OK;
  if (!k_pool || !v_pool || !k_scale || !v_scale || !block_table || !seq_lens || !kv_indptr || !k_out || !v_out)
    return fail(TS_ERR_INVALID_ARG, "%s: null pointer", who);
  for (const void* p : {k_pool, v_pool, static_cast<const void*>(k_out), static_cast<const void*>(v_out)})
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0)
      return fail(TS_ERR_INVALID_ARG, "%s: pools and results must be 16-byte aligned", who);
  for (const void* p : {k_scale, v_scale})
    if (reinterpret_cast<uintptr_t>(p) % 4 != 0)
      return fail(TS_ERR_INVALID_ARG, "%s: scale arrays must be 4-byte aligned", who);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == TS_BF16)
    return launch<__nv_bfloat16>(D, k_pool, v_pool, k_scale, v_scale, block_table, bt_stride, seq_lens, kv_indptr,
                                 rows, B, H_kv, page_size, num_pages, k_out, v_out, s);
  return launch<float>(D, k_pool, v_pool, k_scale, v_scale, block_table, bt_stride, seq_lens, kv_indptr, rows, B,
                       H_kv, page_size, num_pages, k_out, v_out, s);
}
