// ts_kv_append_chunk_rope: the rows of a ragged batch of prompt chunks (or one
// new token per sequence) on their way from the projection to the attention:
// queries and keys normalised per head and rotated by their positions, K and V
// written into their pages, the queries into rows.
//
// Of a head's row x of D values, with weights w:
//   y = w x / sqrt(mean(x^2) + eps)           (no weights: y = x)
//   (y1, y2) -> (y1 cos a - y2 sin a, y2 cos a + y1 sin a),  a = position *
//   inv_freq[j], for the pairs j < rot / 2 of its first rot columns: (j, j +
//   rot / 2), or (2 j, 2 j + 1) where they are interleaved.
// All in float32, rounded once to the stored type.
//
// Each value is read once and written once, and HBM bounds rows of many heads: 18,900
// rows of 32 + 2 x 8 heads of 128 in bf16, a part of a fused projection's, 78.8 us, 464
// MB at 5.9 TB/s, as fast as the plain append's copy. Issue slots are active 62 % of the
// time. Rows of few heads are bound by what each row costs its warp (the sequence's
// search, the table's lookup, sines and two sets of factors) beside its five or six
// steps of data: 18,900 rows of 8 + 2 x 1 heads 33.5 us (97 MB, 2.9 TB/s), 10,000
// float32 rows of 4 + 2 x 2 heads of 64 12.9 us (41 MB, 3.2 TB/s).
//
// A warp takes a row, or one of `parts` shares of its heads where there are few
// rows. D / 8 lanes hold a head, as two groups of four columns a lane, chosen so
// that both columns of a pair are in one lane: nothing is exchanged but the sum
// of squares. The heads of a step are taken kBatch steps at a time, loaded before
// the row's place is known. Weights, cosines and sines of a lane's columns are two
// factors per column, made once per row for the queries and once for the keys:
//   y = inv * (x P + partner Q),
// in packed multiply-adds, since instructions would bound it otherwise.
//
// Angles: a float32 product of position and frequency is off by 2^-24 of the
// angle, a hundredth of a turn at position 131,072. Turns are counted in 64-bit
// fixed point instead: inv_freq / (2 pi) mod 1 as a 64-bit fraction (a float64
// product and its remainder, once per CTA; off by two units at most), times the
// position modulo 2^64, is the angle in turns. Its nearest quarter turn is taken off
// exactly and the 64-bit rest, at most an eighth of a turn, is rounded to float32
// once: by 2^-24 of itself, so that slow pairs keep their small sines.
#include "ts_ragged.cuh"

#include <cmath>
#include <type_traits>

namespace ts {
namespace {

constexpr int kWarps = 8;   // per CTA
constexpr int kBatch = 4;   // steps in flight

template <typename T>
struct RopeParams {
  const T* q;
  const T* k_new;
  const T* v_new;
  const T* q_weight;
  const T* k_weight;
  const float* inv_freq;
  T* k_pool;
  T* v_pool;
  T* q_out;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* q_indptr;
  int64_t q_stride, new_stride, q_out_stride;
  int32_t bt_stride, T_rows, B, H_q, H_kv, num_pages, rot, interleaved, parts;
  float eps;
  PageSize page_size;
};

// Four consecutive values as they are stored.
template <typename T>
struct Quad;
template <>
struct Quad<__nv_bfloat16> {
  uint2 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint2*>(p) = w; }
  __device__ __forceinline__ void get(float (&x)[4]) const {
    const float2 a = bf16x2_to_float2(w.x), b = bf16x2_to_float2(w.y);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
  }
  __device__ __forceinline__ void set(const float (&x)[4]) {
    w.x = float2_to_bf16x2(x[0], x[1]);
    w.y = float2_to_bf16x2(x[2], x[3]);
  }
};
template <>
struct Quad<float> {
  float4 w;
  __device__ __forceinline__ void load(const float* p) { w = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = w; }
  __device__ __forceinline__ void get(float (&x)[4]) const { x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w; }
  __device__ __forceinline__ void set(const float (&x)[4]) { w = make_float4(x[0], x[1], x[2], x[3]); }
};

// inv_freq / (2 pi) modulo 1, in units of 2^-64. Of its magnitude: f - floor(f) of a small negative f would lose
// f's lower bits.
__device__ __forceinline__ unsigned long long turns_per_position(float inv_freq) {
  const double x = fabsf(inv_freq), f = x * 0.15915494309189534;  // 1 / (2 pi); low: what product and constant leave
  const double low = fma(x, 0.15915494309189534, -f) + x * -9.839338337591243e-18;
  const unsigned long long turns = __double2ull_rn((f - floor(f)) * 0x1p64) +
                                   static_cast<unsigned long long>(__double2ll_rn(low * 0x1p64));
  return inv_freq < 0.f ? 0ull - turns : turns;
}

// Cosine and sine of the angle at a position.
__device__ __forceinline__ float2 turn(int pos, unsigned long long step) {
  const unsigned long long t = static_cast<unsigned long long>(pos) * step;
  const uint32_t quarter = static_cast<uint32_t>((t + (1ull << 61)) >> 62);
  // within an eighth of a turn; all of its bits, since a slow pair's angle is small
  const long long rest = static_cast<long long>(t - (static_cast<unsigned long long>(quarter) << 62));
  float s, c;
  sincospif(static_cast<float>(rest) * 0x1p-63f, &s, &c);  // in half turns
  const float u = quarter & 1u ? s : c, v = quarter & 1u ? c : s;
  return make_float2((quarter + 1u) & 2u ? -u : u, quarter & 2u ? -v : v);
}

template <typename T, int D, bool kInterleaved, bool kMixed>
__global__ void __launch_bounds__(kWarps * 32, sizeof(T) == 2 ? 4 : 3) rope_append_kernel(const RopeParams<T> p) {
  // Programmatic dependent launch as in ts_kv_append.
  pdl_wait_primary();
  pdl_launch_dependents();
  constexpr int kLanes = D / 8, kVecs = 32 / kLanes;
  __shared__ unsigned long long steps[D / 2];
  __shared__ float2 angles[kWarps][D / 2];  // cosine and sine of each warp's row
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int parts = kMixed ? p.parts : 1;
  const int64_t r = kMixed ? w / static_cast<uint32_t>(parts) : w;
  const int part = static_cast<int>(w - r * parts);
  const int l = lane % kLanes, vec = lane / kLanes;
  const bool turns = l < p.rot / 8;
  const bool split = turns && !kInterleaved;
  const int oa = split ? 4 * l : 8 * l, ob = split ? p.rot / 2 + 4 * l : 8 * l + 4;

  // Steps of kVecs heads: the row's queries, its keys, its values; a warp takes every parts-th of them in order.
  const int q_steps = (p.H_q + kVecs - 1) / kVecs, kv_steps = (p.H_kv + kVecs - 1) / kVecs;
  const int all_steps = q_steps + 2 * kv_steps;
  // 0: queries, 1: keys, 2: values; and the section's first step, rows and heads
  auto section_of = [&](int g) { return g < q_steps ? 0 : g < q_steps + kv_steps ? 1 : 2; };
  auto first_of = [&](int section) { return section == 0 ? 0 : section == 1 ? q_steps : q_steps + kv_steps; };
  auto source_of = [&](int section) {
    return section == 0 ? p.q + r * p.q_stride : (section == 1 ? p.k_new : p.v_new) + r * p.new_stride;
  };
  Quad<T> xa[kBatch], xb[kBatch];
  auto load_step = [&](int u, const T* src, int h, int heads) {
    if (h < heads) {
      xa[u].load(src + h * D + oa);
      xb[u].load(src + h * D + ob);
    } else {
      xa[u] = {};
      xb[u] = {};
    }
  };
  // Mixed batches are of any steps. Others end with their section, and the warp takes the whole row: section, its
  // next step, heads and rows.
  int section = 0, g = part, heads = p.H_q;
  const T* src = p.q + r * p.q_stride;
  // From a section's end to the next one; false behind the last one.
  auto settle = [&]() {
    if constexpr (kMixed) {
      return g < all_steps;
    } else {
      for (int n = section == 0 ? q_steps : kv_steps; g >= n; n = kv_steps) {
        g = 0;
        if (++section > 2) return false;
        heads = p.H_kv;
        src = source_of(section);
      }
      return true;
    }
  };
  auto load = [&]() {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int step = g + u * parts;
      if constexpr (kMixed) {
        const int of = section_of(step);
        load_step(u, source_of(of), (step - first_of(of)) * kVecs + vec,
                  step >= all_steps ? 0 : of == 0 ? p.H_q : p.H_kv);
      } else {
        load_step(u, src, step * kVecs + vec, heads);
      }
    }
  };
  const bool any = r < p.T_rows && settle();
  if (any) load();
  for (int i = threadIdx.x; i < p.rot / 2; i += kWarps * 32) steps[i] = turns_per_position(p.inv_freq[i]);
  __syncthreads();
  if (!any) return;
  const int b = ragged_sequence(p.q_indptr, p.B, static_cast<int>(r), lane);
  if (b < 0) return;
  const int pos = p.seq_lens[b] - (p.q_indptr[b + 1] - static_cast<int>(r));
  if (pos < 0) return;
  const int64_t row = pool_row(p.block_table, p.bt_stride, b, pos, p.page_size, p.num_pages);

  // pair 4 l + i of the lane, i < 4: each of the kVecs lanes that share them computes 4 / kVecs
  float2* turned = angles[threadIdx.x >> 5];
  if (turns) {
    constexpr int kOwn = 4 / kVecs;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) turned[4 * l + vec * kOwn + i] = turn(pos, steps[4 * l + vec * kOwn + i]);
  }
  __syncwarp();

  // Factors of the columns a[0 .. 3], c[0 .. 3] and of their partners, two columns each.
  float2 P[4], Q[4];
  auto factors = [&](const T* weight) {
    float a[4] = {1.f, 1.f, 1.f, 1.f}, c[4] = {1.f, 1.f, 1.f, 1.f};
    float2 cs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) cs[i] = turns ? turned[4 * l + i] : make_float2(1.f, 0.f);
    if (weight != nullptr) {
      Quad<T> q;
      q.load(weight + oa);
      q.get(a);
      q.load(weight + ob);
      q.get(c);
    }
    if (kInterleaved) {  // partners are neighbours
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        P[i] = make_float2(a[2 * i] * cs[i].x, a[2 * i + 1] * cs[i].x);
        Q[i] = make_float2(-a[2 * i + 1] * cs[i].y, a[2 * i] * cs[i].y);
        P[2 + i] = make_float2(c[2 * i] * cs[2 + i].x, c[2 * i + 1] * cs[2 + i].x);
        Q[2 + i] = make_float2(-c[2 * i + 1] * cs[2 + i].y, c[2 * i] * cs[2 + i].y);
      }
    } else {  // partners of a are c
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        P[i] = make_float2(a[2 * i] * cs[2 * i].x, a[2 * i + 1] * cs[2 * i + 1].x);
        Q[i] = make_float2(-c[2 * i] * cs[2 * i].y, -c[2 * i + 1] * cs[2 * i + 1].y);
        P[2 + i] = make_float2(c[2 * i] * cs[2 * i].x, c[2 * i + 1] * cs[2 * i + 1].x);
        Q[2 + i] = make_float2(a[2 * i] * cs[2 * i].y, a[2 * i + 1] * cs[2 * i + 1].y);
      }
    }
  };
  int made = -1;  // section that P and Q are of
  auto finish_step = [&](int u, int section, const T* weight, T* dst, int h, int heads) {
    if (section < 2 && (weight != nullptr || p.rot > 0)) {
      if (made != section) {
        factors(weight);
        made = section;
      }
      float a[4], c[4];
      xa[u].get(a);
      xb[u].get(c);
      const float2 x[4] = {{a[0], a[1]}, {a[2], a[3]}, {c[0], c[1]}, {c[2], c[3]}};
      float2 y[4];
      float2 inv = make_float2(1.f, 1.f);
      if (weight != nullptr) {
        float2 two = __fmul2_rn(x[0], x[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) two = __ffma2_rn(x[i], x[i], two);
        float ss = two.x + two.y;
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        inv.x = inv.y = rsqrtf(ss * (1.f / D) + p.eps);
      }
      if (turns) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 partner = kInterleaved ? make_float2(x[i].y, x[i].x) : x[i ^ 2];
          y[i] = __fmul2_rn(__ffma2_rn(x[i], P[i], __fmul2_rn(partner, Q[i])), inv);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = __fmul2_rn(__fmul2_rn(x[i], P[i]), inv);
      }
      if (turns || weight != nullptr) {  // columns that nothing touches stay as they are, bit for bit
        const float ya[4] = {y[0].x, y[0].y, y[1].x, y[1].y}, yc[4] = {y[2].x, y[2].y, y[3].x, y[3].y};
        xa[u].set(ya);
        xb[u].set(yc);
      }
    }
    if (h < heads) {
      xa[u].store(dst + h * D + oa);
      xb[u].store(dst + h * D + ob);
    }
  };
  auto weight_of = [&](int section) { return section == 0 ? p.q_weight : section == 1 ? p.k_weight : nullptr; };
  auto target_of = [&](int section) {
    return section == 0 ? p.q_out + r * p.q_out_stride : (section == 1 ? p.k_pool : p.v_pool) + row * p.H_kv * D;
  };
  const int kv_heads = row >= 0 ? p.H_kv : 0;  // that are stored
  for (;;) {
    if constexpr (kMixed) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int step = g + u * parts, of = section_of(step);
        if (step < all_steps)
          finish_step(u, of, weight_of(of), target_of(of), (step - first_of(of)) * kVecs + vec,
                      of == 0 ? p.H_q : kv_heads);
      }
    } else {
      const T* weight = weight_of(section);
      T* dst = target_of(section);
      const int stored = section == 0 ? p.H_q : kv_heads;
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        finish_step(u, section, weight, dst, (g + u * parts) * kVecs + vec, stored);
    }
    g += kBatch * parts;
    if (!settle()) return;
    load();
  }
}

template <typename T>
ts_status launch(int D, const void* q, const void* k_new, const void* v_new, const void* q_weight,
                 const void* k_weight, void* k_pool, void* v_pool, void* q_out, RopeParams<T>& p,
                 cudaStream_t stream) {
  p.q = static_cast<const T*>(q), p.k_new = static_cast<const T*>(k_new), p.v_new = static_cast<const T*>(v_new);
  p.q_weight = static_cast<const T*>(q_weight), p.k_weight = static_cast<const T*>(k_weight);
  p.k_pool = static_cast<T*>(k_pool), p.v_pool = static_cast<T*>(v_pool), p.q_out = static_cast<T*>(q_out);
  const int vecs = 256 / D, steps = (p.H_q + vecs - 1) / vecs + 2 * ((p.H_kv + vecs - 1) / vecs);
  // Shares of a row, for as many warps as the device holds (32 / 8 heads of 128: 256 rows in shares 5.5 us, whole
  // 10.1; 960 rows 8.6 and 10.2; 4,800 rows whole 22.7, in two shares 29.0).
  const int64_t want = static_cast<int64_t>(device_sm_count()) * 32;
  p.parts = static_cast<int32_t>(want / p.T_rows);
  if (p.parts < 1) p.parts = 1;
  if (p.parts > steps) p.parts = steps;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(p.T_rows) * p.parts - 1) / kWarps + 1));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // A row of few steps, or a share of one, is taken in batches that mix queries, keys and values: fewer waits one
  // after another (float32, 4 + 2 x 2 heads of 64: 12.9 us for 10,000 rows, 26 in batches of their own). Whole rows
  // of many steps are not: their batches' places are simpler to compute (18,900 rows of 32 / 8 heads of 128: 78.6
  // us, mixed 94).
  const bool mixed = p.parts > 1 || steps <= 3 * kBatch;
  auto pick = [&](auto interleaved, auto mix) {
    return D == 64 ? rope_append_kernel<T, 64, decltype(interleaved)::value, decltype(mix)::value>
                   : rope_append_kernel<T, 128, decltype(interleaved)::value, decltype(mix)::value>;
  };
  using Yes = std::true_type;
  using No = std::false_type;
  auto kern = p.interleaved ? (mixed ? pick(Yes(), Yes()) : pick(Yes(), No()))
                            : (mixed ? pick(No(), Yes()) : pick(No(), No()));
  LaunchTrace trace("rope_append_kernel", stream);
  return cuda_check(cudaLaunchKernelEx(&cfg, kern, p), "ts_kv_append_chunk_rope: launch");
}

}  // namespace
}  // namespace ts

extern "C" ts_status ts_kv_append_chunk_rope(const void* q, int64_t q_stride, const void* k_new, const void* v_new,
                                             int64_t new_stride, const void* q_weight, const void* k_weight,
                                             float eps, const float* inv_freq, int32_t rot_dim, int32_t interleaved,
                                             void* k_pool, void* v_pool, const int32_t* block_table,
                                             int32_t bt_stride, const int32_t* seq_lens, const int32_t* q_indptr,
                                             int32_t T, int32_t B, int32_t H_q, int32_t H_kv, int32_t D,
                                             int32_t page_size, int32_t num_pages, ts_dtype dtype, void* q_out,
                                             int64_t q_out_stride, void* stream) {
  using namespace ts;
  const char* who = "ts_kv_append_chunk_rope";
  if (T < 0 || B < 0 || H_q <= 0 || H_kv <= 0 || D <= 0 || page_size <= 0 || num_pages <= 0 || bt_stride <= 0)
    return fail(TS_ERR_INVALID_ARG, "%s: bad sizes (T=%d B=%d H_q=%d H_kv=%d D=%d ps=%d P=%d bt=%d)", who, T, B, H_q,
                H_kv, D, page_size, num_pages, bt_stride);
  if (dtype != TS_F32 && dtype != TS_BF16)
    return fail(TS_ERR_INVALID_ARG, "%s: bad dtype %d", who, static_cast<int>(dtype));
  if (rot_dim < 0 || rot_dim > D)
    return fail(TS_ERR_INVALID_ARG, "%s: rot_dim=%d outside [0, D=%d]", who, rot_dim, D);
  if (!std::isfinite(eps) || eps < 0.f) return fail(TS_ERR_INVALID_ARG, "%s: bad eps", who);
  if (D != 64 && D != 128) return fail(TS_ERR_UNSUPPORTED, "%s: D=%d (supported 64, 128)", who, D);
  if (rot_dim % 8 != 0) return fail(TS_ERR_UNSUPPORTED, "%s: rot_dim=%d is not a multiple of 8", who, rot_dim);
  const int64_t es = dtype == TS_F32 ? 4 : 2;
  if (H_q > 4096 || H_kv > 4096) return fail(TS_ERR_UNSUPPORTED, "%s: more than 4096 heads", who);
  const int64_t q_width = static_cast<int64_t>(H_q) * D, width = static_cast<int64_t>(H_kv) * D;
  if (q_stride < q_width || q_out_stride < q_width || new_stride < width)
    return fail(TS_ERR_INVALID_ARG, "%s: rows closer together than they are wide", who);
  if (T == 0 || B == 0) return TS_OK;
  if (!q || !k_new || !v_new || !k_pool || !v_pool || !block_table || !seq_lens || !q_indptr || !q_out ||
      (rot_dim > 0 && !inv_freq))
    return fail(TS_ERR_INVALID_ARG, "%s: null pointer", who);
  if (q_stride * es % 16 != 0 || q_out_stride * es % 16 != 0 || new_stride * es % 16 != 0)
    return fail(TS_ERR_UNSUPPORTED, "%s: row steps must be multiples of 16 B", who);
  for (const void* x : {q, k_new, v_new, q_weight, k_weight, static_cast<const void*>(k_pool),
                        static_cast<const void*>(v_pool), static_cast<const void*>(q_out)})
    if (reinterpret_cast<uintptr_t>(x) % 16 != 0)
      return fail(TS_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", who);
  if (reinterpret_cast<uintptr_t>(inv_freq) % 4 != 0)
    return fail(TS_ERR_INVALID_ARG, "%s: inv_freq must be 4-byte aligned", who);
  auto fill = [&](auto p) {
    p.inv_freq = inv_freq;
    p.block_table = block_table, p.seq_lens = seq_lens, p.q_indptr = q_indptr;
    p.q_stride = q_stride, p.new_stride = new_stride, p.q_out_stride = q_out_stride;
    p.bt_stride = bt_stride, p.T_rows = T, p.B = B, p.H_q = H_q, p.H_kv = H_kv, p.num_pages = num_pages;
    p.rot = rot_dim, p.interleaved = interleaved != 0, p.eps = eps;
    return launch(D, q, k_new, v_new, q_weight, k_weight, k_pool, v_pool, q_out, p,
                  static_cast<cudaStream_t>(stream));
  };
  if (dtype == TS_BF16) return fill(RopeParams<__nv_bfloat16>{.page_size = PageSize(page_size)});
  return fill(RopeParams<float>{.page_size = PageSize(page_size)});
}
