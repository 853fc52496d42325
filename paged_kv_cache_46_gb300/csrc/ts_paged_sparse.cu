// ts_paged_decode_sparse_attn: decode attention over chosen pages, a list for
// every query row and kv head (ts_select_pages makes them).
//
// Of a query row at position p, over the tokens t <= p of the listed pages:
//   s_t = scale * <q, K_t>,  O = sum_t softmax(s)_t V_t,  LSE = log sum_t exp(s_t).
//
// A list entry read is page_size x D values of K and of V, and HBM bounds the
// call: a row of one kv head is 128 to 512 bytes, its neighbours belong to the
// other heads.
//
// Split: the entries of all items (a query row and kv head) in order are cut into
// equal contiguous ranges, one per warp of a grid that fills the device; a row
// counts min(pages, its pages) entries, found on the device, so that short
// sequences cost what they hold. Warps are workers of their own: nothing in a
// CTA is shared but the prefix sums of that plan. A range that ends inside an
// item leaves a float32 state, at most two per warp, which sparse_merge_kernel
// joins; an item within one range is written at once. Few items (take_whole) go to a
// CTA of eight warps each instead, which join their states in shared memory.
//
// bf16 (sparse_mma_kernel): tiles of 16 tokens, two (D = 64: four) per warp in
// flight, brought by the TMA as boxes of one kv head's 8 or 16 rows and 64 columns,
// with the 128-byte swizzle so that ldmatrix meets every bank once. (Copies of a row
// each by its lane, cp.async.bulk, issue one after another: issue slots 32 % active,
// with boxes 23 %.) The g query heads are the rows of an m16n8k16 product, padded to
// 16: a 128-row tcgen05 tile would be 4 / 128 full, and these products keep the
// tensor pipe active 15 % of the time. Both operands of P V are bf16: the weights
// enter as two terms, rounded weights in the rows of the heads and what the rounding
// left in the eight rows of padding, so that they count with 16 bits. 64 rows of 128
// pages of 16 (8 kv heads of 128, 4 queries each): 90 to 92 us with the join, 536 MB at
// 5.9 TB/s; nine tenths of the first kernel's warps end 76 to 85 us after the start. Two
// stages and two CTAs an SM: 93.5 us when that was measured, three stages 97.3, six
// stages and one CTA 103, two stages and three CTAs 96.9, one stage and four CTAs 101.
// float32 (sparse_f32_kernel): on the CUDA cores, packed multiply-adds. Tiles of
// eight tokens, two (D = 64: four) per warp in flight. For the scores a lane takes a
// key and a quarter of its columns, so that a value of K is read once for the g
// heads and the sums need two exchanges, not five per head; for P V it takes four
// columns of all keys, with the weights from shared memory. 20 sequences of 57 pages
// of 32, 4 kv heads of 128 (146 MB): one query a head 30 us, 4.9 TB/s (a row over all
// lanes 48 us); eight queries a head 45 us, 3.2 TB/s, bound by multiply-adds and by
// reading each query's value from shared memory once per key of a lane (85).
#include "ts_ranges.cuh"
#include "ts_tcgen05.cuh"

#include <cmath>

namespace ts {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kWholeWarps = 8;  // of a CTA that takes an item whole
constexpr int kParts = 32;  // ranges that an item is cut into at most, and one more at its end
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
  int64_t* plan;    // [kThreads + 1] entries in front of each chunk of rows, kept for the merge
  float* part_o;    // [2 * warps, g, D]
  float* part_lse;  // [2 * warps, g], base 2
  uint32_t* err_word;
  int32_t bt_stride, rows, q_len, H_kv, page_size, num_pages, pages, warps;
  float scale_log2;
};

// Entries of a row's lists that are taken.
__device__ __forceinline__ int row_entries(const SparseParams& p, int row) {
  const int pos = row_position(p, row);
  return pos < 0 ? 0 : min(p.pages, pos / p.page_size + 1);
}
// Entries of a warp's range, of `total` in all.
__device__ __forceinline__ int64_t range_of(const SparseParams& p, int64_t total) {
  return max(even_range(total, p.warps), static_cast<int64_t>((p.pages + kParts - 1) / kParts));
}

// A listed page: its pool page and how many of its tokens the row sees (0: none).
struct Listed {
  int32_t page, tokens;
};
__device__ __forceinline__ Listed listed_page(const SparseParams& p, const Walk& w, int pos, int i) {
  Listed e{0, 0};
  if (i >= w.i1) return e;
  const int idx = p.page_idx[(static_cast<int64_t>(w.row) * p.H_kv + w.h) * p.pages + i];
  if (idx < 0 || static_cast<int64_t>(idx) * p.page_size > pos) return e;
  const int page =
      idx < p.bt_stride ? p.block_table[static_cast<int64_t>(w.row / p.q_len) * p.bt_stride + idx] : -1;
  if (page < 0 || page >= p.num_pages) {
    set_device_error(p.err_word, TS_DEVERR_PAGE_RANGE);
    return e;
  }
  e.page = page;
  e.tokens = min(p.page_size, pos - idx * p.page_size + 1);
  return e;
}

template <typename T>
__device__ __forceinline__ void store2(T* to, float x, float y) {
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint32_t*>(to) = float2_to_bf16x2(x, y);
  else
    *reinterpret_cast<float2*>(to) = make_float2(x, y);
}

// Where a segment's state of query head i goes: its result, or one of the warp's
// two places in the workspace (0 where the item began before the range).
template <typename T, int D>
struct Target {
  T* out;
  float* lse;
  float* part_o;
  float* part_lse;
  __device__ __forceinline__ Target(const SparseParams& p, const Walk& w, int64_t warp, int g, int i) {
    out = nullptr, lse = nullptr, part_o = nullptr, part_lse = nullptr;
    if (w.whole()) {
      const int64_t at = static_cast<int64_t>(w.row) * p.H_kv * g + w.h * g + i;
      out = static_cast<T*>(p.out) + at * D;
      if (p.lse != nullptr) lse = p.lse + at;
    } else {
      const int64_t at = (2 * warp + (w.i0 == 0)) * g + i;
      part_o = p.part_o + at * D;
      part_lse = p.part_lse + at;
    }
  }
  __device__ __forceinline__ void put(int d, float x, float y) const {
    if (out != nullptr)
      store2(out + d, x, y);
    else
      store2(part_o + d, x, y);
  }
  __device__ __forceinline__ void put_lse(float lse2) const {
    if (part_lse != nullptr)
      *part_lse = lse2;
    else if (lse != nullptr)
      *lse = lse2 * kLn2S;
  }
};

// A warp's part of an item that its CTA takes whole.
template <int kOf>
__device__ __forceinline__ bool start_whole(const SparseParams& p, Walk& w, int warp) {
  w.row = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.H_kv));
  w.h = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.H_kv));
  w.count = row_entries(p, w.row);
  w.i0 = static_cast<int>(static_cast<int64_t>(w.count) * warp / kOf);
  w.i1 = static_cast<int>(static_cast<int64_t>(w.count) * (warp + 1) / kOf);
  w.at = w.end = w.item0 = 0;
  return true;
}

// The warps' states of an item, [warps][G][D] with their references and sums, to its result.
template <typename T, int D, int G, int kOf>
__device__ __forceinline__ void join_warps(const SparseParams& p, const Walk& w, const float* states,
                                           const float (&m)[kOf][G], const float (&sum)[kOf][G]) {
  __syncthreads();
  for (int e = threadIdx.x; e < G * D / 4; e += kOf * 32) {
    const int i = e / (D / 4), d = e % (D / 4) * 4;
    float top = m[0][i];
#pragma unroll
    for (int k = 1; k < kOf; ++k) top = fmaxf(top, m[k][i]);
    const float ref = top == -INFINITY ? 0.f : top;
    float total = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kOf; ++k) {
      const float a = fast_exp2(m[k][i] - ref);
      const float4 x = *reinterpret_cast<const float4*>(states + (k * G + i) * D + d);
      total = fmaf(a, sum[k][i], total);
      o = make_float4(fmaf(a, x.x, o.x), fmaf(a, x.y, o.y), fmaf(a, x.z, o.z), fmaf(a, x.w, o.w));
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;  // (NaN stays NaN)
    const int64_t at = (static_cast<int64_t>(w.row) * p.H_kv + w.h) * G + i;
    T* out = static_cast<T*>(p.out) + at * D + d;
    store2(out, o.x * inv, o.y * inv);
    store2(out + 2, o.z * inv, o.w * inv);
    if (d == 0 && p.lse != nullptr) p.lse[at] = total == 0.f ? -INFINITY : (ref + log2f(total)) * kLn2S;
  }
}

// ---------------------------------------------------------------------------
// bf16
// ---------------------------------------------------------------------------

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// (x, y) += the first eight rows of A (16 x 16, its last eight rows zero) x B (16 x 8).
__device__ __forceinline__ void mma_rows8(float& x, float& y, uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1) {
  [[maybe_unused]] float u, v;  // rows 8 .. 15
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %5}, {%7, %8}, "
      "{%0, %1, %9, %9};"
      : "+f"(x), "+f"(y), "=f"(u), "=f"(v)
      : "r"(a0), "r"(0u), "r"(a2), "r"(b0), "r"(b1), "f"(0.f));
}

// c += A (16 x 16: rows 0 .. 7 in a0, a2; rows 8 .. 15 in a1, a3) x B (16 x 8).
__device__ __forceinline__ void mma_rows16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                           uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// What the two rounded values of a pair leave, rounded in turn.
__device__ __forceinline__ uint32_t rest_bf16x2(float lo, float hi, uint32_t rounded) {
  const float2 f = bf16x2_to_float2(rounded);
  return float2_to_bf16x2(lo - f.x, hi - f.y);
}

// The sum of both terms' products; an infinite value of V times a remainder (0 or negative) must not count.
__device__ __forceinline__ float both_terms(float x, float rest) { return fabsf(x) == INFINITY ? x : x + rest; }

// A stage: 16 rows of K, then of V, in boxes of 64 columns (rows of 128 bytes, 128-byte swizzle).
template <int D>
struct MmaSmem {
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kOperand = 16 * D * 2, kStage = 2 * kOperand;
  static constexpr int bytes(int warps) { return warps * kStages * kStage; }
};

// The bits of the first n of eight rows.
__device__ __forceinline__ unsigned first_rows(int n) { return n >= 8 ? 0xffu : n <= 0 ? 0u : (1u << n) - 1u; }

// kWhole: a CTA per item instead of even ranges.
template <int D, int G, bool kWhole>
__global__ void __launch_bounds__((kWhole ? kWholeWarps : kWarps) * 32, kWhole ? 1 : 2) sparse_mma_kernel(
    const __grid_constant__ SparseParams p, const __grid_constant__ CUtensorMap kmap,
    const __grid_constant__ CUtensorMap vmap) {
  pdl_launch_dependents();
  using S = MmaSmem<D>;
  constexpr int kStages = S::kStages;
  extern __shared__ __align__(1024) unsigned char ring[];
  constexpr int kOf = kWhole ? kWholeWarps : kWarps;
  __shared__ __align__(8) uint64_t bars[kOf][kStages];
  __shared__ int64_t before[kWhole ? 1 : kThreads + 1];
  __shared__ float sh_m[kWhole ? kOf : 1][G], sh_sum[kWhole ? kOf : 1][G];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t worker = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if ((smem_u32(ring) & 1023u) != 0u) {
    if (threadIdx.x == 0) set_device_error(p.err_word, TS_DEVERR_SMEM_ALIGN);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kOf * kStages; ++i) mbar_init(smem_u32(&bars[0][0] + i), 1);
    fence_mbar_init();
  }
  Walk w;
  bool any;
  if constexpr (kWhole) {
    any = start_whole<kOf>(p, w, warp);
    __syncthreads();  // the barriers are set up
  } else {
    make_plan<kThreads>(p, before);
    const int64_t range = range_of(p, before[kThreads] * p.H_kv);
    any = w.start<kThreads>(p, before, worker * range, (worker + 1) * range, lane);
  }
  pdl_wait_primary();  // so far the lengths alone were read
  if (!kWhole && blockIdx.x == 0)
    for (int i = threadIdx.x; i <= kThreads; i += kThreads) p.plan[i] = before[i];
  if (!any) return;

  const uint32_t stage0 = smem_u32(ring) + warp * kStages * S::kStage;
  const uint32_t bar0 = smem_u32(&bars[warp][0]);
  const int quarter = lane & 3, head = lane >> 2;
  const int groups = p.page_size >> 3;  // of eight rows, in a page: 1, 2 or 4
  const int gshift = groups >> 1;       // its logarithm
  // ldmatrix rows and 16-byte chunks of a lane: keys 0 .. 7 and 8 .. 15, columns 0 .. 7 and 8 .. 15 of a step
  const int krow = (lane & 7) + ((lane >> 4) << 3), vrow = (lane & 7) + (lane & 8);
  const uint32_t kat = krow * 128 + ((((lane >> 3) & 1) ^ (krow & 7)) << 4);
  const uint32_t vat = vrow * 128 + (((lane >> 4) ^ (vrow & 7)) << 4);
  uint32_t stage = 0, parity = 0;       // of the next tile to be waited for
  bool ok = true;

  do {
    const int pos = row_position(p, w.row);
    // the item's queries, as rows of A
    uint32_t qa[D / 16][2];
    {
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) +
                                 (static_cast<int64_t>(w.row) * p.H_kv * G + w.h * G + head) * D + 2 * quarter;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qa[k][0] = head < G ? *reinterpret_cast<const uint32_t*>(src + 16 * k) : 0u;
        qa[k][1] = head < G ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 8) : 0u;
      }
    }
    float m = -INFINITY, sum = 0.f;
    float o[D / 8][4];  // of rounded weights, and of what the rounding left
#pragma unroll
    for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

    for (int c0 = w.i0; c0 < w.i1 && ok; c0 += 32) {
      const Listed e = listed_page(p, w, pos, c0 + lane);
      const int entries = min(32, w.i1 - c0);
      const int tiles = (entries * groups + 1) >> 1;
      // pool row and seen rows of the eight-row group i of these entries
      auto group = [&](int i, int& row, unsigned& rows) {
        const int from = i >> gshift, at = (i & (groups - 1)) * 8;
        const int page = __shfl_sync(0xffffffffu, e.page, from & 31), n = __shfl_sync(0xffffffffu, e.tokens, from & 31);
        row = page * p.page_size + at;
        rows = from < 32 ? first_rows(n - at) : 0u;
      };
      auto issue = [&](int t, uint32_t st) {
        int row0, row1;
        unsigned rows0, rows1;
        group(2 * t, row0, rows0);
        group(2 * t + 1, row1, rows1);
        if (lane == 0) {
          const uint32_t bar = bar0 + 8 * st, to = stage0 + st * S::kStage;
          if (groups > 1) {  // the tile is a part of one page
            mbar_arrive_expect_tx(bar, rows0 ? S::kStage : 0);
            if (rows0) {
#pragma unroll
              for (int x = 0; x < D / 64; ++x) {
                tma_load_3d(to + x * 2048, &kmap, 64 * x, w.h, row0, bar);
                tma_load_3d(to + S::kOperand + x * 2048, &vmap, 64 * x, w.h, row0, bar);
              }
            }
          } else {  // of two
            mbar_arrive_expect_tx(bar, (rows0 ? S::kStage / 2 : 0) + (rows1 ? S::kStage / 2 : 0));
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
              if (rows0) {
                tma_load_3d(to + x * 2048, &kmap, 64 * x, w.h, row0, bar);
                tma_load_3d(to + S::kOperand + x * 2048, &vmap, 64 * x, w.h, row0, bar);
              }
              if (rows1) {
                tma_load_3d(to + x * 2048 + 1024, &kmap, 64 * x, w.h, row1, bar);
                tma_load_3d(to + S::kOperand + x * 2048 + 1024, &vmap, 64 * x, w.h, row1, bar);
              }
            }
          }
        }
        __syncwarp();
      };
      uint32_t put = stage;
      for (int t = 0; t < kStages && t < tiles; ++t) {
        issue(t, put);
        put = put + 1 == kStages ? 0 : put + 1;
      }
      for (int t = 0; t < tiles; ++t) {
        int row0, row1;
        unsigned rows, rows1;
        group(2 * t, row0, rows);
        group(2 * t + 1, row1, rows1);
        rows |= rows1 << 8;
        ok = __all_sync(0xffffffffu, mbar_wait(bar0 + 8 * stage, parity));
        if (!ok) {  // leave, but not with copies in flight
          for (int i = t; i < tiles && i < t + kStages; ++i) {
            mbar_wait(bar0 + 8 * stage, parity);
            if (++stage == kStages) stage = 0, parity ^= 1u;
          }
          break;
        }
        if (rows != 0u) {
          const uint32_t ks = stage0 + stage * S::kStage, vs = ks + S::kOperand;
          if (rows != 0xffffu) {  // values of rows that are not seen must not count, not even NaN
            if (!(rows >> (lane & 15) & 1u)) {
              for (int i = lane >> 4; i < D / 8; i += 2)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vs + (i >> 3) * 2048 + (lane & 15) * 128 +
                                                                             (i & 7) * 16),
                             "r"(0u)
                             : "memory");
            }
            fence_async_smem();
            __syncwarp();
          }
          // scores: lane holds keys 2 quarter + {0, 1} and 8 more of query head `head`
          float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            uint32_t b[4];
            ldmatrix4(b, ks + (k >> 2) * 2048 + (kat ^ ((k & 3) << 5)));
            mma_rows8(s[0], s[1], qa[k][0], qa[k][1], b[0], b[1]);
            mma_rows8(s[2], s[3], qa[k][0], qa[k][1], b[2], b[3]);
          }
          const unsigned seen = rows >> (2 * quarter);
          s[0] = seen & 1u ? s[0] * p.scale_log2 : -INFINITY;
          s[1] = seen & 2u ? s[1] * p.scale_log2 : -INFINITY;
          s[2] = seen & 0x100u ? s[2] * p.scale_log2 : -INFINITY;
          s[3] = seen & 0x200u ? s[3] * p.scale_log2 : -INFINITY;
          float top = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          top = fmaxf(top, m);
          if (__any_sync(0xffffffffu, top > m)) {
            const float scale = fast_exp2(m - (top == -INFINITY ? 0.f : top));
            m = top;
            sum *= scale;
#pragma unroll
            for (int j = 0; j < D / 8; ++j) o[j][0] *= scale, o[j][1] *= scale, o[j][2] *= scale, o[j][3] *= scale;
          }
          const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[i] = fast_exp2(s[i] - ref);
            sum += s[i];
          }
          const uint32_t p0 = float2_to_bf16x2(s[0], s[1]), p1 = float2_to_bf16x2(s[2], s[3]);
          const uint32_t r0 = rest_bf16x2(s[0], s[1], p0), r1 = rest_bf16x2(s[2], s[3], p1);
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            uint32_t b[4];
            ldmatrix4_trans(b, vs + (j >> 2) * 2048 + (vat ^ ((j & 3) << 5)));
            mma_rows16(o[2 * j], p0, r0, p1, r1, b[0], b[1]);
            mma_rows16(o[2 * j + 1], p0, r0, p1, r1, b[2], b[3]);
          }
        }
        __syncwarp();
        if (t + kStages < tiles) issue(t + kStages, stage);
        if (++stage == kStages) {
          stage = 0;
          parity ^= 1u;
        }
      }
    }
    if (!kWhole && !ok) break;
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    if constexpr (kWhole) {
      __syncthreads();  // all stages have been read: the ring takes the states
      float* states = reinterpret_cast<float*>(ring);
      if (head < G) {
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
          store2(states + (warp * G + head) * D + 8 * j + 2 * quarter, both_terms(o[j][0], o[j][2]),
                 both_terms(o[j][1], o[j][3]));
        if (quarter == 0) sh_m[warp][head] = m, sh_sum[warp][head] = sum;
      }
      join_warps<__nv_bfloat16, D, G, kOf>(p, w, states, sh_m, sh_sum);
      break;
    } else if (head < G) {
      const Target<__nv_bfloat16, D> to(p, w, worker, G, head);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;  // (NaN stays NaN)
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
        to.put(8 * j + 2 * quarter, both_terms(o[j][0], o[j][2]) * inv, both_terms(o[j][1], o[j][3]) * inv);
      if (quarter == 0) to.put_lse(sum == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m) + log2f(sum));
    }
  } while (w.next(p));
  if (!ok && lane == 0) set_device_error(p.err_word, TS_DEVERR_TIMEOUT);
}

// ---------------------------------------------------------------------------
// float32
// ---------------------------------------------------------------------------

// A stage: 8 rows of K, then of V, in boxes of 32 columns (rows of 128 bytes, 128-byte swizzle). Behind the
// stages, per warp: the item's queries, a quarter of the columns per 16-byte step in the banks, and the
// weights and scales of a tile.
template <int D, int G>
struct F32Smem {
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kOperand = 8 * D * 4, kStage = 2 * kOperand;
  static constexpr int kPart = D / 4 + 4;  // floats of a quarter of a query, and their padding
  static constexpr int kQuery = G * 4 * kPart * 4, kWeights = G * 8 * 4;
  static constexpr int kWarp = kQuery + kWeights + G * 4 + (G < 4 ? 16 - G * 4 : 0);
  static constexpr int bytes(int warps) { return warps * (kStages * kStage + kWarp); }
};

template <int D, int G, bool kWhole>
__global__ void __launch_bounds__((kWhole ? kWholeWarps : kWarps) * 32, kWhole ? 1 : 2) sparse_f32_kernel(
    const __grid_constant__ SparseParams p, const __grid_constant__ CUtensorMap kmap,
    const __grid_constant__ CUtensorMap vmap) {
  pdl_launch_dependents();
  using S = F32Smem<D, G>;
  constexpr int kStages = S::kStages, kPart = S::kPart;
  constexpr int kMine = G >= 4 ? G / 4 : 1;  // heads whose scores a lane keeps
  extern __shared__ __align__(1024) unsigned char ring[];
  constexpr int kOf = kWhole ? kWholeWarps : kWarps;
  __shared__ __align__(8) uint64_t bars[kOf][kStages];
  __shared__ int64_t before[kWhole ? 1 : kThreads + 1];
  __shared__ float sh_m[kWhole ? kOf : 1][G], sh_sum[kWhole ? kOf : 1][G];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t worker = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if ((smem_u32(ring) & 1023u) != 0u) {
    if (threadIdx.x == 0) set_device_error(p.err_word, TS_DEVERR_SMEM_ALIGN);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kOf * kStages; ++i) mbar_init(smem_u32(&bars[0][0] + i), 1);
    fence_mbar_init();
  }
  Walk w;
  bool any;
  if constexpr (kWhole) {
    any = start_whole<kOf>(p, w, warp);
    __syncthreads();  // the barriers are set up
  } else {
    make_plan<kThreads>(p, before);
    const int64_t range = range_of(p, before[kThreads] * p.H_kv);
    any = w.start<kThreads>(p, before, worker * range, (worker + 1) * range, lane);
  }
  pdl_wait_primary();  // so far the lengths alone were read
  if (!kWhole && blockIdx.x == 0)
    for (int i = threadIdx.x; i <= kThreads; i += kThreads) p.plan[i] = before[i];
  if (!any) return;

  unsigned char* stages = ring + warp * kStages * S::kStage;
  unsigned char* own = ring + kOf * kStages * S::kStage + warp * S::kWarp;
  float* qs = reinterpret_cast<float*>(own);
  float* weights = reinterpret_cast<float*>(own + S::kQuery);                 // [G][8]
  float* scales = reinterpret_cast<float*>(own + S::kQuery + S::kWeights);    // [G]
  const uint32_t stage0 = smem_u32(stages), bar0 = smem_u32(&bars[warp][0]);
  // scores: a lane takes one of the eight keys and a quarter of the columns; the heads it keeps follow from it
  const int key = lane & 7, part = lane >> 3;
  int mine = 0;
#pragma unroll
  for (int n = G / 2, o = 16; n > 0 && o >= 8; n >>= 1, o >>= 1) mine += (lane & o) ? n : 0;
  // P V: four columns of all keys (D = 64: of the half of the keys), rows of V as K's
  const int vlane = D == 128 ? lane : lane & 15, vhalf = D == 128 ? 0 : lane >> 4;
  constexpr int kVRows = D == 128 ? 8 : 4;
  const int groups = p.page_size >> 3;  // of eight rows, in a page: 1, 2 or 4
  const int gshift = groups >> 1;       // its logarithm
  uint32_t stage = 0, parity = 0;       // of the next tile to be waited for
  bool ok = true;

  do {
    const int pos = row_position(p, w.row);
    {
      const float* src = static_cast<const float*>(p.q) + (static_cast<int64_t>(w.row) * p.H_kv * G + w.h * G) * D;
      __syncwarp();  // the item before has read its queries
      for (int i = lane; i < G * D / 4; i += 32) {
        const int head = i / (D / 4), d = i % (D / 4) * 4;
        float4 x = *reinterpret_cast<const float4*>(src + head * D + d);
        x = make_float4(x.x * p.scale_log2, x.y * p.scale_log2, x.z * p.scale_log2, x.w * p.scale_log2);
        *reinterpret_cast<float4*>(qs + (head * 4 + d / (D / 4)) * kPart + d % (D / 4)) = x;
      }
      __syncwarp();
    }
    float m[kMine], sum[kMine];
    float2 acc[G][2];
#pragma unroll
    for (int i = 0; i < kMine; ++i) m[i] = -INFINITY, sum[i] = 0.f;
#pragma unroll
    for (int i = 0; i < G; ++i) acc[i][0] = acc[i][1] = make_float2(0.f, 0.f);

    for (int c0 = w.i0; c0 < w.i1 && ok; c0 += 32) {
      const Listed e = listed_page(p, w, pos, c0 + lane);
      const int tiles = min(32, w.i1 - c0) * groups;
      // pool row of tile t, and how many of its rows are seen
      auto tile = [&](int t, int& row) {
        const int from = t >> gshift, at = (t & (groups - 1)) * 8;
        row = __shfl_sync(0xffffffffu, e.page, from) * p.page_size + at;
        return min(8, __shfl_sync(0xffffffffu, e.tokens, from) - at);
      };
      auto issue = [&](int t, uint32_t st) {
        int row;
        const int n = tile(t, row);
        if (lane == 0) {
          const uint32_t bar = bar0 + 8 * st, to = stage0 + st * S::kStage;
          mbar_arrive_expect_tx(bar, n > 0 ? S::kStage : 0);
          if (n > 0) {
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
              tma_load_3d(to + x * 1024, &kmap, 32 * x, w.h, row, bar);
              tma_load_3d(to + S::kOperand + x * 1024, &vmap, 32 * x, w.h, row, bar);
            }
          }
        }
        __syncwarp();
      };
      uint32_t put = stage;
      for (int t = 0; t < kStages && t < tiles; ++t) {
        issue(t, put);
        put = put + 1 == kStages ? 0 : put + 1;
      }
      for (int t = 0; t < tiles; ++t) {
        int row;
        const int n = tile(t, row);
        ok = __all_sync(0xffffffffu, mbar_wait(bar0 + 8 * stage, parity));
        if (!ok) {  // leave, but not with copies in flight
          for (int i = t; i < tiles && i < t + kStages; ++i) {
            mbar_wait(bar0 + 8 * stage, parity);
            if (++stage == kStages) stage = 0, parity ^= 1u;
          }
          break;
        }
        if (n > 0) {
          const unsigned char* ks = stages + stage * S::kStage;
          const unsigned char* vs = ks + S::kOperand;
          // a quarter of the columns of this lane's key
          constexpr int kChunks = D / 16;  // of four columns
          const unsigned char* krow = ks + (D == 128 ? part : part >> 1) * 1024 + key * 128;
          const int chunk0 = D == 128 ? 0 : (part & 1) * 4;
          float2 two[G];
#pragma unroll
          for (int i = 0; i < G; ++i) two[i] = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            const float4 x = *reinterpret_cast<const float4*>(krow + (((chunk0 + c) ^ key) << 4));
#pragma unroll
            for (int i = 0; i < G; ++i) {
              const float4 y = *reinterpret_cast<const float4*>(qs + (i * 4 + part) * kPart + 4 * c);
              two[i] = __ffma2_rn(make_float2(x.x, x.y), make_float2(y.x, y.y), two[i]);
              two[i] = __ffma2_rn(make_float2(x.z, x.w), make_float2(y.z, y.w), two[i]);
            }
          }
          float s[G];
#pragma unroll
          for (int i = 0; i < G; ++i) s[i] = two[i].x + two[i].y;
          int o = 16;
#pragma unroll
          for (int k = G / 2; k > 0 && o >= 8; k >>= 1, o >>= 1) {
            const bool upper = (lane & o) != 0;
#pragma unroll
            for (int i = 0; i < k; ++i) {
              const float send = upper ? s[i] : s[i + k];
              s[i] = (upper ? s[i + k] : s[i]) + __shfl_xor_sync(0xffffffffu, send, o);
            }
          }
#pragma unroll
          for (; o >= 8; o >>= 1) s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
          bool rises = false;
#pragma unroll
          for (int i = 0; i < kMine; ++i) {
            if (key >= n) s[i] = -INFINITY;
            float top = s[i];
#pragma unroll
            for (int x = 4; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            float scale = 1.f;
            if (top > m[i]) {
              scale = fast_exp2(m[i] - top);
              m[i] = top;
              sum[i] *= scale;
              rises = true;
            }
            const float weight = fast_exp2(s[i] - (m[i] == -INFINITY ? 0.f : m[i]));
            sum[i] += weight;
            weights[(mine + i) * 8 + key] = weight;
            if (key == 0) scales[mine + i] = scale;
          }
          rises = __any_sync(0xffffffffu, rises);
          __syncwarp();
          if (rises) {
#pragma unroll
            for (int i = 0; i < G; ++i) {
              const float scale = scales[i];
              acc[i][0] = make_float2(acc[i][0].x * scale, acc[i][0].y * scale);
              acc[i][1] = make_float2(acc[i][1].x * scale, acc[i][1].y * scale);
            }
          }
          const unsigned char* vcol = vs + (vlane >> 3) * 1024;
#pragma unroll
          for (int k4 = 0; k4 < kVRows; k4 += 4) {
            const int first = vhalf * 4 + k4;
            float4 pw[G];
#pragma unroll
            for (int i = 0; i < G; ++i) pw[i] = *reinterpret_cast<const float4*>(weights + i * 8 + first);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int r = first + k;
              if (r >= n) continue;  // (what such rows hold must not count, not even NaN)
              const float4 v = *reinterpret_cast<const float4*>(vcol + r * 128 + (((vlane & 7) ^ r) << 4));
#pragma unroll
              for (int i = 0; i < G; ++i) {
                const float x = k == 0 ? pw[i].x : k == 1 ? pw[i].y : k == 2 ? pw[i].z : pw[i].w;
                acc[i][0] = __ffma2_rn(make_float2(x, x), make_float2(v.x, v.y), acc[i][0]);
                acc[i][1] = __ffma2_rn(make_float2(x, x), make_float2(v.z, v.w), acc[i][1]);
              }
            }
          }
        }
        __syncwarp();
        if (t + kStages < tiles) issue(t + kStages, stage);
        if (++stage == kStages) {
          stage = 0;
          parity ^= 1u;
        }
      }
    }
    if (!kWhole && !ok) break;
    // sums over the keys, to all lanes
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
#pragma unroll
      for (int x = 4; x > 0; x >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], x);
      if (key == 0) weights[mine + i] = sum[i], scales[mine + i] = m[i];
    }
    __syncwarp();
    if constexpr (kWhole) {
      __syncthreads();  // all stages have been read: the ring takes the states
      float* states = reinterpret_cast<float*>(ring);
#pragma unroll
      for (int i = 0; i < G; ++i) {
        float x[4] = {acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y};
        if (D == 64) {
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] += __shfl_xor_sync(0xffffffffu, x[j], 16);
        }
        if (vhalf == 0)
          *reinterpret_cast<float4*>(states + (warp * G + i) * D + 4 * vlane) = make_float4(x[0], x[1], x[2], x[3]);
        if (lane == 0) sh_m[warp][i] = scales[i], sh_sum[warp][i] = weights[i];
      }
      join_warps<float, D, G, kOf>(p, w, states, sh_m, sh_sum);
      break;
    } else {
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const float total = weights[i], top = scales[i];
        const Target<float, D> to(p, w, worker, G, i);
        float x[4] = {acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y};
        if (D == 64) {
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] += __shfl_xor_sync(0xffffffffu, x[j], 16);
        }
        const float inv = total == 0.f ? 0.f : 1.f / total;  // (NaN stays NaN)
        if (vhalf == 0) {
          to.put(4 * vlane, x[0] * inv, x[1] * inv);
          to.put(4 * vlane + 2, x[2] * inv, x[3] * inv);
        }
        if (lane == 0) to.put_lse(total == 0.f ? -INFINITY : (top == -INFINITY ? 0.f : top) + log2f(total));
      }
    }
    __syncwarp();  // before the next item's weights
  } while (w.next(p));
  if (!ok && lane == 0) set_device_error(p.err_word, TS_DEVERR_TIMEOUT);
}

// ---------------------------------------------------------------------------

// Joins the states of items that were cut, and writes the rows that see nothing. A
// CTA per query row and kv head; g D / 4 threads hold four columns each, as often
// as they fit, and share the states.
template <typename T, int D, int G, int kMergeThreads>
__global__ void __launch_bounds__(kMergeThreads) sparse_merge_kernel(const SparseParams p) {
  constexpr int kCols = G * D / 4, kShares = kMergeThreads / kCols;
  __shared__ int32_t warp_sum[kMergeThreads / 32];
  __shared__ float weight[kParts + 2][G];
  __shared__ float4 part[kShares][kCols];
  __shared__ float sh_total[G], sh_top[G];
  pdl_launch_dependents();
  const int row = blockIdx.x / p.H_kv, h = blockIdx.x % p.H_kv, tid = threadIdx.x;
  const int count = row_entries(p, row), each = chunk_rows<kThreads>(p), chunk = row / each;
  // entries in front of the row, in its chunk
  int64_t in_front = 0;
  if (row > chunk * each) {
    int mine = 0;
    for (int r = chunk * each + tid; r < row; r += kMergeThreads) mine += row_entries(p, r);
    mine = __reduce_add_sync(0xffffffffu, mine);
    if ((tid & 31) == 0) warp_sum[tid >> 5] = mine;
    __syncthreads();
    for (int w = 0; w < kMergeThreads / 32; ++w) in_front += warp_sum[w];
  }
  pdl_wait_primary();  // so far the lengths alone were read
  in_front += p.plan[chunk];
  const int64_t range = range_of(p, p.plan[kThreads] * p.H_kv);
  const int64_t first = in_front * p.H_kv + static_cast<int64_t>(h) * count;
  const int64_t w0 = first / range, w1 = (first + count - 1) / range;
  if (count > 0 && w0 == w1) return;  // written already
  const int n = count > 0 ? static_cast<int>(w1 - w0) + 1 : 0;  // at most kParts + 1
  if (tid < 32) {
    for (int i = 0; i < G; ++i) {
      const float a = tid < n ? p.part_lse[(2 * (w0 + tid) + (tid == 0)) * G + i] : -INFINITY;
      const float c = tid + 32 < n ? p.part_lse[2 * (w0 + tid + 32) * G + i] : -INFINITY;
      float top = fmaxf(a, c);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float ref = top == -INFINITY ? 0.f : top, wa = fast_exp2(a - ref), wc = fast_exp2(c - ref);
      float total = wa + wc;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
      weight[tid][i] = wa;
      if (tid + 32 < kParts + 2) weight[tid + 32][i] = wc;
      if (tid == 0) sh_total[i] = total, sh_top[i] = ref;
    }
  }
  __syncthreads();
  const int share = tid / kCols, e = tid % kCols, i = e / (D / 4), d = e % (D / 4) * 4;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = share; k < n; k += kShares) {
    const float a = weight[k][i];
    const float4 x = *reinterpret_cast<const float4*>(p.part_o + ((2 * (w0 + k) + (k == 0)) * G + i) * D + d);
    o = make_float4(fmaf(a, x.x, o.x), fmaf(a, x.y, o.y), fmaf(a, x.z, o.z), fmaf(a, x.w, o.w));
  }
  part[share][e] = o;
  __syncthreads();
  if (share != 0) return;
#pragma unroll
  for (int k = 1; k < kShares; ++k) {
    const float4 x = part[k][e];
    o = make_float4(o.x + x.x, o.y + x.y, o.z + x.z, o.w + x.w);
  }
  const float total = sh_total[i], inv = total == 0.f ? 0.f : 1.f / total;  // (NaN stays NaN)
  const int64_t at = (static_cast<int64_t>(row) * p.H_kv + h) * G + i;
  T* out = static_cast<T*>(p.out) + at * D + d;
  store2(out, o.x * inv, o.y * inv);
  store2(out + 2, o.z * inv, o.w * inv);
  if (d == 0 && p.lse != nullptr) p.lse[at] = total == 0.f ? -INFINITY : (sh_top[i] + log2f(total)) * kLn2S;
}

// Warps of the grid: two CTAs on each SM, or as many as lists of full length keep busy.
int sparse_warps(int64_t items, int pages) {
  const int64_t least = (pages + kParts - 1) / kParts, most = (items * pages + least - 1) / least;
  const int64_t full = static_cast<int64_t>(paged_decode_ctas()) * 2 * kWarps;
  const int64_t n = most < full ? most : full;
  return static_cast<int>((n < 1 ? 1 : n) + kWarps - 1) / kWarps * kWarps;
}

struct SparseWs {
  size_t plan, part_o, part_lse, total;
  SparseWs(int warps, int g, int D) {
    plan = kWorkspaceAlign;
    part_o = align_up(plan + (kThreads + 1) * sizeof(int64_t), kWorkspaceAlign);
    part_lse = part_o + static_cast<size_t>(2) * warps * g * D * sizeof(float);
    total = align_up(part_lse + static_cast<size_t>(2) * warps * g * sizeof(float), kWorkspaceAlign);
  }
};

template <typename K, typename... A>
cudaError_t launch_pdl(K kern, unsigned grid, int threads, size_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// 3-D map over a pool [rows][H_kv][D] of es-byte values with a box of 128 bytes of one
// kv head's `rows` rows, 128-byte swizzle.
ts_status make_pool_map(CUtensorMap* map, const void* pool, int64_t pool_rows, int H_kv, int D, int es, int rows) {
  auto fn = tensor_map_encoder();
  if (!fn) return fail(TS_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H_kv),
                              static_cast<cuuint64_t>(pool_rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * es, static_cast<cuuint64_t>(H_kv) * D * es};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / es), 1, static_cast<cuuint32_t>(rows)}, ones[3] = {1, 1, 1};
  const auto type = es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  const CUresult r = fn(map, type, 3, const_cast<void*>(pool), dims, strides, box, ones,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(TS_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return TS_OK;
}

template <int kBytes>
ts_status prepare_ring(const void* kernel) {
  return cuda_check(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes),
                    "ts_paged_decode_sparse_attn: shared memory");
}

// Up to two items an SM: a CTA takes an item whole and joins its warps' states itself, one launch instead of two,
// unless the lists are so long and the items so few that most SMs would wait for them. Times of the call's kernels,
// whole and cut evenly, 8 kv heads of 128 (items of 0.5 MB are 64 pages of 16 in bf16): 8 items of 0.5 MB 9.6 and
// 8.3 us (the call, host-bound, 10.2 and 13.0), of 1 MB 16.4 and 9.9; 80 of 1 MB 16.9 and 17.6 (float32 with eight
// queries a head, 1.9 MB: 66 and 45); 128 of 0.5 MB 10.4 and 16.1, float32 of 1 MB 28 and 36; 256 of 0.5 MB 26.9 and
// 31.0; 512 of 0.5 MB 54.4 and 52.0.
bool take_whole(int64_t items, int64_t item_bytes) {
  const int64_t sms = paged_decode_ctas();
  return items <= 2 * sms && (item_bytes <= (512 << 10) || (4 * items >= 3 * sms && item_bytes <= (1 << 20)));
}

template <typename T, int D, int G, bool kWhole>
ts_status launch_first(const SparseParams& p, cudaStream_t s) {
  constexpr bool kBf16 = sizeof(T) == 2;
  constexpr int kOf = kWhole ? kWholeWarps : kWarps;
  constexpr int kBytes = kBf16 ? MmaSmem<D>::bytes(kOf) : F32Smem<D, G>::bytes(kOf);
  const auto kern = [] {
    if constexpr (kBf16)
      return sparse_mma_kernel<D, G, kWhole>;
    else
      return sparse_f32_kernel<D, G, kWhole>;
  }();
  ts_status st = prepare_once(reinterpret_cast<const void*>(kern), prepare_ring<kBytes>);
  if (st != TS_OK) return st;
  CUtensorMap kmap, vmap;
  const int64_t pool_rows = static_cast<int64_t>(p.num_pages) * p.page_size;
  const int box = kBf16 && p.page_size >= 16 ? 16 : 8;
  st = make_pool_map(&kmap, p.k_pool, pool_rows, p.H_kv, D, sizeof(T), box);
  if (st == TS_OK) st = make_pool_map(&vmap, p.v_pool, pool_rows, p.H_kv, D, sizeof(T), box);
  if (st != TS_OK) return st;
  const unsigned grid = static_cast<unsigned>(kWhole ? static_cast<int64_t>(p.rows) * p.H_kv : p.warps / kWarps);
  LaunchTrace trace(kBf16 ? "sparse_mma_kernel" : "sparse_f32_kernel", s);
  return cuda_check(launch_pdl(kern, grid, kOf * 32, kBytes, s, p, kmap, vmap), "ts_paged_decode_sparse_attn: launch");
}

template <typename T, int D, int G>
ts_status launch(const SparseParams& p, cudaStream_t s) {
  const int64_t items = static_cast<int64_t>(p.rows) * p.H_kv;
  const int64_t item_bytes = static_cast<int64_t>(p.pages) * p.page_size * (2 * D * sizeof(T));
  if (take_whole(items, item_bytes)) return launch_first<T, D, G, true>(p, s);
  const ts_status st = launch_first<T, D, G, false>(p, s);
  if (st != TS_OK) return st;
  // Items that fill the device are cut into few parts each: small CTAs, so that all are resident at once (512
  // items of 4 x 128: the call 90 us, with 512 threads 93). Few items are cut into many parts, which more
  // threads share. (Joined in the first kernel by the last warp to arrive, the call takes 94 us, and one of 2
  // items 16.0 instead of 8.0: the fences and atomics in a row take longer than a launch that waits early.)
  constexpr int kSmall = G * D / 4 < 128 ? 128 : G * D / 4;
  LaunchTrace trace("sparse_merge_kernel", s);
  const unsigned grid = static_cast<unsigned>(items);
  return cuda_check(items * 4 >= p.warps ? launch_pdl(sparse_merge_kernel<T, D, G, kSmall>, grid, kSmall, 0, s, p)
                                         : launch_pdl(sparse_merge_kernel<T, D, G, 512>, grid, 512, 0, s, p),
                    "ts_paged_decode_sparse_attn: merge launch");
}

template <typename T, int D>
ts_status launch(int g, const SparseParams& p, cudaStream_t s) {
  return g == 1 ? launch<T, D, 1>(p, s) : g == 2 ? launch<T, D, 2>(p, s) : g == 4 ? launch<T, D, 4>(p, s)
                                                                                  : launch<T, D, 8>(p, s);
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
  return SparseWs(sparse_warps(rows * H_kv, pages), H_q / H_kv, D).total;
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
  const int g = H_q / H_kv, warps = sparse_warps(rows * H_kv, pages);
  const SparseWs ws(warps, g, D);
  if (!workspace || workspace_bytes < ws.total || reinterpret_cast<uintptr_t>(workspace) % kWorkspaceAlign != 0)
    return fail(TS_ERR_WORKSPACE, "%s: workspace %zu B < %zu B needed or misaligned", who, workspace_bytes, ws.total);
  unsigned char* w = static_cast<unsigned char*>(workspace);
  const SparseParams p{q, k_pool, v_pool, block_table, seq_lens, page_idx, out, lse,
                       reinterpret_cast<int64_t*>(w + ws.plan), reinterpret_cast<float*>(w + ws.part_o),
                       reinterpret_cast<float*>(w + ws.part_lse), static_cast<uint32_t*>(workspace), bt_stride,
                       static_cast<int32_t>(rows), q_len, H_kv, page_size, num_pages, pages, warps, scale * kLog2eS};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == TS_BF16)
    return D == 64 ? launch<__nv_bfloat16, 64>(g, p, s) : launch<__nv_bfloat16, 128>(g, p, s);
  return D == 64 ? launch<float, 64>(g, p, s) : launch<float, 128>(g, p, s);
}
