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
// page_score_kernel: HBM bounds it (2 D + 4 bytes a page and head). A warp takes
// one kv head; sixteen pages are the rows of an m16n8k32 product of 8-bit whole
// numbers, the g query heads (padded to eight) its columns. The order of the codes
// along the sum is free, so that a lane's operands are 16 bytes of a page's codes as
// they lie in memory, and 16 bytes of a query head's; nothing goes through shared
// memory.
// The tiles of all rows and heads are cut evenly over one wave of warps (ts_ranges):
// 64 sequences of 4,096 .. 32,768 tokens (8 kv heads of 128, 4 queries each, pages of
// 16) 32 us, 158 MB at 4.9 TB/s; the fastest warps are done after 25. The tensor pipe is
// active 41 % of the time (64 clocks a product). With dp4a, sixteen lanes a page, 49 us.
// Every query row is scored by itself: the same with 2 and 4 tokens a sequence takes,
// with the choice, 65 and 122 us (one token: 38).
// page_pick_kernel: a CTA per query row and kv head. One histogram of 2048 equal
// bins between the smallest and the largest key finds the bin of the threshold;
// the few keys in it are ranked against each other (key, then page); a bit per
// chosen page and a sum over the words of bits give each its place in the list.
// Where many keys share the bin, it is cut in 2048 again first. Latency bounds it:
// 8,192 keys 4.9 us, of which loading them is 1.4, the histogram 1.2, the ranking 0.8
// and the list 1.5.
// page_select_kernel: both for smaller calls (whole_threads), a CTA an item, its keys in shared memory.
#include "ts_ranges.cuh"

#include <cmath>

namespace ts {
namespace {

// kResident: CTAs on an SM, 128 registers a thread (64 sequences 37.9 us and 131,072 tokens alone 11.9; with 5 37.1
// and 13.1, with 6 39.8; two waves of 5 42).
constexpr int kThreads = 128, kWarps = kThreads / 32, kResident = 4;
constexpr int kWholePages = 2048;  // at most, of a CTA that scores and chooses
constexpr int kBins = 2048, kKeys = 16, kRanked = 96;  // kKeys: in a thread's registers

struct SelectParams {
  const int8_t* bounds;
  const float* bound_scale;
  const int32_t* block_table;
  const int32_t* seq_lens;
  uint32_t* keys;  // [rows, H_kv, bt_stride]
  int32_t* page_idx;
  uint32_t* err_word;
  int32_t bt_stride, rows, q_len, H_kv, page_size, num_pages, pages, first, last, warps;
};

// Pages of the query at a row's position, as far as the table has slots; none in front of the first token.
__device__ __forceinline__ int pages_of(const SelectParams& p, int row, bool* past) {
  const int pos = row_position(p, row);
  if (pos < 0) return 0;
  const int have = pos / p.page_size + 1;
  *past = have > p.bt_stride;
  return min(have, p.bt_stride);
}
// Tiles of sixteen pages to be scored, where the row has more pages than are listed.
__device__ __forceinline__ int row_entries(const SelectParams& p, int row) {
  bool past;
  const int have = pages_of(p, row, &past);
  return have > p.pages ? (have + 15) / 16 : 0;
}

// Scores as whole numbers of their order: NaN above all, 0 is no score's.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 becomes 0: they are equal
  const uint32_t key = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
  return x != x ? 0xffffffffu : key;
}
// The larger of two scores; NaN if one is.
__device__ __forceinline__ float larger(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

// d += A (16 x 32, 8 bits) x B (32 x 8, 8 bits).
__device__ __forceinline__ void mma_s8(int32_t (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                       uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four consecutive values as floats.
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  const float2 a = bf16x2_to_float2(w.x), b = bf16x2_to_float2(w.y);
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// 16 of a page's bytes of bounds, read once; L2 fetches the rest of them (2 D: 256 or 128 bytes) with the first.
template <int kBytes>
__device__ __forceinline__ uint4 load_codes(const uint4* p) {
  uint4 w;
  if constexpr (kBytes == 256)
    asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "l"(p));
  else
    asm volatile("ld.global.L1::no_allocate.L2::128B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "l"(p));
  return w;
}

// Bytes that hold four whole numbers below zero, and those that do not.
__device__ __forceinline__ uint32_t negative_bytes(uint32_t w) { return ((w >> 7) & 0x01010101u) * 0xffu; }

// Keys of slots i .. end - 1 of a query row and kv head; a whole warp calls it. The first call of a kernel waits for
// the kernel in front of it once it has read lengths and block table.
template <typename T, int D, int G>
__device__ __forceinline__ void score_pages(const T* q, const SelectParams& p, int row, int h, int i, int end,
                                            uint32_t* keys, bool& waited) {
  constexpr int kChunks = 2 * D / 64;       // of 64 codes: a quad of lanes holds 16 each
  constexpr int kTiles = D == 128 ? 1 : 2;  // of sixteen pages, in flight
  const int lane = threadIdx.x & 31, quarter = lane & 3, at = lane >> 2;
  const int32_t* table = p.block_table + static_cast<int64_t>(row / p.q_len) * p.bt_stride;
  // rows `at` and `at` + 8 of the tiles in flight: pages, looked up a step ahead of their codes and scales
  int32_t page[kTiles][2];
  uint4 w[kTiles][2][kChunks];
  float s[kTiles][2];
  bool good[kTiles][2];
  auto look_up = [&](int first) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int slot = first + 16 * t + 8 * r + at;
        page[t][r] = slot < end ? table[slot] : -1;
      }
  };
  auto load = [&](int t) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      good[t][r] = static_cast<uint32_t>(page[t][r]) < static_cast<uint32_t>(p.num_pages);
      const int64_t place = static_cast<int64_t>(good[t][r] ? page[t][r] : 0) * p.H_kv + h;
      const uint4* src = reinterpret_cast<const uint4*>(p.bounds + place * 2 * D) + quarter;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) w[t][r][c] = load_codes<2 * D>(src + 4 * c);
      s[t][r] = p.bound_scale[place];
    }
  };
  look_up(i);
  if (!waited) pdl_wait_primary();  // so far lengths and block table alone were read
  waited = true;
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
    if (i + 16 * t < end) load(t);
  look_up(i + 16 * kTiles);

  // the codes of query head `at`, as columns of B: above zero beside the upper bounds, below beside the lower
  uint32_t code[kChunks][4];
  float q_scale = 0.f;
  {
    const int64_t head = (static_cast<int64_t>(row) * p.H_kv + h) * G + (G < 8 ? min(at, G - 1) : at);
    const T* src = q + head * D + 16 * quarter;
    uint32_t largest = 0u;
#pragma unroll
    for (int c = 0; c < kChunks / 2; ++c)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 x = load4(src + 64 * c + 4 * k);
        largest = max(max(max(magnitude(x.x), magnitude(x.y)), max(magnitude(x.z), magnitude(x.w))), largest);
      }
    largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, 1));
    largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, 2));
    const bool odd = largest >= 0x7f800000u;  // (its scale stays infinite or NaN, and so do its scores)
    q_scale = odd ? __uint_as_float(largest) : fmaxf(__uint_as_float(largest), 1e-10f) * (1.f / 127.f);
    const float inv = reciprocal(q_scale);
    auto quantize = [&](auto&& divide) {
#pragma unroll
      for (int c = 0; c < kChunks / 2; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 x = load4(src + 64 * c + 4 * k);
          // 1.5 * 2^23 more: the rounded number is in the last bits
          auto bits = [&](float v) { return __float_as_uint(divide(v) + 12582912.f); };
          const uint32_t low = __byte_perm(bits(x.x), bits(x.y), 0x0040);
          const uint32_t high = __byte_perm(bits(x.z), bits(x.w), 0x0040);
          const uint32_t word = odd ? 0u : __byte_perm(low, high, 0x5410), below = negative_bytes(word);
          code[c][k] = word & ~below;
          code[kChunks / 2 + c][k] = word & below;
        }
    };
    if (__any_sync(0xffffffffu, all_ones(q_scale)))  // see quotient()
      quantize([&](float x) { return __fdiv_rn(x, q_scale); });
    else
      quantize([&](float x) { return quotient(x, q_scale, inv); });
  }
  const float qs0 = __shfl_sync(0xffffffffu, q_scale, 8 * quarter);
  const float qs1 = __shfl_sync(0xffffffffu, q_scale, 8 * quarter + 4);

  for (; i < end; i += 16 * kTiles) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      const int first = i + 16 * t;
      if (first >= end) break;
      int32_t dot[4] = {0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        mma_s8(dot, w[t][0][c].x, w[t][1][c].x, w[t][0][c].y, w[t][1][c].y, code[c][0], code[c][1]);
        mma_s8(dot, w[t][0][c].z, w[t][1][c].z, w[t][0][c].w, w[t][1][c].w, code[c][2], code[c][3]);
      }
      const float scale[2] = {s[t][0], s[t][1]};
      const bool ok[2] = {good[t][0], good[t][1]};
      if (first + 16 * kTiles < end) load(t);
      float score[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {  // heads 2 quarter and 2 quarter + 1
        float k0 = static_cast<float>(dot[2 * r]) * qs0 * scale[r];
        const float k1 = static_cast<float>(dot[2 * r + 1]) * qs1 * scale[r];
        if (G > 1) k0 = larger(k0, k1);
        if (G < 8) k0 = 2 * quarter < G ? k0 : -INFINITY;
        if (G > 2) k0 = larger(k0, __shfl_xor_sync(0xffffffffu, k0, 1));
        if (G > 4) k0 = larger(k0, __shfl_xor_sync(0xffffffffu, k0, 2));
        if (G <= 2) k0 = __shfl_sync(0xffffffffu, k0, lane & 28);
        score[r] = k0;  // complete in the quad's first two lanes
      }
      const int slot = first + 8 * quarter + at;  // which store rows `at` and `at` + 8
      if (quarter < 2 && slot < end) {
        const bool fine = quarter ? ok[1] : ok[0];
        keys[slot] = fine ? order_key(quarter ? score[1] : score[0]) : 0u;
        if (!fine) set_device_error(p.err_word, TS_DEVERR_PAGE_RANGE);
      }
    }
    look_up(i + 32 * kTiles);
  }
}

template <typename T, int D, int G>
__global__ void __launch_bounds__(kThreads, kResident) page_score_kernel(const T* q, const SelectParams p) {
  pdl_launch_dependents();
  __shared__ int64_t before[kThreads + 1];
  const int64_t worker = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  make_plan<kThreads>(p, before);
  const int64_t range = even_range(before[kThreads] * p.H_kv, p.warps);
  Walk walk;
  if (!walk.start<kThreads>(p, before, worker * range, (worker + 1) * range, threadIdx.x & 31)) {
    pdl_wait_primary();
    return;
  }
  bool waited = false;
  do {
    bool past;
    const int have = pages_of(p, walk.row, &past);
    uint32_t* keys = p.keys + (static_cast<int64_t>(walk.row) * p.H_kv + walk.h) * p.bt_stride;
    score_pages<T, D, G>(q, p, walk.row, walk.h, 16 * walk.i0, min(have, 16 * walk.i1), keys, waited);
  } while (walk.next(p));
}

// Sums of v over the threads in front, and over all (uniform); `sums` is scratch of a word per warp.
template <int kWarpsOf>
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t (&sums)[kWarpsOf], uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();  // the sums of a scan before have been read
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  uint32_t mine = lane < kWarpsOf ? sums[lane] : 0u;
  total = __reduce_add_sync(0xffffffffu, mine);
  mine = lane < warp ? mine : 0u;
  return incl - v + __reduce_add_sync(0xffffffffu, mine);
}

// The list of item (row, kv head) from its `have` pages' keys; a whole CTA calls it.
template <int kPickThreads>
__device__ __forceinline__ void pick_pages(const SelectParams& p, int64_t item, int have, const uint32_t* keys) {
  __shared__ uint32_t bins[kBins];
  __shared__ uint32_t ranked_key[kRanked], ranked_at[kRanked];
  __shared__ uint32_t words[kPickThreads];  // bits of the chosen, a stretch of pages at a time
  __shared__ uint32_t sums[kPickThreads / 32], low[kPickThreads / 32], high[kPickThreads / 32];
  __shared__ uint32_t sh_need, sh_bin, sh_count, sh_ranked;
  static_assert(kPickThreads / 32 <= 32 && kBins % kPickThreads == 0, "one warp adds up the warps' sums");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* out = p.page_idx + item * p.pages;
  if (have <= p.pages) {
    for (int i = tid; i < p.pages; i += kPickThreads) out[i] = i < have ? i : -1;
    return;
  }
  const int n = have - p.first - p.last;
  uint32_t need = static_cast<uint32_t>(p.pages - p.first - p.last);  // of n, which are more
  for (int i = tid; i < p.first; i += kPickThreads) out[i] = i;
  for (int i = tid; i < p.last; i += kPickThreads) out[p.pages - p.last + i] = have - p.last + i;
  if (need == 0u) return;
  keys += p.first;
  uint32_t lo = 0xffffffffu, hi = 0u;
  const bool fits = n <= kKeys * kPickThreads;
  uint32_t kept[kKeys];
  if (fits) {
#pragma unroll
    for (int u = 0; u < kKeys; ++u) kept[u] = tid + u * kPickThreads < n ? keys[tid + u * kPickThreads] : 0u;
  }
  // f(i, key) for this thread's keys
  auto each_key = [&](auto&& f) {
    if (fits) {
#pragma unroll
      for (int u = 0; u < kKeys; ++u) {
        if (u * kPickThreads >= n) break;
        if (tid + u * kPickThreads < n) f(tid + u * kPickThreads, kept[u]);
      }
    } else {
#pragma unroll 8
      for (int i = tid; i < n; i += kPickThreads) f(i, keys[i]);
    }
  };
  each_key([&](int, uint32_t k) { lo = min(lo, k), hi = max(hi, k); });
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) low[warp] = lo, high[warp] = hi;
  for (int i = tid; i < kBins; i += kPickThreads) bins[i] = 0u;
  if (tid == 0) sh_ranked = 0u;
  __syncthreads();
  lo = __reduce_min_sync(0xffffffffu, lane < kPickThreads / 32 ? low[lane] : 0xffffffffu);
  hi = __reduce_max_sync(0xffffffffu, lane < kPickThreads / 32 ? high[lane] : 0u);

  // [lo, hi] holds the need-th largest of the keys that are not above hi
  uint32_t inside = static_cast<uint32_t>(n);  // keys in [lo, hi]
  while (lo < hi && inside > kRanked) {
    const int shift = max(0, 32 - __clz(static_cast<int>(hi - lo)) - 11);
    each_key([&](int, uint32_t k) {
      if (k >= lo && k <= hi) atomicAdd(&bins[(k - lo) >> shift], 1u);
    });
    __syncthreads();
    // counts from the highest bin down, some bins a thread; each is cleared for the next cut
    constexpr int kEach = kBins / kPickThreads;
    uint32_t count[kEach], sum = 0u, total;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int bin = kBins - 1 - (tid * kEach + i);
      count[i] = bins[bin];
      bins[bin] = 0u;
      sum += count[i];
    }
    uint32_t above = block_scan(sum, sums, total);
    if (above < need && above + sum >= need) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        if (above < need && above + count[i] >= need) {
          sh_bin = static_cast<uint32_t>(kBins - 1 - (tid * kEach + i));
          sh_need = need - above;
          sh_count = count[i];
        }
        above += count[i];
      }
    }
    __syncthreads();
    need = sh_need;
    inside = sh_count;
    lo += sh_bin << shift;
    hi = lo + min(hi - lo, (1u << shift) - 1u);
  }
  // Above hi: chosen. In [lo, hi]: the need largest, and of equal keys the lowest pages; where all are one
  // value, simply the first.
  const bool equal = lo == hi;
  if (!equal) {
    each_key([&](int i, uint32_t k) {
      if (k >= lo && k <= hi) {
        const uint32_t to = atomicAdd(&sh_ranked, 1u);  // `inside` in all, in any order
        ranked_key[to] = k;
        ranked_at[to] = static_cast<uint32_t>(i);
      }
    });
    __syncthreads();
    // the key and page of the last one chosen
    for (uint32_t c = tid; c < inside; c += kPickThreads) {
      const uint32_t k = ranked_key[c], at = ranked_at[c];
      uint32_t rank = 0u;
      for (uint32_t j = 0; j < inside; ++j) rank += ranked_key[j] > k || (ranked_key[j] == k && ranked_at[j] < at);
      if (rank == need - 1u) sh_bin = k, sh_count = at;
    }
    __syncthreads();
  }
  const uint32_t last_key = equal ? lo : sh_bin, last_at = equal ? 0u : sh_count;
  uint32_t placed = 0u, equals = 0u;
  for (int base = 0; base < n; base += 32 * kPickThreads) {  // once, for up to 16,384 pages
    const int stretch = min(n - base, 32 * kPickThreads), groups = (stretch + 31) / 32;
    auto mark = [&](int g, uint32_t k) {
      const int i = base + g * 32 + lane;
      const bool same = i < n && k == last_key;
      const bool take = i < n && (k > last_key || (!equal && same && static_cast<uint32_t>(i) <= last_at));
      const unsigned bits = __ballot_sync(0xffffffffu, take), ties = __ballot_sync(0xffffffffu, equal && same);
      if (lane == 0) words[g] = bits, bins[g] = ties;
    };
    if (fits) {  // (then base is 0)
#pragma unroll
      for (int u = 0; u < kKeys; ++u) {
        if (u * kPickThreads >= n) break;
        mark(u * (kPickThreads / 32) + warp, kept[u]);
      }
    } else {
      for (int g = warp; g < groups; g += kPickThreads / 32) {
        const int i = base + g * 32 + lane;
        mark(g, i < n ? keys[i] : 0u);
      }
    }
    __syncthreads();
    uint32_t bits = tid < groups ? words[tid] : 0u, total;
    if (equal) {  // of the ties the first `need`
      uint32_t ties = tid < groups ? bins[tid] : 0u;
      uint32_t room = block_scan(__popc(ties), sums, total) + equals;
      equals += total;
      room = room < need ? need - room : 0u;
      while (__popc(ties) > static_cast<int>(room)) ties &= ~(0x80000000u >> __clz(static_cast<int>(ties)));
      bits |= ties;
    }
    uint32_t to = block_scan(__popc(bits), sums, total) + placed;
    placed += total;
    for (; bits; bits &= bits - 1u) out[p.first + to++] = p.first + base + tid * 32 + __ffs(static_cast<int>(bits)) - 1;
    __syncthreads();
  }
}

template <int kPickThreads>
__global__ void __launch_bounds__(kPickThreads) page_pick_kernel(const SelectParams p) {
  pdl_launch_dependents();
  const int64_t item = blockIdx.x;
  bool past = false;
  const int have = pages_of(p, static_cast<int>(item / p.H_kv), &past);
  pdl_wait_primary();  // so far the lengths alone were read
  if (past && threadIdx.x == 0) set_device_error(p.err_word, TS_DEVERR_PAGE_RANGE);
  pick_pages<kPickThreads>(p, item, have, p.keys + item * p.bt_stride);
}

// Scores and choice of an item by one CTA, keys in shared memory: one launch instead of two.
template <typename T, int D, int G, int kWholeThreads>
__global__ void __launch_bounds__(kWholeThreads, 512 / kWholeThreads)
page_select_kernel(const T* q, const SelectParams p) {
  __shared__ uint32_t keys[kWholePages];
  pdl_launch_dependents();
  constexpr int kOf = kWholeThreads / 32;
  const int64_t item = blockIdx.x;
  const int row = static_cast<int>(item / p.H_kv), h = static_cast<int>(item % p.H_kv), warp = threadIdx.x >> 5;
  bool past = false, waited = false;
  const int have = pages_of(p, row, &past);
  if (have > p.pages && p.pages > p.first + p.last) {
    const int tiles = (have + 15) / 16, t0 = tiles * warp / kOf, t1 = tiles * (warp + 1) / kOf;
    if (t0 < t1) score_pages<T, D, G>(q, p, row, h, 16 * t0, min(have, 16 * t1), keys, waited);
    __syncthreads();
  }
  if (!waited) pdl_wait_primary();
  if (past && threadIdx.x == 0) set_device_error(p.err_word, TS_DEVERR_PAGE_RANGE);
  pick_pages<kWholeThreads>(p, item, have, keys);
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

// One launch, an item a CTA, where the CTAs are resident at once and have few steps: threads of a CTA, or 0. It saves
// the second launch (the call for one sequence of up to 512 pages and 8 kv heads: 11.1 -> 8.6 us; the GPU's own time,
// as in a captured step, is 5.8 us in two launches and 6.5 - 7.8 in one) and lets one item's choice run beside
// another's scores. On the GPU, in two launches and in one:
//   a CTA of 512 threads an SM: 80 items of 1000 pages 13.2, 10.6 us; of 2000 17.1, 15.6; of 4000 25.8, 28.7;
//     152 of 2000 22.6, 17.7; but 8 of 1000 6.7, 10.4: longer tables need the items that fill half of the SMs;
//   two of 256: 304 items of 500 pages 14.7, 11.5 us; of 1000 21.8, 17.9; 192 of 1000 17.0, 16.7; of 2000 26.3, 30.7.
int whole_threads(int64_t items, int64_t slots) {
  const int sms = device_sm_count();
  if (items <= sms) return slots <= 512 || (slots <= kWholePages && 2 * items >= sms) ? 512 : 0;
  return items <= 2 * sms && slots <= 1024 ? 256 : 0;
}

template <typename T, int D, int kWholeThreads>
cudaError_t launch_whole(int g, unsigned grid, cudaStream_t stream, const void* q, const SelectParams& p) {
  const T* src = static_cast<const T*>(q);
  switch (g) {
    case 1: return launch_pdl(page_select_kernel<T, D, 1, kWholeThreads>, grid, kWholeThreads, stream, src, p);
    case 2: return launch_pdl(page_select_kernel<T, D, 2, kWholeThreads>, grid, kWholeThreads, stream, src, p);
    case 4: return launch_pdl(page_select_kernel<T, D, 4, kWholeThreads>, grid, kWholeThreads, stream, src, p);
    default: return launch_pdl(page_select_kernel<T, D, 8, kWholeThreads>, grid, kWholeThreads, stream, src, p);
  }
}

template <int kWholeThreads>
cudaError_t launch_whole(ts_dtype dtype, int D, int g, unsigned grid, cudaStream_t stream, const void* q,
                         const SelectParams& p) {
  if (dtype == TS_BF16)
    return D == 64 ? launch_whole<__nv_bfloat16, 64, kWholeThreads>(g, grid, stream, q, p)
                   : launch_whole<__nv_bfloat16, 128, kWholeThreads>(g, grid, stream, q, p);
  return D == 64 ? launch_whole<float, 64, kWholeThreads>(g, grid, stream, q, p)
                 : launch_whole<float, 128, kWholeThreads>(g, grid, stream, q, p);
}

template <typename T, int D>
cudaError_t launch_score(int g, unsigned grid, cudaStream_t stream, const void* q, const SelectParams& p) {
  const T* src = static_cast<const T*>(q);
  switch (g) {
    case 1: return launch_pdl(page_score_kernel<T, D, 1>, grid, kThreads, stream, src, p);
    case 2: return launch_pdl(page_score_kernel<T, D, 2>, grid, kThreads, stream, src, p);
    case 4: return launch_pdl(page_score_kernel<T, D, 4>, grid, kThreads, stream, src, p);
    default: return launch_pdl(page_score_kernel<T, D, 8>, grid, kThreads, stream, src, p);
  }
}

size_t select_bytes(int64_t rows, int H_kv, int bt_stride) {
  return align_up(kWorkspaceAlign + static_cast<size_t>(rows) * H_kv * bt_stride * sizeof(uint32_t), kWorkspaceAlign);
}

}  // namespace
}  // namespace ts

extern "C" size_t ts_select_pages_workspace_size(int32_t B, int32_t q_len, int32_t H_kv, int32_t bt_stride) {
  if (B < 0 || q_len <= 0 || H_kv <= 0 || H_kv > 8 || bt_stride <= 0 || static_cast<int64_t>(B) * q_len > (1 << 24))
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
  if (rows > (1 << 24)) return fail(TS_ERR_UNSUPPORTED, "%s: more than 2^24 query rows", who);
  if (B == 0) return TS_OK;
  if (!q || !bounds || !bound_scale || !block_table || !seq_lens || !page_idx)
    return fail(TS_ERR_INVALID_ARG, "%s: null pointer", who);
  for (const void* x : {q, static_cast<const void*>(bounds)})
    if (reinterpret_cast<uintptr_t>(x) % 16 != 0)
      return fail(TS_ERR_INVALID_ARG, "%s: queries and bounds must be 16-byte aligned", who);
  const size_t bytes = select_bytes(rows, H_kv, bt_stride);
  if (!workspace || workspace_bytes < bytes || reinterpret_cast<uintptr_t>(workspace) % kWorkspaceAlign != 0)
    return fail(TS_ERR_WORKSPACE, "%s: workspace %zu B < %zu B needed or misaligned", who, workspace_bytes, bytes);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // Warps: those the device holds, or one for each tile of the longest sequences there can be.
  const int64_t tiles = rows * H_kv * ((static_cast<int64_t>(bt_stride) + 15) / 16);
  const int64_t full = static_cast<int64_t>(device_sm_count()) * kResident * kWarps;
  const unsigned ctas = static_cast<unsigned>(((tiles < full ? tiles : full) + kWarps - 1) / kWarps);
  const SelectParams p{bounds,    bound_scale, block_table, seq_lens,
                       reinterpret_cast<uint32_t*>(static_cast<unsigned char*>(workspace) + kWorkspaceAlign),
                       page_idx,  static_cast<uint32_t*>(workspace), bt_stride, static_cast<int32_t>(rows), q_len, H_kv,
                       page_size, num_pages, pages, first, last, static_cast<int32_t>(ctas) * kWarps};
  if (const int threads = whole_threads(rows * H_kv, bt_stride)) {
    LaunchTrace trace("page_select_kernel", s);
    const unsigned items = static_cast<unsigned>(rows * H_kv);
    const cudaError_t e = threads == 512 ? launch_whole<512>(dtype, D, g, items, s, q, p)
                                         : launch_whole<256>(dtype, D, g, items, s, q, p);
    return cuda_check(e, "ts_select_pages: launch");
  }
  if (bt_stride > pages && pages > first + last) {  // else nothing is ranked
    LaunchTrace trace("page_score_kernel", s);
    const cudaError_t e = dtype == TS_BF16 ? (D == 64 ? launch_score<__nv_bfloat16, 64>(g, ctas, s, q, p)
                                                      : launch_score<__nv_bfloat16, 128>(g, ctas, s, q, p))
                                           : (D == 64 ? launch_score<float, 64>(g, ctas, s, q, p)
                                                      : launch_score<float, 128>(g, ctas, s, q, p));
    const ts_status st = cuda_check(e, "ts_select_pages: launch");
    if (st != TS_OK) return st;
  }
  // Threads of a choosing CTA: as many as hold all of its keys in registers, 16 each; more keys are read again for
  // every step. Small CTAs leave room for others (64 sequences of 2,048 pages: 256 threads, all 512 CTAs at once). The
  // table's width decides, lengths are the device's: 64 sequences of 63 .. 250 pages 17.6 us, 28.0 in a table of 8,192.
  LaunchTrace trace("page_pick_kernel", s);
  const unsigned items = static_cast<unsigned>(rows * H_kv);
  return cuda_check(bt_stride <= 256 * kKeys ? launch_pdl(page_pick_kernel<256>, items, 256, s, p)
                                             : launch_pdl(page_pick_kernel<1024>, items, 1024, s, p),
                    "ts_select_pages: launch");
}
