// Work cut evenly over the warps of a grid: items (a query row and kv head) of a
// number of entries each that the device finds from the sequences' lengths, in
// order, cut into equal contiguous ranges, a warp each.
//
// P has rows, H_kv, seq_lens and q_len, and row_entries(p, row) gives the entries of
// each of a row's H_kv items.
#pragma once

#include "ts_common.cuh"

namespace ts {
namespace {

// Position of a query row: token j of q_len of a sequence.
template <typename P>
__device__ __forceinline__ int row_position(const P& p, int row) {
  const int b = row / p.q_len;
  return max(p.seq_lens[b], 0) - p.q_len + (row - b * p.q_len);
}

// Rows of a chunk: a CTA's threads take a chunk each.
template <int kThreads, typename P>
__device__ __forceinline__ int chunk_rows(const P& p) {
  return (p.rows + kThreads - 1) / kThreads;
}

// Entries in front of each chunk of rows, for one kv head; the whole CTA calls it.
template <int kThreads, typename P>
__device__ __forceinline__ void make_plan(const P& p, int64_t (&before)[kThreads + 1]) {
  __shared__ int64_t warp_sum[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, each = chunk_rows<kThreads>(p);
  int64_t sum = 0;
  const int64_t r1 = min(static_cast<int64_t>(p.rows), static_cast<int64_t>(tid + 1) * each);
  for (int64_t r = static_cast<int64_t>(tid) * each; r < r1; ++r) sum += row_entries(p, static_cast<int>(r));
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  for (int w = 0; w < warp; ++w) incl += warp_sum[w];
  before[tid + 1] = incl;
  if (tid == 0) before[0] = 0;
  __syncthreads();
}

// Entries of each of `warps` ranges.
__device__ __forceinline__ int64_t even_range(int64_t total, int32_t warps) {
  if (total < (1ll << 31)) {  // (a division of 64 bits takes several times as long)
    const uint32_t n = static_cast<uint32_t>(warps);
    return (static_cast<uint32_t>(total) + n - 1u) / n;
  }
  return (total + warps - 1) / warps;
}

// Walks the items of entries [at, end): row, head and the part [i0, i1) of the item's entries.
struct Walk {
  int64_t at, end, item0;  // item0: first entry of the item
  int32_t row, h, count, i0, i1;

  // Finds the item of entry `from`; a whole warp calls it.
  template <int kThreads, typename P>
  __device__ __forceinline__ bool start(const P& p, const int64_t (&before)[kThreads + 1], int64_t from, int64_t to,
                                        int lane) {
    at = from;
    end = min(to, before[kThreads] * p.H_kv);
    if (at >= end) return false;
    int chunk = 0;  // the last one with before * H_kv <= at
#pragma unroll
    for (int c0 = 0; c0 < kThreads; c0 += 32)
      chunk += __popc(__ballot_sync(0xffffffffu, before[c0 + lane + 1] * p.H_kv <= at));
    int64_t sum = before[chunk] * p.H_kv;
    for (int64_t r0 = static_cast<int64_t>(chunk) * chunk_rows<kThreads>(p);; r0 += 32) {
      const int64_t r = r0 + lane;
      const int n = r < p.rows ? row_entries(p, static_cast<int>(r)) : 0;
      int64_t incl = static_cast<int64_t>(n) * p.H_kv;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, sum + incl > at);
      if (hit) {
        const int found = __ffs(static_cast<int>(hit)) - 1;
        row = static_cast<int>(r0) + found;
        count = __shfl_sync(0xffffffffu, n, found);
        sum += __shfl_sync(0xffffffffu, incl, found) - static_cast<int64_t>(count) * p.H_kv;
        break;
      }
      sum += __shfl_sync(0xffffffffu, incl, 31);
      if (r0 + 32 >= p.rows) return false;  // (lengths changed under the call)
    }
    item0 = sum;
    for (h = 0; at - item0 >= count; ++h) item0 += count;
    settle();
    return true;
  }
  __device__ __forceinline__ void settle() {
    i0 = static_cast<int>(at - item0);
    i1 = static_cast<int>(min(static_cast<int64_t>(count), end - item0));
  }
  template <typename P>
  __device__ __forceinline__ bool next(const P& p) {
    at = item0 + i1;
    if (at >= end) return false;
    item0 += count;
    if (++h == p.H_kv) {
      h = 0;
      do {
        if (++row >= p.rows) return false;
        count = row_entries(p, row);
      } while (count == 0);
    }
    settle();
    return true;
  }
  __device__ __forceinline__ bool whole() const { return i0 == 0 && i1 == count; }
};

}  // namespace
}  // namespace ts
