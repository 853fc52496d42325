// Device helpers for ragged batches: rows of all sequences one after another,
// sequence b's in [indptr[b], indptr[b + 1]).
#pragma once

#include "ts_common.cuh"

namespace ts {

// The last sequence that begins at `row` or in front of it, or -1. A whole warp
// calls it with one row; each step compares 32 entries, so a batch of up to 1024
// sequences takes two dependent loads. Entries out of order cannot lead out of
// [0, B).
__device__ __forceinline__ int ragged_floor(const int32_t* __restrict__ indptr, int B, int row, int lane) {
  int lo = 0, hi = B;  // the last b in [lo, hi) with indptr[b] <= row
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int probe = lo + lane * step;
    const unsigned below = __ballot_sync(0xffffffffu, probe < hi && indptr[probe] <= row);
    if (below == 0u) return -1;
    lo += (31 - __clz(static_cast<int>(below))) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// The sequence whose rows hold `row`, or -1; as ragged_floor, and checked against
// the sequence's own bounds.
__device__ __forceinline__ int ragged_sequence(const int32_t* __restrict__ indptr, int B, int row, int lane) {
  const int b = ragged_floor(indptr, B, row, lane);
  return b >= 0 && indptr[b] <= row && row < indptr[b + 1] ? b : -1;
}

// A page size and its logarithm (-1 where it is no power of two: the appends and
// the read-back take pages of any size, the attention calls do not): a division
// per row is a fifth of a short row's work.
struct PageSize {
  int32_t rows, shift;
  explicit PageSize(int32_t r) : rows(r), shift(-1) {
    for (int32_t i = 0; i < 31; ++i)
      if (r == (1 << i)) shift = i;
  }
};

// Pool row (page * rows + row in it) of the token at `pos` of sequence b; -1
// where its block-table slot or page id is out of range.
__device__ __forceinline__ int64_t pool_row(const int32_t* __restrict__ block_table, int bt_stride, int b, int pos,
                                            PageSize page_size, int num_pages) {
  if (pos < 0) return -1;
  const int slot = page_size.shift >= 0 ? pos >> page_size.shift : pos / page_size.rows;
  if (slot >= bt_stride) return -1;
  const int page = block_table[static_cast<int64_t>(b) * bt_stride + slot];
  if (page < 0 || page >= num_pages) return -1;
  return static_cast<int64_t>(page) * page_size.rows + (pos - slot * page_size.rows);
}

}  // namespace ts
