// Instantiations of the paged split-KV decode kernel for a sliding window with
// a few first tokens that stay visible (ts_paged_decode_sink_attn): a sequence
// of L tokens attends tokens t < sinks and t >= L - window. Its own pages are
// those of the first tokens, then the window's, and the batch's list of own
// pages is cut over the SMs as for the other variants, so the kernel moves the
// visible rows only. Own translation unit: the other variants' code does not
// change, and the parallel build compiles it beside them.
//
// What bounds it: HBM, as the plain window. The rows are those of the window
// plus one or a few pages per sequence: 64 sequences, window 4096 and 64 first
// tokens, 32 / 8 heads of 128, bf16: 164.5 us, 1,092 MB at 6.6 TB/s (98 % of the
// device's copy rate). One float32 sequence, window 250: 8.1 to 8.9 us, the
// latency of the launch, the prologue and one round of loads.
#include "ts_paged_decode_kernel.cuh"

namespace ts {
namespace {

template <typename T, int D>
PagedKernelFn pick_rows(int G) {
  switch (G) {
    case 1: return paged_decode_kernel<T, D, 1, false, false, false, true, true>;
    case 2: return paged_decode_kernel<T, D, 2, false, false, false, true, true>;
    case 4: return paged_decode_kernel<T, D, 4, false, false, false, true, true>;
    case 8: return paged_decode_kernel<T, D, 8, false, false, false, true, true>;
    default: return nullptr;
  }
}

}  // namespace

PagedKernelFn pick_paged_sink_kernel(ts_dtype dt, int D, int G) {
  if (dt == TS_BF16) {
    if (D == 64) return pick_rows<__nv_bfloat16, 64>(G);
    if (D == 128) return pick_rows<__nv_bfloat16, 128>(G);
  } else if (dt == TS_F32) {
    if (D == 64) return pick_rows<float, 64>(G);
    if (D == 128) return pick_rows<float, 128>(G);
  }
  return nullptr;
}

}  // namespace ts
