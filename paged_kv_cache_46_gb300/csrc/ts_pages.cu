// ts_kv_fork and ts_kv_compact: sequences that share their pages with a copy of
// themselves, and pages moved to the front of the pool.
//
// Both move whole pages of any number of buffers (K, V, scales, bounds, of every
// layer) that one block table serves, and are bound by HBM: each page read once
// and written once. A page of a buffer is cut into pieces of kPiece bytes; a CTA
// takes a piece, found by a search over the buffers' first pieces, which are
// kernel parameters: nothing is kept on the device between calls. 48 buffers (K, V,
// bounds and scales of 12 layers, pages of 32 KB): 64 forks 14.9 us, 97 MB at 6.6 TB/s;
// 32 sequences' pages moved to the front 157 us, 966 MB at 6.1 TB/s. Pieces of 8 KB:
// 172 us; of 32 KB: the same.
//
// Compaction: a bit for every page that some row names; a prefix sum over the words
// of bits gives each page its rank, the number of pages U, and the lists of what
// moves where. Nothing is sorted, and equal calls give equal pages.
//
// They write the block table, which the attention kernels of a stream read
// before they wait for the kernel in front of them: so neither lets its
// successor start early.
#include "ts_common.cuh"

namespace ts {
namespace {

constexpr int kMaxBuffers = 128;  // of a launch
constexpr int kThreads = 256;
constexpr int kPiece = 16384;
constexpr int kScanThreads = 1024;
// Tables and pools that one CTA plans alone, in one launch instead of three (a pool of 70 pages: the call 9.8 us,
// with three 15; 32 sequences, 80 MB to move: 13.9 us, in a table of 32 x 8,192 entries and three launches 17.4).
constexpr int kPlanEntries = 32768, kPlanWords = 8192;

struct Buffers {
  uint8_t* data[kMaxBuffers];
  int64_t page_bytes[kMaxBuffers];
  int64_t first_piece[kMaxBuffers + 1];
  int32_t n;
};

// Copies piece `piece` of page `src` to page `dst`; the whole CTA.
__device__ __forceinline__ void copy_piece(const Buffers& b, int64_t piece, int64_t src, int64_t dst) {
  int lo = 0, hi = b.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.first_piece[mid] <= piece)
      lo = mid;
    else
      hi = mid;
  }
  const int64_t page = b.page_bytes[lo], at = (piece - b.first_piece[lo]) * kPiece;
  const int bytes = static_cast<int>(min(static_cast<int64_t>(kPiece), page - at));
  const uint8_t* from = b.data[lo] + src * page + at;
  uint8_t* to = b.data[lo] + dst * page + at;
  if (((page | reinterpret_cast<int64_t>(b.data[lo])) & 15) == 0) {
    const uint4* f = reinterpret_cast<const uint4*>(from);
    uint4* t = reinterpret_cast<uint4*>(to);
    const int vecs = bytes / 16;
    constexpr int kEach = kPiece / 16 / kThreads;
    uint4 w[kEach];
#pragma unroll
    for (int u = 0; u < kEach; ++u)
      if (static_cast<int>(threadIdx.x) + u * kThreads < vecs) w[u] = f[threadIdx.x + u * kThreads];
#pragma unroll
    for (int u = 0; u < kEach; ++u)
      if (static_cast<int>(threadIdx.x) + u * kThreads < vecs) t[threadIdx.x + u * kThreads] = w[u];
  } else if (((page | reinterpret_cast<int64_t>(b.data[lo])) & 3) == 0) {
    for (int i = threadIdx.x; i < bytes / 4; i += kThreads)
      reinterpret_cast<uint32_t*>(to)[i] = reinterpret_cast<const uint32_t*>(from)[i];
  } else {
    for (int i = threadIdx.x; i < bytes; i += kThreads) to[i] = from[i];
  }
}

struct ForkParams {
  int32_t* block_table;
  int32_t* seq_lens;
  const int32_t* parents;
  const int32_t* children;
  const int32_t* fresh;
  int32_t bt_stride, B, page_size, num_pages, tables;  // tables: this launch writes rows and lengths
};

// grid: (pieces of a page, one at least) x forks
__global__ void __launch_bounds__(kThreads) kv_fork_kernel(const __grid_constant__ Buffers buffers,
                                                           const ForkParams p, int64_t pieces) {
  pdl_wait_primary();
  const int64_t i = blockIdx.x / pieces, piece = blockIdx.x % pieces;
  const int parent = p.parents[i], child = p.children[i];
  if (parent < 0 || parent >= p.B || child < 0 || child >= p.B || parent == child) return;
  const int L = p.seq_lens[parent];
  if (L < 0) return;
  const int64_t slots = (static_cast<int64_t>(L) + p.page_size - 1) / p.page_size;
  if (slots > p.bt_stride) return;
  const int32_t* from = p.block_table + static_cast<int64_t>(parent) * p.bt_stride;
  int32_t* to = p.block_table + static_cast<int64_t>(child) * p.bt_stride;
  const bool cut = L % p.page_size != 0;
  int src = -1, dst = -1;
  if (cut) {
    src = from[slots - 1];
    dst = p.fresh[i];
    if (src < 0 || src >= p.num_pages || dst < 0 || dst >= p.num_pages) return;
    if (piece < buffers.first_piece[buffers.n] && src != dst) copy_piece(buffers, piece, src, dst);
  }
  if (piece == 0 && p.tables) {
    for (int s = threadIdx.x; s < slots; s += kThreads) to[s] = cut && s == slots - 1 ? dst : from[s];
    if (threadIdx.x == 0) p.seq_lens[child] = L;
    __threadfence();  // seen by a kernel that reads tables and lengths before it waits for this one
  }
}

struct CompactParams {
  const int32_t* block_table;
  int32_t* table_out;
  const int32_t* seq_lens;
  int32_t* page_map;
  int32_t* used;
  uint32_t* bits;     // [words] a bit per page that some row holds
  int32_t* before;    // [words] held pages in front of the word
  int32_t* counts;    // [0] held pages U, [1] those in front of page U, [2] pages that move
  int32_t* sources;   // held pages from U on, ascending
  int32_t* targets;   // free pages in front of U, ascending
  int32_t bt_stride, B, page_size, num_pages, words, tables;
};

__device__ __forceinline__ bool holds(const CompactParams& p, int64_t entry) {
  int64_t b, slot;
  if (entry < (1ll << 31)) {  // (a division of 64 bits takes several times as long)
    b = static_cast<uint32_t>(entry) / static_cast<uint32_t>(p.bt_stride);
    slot = entry - b * p.bt_stride;
  } else {
    b = entry / p.bt_stride;
    slot = entry % p.bt_stride;
  }
  return slot * p.page_size < p.seq_lens[b];
}

__global__ void __launch_bounds__(kThreads) page_clear_kernel(const CompactParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < p.words;
       i += static_cast<int64_t>(gridDim.x) * kThreads)
    p.bits[i] = 0u;
}

__global__ void __launch_bounds__(kThreads) page_mark_kernel(const CompactParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int64_t entries = static_cast<int64_t>(p.B) * p.bt_stride;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < entries;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    if (!holds(p, i)) continue;
    const int page = p.block_table[i];
    if (page >= 0 && page < p.num_pages) atomicOr(p.bits + (page >> 5), 1u << (page & 31));
  }
}

// Prefix sums over the words of `bits` by a CTA of kScanThreads, then the lists of moves.
__device__ __forceinline__ void scan_pages(const CompactParams& p, const uint32_t* bits) {
  __shared__ int32_t warp_sum[32];
  __shared__ int32_t front;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = (p.words + kScanThreads - 1) / kScanThreads;
  const int64_t w0 = min(static_cast<int64_t>(p.words), static_cast<int64_t>(tid) * each);
  const int64_t w1 = min(static_cast<int64_t>(p.words), w0 + each);
  int sum = 0;
  for (int64_t w = w0; w < w1; ++w) sum += __popc(bits[w]);
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  const int of_lane = warp_sum[lane];
  const int U = __reduce_add_sync(0xffffffffu, of_lane);
  const int at = incl - sum + __reduce_add_sync(0xffffffffu, lane < warp ? of_lane : 0);
  int rank = at;
  if (tid == 0) front = U;  // of pages 0 .. P - 1 with U == P
  __syncthreads();
  for (int64_t w = w0; w < w1; ++w) {
    const uint32_t x = bits[w];
    p.before[w] = rank;
    if (w == U >> 5) front = rank + __popc(x & ((1u << (U & 31)) - 1u));
    rank += __popc(x);
  }
  __syncthreads();
  const int kept = front;  // held pages in front of page U: they stay
  rank = at;
  for (int64_t w = w0; w < w1; ++w) {
    const uint32_t x = bits[w];
    const int64_t page0 = w * 32;
    if (page0 + 32 > U) {  // held pages from U on
      uint32_t far = page0 >= U ? x : x & ~((1u << (U - page0)) - 1u);
      int k = rank + __popc(x & ~far);
      for (; far; far &= far - 1) p.sources[k++ - kept] = static_cast<int32_t>(page0) + __ffs(far) - 1;
    }
    if (page0 < U) {  // free pages in front of U
      uint32_t free = ~x;
      if (U - page0 < 32) free &= (1u << (U - page0)) - 1u;
      int k = static_cast<int>(page0) - rank;
      for (; free; free &= free - 1) p.targets[k++] = static_cast<int32_t>(page0) + __ffs(free) - 1;
    }
    rank += __popc(x);
  }
  if (tid == 0) {
    p.counts[0] = U;
    p.counts[1] = kept;
    p.counts[2] = U - kept;
  }
}

__global__ void __launch_bounds__(kScanThreads) page_scan_kernel(const CompactParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  scan_pages(p, p.bits);
}

// All three steps of a small plan by one CTA: bits in shared memory, kept in the workspace for the moves.
__global__ void __launch_bounds__(kScanThreads) page_plan_kernel(const CompactParams p) {
  __shared__ uint32_t bits[kPlanWords];
  pdl_launch_dependents();
  for (int i = threadIdx.x; i < p.words; i += kScanThreads) bits[i] = 0u;
  __syncthreads();
  pdl_wait_primary();
  const int entries = p.B * p.bt_stride;  // kPlanEntries at most
#pragma unroll 4
  for (int i = threadIdx.x; i < entries; i += kScanThreads) {
    const int page = p.block_table[i];
    if (holds(p, i) && page >= 0 && page < p.num_pages) atomicOr(bits + (page >> 5), 1u << (page & 31));
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.words; i += kScanThreads) p.bits[i] = bits[i];
  scan_pages(p, bits);
}

// Where a page moves: itself below U, a target from U on, -1 if no row holds it.
__device__ __forceinline__ int moved_to(const CompactParams& p, int page, int U, int kept) {
  const uint32_t x = p.bits[page >> 5];
  if (!(x >> (page & 31) & 1u)) return -1;
  if (page < U) return page;
  return p.targets[p.before[page >> 5] + __popc(x & ((1u << (page & 31)) - 1u)) - kept];
}

__global__ void __launch_bounds__(kThreads) page_move_kernel(const __grid_constant__ Buffers buffers,
                                                             const CompactParams p, int64_t pieces) {
  pdl_wait_primary();
  const int U = p.counts[0], kept = p.counts[1];
  if (p.tables) {
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
    for (int64_t i = i0; i < p.num_pages; i += step) p.page_map[i] = moved_to(p, static_cast<int>(i), U, kept);
    const int64_t entries = static_cast<int64_t>(p.B) * p.bt_stride;
    for (int64_t i = i0; i < entries; i += step) {
      const int page = p.block_table[i];
      p.table_out[i] = holds(p, i) && page >= 0 && page < p.num_pages ? moved_to(p, page, U, kept) : page;
    }
    if (i0 == 0) p.used[0] = U;
    __threadfence();  // seen by a kernel that reads the table before it waits for this one
  }
  const int64_t todo = static_cast<int64_t>(p.counts[2]) * pieces;
  for (int64_t u = blockIdx.x; u < todo; u += gridDim.x)
    copy_piece(buffers, u % pieces, p.sources[u / pieces], p.targets[u / pieces]);
}

// Up to kMaxBuffers of the caller's buffers from `at` on; pieces of one page.
int64_t take_buffers(Buffers& b, void* const* data, const int64_t* page_bytes, int32_t at, int32_t n) {
  b.n = n - at < kMaxBuffers ? n - at : kMaxBuffers;
  int64_t pieces = 0;
  for (int i = 0; i < b.n; ++i) {
    b.data[i] = static_cast<uint8_t*>(data[at + i]);
    b.page_bytes[i] = page_bytes[at + i];
    b.first_piece[i] = pieces;
    pieces += (page_bytes[at + i] + kPiece - 1) / kPiece;
  }
  b.first_piece[b.n] = pieces;
  return pieces;
}

ts_status check_buffers(const char* who, void* const* data, const int64_t* page_bytes, int32_t n) {
  if (n < 0) return fail(TS_ERR_INVALID_ARG, "%s: n_buffers=%d", who, n);
  if (n > 0 && (!data || !page_bytes)) return fail(TS_ERR_INVALID_ARG, "%s: null pointer", who);
  for (int i = 0; i < n; ++i)
    if (!data[i] || page_bytes[i] <= 0 || page_bytes[i] > (1 << 30))
      return fail(TS_ERR_INVALID_ARG, "%s: buffer %d is null or its page of %lld B outside [1, 2^30]", who, i,
                  static_cast<long long>(page_bytes[i]));
  return TS_OK;
}

template <typename K, typename... A>
cudaError_t launch_pdl(K kern, unsigned grid, int threads, cudaStream_t stream, const A&... args) {
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

struct CompactWs {
  size_t bits, before, sources, targets, total;
  explicit CompactWs(int32_t num_pages) {
    const size_t words = (static_cast<size_t>(num_pages) + 31) / 32, half = static_cast<size_t>(num_pages) / 2 + 1;
    bits = 2 * kWorkspaceAlign;  // behind the error word and the counts
    before = align_up(bits + words * 4, kWorkspaceAlign);
    sources = align_up(before + words * 4, kWorkspaceAlign);
    targets = align_up(sources + half * 4, kWorkspaceAlign);
    total = align_up(targets + half * 4, kWorkspaceAlign);
  }
};

unsigned grid_for(int64_t threads, unsigned most) {
  const int64_t n = (threads + kThreads - 1) / kThreads;
  return n < 1 ? 1u : n > most ? most : static_cast<unsigned>(n);
}

}  // namespace
}  // namespace ts

extern "C" ts_status ts_kv_fork(void* const* buffers, const int64_t* page_bytes, int32_t n_buffers,
                                int32_t* block_table, int32_t bt_stride, int32_t* seq_lens, int32_t B,
                                const int32_t* parents, const int32_t* children, const int32_t* fresh, int32_t n,
                                int32_t page_size, int32_t num_pages, void* stream) {
  using namespace ts;
  const char* who = "ts_kv_fork";
  if (n < 0 || B < 0 || bt_stride <= 0 || page_size <= 0 || num_pages <= 0)
    return fail(TS_ERR_INVALID_ARG, "%s: bad sizes (n=%d B=%d bt=%d ps=%d P=%d)", who, n, B, bt_stride, page_size,
                num_pages);
  const ts_status st = check_buffers(who, buffers, page_bytes, n_buffers);
  if (st != TS_OK) return st;
  if (n == 0 || B == 0) return TS_OK;
  if (!block_table || !seq_lens || !parents || !children || !fresh)
    return fail(TS_ERR_INVALID_ARG, "%s: null pointer", who);
  for (int32_t at = 0; at < n_buffers; at += kMaxBuffers) {
    Buffers b;
    if (take_buffers(b, buffers, page_bytes, at, n_buffers) * n > 0x7fffffff)
      return fail(TS_ERR_UNSUPPORTED, "%s: more than 2^31 pieces to copy", who);
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ForkParams p{block_table, seq_lens, parents, children, fresh, bt_stride, B, page_size, num_pages, 1};
  for (int32_t at = 0; at == 0 || at < n_buffers; at += kMaxBuffers, p.tables = 0) {
    Buffers b;
    int64_t pieces = take_buffers(b, buffers, page_bytes, at, n_buffers);
    if (pieces == 0) pieces = 1;
    LaunchTrace trace("kv_fork_kernel", s);
    const ts_status done = cuda_check(
        launch_pdl(kv_fork_kernel, static_cast<unsigned>(pieces * n), kThreads, s, b, p, pieces), "ts_kv_fork: launch");
    if (done != TS_OK) return done;
  }
  return TS_OK;
}

extern "C" size_t ts_kv_compact_workspace_size(int32_t num_pages) {
  return num_pages <= 0 ? 0 : ts::CompactWs(num_pages).total;
}

extern "C" ts_status ts_kv_compact(void* const* buffers, const int64_t* page_bytes, int32_t n_buffers,
                                   const int32_t* block_table, int32_t* table_out, int32_t bt_stride,
                                   const int32_t* seq_lens, int32_t B, int32_t page_size, int32_t num_pages,
                                   int32_t* page_map, int32_t* used, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  using namespace ts;
  const char* who = "ts_kv_compact";
  if (B < 0 || bt_stride <= 0 || page_size <= 0 || num_pages <= 0)
    return fail(TS_ERR_INVALID_ARG, "%s: bad sizes (B=%d bt=%d ps=%d P=%d)", who, B, bt_stride, page_size, num_pages);
  const ts_status st = check_buffers(who, buffers, page_bytes, n_buffers);
  if (st != TS_OK) return st;
  if (!page_map || !used || (B > 0 && (!block_table || !table_out || !seq_lens)))
    return fail(TS_ERR_INVALID_ARG, "%s: null pointer", who);
  const CompactWs ws(num_pages);
  if (!workspace || workspace_bytes < ws.total || reinterpret_cast<uintptr_t>(workspace) % kWorkspaceAlign != 0)
    return fail(TS_ERR_WORKSPACE, "%s: workspace %zu B < %zu B needed or misaligned", who, workspace_bytes, ws.total);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned char* w = static_cast<unsigned char*>(workspace);
  CompactParams p{block_table, table_out, seq_lens, page_map, used, reinterpret_cast<uint32_t*>(w + ws.bits),
                  reinterpret_cast<int32_t*>(w + ws.before), reinterpret_cast<int32_t*>(w + kWorkspaceAlign),
                  reinterpret_cast<int32_t*>(w + ws.sources), reinterpret_cast<int32_t*>(w + ws.targets),
                  bt_stride, B, page_size, num_pages,
                  static_cast<int32_t>((static_cast<int64_t>(num_pages) + 31) / 32), 1};
  const unsigned sms = static_cast<unsigned>(device_sm_count());
  const int64_t entries = static_cast<int64_t>(B) * bt_stride;
  auto step = [&](const char* name, auto kern, unsigned grid, int threads) {
    LaunchTrace trace(name, s);
    return cuda_check(launch_pdl(kern, grid, threads, s, p), "ts_kv_compact: launch");
  };
  ts_status done = TS_OK;
  if (entries <= kPlanEntries && p.words <= kPlanWords) {
    done = step("page_plan_kernel", page_plan_kernel, 1u, kScanThreads);
  } else {
    done = step("page_clear_kernel", page_clear_kernel, grid_for(p.words, 8 * sms), kThreads);
    if (done == TS_OK && B > 0) done = step("page_mark_kernel", page_mark_kernel, grid_for(entries, 8 * sms), kThreads);
    if (done == TS_OK) done = step("page_scan_kernel", page_scan_kernel, 1u, kScanThreads);
  }
  if (done != TS_OK) return done;
  for (int32_t at = 0; at == 0 || at < n_buffers; at += kMaxBuffers, p.tables = 0) {
    Buffers b;
    const int64_t pieces = take_buffers(b, buffers, page_bytes, at, n_buffers);
    LaunchTrace trace("page_move_kernel", s);
    done = cuda_check(launch_pdl(page_move_kernel, 8 * sms, kThreads, s, b, p, pieces), "ts_kv_compact: launch");
    if (done != TS_OK) return done;
  }
  return TS_OK;
}
