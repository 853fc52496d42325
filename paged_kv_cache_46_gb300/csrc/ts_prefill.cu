// ts_paged_prefill_attn, bf16: attention of a ragged batch of prompt chunks
// over the paged cache that already holds their K/V rows.
//
// Token j of sequence b's n new ones sits at position p = L - n + j and sees
// keys t <= p; with a window W only t > p - W, and the first S tokens besides.
//
// Rows. One kv head's g query heads of a token are neighbouring rows of a tile
// (row r of a tile: token r / g, head h * g + r % g), so that a K/V tile read
// once serves all of them (TokenSpeed deep dive, section 7.2: tokens and heads
// fold into the rows of a tile). A work item is two 128-row tiles (2 * (128 /
// g) tokens) of one kv head of one sequence, and 128 keys at a time.
//
// Split. Items have 1 to thousands of key tiles, so the key tiles of all items
// (in order of sequence, kv head, token block; some extra units per item for its
// queries and epilogue) are cut into equal contiguous ranges, one per SM. Each
// CTA computes the cut in its prologue from the lengths. An item cut between
// CTAs leaves float32 states that prefill_merge_kernel joins by LSE
// (TokenSpeed deep dive, section 7.1): at most two per CTA, whatever the sizes.
//
// Inside a CTA (384 threads):
//   warps 0-3, 4-7  softmax of tile 0 and tile 1, one query row per thread
//   warps 8, 10     TMA of K and of V: one box per page and 64-column atom
//   warp 9          issues the products
//   warp 11         walks the range, hands its pieces to the others, loads queries
// S = Q K^T goes to TMEM (128 columns a tile); the softmax takes its row into
// registers and writes P, as bf16, over the front half of the same columns,
// where it is the A operand of O += P V; the next S into those columns waits
// until that product has completed. The two tiles take turns: while one tile's
// softmax runs, the tensor pipe works on the other.
//
// What bounds it, by clock stamps inside a 32k-token run at head dim 128 (a step
// of both tiles takes 3,000 clocks, 3,575 with the stamps; the products alone
// would take 2,048): each tile's own chain of S (512, and 350 until the softmax
// sees it), loads from TMEM (470), weights (980; 710 for a warp that has the SM
// to itself, 510 of them the exponentials), issue and run of P V (512 + 540),
// since TMEM has room for one score tile per query tile there. 4096 tokens over
// 32,768, 32 / 8 heads of 128: 2.66 million clocks, which is 1.38 ms (1.49
// PFLOP/s) for the first tens of calls and 1.49 ms (1.38) where calls go on for
// seconds and the power limit takes the clock from 1.93 to 1.79 GHz; 16 ragged
// prompts of 7,900 tokens in all, over up to 4,096 each: 294 us, 1.13 PFLOP/s,
// and 303 us. At head dim 64 a third score buffer takes S off the chain (window
// 1024, 7,300 tokens: 135 us); the tensor pipe and the exponential unit are
// active 28 % of the time there and issue slots 47 %: latency, with two softmax
// warps a scheduler to hide it. Tried against this: products of 64 keys with four
// score buffers (1.73 ms: an N = 64 product costs 47 clocks, not 32), the second
// half of P through shared memory (1.63 ms), a row's keys over two warps (1.45
// ms), scores loaded 32 at a time between the weights (1.56 ms).
//
// A row's reference for the exponents is the maximum of its first key tile and
// moves only when a later tile's weights sum up to 2^14, so most tiles need no
// maximum, and O in TMEM is rescaled rarely.
// P is rounded to bf16 because the product's operands share one type; O is
// divided by the sum of the weights before that rounding.
#include <cmath>
#include <cstdlib>
#include <type_traits>

#include "ts_tcgen05.cuh"

namespace ts {
namespace {

constexpr int kBM = 128;  // query rows per tile
constexpr int kBN = 128;  // keys per tile
constexpr int kThreads = 384;
constexpr int kAtom = kBN * 128;  // one [128 rows x 64 bf16] SW128 atom
constexpr int kBadRing = 16;      // key tiles whose bad-page mask is kept
constexpr float kLog2eC = 1.4426950408889634f;
constexpr float kLn2C = 0.6931471805599453f;
constexpr float kMostSum = 16384.f;  // sum of a tile's weights at which a row's reference moves
// 256 threads of softmax and 128 others: 256 * 216 + 128 * 72 == 384 * 168.
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 216, kOtherRegs = 72;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "register split");

template <int D>
struct Lay {
  static constexpr int kAtoms = D / 64;
  static constexpr int kTileBytes = kAtoms * kAtom;  // K, V or Q tile
  static constexpr int kRing = D == 128 ? 5 : 8;     // K and V tiles in flight
  static constexpr int kOffQ = 0;
  static constexpr int kOffKV = 2 * kTileBytes;
  static constexpr int kOffBar = kOffKV + kRing * kTileBytes;
  static constexpr int kOffBad = kOffBar + 384;
  static constexpr int kOffPieces = kOffBad + kBadRing * 4;
  static constexpr int kOffMisc = kOffPieces + 4 * 48;
  static constexpr int kSmem = kOffMisc + 64 + 12 * 8;
  // TMEM: kBufs score buffers of 128 columns taken in turn by the products of
  // both tiles, then O of tile 0 and of tile 1. P goes over the front half of
  // its scores. A third buffer (head dim 64 leaves the columns) lets a tile's
  // next scores be computed before its P V.
  static constexpr int kBufs = D == 128 ? 2 : 3;
  static constexpr uint32_t kTmemO = kBufs * 128;
  static_assert(kTmemO + 2 * D <= 512, "TMEM columns");
};
static_assert(Lay<128>::kSmem <= 227 * 1024, "shared memory");

// An item cut between CTAs: written by the CTA that holds its first key tile.
struct SplitItem {
  int32_t row0;    // its first token's row in the batch, -1: no such item
  int32_t tokens;  // its tokens
  int32_t head;    // kv head
  int32_t parts;   // CTAs that hold its key tiles, this one and the next ones
  int32_t slot;    // the first part's slot; part i > 0 of CTA k + i is slot 2 (k + i)
  int32_t pad[3];
};

struct PrefillParams {
  __nv_bfloat16* out;          // [T, H_q, D]
  float* lse;                  // [T, H_q] or nullptr
  const int32_t* block_table;  // [B, bt_stride]
  const int32_t* seq_lens;     // [B], the new tokens included
  const int32_t* q_indptr;     // [B + 1]
  int32_t T, B, bt_stride, H_q, H_kv, g, page_size, num_pages, window, sinks;
  int32_t tile_tokens;  // tokens per tile: 128 / g
  int32_t item_units;   // units an item counts beyond its key tiles
  int32_t min_units;    // units a CTA takes at least, while there are any
  int32_t slot_rows;    // rows of a partial state: 128 or 256
  float scale_log2;
  uint32_t* err_word;
  SplitItem* split;  // [CTAs]
  float* part_o;     // [2 * CTAs, D / 4, slot_rows, 4]: neighbouring rows (threads) write neighbouring places
  float* part_lse;   // [2 * CTAs, slot_rows]
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// Waits for this thread's loads from TMEM. It takes the registers of one of
// them, so that the compiler neither reads nor copies them before.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// True for one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// The lowest n bits (none below 0, all from 32 on).
__device__ __forceinline__ uint32_t ones(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

// A sequence of the batch, and an item of it.
struct Seq {
  int row0, n, L, blocks;  // first row, new tokens, tokens in the cache, token blocks
};
struct Item {
  int j0, tokens;  // first token and number of tokens
  int p0;          // position of token j0
  int klo, khi;    // keys some row sees: [klo, khi) and [0, sinks)
  int w0, ns, nt;  // first key tile of [klo, khi), tiles of first tokens in front of it, all tiles
};

__device__ __forceinline__ Seq load_seq(const PrefillParams& p, int b) {
  const int r0 = p.q_indptr[b], r1 = p.q_indptr[b + 1];
  Seq s;
  s.row0 = r0;
  s.n = (r0 >= 0 && r0 <= r1 && r1 <= p.T) ? r1 - r0 : 0;  // rows outside the batch: none
  s.L = max(p.seq_lens[b], 0);
  s.blocks = (s.n + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens);
  return s;
}

__device__ __forceinline__ int tiles_of(int keys) { return keys > 0 ? (keys - 1) / kBN + 1 : 0; }

__device__ __forceinline__ Item load_item(const PrefillParams& p, const Seq& s, int block) {
  Item it;
  it.j0 = block * 2 * p.tile_tokens;
  it.tokens = min(s.n - it.j0, 2 * p.tile_tokens);
  it.p0 = s.L - s.n + it.j0;
  // keys past the block table's row do not exist
  const long long cap = min(static_cast<long long>(p.bt_stride) * p.page_size, 1ll << 30);
  const int end = it.p0 + it.tokens;
  it.khi = static_cast<int>(min(static_cast<long long>(max(end, 0)), cap));
  it.klo = (p.window > 0 && it.p0 >= p.window) ? it.p0 - p.window + 1 : 0;
  if (it.klo <= p.sinks) it.klo = 0;  // the window meets the first tokens
  it.w0 = it.klo / kBN;
  it.ns = it.klo > 0 ? min(tiles_of(p.sinks), it.w0) : 0;
  it.nt = it.ns + max(0, tiles_of(it.khi) - it.w0);
  return it;
}

// a / b of non-negative numbers, in 32 bits where they fit.
__device__ __forceinline__ long long div_units(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// Four lanes hold one row each, as four 16-byte chunks; afterwards lane i of
// the four holds chunk i of the four rows. A store of the result then covers
// 64 contiguous bytes of eight rows instead of 16 bytes of 32 rows.
__device__ __forceinline__ void transpose4(uint4 (&v)[4], int lane) {
  auto swap = [&](uint4& keep_lo, uint4& keep_hi, int mask, bool hi) {
    uint4 send = hi ? keep_lo : keep_hi;
    send.x = __shfl_xor_sync(0xffffffffu, send.x, mask);
    send.y = __shfl_xor_sync(0xffffffffu, send.y, mask);
    send.z = __shfl_xor_sync(0xffffffffu, send.z, mask);
    send.w = __shfl_xor_sync(0xffffffffu, send.w, mask);
    if (hi)
      keep_lo = send;
    else
      keep_hi = send;
  };
  swap(v[0], v[1], 1, lane & 1);
  swap(v[2], v[3], 1, lane & 1);
  swap(v[0], v[2], 2, lane & 2);
  swap(v[1], v[3], 2, lane & 2);
}

// A place in a ring and the phase of its barrier.
struct Turn {
  uint32_t at, phase;
  __device__ __forceinline__ explicit Turn(uint32_t a) : at(a), phase(0) {}
  template <uint32_t kPlaces, uint32_t kStep = 1>
  __device__ __forceinline__ void next() {
    at += kStep;
    if (at >= kPlaces) {
      at -= kPlaces;
      phase ^= 1;
    }
  }
};

// A piece of the CTA's range: key tiles [t0, t0 + nk) of one item. Warp 11
// writes them to a ring in shared memory, ahead of the roles that read them.
struct alignas(16) Piece {
  int nk, t0;            // key tiles; nk = 0: an item without keys, nk < 0: the range's end
  int ns, w0;            // key tile i of the item is tile i < ns ? i : w0 + i - ns of the sequence
  int klo, khi;          // keys some row of the item sees: [klo, khi) and [0, sinks)
  int p0, tokens;        // position of its first token, its tokens
  int head, row0, slot;  // kv head; first token's row in the batch; slot of the state, -1: the whole item
  int seq;               // sequence
};
constexpr int kPieces = 4;        // pieces in the ring
constexpr int kPieceReaders = 11;  // warps that read each piece

// The CTA's range of units, walked piece by piece.
struct Walk {
  long long left;        // units of the range still to walk
  int b, h, block, rem;  // the next unit: item, and unit within it
  Seq s;
  bool first;  // no piece returned yet

  // A whole warp finds the item: unit `off` of sequence b0, `n` units to walk.
  __device__ __forceinline__ void init(const PrefillParams& p, int b0, long long off, long long n, int lane) {
    left = n;
    b = b0;
    first = true;
    h = block = rem = 0;
    if (n <= 0) return;
    s = load_seq(p, b);
    long long c = 0;  // units of one kv head
    for (int i = lane; i < s.blocks; i += 32) c += load_item(p, s, i).nt + p.item_units;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    h = static_cast<int>(div_units(off, c));
    off -= h * c;
    for (int base = 0; base < s.blocks; base += 32) {
      const int mine = base + lane < s.blocks ? load_item(p, s, base + lane).nt + p.item_units : 0;
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, off < incl);
      if (hit != 0u) {
        const int at = __ffs(hit) - 1;
        block = base + at;
        rem = static_cast<int>(off) - __shfl_sync(0xffffffffu, incl - mine, at);
        return;
      }
      off -= __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  // The next piece; also whether the item goes on in later CTAs from its first
  // key tile here (then `rest` is the number of its key tiles there).
  __device__ __forceinline__ bool next(const PrefillParams& p, int k, Piece& q, int& rest) {
    while (left > 0) {
      const Item it = load_item(p, s, block);
      const int cost = it.nt + p.item_units;
      const int here = static_cast<int>(min(static_cast<long long>(cost - rem), left));
      const bool owner = rem == 0;
      const int t0 = max(0, rem - p.item_units), t1 = max(t0, rem + here - p.item_units);
      q.nk = t1 - t0;
      q.t0 = t0;
      q.ns = it.ns;
      q.w0 = it.w0;
      q.klo = it.klo;
      q.khi = it.khi;
      q.p0 = it.p0;
      q.tokens = it.tokens;
      q.head = h;
      q.row0 = s.row0 + it.j0;
      q.seq = b;
      left -= here;
      rem += here;
      if (rem == cost) {
        rem = 0;
        if (++block == s.blocks) {
          block = 0;
          if (++h == p.H_kv) {
            h = 0;
            if (left > 0) {
              do {  // a sequence with rows follows
                if (++b >= p.B) {
                  left = 0;
                  break;
                }
                s = load_seq(p, b);
              } while (s.n == 0);
            }
          }
        }
      }
      if (t1 > t0 || (it.nt == 0 && owner)) {
        const bool whole = t0 == 0 && t1 == it.nt;
        q.slot = whole ? -1 : 2 * k + (first ? 0 : 1);
        rest = t0 == 0 ? it.nt - t1 : 0;
        first = false;
        return true;
      }
    }
    return false;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const PrefillParams p,
                                                              const __grid_constant__ CUtensorMap qmap,
                                                              const __grid_constant__ CUtensorMap kmap,
                                                              const __grid_constant__ CUtensorMap vmap) {
  using L = Lay<D>;
  constexpr int kAtoms = L::kAtoms, kRing = L::kRing, kTile = L::kTileBytes;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int k = blockIdx.x;
  pdl_launch_dependents();
  if ((smem_u32(smem) & 1023u) != 0) {
    if (tid == 0) set_device_error(p.err_word, TS_DEVERR_SMEM_ALIGN);
    return;
  }
  constexpr int kBufs = L::kBufs;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  auto b_full = [&](int i) { return smem_u32(&bars[i]); };                 // K or V tile landed
  auto b_empty = [&](int i) { return smem_u32(&bars[kRing + i]); };        // and no longer needed
  // scores, weights of tile t's product number n (of the CTA's): kBufs barriers
  // each in turn. They are a tile's own, so that a tile without rows in some
  // pieces cannot see another's phases pass.
  auto b_sfull = [&](int t, uint32_t n) { return smem_u32(&bars[2 * kRing + t * kBufs + n % kBufs]); };
  auto b_pfull = [&](int t, uint32_t n) { return smem_u32(&bars[2 * kRing + (2 + t) * kBufs + n % kBufs]); };
  auto buf_phase = [&](uint32_t n) { return (n / kBufs) & 1; };
  constexpr int kBar0 = 2 * kRing + 4 * kBufs;
  auto b_ofree = [&](int t) { return smem_u32(&bars[kBar0 + t]); };  // O of tile t has been read out
  // Tile t's P V number n has completed. With three score buffers the one before
  // may be running still when it is asked for: two barriers in turn.
  constexpr uint32_t kDone = kBufs == 3 ? 2 : 1;
  auto b_pvdone = [&](int t, uint32_t n) { return smem_u32(&bars[kBar0 + 2 + 2 * t + n % kDone]); };
  auto pv_phase = [&](uint32_t n) { return (n / kDone) & 1; };
  const uint32_t b_qfull = smem_u32(&bars[kBar0 + 6]), b_qempty = smem_u32(&bars[kBar0 + 7]);
  auto b_piece = [&](int i) { return smem_u32(&bars[kBar0 + 8 + i]); };
  auto b_taken = [&](int i) { return smem_u32(&bars[kBar0 + 8 + kPieces + i]); };
  static_assert((kBar0 + 8 + 2 * kPieces) * 8 <= L::kOffBad - L::kOffBar, "mbarriers fit their place");
  static_assert(kPieces * sizeof(Piece) == L::kOffMisc - L::kOffPieces, "piece ring");
  Piece* ring = reinterpret_cast<Piece*>(smem + L::kOffPieces);
  volatile uint32_t* bad_ring = reinterpret_cast<volatile uint32_t*>(smem + L::kOffBad);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  int* start_seq = reinterpret_cast<int*>(smem + L::kOffMisc + 16);
  long long* start_off = reinterpret_cast<long long*>(smem + L::kOffMisc + 24);
  long long* warp_tot = reinterpret_cast<long long*>(smem + L::kOffMisc + 64);

  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(b_full(i), 1);
      mbar_init(b_empty(i), 1);
    }
    for (int t = 0; t < 2; ++t) {
      for (int i = 0; i < kBufs; ++i) {
        mbar_init(b_sfull(t, i), 2);  // the products' commit and the issuer's own arrival
        mbar_init(b_pfull(t, i), 4);
      }
      for (int i = 0; i < 2; ++i) mbar_init(b_pvdone(t, i), 1);
      mbar_init(b_ofree(t), 4);
    }
    mbar_init(b_qfull, 1);
    mbar_init(b_qempty, 1);
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(b_piece(i), 1);
      mbar_init(b_taken(i), kPieceReaders);
    }
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    prefetch_map(&qmap);
    prefetch_map(&kmap);
    prefetch_map(&vmap);
  }
  if (warp == 0) tmem_alloc(smem_u32(tmem_slot), 512);

  // ---- prologue: this CTA's range of units --------------------------------
  // Units of every sequence, by eight lanes (up to 48 sequences) or one each,
  // and their prefix sums over the threads; the sums of a sequence are kept in
  // the K/V area, free until the first copy, for the search. (One sequence of
  // 65,536 tokens, window 64: 98.6 us with one lane, 73.8 with eight, 69.2 with
  // 32, which take 0.2 us longer for 33 tokens; 48 of 2,048: 86.8 with one, 84.7
  // with eight.)
  const int lps = p.B <= kThreads / 8 ? 8 : 1;
  const int chunk = (p.B + kThreads / lps - 1) / (kThreads / lps);
  const int lo = min(p.B, tid / lps * chunk), hi = min(p.B, lo + chunk);
  long long* kept = reinterpret_cast<long long*>(smem + L::kOffKV);
  const bool keep = p.B <= 8192;  // 64 KB
  auto seq_units = [&](int b, int first, int step) {
    const Seq s = load_seq(p, b);
    long long c = 0;
    for (int i = first; i < s.blocks; i += step) c += load_item(p, s, i).nt + p.item_units;
    return c * p.H_kv;
  };
  long long mine = 0;
  for (int x = 0; x < chunk; ++x) {
    const int b = lo + x;
    long long c = b < hi ? seq_units(b, tid % lps, lps) : 0;
    for (int o = lps / 2; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    if (tid % lps == 0 && b < hi) {
      if (keep) kept[b] = c;
      mine += c;
    }
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_tot[warp] = incl;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  long long wbase = 0, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    const long long v = warp_tot[w];
    if (w < warp) wbase += v;
    total += v;
  }
  const long long excl = wbase + incl - mine;
  const long long G = max(1ll, min(static_cast<long long>(gridDim.x), div_units(total, p.min_units)));
  const long long q_units = div_units(total, G), r_units = total - q_units * G;
  const long long u0 = k < G ? k * q_units + min(static_cast<long long>(k), r_units) : total;
  const long long u1 = k < G ? u0 + q_units + (k < r_units ? 1 : 0) : total;
  if (u0 < u1 && excl <= u0 && u0 < excl + mine) {
    long long off = excl;
    for (int b = lo; b < hi; ++b) {
      const long long c = keep ? kept[b] : seq_units(b, 0, 1);
      if (u0 < off + c) {
        *start_seq = b;
        *start_off = u0 - off;
        break;
      }
      off += c;
    }
  }
  fence_async_smem();  // the sums' place is written by copies next
  __syncthreads();
  constexpr uint32_t tmem = 0;  // all 512 columns: there is no other place for them
  const uint32_t sQ = smem_u32(smem + L::kOffQ), sKV = smem_u32(smem + L::kOffKV);

  const int tt = p.tile_tokens;
  bool ok = true;
  // A reader waits for piece n (all its threads that use it), copies what it
  // needs, and hands the entry back once per warp.
  auto piece_ready = [&](uint32_t n) { return mbar_wait(b_piece(n % kPieces), (n / kPieces) & 1); };
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 11) {
      // ---------------- pieces ------------------------------------------------
      Walk w;
      w.init(p, *start_seq, *start_off, u1 - u0, lane);
      pdl_wait_primary();  // lengths and row offsets are read before it, all else behind it
      if (lane == 0) {
        p.split[k].row0 = -1;
        bool more = true;
        uint32_t pieces = 0;  // with queries
        for (uint32_t n = 0; more; ++n) {
          Piece q;
          int rest = 0;
          more = w.next(p, k, q, rest);
          if (!more) q.nk = -1;
          if (n >= kPieces && !mbar_wait(b_taken(n % kPieces), (n / kPieces - 1) & 1)) {
            set_device_error(p.err_word, TS_DEVERR_TIMEOUT);
            break;
          }
          ring[n % kPieces] = q;
          mbar_arrive(b_piece(n % kPieces));
          if (q.nk > 0) {  // its queries, once the products have read the last piece's
            if (pieces > 0 && !mbar_wait(b_qempty, (pieces - 1) & 1)) {
              set_device_error(p.err_word, TS_DEVERR_TIMEOUT);
              mbar_wait(b_qfull, (pieces - 1) & 1);  // a copy in flight lands first
              break;
            }
            const int nq = q.tokens > tt ? 2 : 1;
            mbar_arrive_expect_tx(b_qfull, nq * kAtoms * tt * p.g * 128);
            for (int t2 = 0; t2 < nq; ++t2)
              for (int a = 0; a < kAtoms; ++a)
                tma_load_3d(sQ + t2 * kTile + a * kAtom, &qmap, a * 64, q.head * p.g, q.row0 + t2 * tt, b_qfull);
            ++pieces;
          }
          if (more && rest > 0) {  // its last key tile lies `rest` units behind this CTA's range
            const long long big = r_units * (q_units + 1), last = u1 + rest - 1;
            SplitItem si;
            si.tokens = q.tokens;
            si.head = q.head;
            si.parts =
                static_cast<int>(last < big ? div_units(last, q_units + 1)
                                            : r_units + div_units(last - big, max(q_units, 1ll))) - k + 1;
            si.slot = q.slot;
            si.row0 = q.row0;
            p.split[k] = si;
          }
        }
      }
    } else if (warp != 9) {
      // ---------------- K (warp 8) and V (warp 10): lane i holds page i of the key tile
      pdl_wait_primary();
      const bool is_v = warp == 10;
      const CUtensorMap* map = is_v ? &vmap : &kmap;
      const int npg = kBN / p.page_size;
      const int oob = p.num_pages * p.page_size;  // a row past the pool: zero fill
      uint32_t tiles = 0;                         // key tiles loaded; K of tile j is tile 2 j of the ring, V 2 j + 1
      for (uint32_t n = 0;; ++n) {
        ok = __all_sync(0xffffffffu, piece_ready(n));
        if (!ok) break;
        const Piece q = ring[n % kPieces];
        __syncwarp();
        if (lane == 0) mbar_arrive(b_taken(n % kPieces));
        if (q.nk < 0) break;
        // tokens past the block table's row: absent, as those of a bad page
        if (lane == 0 && q.p0 + q.tokens > max(q.khi, 0)) set_device_error(p.err_word, TS_DEVERR_PAGE_RANGE);
        const int64_t bt = static_cast<int64_t>(q.seq) * p.bt_stride;
        auto page_row = [&](int i, uint32_t& bad) {  // this lane's page of tile i of the item
          const int pi = (i < q.ns ? i : q.w0 + i - q.ns) * npg + lane, t = pi * p.page_size;
          int row = oob;
          bool wrong = false;
          if (lane < npg && t < q.khi && (t + p.page_size > q.klo || t < p.sinks)) {
            const int page = p.block_table[bt + pi];
            wrong = page < 0 || page >= p.num_pages;
            if (!wrong) row = page * p.page_size;
          }
          bad = __ballot_sync(0xffffffffu, wrong);
          return row;
        };
        const int t1 = q.t0 + q.nk;
        uint32_t bad = 0;
        int row = q.nk > 0 ? page_row(q.t0, bad) : oob;
        for (int i = q.t0; i < t1; ++i) {
          uint32_t bad_next = 0;
          const int row_next = i + 1 < t1 ? page_row(i + 1, bad_next) : oob;
          if (lane == 0 && !is_v) {
            bad_ring[tiles % kBadRing] = bad;
            if (bad) set_device_error(p.err_word, TS_DEVERR_PAGE_RANGE);
          }
          const uint32_t seq = 2 * tiles + (is_v ? 1 : 0), s = seq % kRing;
          if (seq >= kRing) {
            ok = __all_sync(0xffffffffu, mbar_wait(b_empty(s), (seq / kRing - 1) & 1));
            if (!ok) break;
          }
          if (lane == 0) mbar_arrive_expect_tx(b_full(s), kTile);
          __syncwarp();
          const int pg = lane / kAtoms, a = lane % kAtoms;
          const int r = __shfl_sync(0xffffffffu, row, pg);
          if (lane < npg * kAtoms)
            tma_load_3d(sKV + s * kTile + a * kAtom + pg * p.page_size * 128, map, a * 64, r, q.head, b_full(s));
          ++tiles;
          row = row_next;
          bad = bad_next;
        }
        if (!ok) break;
      }
      if (!ok && lane == 0) {
        set_device_error(p.err_word, TS_DEVERR_TIMEOUT);
        // let the copies in flight land before the CTA's shared memory goes
        for (uint32_t i = tiles > kRing ? tiles - kRing : 0; i < tiles; ++i) {
          const uint32_t seq = 2 * i + (is_v ? 1 : 0);
          mbar_wait(b_full(seq % kRing), (seq / kRing) & 1);
        }
      }
    } else if (warp == 9) {
      // ---------------- products --------------------------------------------
      pdl_wait_primary();  // no bounded wait runs while the previous kernel does
      // The whole warp runs this code and one elected lane issues: descriptors
      // and loop counts stay in uniform registers, as the instruction wants
      // them. (Run by one lane in a branch of its own, every product moved its
      // operands there first and took 119 cycles instead of 64.)
      constexpr uint32_t iS = idesc_bf16(kBM, kBN, 0);
      constexpr uint32_t iO = idesc_bf16(kBM, D, 1);
      // descriptors of the first Q and ring tile; others differ by an address
      // difference in 16-byte units, which stays within the address field
      const uint64_t dQ = desc_sw128(sQ), dK = desc_sw128(sKV), dV = desc_sw128(sKV, kAtom, 1024);
      constexpr uint64_t kTileStep = kTile >> 4;
      // Counters are kept as (place, phase) pairs and tile numbers are compile-
      // time: what this warp computes between two products delays them.
      Turn kt(0), vt(1);                            // ring places of the next K and V tile
      Turn st[2] = {Turn(0), Turn(0)}, pt[2] = {Turn(0), Turn(0)};  // barriers of each tile's next S and P V
      uint32_t pieces = 0, used[2] = {0, 0};        // with products; of each tile
      uint32_t pvs[2] = {0, 0};                     // P V products of each tile
      auto run_piece = [&](auto tiles_tag, const int nk) {
        constexpr int NQ = decltype(tiles_tag)::value;  // tiles with rows
        int left = nk;         // K tiles whose S products are not all issued
        uint32_t sb = 0, pb = 0;  // buffers of the next S and P V: the last piece's products are all issued
        // S of tile t; the last tile's hands the K tile back, the last K tile's the queries
        auto issue_s = [&](auto tag) {
          constexpr int t = decltype(tag)::value;
          const uint64_t q = dQ + t * kTileStep, kb = dK + kt.at * kTileStep;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            constexpr uint64_t kAtomStep = kAtom >> 4;
            const uint64_t off = (ks >> 2) * kAtomStep + (ks & 3) * 2;
            mma_bf16(sb * 128, q + off, kb + off, iS, ks > 0);
          }
          const uint32_t done = b_sfull(t, st[t].at);
          mma_commit(done);
          // the arrival carries what the key tile's barrier carried here: the
          // softmax reads the tile's bad-page mask after it
          mbar_arrive(done);
          if (t == NQ - 1) {
            mma_commit(b_empty(kt.at));
            if (left == 1) mma_commit(b_qempty);
          }
        };
        auto after_s = [&](auto tag) {
          constexpr int t = decltype(tag)::value;
          st[t].template next<kBufs>();
          if (++sb == kBufs) sb = 0;
          if (t == NQ - 1) {
            kt.template next<kRing, 2>();
            --left;
          }
        };
        using T0 = std::integral_constant<int, 0>;
        using T1 = std::integral_constant<int, NQ - 1>;
        auto prime = [&](auto tag) {
          constexpr int t = decltype(tag)::value;
          if (!ok || left == 0) return;
          if (t == 0) ok = __all_sync(0xffffffffu, mbar_wait(b_full(kt.at), kt.phase));
          if (!ok) return;
          tc_fence_after();
          if (elect_one()) issue_s(tag);
          __syncwarp();
          after_s(tag);
        };
        // Products on different accumulators may overlap, so a buffer's next S
        // waits until the P V that read its weights has completed.
        auto pv_done = [&](int t) { return pvs[t] == 0 || mbar_wait(b_pvdone(t, pvs[t] - 1), pv_phase(pvs[t] - 1)); };
        ok = __all_sync(0xffffffffu, pv_done(0) && pv_done(1));
        prime(T0());
        prime(T1());
        // P V of tile t and the tile's next S. With three buffers S goes into that
        // of the product before and is issued first, so that it is there when the
        // softmax has written this step's weights; with two it goes into that of
        // this P V and comes behind it.
        auto step = [&](auto tag, const bool first) {
          constexpr int t = decltype(tag)::value;
          constexpr int ts = NQ == 1 ? 0 : t, before = NQ == 1 ? 0 : 1 - t;
          const bool more = left > 0;
          const uint32_t vbar = b_full(vt.at), kbar = b_full(kt.at), pbar = b_pfull(t, pt[t].at);
          if (kBufs == 3 && more) {
            ok = __all_sync(0xffffffffu, (ts > 0 || mbar_wait(kbar, kt.phase)) && pv_done(before));
            if (!ok) return;
            tc_fence_after();
            if (elect_one()) issue_s(std::integral_constant<int, ts>());
            __syncwarp();
            after_s(std::integral_constant<int, ts>());
          }
          // what is left to wait for, asked for all at once
          const bool have_v = t > 0 || mbar_try_wait(vbar, vt.phase);
          const bool have_k = kBufs == 3 || ts > 0 || !more || mbar_try_wait(kbar, kt.phase);
          const bool have_p = mbar_try_wait(pbar, pt[t].phase);
          bool good = have_v && have_k && have_p;
          if (!good)
            good = (have_v || mbar_wait(vbar, vt.phase)) && (have_k || mbar_wait(kbar, kt.phase)) &&
                   (have_p || mbar_wait(pbar, pt[t].phase));
          // O of the tile's last piece has been read out
          if (first && used[t] > 0) good = good && mbar_wait(b_ofree(t), (used[t] - 1) & 1);
          ok = __all_sync(0xffffffffu, good);
          if (!ok) return;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t vb = dV + vt.at * kTileStep;
#pragma unroll
            for (int ks = 0; ks < kBN / 16; ++ks)
              mma_bf16_tmem_a(L::kTmemO + t * D, pb * 128 + ks * 8, vb + ks * 128, iO, (!first || ks > 0) ? 1u : 0u);
            mma_commit(b_pvdone(t, pvs[t]));
            if (t == NQ - 1) mma_commit(b_empty(vt.at));
          }
          __syncwarp();
          ++pvs[t];
          if (kBufs == 2 && more) {
            ok = __all_sync(0xffffffffu, pv_done(t));
            if (!ok) return;
            tc_fence_after();
            if (elect_one()) issue_s(std::integral_constant<int, ts>());
            __syncwarp();
          }
          if (kBufs == 2 && more) after_s(std::integral_constant<int, ts>());
          pt[t].template next<kBufs>();
          if (++pb == kBufs) pb = 0;
          if (t == NQ - 1) vt.template next<kRing, 2>();
        };
        for (int i = 0; ok && i < nk; ++i) {
          step(T0(), i == 0);
          if (NQ == 2 && ok) step(T1(), i == 0);
        }
        ++used[0];
        if (NQ == 2) ++used[1];
      };
      for (uint32_t n = 0;; ++n) {
        ok = __all_sync(0xffffffffu, piece_ready(n));
        if (!ok) break;
        // a reduction's result is known to be the same in all lanes
        const int nk = __reduce_max_sync(0xffffffffu, ring[n % kPieces].nk);
        const bool two = __reduce_max_sync(0xffffffffu, ring[n % kPieces].tokens) > tt;
        if (lane == 0) mbar_arrive(b_taken(n % kPieces));
        __syncwarp();
        if (nk < 0) break;
        if (nk == 0) continue;
        ok = __all_sync(0xffffffffu, mbar_wait(b_qfull, pieces & 1));
        if (!ok) break;
        if (two)
          run_piece(std::integral_constant<int, 2>(), nk);
        else
          run_piece(std::integral_constant<int, 1>(), nk);
        if (!ok) break;
        ++pieces;
      }
      if (!ok && lane == 0) set_device_error(p.err_word, TS_DEVERR_TIMEOUT);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---------------- softmax: one query row per thread -----------------------
    pdl_wait_primary();
    const int t = warp >> 2, r = tid & 127;
    const int rt = r / p.g, rh = r - rt * p.g, j = t * tt + rt;  // its token of the tile, head, token of the item
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + lanes + L::kTmemO + t * D;
    uint32_t steps = 0, tiles = 0;  // products of this tile; key tiles of the CTA's pieces so far
    for (uint32_t n = 0;; ++n) {
      ok = __all_sync(0xffffffffu, piece_ready(n));
      if (!ok) break;
      const Piece& q = ring[n % kPieces];  // read until this warp hands it back
      const int nk = q.nk;
      if (nk < 0) break;
      if (q.tokens <= t * tt) {  // no row in this tile
        __syncwarp();
        if (lane == 0) mbar_arrive(b_taken(n % kPieces));
        tiles += nk;
        continue;
      }
      const int pos = q.p0 + j;
      const bool real = rt < tt && j < q.tokens;
      const int nq = q.tokens > tt ? 2 : 1;
      float m = -INFINITY, l = 0.f;
      const int klo = q.klo, khi = q.khi, ns = q.ns, w0 = q.w0, t0 = q.t0;
      const int pfirst = q.p0 + t * tt, plast = pfirst + tt - 1;  // positions of the tile's rows
      bool fresh = true;  // some row has no reference yet
      for (int i = 0; i < nk; ++i) {
        // before the scores are there: what is known of the key tile
        const int k0 = (t0 + i < ns ? t0 + i : w0 + t0 + i - ns) * kBN;
        const int first = (p.window > 0 && pos >= p.window) ? pos - p.window + 1 - k0 : 0;
        const int end = min(pos + 1, khi) - k0, keep = p.sinks - k0;
        // every row of the tile sees every key: no masks
        const bool all = k0 + kBN - 1 <= pfirst && k0 + kBN <= khi && p.scale_log2 > 0.f &&
                         (p.window == 0 || k0 > plast - p.window || k0 + kBN <= p.sinks);
        auto cuts_page = [&](int x) { return x > k0 && x < k0 + kBN && (x & (p.page_size - 1)) != 0; };
        const bool ragged = cuts_page(khi) || cuts_page(klo) || (klo > 0 && cuts_page(p.sinks));
        const uint32_t tS = tmem + lanes + (i * nq + t) % kBufs * 128;
        ok = __all_sync(0xffffffffu, mbar_wait(b_sfull(t, steps), buf_phase(steps)));
        if (!ok) break;
        tc_fence_after();
        float s[kBN];
#pragma unroll
        for (int c = 0; c < kBN; c += 32) tmem_ld32(tS + c, reinterpret_cast<uint32_t*>(s) + c);
        // Rows of a loaded page that no row sees (past the sequence's end, in
        // front of the window, behind the first tokens) may hold anything, and
        // 0 * NaN is NaN in the product: zero them once landed. Both tiles'
        // warps do, each before its own product. (Not before the scores: a tile
        // without rows in some pieces may be pieces ahead of the copies.)
        if (ragged) {
          const uint32_t vseq = 2 * tiles + 1;
          ok = __all_sync(0xffffffffu, mbar_wait(b_full(vseq % kRing), (vseq / kRing) & 1));
          if (!ok) break;
          const int key = k0 + r;
          if (!(key < khi && (key >= klo || key < p.sinks))) {
            unsigned char* v = smem + L::kOffKV + (vseq % kRing) * kTile + r * 128;
#pragma unroll
            for (int a = 0; a < kAtoms; ++a)
#pragma unroll
              for (int c = 0; c < 8; ++c)
                *reinterpret_cast<uint4*>(v + a * kAtom + c * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_async_smem();
        }
        const uint32_t bad = bad_ring[tiles % kBadRing];
        const bool full = all && bad == 0u;
        const float f = full ? p.scale_log2 : 1.f;  // what the scores are still to be multiplied by
        auto weigh = [&](int c0, float ms, float2& l2) {  // weights of 32 keys, written as bf16
          const float2 f2 = make_float2(f, f), nm = make_float2(-ms, -ms);
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 x = __ffma2_rn(make_float2(s[c0 + c], s[c0 + c + 1]), f2, nm);
            const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
            pk[c / 2] = float2_to_bf16x2(e.x, e.y);
            l2 = __fadd2_rn(l2, e);
          }
          tmem_st16(tS + c0 / 2, pk);
        };
        // The reference m is a maximum over earlier keys, and any reference
        // gives the same quotient while nothing overflows: a tile's weights are
        // taken against the old one without looking for the tile's maximum, and
        // only where a row's sum reaches kMostSum is it moved. Rows that no one
        // reads do not count.
        bool move = fresh;
        float2 l2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kBN; c += 32) tmem_wait_ld32(reinterpret_cast<uint32_t*>(s) + c);
        if (!full) {
#pragma unroll
          for (int c0 = 0; c0 < kBN; c0 += 32) {
            uint32_t vis = ones(end - c0) & (~ones(first - c0) | ones(keep - c0));
            if (bad != 0u) {
              for (int c = 0; c < 32; c += p.page_size)
                if ((bad >> ((c0 + c) / p.page_size)) & 1u) vis &= ~(ones(c + p.page_size) & ~ones(c));
            }
#pragma unroll
            for (int c = 0; c < 32; ++c) s[c0 + c] = (vis >> c) & 1u ? s[c0 + c] * p.scale_log2 : -INFINITY;
          }
        }
        if (!move) {
#pragma unroll
          for (int c0 = 0; c0 < kBN; c0 += 32) weigh(c0, m, l2);
          move = __any_sync(0xffffffffu, real && !(l2.x + l2.y < kMostSum));
        }
        if (move) {
          float mx = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
          for (int c = 0; c < kBN; c += 8) {
            mx = fmax3(mx, s[c], s[c + 1]);
            mx1 = fmax3(mx1, s[c + 2], s[c + 3]);
            mx2 = fmax3(mx2, s[c + 4], s[c + 5]);
            mx3 = fmax3(mx3, s[c + 6], s[c + 7]);
          }
          mx = fmaxf(fmaxf(mx, mx1), fmaxf(mx2, mx3)) * f;
          const float mnew = fmaxf(m, mx);
          if (i > 0) {  // O so far is rescaled: every P V of it must be done
            ok = __all_sync(0xffffffffu, mbar_wait(b_pvdone(t, steps - 1), pv_phase(steps - 1)));
            if (!ok) break;
            tc_fence_after();
            const float alpha = m == -INFINITY ? 0.f : fast_exp2(m - mnew);
            l *= alpha;
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
              uint32_t u[32];
              tmem_ld32(tO + c0, u);
              tmem_wait_ld32(u);
#pragma unroll
              for (int x = 0; x < 32; ++x) u[x] = __float_as_uint(__uint_as_float(u[x]) * alpha);
              tmem_st32(tO + c0, u);
            }
          }
          m = mnew;
          fresh = __any_sync(0xffffffffu, real && m == -INFINITY);
          l2 = make_float2(0.f, 0.f);
#pragma unroll
          for (int c0 = 0; c0 < kBN; c0 += 32) weigh(c0, m == -INFINITY ? 0.f : m, l2);
        }
        l += l2.x + l2.y;
        // The last weights are handed over once the P V before has completed: a
        // barrier tells its newest phase only from the one before, and a tile that
        // has the buffers for itself may be two products ahead of a late V tile.
        if (i > 0 && i == nk - 1) {
          ok = __all_sync(0xffffffffu, mbar_wait(b_pvdone(t, steps - 1), pv_phase(steps - 1)));
          if (!ok) break;
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_pfull(t, steps));
        ++steps;
        ++tiles;
      }
      if (!ok) break;
      // epilogue: O / sum and the LSE (no key: O = 0, LSE = -inf; a score that
      // is NaN or +inf makes the sum NaN, and O and the LSE with it)
      const float inv = l == 0.f ? 0.f : 1.0f / l;
      const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
      const int slot = q.slot;
      const int64_t row = static_cast<int64_t>(q.row0 + j) * p.H_q + q.head * p.g + rh;
      __syncwarp();
      if (lane == 0) mbar_arrive(b_taken(n % kPieces));
      if (nk > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(b_pvdone(t, steps - 1), pv_phase(steps - 1)));
        if (!ok) break;
        tc_fence_after();
      }
      auto read_o = [&](int c0, float* o) {
        if (nk > 0) {
          tmem_ld32(tO + c0, reinterpret_cast<uint32_t*>(o));
          tmem_wait_ld32(reinterpret_cast<uint32_t*>(o));
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = 0.f;
        }
#pragma unroll
        for (int x = 0; x < 32; ++x) o[x] *= inv;
      };
      if (slot < 0) {
        // lane i of each four writes chunk i of the four's rows
        long long rows[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
          rows[x] = __shfl_sync(0xffffffffu, real ? static_cast<long long>(row) : -1ll, (lane & ~3) + x);
        for (int c0 = 0; c0 < D; c0 += 32) {
          float o[32];
          read_o(c0, o);
          uint4 v[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            v[x] = make_uint4(float2_to_bf16x2(o[8 * x], o[8 * x + 1]), float2_to_bf16x2(o[8 * x + 2], o[8 * x + 3]),
                              float2_to_bf16x2(o[8 * x + 4], o[8 * x + 5]),
                              float2_to_bf16x2(o[8 * x + 6], o[8 * x + 7]));
          transpose4(v, lane);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (rows[x] >= 0) *reinterpret_cast<uint4*>(p.out + rows[x] * D + c0 + (lane & 3) * 8) = v[x];
        }
        if (real && p.lse) p.lse[row] = lse2 * kLn2C;
      } else {
        float* dst = p.part_o + (static_cast<int64_t>(slot) * (D / 4) * p.slot_rows + t * kBM + r) * 4;
        for (int c0 = 0; c0 < D; c0 += 32) {
          float o[32];
          read_o(c0, o);
          if (real) {
#pragma unroll
            for (int x = 0; x < 32; x += 4)
              *reinterpret_cast<float4*>(dst + static_cast<int64_t>(c0 + x) * p.slot_rows) =
                  make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
          }
        }
        if (real) p.part_lse[static_cast<int64_t>(slot) * p.slot_rows + t * kBM + r] = lse2 * kLn2C;
      }
      if (nk > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_ofree(t));
      }
    }
    if (!ok && lane == 0) set_device_error(p.err_word, TS_DEVERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the states of the items cut between CTAs: block (x, k) takes 32 rows
// of the item whose first part CTA k holds. Lane r of every warp holds row r,
// warp w its columns 4 (w + 8 i); the joined rows leave through shared memory.
template <int D>
__global__ void __launch_bounds__(256) prefill_merge_kernel(const PrefillParams p) {
  constexpr int kN = D / 32;  // groups of four columns per thread
  __shared__ uint2 rows_s[32][D / 4 + 1];
  __shared__ float top_s[8][32];
  pdl_launch_dependents();
  pdl_wait_primary();
  const int k = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SplitItem si = p.split[k];
  const int r = blockIdx.x * 32 + lane;  // row of the slot
  const int tile = r / kBM, rt = r % kBM / p.g, j = tile * p.tile_tokens + rt;
  const bool real = rt < p.tile_tokens && j < si.tokens;
  if (si.row0 < 0 || !__syncthreads_or(real)) return;
  // the rows' largest LSE: the parts shared out among the warps
  float mx = -INFINITY;
  auto at = [&](int i) { return static_cast<int64_t>(i == 0 ? si.slot : 2 * (k + i)) * p.slot_rows; };
  if (real)
    for (int i = warp; i < si.parts; i += 8) mx = fmaxf(mx, p.part_lse[at(i) + r]);
  top_s[warp][lane] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) mx = fmaxf(mx, top_s[w][lane]);
  const float ms = mx == -INFINITY ? 0.f : mx;
  float4 a[kN];
  float sum = 0.f;
#pragma unroll
  for (int x = 0; x < kN; ++x) a[x] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (real) {
    // four parts' loads in flight (33 tokens over 1,000, cut into 5 parts
    // each: 16.1 us both kernels, with one in flight 17.6)
    for (int i0 = 0; i0 < si.parts; i0 += 4) {
      float lse[4];
      float4 v[4][kN];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = min(i0 + u, si.parts - 1);
        const float4* o = reinterpret_cast<const float4*>(p.part_o) + at(i) * (D / 4) + r;
        lse[u] = i0 + u < si.parts ? p.part_lse[at(i) + r] : -INFINITY;
#pragma unroll
        for (int x = 0; x < kN; ++x) v[u][x] = o[static_cast<int64_t>(warp + 8 * x) * p.slot_rows];
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (i0 + u >= si.parts) break;
        const float wt = __expf(lse[u] - ms);
        sum += wt;
#pragma unroll
        for (int x = 0; x < kN; ++x) {
          a[x].x += wt * v[u][x].x;
          a[x].y += wt * v[u][x].y;
          a[x].z += wt * v[u][x].z;
          a[x].w += wt * v[u][x].w;
        }
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a part's NaN stays one
#pragma unroll
  for (int x = 0; x < kN; ++x)
    rows_s[lane][warp + 8 * x] =
        make_uint2(float2_to_bf16x2(a[x].x * inv, a[x].y * inv), float2_to_bf16x2(a[x].z * inv, a[x].w * inv));
  const int64_t out = real ? static_cast<int64_t>(si.row0 + j) * p.H_q + si.head * p.g + r % kBM % p.g : -1;
  if (warp == 0 && real && p.lse) p.lse[out] = sum == 0.f ? -INFINITY : ms + logf(sum);
  __syncthreads();
  // warp w writes rows w, w + 8, ...: one row of D / 4 pairs of words at a time
  for (int rr = warp; rr < 32; rr += 8) {
    const long long to = __shfl_sync(0xffffffffu, static_cast<long long>(out), rr);
    if (to >= 0 && lane < D / 4) reinterpret_cast<uint2*>(p.out + to * D)[lane] = rows_s[rr][lane];
  }
}

// 3-D map over rows of `heads` vectors of D bf16, `row_step` elements apart:
// (column, row or head, head or row) with 128-byte swizzle and zero fill.
ts_status make_map(CUtensorMap* map, const void* base, uint64_t D, uint64_t dim1, uint64_t step1, uint64_t dim2,
                   uint64_t step2, uint32_t box1, uint32_t box2) {
  auto fn = tensor_map_encoder();
  if (!fn) return fail(TS_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[3] = {D, dim1, dim2};
  cuuint64_t strides[2] = {step1 * 2, step2 * 2};
  cuuint32_t box[3] = {64, box1, box2};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult res = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (res != CUDA_SUCCESS) return fail(TS_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(res));
  return TS_OK;
}

struct WsLayout {
  size_t split, part_o, part_lse, total;
};

WsLayout workspace_layout(int ctas, int slot_rows, int D) {
  WsLayout w;
  w.split = kWorkspaceAlign;  // behind the error word
  w.part_o = align_up(w.split + static_cast<size_t>(ctas) * sizeof(SplitItem), kWorkspaceAlign);
  w.part_lse = align_up(w.part_o + 2ull * ctas * slot_rows * D * sizeof(float), kWorkspaceAlign);
  w.total = align_up(w.part_lse + 2ull * ctas * slot_rows * sizeof(float), kWorkspaceAlign);
  return w;
}

int slot_rows_of(int T, int g) { return T > kBM / g ? 2 * kBM : kBM; }

template <int D>
ts_status launch(const PrefillParams& prm, const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                 int ctas, cudaStream_t s) {
  ts_status st = prepare_once(reinterpret_cast<const void*>(prefill_kernel<D>), [](const void* f) {
    ts_status s2 = cuda_check(cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::kSmem),
                              "prefill smem attribute");
    if (s2 != TS_OK) return s2;
    cudaFuncAttributes fa;
    s2 = cuda_check(cudaFuncGetAttributes(&fa, f), "query kernel attributes");
    if (s2 != TS_OK) return s2;
    if (fa.numRegs < kLaunchRegs)
      return fail(TS_ERR_UNSUPPORTED, "prefill kernel compiled with %d registers/thread, the register split needs %d",
                  fa.numRegs, kLaunchRegs);
    return TS_OK;
  });
  if (st != TS_OK) return st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Lay<D>::kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  {
    LaunchTrace trace("prefill_kernel", s);
    st = cuda_check(cudaLaunchKernelEx(&cfg, prefill_kernel<D>, prm, qmap, kmap, vmap), "prefill launch");
  }
  if (st != TS_OK) return st;
  cfg.gridDim = dim3(static_cast<unsigned>(prm.slot_rows / 32), static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  LaunchTrace trace("prefill_merge_kernel", s);
  return cuda_check(cudaLaunchKernelEx(&cfg, prefill_merge_kernel<D>, prm), "prefill merge launch");
}

}  // namespace

// float32 path (ts_prefill_f32.cu).
ts_status launch_prefill_f32(const float* q, int64_t q_stride, const float* k_pool, const float* v_pool,
                             const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens,
                             const int32_t* q_indptr, int32_t T, int32_t B, int32_t H_q, int32_t H_kv, int32_t D,
                             int32_t page_size, int32_t num_pages, int32_t window, int32_t sinks, float scale,
                             float* out, float* lse, uint32_t* err_word, float* part_o, float* part_lse, int32_t ctas,
                             cudaStream_t stream);

}  // namespace ts

extern "C" size_t ts_paged_prefill_workspace_size(int32_t T, int32_t B, int32_t H_q, int32_t H_kv, int32_t D) {
  using namespace ts;
  if (T < 0 || B < 0 || H_q <= 0 || H_kv <= 0 || H_q % H_kv != 0 || H_q / H_kv > 64 || (D != 64 && D != 128)) return 0;
  const int ctas = paged_decode_ctas();
  return ctas > 0 ? workspace_layout(ctas, slot_rows_of(T, H_q / H_kv), D).total : 0;
}

extern "C" ts_status ts_paged_prefill_attn(const void* q, int64_t q_stride, const void* k_pool, const void* v_pool,
                                           const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens,
                                           const int32_t* q_indptr, int32_t T, int32_t B, int32_t H_q, int32_t H_kv,
                                           int32_t D, int32_t page_size, int32_t num_pages, int32_t window,
                                           int32_t sinks, float scale, ts_dtype dtype, void* out, float* lse,
                                           void* workspace, size_t workspace_bytes, void* stream) {
  using namespace ts;
  const char* who = "ts_paged_prefill_attn";
  if (T < 0 || T > (1 << 30) || B < 0 || H_q <= 0 || H_kv <= 0 || D <= 0 || page_size <= 0 || num_pages <= 0 ||
      bt_stride <= 0 || static_cast<long long>(num_pages) * page_size > INT32_MAX)
    return fail(TS_ERR_INVALID_ARG, "%s: bad sizes (T=%d B=%d H_q=%d H_kv=%d D=%d ps=%d P=%d bt=%d)", who, T, B, H_q,
                H_kv, D, page_size, num_pages, bt_stride);
  if (H_q % H_kv != 0)
    return fail(TS_ERR_INVALID_ARG, "%s: H_q=%d not a multiple of H_kv=%d", who, H_q, H_kv);
  if (window < 0 || sinks < 0)
    return fail(TS_ERR_INVALID_ARG, "%s: window=%d (0: none, or >= 1 token), sinks=%d (>= 0 tokens)", who, window,
                sinks);
  if (dtype != TS_F32 && dtype != TS_BF16)
    return fail(TS_ERR_INVALID_ARG, "%s: bad dtype %d", who, static_cast<int>(dtype));
  if (!std::isfinite(scale)) return fail(TS_ERR_INVALID_ARG, "%s: scale not finite", who);
  if (q_stride < static_cast<int64_t>(H_q) * D)
    return fail(TS_ERR_INVALID_ARG, "%s: query rows %lld elements apart are narrower than H_q*D", who,
                static_cast<long long>(q_stride));
  const int g = H_q / H_kv;
  if ((D != 64 && D != 128) || g > 64 || H_q > 65535 ||
      (page_size != 8 && page_size != 16 && page_size != 32))
    return fail(TS_ERR_UNSUPPORTED, "%s: D=%d (supported 64, 128), H_q=%d, H_kv=%d (H_q/H_kv up to 64), "
                "page_size=%d (supported 8, 16, 32)", who, D, H_q, H_kv, page_size);
  if (T == 0 || B == 0) return TS_OK;
  if (!q || !k_pool || !v_pool || !block_table || !seq_lens || !q_indptr || !out)
    return fail(TS_ERR_INVALID_ARG, "%s: null pointer", who);
  const int64_t es = dtype == TS_F32 ? 4 : 2;
  for (const void* ptr : {q, k_pool, v_pool, static_cast<const void*>(out)})
    if (reinterpret_cast<uintptr_t>(ptr) % 16 != 0)
      return fail(TS_ERR_INVALID_ARG, "%s: q, pools and out must be 16-byte aligned", who);
  if (q_stride * es % 16 != 0)
    return fail(TS_ERR_UNSUPPORTED, "%s: query rows %lld B apart (a multiple of 16 B is needed)", who,
                static_cast<long long>(q_stride * es));
  const size_t need = ts_paged_prefill_workspace_size(T, B, H_q, H_kv, D);
  if (need == 0) return fail(TS_ERR_CUDA, "%s: cannot query the SM count", who);
  if (!workspace || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % kWorkspaceAlign != 0)
    return fail(TS_ERR_WORKSPACE, "%s: workspace %zu B < %zu B needed, or not 256-byte aligned", who, workspace_bytes,
                need);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t* err_word = static_cast<uint32_t*>(workspace);
  const int ctas = paged_decode_ctas();
  const WsLayout ws = workspace_layout(ctas, slot_rows_of(T, g), D);
  unsigned char* wsb = static_cast<unsigned char*>(workspace);
  float* part_o = reinterpret_cast<float*>(wsb + ws.part_o);
  float* part_lse = reinterpret_cast<float*>(wsb + ws.part_lse);
  if (dtype == TS_F32)
    return launch_prefill_f32(static_cast<const float*>(q), q_stride, static_cast<const float*>(k_pool),
                              static_cast<const float*>(v_pool), block_table, bt_stride, seq_lens, q_indptr, T, B, H_q,
                              H_kv, D, page_size, num_pages, window, sinks, scale, static_cast<float*>(out), lse,
                              err_word, part_o, part_lse, ctas, s);
  PrefillParams prm;
  prm.out = static_cast<__nv_bfloat16*>(out);
  prm.lse = lse;
  prm.block_table = block_table;
  prm.seq_lens = seq_lens;
  prm.q_indptr = q_indptr;
  prm.T = T;
  prm.B = B;
  prm.bt_stride = bt_stride;
  prm.H_q = H_q;
  prm.H_kv = H_kv;
  prm.g = g;
  prm.page_size = page_size;
  prm.num_pages = num_pages;
  prm.window = window;
  prm.sinks = sinks;
  prm.tile_tokens = kBM / g;
  // A whole item's queries, first scores and epilogue take about as long as
  // three of its key tiles (4.3 us against 1.5 at head dim 128): with more of
  // them than CTAs that is what balances the cut (16 ragged prompts: 310 us with
  // one unit, 290 with four; 8 of 300 tokens: 62.3 and 60.9). With fewer, every
  // item is cut and each part has that cost anyway (33 tokens: 15.4 us with one,
  // 15.7 with four; 512 tokens: 26.4 and 26.6). Only whole items' rows count
  // here: the items of short chunks, one tile and bound by their loads, cost
  // little beside their keys (64 chunks of 16 tokens over up to 4,096: 126 us
  // with one unit, 130 with four; 256 of one token over up to 8,192: 791 and 814;
  // 128 of up to 64 over up to 2,048: 162 both).
  const int64_t items = static_cast<int64_t>(H_kv) * T / (2 * prm.tile_tokens);
  prm.item_units = items >= ctas ? 4 : 1;
  // Fewer, larger parts where there are few units: each part costs the merge
  // (one unit, two, four; 33 tokens over 200: 12.0, 14.1, 18.2 us; over 1,000:
  // 16.7, 16.7, 20.0; over 4,000: 26.7, 21.8, 21.8; 64 tokens over 2,000 with two
  // kv heads: 17.7, 16.1, 19.3).
  prm.min_units = 2;
  prm.slot_rows = slot_rows_of(T, g);
  prm.scale_log2 = scale * kLog2eC;
  prm.err_word = err_word;
  prm.split = reinterpret_cast<SplitItem*>(wsb + ws.split);
  prm.part_o = part_o;
  prm.part_lse = part_lse;
  CUtensorMap qmap, kmap, vmap;
  ts_status st = make_map(&qmap, q, D, H_q, D, T, q_stride, g, prm.tile_tokens);
  const uint64_t rows = static_cast<uint64_t>(num_pages) * page_size, width = static_cast<uint64_t>(H_kv) * D;
  if (st == TS_OK) st = make_map(&kmap, k_pool, D, rows, width, H_kv, D, page_size, 1);
  if (st == TS_OK) st = make_map(&vmap, v_pool, D, rows, width, H_kv, D, page_size, 1);
  if (st != TS_OK) return st;
  return D == 64 ? launch<64>(prm, qmap, kmap, vmap, ctas, s) : launch<128>(prm, qmap, kmap, vmap, ctas, s);
}
