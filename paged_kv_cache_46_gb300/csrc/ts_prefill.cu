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
// (in order of sequence, kv head, token block; one extra unit per item for its
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
// where it is the A operand of O += P V. Products of one thread complete in
// order, so S(j + 1) of a tile may follow its P V(j) without a wait, and the
// two tiles take turns: while one tile's softmax runs, the tensor pipe works
// on the other. The running maximum moves only when a score exceeds it by more
// than 2^8 (a row's weights stay below that), so O in TMEM is rescaled rarely.
// P is rounded to bf16 because the product's operands share one type; O is
// divided by the sum of the rounded weights, the LSE takes the exact sum.
#include <cmath>
#include <cstdlib>

#include "ts_tcgen05.cuh"

namespace ts {
namespace {

constexpr int kBM = 128;  // query rows per tile
constexpr int kBN = 128;  // keys per tile
constexpr int kThreads = 384;
constexpr int kAtom = kBN * 128;  // one [128 rows x 64 bf16] SW128 atom
constexpr int kItemUnits = 1;     // units an item counts beyond its key tiles
constexpr int kBadRing = 16;      // key tiles whose bad-page mask is kept
constexpr float kLog2eC = 1.4426950408889634f;
constexpr float kLn2C = 0.6931471805599453f;
constexpr float kSlack = 8.0f;
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
  static constexpr int kOffBad = kOffBar + 320;
  static constexpr int kOffPieces = kOffBad + kBadRing * 4;
  static constexpr int kOffMisc = kOffPieces + 4 * 48;
  static constexpr int kSmem = kOffMisc + 128 + 12 * 8;
  // TMEM columns of tile t: S at 128 t, O at 256 + D t. P (64 columns) goes over
  // the front of S at D = 128, where all 512 columns are taken, and has its own
  // place at D = 64: the next S product then need not wait for P V.
  static constexpr uint32_t kTmemO = 256;
  static constexpr bool kOwnP = D == 64;
  static constexpr uint32_t kTmemP = kOwnP ? 256 + 2 * D : 0, kTmemPStep = kOwnP ? 64 : 128;
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
  int32_t min_units;    // units a CTA takes at least, while there are any
  int32_t slot_rows;    // rows of a partial state: 128 or 256
  float scale_log2;
  uint32_t* err_word;
  SplitItem* split;  // [CTAs]
  float* part_o;     // [2 * CTAs, slot_rows, D]
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

__device__ __forceinline__ Item load_item(const PrefillParams& p, const Seq& s, int block) {
  Item it;
  it.j0 = block * 2 * p.tile_tokens;
  it.tokens = min(s.n - it.j0, 2 * p.tile_tokens);
  it.p0 = s.L - s.n + it.j0;
  // keys past the block table's row do not exist
  const long long cap = static_cast<long long>(p.bt_stride) * p.page_size;
  const int end = it.p0 + it.tokens;
  it.khi = static_cast<int>(min(static_cast<long long>(max(end, 0)), cap));
  it.klo = (p.window > 0 && it.p0 >= p.window) ? it.p0 - p.window + 1 : 0;
  if (it.klo <= p.sinks) it.klo = 0;  // the window meets the first tokens
  it.w0 = it.klo / kBN;
  it.ns = it.klo > 0 ? min((p.sinks + kBN - 1) / kBN, it.w0) : 0;
  it.nt = it.ns + max(0, (it.khi + kBN - 1) / kBN - it.w0);
  return it;
}

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
  int left;              // units of the range still to walk
  int b, h, block, rem;  // the next unit: item, and unit within it
  Seq s;
  bool first;  // no piece returned yet

  __device__ __forceinline__ void init(const PrefillParams& p, const int* start) {
    left = start[4];
    b = start[0];
    h = start[1];
    block = start[2];
    rem = start[3];
    first = true;
    if (left > 0) s = load_seq(p, b);
  }
  // The next piece; also whether the item goes on in later CTAs from its first
  // key tile here (then `rest` is the number of its key tiles there).
  __device__ __forceinline__ bool next(const PrefillParams& p, int k, Piece& q, int& rest) {
    while (left > 0) {
      const Item it = load_item(p, s, block);
      const int cost = it.nt + kItemUnits;
      const int here = min(cost - rem, left);
      const bool owner = rem == 0;
      const int t0 = max(0, rem - kItemUnits), t1 = max(t0, rem + here - kItemUnits);
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
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  auto b_full = [&](int s) { return smem_u32(&bars[s]); };
  auto b_empty = [&](int s) { return smem_u32(&bars[kRing + s]); };
  auto b_sfull = [&](int t) { return smem_u32(&bars[2 * kRing + t]); };
  auto b_pfull = [&](int t, int half) { return smem_u32(&bars[2 * kRing + 18 + 2 * t + half]); };
  auto b_sfree = [&](int t) { return smem_u32(&bars[2 * kRing + 2 + t]); };
  auto b_pvdone = [&](int t) { return smem_u32(&bars[2 * kRing + 4 + t]); };
  auto b_ofree = [&](int t) { return smem_u32(&bars[2 * kRing + 6 + t]); };
  const uint32_t b_qfull = smem_u32(&bars[2 * kRing + 8]), b_qempty = smem_u32(&bars[2 * kRing + 9]);
  auto b_piece = [&](int s) { return smem_u32(&bars[2 * kRing + 10 + s]); };
  auto b_taken = [&](int s) { return smem_u32(&bars[2 * kRing + 10 + kPieces + s]); };
  static_assert(kPieces == 4 && (2 * kRing + 22) * 8 <= 320, "mbarriers fit their slot");
  static_assert(kPieces * sizeof(Piece) == L::kOffMisc - L::kOffPieces, "piece ring");
  Piece* ring = reinterpret_cast<Piece*>(smem + L::kOffPieces);
  volatile uint32_t* bad_ring = reinterpret_cast<volatile uint32_t*>(smem + L::kOffBad);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  int* start = reinterpret_cast<int*>(smem + L::kOffMisc + 16);
  long long* cut = reinterpret_cast<long long*>(smem + L::kOffMisc + 64);  // the batch's cut: range end, q, r
  long long* warp_tot = reinterpret_cast<long long*>(smem + L::kOffMisc + 128);

  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(b_full(i), 1);
      mbar_init(b_empty(i), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(b_sfull(t), 2);  // the products' commit and the issuer's own arrival
      mbar_init(b_pfull(t, 0), 4);
      mbar_init(b_pfull(t, 1), 4);
      mbar_init(b_sfree(t), 4);
      mbar_init(b_pvdone(t), 1);
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
  if (warp == 0) tmem_alloc(smem_u32(tmem_slot), 512);

  // ---- prologue: this CTA's range of units --------------------------------
  const int chunk = (p.B + kThreads - 1) / kThreads;
  const int lo = min(p.B, tid * chunk), hi = min(p.B, lo + chunk);
  auto seq_cost = [&](const Seq& s) {  // of one kv head
    long long c = 0;
    for (int i = 0; i < s.blocks; ++i) c += load_item(p, s, i).nt + kItemUnits;
    return c;
  };
  long long mine = 0;
  for (int b = lo; b < hi; ++b) mine += seq_cost(load_seq(p, b)) * p.H_kv;
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
  const long long G = max(1ll, min(static_cast<long long>(gridDim.x), total / p.min_units));
  const long long q_units = total / G, r_units = total % G;
  const long long u0 = k < G ? k * q_units + min(static_cast<long long>(k), r_units) : total;
  const long long u1 = k < G ? u0 + q_units + (k < r_units ? 1 : 0) : total;
  if (tid == 0) {
    start[4] = static_cast<int>(u1 - u0);
    cut[0] = u1;
    cut[1] = q_units;
    cut[2] = r_units;
  }
  if (u0 < u1 && excl <= u0 && u0 < excl + mine) {
    long long off = excl;
    for (int b = lo; b < hi; ++b) {
      const Seq s = load_seq(p, b);
      const long long c = seq_cost(s);
      if (u0 < off + c * p.H_kv) {
        int rem_h = static_cast<int>((u0 - off) / c);
        long long rem = (u0 - off) - rem_h * c;
        int i = 0;
        while (true) {
          const int ci = load_item(p, s, i).nt + kItemUnits;
          if (rem < ci) break;
          rem -= ci;
          ++i;
        }
        start[0] = b;
        start[1] = rem_h;
        start[2] = i;
        start[3] = static_cast<int>(rem);
        break;
      }
      off += c * p.H_kv;
    }
  }
  __syncthreads();
  constexpr uint32_t tmem = 0;  // all 512 columns: there is no other place for them
  const uint32_t sQ = smem_u32(smem + L::kOffQ), sKV = smem_u32(smem + L::kOffKV);
  pdl_wait_primary();

  const int tt = p.tile_tokens;
  bool ok = true;
  // A reader waits for piece n (all its threads that use it), copies what it
  // needs, and hands the entry back once per warp.
  auto piece_ready = [&](uint32_t n) { return mbar_wait(b_piece(n % kPieces), (n / kPieces) & 1); };
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 11) {
      // ---------------- pieces ------------------------------------------------
      if (lane == 0) {
        Walk w;
        w.init(p, start);
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
            const long long qu = cut[1], r = cut[2], big = r * (qu + 1), last = cut[0] + rest - 1;
            SplitItem si;
            si.tokens = q.tokens;
            si.head = q.head;
            si.parts = static_cast<int>(last < big ? last / (qu + 1) : r + (last - big) / max(qu, 1ll)) - k + 1;
            si.slot = q.slot;
            si.row0 = q.row0;
            p.split[k] = si;
          }
        }
      }
    } else if (warp != 9) {
      // ---------------- K (warp 8) and V (warp 10): lane i holds page i of the key tile
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
      uint32_t seq = 0;     // K tile of the current step in the ring (V: the one after it)
      uint32_t pieces = 0;  // with products
      uint32_t sn0 = 0, sn1 = 0, pn0 = 0, pn1 = 0, used0 = 0, used1 = 0;  // S, P V products, pieces of each tile
      auto landed = [&](uint32_t x) { return mbar_wait(b_full(x % kRing), (x / kRing) & 1); };
      // S of tile t from ring tile x; `last`: no other product reads it, `q_last`: nor the queries
      auto issue_s = [&](int t, uint32_t x, bool last, bool q_last) {
        const uint64_t q = dQ + t * kTileStep, kb = dK + (x % kRing) * kTileStep;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            constexpr uint64_t kAtomStep = kAtom >> 4;
            const uint64_t off = (ks >> 2) * kAtomStep + (ks & 3) * 2;
            mma_bf16(t * 128, q + off, kb + off, iS, ks > 0);
          }
          mma_commit(b_sfull(t));
          // the arrival carries what the key tile's barrier carried here: the
          // softmax reads the tile's bad-page mask after it
          mbar_arrive(b_sfull(t));
          if (last) mma_commit(b_empty(x % kRing));
          if (q_last) mma_commit(b_qempty);
        }
        __syncwarp();
      };
      // half of P V of tile t (64 keys), V in ring tile x; `last` as above
      auto issue_pv = [&](int t, int half, uint32_t x, uint32_t add, bool last) {
        const uint64_t vb = dV + (x % kRing) * kTileStep + half * 512;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < kBN / 32; ++ks)
            mma_bf16_tmem_a(L::kTmemO + t * D, L::kTmemP + t * L::kTmemPStep + half * 32 + ks * 8, vb + ks * 128, iO,
                            ks > 0 ? 1u : add);
          if (half == 1) mma_commit(b_pvdone(t));
          if (last) mma_commit(b_empty(x % kRing));
        }
        __syncwarp();
      };
      // S may be overwritten once the softmax has read it (with P over it: once
      // P V is issued, which it is by then)
      auto s_free = [&](int t, uint32_t sn) { return !L::kOwnP || sn == 0 || mbar_wait(b_sfree(t), (sn - 1) & 1); };
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
        ok = __all_sync(0xffffffffu, mbar_wait(b_qfull, pieces & 1) && landed(seq) && s_free(0, sn0));
        if (!ok) break;
        issue_s(0, seq, !two, !two && nk == 1);
        ++sn0;
        if (two) {
          ok = __all_sync(0xffffffffu, s_free(1, sn1));
          if (!ok) break;
          issue_s(1, seq, true, nk == 1);
          ++sn1;
        }
        for (int i = 0; i < nk; ++i) {
          const bool more = i + 1 < nk, q_last = i + 2 == nk;
          const uint32_t add = i > 0 ? 1u : 0u;
          bool good = landed(seq + 1) && (!more || landed(seq + 2));
          if (i == 0) {  // O of the last piece has been read
            if (used0 > 0) good = good && mbar_wait(b_ofree(0), (used0 - 1) & 1);
            if (two && used1 > 0) good = good && mbar_wait(b_ofree(1), (used1 - 1) & 1);
          }
          if constexpr (L::kOwnP) {
            if (more) {
              ok = __all_sync(0xffffffffu, good && s_free(0, sn0));
              if (!ok) break;
              issue_s(0, seq + 2, !two, !two && q_last);
              ++sn0;
              if (two) {
                good = s_free(1, sn1);
                ok = __all_sync(0xffffffffu, good);
                if (!ok) break;
                issue_s(1, seq + 2, true, q_last);
                ++sn1;
              }
            }
          }
          ok = __all_sync(0xffffffffu, good && mbar_wait(b_pfull(0, 0), pn0 & 1));
          if (!ok) break;
          issue_pv(0, 0, seq + 1, add, false);
          ok = __all_sync(0xffffffffu, mbar_wait(b_pfull(0, 1), pn0 & 1));
          if (!ok) break;
          issue_pv(0, 1, seq + 1, 1u, !two);
          ++pn0;
          if (!L::kOwnP && more) issue_s(0, seq + 2, !two, !two && q_last);
          if (two) {
            ok = __all_sync(0xffffffffu, mbar_wait(b_pfull(1, 0), pn1 & 1));
            if (!ok) break;
            issue_pv(1, 0, seq + 1, add, false);
            ok = __all_sync(0xffffffffu, mbar_wait(b_pfull(1, 1), pn1 & 1));
            if (!ok) break;
            issue_pv(1, 1, seq + 1, 1u, true);
            ++pn1;
            if (!L::kOwnP && more) issue_s(1, seq + 2, true, q_last);
          }
          seq += 2;
        }
        if (!ok) break;
        ++used0;
        if (two) ++used1;
        ++pieces;
      }
      if (!ok && lane == 0) set_device_error(p.err_word, TS_DEVERR_TIMEOUT);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---------------- softmax: one query row per thread -----------------------
    const int t = warp >> 2, r = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + t * 128, tO = tmem + lanes + L::kTmemO + t * D;
    const uint32_t tP = tmem + lanes + L::kTmemP + t * L::kTmemPStep;
    uint32_t steps = 0, tiles = 0;  // P V products of this tile; key tiles of the CTA
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
      const int pos = q.p0 + t * tt + r / p.g;  // this row's token
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < nk; ++i) {
        const int ti = q.t0 + i;
        const int k0 = (ti < q.ns ? ti : q.w0 + ti - q.ns) * kBN;
        ok = __all_sync(0xffffffffu, mbar_wait(b_sfull(t), steps & 1));
        if (!ok) break;
        tc_fence_after();
        float s[kBN];
#pragma unroll
        for (int c = 0; c < kBN; c += 32) tmem_ld32(tS + c, reinterpret_cast<uint32_t*>(s) + c);
        const uint32_t bad = bad_ring[tiles % kBadRing];
        // every row of the tile sees every key: no masks
        const int pfirst = q.p0 + t * tt, plast = pfirst + tt - 1;
        const bool full = k0 + kBN - 1 <= pfirst && k0 + kBN <= q.khi && bad == 0u && p.scale_log2 > 0.f &&
                          (p.window == 0 || k0 > plast - p.window || k0 + kBN <= p.sinks);
        float f = p.scale_log2;  // what the scores are still to be multiplied by
        tmem_wait_ld();
        if constexpr (L::kOwnP) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(b_sfree(t));
        }
        float mx = -INFINITY;
        if (full) {
          float mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
          for (int c = 0; c < kBN; c += 8) {
            mx = fmax3(mx, s[c], s[c + 1]);
            mx1 = fmax3(mx1, s[c + 2], s[c + 3]);
            mx2 = fmax3(mx2, s[c + 4], s[c + 5]);
            mx3 = fmax3(mx3, s[c + 6], s[c + 7]);
          }
          mx = fmaxf(fmaxf(mx, mx1), fmaxf(mx2, mx3)) * f;
        } else {
          const int first = (p.window > 0 && pos >= p.window) ? pos - p.window + 1 - k0 : 0;
          const int end = min(pos + 1, q.khi) - k0, keep = p.sinks - k0;
#pragma unroll
          for (int c0 = 0; c0 < kBN; c0 += 32) {
            uint32_t vis = ones(end - c0) & (~ones(first - c0) | ones(keep - c0));
            if (bad != 0u) {
              for (int c = 0; c < 32; c += p.page_size)
                if ((bad >> ((c0 + c) / p.page_size)) & 1u) vis &= ~(ones(c + p.page_size) & ~ones(c));
            }
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              s[c0 + c] = (vis >> c) & 1u ? s[c0 + c] * f : -INFINITY;
              mx = fmaxf(mx, s[c0 + c]);
            }
          }
          f = 1.f;
        }
        if (i == 0) {
          m = mx;
        } else if (__any_sync(0xffffffffu, mx > m + kSlack)) {
          ok = __all_sync(0xffffffffu, mbar_wait(b_pvdone(t), (steps - 1) & 1));
          if (!ok) break;
          tc_fence_after();
          const float mnew = fmaxf(m, mx);
          const float alpha = m == -INFINITY ? 0.f : fast_exp2(m - mnew);
          m = mnew;
          l *= alpha;
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 16) {
            uint32_t u[16];
            tmem_ld16(tO + c0, u);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 16; ++x) u[x] = __float_as_uint(__uint_as_float(u[x]) * alpha);
            tmem_st16(tO + c0, u);
          }
        }
        // Rows of a loaded page that no row sees (past the sequence's end, in
        // front of the window, behind the first tokens) may hold anything, and
        // 0 * NaN is NaN in the product: zero them once landed. Both tiles'
        // warps do, each before its own product.
        auto cuts_page = [&](int x) { return x > k0 && x < k0 + kBN && (x & (p.page_size - 1)) != 0; };
        if (cuts_page(q.khi) || cuts_page(q.klo) || (q.klo > 0 && cuts_page(p.sinks))) {
          const uint32_t vseq = 2 * tiles + 1;
          ok = __all_sync(0xffffffffu, mbar_wait(b_full(vseq % kRing), (vseq / kRing) & 1));
          if (!ok) break;
          const int key = k0 + r;
          if (!(key < q.khi && (key >= q.klo || key < p.sinks))) {
            unsigned char* v = smem + L::kOffKV + (vseq % kRing) * kTile + r * 128;
#pragma unroll
            for (int a = 0; a < kAtoms; ++a)
#pragma unroll
              for (int c = 0; c < 8; ++c)
                *reinterpret_cast<uint4*>(v + a * kAtom + c * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_async_smem();
        }
        if (L::kOwnP && steps > 0) {  // P V has read the last P
          ok = __all_sync(0xffffffffu, mbar_wait(b_pvdone(t), (steps - 1) & 1));
          if (!ok) break;
          tc_fence_after();
        }
        const float ms = m == -INFINITY ? 0.f : m;
        const float2 f2 = make_float2(f, f), nm = make_float2(-ms, -ms);
        float2 l2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int c0 = 0; c0 < kBN; c0 += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 x = __ffma2_rn(make_float2(s[c0 + c], s[c0 + c + 1]), f2, nm);
            const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
            pk[c / 2] = float2_to_bf16x2(e.x, e.y);
            l2 = __fadd2_rn(l2, e);
          }
          tmem_st16(tP + c0 / 2, pk);
          if (c0 == 32 || c0 == 96) {  // half of P is there: its product may start
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b_pfull(t, c0 / 64));
          }
        }
        l += l2.x + l2.y;
        ++steps;
        ++tiles;
      }
      if (!ok) break;
      // epilogue: O / sum and the LSE (no key: O = 0, LSE = -inf)
      if (nk > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(b_pvdone(t), (steps - 1) & 1));
        if (!ok) break;
        tc_fence_after();
      }
      const float inv = l > 0.f ? 1.0f / l : 0.f;
      const float lse2 = l > 0.f ? m + log2f(l) : -INFINITY;
      const int rt = r / p.g, j = t * tt + rt;  // token of the tile, of the item
      const bool real = rt < tt && j < q.tokens;
      const int slot = q.slot;
      const int64_t row = static_cast<int64_t>(q.row0 + j) * p.H_q + q.head * p.g + r % p.g;
      const int64_t prow = static_cast<int64_t>(slot) * p.slot_rows + t * kBM + r;
      __syncwarp();
      if (lane == 0) mbar_arrive(b_taken(n % kPieces));
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 32) {
        float o[32];
        if (nk > 0) {
          tmem_ld32(tO + c0, reinterpret_cast<uint32_t*>(o));
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = 0.f;
        }
#pragma unroll
        for (int x = 0; x < 32; ++x) o[x] *= inv;
        if (real && slot < 0) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + row * D + c0);
#pragma unroll
          for (int x = 0; x < 32; x += 8)
            dst[x / 8] = make_uint4(float2_to_bf16x2(o[x], o[x + 1]), float2_to_bf16x2(o[x + 2], o[x + 3]),
                                    float2_to_bf16x2(o[x + 4], o[x + 5]), float2_to_bf16x2(o[x + 6], o[x + 7]));
        } else if (real) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + prow * D + c0);
#pragma unroll
          for (int x = 0; x < 32; x += 4) dst[x / 4] = make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
        }
      }
      if (real && slot >= 0) p.part_lse[prow] = lse2 * kLn2C;
      if (real && slot < 0 && p.lse) p.lse[row] = lse2 * kLn2C;
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
// of the item whose first part CTA k holds, a warp one row at a time.
template <int D>
__global__ void __launch_bounds__(256) prefill_merge_kernel(const PrefillParams p) {
  pdl_launch_dependents();
  pdl_wait_primary();
  const int k = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SplitItem si = p.split[k];
  if (si.row0 < 0) return;
  constexpr int kV = D / 32;  // values per lane
  for (int rr = warp; rr < 32; rr += 8) {
    const int r = blockIdx.x * 32 + rr;
    const int rt = (r % kBM) / p.g, j = (r / kBM) * p.tile_tokens + rt;
    if (rt >= p.tile_tokens || j >= si.tokens) continue;
    float mx = -INFINITY;
    for (int i = 0; i < si.parts; ++i) {
      const int slot = i == 0 ? si.slot : 2 * (k + i);
      mx = fmaxf(mx, p.part_lse[static_cast<int64_t>(slot) * p.slot_rows + r]);
    }
    const float ms = mx == -INFINITY ? 0.f : mx;
    float a[kV], sum = 0.f;
#pragma unroll
    for (int x = 0; x < kV; ++x) a[x] = 0.f;
    for (int i = 0; i < si.parts; ++i) {
      const int64_t row = static_cast<int64_t>(i == 0 ? si.slot : 2 * (k + i)) * p.slot_rows + r;
      const float wt = __expf(p.part_lse[row] - ms);
      const float* o = p.part_o + row * D + lane * kV;
      sum += wt;
#pragma unroll
      for (int x = 0; x < kV; ++x) a[x] += wt * o[x];
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const int64_t out = static_cast<int64_t>(si.row0 + j) * p.H_q + si.head * p.g + r % kBM % p.g;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + out * D) + lane * (kV / 2);
#pragma unroll
    for (int x = 0; x < kV; x += 2) dst[x / 2] = float2_to_bf16x2(a[x] * inv, a[x + 1] * inv);
    if (lane == 0 && p.lse) p.lse[out] = sum > 0.f ? ms + logf(sum) : -INFINITY;
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
                             float* out, float* lse, uint32_t* err_word, cudaStream_t stream);

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
  if (dtype == TS_F32)
    return launch_prefill_f32(static_cast<const float*>(q), q_stride, static_cast<const float*>(k_pool),
                              static_cast<const float*>(v_pool), block_table, bt_stride, seq_lens, q_indptr, T, B, H_q,
                              H_kv, D, page_size, num_pages, window, sinks, scale, static_cast<float*>(out), lse,
                              err_word, s);
  const int ctas = paged_decode_ctas();
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
  prm.min_units = 2;
  prm.slot_rows = slot_rows_of(T, g);
  prm.scale_log2 = scale * kLog2eC;
  prm.err_word = err_word;
  const WsLayout ws = workspace_layout(ctas, prm.slot_rows, D);
  unsigned char* wsb = static_cast<unsigned char*>(workspace);
  prm.split = reinterpret_cast<SplitItem*>(wsb + ws.split);
  prm.part_o = reinterpret_cast<float*>(wsb + ws.part_o);
  prm.part_lse = reinterpret_cast<float*>(wsb + ws.part_lse);
  CUtensorMap qmap, kmap, vmap;
  ts_status st = make_map(&qmap, q, D, H_q, D, T, q_stride, g, prm.tile_tokens);
  const uint64_t rows = static_cast<uint64_t>(num_pages) * page_size, width = static_cast<uint64_t>(H_kv) * D;
  if (st == TS_OK) st = make_map(&kmap, k_pool, D, rows, width, H_kv, D, page_size, 1);
  if (st == TS_OK) st = make_map(&vmap, v_pool, D, rows, width, H_kv, D, page_size, 1);
  if (st != TS_OK) return st;
  return D == 64 ? launch<64>(prm, qmap, kmap, vmap, ctas, s) : launch<128>(prm, qmap, kmap, vmap, ctas, s);
}
