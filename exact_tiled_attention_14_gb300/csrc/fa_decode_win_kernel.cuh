// fa_decode_win_kernel.cuh — a few new queries per sequence against its
// key/value cache, on the tensor cores: the last tokens of a sequence under
// a sliding window with sinks, or the tokens of a drafted tree.
//
// For one (batch, key/value head) the G query heads that share the head and
// their Nq tokens are R = G * Nq rows of one problem, O = softmax(Q K^T) V
// with a mask per row, and every key and value of the span that some row
// sees is read once for all of them.  The cache is what the call reads:
// 4 * d bytes a key against 4 * d * R operations, so up to a few hundred
// rows HBM bounds it.  A tile of 128 keys is 64 KB at d = 128 and takes an
// SM 1.5 us at its share of 6.8 TB/s; the products of 128 rows with it take
// 0.3 us and their softmax about 0.5 us, so rows are simply padded to the
// 128 lanes of TMEM and the tile's work hides behind the next tile's load.
//
// Split.  The key tiles of all units (a unit: batch, key/value head, block
// of 128 * kTiles rows) are laid end to end and cut into equal runs, one
// per CTA, so every SM reads the same amount whatever the sequences'
// lengths, which only the device knows.  A unit that lies in one run is
// finished there; of a cut unit each CTA writes the unnormalised output and
// the softmax statistics of its part, and a second kernel adds the parts up
// by the rescale identity ("FlashAttention: The Matrix You Never Have to
// Write Down", section "What it doesn't solve", on splitting the key axis
// and combining partial results) in the order of the runs: no atomics.
//
// Keys.  A unit's keys are the sinks before the window, padded to whole
// boxes of 16, and then the span lo .. hi - 1: tile 0 usually holds both, so
// a few sinks cost one box, not a tile.  Only boxes that hold a needed key
// are loaded.
//
// One CTA: warps 0-3 and 4-7 are two softmax groups, warp 8 issues S = Q K^T,
// warp 9 the TMA loads, warp 10 O += P V.  With up to 128 rows (kTiles = 1)
// the groups take alternate key tiles, each with its own S, P, O and
// statistics, and are merged at the end of the unit; with more (kTiles = 2)
// each group owns a row tile and both take every key tile.
//
// Copies.  A thread works on the lane its warp owns, and one row's 128 scores
// of a tile take a thread about 2000 cycles from S to P: latency at the start
// and end of each unit.  So with few rows the query tile holds kCopies copies
// of them (4 up to 32 rows, 2 up to 64), S comes out once per copy, and copy
// g weighs only keys g * 128 / kCopies ...: its rows of P are zero elsewhere,
// and its O is the part of those keys.  The copies are parts like the groups'
// and are merged with them.  Measured with 4 rows against one copy: one tile
// 7.2 and 7.9 us, 16 caches of 2005 keys (256 units, d = 64) 37.8 and 44.6;
// in a long unit a tile takes 0.73 us instead of 0.68, so that units of more
// than about 40 tiles would gain a little from one copy.
//
// Measured (key tiles of one unit a CTA, 152 CTAs, inputs larger than L2):
// d = 128 1.34 us a tile of 64 KB, 7.4 TB/s with what L2 keeps, up to 128
// rows, and 1.68 at 256 rows (in short runs; a call of 8 caches of 131k keys
// repeated for seconds runs into the power cap, 1670 MHz, and takes 1.97 us a
// tile, 850 us); d = 64 0.73 us a tile of 32 KB (6.8 TB/s), and
// 1.16 at 256 rows.  A unit costs about 2 us more than its tiles and a call
// about 7 us.  Up to 128 rows the loads bound the time; at 256 rows the
// softmax of two row tiles a key tile does, with the two products' chain.
#pragma once

#include <cuda.h>
#include <cstdint>

#include "ptx_sm103.cuh"

namespace fa {

constexpr int kDwThreads = 384;
constexpr int kDwTile = 128;          // keys per tile, rows per row tile
constexpr int kDwBox = 16;            // rows of the small load box
// Rows of the other.  With one row tile 64, in which sink tiles and spans'
// last tiles take fewer copies (16 caches of 2000 keys and 5 sinks, d = 64:
// 41.4 -> 38.9 us); with two, which wait less for copies than for products,
// 128 (8 caches of 131k keys, d = 128: 13 % less time than with 64 in one run).
constexpr int dec_big_box(int tiles) { return tiles == 2 ? 128 : 64; }
constexpr int kDwSWarp = 8, kDwLoadWarp = 9, kDwPvWarp = 10;
constexpr uint32_t kDwSoftmaxRegs = 208, kDwIssueRegs = 88;
static_assert(2 * 128 * kDwSoftmaxRegs + 128 * kDwIssueRegs <= 168 * kDwThreads, "register split");
constexpr float kDwTau = 8.0f;        // lazy-rescale threshold, log2 units
constexpr int kDwMaxTree = 64;        // drafted tokens (bits of a row's mask)
constexpr int kDwMaxTokens = 16;      // new tokens of a window call

enum DwWaitSite : uint32_t {
  kSiteDwQEmpty = 40, kSiteDwKvEmpty = 41, kSiteDwQFull = 42, kSiteDwKvFull = 43,
  kSiteDwPFull = 44, kSiteDwOFree = 45, kSiteDwSFull = 46, kSiteDwSFree = 47, kSiteDwPvDone = 48
};

struct DecWinParams {
  CUtensorMap tm_q;        // [B * Hk, R, d], boxes of 128 / kCopies rows x 64 columns, 128-byte swizzle
  CUtensorMap tm_k;        // [B * Hk, Nk, d], boxes of dec_big_box rows
  CUtensorMap tm_v;
  CUtensorMap tm_k16;      // the same tensors in boxes of 16 rows
  CUtensorMap tm_v16;
  void* o;                 // [B * Hk, R, d]
  float* lse;              // [B * Hk, R]
  float4* part_o;          // [2 * grid, d / 4, slot_rows] unnormalised parts, 4 columns each
                           // ([2 * grid, slot_rows, d / 4] where rows have copies)
  float2* part_ml;         // [2 * grid, slot_rows] (-m in log2 units, l)
  int4* cut;               // [grid] the cut unit that starts in the run: (head, row block,
                           // slot of its first part, run of its last part), run -1: none
  unsigned int* status;
  unsigned long long watchdog_cycles;
  const int* seqlens;      // [B] or NULL: every count is len_all
  const unsigned long long* tree;   // [B, Nq] visible drafted tokens, NULL for a window call
  int len_all;
  int B, Hk, Nq, Nk;
  int R;                   // rows of a unit's head: G * Nq, row g * Nq + i
  int row_span;            // rows of a unit: 128 * kTiles
  int row_blocks;          // units per head: ceil(R / row_span)
  int slot_rows;
  int combine_rows;        // log2 of a combine block's rows
  int grid;
  int win;                 // >= 1; larger than every position: no window
  int sinks;
  float scale_log2;
};

// Keys of batch b: count len (window: keys with the new tokens, tree:
// history), the span lo .. hi - 1, the sinks before it and the rows they
// take in the list (whole boxes).
struct DecSpan {
  int len, lo, hi, sink, sink_rows;
};
__host__ __device__ __forceinline__ DecSpan dec_span(int count, int Nk, int Nq, int win, int sinks,
                                                     bool tree) {
  DecSpan s;
  s.len = count < 0 ? 0 : (count > Nk ? Nk : count);
  if (tree) {
    s.hi = s.len + Nq < Nk ? s.len + Nq : Nk;
    s.lo = s.len - win;              // a row that marks no drafted token sits at len - 1
  } else {
    s.hi = s.len;
    s.lo = s.len - Nq - win + 1;     // the first token's window
  }
  if (s.lo < 0) s.lo = 0;
  s.sink = sinks < s.lo ? sinks : s.lo;
  s.sink_rows = (s.sink + kDwBox - 1) / kDwBox * kDwBox;
  return s;
}
// Key tiles of a unit: at least one, so that every unit has a writer.
__host__ __device__ __forceinline__ int dec_tiles(const DecSpan& s) {
  const int rows = s.sink_rows + (s.hi - s.lo);
  return rows <= kDwTile ? 1 : (rows + kDwTile - 1) / kDwTile;
}
// Tile t of the list: ns rows of sinks from key sink0 on, then the span from
// key key0 on, nw of whose rows are keys.
struct DecTile {
  int ns, sink0, key0, nw;
};
__host__ __device__ __forceinline__ DecTile dec_tile(const DecSpan& s, int t) {
  DecTile d;
  d.sink0 = t * kDwTile;
  const int left = s.sink_rows - d.sink0;
  d.ns = left < 0 ? 0 : (left > kDwTile ? kDwTile : left);
  d.key0 = s.lo + d.sink0 + d.ns - s.sink_rows;
  const int nw = s.hi - d.key0;
  d.nw = nw < 0 ? 0 : (nw > kDwTile - d.ns ? kDwTile - d.ns : nw);
  return d;
}

// Tiles [from, to) that hold 128 span keys from max(lo, first) to min(hi,
// last) and no sinks before the span: tile t's keys start at base + 128 t.
struct DecRange {
  int from, to, base;
};
__host__ __device__ __forceinline__ DecRange dec_plain(const DecSpan& s, int first, int last) {
  DecRange r;
  r.base = s.lo - s.sink_rows;
  const int skip = first - r.base > s.sink_rows ? first - r.base : s.sink_rows;
  const int end = last < s.hi ? last : s.hi;
  r.from = (skip + kDwTile - 1) / kDwTile;
  r.to = end <= r.base ? 0 : (end - r.base) / kDwTile;
  return r;
}

__device__ __forceinline__ DecSpan dec_span_of(const DecWinParams& p, int b) {
  return dec_span(p.seqlens ? p.seqlens[b] : p.len_all, p.Nk, p.Nq, p.win, p.sinks,
                  p.tree != nullptr);
}

// The deal of `total` key tiles to `grid` CTAs: the first `extra` runs have
// per + 1 tiles, the others per; with fewer tiles than CTAs the CTAs past the
// last tile have none (total < 2^31, see the host's check).
struct DecDeal {
  int per, extra, runs;
};
__host__ __device__ __forceinline__ DecDeal dec_deal(int total, int grid) {
  DecDeal d;
  d.runs = total < grid ? total : grid;
  d.per = total / d.runs;
  d.extra = total - d.per * d.runs;
  return d;
}
__host__ __device__ __forceinline__ int dec_run_start(const DecDeal& d, int run) {
  return run * d.per + (run < d.extra ? run : d.extra);
}
__host__ __device__ __forceinline__ int dec_run_of(const DecDeal& d, int tile) {
  const int longer = d.extra * (d.per + 1);
  return tile < longer ? tile / (d.per + 1) : d.extra + (tile - longer) / d.per;
}
// Key tiles of batches [0, n) and of all batches, by one warp.
__device__ __forceinline__ void dec_tile_sums(const DecWinParams& p, int n, int& before,
                                              int& total) {
  const int units = p.Hk * p.row_blocks;
  int bsum = 0, tsum = 0;
  if (p.seqlens == nullptr) {   // all batches alike
    const int t = dec_tiles(dec_span_of(p, 0)) * units;
    before = n * t;
    total = p.B * t;
    return;
  }
  for (int b = threadIdx.x & 31; b < p.B; b += 32) {
    const int t = dec_tiles(dec_span_of(p, b)) * units;
    tsum += t;
    if (b < n) bsum += t;
  }
  before = __reduce_add_sync(0xffffffffu, bsum);
  total = __reduce_add_sync(0xffffffffu, tsum);
}

// A CTA's place in its run: batch, unit within the batch, tile within the
// unit, tiles left.
struct DecCursor {
  int b, unit, tile, left;
  int n_done;          // pieces taken so far
};
struct DecPiece {
  int b, unit, t0, n;  // tiles t0 .. t0 + n - 1 of the unit
  bool whole;
  int slot;            // where a part goes: 0 the run's first piece, 1 its last
  DecSpan s;
};
__device__ __forceinline__ bool dec_next(const DecWinParams& p, DecCursor& c, DecPiece& pc) {
  if (c.left <= 0) return false;
  pc.b = c.b;
  pc.unit = c.unit;
  pc.t0 = c.tile;
  pc.s = dec_span_of(p, c.b);
  const int nt = dec_tiles(pc.s);
  pc.n = nt - c.tile < c.left ? nt - c.tile : c.left;
  pc.whole = c.tile == 0 && pc.n == nt;
  pc.slot = c.n_done == 0 ? 0 : 1;
  c.left -= pc.n;
  ++c.n_done;
  c.tile = 0;
  if (++c.unit == p.Hk * p.row_blocks) {
    c.unit = 0;
    ++c.b;
  }
  return true;
}

// Columns 4 c .. 4 c + 3 of row r of a part: next to each other for the rows of
// a warp that holds a row a lane, which so writes 512 bytes at a time, and
// row by row where neighbouring threads hold a row's columns (copies).
template <int D>
__device__ __forceinline__ float4* dec_part(const DecWinParams& p, size_t slot, int r, int c) {
  const bool by_row = p.slot_rows <= kDwTile / 2;
  return p.part_o + slot * (D / 4) * p.slot_rows + (by_row ? r * (D / 4) + c : c * p.slot_rows + r);
}

// Where P is.  S of the two groups fills TMEM columns 0-255, their O the
// columns from 256 on.  At d = 64 there is room behind O for P (16 bit, 64
// columns a group).  At d = 128 TMEM is full: with one row tile P goes over
// the S it was formed from, and the group's next S waits for the product that
// reads P (the loads bound these calls, not that chain); with two row tiles
// P goes to shared memory, which costs two ring stages but lets the next S
// be formed during the softmax (measured for 256 rows: 1.80 us a tile against
// 2.07 with P over S, the chain of softmax and both products; 1.68 since the
// issuing warps keep their descriptors in uniform registers).
//
// Shared memory: query tiles (two buffers, so a unit's queries load while the
// previous unit runs; one at d = 128 with two row tiles, where there is no
// room), a ring of K and V tiles, and P where it is there.
template <int D, int kTiles>
struct DwLayout {
  static constexpr int kChunks = D / 64;
  static constexpr int kTile = kDwTile * D * 2;
  static constexpr int kChunkBytes = kDwTile * 128;
  static constexpr int kPTile = kDwTile * kDwTile * 2;
  static constexpr bool kSmemP = D == 128 && kTiles == 2;
  static constexpr bool kOwnP = D == 64 || kSmemP;     // P is not over S
  static constexpr int kQBufs = (D == 128 && kTiles == 2) ? 1 : 2;
  static constexpr int kStages = (D == 128) ? (kSmemP ? 3 : 5) : (kTiles == 2 ? 10 : 12);
  static constexpr int kQ = 0;
  static constexpr int kKV = kQ + kQBufs * kTiles * kTile;
  static constexpr int kP = kKV + kStages * kTile;
  static constexpr int kBar = kP + (kSmemP ? 2 * kPTile : 0);
  // K and V uses of a ring slot have a full barrier each: a wait by parity is
  // only sound where the waiting thread waits for every phase, and the S warp
  // waits for K tiles, the P V warp for V tiles.
  static constexpr int bQFull = 0, bQEmpty = kQBufs, bKFull = 2 * kQBufs,
                       bVFull = bKFull + kStages, bKvEmpty = bVFull + kStages,
                       bSFull = bKvEmpty + kStages,
                       bSFree = bSFull + 2, bPFull = bSFree + 2, bPvDone = bPFull + 2,
                       bOFree = bPvDone + 2, bFinalS = bOFree + 2, bFinalPv = bFinalS + 1,
                       kNumBars = bFinalPv + 1;
  static constexpr int kMisc = kBar + 8 * kNumBars;   // tmem base, abort flag, cursor, deal
  static constexpr int kBytes = kMisc + 48;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kAlloc <= 232448, "shared memory budget");
  static constexpr uint32_t s_col(int w) { return 128u * w; }
  static constexpr uint32_t o_col(int w) { return 256u + static_cast<uint32_t>(D) * w; }
  static constexpr uint32_t p_col(int w) { return kOwnP ? 256u + 2u * D + 64u * w : 128u * w; }
};

// Place in the ring: slot and the parity of its current use.
template <int kStages>
struct DwRing {
  uint32_t slot = 0, parity = 0;
  __device__ __forceinline__ void step(uint32_t n = 1) {
    slot += n;
    if (slot >= kStages) {
      slot -= kStages;
      parity ^= 1u;
    }
  }
};

// What one row sees: its position and, of a tree, the drafted tokens.
struct DecRow {
  int pos;
  unsigned long long bits;
};
__host__ __device__ __forceinline__ int dec_popc(unsigned long long x) {
#ifdef __CUDA_ARCH__
  return __popcll(x);
#else
  return __builtin_popcountll(x);
#endif
}
// Token i of a batch with count len (rows: its tree, NULL for a window call).
__host__ __device__ __forceinline__ DecRow dec_row(const unsigned long long* rows, int i, int Nq,
                                                   int len, int win, int sinks) {
  DecRow r;
  r.bits = 0;
  if (rows == nullptr) {
    r.pos = len - Nq + i;
    return r;
  }
  const unsigned long long used = Nq == 64 ? ~0ull : (1ull << Nq) - 1ull;   // later bits: nothing
  r.bits = rows[i] & used;
  r.pos = len + dec_popc(r.bits) - 1;
  if (win <= kDwMaxTree) {   // positions lie up to 64 apart (a row of 0, one of 64 marks)
    // drop drafted tokens that lie before the row's window and are no sinks
    unsigned long long in = 0;
    for (int j = 0; j < Nq; ++j) {
      const int pj = len + dec_popc(rows[j] & used) - 1;
      if (pj > r.pos - win || pj < sinks) in |= 1ull << j;
    }
    r.bits &= in;
  }
  return r;
}
// Tiles whose 128 columns a row sees whole: from its window on, up to its
// position (of a tree: up to the history's end).
__host__ __device__ __forceinline__ DecRange dec_whole(const DecSpan& s, const DecRow& r, bool tree,
                                                       int win) {
  return dec_plain(s, r.pos - win + 1, tree ? s.len : r.pos + 1);
}
// Visible columns 32 q .. 32 q + 31 of tile tl for a row, as bits.
// seen: keys of the span part up to the row's position (tree: its history).
__host__ __device__ __forceinline__ uint32_t dec_visible(const DecSpan& s, const DecTile& tl,
                                                         const DecRow& r, bool tree, int win,
                                                         int sinks, int q) {
  const int c = 32 * q;
  const int upto = (tree ? s.len : r.pos + 1) - tl.key0;
  const int seen = tl.nw < upto ? tl.nw : upto;
  const int first = r.pos - win + 1 - tl.key0;
  const int ns = s.sink - tl.sink0 < tl.ns ? s.sink - tl.sink0 : tl.ns;
  const int sk = sinks - tl.key0 < seen ? sinks - tl.key0 : seen;
  uint32_t vis = ptx::bit_range(-c, ns - c) |                              // sinks before the span
                 ptx::bit_range(tl.ns + (first > 0 ? first : 0) - c, tl.ns + seen - c) |   // window
                 ptx::bit_range(tl.ns - c, tl.ns + sk - c);                // sinks in the span
  if (tree) {
    // drafted token 0 sits at column ns + len - key0
    const long long at = static_cast<long long>(tl.ns) + s.len - tl.key0 - c;
    uint32_t dv = 0;
    if (at > -64 && at <= 0) dv = static_cast<uint32_t>(r.bits >> -at);
    if (at > 0 && at < 32) dv = static_cast<uint32_t>(r.bits) << at;
    vis |= dv & ptx::bit_range(tl.ns - c, tl.ns + tl.nw - c);
  }
  return vis;
}

template <int D, bool kBf16, int kTiles, int kCopies>
__global__ void __launch_bounds__(kDwThreads, 1)
    fa_decode_win_kernel(const __grid_constant__ DecWinParams p) {
  using L = DwLayout<D, kTiles>;
  constexpr int kRows = kDwTile / kCopies;     // rows of a copy
  static_assert(kTiles == 1 || kCopies == 1, "copies of one row tile");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = ptx::smem_u32(smem_raw);
  const uint32_t sbase = (raw_base + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - raw_base);
  const int warp = ptx::warp_same(threadIdx.x >> 5), lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return sbase + L::kBar + 8u * i; };
  uint32_t* tmem_base_ptr = reinterpret_cast<uint32_t*>(sgen + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sgen + L::kMisc + 4);
  // batch, unit, tile, tiles left, and the deal's per, extra, runs
  int* cursor_s = reinterpret_cast<int*>(sgen + L::kMisc + 8);

  // the combine kernel may be scheduled once every CTA has started (it waits
  // for this grid to complete before reading the parts)
  ptx::griddep_launch_dependents();
  if (warp == kDwSWarp) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_base_ptr), 512);
    ptx::tmem_relinquish();
  }
  if (threadIdx.x == kDwLoadWarp * 32) {
    *abort_flag = 0;
    for (int i = 0; i < L::kQBufs; ++i) {
      ptx::mbar_init(bar(L::bQFull + i), 1);
      // the last S has read the buffer, and (kTiles == 1) every softmax
      // thread is done with it as the scratch of the unit's merge
      ptx::mbar_init(bar(L::bQEmpty + i), kTiles == 1 ? 257 : 1);
    }
    for (int s = 0; s < L::kStages; ++s) {
      ptx::mbar_init(bar(L::bKFull + s), 1);
      ptx::mbar_init(bar(L::bVFull + s), 1);
      ptx::mbar_init(bar(L::bKvEmpty + s), 1);
    }
    for (int w = 0; w < 2; ++w) {
      ptx::mbar_init(bar(L::bSFull + w), 1);
      ptx::mbar_init(bar(L::bSFree + w), 128);
      ptx::mbar_init(bar(L::bPFull + w), 128);
      ptx::mbar_init(bar(L::bPvDone + w), 1);
      ptx::mbar_init(bar(L::bOFree + w), kTiles == 1 ? 256 : 128);
    }
    ptx::mbar_init(bar(L::bFinalS), 1);
    ptx::mbar_init(bar(L::bFinalPv), 1);
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
    ptx::prefetch_tmap(&p.tm_q);
    ptx::prefetch_tmap(&p.tm_k);
    ptx::prefetch_tmap(&p.tm_v);
    ptx::prefetch_tmap(&p.tm_k16);
    ptx::prefetch_tmap(&p.tm_v16);
  }
  if (warp == kDwPvWarp) {
    // this CTA's run and the batch, unit and tile that it starts in
    const int units = p.Hk * p.row_blocks;
    int before, total;
    dec_tile_sums(p, 0, before, total);
    const DecDeal deal = dec_deal(total, p.grid);
    const int run = blockIdx.x;
    const int start = dec_run_start(deal, run);
    const int left = run < deal.runs ? dec_run_start(deal, run + 1) - start : 0;
    if (left > 0) {
      if (p.seqlens == nullptr) {
        const int nt = dec_tiles(dec_span_of(p, 0));
        const int unit = start / nt;
        if (lane == 0) {
          cursor_s[0] = unit / units;
          cursor_s[1] = unit % units;
          cursor_s[2] = start - unit * nt;
        }
      } else {
        int base = 0;
        for (int b0 = 0; base <= start; b0 += 32) {
          const int b = b0 + lane;
          const int nt = b < p.B ? dec_tiles(dec_span_of(p, b)) : 0;
          const int mine = nt * units;
          int incl = mine;
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += up;
          }
          const int first = base + incl - mine;
          if (first <= start && start < first + mine) {
            cursor_s[0] = b;
            cursor_s[1] = (start - first) / nt;
            cursor_s[2] = (start - first) % nt;
          }
          base += __shfl_sync(0xffffffffu, incl, 31);
        }
      }
    }
    if (lane == 0) {
      cursor_s[3] = left;
      cursor_s[4] = deal.per;
      cursor_s[5] = deal.extra;
      cursor_s[6] = deal.runs;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_base_ptr;
  const ptx::Watchdog wd{p.watchdog_cycles, abort_flag, p.status};
  DecCursor cu{cursor_s[0], cursor_s[1], cursor_s[2], cursor_s[3], 0};
  DecPiece pc;
  // rows of row tile w of a piece (kTiles == 1: both groups share tile 0)
  auto rows_of = [&](const DecPiece& x, int w) {
    const int first = (kTiles * (x.unit % p.row_blocks) + (kTiles == 2 ? w : 0)) * kDwTile;
    return min(max(p.R - first, 0), kDwTile);
  };

  if (warp >= 8) {
    ptx::setmaxnreg_dec<kDwIssueRegs>();
    if (warp == kDwLoadWarp) {
      // ============================================================ TMA producer
      if (lane == 0) {
        uint32_t loads = 0, pieces = 0;
        uint32_t k_odd = 0, v_odd = 0, k_used = 0, v_used = 0;   // per slot, as in the waits below
        DwRing<L::kStages> ring;
        bool alive = true;
        while (alive && dec_next(p, cu, pc)) {
          const int head = pc.b * p.Hk + pc.unit / p.row_blocks;
          const DecRange plain = dec_plain(pc.s, 0, pc.s.hi);
          auto load_kv = [&](bool v, int j) {
            const uint32_t slot = ring.slot;
            if (loads >= (uint32_t)L::kStages)   // the slot's previous use is over
              alive = alive && ptx::wait_bounded(bar(L::bKvEmpty + slot), ring.parity ^ 1u, wd,
                                                 kSiteDwKvEmpty);
            if (!alive) return;
            const uint32_t dst = sbase + L::kKV + slot * L::kTile, full = bar((v ? L::bVFull : L::bKFull) + slot);
            (v ? v_odd : k_odd) ^= 1u << slot;
            (v ? v_used : k_used) |= 1u << slot;
            constexpr int kBig = dec_big_box(kTiles);
            const CUtensorMap* big = v ? &p.tm_v : &p.tm_k;
            if (pc.t0 + j >= plain.from && pc.t0 + j < plain.to) {   // 128 rows of the cache
              ptx::mbar_arrive_expect_tx(full, L::kTile);
#pragma unroll
              for (int c = 0; c < L::kChunks; ++c)
#pragma unroll
                for (int i = 0; i < kDwTile; i += kBig)
                  ptx::tma_load_3d(dst + c * L::kChunkBytes + i * 128, big, full, c * 64,
                                   plain.base + (pc.t0 + j) * kDwTile + i, head);
            } else {
              const DecTile t = dec_tile(pc.s, pc.t0 + j);
              // boxes of 16 rows; a tile without keys still loads one box,
              // whose rows are masked
              const int bs = t.ns / kDwBox;
              const int bw = max((t.nw + kDwBox - 1) / kDwBox, bs == 0 ? 1 : 0);
              const CUtensorMap* tm = v ? &p.tm_v16 : &p.tm_k16;
              ptx::mbar_arrive_expect_tx(full, (bs + bw) * kDwBox * 128 * L::kChunks);
              for (int c = 0; c < L::kChunks; ++c) {
                for (int i = 0; i < bs; ++i)
                  ptx::tma_load_3d(dst + c * L::kChunkBytes + i * kDwBox * 128, tm, full, c * 64,
                                   t.sink0 + i * kDwBox, head);
                for (int i = 0; i < bw;) {
                  const bool wide = bw - i >= kBig / kDwBox;
                  ptx::tma_load_3d(dst + c * L::kChunkBytes + (bs + i) * kDwBox * 128,
                                   wide ? big : tm, full, c * 64, t.key0 + i * kDwBox, head);
                  i += wide ? kBig / kDwBox : 1;
                }
              }
            }
            ++loads;
            ring.step();
          };
          load_kv(false, 0);
          const uint32_t qb = pieces % L::kQBufs, quse = pieces / L::kQBufs;
          if (quse > 0)
            alive = alive && ptx::wait_bounded(bar(L::bQEmpty + qb), (quse - 1) & 1, wd,
                                               kSiteDwQEmpty);
          if (!alive) break;
          {
            // the rows of each row tile, or every copy of them
            const int nq = kTiles == 2 ? (rows_of(pc, 1) > 0 ? 2 : 1) : kCopies;
            const int row0 = kTiles * (pc.unit % p.row_blocks) * kDwTile;
            const uint32_t dst = sbase + L::kQ + qb * kTiles * L::kTile;
            ptx::mbar_arrive_expect_tx(bar(L::bQFull + qb),
                                       kTiles == 2 ? nq * L::kTile : L::kTile);
            for (int w = 0; w < nq; ++w)
              for (int c = 0; c < L::kChunks; ++c)
                ptx::tma_load_3d(dst + (kTiles == 2 ? w * L::kTile : w * kRows * 128) +
                                     c * L::kChunkBytes,
                                 &p.tm_q, bar(L::bQFull + qb), c * 64,
                                 kTiles == 2 ? row0 + w * kDwTile : row0, head);
            ++pieces;
          }
          for (int j = 0; alive && j < pc.n; ++j) {
            if (j + 1 < pc.n) load_kv(false, j + 1);
            load_kv(true, j);
          }
        }
        // Drain: every issued copy has landed before the CTA can exit.
        const unsigned long long drain = 200000000ull;
        for (int s = 0; s < L::kStages; ++s) {
          if ((k_used >> s) & 1u)
            ptx::wait_drain(bar(L::bKFull + s), ((k_odd >> s) & 1u) ^ 1u, drain);
          if ((v_used >> s) & 1u)
            ptx::wait_drain(bar(L::bVFull + s), ((v_odd >> s) & 1u) ^ 1u, drain);
        }
        for (uint32_t i = pieces > (uint32_t)L::kQBufs ? pieces - L::kQBufs : 0; i < pieces; ++i)
          ptx::wait_drain(bar(L::bQFull + i % L::kQBufs), (i / L::kQBufs) & 1, drain);
      }
      __syncwarp();
    } else if (warp == kDwSWarp) {
      // ============================================================ S = Q K^T
      // The whole warp walks the tiles and one elected lane issues: conditions,
      // descriptors and addresses then stay in uniform registers (64 rows of
      // 8 caches of 131k keys, d = 128: 8 % less time than with lane 0 walking
      // alone, in one run).
      {
        const uint32_t tmem = ptx::warp_same(tmem_base);
        constexpr uint32_t idesc = ptx::idesc_f16(kDwTile, kDwTile, kBf16 ? 1 : 0, 0);
        const uint32_t q_lo = ptx::desc_lo(sbase + L::kQ, 16);
        const uint32_t k_lo = ptx::desc_lo(sbase + L::kKV, 16);
        // K tiles sit at ring positions 0, 1, 3, 5, ... of a piece's 2 n
        DwRing<L::kStages> ring;
        uint32_t pieces = 0, sc[2] = {0, 0}, odd = 0;
        bool alive = true, issued = false;
        while (ptx::warp_all(dec_next(p, cu, pc))) {
          const uint32_t qb = pieces % L::kQBufs;
          alive = ptx::warp_all(alive && ptx::wait_bounded(bar(L::bQFull + qb),
                                                           (pieces / L::kQBufs) & 1, wd,
                                                           kSiteDwQFull));
          const bool second = kTiles == 2 && ptx::warp_all(rows_of(pc, 1) > 0);
          const int n = ptx::warp_same(pc.n);
          for (int j = 0; j < n; ++j) {
            const uint32_t slot = ring.slot;
            alive = ptx::warp_all(alive && ptx::wait_bounded(bar(L::bKFull + slot),
                                                             (odd >> slot) & 1u, wd,
                                                             kSiteDwKvFull));
            odd ^= 1u << slot;   // per slot: parity of its K tiles so far
            ring.step(j == 0 ? (n == 1 ? 2 : 1) : (j + 1 == n ? 3 : 2));
            ptx::tc_fence_after();
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              if (kTiles == 1 ? (j & 1) != w : w == 1 && !second) continue;
              if (sc[w] > 0)   // the softmax has read this group's previous S (over
                               // which, at d = 128, P was written and must be read too)
                alive = ptx::warp_all(
                    alive && ptx::wait_bounded(bar((L::kOwnP ? L::bSFree : L::bPvDone) + w),
                                               (sc[w] - 1) & 1, wd, kSiteDwSFree));
              ++sc[w];
              ptx::tc_fence_after();
              if (!alive) continue;
              issued = true;
              if (!ptx::elect_one()) continue;
              const uint32_t a = q_lo + (qb * kTiles + (kTiles == 2 ? w : 0)) * (L::kTile >> 4);
              const uint32_t b = k_lo + slot * (L::kTile >> 4);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off =
                    static_cast<uint32_t>((kk >> 2) * L::kChunkBytes + (kk & 3) * 32) >> 4;
                ptx::mma_ss(tmem + L::s_col(w), ptx::desc_sw128(a + off), ptx::desc_sw128(b + off),
                            idesc, kk > 0);
              }
              ptx::mma_commit(bar(L::bSFull + w));
            }
            if (alive && ptx::elect_one()) {
              ptx::mma_commit(bar(L::bKvEmpty + slot));
              if (j + 1 == n) ptx::mma_commit(bar(L::bQEmpty + qb));
            }
          }
          ++pieces;
        }
        if (issued) {
          if (ptx::elect_one()) ptx::mma_commit(bar(L::bFinalS));
          ptx::wait_drain(bar(L::bFinalS), 0, 200000000ull);
        }
      }
      __syncwarp();
    } else if (warp == kDwPvWarp) {
      // ============================================================ O += P V
      // The whole warp walks the tiles, as above.  Rows of V that are no key
      // some row sees (box padding, past the keys, drafted slots that no row
      // marks) meet weights 0, but 0 times a value that is not finite is not
      // 0, so they are overwritten with zeros.
      const uint32_t tmem = ptx::warp_same(tmem_base);
      constexpr uint32_t idesc = ptx::idesc_f16(kDwTile, D, kBf16 ? 1 : 0, 1);
      const uint32_t v_lo = ptx::desc_lo(sbase + L::kKV, L::kChunkBytes);
      const uint32_t p_lo = ptx::desc_lo(sbase + L::kP, 16);   // where P is in shared memory
      DwRing<L::kStages> ring;
      uint32_t pcn[2] = {0, 0}, units[2] = {0, 0}, odd = 0;
      bool alive = true, issued = false, cut_here = false;
      while (ptx::warp_all(dec_next(p, cu, pc))) {
        // a tree's keys below `from` are before the window of its shallowest
        // token; `holes` are the drafted tokens that no row marks
        int from = 0;
        unsigned long long holes = 0;
        if (p.tree) {
          const unsigned long long* rows = p.tree + static_cast<size_t>(pc.b) * p.Nq;
          const unsigned long long used = p.Nq == 64 ? ~0ull : (1ull << p.Nq) - 1ull;
          const unsigned long long r0 = lane < p.Nq ? rows[lane] & used : 0ull;
          const unsigned long long r1 = lane + 32 < p.Nq ? rows[lane + 32] & used : 0ull;
          const int depth = min(lane < p.Nq ? dec_popc(r0) : 64, lane + 32 < p.Nq ? dec_popc(r1) : 64);
          from = pc.s.len + __reduce_min_sync(0xffffffffu, depth) - p.win;
          const unsigned long long any = r0 | r1;
          const uint32_t lo = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(any));
          const uint32_t hi = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(any >> 32));
          holes = used & ~((static_cast<unsigned long long>(hi) << 32) | lo);
        }
        const int lead = min(from, pc.s.len);          // keys before every window end here
        const DecRange plain = dec_plain(pc.s, lead, holes ? pc.s.len : pc.s.hi);
        const bool second = kTiles == 2 && ptx::warp_all(rows_of(pc, 1) > 0);
        const int n = ptx::warp_same(pc.n);
        const int keep0 = ptx::warp_same(plain.from - pc.t0), keep1 = ptx::warp_same(plain.to - pc.t0);
        // tile j's product for the groups that take it
        auto wait_v = [&](uint32_t slot) {
          alive = ptx::warp_all(alive && ptx::wait_bounded(bar(L::bVFull + slot),
                                                           (odd >> slot) & 1u, wd, kSiteDwKvFull));
          odd ^= 1u << slot;   // per slot: parity of its V tiles so far
        };
        auto issue = [&](int j, uint32_t slot) {
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            if (kTiles == 1 ? (j & 1) != w : w == 1 && !second) continue;
            const bool first = kTiles == 1 ? j == w : j == 0;
            if (first && units[w] > 0)   // the previous unit's O has been read
              alive = ptx::warp_all(alive && ptx::wait_bounded(bar(L::bOFree + w),
                                                               (units[w] - 1) & 1, wd,
                                                               kSiteDwOFree));
            alive = ptx::warp_all(alive && ptx::wait_bounded(bar(L::bPFull + w), pcn[w] & 1, wd,
                                                             kSiteDwPFull));
            ++pcn[w];
            ptx::tc_fence_after();
            if (alive) issued = true;
            if (alive && ptx::elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kDwTile / 16; ++kk) {
                const uint64_t vd =
                    ptx::desc_sw128(v_lo + slot * (L::kTile >> 4) + kk * (2048 >> 4));
                const uint32_t acc = (kk > 0 || !first) ? 1u : 0u;
                if constexpr (L::kSmemP) {   // K-major, 64 keys to a chunk
                  const uint32_t off = (kk >> 2) * L::kChunkBytes + (kk & 3) * 32;
                  ptx::mma_ss(tmem + L::o_col(w),
                              ptx::desc_sw128(p_lo + ((w * L::kPTile + off) >> 4)), vd, idesc, acc);
                } else {
                  ptx::mma_ts(tmem + L::o_col(w), tmem + L::p_col(w) + kk * 8, vd, idesc,
                              acc);
                }
              }
              ptx::mma_commit(bar(L::bPvDone + w));
            }
          }
          if (alive && ptx::elect_one()) ptx::mma_commit(bar(L::bKvEmpty + slot));
        };
        // V tiles sit at ring positions 2, 4, ..., 2 n - 2 and 2 n - 1 of the
        // piece's 2 n.  Tiles with rows to clear: sinks' padding, past the keys,
        // before every window, drafted slots.
        for (int j = 0; j < n; ++j) {
          ring.step(j + 1 < n ? 2 : 1);
          wait_v(ring.slot);
          if (j < keep0 || j >= keep1) {
            const DecTile t = dec_tile(pc.s, pc.t0 + j);
            auto clear = [&](int r0, int r1) {
              for (int c = 0; c < L::kChunks; ++c) {
                uint4* rows = reinterpret_cast<uint4*>(sgen + L::kKV + ring.slot * L::kTile +
                                                       c * L::kChunkBytes);
                for (int i = r0 * 8 + lane; i < r1 * 8; i += 32) rows[i] = make_uint4(0, 0, 0, 0);
              }
            };
            clear(min(max(pc.s.sink - t.sink0, 0), t.ns), t.ns);
            clear(t.ns + t.nw, kDwTile);
            clear(t.ns + max(p.sinks - t.key0, 0), t.ns + min(lead - t.key0, t.nw));
            if (holes)
              for (int i = max(pc.s.len - t.key0, 0); i < t.nw; ++i)
                if (holes >> (t.key0 + i - pc.s.len) & 1) clear(t.ns + i, t.ns + i + 1);
            ptx::fence_proxy_async_smem();
            __syncwarp();
          }
          issue(j, ring.slot);
        }
        ring.step();
        // kTiles == 1: both groups read both outputs, and arrive for a group
        // that had no tile too
        ++units[0];
        units[1] += kTiles == 1 || second;
        // a unit that starts here and ends in a later run: its parts' place
        if (pc.t0 == 0 && !pc.whole && lane == 0) {
          const DecDeal deal{cursor_s[4], cursor_s[5], cursor_s[6]};
          const int end_tile = dec_run_start(deal, blockIdx.x + 1) - pc.n + dec_tiles(pc.s) - 1;
          p.cut[blockIdx.x] = make_int4(pc.b * p.Hk + pc.unit / p.row_blocks,
                                        pc.unit % p.row_blocks, 2 * blockIdx.x + pc.slot,
                                        dec_run_of(deal, end_tile));
          cut_here = true;
        }
      }
      if (lane == 0 && !cut_here) p.cut[blockIdx.x] = make_int4(0, 0, 0, -1);
      if (issued) {
        if (ptx::elect_one()) ptx::mma_commit(bar(L::bFinalPv));
        ptx::wait_drain(bar(L::bFinalPv), 0, 200000000ull);
      }
      __syncwarp();
    }
  } else {
    ptx::setmaxnreg_inc<kDwSoftmaxRegs>();
    // ============================================================ softmax
    constexpr int kCols = kDwTile / kCopies;     // key columns of a thread
    const int w = warp >> 2, t = threadIdx.x & 127;
    const int seg = t / kRows, r = t % kRows;    // copy (and its keys), row of the row tile
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem_base + lane_off + L::s_col(w) + seg * kCols;
    const uint32_t tP = tmem_base + lane_off + L::p_col(w);
    const uint32_t tO = tmem_base + lane_off + L::o_col(w);
    const float c = p.scale_log2;
    constexpr uint32_t kZero[16] = {};
    if constexpr (kCopies > 1 && L::kOwnP) {     // P outside the copy's keys stays zero
#pragma unroll
      for (int k = 0; k < 4; ++k) ptx::tmem_st16(tP + 16 * k, kZero);
      ptx::tmem_wait_st();
    }
    uint32_t scnt = 0, pieces = 0;
    while (dec_next(p, cu, pc)) {
      const int nrows = rows_of(pc, w);
      const uint32_t qb = pieces++ % L::kQBufs;
      if (kTiles == 2 && nrows == 0) continue;
      const bool has = (kCopies > 1 ? (warp & 3) * 32 % kRows : (warp & 3) * 32) < nrows;
      const int row = (kTiles * (pc.unit % p.row_blocks) + (kTiles == 2 ? w : 0)) * kDwTile + r;
      // what the row sees: most tiles whole, the others column by column
      auto my_row = [&]() {
        return dec_row(p.tree ? p.tree + static_cast<size_t>(pc.b) * p.Nq : nullptr,
                       min(row, p.R - 1) % p.Nq, p.Nq, pc.s.len, p.win, p.sinks);
      };
      const DecRange whole = dec_whole(pc.s, my_row(), p.tree != nullptr, p.win);
      float m_ref = -INFINITY, neg_m = 0.f, l = 0.f;
      int it = 0;                                // tiles of this group so far
      for (int j = 0; j < pc.n; ++j) {
        if (kTiles == 1 && (j & 1) != w) continue;
        // P_w and O_w are in use until the group's previous product is done
        // (at d = 128 this S could only come after it)
        auto wait_pv = [&]() {
          if (L::kOwnP && it > 0) {
            ptx::wait_bounded(bar(L::bPvDone + w), (scnt - 2) & 1, wd, kSiteDwPvDone);
            __syncwarp();
            ptx::tc_fence_after();
          }
        };
        if (!has) {   // a warp without rows only keeps the order
          ptx::wait_bounded(bar(L::bSFull + w), scnt & 1, wd, kSiteDwSFull);
          ++scnt;
          if (L::kOwnP) ptx::mbar_arrive(bar(L::bSFree + w));
          wait_pv();
        } else {
          ptx::wait_bounded(bar(L::bSFull + w), scnt & 1, wd, kSiteDwSFull);
          ++scnt;
          __syncwarp();
          ptx::tc_fence_after();
          if (__any_sync(0xffffffffu, pc.t0 + j < whole.from || pc.t0 + j >= whole.to)) {
            const DecTile tl = dec_tile(pc.s, pc.t0 + j);
            const DecRow me = my_row();
            ptx::tmem_mask_scores(tS, kCols / 32, [&](int q) {
              return dec_visible(pc.s, tl, me, p.tree != nullptr, p.win, p.sinks,
                                 seg * (kCols / 32) + q);
            });
          }
          uint32_t sr[kCols];
#pragma unroll
          for (int q4 = 0; q4 < kCols / 32; ++q4) ptx::tmem_ld32(tS + q4 * 32, sr + q4 * 32);
          ptx::tmem_wait_ld();
          float sv[kCols];
#pragma unroll
          for (int e = 0; e < kCols; ++e) sv[e] = __uint_as_float(sr[e]);
          if (L::kOwnP) {
            ptx::tc_fence_before();
            ptx::mbar_arrive(bar(L::bSFree + w));       // S_w may be overwritten now
          }
          float a0 = -INFINITY, a1 = -INFINITY, a2 = -INFINITY, a3 = -INFINITY;
#pragma unroll
          for (int e = 0; e < kCols; e += 8) {
            a0 = ptx::max3(a0, sv[e + 0], sv[e + 1]);
            a1 = ptx::max3(a1, sv[e + 2], sv[e + 3]);
            a2 = ptx::max3(a2, sv[e + 4], sv[e + 5]);
            a3 = ptx::max3(a3, sv[e + 6], sv[e + 7]);
          }
          const float mx = fmaxf(fmaxf(a0, a1), fmaxf(a2, a3));
          // lazy rescale, as in the prompt kernel: the reference moves only
          // when a tile exceeds it by 2^kDwTau
          const bool grow = (mx - m_ref) * c > kDwTau;
          float alpha = 1.f;
          if (grow) {
            const float nm = -mx * c;
            alpha = (m_ref == -INFINITY) ? 0.f : ptx::ex2(nm - neg_m);
            l *= alpha;
            m_ref = mx;
            neg_m = nm;
          }
          const bool rescale = it > 0 && __any_sync(0xffffffffu, grow);
          const uint64_t c2 = ptx::f2_pack(c, c), nm2 = ptx::f2_pack(neg_m, neg_m);
          uint64_t acc0 = ptx::f2_pack(0.f, 0.f), acc1 = acc0;
          uint32_t pk[kCols / 2];
#pragma unroll
          for (int e = 0; e < kCols / 2; e += 2) {
            float x0, x1, x2, x3;
            ptx::f2_unpack(ptx::ffma2(ptx::f2_pack(sv[2 * e + 0], sv[2 * e + 1]), c2, nm2), x0, x1);
            ptx::f2_unpack(ptx::ffma2(ptx::f2_pack(sv[2 * e + 2], sv[2 * e + 3]), c2, nm2), x2, x3);
            const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1), p2 = ptx::ex2(x2), p3 = ptx::ex2(x3);
            acc0 = ptx::fadd2(acc0, ptx::f2_pack(p0, p1));
            acc1 = ptx::fadd2(acc1, ptx::f2_pack(p2, p3));
            // weights to 16 bits, the operand type of the tensor core; their
            // sum l stays fp32
            pk[e] = ptx::pack2<kBf16>(p0, p1);
            pk[e + 1] = ptx::pack2<kBf16>(p2, p3);
          }
          {
            float s0, s1, s2, s3;
            ptx::f2_unpack(acc0, s0, s1);
            ptx::f2_unpack(acc1, s2, s3);
            l += (s0 + s1) + (s2 + s3);
          }
          wait_pv();
          if (rescale) {
#pragma unroll 1
            for (int q4 = 0; q4 < D / 32; ++q4) {
              uint32_t orr[32];
              ptx::tmem_ld32(tO + q4 * 32, orr);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e)
                orr[e] = __float_as_uint(__uint_as_float(orr[e]) * alpha);
              ptx::tmem_st32(tO + q4 * 32, orr);
            }
          }
          if constexpr (L::kSmemP) {
            uint8_t* prow = sgen + L::kP + w * L::kPTile + t * 128;   // 128-byte swizzle
#pragma unroll
            for (int k = 0; k < kDwTile / 8; ++k)
              *reinterpret_cast<uint4*>(prow + (k >> 3) * L::kChunkBytes +
                                        (((k & 7) ^ (t & 7)) << 4)) =
                  make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
            ptx::fence_proxy_async_smem();
          } else if constexpr (kCopies == 1) {
            ptx::tmem_st32(tP, pk);
            ptx::tmem_st32(tP + 32, pk + 32);
          } else {
            // this copy's keys; the others' columns hold zeros (at d = 128
            // the scores of this lane, until they are overwritten here)
#pragma unroll
            for (int k = 0; k < kCopies; ++k) {
              if (k == seg) {   // the same for the whole warp
                if constexpr (kCopies == 2) {
                  ptx::tmem_st32(tP + 32 * k, pk);
                } else {
                  ptx::tmem_st16(tP + 16 * k, pk);
                }
              } else if (!L::kOwnP) {
#pragma unroll
                for (int i = 0; i < 4 / kCopies; ++i)
                  ptx::tmem_st16(tP + (64 / kCopies) * k + 16 * i, kZero);
              }
            }
          }
          ptx::tmem_wait_st();
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(bar(L::bPFull + w));
        ++it;
      }
      // ---- end of the piece: the group's last product
      if (it > 0) {
        ptx::wait_bounded(bar(L::bPvDone + w), (scnt - 1) & 1, wd, kSiteDwPvDone);
        __syncwarp();
      }
      ptx::tc_fence_after();
      const size_t head = static_cast<size_t>(pc.b) * p.Hk + pc.unit / p.row_blocks;
      const size_t slot = 2ull * blockIdx.x + pc.slot;
      if constexpr (kTiles == 1) {
        // Merge the parts of a row, two groups times kCopies, to their largest
        // maximum.  The statistics go through the unit's query buffer, which
        // S no longer reads; group w then handles half w of the columns of
        // both groups' O (both groups' warps reach the same TMEM lanes).
        // A part takes no part only where its sum is exactly 0 (nothing seen):
        // a sum of NaN, from a key that is not finite, makes the row NaN.
        uint8_t* scratch = sgen + L::kQ + qb * L::kTile;
        float2* ml_s = reinterpret_cast<float2*>(scratch);
        ptx::named_bar_sync(1, 256);             // both groups have their last S
        ml_s[w * kDwTile + t] = make_float2(neg_m, l);
        ptx::tc_fence_before();
        ptx::named_bar_sync(1, 256);
        ptx::tc_fence_after();
        float nm = INFINITY, lt = 0.f;
#pragma unroll
        for (int g = 0; g < 2 * kCopies; ++g) {
          const float2 x = ml_s[g * kRows + r];
          if (x.y != 0.f) nm = fminf(nm, x.x);
        }
#pragma unroll
        for (int g = 0; g < 2 * kCopies; ++g) {
          const float2 x = ml_s[g * kRows + r];
          if (x.y != 0.f) lt = fmaf(ptx::ex2(nm - x.x), x.y, lt);
        }
        // this lane's parts
        const float2 y0 = ml_s[t], y1 = ml_s[kDwTile + t];
        // (a finished unit's are divided by l here)
        const float inv = pc.whole && lt != 0.f ? 1.0f / lt : 1.f;
        const bool live0 = y0.y != 0.f, live1 = y1.y != 0.f;
        const float f0 = ptx::ex2(nm - y0.x) * inv, f1 = ptx::ex2(nm - y1.x) * inv;
        const size_t out_row = head * p.R + row;
        const bool two = pc.n > 1;               // the second group had a tile
        // 16 columns of this lane, both groups' parts added
        auto load16 = [&](int col, float* x) {
          uint32_t a[16];
          ptx::tmem_ld16(tmem_base + lane_off + L::o_col(0) + col, a);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = live0 ? __uint_as_float(a[e]) * f0 : 0.f;
          if (two) {
            ptx::tmem_ld16(tmem_base + lane_off + L::o_col(1) + col, a);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e)
              x[e] = live1 ? fmaf(__uint_as_float(a[e]), f1, x[e]) : x[e];
          }
        };
        if (r < nrows && seg == 0 && w == 0) {
          if (pc.whole)
            p.lse[out_row] = lt != 0.f ? (ptx::lg2(lt) - nm) * 0.693147180559945309f : -INFINITY;
          else
            p.part_ml[slot * p.slot_rows + r] = make_float2(lt != 0.f ? nm : 0.f, lt);
        }
        if constexpr (kCopies == 1) {
          if (has) {
#pragma unroll 1
            for (int col = w * (D / 2); col < (w + 1) * (D / 2); col += 16) {
              float x[16];
              load16(col, x);
              if (r < nrows) {
                if (pc.whole) {
                  uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + out_row * D + col);
#pragma unroll
                  for (int v = 0; v < 2; ++v)
                    dst[v] = make_uint4(ptx::pack2<kBf16>(x[8 * v], x[8 * v + 1]),
                                        ptx::pack2<kBf16>(x[8 * v + 2], x[8 * v + 3]),
                                        ptx::pack2<kBf16>(x[8 * v + 4], x[8 * v + 5]),
                                        ptx::pack2<kBf16>(x[8 * v + 6], x[8 * v + 7]));
                } else {
#pragma unroll
                  for (int v = 0; v < 4; ++v)
                    *dec_part<D>(p, slot, r, col / 4 + v) =
                        make_float4(x[4 * v], x[4 * v + 1], x[4 * v + 2], x[4 * v + 3]);
                }
              }
            }
          }
        } else {
          // The copies' rows meet in the scratch, D / 2 columns at a time
          // (D / 4 of each group's half): [lane][D / 2] floats, 16-byte pieces
          // permuted by the lane so that lanes a row apart use other banks.
          // Then every thread adds the copies of a few pieces and writes them.
          constexpr int kPieces = D / 8;         // 16-byte pieces of a lane's row
          float4* sc4 = reinterpret_cast<float4*>(scratch);
#pragma unroll 1
          for (int pass = 0; pass < 2; ++pass) {
            ptx::named_bar_sync(1, 256);         // the scratch's last use is over
            if (has) {
#pragma unroll
              for (int q = 0; q < D / 64; ++q) {
                float x[16];
                load16(w * (D / 2) + pass * (D / 4) + q * 16, x);
                if (r < nrows) {
#pragma unroll
                  for (int v = 0; v < 4; ++v)
                    sc4[t * kPieces + ((w * (kPieces / 2) + q * 4 + v) ^ (t & 7))] =
                        make_float4(x[4 * v], x[4 * v + 1], x[4 * v + 2], x[4 * v + 3]);
                }
              }
            }
            ptx::named_bar_sync(1, 256);
            for (int i = threadIdx.x; i < nrows * kPieces; i += 256) {
              const int rr = i / kPieces, v = i % kPieces;
              float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int g = 0; g < kCopies; ++g) {
                const int ln = g * kRows + rr;
                const float4 x = sc4[ln * kPieces + (v ^ (ln & 7))];
                sum.x += x.x; sum.y += x.y; sum.z += x.z; sum.w += x.w;
              }
              const int half = v / (kPieces / 2);
              const int col = half * (D / 2) + pass * (D / 4) + (v % (kPieces / 2)) * 4;
              if (pc.whole) {
                uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) +
                                                      (head * p.R + rr) * D + col);
                *dst = make_uint2(ptx::pack2<kBf16>(sum.x, sum.y), ptx::pack2<kBf16>(sum.z, sum.w));
              } else {
                *dec_part<D>(p, slot, rr, col / 4) = sum;
              }
            }
          }
        }
        ptx::fence_proxy_async_smem();           // the next queries may be loaded over the scratch
        ptx::tc_fence_before();
        ptx::mbar_arrive(bar(L::bQEmpty + qb));
        ptx::mbar_arrive(bar(L::bOFree + 0));
        ptx::mbar_arrive(bar(L::bOFree + 1));
      } else {
        const size_t out_row = head * p.R + row;
        const float inv = l != 0.f ? 1.0f / l : 0.f;
        if (has) {
#pragma unroll 1
          for (int col = 0; col < D; col += 32) {
            uint32_t a[32];
            ptx::tmem_ld32(tO + col, a);
            ptx::tmem_wait_ld();
            float x[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = l != 0.f ? __uint_as_float(a[e]) : 0.f;
            if (r < nrows) {
              if (pc.whole) {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + out_row * D + col);
#pragma unroll
                for (int v = 0; v < 4; ++v)
                  dst[v] = make_uint4(ptx::pack2<kBf16>(x[8 * v] * inv, x[8 * v + 1] * inv),
                                      ptx::pack2<kBf16>(x[8 * v + 2] * inv, x[8 * v + 3] * inv),
                                      ptx::pack2<kBf16>(x[8 * v + 4] * inv, x[8 * v + 5] * inv),
                                      ptx::pack2<kBf16>(x[8 * v + 6] * inv, x[8 * v + 7] * inv));
              } else {
#pragma unroll
                for (int v = 0; v < 8; ++v)
                  *dec_part<D>(p, slot, w * kDwTile + r, col / 4 + v) =
                      make_float4(x[4 * v], x[4 * v + 1], x[4 * v + 2], x[4 * v + 3]);
              }
            }
          }
          if (r < nrows) {
            if (pc.whole)
              p.lse[out_row] = l != 0.f ? (ptx::lg2(l) - neg_m) * 0.693147180559945309f : -INFINITY;
            else
              p.part_ml[slot * p.slot_rows + w * kDwTile + r] = make_float2(neg_m, l);
          }
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(bar(L::bOFree + w));
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kDwSWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, 512);
  }
}

// The cut units: block (run, y) adds up the parts of rows of the unit that
// starts in that run and ends in a later one (most runs have one, the run
// table says which), 4 columns a thread: every part is scaled to the largest
// maximum, added in the order of the runs, and the sum divided once.  A row
// without a visible key has no live part (all sums are 0; a sum of NaN is live):
// O = 0 and LSE = -inf.  A block takes 2^combine_rows rows (up to 32) and as
// many columns as its threads reach; four neighbours share a row, so that a
// warp reads 128 bytes of each of four columns' parts and writes 32 of each
// row.  kBatch parts are loaded together.
constexpr int kDwCombineThreads = 128;
template <int D, bool kBf16, int kBatch>
__global__ void __launch_bounds__(kDwCombineThreads)
    fa_decode_win_combine_kernel(const __grid_constant__ DecWinParams p) {
  constexpr int kPer = D / 4;
  const int lr = p.combine_rows, pieces = kDwCombineThreads >> lr;
  const int groups = max(kPer / pieces, 1);      // blocks that share rows
  const int srow = ((threadIdx.x >> 2) & ((1 << lr) - 1)) + (blockIdx.y / groups << lr);
  const int c = (threadIdx.x & 3) + (threadIdx.x >> (2 + lr)) * 4 + blockIdx.y % groups * pieces;
  ptx::griddep_wait();   // the parts are complete, and this grid ends after the main one
  const int run0 = blockIdx.x;
  const int4 cut = p.cut[run0];
  if (cut.w < 0) return;
  const int row = cut.y * p.row_span + srow;
  if (srow >= p.slot_rows || row >= p.R || c >= kPer) return;
  // the unit's first part is the last piece of its run, the others are the
  // first of theirs
  auto slot_of = [&](int run) { return static_cast<size_t>(run == run0 ? cut.z : 2 * run); };
  const float4* const part = dec_part<D>(p, 0, srow, c);
  const size_t part_step = static_cast<size_t>(D / 4) * p.slot_rows;
  float nm = INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int run = run0; run <= cut.w; run += kBatch) {
    // a batch of parts, their loads in flight together
    float2 ml[kBatch];
    float4 x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (run + i <= cut.w) {
        const size_t slot = slot_of(run + i);
        ml[i] = p.part_ml[slot * p.slot_rows + srow];
        x[i] = part[slot * part_step];
      } else {
        ml[i] = make_float2(0.f, 0.f);
      }
    }
    float m = nm;
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (ml[i].y != 0.f) m = fminf(m, ml[i].x);
    const float fo = nm == INFINITY ? 0.f : ptx::ex2(m - nm);
    acc = make_float4(acc.x * fo, acc.y * fo, acc.z * fo, acc.w * fo);
    l *= fo;
    nm = m;
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (ml[i].y != 0.f) {
        const float f = ptx::ex2(m - ml[i].x);
        acc.x = fmaf(f, x[i].x, acc.x);
        acc.y = fmaf(f, x[i].y, acc.y);
        acc.z = fmaf(f, x[i].z, acc.z);
        acc.w = fmaf(f, x[i].w, acc.w);
        l = fmaf(f, ml[i].y, l);
      }
  }
  const size_t out = static_cast<size_t>(cut.x) * p.R + row;
  const float inv = l != 0.f ? 1.0f / l : 0.f;
  reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + out * D)[c] =
      make_uint2(ptx::pack2<kBf16>(acc.x * inv, acc.y * inv),
                 ptx::pack2<kBf16>(acc.z * inv, acc.w * inv));
  if (c == 0) p.lse[out] = l != 0.f ? (ptx::lg2(l) - nm) * 0.693147180559945309f : -INFINITY;
}

}  // namespace fa
