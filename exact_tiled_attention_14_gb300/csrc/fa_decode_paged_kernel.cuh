// fa_decode_paged_kernel.cuh — the last tokens of each sequence against its
// pages of 8-bit keys and values (see fa_paged.cuh), under a sliding window
// with sinks or none.
//
// For one (batch, key/value head) the G query heads that share it and their
// Nq tokens are R = G * Nq rows of one problem.  With k_j = ks * a_j and
// v_j = vs * b_j (codes a, b, scales of the key's page),
//     s_rj = scale * ks * (q_r . a_j),   O_r = sum_j softmax_j(s_r) vs b_j.
// Codes are exact in half precision, and so are the queries once each row is
// multiplied by a power of two that brings its largest element to 2^12 (an element
// under 2^-26 of it, 2^-29 of bf16, loses bits): the products
// accumulate exactly what float32 sums of the codes' values do.  K's scale joins
// the scores in float32.  V's scale joins the weights: O is held in units of a power
// of two that follows the scales, and p * vs / unit is rounded to half precision:
// by 2^-11 of a weight, or by 2^-25 units where it is below 2^-14 of them.  A weight
// p is up to 2^8 (its row's reference rises with scores that pass it by more), the
// largest scale up to 2^6 units, and while no scale but 0 is under 2^-4 of the largest
// the smallest step is 2^-27 of a weight of 1 at most.  Once one is, each row
// has a unit of its own (paged_row_unit), so that pages that a row does not see,
// or gives no weight, cost it nothing.  (As a multiply of each page's product before
// it joined the output the scale took a second set of accumulators and a quarter of
// a tile's instructions.  A threshold of 2^6 with 2^8 units, references that rise more
// often, took 64 rows of 8 caches 66 us instead of 63.5.)
//
// Bound.  A key costs 2 d bytes and 4 d R operations: HBM bounds it, an SM's
// share is 23 bytes a cycle.  The codes have to be turned into 16-bit
// registers before any tensor-core product, which is most of the issue slots
// (about 230 instructions for 16 keys of 8 rows at d = 128, which arrive
// every 174 cycles), and mma.sync takes registers as they are.  tcgen05 would
// need them written to shared memory or TMEM first, and its 8-bit kinds would
// need the queries and weights in 8 bits too.  Measured: 64 caches of 16384, 8
// K/V heads, 4 rows, d = 128 (1.34 GB): 213 us for this kernel, 6.3 TB/s of 6.8,
// and 6 for the second; 8 caches of 131072 as int8, 8 rows: 325 to 345 us, 6.2 to
// 6.6 TB/s.  One cache of 8192 takes 14 us against 2.5 of its bytes: two launches
// and the chain of a run's start, two tiles and the parts' sum.
// The tile's loops stay rolled where registers allow it: all of them unrolled were
// 24 KB of code, warps waited 3.3 of 8.4 cycles an instruction for it to arrive,
// and the 219 us above were 298.
//
// Layout.  S^T = K Q^T and O^T += V^T P^T: the 16-row side of m16n8k16 goes
// to keys (head elements for O), the 8-row side to the query rows, since few
// rows are the usual case.  The order of a product's contraction is free, so
// a thread takes 16 bytes of a row at a time (below) without ldmatrix.
//
// Split.  A unit is (batch, K/V head, block of 8 kTiles rows); its keys are
// tiles of kKeys (4 KB of K and of V).  The tiles of all units are laid end to
// end and cut into equal runs, one per warp, whatever the sequences' lengths,
// which only the device knows.  Warps share nothing: each has its ring, which
// its lanes fill by TMA, and its queries, so none ever waits for another.  A
// unit that lies in one run is finished there; of a cut unit each warp leaves
// its part in the workspace, and a second kernel adds the parts up in the order
// of the runs: no atomics.  (Warps of a CTA sharing its tiles, merged at the
// end of each unit, cost 3.6 us a unit: 4096 units of one tile took 98 us.)
#pragma once

#include <cuda.h>
#include <cstdint>

#include "fa_decode_win_kernel.cuh"
#include "fa_paged.cuh"
#include "ptx_sm103.cuh"

namespace fa {

// Warps of a CTA by its row tiles (8 rows each).
__host__ __device__ constexpr int dp_warps(int tiles) { return tiles == 1 ? 12 : 10; }
constexpr int kDpTileBytes = 4096;       // of K, and of V
// A run takes this many tiles at least: a part is 4 KB for each row tile at
// d = 128, a tile 8 KB.
__host__ __device__ constexpr int dp_min_tiles(int tiles) { return tiles + 1; }
constexpr float kDpTau = 8.0f;           // lazy-rescale threshold, log2 units
constexpr uint32_t kSiteDpFull = 50;
__host__ __device__ constexpr int dp_keys(int d) { return kDpTileBytes / d; }

struct DecPagedParams {
  CUtensorMap tm_k;        // [pages * Hk * page, d] bytes, boxes of box_rows rows
  CUtensorMap tm_v;
  const void* q;           // [B * Hk, R, d]
  void* o;                 // [B * Hk, R, d]
  float* lse;              // [B * Hk, R]
  float4* part_o;          // [2 * runs, slot_rows, d / 4] parts, each the mean of its values
  float2* part_ml;         // [2 * runs, slot_rows] (m in log2 units, l)
  int2* cut;               // [units] (slot of the unit's first part, run of its last), (-1, 0): whole
  const float* k_scale;    // [pages, Hk]
  const float* v_scale;
  const int* table;        // [B, per_seq]
  const int* seqlens;      // [B]
  unsigned int* status;
  unsigned long long watchdog_cycles;
  int B, Hk, Nq;
  int R;                   // rows of a head: G * Nq, row g * Nq + i
  int row_blocks;          // units per head
  int slot_rows;           // rows of a unit's part
  int per_seq, pages, page;
  uint32_t page_magic;     // ceil(2^32 / (page / 16)), 0 for pages of 16
  int boxes;               // boxes of a tile, all of one page each: 16 to a tile's keys
  int runs;                // at most
  int grid;
  int win;                 // >= 1; larger than every position: no window
  int sinks;
  float scale_log2;
};

// Keys that the rows of a batch see, as tiles: the sinks' tiles before the
// window's first, then tiles from `first` on.  A batch has one tile at least,
// so that each unit has a writer.
struct PagedSpan {
  int len, lo, sink_tiles, first, tiles;
};
__host__ __device__ __forceinline__ PagedSpan paged_span(int count, int capacity, int Nq, int win,
                                                         int sinks, int keys) {
  PagedSpan s;
  s.len = count < 0 ? 0 : (count > capacity ? capacity : count);
  s.lo = s.len - Nq - win + 1;                  // the first token's window
  if (s.lo < 0) s.lo = 0;
  s.first = s.lo / keys;
  const int st = (sinks < s.lo ? sinks : s.lo) + keys - 1;
  s.sink_tiles = st / keys < s.first ? st / keys : s.first;
  const int last = (s.len + keys - 1) / keys;
  s.tiles = s.sink_tiles + (last > s.first ? last - s.first : 0);
  if (s.tiles < 1) s.tiles = 1;
  return s;
}
// First key of tile t of the list.
__host__ __device__ __forceinline__ int paged_key0(const PagedSpan& s, int t, int keys) {
  return (t < s.sink_tiles ? t : s.first + t - s.sink_tiles) * keys;
}
// Whether some row of a batch, at positions len - Nq .. len - 1, sees some key of
// [key0, key0 + n).
__host__ __device__ __forceinline__ bool paged_seen(const PagedSpan& s, int Nq, int key0, int n,
                                                    int win, int sinks) {
  return key0 < s.len && (key0 + n - 1 > s.len - Nq - win || key0 < sinks);
}
// Whether the row at position pos sees some key of [key0, key0 + n).
__host__ __device__ __forceinline__ bool paged_sees(int key0, int n, int pos, int win, int sinks) {
  return key0 <= pos && (key0 + n - 1 > pos - win || key0 < sinks);
}

// The unit of O is 2^-6 of a power of two that is not below the scales so far: a
// weight of up to 2^8 is at most 2^14 units (2^15 for scales over 2^127).  Once the
// smallest scale but 0 is under 2^-4 of that power (they are apart), each row has
// a unit of its own, by the largest product c of a weight (over 2^8) and its
// scale: it falls as the row's reference rises, instead of O, and rises with c.
constexpr float kDpUnit = 0x1p6f, kDpSpread = 0x1p4f;
__host__ __device__ __forceinline__ bool paged_new_unit(float unit, float top) {
  return top > unit * kDpUnit;
}
__host__ __device__ __forceinline__ bool paged_apart(float unit, float least) {
  return least < unit * (kDpUnit / kDpSpread);
}
__device__ __forceinline__ float paged_unit(float top) {
  const float up = __uint_as_float((__float_as_uint(top) + 0x7fffffu) & 0x7f800000u);
  return fminf(fmaxf(up, kDpUnit * 0x1p-126f), 0x1p127f) / kDpUnit;
}
// 1 / unit, 0 before there is one
__device__ __forceinline__ float paged_per_unit(float unit) {
  return unit > 0.f ? __uint_as_float(0x7f000000u - __float_as_uint(unit)) : 0.f;
}
// A row's next unit, its reference having made O a factor f smaller; returns O's factor.
__device__ __forceinline__ float paged_row_unit(float& unit, float f, float c) {
  const float was = unit * f;
  unit = paged_unit(fmaxf(c, was * kDpUnit));
  return was * paged_per_unit(unit);
}

// Key rows of the 16 of a product.  At d = 128 a row is 128 bytes, its 16-byte
// chunks permuted by its number (128-byte swizzle); at d = 64 two rows share
// 128 bytes (64-byte swizzle).  A quarter warp reads K as two rows of four
// chunks and V as four rows of two chunks; slot order dp_row makes both touch
// all banks once: at d = 64 slots 2 t and 2 t + 1 are rows of different parity,
// and slots 0, 2, 4, 6 (1, 3, 5, 7) differ in parity or in the row's bit 2.
template <int D>
__host__ __device__ constexpr int dp_row(int slot) {
  return D == 128 ? slot
                  : ((slot >> 1 & 1) + (slot >> 2 & 1) * 4) ^ (slot & 1 ? 3 : 0);
}
// Byte offset of 16-byte chunk c of row r.
template <int D>
__host__ __device__ constexpr uint32_t dp_chunk(int r, int c) {
  return D == 128 ? r * 128u + ((c ^ (r & 7)) << 4) : r * 64u + ((c ^ (r >> 1 & 3)) << 4);
}

// Shared memory: the warps' rings, then each warp's queries, weights and scales.
template <int D, int kTiles>
struct DpLayout {
  static_assert(kTiles == 1 || kTiles == 2, "row tiles of 8 rows");
  static constexpr int kRows = 8 * kTiles;
  static constexpr int kWarps = dp_warps(kTiles), kThreads = 32 * kWarps;
  static constexpr int kStages = 2;
  static constexpr int kRing = kStages * 2 * kDpTileBytes;    // of a warp
  static constexpr int kQ = 0;                                // within a warp's own
  static constexpr int kP = kQ + kRows * D * 2;
  static constexpr int kQmul = kP + dp_keys(D) / 16 * kTiles * 256;
  static constexpr int kMeta = kQmul + kRows * 4;             // [stage]: 4 K, 4 V scales
  static constexpr int kBar = kMeta + kStages * 32;
  static constexpr int kOwn = kBar + kStages * 8;
  static constexpr int kMisc = kWarps * (kRing + kOwn);
  static constexpr int kAlloc = kMisc + 16 + 1024;
  static_assert(kOwn % 16 == 0 && kAlloc <= 232448, "shared memory budget");
};

__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* tm, uint32_t bar,
                                              int row) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(0), "r"(row), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// x, its magnitude at most `most` (NaN stays).
__device__ __forceinline__ float dp_cap(float x, float most) {
  float y;
  asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(most));
  return y;
}

// A place in the list of all tiles.
struct DpPlace {
  int b, hk, block, tile;
  PagedSpan s;
};
__device__ __forceinline__ PagedSpan dp_span(const DecPagedParams& p, int b, int keys) {
  return paged_span(p.seqlens[b], p.per_seq * p.page, p.Nq, p.win, p.sinks, keys);
}
// (past the last unit: a place never used)
__device__ __forceinline__ void dp_next_unit(const DecPagedParams& p, DpPlace& x, int keys) {
  x.tile = 0;
  if (++x.block < p.row_blocks) return;
  x.block = 0;
  if (++x.hk < p.Hk) return;
  x.hk = 0;
  if (++x.b < p.B) x.s = dp_span(p, x.b, keys);
}

// Run `run` of the deal of all tiles, at least min_tiles each, to at most `runs`
// runs: its tiles start .. start + left - 1 and its first place; by one warp.
struct DpRun {
  DecDeal deal;
  DpPlace at;
  int start, left;
};
__device__ __forceinline__ DpRun dp_run(const DecPagedParams& p, int keys, int runs, int min_tiles,
                                        int run) {
  const int lane = threadIdx.x & 31, units = p.Hk * p.row_blocks;   // of a batch
  DpRun r{};
  int total = 0;
  for (int b = lane; b < p.B; b += 32) total += dp_span(p, b, keys).tiles * units;
  total = __reduce_add_sync(0xffffffffu, total);
  r.deal = dec_deal(total, min(runs, (total + min_tiles - 1) / min_tiles));
  if (run >= r.deal.runs) return r;
  r.start = dec_run_start(r.deal, run);
  r.left = dec_run_start(r.deal, run + 1) - r.start;
  int before = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int mine = b0 + lane < p.B ? dp_span(p, b0 + lane, keys).tiles * units : 0;
    int upto = mine;
#pragma unroll
    for (int i = 1; i < 32; i *= 2) {
      const int x = __shfl_up_sync(0xffffffffu, upto, i);
      if (lane >= i) upto += x;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, before + upto > r.start);
    if (past != 0) {
      const int k = __ffs(past) - 1;
      r.at.b = b0 + k;
      r.at.s = dp_span(p, r.at.b, keys);
      const int skip = r.start - (before + __shfl_sync(0xffffffffu, upto - mine, k));
      const int unit = skip / r.at.s.tiles;
      r.at.tile = skip - unit * r.at.s.tiles;
      r.at.hk = unit / p.row_blocks;
      r.at.block = unit - r.at.hk * p.row_blocks;
      break;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return r;
}

// Four elements a lane of a query row, times the power of two (returned) that
// brings the row's largest to 2^12; by one warp.
template <bool kBf16>
__device__ __forceinline__ int dp_query_row(const uint2 raw, float* x) {
  ptx::unpack2<kBf16>(raw.x, x[0], x[1]);
  ptx::unpack2<kBf16>(raw.y, x[2], x[3]);
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
  top = __reduce_max_sync(0xffffffffu, top);
  int shift = 0;
  if (top != 0 && top < kInfBits) shift = min(12 - (static_cast<int>(top >> 23) - 127), 120);
  const float mul = __uint_as_float(static_cast<uint32_t>(shift + 127) << 23);
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] *= mul;
  return shift;
}

template <int D, bool kBf16, bool kInt8, int kTiles>
__global__ void __launch_bounds__(32 * dp_warps(kTiles), 1)
    fa_decode_paged_kernel(const __grid_constant__ DecPagedParams p) {
  using L = DpLayout<D, kTiles>;
  constexpr int kKeys = dp_keys(D);          // of a tile
  constexpr int kMt = kKeys / 16;            // products' key blocks of a tile
  constexpr int kJ = D / 16;
  constexpr int kWords = D / 16;             // 4-byte words of a thread's part of a K row
  constexpr int kStages = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = ptx::smem_u32(smem_raw);
  const uint32_t sbase = (raw_base + 1023u) & ~1023u;
  uint8_t* const sgen = smem_raw + (sbase - raw_base);
  const int warp = ptx::warp_same(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(sgen + L::kMisc);
  const ptx::Watchdog wd{p.watchdog_cycles, abort_flag, p.status};
  const uint32_t ring = sbase + warp * L::kRing;
  uint8_t* const ring_gen = sgen + warp * L::kRing;
  const uint32_t own = sbase + L::kWarps * L::kRing + warp * L::kOwn;
  uint8_t* const own_gen = sgen + L::kWarps * L::kRing + warp * L::kOwn;
  uint2* const q_s = reinterpret_cast<uint2*>(own_gen + L::kQ);
  uint2* const p_s = reinterpret_cast<uint2*>(own_gen + L::kP);
  float* const qmul_s = reinterpret_cast<float*>(own_gen + L::kQmul);
  const float* const meta_gen = reinterpret_cast<const float*>(own_gen + L::kMeta);
  auto bar = [&](int stage) -> uint32_t { return own + L::kBar + 8u * stage; };

  ptx::griddep_launch_dependents();
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    ptx::prefetch_tmap(&p.tm_k);
    ptx::prefetch_tmap(&p.tm_v);
  }
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) ptx::mbar_init(bar(i), 1);
    ptx::fence_mbar_init();
  }
  __syncthreads();                           // (the abort flag; the only one)

  // ---- the warp's run and its first place
  const int run = warp * p.grid + blockIdx.x;    // few runs spread over the SMs
  const DpRun rn = dp_run(p, kKeys, p.runs, dp_min_tiles(kTiles), run);
  const DecDeal deal = rn.deal;
  if (run >= deal.runs) return;
  DpPlace at = rn.at;
  int left = rn.left;                        // tiles not begun

  // ---- queries of row tile nt of the unit at `at`, four elements of each row a lane;
  // with one row tile the first unit's are asked for before the loads, behind which
  // they wait (5000 cycles of 33000 where every warp has five tiles)
  uint2 raw[8];
  auto ask = [&](int nt) {
    const int row0 = at.block * L::kRows + nt * 8, rows = min(p.R - row0, 8);
    const size_t first = (static_cast<size_t>(at.b) * p.Hk + at.hk) * p.R + row0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      raw[i] = make_uint2(0, 0);
      if (i < rows && lane * 4 < D)
        raw[i] = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.q) +
                                                 (first + i) * D + lane * 4);
    }
  };
  if (kTiles == 1) ask(0);

  // ---- the warp's loads
  const int box_rows = kKeys / p.boxes;
  DpPlace nx = at;                           // the next tile to load
  int nx_left = left;                        // tiles from it on
  int nx_page = -1, nx_row = 0;              // page of the lane's box, its first row in the page
  uint32_t valid = 0;                        // 4 bits per stage: boxes that name a page
  int loaded = 0, waited = 0;                // tiles asked for, tiles that have arrived
  auto look = [&]() {                        // the page of the lane's box of tile nx
    nx_page = -1;
    if (nx_left > 0 && lane < p.boxes) {
      const int key = paged_key0(nx.s, nx.tile, kKeys) + lane * box_rows;
      const int nth = p.page_magic ? __umulhi(key >> 4, p.page_magic) : key >> 4;
      nx_row = key - nth * p.page;
      if (key < nx.s.len) nx_page = p.table[static_cast<size_t>(nx.b) * p.per_seq + nth];
    }
  };
  auto load = [&](int stage) {               // into the stage; then look at the one after
    if (nx_left > 0) {
      const bool ok = nx_page >= 0 && nx_page < p.pages;
      const uint32_t have = __ballot_sync(0xffffffffu, ok);
      valid = (valid & ~(15u << (4 * stage))) | have << (4 * stage);
      if (lane == 0)
        ptx::mbar_arrive_expect_tx(bar(stage), __popc(have) * 2 * box_rows * D);
      __syncwarp();
      if (ok) {
        const int head = nx_page * p.Hk + nx.hk;
        const int row = head * p.page + nx_row;
        const uint32_t dst = ring + stage * (2 * kDpTileBytes) + lane * box_rows * D;
        tma_load_rows(dst, &p.tm_k, bar(stage), row);
        tma_load_rows(dst + kDpTileBytes, &p.tm_v, bar(stage), row);
        const uint32_t meta = own + L::kMeta + stage * 32 + lane * 4;
        cp_async4(meta, p.k_scale + head);
        cp_async4(meta + 16, p.v_scale + head);
      }
      ++loaded;
      --nx_left;
      if (++nx.tile == nx.s.tiles) dp_next_unit(p, nx, kKeys);
      look();
    }
    cp_async_commit();                       // one group per tile, empty ones too
  };
  look();
  for (int i = 0; i < kStages; ++i) load(i);

  // ---- pieces of units, in the order of the run
  bool alive = true;
  int stage = 0, parity = 0, pieces = 0, done = 0;
  for (; left > 0; dp_next_unit(p, at, kKeys), ++pieces) {
    const int tile0 = at.tile;
    const int n = min(at.s.tiles - tile0, left);
    const bool whole = tile0 == 0 && n == at.s.tiles;
    const size_t head = static_cast<size_t>(at.b) * p.Hk + at.hk;
    const int row0 = at.block * L::kRows, rows = min(p.R - row0, L::kRows);
    const PagedSpan s = at.s;
    left -= n;

    // the queries: row r, elements 4 c .. 4 c + 3 as the B operand's
    // registers of lane (r % 8, 4 c / (D / 4)), in half precision
#pragma unroll 1
    for (int nt = 0; nt < kTiles; ++nt) {
      if (kTiles > 1 || pieces > 0) ask(nt);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float x[4];
        const int shift = dp_query_row<kBf16>(raw[i], x);
        if (lane * 4 < D)
          q_s[(lane % (D / 16) * kTiles + nt) * 32 + i * 4 + lane / (D / 16)] =
              make_uint2(ptx::pack2<false>(x[0], x[1]), ptx::pack2<false>(x[2], x[3]));
        if (lane == 0)
          qmul_s[nt * 8 + i] =
              p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
      }
    }
    __syncwarp();

    float qmul[kTiles][2];
    int pos[kTiles][2];
    float m[kTiles][2], l[kTiles][2];
#pragma unroll
    for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = nt * 8 + 2 * t + e;
        qmul[nt][e] = qmul_s[r];
        pos[nt][e] = s.len - p.Nq + (row0 + r) % p.Nq;
        m[nt][e] = 0.f;                      // the reference, 0 before the first score
        l[nt][e] = 0.f;
      }
    float o[kJ][kTiles][4] = {};
    float o_unit[kTiles][2] = {};            // of O, by rows (0: nothing summed yet)
    float vs_least = INFINITY;               // smallest scale of values but 0; 0: they are apart
    uint32_t seen = 0;                       // rows (2 nt + e) with a reference
    const int pos_lo = s.len - p.Nq, pos_hi = s.len - 1;

#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int key0 = paged_key0(s, tile0 + i, kKeys);
      alive = ptx::warp_all(alive && ptx::wait_bounded(bar(stage), parity, wd, kSiteDpFull));
      cp_async_wait<kStages - 1>();
      __syncwarp();
      waited += alive;
      const uint8_t* const kt = ring_gen + stage * (2 * kDpTileBytes);
      uint8_t* const vt = ring_gen + stage * (2 * kDpTileBytes) + kDpTileBytes;
      const float* const sc = meta_gen + stage * 8;
      const uint32_t have = valid >> (4 * stage) & 15u;
      // every row sees every key of the tile
      const bool full = have == (1u << p.boxes) - 1u && key0 + kKeys - 1 <= pos_lo &&
                        (key0 > pos_hi - p.win || key0 + kKeys <= p.sinks);
      auto box_of = [&](int mt) { return mt * p.boxes / kMt; };
      if (!full) {
        // values that no row sees weigh 0, and 0 times what they hold must be 0
        for (int i = lane; i < kKeys; i += 32) {
          const int key = key0 + i;
          const bool seen = (have >> box_of(i >> 4) & 1u) && key <= pos_hi &&
                            (key > pos_lo - p.win || key < p.sinks);
          if (!seen)
            for (int c = 0; c < D / 16; ++c)
              *reinterpret_cast<uint4*>(vt + i * D + c * 16) = make_uint4(0, 0, 0, 0);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
      }

      // ---- S^T, 16 bytes of each key row at a time
      float sv[kMt][kTiles][4] = {};
#pragma unroll 1
      for (int c = 0; c < kWords / 4; ++c) {
        uint32_t w[kMt][2][4];               // rows dp_row(g) and + 8 of each 16
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 x = *reinterpret_cast<const uint4*>(
                kt + dp_chunk<D>(mt * 16 + h * 8 + dp_row<D>(g), t * (kWords / 4) + c));
            w[mt][h][0] = x.x;
            w[mt][h][1] = x.y;
            w[mt][h][2] = x.z;
            w[mt][h][3] = x.w;
          }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint2 qb[kTiles];
#pragma unroll
          for (int nt = 0; nt < kTiles; ++nt) qb[nt] = q_s[((c * 4 + j) * kTiles + nt) * 32 + lane];
#pragma unroll
          for (int mt = 0; mt < kMt; ++mt) {
            uint32_t a0, a1, a2, a3;
            codes4<kInt8>(w[mt][0][j], a0, a2);
            codes4<kInt8>(w[mt][1][j], a1, a3);
#pragma unroll
            for (int nt = 0; nt < kTiles; ++nt)
              mma16816(sv[mt][nt], a0, a1, a2, a3, qb[nt].x, qb[nt].y);
          }
        }
      }

      // ---- scores less the row's reference, in log2 units
      float vs[kMt], vs_top = 0.f;
      bool odd = false;                      // a scale of values that is not finite
      float mx[kTiles][2];
#pragma unroll
      for (int nt = 0; nt < kTiles; ++nt) mx[nt][0] = mx[nt][1] = -INFINITY;
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt) {
        // (an infinite one may make scores of -inf, which would weigh nothing)
        const float ks = fabsf(sc[box_of(mt)]) < INFINITY ? sc[box_of(mt)] : NAN;
        const uint64_t k2 = ptx::f2_pack(ks, ks);
        vs[mt] = (have >> box_of(mt) & 1u) ? sc[4 + box_of(mt)] : 0.f;
        // (a page that no row sees may have any scale)
        if (!full && !paged_seen(s, p.Nq, key0 + mt * 16, 16, p.win, p.sinks)) vs[mt] = 0.f;
        if (!(fabsf(vs[mt]) < INFINITY)) {
          vs[mt] = 0.f;
          odd = true;
        }
        vs_top = fmaxf(vs_top, fabsf(vs[mt]));
        vs_least = fminf(vs_least, vs[mt] != 0.f ? fabsf(vs[mt]) : INFINITY);
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt) {
          const uint64_t q2 = ptx::f2_pack(qmul[nt][0], qmul[nt][1]);
          const uint64_t n2 = ptx::f2_pack(-m[nt][0], -m[nt][1]);
          // (a score of 0 is one whatever its factor; another one passes 2^87 at 2^120)
          float c0, c1;
          ptx::f2_unpack(ptx::fmul2(q2, k2), c0, c1);
          const uint64_t c2 = ptx::f2_pack(dp_cap(c0, 0x1p120f), dp_cap(c1, 0x1p120f));
#pragma unroll
          for (int e = 0; e < 4; e += 2)
            ptx::f2_unpack(ptx::ffma2(ptx::f2_pack(sv[mt][nt][e], sv[mt][nt][e + 1]), c2, n2),
                           sv[mt][nt][e], sv[mt][nt][e + 1]);
        }
      }
      if (!full) {
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
          for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + mt * 16 + (e >> 1) * 8 + dp_row<D>(g), ps = pos[nt][e & 1];
              const bool see = (have >> box_of(mt) & 1u) && key <= ps &&
                               (key > ps - p.win || key < p.sinks);
              if (!see) sv[mt][nt][e] = -INFINITY;
            }
      }
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            mx[nt][e] = ptx::max3(mx[nt][e], sv[mt][nt][e], sv[mt][nt][e + 2]);
      // what O is multiplied by
      float f[kTiles][2];
#pragma unroll
      for (int nt = 0; nt < kTiles; ++nt) f[nt][0] = f[nt][1] = 1.f;
      // a row keeps its reference until a score passes it by the threshold (or is
      // its first): only then do its lanes look for its largest
      bool raise = false;
#pragma unroll
      for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          raise |= mx[nt][e] > kDpTau || (!(seen >> (2 * nt + e) & 1u) && mx[nt][e] > -INFINITY);
      raise = __any_sync(0xffffffffu, raise);
      if (raise) {
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int i = 4; i < 32; i *= 2)
              mx[nt][e] = fmaxf(mx[nt][e], __shfl_xor_sync(0xffffffffu, mx[nt][e], i));
            const uint32_t bit = 1u << (2 * nt + e);
            const bool fresh = !(seen & bit);
            if (mx[nt][e] > kDpTau || (fresh && mx[nt][e] > -INFINITY)) {
              // (a row without a reference so far holds zeros, or NaN, which stays)
              f[nt][e] = fresh ? 0.f : ptx::ex2(-mx[nt][e]);
              m[nt][e] += mx[nt][e];
              l[nt][e] *= f[nt][e];
              seen |= bit;
#pragma unroll
              for (int mt = 0; mt < kMt; ++mt) {
                sv[mt][nt][e] -= mx[nt][e];
                sv[mt][nt][e + 2] -= mx[nt][e];
              }
            }
          }
      }
      // the unit of O: alike for all rows, until the scales are apart
      const bool rise = paged_new_unit(o_unit[0][0], vs_top);
      const float now = rise ? paged_unit(vs_top) : o_unit[0][0];
      if (paged_apart(now, vs_least)) {
        vs_least = 0.f;
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float c = 0.f;
#pragma unroll
            for (int mt = 0; mt < kMt; ++mt)
              c = fmaxf(c, ptx::ex2(fmaxf(sv[mt][nt][e], sv[mt][nt][e + 2]) - kDpTau) *
                               fabsf(vs[mt]));
#pragma unroll
            for (int i = 4; i < 32; i *= 2) c = fmaxf(c, __shfl_xor_sync(0xffffffffu, c, i));
            f[nt][e] = paged_row_unit(o_unit[nt][e], f[nt][e], c);
          }
        raise = true;
      } else if (rise) {
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            f[nt][e] *= o_unit[nt][e] * paged_per_unit(now);
            o_unit[nt][e] = now;
          }
        raise = true;
      }
      if (raise) {
#pragma unroll
        for (int j = 0; j < kJ; ++j)
#pragma unroll
          for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][nt][e] *= f[nt][e & 1];
      }
#pragma unroll
      for (int nt = 0; nt < kTiles; ++nt) {
        const uint64_t per = ptx::f2_pack(paged_per_unit(o_unit[nt][0]), paged_per_unit(o_unit[nt][1]));
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt) {
          const uint64_t r2 = ptx::fmul2(ptx::f2_pack(vs[mt], vs[mt]), per);
          const uint64_t ab = ptx::f2_pack(ptx::ex2(sv[mt][nt][0]), ptx::ex2(sv[mt][nt][1]));
          const uint64_t cd = ptx::f2_pack(ptx::ex2(sv[mt][nt][2]), ptx::ex2(sv[mt][nt][3]));
          const uint64_t sum =
              ptx::fadd2(ptx::f2_pack(l[nt][0], l[nt][1]), ptx::fadd2(ab, cd));
          ptx::f2_unpack(sum, l[nt][0], l[nt][1]);
          float a, b, c, d;
          ptx::f2_unpack(ptx::fmul2(ab, r2), a, b);
          ptx::f2_unpack(ptx::fmul2(cd, r2), c, d);
          // P^T as the B operand
          p_s[(mt * kTiles + nt) * 32 + lane] = make_uint2(transpose8x8(ptx::pack2<false>(a, b)),
                                                           transpose8x8(ptx::pack2<false>(c, d)));
        }
      }
      if (odd) {                             // rows that see such a page: NaN
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt) {
          if (!(have >> box_of(mt) & 1u) || fabsf(sc[4 + box_of(mt)]) < INFINITY) continue;
#pragma unroll
          for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (paged_sees(key0 + box_of(mt) * box_rows, box_rows, pos[nt][e & 1], p.win,
                             p.sinks))
#pragma unroll
                for (int j = 0; j < kJ; ++j) o[j][nt][e] = NAN;
        }
      }

      // ---- O^T: element 2 j (+ 1) of the thread's D / 8 of a row, 16 keys at a time
#pragma unroll 1
      for (int mt = 0; mt < kMt; ++mt) {
        constexpr int kVw = D / 32;          // 4-byte words
        uint32_t v[4][kVw];                  // keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // (the 16 rows of a block do not change a row's chunk order)
          const uint8_t* const row = vt + mt * 16 * D;
          const int r = (i >> 1) * 8 + dp_row<D>(2 * t + (i & 1));
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(row + dp_chunk<D>(r, g));
            v[i][0] = x.x;
            v[i][1] = x.y;
            v[i][2] = x.z;
            v[i][3] = x.w;
          } else {
            const uint2 x =
                *reinterpret_cast<const uint2*>(row + dp_chunk<D>(r, g >> 1) + (g & 1) * 8);
            v[i][0] = x.x;
            v[i][1] = x.y;
          }
        }
        uint2 pb[kTiles];
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt) pb[nt] = p_s[(mt * kTiles + nt) * 32 + lane];
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          uint32_t a0, a1, a2, a3;
          constexpr uint32_t kSel[2] = {0x5140, 0x7362};
          codes4<kInt8>(__byte_perm(v[0][j >> 1], v[1][j >> 1], kSel[j & 1]), a0, a1);
          codes4<kInt8>(__byte_perm(v[2][j >> 1], v[3][j >> 1], kSel[j & 1]), a2, a3);
#pragma unroll
          for (int nt = 0; nt < kTiles; ++nt)
            mma16816(o[j][nt], a0, a1, a2, a3, pb[nt].x, pb[nt].y);
        }
      }
      __syncwarp();                          // the stage has been read
      if (alive) load(stage);
      if (++stage == kStages) {
        stage = 0;
        parity ^= 1;
      }
    }

    // ---- the unit's result or its part: a thread has D / 8 elements in a row of
    // each of its rows
    const int unit = (static_cast<int>(head) * p.row_blocks + at.block);
    const size_t slot = 2 * static_cast<size_t>(run) + (pieces == 0 ? 0 : 1);
#pragma unroll
    for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float lt = l[nt][e];
#pragma unroll
        for (int k = 4; k < 32; k *= 2) lt += __shfl_xor_sync(0xffffffffu, lt, k);
        const float mt = m[nt][e];
        const int r = nt * 8 + 2 * t + e;
        if (r >= rows) continue;
        // (in this order nothing leaves float32's range that the result does not)
        const float inv = ptx::rcp(lt);
        float x[2 * kJ];
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          x[2 * j] = lt != 0.f ? o[j][nt][e] * inv * o_unit[nt][e] : 0.f;
          x[2 * j + 1] = lt != 0.f ? o[j][nt][e + 2] * inv * o_unit[nt][e] : 0.f;
        }
        if (whole) {
          const size_t row = head * p.R + row0 + r;
          uint4* const out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + row * D) +
                             g * (kJ / 4);
#pragma unroll
          for (int j = 0; j < kJ / 4; ++j)
            out[j] = make_uint4(ptx::pack2<kBf16>(x[8 * j], x[8 * j + 1]),
                                ptx::pack2<kBf16>(x[8 * j + 2], x[8 * j + 3]),
                                ptx::pack2<kBf16>(x[8 * j + 4], x[8 * j + 5]),
                                ptx::pack2<kBf16>(x[8 * j + 6], x[8 * j + 7]));
          if (g == 0)
            p.lse[row] = lt != 0.f ? (ptx::lg2(lt) + mt) * 0.693147180559945309f : -INFINITY;
        } else {
          float4* const out = p.part_o + (slot * p.slot_rows + r) * (D / 4) + g * (kJ / 2);
#pragma unroll
          for (int j = 0; j < kJ / 2; ++j)
            out[j] = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
          if (g == 0) p.part_ml[slot * p.slot_rows + r] = make_float2(mt, lt);
        }
      }
    if (tile0 == 0 && lane == 0)
      p.cut[unit] = whole ? make_int2(-1, 0)
                          : make_int2(static_cast<int>(slot),
                                      dec_run_of(deal, rn.start + done + s.tiles - 1));
    done += n;
    __syncwarp();                            // the queries have been read
  }
  // after a wait that ran out: the loads in flight land before the block ends
  cp_async_wait<0>();
  for (; waited < loaded; ++waited)
    ptx::wait_drain(bar(waited % kStages), waited / kStages & 1, 200000000ull);
}

// The cut units: a block takes `per_block` units and adds up the unit's parts of
// a row, 4 columns a thread.  With few parts D / 4 threads do a row alone, and a
// block several rows (kGroups = 1); with many, kGroups such groups take other
// parts of one row each and meet in shared memory.  kBatch parts are in flight at
// a time.  Each part is a mean with its weight, and so is what they add up to: every
// factor is at most 1, and values of any size stay in range.
// A row without a visible key has no live part (a sum of NaN is live).
// (5 parts of 512 units, 4 rows: 8.0 us with four groups a row, 5.8 alone.)
constexpr int kDpCombineThreads = 128;       // of kGroups = 1
template <int D, bool kBf16, int kGroups>
__global__ void __launch_bounds__(kGroups == 1 ? kDpCombineThreads : kGroups * (D / 4))
    fa_decode_paged_combine_kernel(const __grid_constant__ DecPagedParams p, int units,
                                   int per_block) {
  constexpr int kPer = D / 4, kBatch = 8;
  constexpr int kRowsOf = kGroups == 1 ? kDpCombineThreads / kPer : 1;   // of a block
  __shared__ float4 acc_s[kGroups][kPer];
  __shared__ float2 ml_s[kGroups];
  const int c = threadIdx.x % kPer, of = threadIdx.x / kPer;
  const int group = kGroups == 1 ? 0 : of, r = blockIdx.y * kRowsOf + (kGroups == 1 ? of : 0);
  ptx::griddep_wait();   // the parts are complete, and this grid ends after the main one
  const int u1 = min((static_cast<int>(blockIdx.x) + 1) * per_block, units);
  for (int u = blockIdx.x * per_block; u < u1; ++u) {
    const int2 cut = p.cut[u];
    if (cut.x < 0) continue;
    const int head = u / p.row_blocks, row = (u - head * p.row_blocks) * p.slot_rows + r;
    if (r >= p.slot_rows || row >= p.R) continue;
    const int run0 = cut.x >> 1, parts = cut.y - run0 + 1;
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = group; i < parts; i += kGroups * kBatch) {
      float2 ml[kBatch];
      float4 x[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int part = i + k * kGroups;
        ml[k] = make_float2(0.f, 0.f);
        if (part < parts) {
          const size_t slot = part == 0 ? cut.x : 2 * static_cast<size_t>(run0 + part);
          ml[k] = p.part_ml[slot * p.slot_rows + r];
          x[k] = p.part_o[(slot * p.slot_rows + r) * kPer + c];
        }
      }
      float now = m;
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (ml[k].y != 0.f) now = fmaxf(now, ml[k].x);
      // the weight of what there was, then those of the batch
      const float was = m == -INFINITY ? 0.f : ptx::ex2(m - now) * l;
      float w[kBatch];
      l = was;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        w[k] = ml[k].y != 0.f ? ptx::ex2(ml[k].x - now) * ml[k].y : 0.f;
        l += w[k];
      }
      m = now;
      const float inv = l != 0.f ? ptx::rcp(l) : 0.f, fo = was * inv;
      acc = make_float4(acc.x * fo, acc.y * fo, acc.z * fo, acc.w * fo);
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (ml[k].y != 0.f) {
          const float f = w[k] * inv;
          acc.x = fmaf(f, x[k].x, acc.x);
          acc.y = fmaf(f, x[k].y, acc.y);
          acc.z = fmaf(f, x[k].z, acc.z);
          acc.w = fmaf(f, x[k].w, acc.w);
        }
    }
    float top = m, lt = l;
    float4 sum = acc;
    if constexpr (kGroups > 1) {
      acc_s[group][c] = acc;
      if (c == 0) ml_s[group] = make_float2(m, l);
      __syncthreads();
      if (threadIdx.x < 32) {              // group 0's warp: a lane for each group's weight
        const float2 part = threadIdx.x < kGroups ? ml_s[threadIdx.x] : make_float2(0.f, 0.f);
        top = part.y != 0.f ? part.x : -INFINITY;
#pragma unroll
        for (int k = 1; k < 32; k *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        float f = part.y != 0.f ? ptx::ex2(part.x - top) * part.y : 0.f;
        lt = f;
#pragma unroll
        for (int k = 1; k < 32; k *= 2) lt += __shfl_xor_sync(0xffffffffu, lt, k);
        f *= lt != 0.f ? ptx::rcp(lt) : 0.f;
        sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < kGroups; ++k) {
          const float fk = __shfl_sync(0xffffffffu, f, k);
          const float4 x = acc_s[k][c];
          sum.x = fmaf(fk, x.x, sum.x);
          sum.y = fmaf(fk, x.y, sum.y);
          sum.z = fmaf(fk, x.z, sum.z);
          sum.w = fmaf(fk, x.w, sum.w);
        }
      }
    }
    if (group == 0) {
      const size_t out = static_cast<size_t>(head) * p.R + row;
      reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + out * D)[c] =
          make_uint2(ptx::pack2<kBf16>(sum.x, sum.y), ptx::pack2<kBf16>(sum.z, sum.w));
      if (c == 0) p.lse[out] = lt != 0.f ? (ptx::lg2(lt) + top) * 0.693147180559945309f : -INFINITY;
    }
    if constexpr (kGroups > 1) __syncthreads();
  }
}

}  // namespace fa
