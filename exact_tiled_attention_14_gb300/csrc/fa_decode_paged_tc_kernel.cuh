// fa_decode_paged_tc_kernel.cuh — decoding over pages of 8-bit keys and values
// (see fa_paged.cuh) for many rows: 17 to 128 query rows of a key/value head in
// one unit, on the tensor cores through TMEM.
//
// The function, the queries' powers of two, the placing of the scales and the
// unit of O are those of fa_decode_paged_kernel.cuh.  There a warp turns codes
// into 16-bit registers for its own products, which costs as many issue slots
// again for each 16 rows (figures at row_tiles in fa_decode_paged.cu).  Here codes are turned once for all rows, by warps of their own, into
// half-precision tiles in shared memory, and a product of 128 rows costs a
// tile 544 cycles whatever their number.
//
// Cost (d = 128, a tile of 128 keys, 32 KB): its share of HBM 1394 cycles of
// an SM, the products 1088, 1800 of shared-memory traffic (codes in and out 64
// KB, half-precision tiles in and out 128 KB, queries 32 KB).  What bounds it is
// none of them but a softmax thread's chain, some 2650 cycles a tile at 64 rows and
// 2900 at 128 (of 20 parts about 3 to read the scores, 3 to their maximum, 2 to
// meet, 6 for the weights, 3 to store them, 3 around the loop), and at the ends of a
// run 12000 cycles to the first scores and 4000 to leave a part.  8 caches to
// 32768, 4 K/V heads (169 MB, 25 us): 32 and 64 rows 63.5 us, 128 rows 73.5; at
// d = 64 64 rows take 59.5.  Scales of V that differ by more than 2^4, for which a
// row's threads meet in every tile, add 10 %.
//
// One CTA (27 warps) per SM, persistent over its run of key tiles:
//   warps 0-15   softmax: warp w has rows 32 (w % 4) .. + 31, one a lane, and
//                quarter w / 4 of a tile's keys; the four threads of a row agree
//                on its reference;
//   warps 16-19  K tiles to half precision, and the queries at a unit's start;
//   warps 20-23  V tiles, rows that no row of the unit sees as zeros
//                (up to 64 rows softmax warps without rows do both: see `turner`);
//   warps 24, 25 pages, scales and the TMA loads, of K and of V (and, with V's
//                scales, the unit of O that they call for);
//   warp 26      S = Q K^T of the next tile, then O += P V of this one.
// 64 keys a softmax thread instead of 32 took twice as long.  A second copy of up
// to 64 rows in the idle lanes, which takes every other tile, gained 1 us of 71 and
// cost 128 rows 12 (the products' order, the copies' sum); weights formed before
// the row's threads have met, done again where a score passes, cost 20 of 68.
// S and P are double buffered in TMEM (at d = 128 it is full), O is not.  A unit
// that lies in one run is finished there; parts of the others go to the
// workspace for fa_decode_paged_combine_kernel.
#pragma once

#include "fa_decode_paged_kernel.cuh"

namespace fa {

constexpr int kDtKeys = 128, kDtRows = 128, kDtThreads = 864;
constexpr int kDtConvert = 16, kDtLoad = 24, kDtMma = 26;   // first warp of a role
constexpr int kDtTurners = 4;            // warps that turn K, and V
constexpr int kDtMetas = 3;              // tiles whose scales are kept

enum DtWaitSite : uint32_t {
  kSiteDtCodesFull = 51, kSiteDtCodesEmpty = 52, kSiteDtMetaFull = 53, kSiteDtMetaEmpty = 54,
  kSiteDtKFull = 55, kSiteDtKEmpty = 56, kSiteDtVFull = 57, kSiteDtVEmpty = 58, kSiteDtSFull = 59,
  kSiteDtPFull = 60, kSiteDtPvDone = 61, kSiteDtOFree = 62,
  kSiteDtQReady = 63
};

// Scales of a tile by 16 keys (V's in units of `unit`, see paged_unit), and which of
// the eight name a page; bit 8: the scales of V so far are apart (paged_apart).
struct DtMeta {
  float ks[8], vs[8];
  uint32_t have;
  float unit;
  uint32_t pad[2];
};

template <int D>
struct DtLayout {
  static constexpr int kChunks = D / 64, kChunkBytes = kDtKeys * 128;
  static constexpr int kTile = kDtKeys * D * 2;               // half precision
  static constexpr int kCodes = kDtKeys * D;                  // of K, and of V
  static constexpr int kSlots = D == 128 ? 4 : 8;              // of the ring: K, V, K, V ...
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + kTile;                       // two tiles each
  static constexpr int kV = kK + 2 * kTile;
  static constexpr int kRing = kV + 2 * kTile;
  static constexpr int kMeet = kRing + kSlots * kCodes;  // [2][row], where a row's threads meet
  static constexpr int kMeta = kMeet + 2 * kDtRows * 4;
  // the queries' powers of two, of the units whose first tile has the meta's slot
  static constexpr int kShift = kMeta + kDtMetas * static_cast<int>(sizeof(DtMeta));   // [row] int8
  static constexpr int kBar = kShift + kDtMetas * kDtRows;
  static constexpr int bCodesFull = 0, bCodesEmpty = kSlots, bMetaFull = 2 * kSlots,
                       bMetaEmpty = bMetaFull + kDtMetas, bKFull = bMetaEmpty + kDtMetas,
                       bKEmpty = bKFull + 2, bVFull = bKEmpty + 2, bVEmpty = bVFull + 2,
                       bSFull = bVEmpty + 2, bPFull = bSFull + 2, bPvDone = bPFull + 2,
                       bQReady = bPvDone + 2, bOFree = bQReady + kDtMetas,
                       bFinal = bOFree + 1, kNumBars = bFinal + 1;
  static constexpr int kMisc = kBar + 8 * kNumBars;           // TMEM base, abort flag, a word for stores
  static constexpr int kAlloc = kMisc + 16 + 1024;
  static_assert(kBar % 8 == 0 && kAlloc <= 232448, "shared memory budget");
  static constexpr uint32_t s_col(int b) { return 128u * b; }
  static constexpr uint32_t kOCol = 256;
  static constexpr uint32_t p_col(int b) { return 256u + D + 64u * b; }
};

// Row in its eight and 16-byte piece of a lane in step k of turning codes, four
// (d = 128) or eight (64) rows a step: reads (swizzled by the copy) and both
// 16-byte writes of every quarter warp touch all banks once.  At d = 128 a
// quarter takes four pieces of one 64-column chunk of two rows whose numbers
// differ in bits 0 (the writes' other banks) and 2 (the reads').
struct DtPiece {
  int row, piece;
};
template <int D>
__host__ __device__ __forceinline__ DtPiece dt_piece(int lane, int k) {
  DtPiece p;
  if (D == 128) {
    const int q = lane >> 3, i = lane & 7, a = 2 * (k & 1) + (q & 1);
    p.row = i & 4 ? a ^ 5 : a;
    p.piece = (i & 3) + 4 * (q >> 1);
  } else {
    p.row = lane >> 2;
    p.piece = lane & 3;
  }
  return p;
}
// Where half h (8 elements, 16 bytes) of piece c of row r goes in a tile of half
// precision: chunks of 64 columns, rows of 128 bytes, 128-byte swizzle.
__host__ __device__ __forceinline__ uint32_t dt_place(int r, int c, int h) {
  return (c >> 2) * static_cast<uint32_t>(kDtKeys * 128) + r * 128u +
         (((2 * (c & 3) + h) ^ (r & 7)) << 4);
}

template <int D, bool kBf16, bool kInt8>
__global__ void __launch_bounds__(kDtThreads, 1)
    fa_decode_paged_tc_kernel(const __grid_constant__ DecPagedParams p) {
  using L = DtLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = ptx::smem_u32(smem_raw);
  const uint32_t sbase = (raw_base + 1023u) & ~1023u;
  uint8_t* const sgen = smem_raw + (sbase - raw_base);
  const int warp = ptx::warp_same(threadIdx.x >> 5), lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return sbase + L::kBar + 8u * i; };
  uint32_t* const tmem_ptr = reinterpret_cast<uint32_t*>(sgen + L::kMisc);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(sgen + L::kMisc + 4);
  DtMeta* const metas = reinterpret_cast<DtMeta*>(sgen + L::kMeta);
  // (volatile: read before the slot is given back, not where the values are used)
  auto meta_of = [&](int ms) { return static_cast<const volatile DtMeta*>(metas + ms); };
  volatile signed char* const shift_s = reinterpret_cast<volatile signed char*>(sgen + L::kShift);
  const ptx::Watchdog wd{p.watchdog_cycles, abort_flag, p.status};

  // softmax warps: with one unit a head, those that have rows
  const int quarters = p.row_blocks > 1 ? 4 : (p.R + 31) / 32, active = 4 * quarters;
  // The turners' numbers.  A warp's softmax rows are given by the part of the SM that
  // it runs on (w % 4), so up to 64 rows keep two of the four parts busy: there the
  // other two parts' softmax warps, which have no rows, turn the codes.
  const int turner = quarters > 2 ? (warp < kDtLoad ? warp - kDtConvert : -1)
                     : warp < kDtConvert && (warp & 2) ? (warp >> 2) * 2 + (warp & 1)
                                                       : -1;

  ptx::griddep_launch_dependents();
  if (warp == kDtMma) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_ptr), 512);
    ptx::tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < L::kSlots; ++i) {
      ptx::mbar_init(bar(L::bCodesFull + i), 1);
      ptx::mbar_init(bar(L::bCodesEmpty + i), kDtTurners);
    }
    for (int i = 0; i < kDtMetas; ++i) {
      ptx::mbar_init(bar(L::bMetaFull + i), 2);
      ptx::mbar_init(bar(L::bMetaEmpty + i), active + kDtTurners);
      ptx::mbar_init(bar(L::bQReady + i), kDtTurners);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(L::bKFull + i), kDtTurners);
      ptx::mbar_init(bar(L::bKEmpty + i), 1);
      ptx::mbar_init(bar(L::bVFull + i), kDtTurners);
      ptx::mbar_init(bar(L::bVEmpty + i), 1);
      ptx::mbar_init(bar(L::bSFull + i), 1);
      ptx::mbar_init(bar(L::bPFull + i), active);
      ptx::mbar_init(bar(L::bPvDone + i), 1);
    }
    ptx::mbar_init(bar(L::bOFree), active);
    ptx::mbar_init(bar(L::bFinal), 1);
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&p.tm_k);
    ptx::prefetch_tmap(&p.tm_v);
  }
  // ---- the CTA's run and its first place (each warp for itself)
  const DpRun rn = dp_run(p, kDtKeys, p.runs, 1, blockIdx.x);
  const DecDeal deal = rn.deal;
  const int run = blockIdx.x;
  DpPlace at = rn.at;
  int left = rn.left;
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = ptx::warp_same(*tmem_ptr);

  const int box_rows = kDtKeys / p.boxes;
  auto piece_of = [&](int& n, bool& whole) {     // of the place `at`
    n = min(at.s.tiles - at.tile, left);
    whole = at.tile == 0 && n == at.s.tiles;
  };

  if (warp == kDtLoad || warp == kDtLoad + 1) {
    // ============================================================ pages, scales, loads
    // Lane 8 a + i looks up box i of every fourth tile from tile a on: pages are
    // asked for eight tiles and scales four tiles before they are needed, and no
    // tile waits for them.
    const bool is_v = warp != kDtLoad;
    const CUtensorMap* const tm = is_v ? &p.tm_v : &p.tm_k;
    const float* const scales = is_v ? p.v_scale : p.k_scale;
    const int box = lane & 7, ahead = lane >> 3;
    DpPlace nx = at;                             // the lane's next tile, and its number
    int nx_j = 0;
    auto skip = [&](int n) {
      nx_j += n;
      nx.tile += n;
      while (nx_j < left && nx.tile >= nx.s.tiles) {
        const int over = nx.tile - nx.s.tiles;
        dp_next_unit(p, nx, kDtKeys);
        nx.tile = over;
      }
    };
    skip(ahead);
    struct Box {
      int page = -1, hk = 0, row = 0;            // page (-1: none), head, first row in the page
      bool seen = false;                         // by some row
      bool first = false;                        // of a piece of a unit
    };
    auto look = [&]() {
      Box x;
      if (nx_j < left && box < p.boxes) {
        const int key = paged_key0(nx.s, nx.tile, kDtKeys) + box * box_rows;
        const int nth = p.page_magic ? __umulhi(key >> 4, p.page_magic) : key >> 4;
        x.row = key - nth * p.page;
        x.hk = nx.hk;
        x.seen = paged_seen(nx.s, p.Nq, key, box_rows, p.win, p.sinks);
        x.first = nx_j == 0 || nx.tile == 0;
        if (key < nx.s.len) x.page = p.table[static_cast<size_t>(nx.b) * p.per_seq + nth];
      }
      skip(4);
      return x;
    };
    struct Code {
      int row;                                   // of the cache (-1: none)
      float scale;
      bool seen, first;
    };
    auto resolve = [&](const Box& x) {
      Code c{-1, 0.f, x.seen, x.first};
      if (x.page >= 0 && x.page < p.pages) {
        const int head = x.page * p.Hk + x.hk;
        c.row = head * p.page + x.row;
        c.scale = scales[head];
        // (an infinite one of K may make scores of -inf, which would weigh nothing)
        if (!is_v && !(fabsf(c.scale) < INFINITY)) c.scale = NAN;
      }
      return c;
    };
    Box x0 = look(), x1 = look();
    Code now = resolve(x0), next = resolve(x1);
    x0 = look();
    bool alive = true;
    int issued = 0;
    const int per = 8 / p.boxes;
    float unit = 0.f, vs_least = INFINITY;       // of O, and the smallest scale of V but 0, in the piece
#pragma unroll 1
    for (int j = 0; j < left && alive; ++j) {
      const int ms = j % kDtMetas, use = 2 * j + is_v, slot = use % L::kSlots;
      const bool mine = ahead == (j & 3) && now.row >= 0;
      const uint32_t have = __ballot_sync(0xffffffffu, mine) >> (8 * (j & 3)) & 255u;
      if (use >= L::kSlots)
        alive = ptx::warp_all(alive && ptx::wait_bounded(bar(L::bCodesEmpty + slot),
                                                         (use / L::kSlots - 1) & 1, wd,
                                                         kSiteDtCodesEmpty));
      if (!alive) break;
      if (lane == 0)
        ptx::mbar_arrive_expect_tx(bar(L::bCodesFull + slot), __popc(have) * box_rows * D);
      __syncwarp();
      if (mine)
        tma_load_rows(sbase + L::kRing + slot * L::kCodes + box * box_rows * D, tm,
                      bar(L::bCodesFull + slot), now.row);
      ++issued;
      if (j >= kDtMetas)
        alive = ptx::warp_all(alive && ptx::wait_bounded(bar(L::bMetaEmpty + ms),
                                                         (j / kDtMetas - 1) & 1, wd,
                                                         kSiteDtMetaEmpty));
      float per_unit = 1.f;
      if (is_v) {
        // the unit of O rises with the scales that some row sees, until they are apart
        const float size = mine && now.seen && fabsf(now.scale) < INFINITY ? fabsf(now.scale) : 0.f;
        const float top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(size)));
        const float least = __uint_as_float(
            __reduce_min_sync(0xffffffffu, size > 0.f ? __float_as_uint(size) : kInfBits));
        if (__any_sync(0xffffffffu, ahead == (j & 3) && now.first)) {
          unit = 0.f;
          vs_least = INFINITY;
        }
        if (paged_new_unit(unit, top)) unit = paged_unit(top);
        per_unit = paged_per_unit(unit);
        vs_least = fminf(vs_least, least);
        // (a box's bit for each 16 keys of it)
        const uint32_t bits =
            __ballot_sync(0xffffffffu, lane < 8 && (have >> (lane * p.boxes / 8) & 1u));
        if (lane == 0) {
          metas[ms].have = bits | (paged_apart(unit, vs_least) ? 256u : 0u);
          metas[ms].unit = unit;
        }
      }
      if (ahead == (j & 3) && box < p.boxes) {
        float* const to = is_v ? metas[ms].vs : metas[ms].ks;
        const float x = is_v ? now.scale * per_unit : now.scale;
        for (int i = box * per; i < (box + 1) * per; ++i) to[i] = x;
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(L::bMetaFull + ms));
      if ((j & 3) == 3) {
        now = next;
        next = resolve(x0);
        x0 = look();
      }
    }
    // the loads land before the block ends, whatever became of their readers
    for (int i = max(issued - L::kSlots / 2, 0); i < issued; ++i) {
      const int use = 2 * i + is_v;
      ptx::wait_drain(bar(L::bCodesFull + use % L::kSlots), use / L::kSlots & 1, 200000000ull);
    }
    __syncwarp();
  } else if (warp == kDtMma) {
    // ============================================================ products
    constexpr uint32_t idesc_s = ptx::idesc_f16(kDtRows, kDtKeys, 0, 0);
    constexpr uint32_t idesc_o = ptx::idesc_f16(kDtRows, D, 0, 1);
    const uint32_t q_lo = ptx::desc_lo(sbase + L::kQ, 16);
    const uint32_t k_lo = ptx::desc_lo(sbase + L::kK, 16);
    const uint32_t v_lo = ptx::desc_lo(sbase + L::kV, L::kChunkBytes);
    bool alive = true, issued = false;
    auto issue_s = [&](int j) {
      const int b = j & 1;
      // (S of two tiles ago has been read: its P was waited for)
      alive = ptx::warp_all(alive && ptx::wait_bounded(bar(L::bKFull + b), j >> 1 & 1, wd,
                                                       kSiteDtKFull));
      ptx::tc_fence_after();
      if (!alive) return;
      issued = true;
      if (ptx::elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off =
              static_cast<uint32_t>((kk >> 2) * L::kChunkBytes + (kk & 3) * 32) >> 4;
          ptx::mma_ss(tmem + L::s_col(b), ptx::desc_sw128(q_lo + off),
                      ptx::desc_sw128(k_lo + b * (L::kTile >> 4) + off), idesc_s, kk > 0);
        }
        ptx::mma_commit(bar(L::bSFull + b));
        ptx::mma_commit(bar(L::bKEmpty + b));
      }
    };
    const int total = left;
    if (total > 0) issue_s(0);
    int j = 0;
    for (int pieces = 0; left > 0; ++pieces, dp_next_unit(p, at, kDtKeys)) {
      int n;
      bool whole;
      piece_of(n, whole);
      left -= n;
      for (int i = 0; i < n; ++i, ++j) {
        if (j + 1 < total) issue_s(j + 1);
        const int b = j & 1;
        alive = ptx::warp_all(alive && ptx::wait_bounded(bar(L::bVFull + b), j >> 1 & 1, wd,
                                                         kSiteDtVFull));
        if (i == 0 && pieces > 0)                // the previous unit's O has been read
          alive = ptx::warp_all(alive && ptx::wait_bounded(bar(L::bOFree), (pieces - 1) & 1, wd,
                                                           kSiteDtOFree));
        alive = ptx::warp_all(alive && ptx::wait_bounded(bar(L::bPFull + b), j >> 1 & 1, wd,
                                                         kSiteDtPFull));
        ptx::tc_fence_after();
        if (alive && ptx::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kDtKeys / 16; ++kk)
            ptx::mma_ts(tmem + L::kOCol, tmem + L::p_col(b) + kk * 8,
                        ptx::desc_sw128(v_lo + b * (L::kTile >> 4) + kk * (2048 >> 4)), idesc_o,
                        kk > 0 || i > 0);
          ptx::mma_commit(bar(L::bPvDone + b));
          ptx::mma_commit(bar(L::bVEmpty + b));
        }
      }
    }
    if (issued) {                                // nothing is in flight when TMEM goes
      if (ptx::elect_one()) ptx::mma_commit(bar(L::bFinal));
      ptx::wait_drain(bar(L::bFinal), 0, 200000000ull);
    }
    __syncwarp();
  } else if (turner >= 0) {
    // ============================================================ codes to half precision
    constexpr int kRowsOf = kDtKeys / kDtTurners;            // rows of a warp
    constexpr int kBatch = 8;                                // query rows at a time
    constexpr int kStep = D == 128 ? 4 : 8, kSteps = kRowsOf / kStep;
    const bool is_v = turner >= kDtTurners;
    const int first = (turner & (kDtTurners - 1)) * kRowsOf;
    // where the lane's piece of step k comes from and goes to, but for its eight
    // rows, in which a row has the same place in each
    uint32_t from[2], to[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const DtPiece x = dt_piece<D>(lane, k);
      from[k] = dp_chunk<D>(first + x.row, x.piece);
      to[k] = dt_place(first + x.row, x.piece, 0);
    }
    uint8_t* const tiles = sgen + (is_v ? L::kV : L::kK);
    const int b_full = is_v ? L::bVFull : L::bKFull, b_empty = is_v ? L::bVEmpty : L::bKEmpty;
    const uint32_t site = is_v ? kSiteDtVEmpty : kSiteDtKEmpty;
    bool alive = true;
    int j = 0;
    for (; left > 0; dp_next_unit(p, at, kDtKeys)) {
      int n;
      bool whole;
      piece_of(n, whole);
      left -= n;
      const PagedSpan s = at.s;
      const int pos_lo = s.len - p.Nq, pos_hi = s.len - 1;
      if (!is_v) {
        // Queries, asked for before the previous unit's last S has read its own; rows
        // that no softmax warp takes may hold anything.
        const size_t head = static_cast<size_t>(at.b) * p.Hk + at.hk;
        const int row0 = at.block * kDtRows, rows = min(p.R - row0, kDtRows);
        volatile signed char* const shifts = shift_s + j % kDtMetas * kDtRows;
        const int of = 8 * quarters;             // the warp's rows
#pragma unroll 1
        for (int r0 = turner * of; r0 < (turner + 1) * of; r0 += kBatch) {
          uint2 raw[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            raw[i] = make_uint2(0, 0);
            if (r0 + i < rows && lane * 4 < D)
              raw[i] = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.q) +
                                                       (head * p.R + row0 + r0 + i) * D + lane * 4);
          }
          if (r0 == turner * of && j > 0) {
            alive = ptx::warp_all(alive && ptx::wait_bounded(bar(L::bKEmpty + ((j - 1) & 1)),
                                                             (j - 1) >> 1 & 1, wd, kSiteDtKEmpty));
            // (the powers' slot is free with the first tile's meta)
            if (j >= kDtMetas)
              alive = ptx::warp_all(alive && ptx::wait_bounded(bar(L::bMetaFull + j % kDtMetas),
                                                               j / kDtMetas & 1, wd,
                                                               kSiteDtMetaFull));
          }
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            float x[4];
            const int shift = dp_query_row<kBf16>(raw[i], x);
            if (lane * 4 < D)
              *reinterpret_cast<uint2*>(sgen + L::kQ + dt_place(r0 + i, lane >> 2, lane >> 1 & 1) +
                                        (lane & 1) * 8) =
                  make_uint2(ptx::pack2<false>(x[0], x[1]), ptx::pack2<false>(x[2], x[3]));
            if (lane == 0) shifts[r0 + i] = static_cast<signed char>(shift);
          }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(L::bQReady + j % kDtMetas));
      }
      for (int i = 0; i < n; ++i, ++j) {
        const int ms = j % kDtMetas, b = j & 1;
        const int slot = 2 * j % L::kSlots + is_v;
        const int key0 = paged_key0(s, at.tile + i, kDtKeys);
        if (is_v)
          alive = ptx::warp_all(alive && ptx::wait_bounded(bar(L::bMetaFull + ms), j / kDtMetas & 1,
                                                           wd, kSiteDtMetaFull));
        alive = ptx::warp_all(alive && ptx::wait_bounded(bar(L::bCodesFull + slot),
                                                         2 * j / L::kSlots & 1, wd,
                                                         kSiteDtCodesFull));
        const uint8_t* const codes = sgen + L::kRing + slot * L::kCodes;
        uint4 x[kSteps];
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
          x[k] = *reinterpret_cast<const uint4*>(codes + from[k & 1] + (k * kStep & ~7) * D);
        // The next copy may write the slot once this arrives, and nothing orders a copy
        // behind loads whose results are not used yet.  So every lane first stores a word
        // that it can form only from all of its loads (nobody reads it, and whose store
        // stays does not matter); the warp meets behind the stores, and only then does
        // one lane arrive.  Without it up to a third of the runs over short units had a
        // tile with the next but one's codes; it costs 1 us of 63.
        uint32_t all = 0;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) all |= x[k].x | x[k].y | x[k].z | x[k].w;
        ptx::st_shared(sbase + L::kMisc + 8, all);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(L::bCodesEmpty + slot));
        if (is_v) {
          const uint32_t have = meta_of(ms)->have & 255u;
          const bool full = have == 255u && key0 + kDtKeys - 1 <= pos_hi &&
                            (key0 > pos_lo - p.win || key0 + kDtKeys <= p.sinks);
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(L::bMetaEmpty + ms));
          if (!full) {
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
              const int r = first + (k * kStep & ~7) + dt_piece<D>(lane, k).row;
              if (!(have >> (r >> 4) & 1u && key0 + r <= pos_hi &&
                    (key0 + r > pos_lo - p.win || key0 + r < p.sinks)))
                x[k] = make_uint4(0, 0, 0, 0);
            }
          }
        }
        if (j >= 2)
          alive = ptx::warp_all(alive && ptx::wait_bounded(bar(b_empty + b), (j - 2) >> 1 & 1, wd,
                                                           site));
        uint8_t* const tile = tiles + b * L::kTile;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint4 y, z;
          codes4<kInt8>(x[k].x, y.x, y.y);
          codes4<kInt8>(x[k].y, y.z, y.w);
          codes4<kInt8>(x[k].z, z.x, z.y);
          codes4<kInt8>(x[k].w, z.z, z.w);
          uint8_t* const eight = tile + (k * kStep & ~7) * 128;
          *reinterpret_cast<uint4*>(eight + to[k & 1]) = y;
          *reinterpret_cast<uint4*>(eight + (to[k & 1] ^ 16u)) = z;
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(b_full + b));
      }
    }
  } else if (warp < kDtConvert && (warp & 3) < quarters) {
    // ============================================================ softmax
    const int quarter = warp & 3, part = warp >> 2, r = quarter * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    float* const meet = reinterpret_cast<float*>(sgen + L::kMeet) + r;
    // the four threads of a row, in warps four apart, come to one value
    auto row_sync = [&]() { ptx::named_bar_sync(1 + quarter, 128); };
    auto row_all = [&](float v, auto&& join) {
      if (part >= 2) meet[(part - 2) * kDtRows] = v;
      row_sync();
      if (part < 2) {
        v = join(v, meet[part * kDtRows]);
        meet[part * kDtRows] = v;
      }
      row_sync();
      v = join(meet[0], meet[kDtRows]);
      row_sync();
      return v;
    };
    int j = 0;
    uint32_t q_parity = 0;
    for (int pieces = 0; left > 0; ++pieces, dp_next_unit(p, at, kDtKeys)) {
      int n;
      bool whole;
      piece_of(n, whole);
      const int done = rn.left - left;           // tiles of the run before the piece
      left -= n;
      const PagedSpan s = at.s;
      const size_t head = static_cast<size_t>(at.b) * p.Hk + at.hk;
      const int row0 = at.block * kDtRows, rows = min(p.R - row0, kDtRows);
      const bool has = quarter * 32 < rows;      // a warp without rows only keeps the order
      const int pos = s.len - p.Nq + (row0 + r) % p.Nq;
      const int pos_lo = s.len - p.Nq, pos_hi = s.len - 1;
      float m = 0.f, l = 0.f,                    // the reference, 0 before the first score
            o_unit = 0.f, qmul = 0.f;            // the unit of O
      bool fresh = true, poison = false;         // no reference yet; a page's scale of values is not finite
      for (int i = 0; i < n; ++i, ++j) {
        const int ms = j % kDtMetas, b = j & 1;
        const int key0 = paged_key0(s, at.tile + i, kDtKeys) + part * 32;   // of the thread's keys
        ptx::wait_bounded(bar(L::bMetaFull + ms), j / kDtMetas & 1, wd, kSiteDtMetaFull);
        ptx::wait_bounded(bar(L::bSFull + b), j >> 1 & 1, wd, kSiteDtSFull);
        __syncwarp();
        ptx::tc_fence_after();
        const volatile DtMeta* const meta = meta_of(ms);
        const uint32_t bits = meta->have, have = bits >> (2 * part) & 3u;
        const float unit = meta->unit;
        const float ks[2] = {meta->ks[2 * part], meta->ks[2 * part + 1]};
        float vs[2] = {meta->vs[2 * part], meta->vs[2 * part + 1]};
        // every row sees every key of the thread's
        const bool full = have == 3u && key0 + 31 <= pos_lo &&
                          (key0 > pos_hi - p.win || key0 + 32 <= p.sinks);
        if (!full) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (!(have >> k & 1u) || !paged_seen(s, p.Nq, key0 + 16 * k, 16, p.win, p.sinks))
              vs[k] = 0.f;
        }
        if (!(fabsf(vs[0]) < INFINITY && fabsf(vs[1]) < INFINITY)) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (!(fabsf(vs[k]) < INFINITY)) {
              poison |= paged_sees(key0 + 16 * k, 16, pos, p.win, p.sinks);
              vs[k] = 0.f;
            }
        }
        if (i == 0) {                            // (a slot's parity turns with each unit on it)
          ptx::wait_bounded(bar(L::bQReady + ms), q_parity >> ms & 1, wd, kSiteDtQReady);
          q_parity ^= 1u << ms;
          const int shift = shift_s[ms * kDtRows + r];
          qmul = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(L::bMetaEmpty + ms));
        if (has) {
          uint32_t sr[32];
          ptx::tmem_ld32(lanes + L::s_col(b) + part * 32, sr);
          ptx::tmem_wait_ld();
          // scores less the row's reference, in log2 units
          float x[32];
          const uint64_t n2 = ptx::f2_pack(-m, -m);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float c = qmul * ks[k];
            if (fabsf(c) < 0x1p100f && fabsf(c) > 0x1p-100f) {
              const uint64_t c2 = ptx::f2_pack(c, c);
#pragma unroll
              for (int e = 16 * k; e < 16 * k + 16; e += 2)
                ptx::f2_unpack(ptx::ffma2(ptx::f2_pack(__uint_as_float(sr[e]),
                                                       __uint_as_float(sr[e + 1])),
                                          c2, n2),
                               x[e], x[e + 1]);
            } else {   // factors whose product may leave the range that the score stays in
#pragma unroll
              for (int e = 16 * k; e < 16 * k + 16; ++e)
                x[e] = fmaf(__uint_as_float(sr[e]) * qmul, ks[k], -m);
            }
          }
          if (!full) {
            const uint32_t vis = (ptx::bit_range(pos - p.win + 1 - key0, pos + 1 - key0) |
                                  ptx::bit_range(0, min(p.sinks, pos + 1) - key0)) &
                                 ((have & 1u ? 0xffffu : 0u) | (have & 2u ? 0xffff0000u : 0u));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(vis >> e & 1u)) x[e] = -INFINITY;
          }
          float a0 = -INFINITY, a1 = -INFINITY;
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            a0 = ptx::max3(a0, x[e], x[e + 1]);
            a1 = ptx::max3(a1, x[e + 16], x[e + 17]);
          }
          float mx = fmaxf(a0, a1);
          // a row keeps its reference until a score passes it by the threshold (or
          // is its first); its threads meet only then
          float f = 1.f;
          auto passes = [&]() { return mx > kDpTau || (fresh && mx > -INFINITY); };
          if (ptx::named_bar_any(1 + quarter, 128, passes())) {
            mx = row_all(mx, [](float u, float v) { return fmaxf(u, v); });
            if (passes()) {
              f = fresh ? 0.f : ptx::ex2(-mx);   // (nothing so far: zeros, or NaN, which stays)
              fresh = false;
              m += mx;
              l *= f;
              a0 -= mx;
              a1 -= mx;
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] -= mx;
            }
          }
          // the unit of O: the tile's, until the scales are apart
          if (bits & 256u) {
            vs[0] *= unit;
            vs[1] *= unit;
            const float c = fmaxf(ptx::ex2(a0 - kDpTau) * fabsf(vs[0]), ptx::ex2(a1 - kDpTau) * fabsf(vs[1]));
            f = paged_row_unit(o_unit, f, row_all(c, [](float u, float v) { return fmaxf(u, v); }));
            const float per_unit = paged_per_unit(o_unit);
            vs[0] *= per_unit;
            vs[1] *= per_unit;
          } else if (unit != o_unit) {
            f *= o_unit * paged_per_unit(unit);
            o_unit = unit;
          }
          uint64_t acc = ptx::f2_pack(0.f, 0.f);
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint64_t r2 = ptx::f2_pack(vs[k], vs[k]);
#pragma unroll
            for (int e = 16 * k; e < 16 * k + 16; e += 2) {
              float p0, p1;
              const uint64_t pr = ptx::f2_pack(ptx::ex2(x[e]), ptx::ex2(x[e + 1]));
              acc = ptx::fadd2(acc, pr);
              ptx::f2_unpack(ptx::fmul2(pr, r2), p0, p1);
              pk[e / 2] = ptx::pack2<false>(p0, p1);
            }
          }
          float s0, s1;
          ptx::f2_unpack(acc, s0, s1);
          l += s0 + s1;
          // O and the other P are in use until the previous products are done
          if (i > 0 && __any_sync(0xffffffffu, f != 1.f)) {
            ptx::wait_bounded(bar(L::bPvDone + (b ^ 1)), (j - 1) >> 1 & 1, wd, kSiteDtPvDone);
            __syncwarp();
            ptx::tc_fence_after();
#pragma unroll 1
            for (int c = part * (D / 4); c < (part + 1) * (D / 4); c += 16) {
              uint32_t a[16];
              ptx::tmem_ld16(lanes + L::kOCol + c, a);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) a[e] = __float_as_uint(__uint_as_float(a[e]) * f);
              ptx::tmem_st16(lanes + L::kOCol + c, a);
            }
          }
          if (j >= 2) {
            ptx::wait_bounded(bar(L::bPvDone + b), (j - 2) >> 1 & 1, wd, kSiteDtPvDone);
            __syncwarp();
            ptx::tc_fence_after();
          }
          ptx::tmem_st16(lanes + L::p_col(b) + part * 16, pk);
          ptx::tmem_wait_st();
        } else if (j >= 2) {
          ptx::wait_bounded(bar(L::bPvDone + b), (j - 2) >> 1 & 1, wd, kSiteDtPvDone);
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(L::bPFull + b));
      }

      // ---- the unit's result or its part
      ptx::wait_bounded(bar(L::bPvDone + ((j - 1) & 1)), (j - 1) >> 1 & 1, wd, kSiteDtPvDone);
      __syncwarp();
      ptx::tc_fence_after();
      const int unit = static_cast<int>(head) * p.row_blocks + at.block;
      const size_t slot = 2 * static_cast<size_t>(run) + (pieces == 0 ? 0 : 1);
      if (has) {
        // (l is not negative: its sign carries the poison)
        float lt = row_all(copysignf(l, poison ? -1.f : 1.f), [](float u, float v) {
          return copysignf(fabsf(u) + fabsf(v), signbit(u) || signbit(v) ? -1.f : 1.f);
        });
        poison = signbit(lt);
        lt = fabsf(lt);
        const float inv = ptx::rcp(lt);
        const size_t row = head * p.R + row0 + r;
#pragma unroll 1
        for (int c = part * (D / 4); c < (part + 1) * (D / 4); c += 16) {
          uint32_t a[16];
          ptx::tmem_ld16(lanes + L::kOCol + c, a);
          ptx::tmem_wait_ld();
          float x[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            x[e] = __uint_as_float(a[e]) * inv * o_unit;
            if (lt == 0.f) x[e] = 0.f;
            if (poison) x[e] = NAN;
          }
          if (r < rows) {
            if (whole) {
              uint4* const out =
                  reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + row * D + c);
#pragma unroll
              for (int v = 0; v < 2; ++v)
                out[v] = make_uint4(ptx::pack2<kBf16>(x[8 * v], x[8 * v + 1]),
                                    ptx::pack2<kBf16>(x[8 * v + 2], x[8 * v + 3]),
                                    ptx::pack2<kBf16>(x[8 * v + 4], x[8 * v + 5]),
                                    ptx::pack2<kBf16>(x[8 * v + 6], x[8 * v + 7]));
            } else {
              float4* const out = p.part_o + (slot * p.slot_rows + r) * (D / 4) + c / 4;
#pragma unroll
              for (int v = 0; v < 2; ++v) {
                auto bits = [&](int e) {
                  return make_uint4(__float_as_uint(x[e]), __float_as_uint(x[e + 1]),
                                    __float_as_uint(x[e + 2]), __float_as_uint(x[e + 3]));
                };
                ptx::store32(out + 2 * v, bits(8 * v), bits(8 * v + 4));
              }
            }
          }
        }
        if (part == 0 && r < rows) {
          if (whole)
            p.lse[row] = lt != 0.f ? (ptx::lg2(lt) + m) * 0.693147180559945309f : -INFINITY;
          else
            p.part_ml[slot * p.slot_rows + r] = make_float2(m, lt);
        }
      }
      if (at.tile == 0 && threadIdx.x == 0)
        p.cut[unit] = whole ? make_int2(-1, 0)
                            : make_int2(static_cast<int>(slot),
                                        dec_run_of(deal, rn.start + done + s.tiles - 1));
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(L::bOFree));
    }
  }

  // ---------------------------------------------------------------- teardown
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kDtMma) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

}  // namespace fa
