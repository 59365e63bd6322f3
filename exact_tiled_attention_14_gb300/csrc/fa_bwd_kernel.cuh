// fa_bwd_kernel.cuh — gradients of exact attention for sm_103a (tcgen05 + TMEM + TMA).
//
// What it computes: dQ, dK, dV of sum(dO * O) for O = softmax(scale Q K^T) V
// (causal or not).  Like the forward pass, no N x N matrix is stored: the
// score and probability tiles are rebuilt from Q, K and the per-row LSE the
// forward pass emitted ("FlashAttention: The Matrix You Never Have to Write
// Down", section "The forward pass is only half of it"; "Why FlashAttention
// Can Avoid a Square Attention Array Without Making Attention Linear",
// section "Backward can recreate tiles instead of retaining the square").
// With P = exp(scale S - LSE) and D = rowsum(dO * O), the chain rule through
// the softmax gives, per (query tile i, key tile j):
//   dV_j += P^T dO_i,   dP = dO_i V_j^T,   dS = P * (dP - D),
//   dK_j += scale dS^T Q_i,   dQ_i += scale dS K_j.
//
// Two kernels, launched in this order on one stream:
//   fa_bwd_delta_kernel  D = rowsum(dO * O), memory-bound, one pass over O, dO.
//   fa_bwd_kernel        both tensor-core passes in one grid:
//   - dK/dV CTAs         one per (batch*head, key tile j): K_j, V_j stay in
//                        shared memory while Q_i and dO_i stream past; rebuilds
//                        S^T = K_j Q_i^T and dP^T = V_j dO_i^T on the tensor
//                        core, forms P^T and dS^T in registers, accumulates
//                        dV_j and dK_j in TMEM.
//   - dQ CTAs            one per (batch*head, query tile i): Q_i, dO_i stay
//                        while K_j and V_j stream past; rebuilds S and dP, forms
//                        dS, accumulates dQ_i in TMEM.
// Each gradient row is written by exactly one CTA, so there are no atomics
// and the result is deterministic; the price is that S and dP are formed
// twice (seven tile GEMMs per (i, j) instead of five).  fa_bwd_onepass.cuh
// holds the other trade: five tile GEMMs per pair, dQ summed in fp32 by the
// TMA engine in no fixed order.
//
// CTA layout (both tensor-core passes; the sliding-window variants' is
// below): warps 0-7 do the element-wise work, warp w on TMEM lanes 32*(w%4)
// .. +31 (key rows in dkdv, query rows in dq) and on column half w/4 of each
// 128-column tile, so a row's 128 scores are shared by two threads; warp 8
// issues the tcgen05 MMAs from one thread; warp 9 issues the TMA loads from
// one thread.  TMEM: S (or S^T) in columns 0-127, dP (dP^T) in 128-255, the
// fp32 accumulators from 256.  The streamed operands come through two rings:
// ring A holds the operand the last product of a tile still reads (Q_i in
// dkdv, K_j in dq), ring B the other one (dO_i, V_j), so B's slots free up
// earlier.
//
// Overlap.  The tensor core is kept busy while the element-wise warps work:
//   dkdv  the element-wise pass runs in two phases.  Phase 1 turns S^T_i into
//         P^T_i and writes it, 16-bit, over the S^T columns the same warp has
//         just read (the first half of each group's columns: 0-31 and
//         64-95); phase 2 does the same with dP^T_i and dS^T_i (columns
//         128-159 and 192-223).  The MMA thread
//         issues dV_j += P^T_i dO_i as soon as phase 1 is done, then S^T_{i+1},
//         then dK_j += dS^T_i Q_i once phase 2 is done, then dP^T_{i+1}: each
//         product that overwrites a 16-bit operand follows the one that reads
//         it in the thread's order.  Phase 1 of tile i+1 runs while the
//         tensor core works on dK_j and dP^T_{i+1}.
//   dq    dS goes to TMEM columns of its own (two buffers after dQ), so
//         S_{j+1} and dP_{j+1} are issued as soon as the element-wise warps
//         have read S_j and dP_j, and dQ_i += dS_j K_j when dS_j is written.
//
// Sliding-window calls (kWin: the query at position p sees the keys j <= p
// with j > p - win or j < sinks; H query heads share Hk key/value heads)
// walk only the tile pairs that hold a visible (query, key): a dQ item the
// sink tiles and the tiles of its rows' windows, a dK/dV item the query
// tiles of every head of its group that see the key tile.  There warps 0-15 do
// the element-wise work (four column groups of 32, so P^T and dS^T sit in four
// blocks of 16 columns, 32 apart; 8 warps measured 353 us where 16 take 339,
// B4 H16/4 N4096 d64 window 1024, and the same at d = 128), warp 16 issues and
// warp 17 loads.  The whole MMA warp walks the steps with one elected lane
// issuing, so that descriptors and conditions stay in uniform registers: with
// lane 0 walking alone the issue of a step's 16 to 32 products outlasted them
// (400 us against 343; d = 128, B1 H32/8 N16384 window 2048 64 sinks: 1520
// against 1400).  Measured on the present sources: 342 us (441 TFLOP/s of the
// visible pairs) and 1450 to 1460 us (910).  What bounds it: at d = 128 the chain S,
// dP, element-wise work of a tile beside 3 or 4 products of about 550 cycles
// (2400 and 2670 cycles a step), at d = 64 the element-wise work (about 2000
// of 2300 cycles).  Measured and not kept: an issuing warp for each of S and
// dP (1466, 346: dV and dQ get ahead of the S that the warps wait for), LSE
// and D staged through a barrier in shared memory (1419, 363), the two halves
// of a tile on barriers of their own (d = 64: 389).
#pragma once

#include <cuda.h>
#include <cstdint>

#include "fa_philox.cuh"
#include "ptx_sm103.cuh"

namespace fa {

// (of the variants without a window; see BwdRoles for theirs)
constexpr int kBwdThreads = 320;
constexpr int kBwdEwThreads = 256;       // element-wise warps 0-7
constexpr int kBwdMmaWarp = 8;
constexpr int kBwdLoadWarp = 9;
constexpr int kBwdTile = 128;            // rows of a query or key tile = TMEM lanes
constexpr uint32_t kBwdTmemCols = 512;
constexpr int kBwdNarrow = 32;           // keys of a sink tile worked on at that width

// Roles of the tensor-core kernel.  kGroups element-wise warps share a TMEM
// lane quarter, each on kCols of a tile's 128 columns.
template <bool kWin>
struct BwdRoles {
  static constexpr int kGroups = kWin ? 4 : 2;
  static constexpr int kCols = kBwdTile / kGroups;
  static constexpr int kEwThreads = kGroups * 128;
  static constexpr int kMmaWarp = kEwThreads / 32;
  static constexpr int kLoadWarp = kMmaWarp + 1;
  static constexpr int kThreads = kEwThreads + 64;
};

// The MMA warp.  kWin: every lane walks the loop and one elected lane issues
// (elected() is true in it), which keeps descriptors and addresses in uniform
// registers; a wait's outcome is the warp's.  Otherwise lane 0 walks alone.
template <bool kWin>
__device__ __forceinline__ bool bwd_elected() {
  return !kWin || ptx::elect_one();
}
template <bool kWin>
__device__ __forceinline__ int bwd_uniform(int x) {   // x is the same in every lane
  return kWin ? ptx::warp_same(x) : x;
}
template <bool kWin>
__device__ __forceinline__ bool bwd_warp_ok(bool ok) {
  return kWin ? ptx::warp_all(ok) : ok;
}

// Sites recorded in the status word when a wait of a backward kernel runs out.
enum BwdWaitSite : uint32_t {
  kSiteBwdEmpty = 20, kSiteBwdRes = 21, kSiteBwdFull = 22, kSiteBwdSFull = 23,
  kSiteBwdPFull = 24, kSiteBwdDone = 25, kSiteBwdDpFull = 26, kSiteBwdDsReady = 27,
  kSiteBwdDsFree = 28, kSiteBwdSFree = 29, kSiteBwdDqFull = 32, kSiteBwdDqFree = 33
};

struct BwdParams {
  CUtensorMap tm_q;    // [BH, N, d], boxes of 128 rows x 64 columns, 128-byte swizzle
  CUtensorMap tm_k;
  CUtensorMap tm_v;
  CUtensorMap tm_do;
  const float* lse;    // [BH, N] natural-log LSE of the scaled scores (forward output)
  const float* delta;  // [BH, N] rowsum(dO * O)
  void* dq;            // [BH, N, d]
  void* dk;
  void* dv;
  unsigned int* status;
  unsigned long long watchdog_cycles;
  int BH;
  int N;
  int n_tiles;         // ceil(N / 128)
  float scale;
  float scale_log2;    // scale * log2(e)
  // Dropout of the forward pass (kDrop variants only): keep threshold t,
  // seed words, offset and 256 / t.  The mask is regenerated from them:
  // dV += (P Z)^T dO and dS = P (Z dP 256/t - D), dV scaled by 256 / t.
  uint32_t drop_t;
  uint32_t drop_k0, drop_k1;
  uint32_t drop_off;
  float drop_scale;
  // Queries against a key set of another length (kKv variants; N and
  // n_tiles then count queries): Nk keys per head in n_ktiles tiles (K, V,
  // dK, dV are [BH, Nk, d]), per-batch key counts seqlens_k[b] (NULL: all
  // Nk; batch b = bh / H), and the causal alignment: align_br = 0 puts
  // query i at position i, 1 at len_b - N + i.  Square calls set
  // Nk = N, n_ktiles = n_tiles.
  int Nk;
  int n_ktiles;
  int H;
  const int* seqlens_k;
  int align_br;
  // Widths (kKv variants; square calls set both to D): width_qk of Q, K,
  // dQ, dK and width_v of V, dO, O, dV, each 64 or 128 with D the larger.
  // Each tensor map has its tensor's own width and only those 64-column
  // chunks are loaded; products over the head width take width_qk / 16 (S)
  // or width_v / 16 (dP) K steps, and dV is accumulated over width_v
  // columns, dK and dQ over width_qk.
  int width_qk;
  int width_v;
  // Packed variable-length batches (kKv variants with varlen = 1): Q, dO, O,
  // dQ token-major [total_q, H, d], K, V, dK, dV [Nk = total_k, H, d], LSE
  // [H, total_q] (as the forward writes it), D [total_q, H]; sequence b owns
  // query tokens cu_q[b] .. cu_q[b+1] - 1 and key tokens cu_k[b] ..
  // cu_k[b+1] - 1 (clamped to the totals).  N and n_tiles are then the
  // longest query count and its tiles, n_ktiles the longest key count's.
  // The tensor maps are (column, head, token).
  const int* cu_q;
  const int* cu_k;
  int varlen;
  int total_q;
  // One-pass kernel: dQ is accumulated, unscaled, in fp32 in blocks of 32
  // queries x 16 columns: block (bh, query tile qt, column block cb, row
  // quarter rq) holds element (column cc, row rr) at
  // dq_acc[((((bh * n_tiles + qt) * (width_qk / 16) + cb) * 4 + rq) * 16 + cc) * 32 + rr]
  // (dq_pad = n_tiles * 128 rows per head).  Zeroed before the launch and
  // converted to dQ by fa_bwd_dq_convert_kernel afterwards.
  float* dq_acc;
  int dq_pad;
  // Work items (key tiles of dK/dV or one-pass CTAs, query tiles of dQ
  // CTAs) are dealt in groups of item_group heads, tile by tile within a
  // group, so the CTAs at work share a few heads' streamed tiles in L2.
  int item_group;
  // Sliding window (kWin variants, which are kKv and kCausal): window and
  // sink counts (win >= 1), key/value heads per batch Hk (K, V, dK, dV are
  // [BHk, Nk, d]) and the G = H / Hk query heads that share each.
  int win;
  int sinks;
  int Hk;
  int G;
  int BHk;
  // Sink tiles (key tiles 0 .. split_tiles - 1 of each key/value head) are
  // seen by every later query tile, many times the steps of a window's tile,
  // so each is cut into split_parts items of equal steps that leave fp32 dK
  // and dV in split_ws ([BHk, split_tiles, split_parts, 128, 2 d]); a last
  // kernel adds the parts up in order.  split_tiles = 0: nothing is cut.
  int split_tiles;
  int split_parts;
  float* split_ws;
};

// Tile index and head of work item `blk` among BH * n_tiles items dealt in
// groups of p.item_group heads (the last group may be smaller).
__host__ __device__ __forceinline__ void bwd_item(const BwdParams& p, int blk, int n_tiles,
                                                  int& tile, int& bh) {
  const int per_group = p.item_group * n_tiles;
  const int g = blk / per_group, r = blk - g * per_group;
  const int left = p.BH - g * p.item_group;
  const int gh = p.item_group < left ? p.item_group : left;
  tile = r / gh;
  bh = g * p.item_group + (r - tile * gh);
}

// Where head bh's rows sit in a kKv call: its key count len and query
// offset off (query i at position i + off), its query count lenq, and with
// packed batches the first query and key token q0, k0.
struct BwdHead {
  int len, off, lenq, q0, k0;
};
__device__ __forceinline__ BwdHead bwd_kv_head(const BwdParams& p, int bh, bool causal) {
  BwdHead h;
  const int b = bh / p.H;
  h.lenq = p.N;
  h.q0 = 0;
  h.k0 = 0;
  if (p.varlen) {
    h.q0 = min(max(p.cu_q[b], 0), p.total_q);
    h.lenq = min(max(p.cu_q[b + 1], h.q0), p.total_q) - h.q0;
    h.k0 = min(max(p.cu_k[b], 0), p.Nk);
    h.len = min(max(p.cu_k[b + 1], h.k0), p.Nk) - h.k0;
  } else {
    h.len = p.seqlens_k ? p.seqlens_k[b] : p.Nk;
    h.len = min(max(h.len, 0), p.Nk);
  }
  h.off = (causal && p.align_br) ? h.len - h.lenq : 0;
  return h;
}

// Sliding window (kWin): one past the last query tile of a head (n_tiles in
// all, query i at position i + off) that sees a key of key tile kt of a
// batch of len keys.  Unless the tile holds a sink, the last query that sees
// its last key sits win - 1 positions after it.
__host__ __device__ __forceinline__ int bwd_win_q_end(int kt, int len, int off, int n_tiles,
                                                      int win, int sinks) {
  if (kt * kBwdTile < sinks) return n_tiles;
  const int key = (kt + 1) * kBwdTile < len ? (kt + 1) * kBwdTile - 1 : len - 1;
  const int last = key + win - 1 - off;
  if (last < 0) return 0;
  return last / kBwdTile + 1 < n_tiles ? last / kBwdTile + 1 : n_tiles;
}
// Sliding window: the key tiles that the query tile with rows r0 .. r1 - 1
// walks, of the n_end tiles up to its last row: ns sink tiles, then those
// from wa on, count in all.  Of the keys in them some row sees those below
// min(sinks, hi) and lo .. hi - 1.
struct BwdWinKeys {
  int ns, wa, count, lo, hi;
};
__host__ __device__ __forceinline__ BwdWinKeys bwd_win_keys(int r0, int r1, int len, int off,
                                                            int n_end, int win, int sinks) {
  BwdWinKeys k;
  const int used = sinks < len ? sinks : len;
  const int n_sink = (used + kBwdTile - 1) / kBwdTile;
  const int lo = r0 + off - win + 1, end = r1 + off;
  k.lo = lo > 0 ? lo : 0;
  k.hi = end < 0 ? 0 : (end < len ? end : len);
  k.ns = n_sink < n_end ? n_sink : n_end;
  k.wa = k.lo / kBwdTile > n_sink ? k.lo / kBwdTile : n_sink;
  k.count = k.ns + (n_end > k.wa ? n_end - k.wa : 0);
  return k;
}

// Row indices of head bh (h = bh % H): of query row qrow in Q, dO, dQ (rows
// of d values), of key row key in K, V, dK, dV, and of the query's LSE and D.
__device__ __forceinline__ long long bwd_qrow(const BwdParams& p, bool tok, const BwdHead& hd,
                                              int bh, long long qrow) {
  return tok ? (hd.q0 + qrow) * p.H + bh % p.H : static_cast<long long>(bh) * p.N + qrow;
}
__device__ __forceinline__ long long bwd_krow(const BwdParams& p, bool tok, const BwdHead& hd,
                                              int bh, long long key) {
  return tok ? (hd.k0 + key) * p.H + bh % p.H : static_cast<long long>(bh) * p.Nk + key;
}
__device__ __forceinline__ long long bwd_lse_at(const BwdParams& p, bool tok, const BwdHead& hd,
                                                int bh, long long qrow) {
  return tok ? static_cast<long long>(bh % p.H) * p.total_q + hd.q0 + qrow
             : static_cast<long long>(bh) * p.N + qrow;
}

// Shared memory of the tensor-core kernels: the resident pair of tiles
// (K_j, V_j or Q_i, dO_i), ring A and ring B of streamed tiles, in the
// one-pass kernel (kOne, fa_bwd_onepass.cuh) a 128 x 128 tile of dS and
// 32 KB of dQ staging blocks, kVecBytes of per-query vectors (dkdv: -LSE in
// log2 units and D of the current query tile), the ring barriers and ten
// kernel-specific barriers.  The dS tile and the staging blocks take the
// room of ring stages.
template <int D, int kVecBytes, bool kOne = false>
struct BwdSmem {
  static constexpr int kChunks = D / 64;
  static constexpr int kTile = kBwdTile * D * 2;
  static constexpr int kChunkBytes = kBwdTile * 128;
  static constexpr int kStagesA = (D == 128) ? (kOne ? 2 : 3) : (kOne ? 4 : 6);
  static constexpr int kStagesB = (D == 128) ? (kOne ? 1 : 2) : (kOne ? 3 : 4);
  static constexpr int kRes = 0;
  static constexpr int kRingA = kRes + 2 * kTile;
  static constexpr int kRingB = kRingA + kStagesA * kTile;
  static constexpr int kDs = kRingB + kStagesB * kTile;   // 1024-aligned like the tiles
  static constexpr int kStg = kDs + (kOne ? kBwdTile * kBwdTile * 2 : 0);
  static constexpr int kStgBytes = 32 * 1024;
  static constexpr int kVec = kStg + (kOne ? kStgBytes : 0);
  static constexpr int kBar = kVec + kVecBytes;
  static constexpr int bFullA = 0, bEmptyA = kStagesA, bFullB = 2 * kStagesA,
                       bEmptyB = bFullB + kStagesB, bRes = bEmptyB + kStagesB, bX = bRes + 1,
                       kNumBars = bX + 10;
  static constexpr int kMisc = kBar + 8 * kNumBars;   // tmem base, abort flag
  static constexpr int kBytes = kMisc + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kAlloc <= 232448, "shared memory budget");
};

// Kernel-specific barriers (offsets from bX).
struct DkdvBars {
  static constexpr int kSFull = 0, kDpFull = 1, kPReady = 2, kDsReady = 3, kDone = 4;
  static constexpr int kDqFull = 5, kDqFree = 7;   // one-pass kernel: two each (per dQ buffer)
};
struct DqBars {
  static constexpr int kSFull = 0, kSFree = 1, kPFull = 2, kDsFree = 4, kDone = 6;   // PFull, DsFree: 2 each
};

// ---------------------------------------------------------------- D = rowsum(dO * O)
// Each row is read as 16-byte pieces (8 values), D/8 consecutive threads per
// row, reduced with shuffles.  The loop runs warp-uniformly so every lane
// takes part in every shuffle.
template <int D, bool kBf16>
__global__ void __launch_bounds__(256) fa_bwd_delta_kernel(const uint4* __restrict__ o,
                                                           const uint4* __restrict__ dout,
                                                           float* __restrict__ delta,
                                                           long long rows) {
  // the tensor-core grid may be scheduled once every CTA here has started:
  // its prologue and first loads overlap this pass, and its element-wise
  // warps wait for D before reading it
  ptx::griddep_launch_dependents();
  constexpr int kPer = D / 8;   // threads per row
  const long long total = rows * kPer;
  const int lane = threadIdx.x & 31;
  const long long warp_id = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const long long nwarps = (static_cast<long long>(gridDim.x) * blockDim.x) >> 5;
  for (long long base = warp_id * 32; base < total; base += nwarps * 32) {
    const long long idx = base + lane;
    float acc = 0.f;
    if (idx < total) {
      const uint4 a = o[idx], b = dout[idx];
      const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float a0, a1, b0, b1;
        ptx::unpack2<kBf16>(av[e], a0, a1);
        ptx::unpack2<kBf16>(bv[e], b0, b1);
        acc = fmaf(a0, b0, acc);
        acc = fmaf(a1, b1, acc);
      }
    }
#pragma unroll
    for (int off = kPer / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if (idx < total && (lane % kPer) == 0) delta[idx / kPer] = acc;
  }
}

// ---------------------------------------------------------------- dQ = scale * accumulator
// The one-pass kernel leaves dQ unscaled in fp32 in blocks of 32 queries x
// 16 columns, column by column within a block (BwdParams::dq_acc); the
// blocks of one (batch*head, 128-query tile) are contiguous, 128 x W floats.
// One CTA per (batch*head, query tile) moves them, 64 columns at a time,
// through a shared-memory tile with 16-byte loads and writes the rows in
// the storage dtype, scaled, with 16-byte stores.  Blocks: bh * n_tiles +
// query tile.
template <bool kBf16>
__global__ void __launch_bounds__(256) fa_bwd_dq_convert_kernel(const float* __restrict__ acc,
                                                                uint32_t* __restrict__ dq,
                                                                int N, int W, int pad,
                                                                float scale) {
  __shared__ float tile[kBwdTile][65];
  const int n_tiles = pad / kBwdTile;
  const int bh = blockIdx.x / n_tiles;
  const int qt = blockIdx.x - bh * n_tiles;
  const float4* src = reinterpret_cast<const float4*>(
      acc + (static_cast<long long>(bh) * n_tiles + qt) * kBwdTile * W);
  for (int h = 0; h < W / 64; ++h) {
    // blocks cb = 4h .. 4h + 3 of the tile: 4 x 4 blocks of 512 floats
    const float4* s4 = src + h * (4 * 4 * 512 / 4);
    for (int idx = threadIdx.x; idx < 4 * 4 * 512 / 4; idx += 256) {
      const float4 v = s4[idx];
      const int e = idx * 4;                          // float index within the half
      const int blk = e >> 9, in = e & 511;           // block (cb - 4h) * 4 + rq, offset
      const int cc = in >> 5, rr = in & 31;           // column within the block, row
      const int row = (blk & 3) * 32 + rr, col = (blk >> 2) * 16 + cc;
      tile[row][col] = v.x;
      tile[row + 1][col] = v.y;
      tile[row + 2][col] = v.z;
      tile[row + 3][col] = v.w;
    }
    __syncthreads();
    // 128 rows x 8 pieces of 8 columns
    for (int idx = threadIdx.x; idx < kBwdTile * 8; idx += 256) {
      const int r = idx >> 3, c8 = (idx & 7) * 8;
      const int q = qt * kBwdTile + r;
      if (q < N) {
        uint4 out;
        out.x = ptx::pack2<kBf16>(tile[r][c8] * scale, tile[r][c8 + 1] * scale);
        out.y = ptx::pack2<kBf16>(tile[r][c8 + 2] * scale, tile[r][c8 + 3] * scale);
        out.z = ptx::pack2<kBf16>(tile[r][c8 + 4] * scale, tile[r][c8 + 5] * scale);
        out.w = ptx::pack2<kBf16>(tile[r][c8 + 6] * scale, tile[r][c8 + 7] * scale);
        *reinterpret_cast<uint4*>(dq + (static_cast<long long>(bh) * N + q) * (W / 2) +
                                  (h * 64 + c8) / 2) = out;
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- shared pieces
// TMEM columns.
constexpr uint32_t kColS = 0, kColDp = 128, kColAcc = 256;

// Issue A (K-major, shared memory) x B^T (K-major) over the head width into
// d_tmem: M = N = 128, K = D in steps of 16 columns.
template <int D, int Chunk>
__device__ __forceinline__ void issue_kmajor(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                             uint32_t idesc, int steps = D / 16) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    if (kk >= steps) break;
    const uint32_t off = static_cast<uint32_t>((kk >> 2) * Chunk + (kk & 3) * 32) >> 4;
    ptx::mma_ss(d_tmem, ptx::desc_sw128(a_lo + off), ptx::desc_sw128(b_lo + off), idesc, kk > 0);
  }
}

// Issue A (16-bit, in TMEM, 128 rows x 128 along K) x B (MN-major tile of 128
// rows along K, D columns) into d_tmem (N = D).  A's 64 packed columns sit
// in kBlocks equal blocks, 128 / kBlocks columns apart (more than one: a
// 16-bit tile written over the fp32 columns that each group of warps read).
// `narrow`: the first kBwdNarrow along K only.
template <int kBlocks>
__device__ __forceinline__ void issue_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                             uint32_t idesc, uint32_t acc, bool narrow = false) {
#pragma unroll
  for (int kk = 0; kk < kBwdTile / 16; ++kk) {
    if (kk == kBwdNarrow / 16 && narrow) break;
    constexpr int kPer = 8 / kBlocks;   // K steps of a block
    const uint32_t acol = kk / kPer * (kBwdTile / kBlocks) + kk % kPer * 8;
    ptx::mma_ts(d_tmem, a_tmem + acol, ptx::desc_sw128(b_lo + kk * (2048 >> 4)), idesc,
                kk > 0 ? 1u : acc);
  }
}

// Issue A (K-major, shared memory, 128 rows x 128 along K in two 64-column
// chunks) x B (MN-major tile of 128 rows along K) into d_tmem.
template <int Chunk>
__device__ __forceinline__ void issue_smem_a(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                             uint32_t idesc, uint32_t acc) {
#pragma unroll
  for (int kk = 0; kk < kBwdTile / 16; ++kk) {
    const uint32_t aoff = static_cast<uint32_t>((kk >> 2) * Chunk + (kk & 3) * 32) >> 4;
    ptx::mma_ss(d_tmem, ptx::desc_sw128(a_lo + aoff), ptx::desc_sw128(b_lo + kk * (2048 >> 4)),
                idesc, kk > 0 ? 1u : acc);
  }
}

// Issue A x B with both operands MN-major in shared memory (128 rows along
// K each, 16 rows = 2 KB per K step) into a fresh accumulator at d_tmem.
__device__ __forceinline__ void issue_mn_mn(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                            uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < kBwdTile / 16; ++kk)
    ptx::mma_ss(d_tmem, ptx::desc_sw128(a_lo + kk * (2048 >> 4)),
                ptx::desc_sw128(b_lo + kk * (2048 >> 4)), idesc, kk > 0 ? 1u : 0u);
}

// Instruction-descriptor bit that marks A as MN-major (kind::f16).
constexpr uint32_t kIdescAMnMajor = 1u << 15;

// Element-wise fp32 addition of `bytes` (a multiple of 16) of shared memory
// into global memory by the TMA engine, in this thread's bulk group.
__device__ __forceinline__ void bulk_reduce_add_f32(float* gdst, uint32_t ssrc, uint32_t bytes) {
  asm volatile(
      "cp.reduce.async.bulk.global.shared::cta.bulk_group.add.f32 [%0], [%1], %2;\n\t"
      "cp.async.bulk.commit_group;" ::"l"(gdst),
      "r"(ssrc), "r"(bytes)
      : "memory");
}
// Wait until this thread's bulk groups have finished reading shared memory
// (the source may be overwritten), or have completed entirely.
__device__ __forceinline__ void bulk_wait_read_all() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// One-pass kernel: TMEM column of dQ buffer b.  At d = 128 TMEM holds S^T,
// dP^T, dV and dK (512 columns), so the single dQ buffer takes the dP^T
// columns once the element-wise warps have read them; at d = 64 two
// buffers of 64 columns follow dV and dK.
template <int D>
struct DqBuf {
  static constexpr int kBufs = (D == 128) ? 1 : 2;
  static __device__ __forceinline__ uint32_t col(int b) {
    return D == 128 ? kColDp : kColAcc + 2u * D + 64u * b;
  }
};

// Zero rows [r0, r1) of a 128-row tile (64-column chunks of 128-byte rows),
// 16 bytes at a time, by threads tid of nthreads.  The swizzle permutes the
// 16-byte pieces within a row, so whole rows need no address arithmetic.
__device__ __forceinline__ void zero_rows(uint8_t* tile, int chunks, int r0, int r1, int tid,
                                          int nthreads) {
  for (int i = r0 * 8 + tid; i < r1 * 8; i += nthreads)
    for (int c = 0; c < chunks; ++c)
      *reinterpret_cast<uint4*>(tile + c * (kBwdTile * 128) + i * 16) = make_uint4(0u, 0u, 0u, 0u);
}

// Write columns [c0, c0 + nc) (nc a multiple of 32) of one row of a TMEM
// accumulator (fp32), times `mul`, to global memory in the storage dtype, in
// rows of `width` values (rows past N are skipped).
template <bool kBf16>
__device__ __forceinline__ void store_acc_cols(uint32_t t_acc, int c0, int nc, int width, float mul,
                                               void* base, long long row, bool in_range) {
  uint4* out = reinterpret_cast<uint4*>(static_cast<uint8_t*>(base) + row * (width * 2) + c0 * 2);
#pragma unroll 1
  for (int q4 = 0; q4 < nc / 32; ++q4) {
    uint32_t r[32];
    ptx::tmem_ld32(t_acc + c0 + q4 * 32, r);
    ptx::tmem_wait_ld();
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e)
      pk[e] = ptx::pack2<kBf16>(__uint_as_float(r[2 * e]) * mul, __uint_as_float(r[2 * e + 1]) * mul);
    if (in_range) {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        out[q4 * 4 + v] = make_uint4(pk[4 * v], pk[4 * v + 1], pk[4 * v + 2], pk[4 * v + 3]);
    }
  }
}

// Columns [c0, c0 + nc) (nc a multiple of 32) of one row of a TMEM
// accumulator, times `mul`, to the fp32 row `out` (16-byte aligned).
__device__ __forceinline__ void store_acc_f32(uint32_t t_acc, int c0, int nc, float mul, float* out) {
#pragma unroll 1
  for (int c = c0; c < c0 + nc; c += 32) {
    uint32_t r[32];
    ptx::tmem_ld32(t_acc + c, r);
    ptx::tmem_wait_ld();
#pragma unroll
    for (int v = 0; v < 8; ++v)
      reinterpret_cast<float4*>(out + c)[v] =
          make_float4(__uint_as_float(r[4 * v]) * mul, __uint_as_float(r[4 * v + 1]) * mul,
                      __uint_as_float(r[4 * v + 2]) * mul, __uint_as_float(r[4 * v + 3]) * mul);
  }
}

// Adds up the parts of the cut sink tiles (BwdParams::split_ws) in their order
// and writes dK and dV in the storage dtype: one thread per 4 columns of a
// row's dK and dV, blocks over (head, sink tile).
template <int D, bool kBf16>
__global__ void __launch_bounds__(256) fa_bwd_win_parts_kernel(const __grid_constant__ BwdParams p) {
  constexpr int kPer = 2 * D / 4;   // threads of a row
  const int bh = blockIdx.x / p.split_tiles, kt = blockIdx.x % p.split_tiles;
  const int r = blockIdx.y * (256 / kPer) + threadIdx.x / kPer, c = threadIdx.x % kPer * 4;
  const long long key = static_cast<long long>(kt) * kBwdTile + r;
  if (key >= p.Nk) return;
  const float4* src = reinterpret_cast<const float4*>(
      p.split_ws + (static_cast<size_t>(blockIdx.x) * p.split_parts * kBwdTile + r) * (2 * D) + c);
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int i = 0; i < p.split_parts; ++i) {
    const float4 x = src[static_cast<size_t>(i) * (kBwdTile * 2 * D / 4)];
    a.x += x.x;
    a.y += x.y;
    a.z += x.z;
    a.w += x.w;
  }
  uint16_t* out = static_cast<uint16_t*>(c < D ? p.dk : p.dv) +
                  (static_cast<size_t>(bh) * p.Nk + key) * D + c % D;
  *reinterpret_cast<uint2*>(out) =
      make_uint2(ptx::pack2<kBf16>(a.x, a.y), ptx::pack2<kBf16>(a.z, a.w));
}

// Shared setup of one work item of the tensor-core grid: the ring barriers
// and, through `init_x(bar)`, the item's own barriers, initialised by one
// thread (the load thread without a window).  The CTA's TMEM is allocated once for all its items.
template <class L, class InitX>
__device__ __forceinline__ void bwd_setup(uint32_t sbase, uint8_t* sgen, InitX init_x) {
  if (threadIdx.x == kBwdLoadWarp * 32) {
    *reinterpret_cast<volatile int*>(sgen + L::kMisc + 4) = 0;
    auto bar = [&](int i) -> uint32_t { return sbase + L::kBar + 8u * i; };
    for (int s = 0; s < L::kStagesA; ++s) {
      ptx::mbar_init(bar(L::bFullA + s), 1);
      ptx::mbar_init(bar(L::bEmptyA + s), 1);
    }
    for (int s = 0; s < L::kStagesB; ++s) {
      ptx::mbar_init(bar(L::bFullB + s), 1);
      ptx::mbar_init(bar(L::bEmptyB + s), 1);
    }
    ptx::mbar_init(bar(L::bRes), 1);
    init_x(bar);
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
}

// End of one work item: every role is done (the MMA thread has seen its
// last commit, the load thread its last copy), so the thread that set them up
// invalidates the item's barriers; the next item, whose layout may put
// other data there, initialises its own.
template <class L>
__device__ __forceinline__ void bwd_teardown(uint32_t sbase) {
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (threadIdx.x == kBwdLoadWarp * 32)
    for (int i = 0; i < L::kNumBars; ++i) ptx::mbar_inval(sbase + L::kBar + 8u * i);
}

// The load thread: the resident pair (res_a, res_b at tile `res_tile`), then
// tiles first .. first + count - 1 of str_a into ring A and of str_b into
// ring B, in the order A_0, B_0, A_1, B_1, ...  The "a" tensors (K and Q)
// have chunks_a 64-column chunks, the "b" tensors (V and dO) chunks_b; only
// those are loaded.
template <class L>
__device__ __forceinline__ void bwd_producer(uint32_t sbase, const CUtensorMap* res_a,
                                             const CUtensorMap* res_b, int res_tile,
                                             const CUtensorMap* str_a, const CUtensorMap* str_b,
                                             int first, int count, int bh,
                                             const ptx::Watchdog& wd, int tok_h = -1,
                                             int res_tok0 = 0, int str_tok0 = 0,
                                             int chunks_a = L::kChunks, int chunks_b = L::kChunks) {
  auto bar = [&](int i) -> uint32_t { return sbase + L::kBar + 8u * i; };
  bool alive = true;
  // tile `tile` of a [BH, rows, d] map: (column, row, batch*head); with
  // packed batches (tok_h = head) of a (column, head, token) map from token
  // tok0 on
  auto y_of = [&](int tile, int tok0) { return tok_h < 0 ? tile * kBwdTile : tok_h; };
  auto z_of = [&](int tile, int tok0) { return tok_h < 0 ? bh : tok0 + tile * kBwdTile; };
  ptx::mbar_arrive_expect_tx(bar(L::bRes), (chunks_a + chunks_b) * L::kChunkBytes);
  for (int c = 0; c < chunks_a; ++c)
    ptx::tma_load_3d(sbase + L::kRes + c * L::kChunkBytes, res_a, bar(L::bRes), c * 64,
                     y_of(res_tile, res_tok0), z_of(res_tile, res_tok0));
  for (int c = 0; c < chunks_b; ++c)
    ptx::tma_load_3d(sbase + L::kRes + L::kTile + c * L::kChunkBytes, res_b, bar(L::bRes), c * 64,
                     y_of(res_tile, res_tok0), z_of(res_tile, res_tok0));
  // one tile of `tm` into slot `slot` of a ring, once its previous use is over
  auto load = [&](const CUtensorMap* tm, int ring, int full0, int empty0, int stages, int it,
                  int chunks) {
    const int slot = it % stages, use = it / stages;
    if (use > 0)
      alive = ptx::wait_bounded(bar(empty0 + slot), (use - 1) & 1, wd, kSiteBwdEmpty) && alive;
    if (!alive) return;
    const uint32_t dst = sbase + ring + slot * L::kTile;
    ptx::mbar_arrive_expect_tx(bar(full0 + slot), chunks * L::kChunkBytes);
    for (int c = 0; c < chunks; ++c)
      ptx::tma_load_3d(dst + c * L::kChunkBytes, tm, bar(full0 + slot), c * 64,
                       y_of(first + it, str_tok0), z_of(first + it, str_tok0));
  };
  int loads = 0;
  for (int it = 0; it < count && alive; ++it) {
    load(str_a, L::kRingA, L::bFullA, L::bEmptyA, L::kStagesA, it, chunks_a);
    if (!alive) break;
    load(str_b, L::kRingB, L::bFullB, L::bEmptyB, L::kStagesB, it, chunks_b);
    if (!alive) {   // tile `it` of ring A was issued: drain it too
      ptx::wait_drain(bar(L::bFullA + it % L::kStagesA), (it / L::kStagesA) & 1, 200000000ull);
      break;
    }
    ++loads;
  }
  // Drain: every issued copy has landed before the CTA can exit.
  const unsigned long long drain = 200000000ull;
  ptx::wait_drain(bar(L::bRes), 0, drain);
  for (int l = loads > L::kStagesA ? loads - L::kStagesA : 0; l < loads; ++l)
    ptx::wait_drain(bar(L::bFullA + l % L::kStagesA), (l / L::kStagesA) & 1, drain);
  for (int l = loads > L::kStagesB ? loads - L::kStagesB : 0; l < loads; ++l)
    ptx::wait_drain(bar(L::bFullB + l % L::kStagesB), (l / L::kStagesB) & 1, drain);
}

// The same with tiles named by functions: res(y, z) and str(it, y, z) give
// the row and head coordinates of the resident pair and of the it-th
// streamed pair (kWin: tiles and heads are not consecutive).
template <class L, class Res, class Str>
__device__ __forceinline__ void bwd_producer_map(uint32_t sbase, const CUtensorMap* res_a,
                                                 const CUtensorMap* res_b, Res res,
                                                 const CUtensorMap* str_a,
                                                 const CUtensorMap* str_b, Str str, int count,
                                                 const ptx::Watchdog& wd) {
  auto bar = [&](int i) -> uint32_t { return sbase + L::kBar + 8u * i; };
  int y, z;
  res(y, z);
  ptx::mbar_arrive_expect_tx(bar(L::bRes), 2 * L::kTile);
  for (int c = 0; c < L::kChunks; ++c) {
    ptx::tma_load_3d(sbase + L::kRes + c * L::kChunkBytes, res_a, bar(L::bRes), c * 64, y, z);
    ptx::tma_load_3d(sbase + L::kRes + L::kTile + c * L::kChunkBytes, res_b, bar(L::bRes), c * 64,
                     y, z);
  }
  int na = 0, nb = 0;   // tiles issued into ring A / B
  for (int it = 0; it < count; ++it) {
    str(it, y, z);
    const int sa = it % L::kStagesA, ua = it / L::kStagesA;
    if (ua > 0 && !ptx::wait_bounded(bar(L::bEmptyA + sa), (ua - 1) & 1, wd, kSiteBwdEmpty)) break;
    ptx::mbar_arrive_expect_tx(bar(L::bFullA + sa), L::kTile);
    for (int c = 0; c < L::kChunks; ++c)
      ptx::tma_load_3d(sbase + L::kRingA + sa * L::kTile + c * L::kChunkBytes, str_a,
                       bar(L::bFullA + sa), c * 64, y, z);
    ++na;
    const int sb = it % L::kStagesB, ub = it / L::kStagesB;
    if (ub > 0 && !ptx::wait_bounded(bar(L::bEmptyB + sb), (ub - 1) & 1, wd, kSiteBwdEmpty)) break;
    ptx::mbar_arrive_expect_tx(bar(L::bFullB + sb), L::kTile);
    for (int c = 0; c < L::kChunks; ++c)
      ptx::tma_load_3d(sbase + L::kRingB + sb * L::kTile + c * L::kChunkBytes, str_b,
                       bar(L::bFullB + sb), c * 64, y, z);
    ++nb;
  }
  // Drain: every issued copy has landed before the CTA can exit.
  const unsigned long long drain = 200000000ull;
  ptx::wait_drain(bar(L::bRes), 0, drain);
  for (int l = na > L::kStagesA ? na - L::kStagesA : 0; l < na; ++l)
    ptx::wait_drain(bar(L::bFullA + l % L::kStagesA), (l / L::kStagesA) & 1, drain);
  for (int l = nb > L::kStagesB ? nb - L::kStagesB : 0; l < nb; ++l)
    ptx::wait_drain(bar(L::bFullB + l % L::kStagesB), (l / L::kStagesB) & 1, drain);
}

// ---------------------------------------------------------------- dK, dV
// Per-query vectors of the dkdv kernel: one buffer at d = 128 (shared memory
// is full), two at d = 64.
template <int D>
struct DkdvVec {
  static constexpr int kBufs = (D == 128) ? 1 : 2;
  static constexpr int kBytes = kBufs * 2 * kBwdTile * 4;
};

// One CTA of the dK/dV pass: block `blk` of BH * n_tiles.
template <int D, bool kBf16, bool kCausal, bool kDrop, bool kKv, bool kWin = false>
__device__ __forceinline__ void bwd_dkdv_cta(const BwdParams& p, int blk, uint32_t tmem_base) {
  using L = BwdSmem<D, DkdvVec<D>::kBytes>;
  using X = DkdvBars;
  using W = BwdRoles<kWin>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = ptx::smem_u32(smem_raw);
  const uint32_t sbase = (raw_base + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - raw_base);
  const int warp = bwd_uniform<kWin>(threadIdx.x >> 5), lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return sbase + L::kBar + 8u * i; };
  auto xbar = [&](int i) -> uint32_t { return bar(L::bX + i); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sgen + L::kMisc + 4);

  // Key tile kt of head bh; for causal runs the first key tiles of a group
  // of heads (the most query tiles to visit) are dealt first.
  int kt, bh;                                // kWin: bh is the key/value head
  int part = 0, parts = 1;                   // kWin: of a cut sink tile
  if constexpr (kWin) {
    const int cut = p.BHk * p.split_tiles * p.split_parts;
    if (blk < cut) {
      parts = p.split_parts;
      part = blk % parts;
      kt = blk / parts % p.split_tiles;
      bh = blk / (parts * p.split_tiles);
    } else {
      const int rest = p.n_ktiles - p.split_tiles;
      bh = (blk - cut) / rest;
      kt = p.split_tiles + (blk - cut) - bh * rest;
    }
  } else {
    bwd_item(p, blk, p.n_ktiles, kt, bh);
  }
  int i0 = kCausal ? kt : 0;                 // query tiles i >= kt see this key tile
  int len = p.N, off = 0;                    // keys of this head, query offset (kKv)
  int n_q = p.n_tiles;                       // query tiles of this head
  const bool tok = kKv && p.varlen;          // packed batch: token-major rows
  BwdHead hd{p.N, 0, p.N, 0, 0};
  if constexpr (kKv) {
    // the first query that sees key kt * 128 sits at row kt * 128 - off
    hd = bwd_kv_head(p, kWin ? bh / p.Hk * p.H : bh, kCausal);
    len = hd.len;
    off = hd.off;
    if (tok) n_q = (hd.lenq + kBwdTile - 1) / kBwdTile;
    const int first = kt * kBwdTile - off;
    i0 = !kCausal || first <= 0 ? 0 : first / kBwdTile;
    if (kt * kBwdTile >= len) i0 = n_q;      // padding: no query sees these keys
  }
  if constexpr (kWin) n_q = bwd_win_q_end(kt, len, off, n_q, p.win, p.sinks);
  // key rows this CTA owns: padded keys are written (as zeros); a packed
  // sequence's rows end at its key count
  const int key_rows = tok ? len : p.Nk;
  const int q_rows = tok ? hd.lenq : p.N;
  // Steps: the query tiles i0 .. n_q - 1; kWin: of every head that reads this
  // one, head after head, and of those the part's share.
  const int nq1 = n_q - i0;
  int nq = nq1, it0 = 0;
  if constexpr (kWin) {
    const int all = max(nq1, 0) * p.G;
    it0 = static_cast<int>(static_cast<long long>(all) * part / parts);
    nq = static_cast<int>(static_cast<long long>(all) * (part + 1) / parts) - it0;
  }
  struct Step {
    int tile, head;   // query tile and head
  };
  auto first_step = [&]() -> Step {
    if constexpr (kWin) {
      if (nq <= 0) return {0, 0};
      const int g = it0 / nq1;
      return {i0 + it0 - g * nq1, bh / p.Hk * p.H + bh % p.Hk * p.G + g};
    }
    return {i0, bh};
  };
  auto next_step = [&](Step& x) {
    if (++x.tile == n_q && kWin) {
      x.tile = i0;
      ++x.head;
    }
  };
  // a cut tile's part: rows of dK (d floats) and dV
  float* part_ws = nullptr;
  if constexpr (kWin) {
    if (parts > 1)
      part_ws = p.split_ws + ((static_cast<size_t>(bh) * p.split_tiles + kt) * parts + part) *
                                 (kBwdTile * 2 * D);
  }
  if (kWin && nq <= 0 && part_ws != nullptr) {
    for (int i = threadIdx.x; i < kBwdTile * 2 * D / 4; i += W::kThreads)
      reinterpret_cast<float4*>(part_ws)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    return;
  }
  if (kKv && nq <= 0) {
    // no query sees this key tile: its dK and dV rows are zero
    if (threadIdx.x < 256) {
      const int t = threadIdx.x & 127;
      const long long key = static_cast<long long>(kt) * kBwdTile + t;
      if (key < key_rows) {
        const int width = threadIdx.x < 128 ? p.width_v : p.width_qk;
        uint4* row = reinterpret_cast<uint4*>(static_cast<uint8_t*>(threadIdx.x < 128 ? p.dv : p.dk) +
                                              bwd_krow(p, tok, hd, bh, key) * (width * 2));
        for (int c = 0; c < width / 8; ++c) row[c] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    return;
  }

  bwd_setup<L>(sbase, sgen, [&](auto b) {
    ptx::mbar_init(b(L::bX + X::kSFull), 1);
    ptx::mbar_init(b(L::bX + X::kDpFull), 1);
    ptx::mbar_init(b(L::bX + X::kPReady), W::kEwThreads);
    ptx::mbar_init(b(L::bX + X::kDsReady), W::kEwThreads);
    ptx::mbar_init(b(L::bX + X::kDone), 1);
  });
  const ptx::Watchdog wd{p.watchdog_cycles, abort_flag, p.status};

  if (warp == W::kLoadWarp) {
    if constexpr (kWin) {
      if (lane == 0) {
        Step at = first_step();
        bwd_producer_map<L>(
            sbase, &p.tm_k, &p.tm_v, [&](int& y, int& z) { y = kt * kBwdTile; z = bh; }, &p.tm_q,
            &p.tm_do,
            [&](int, int& y, int& z) {
              y = at.tile * kBwdTile;
              z = at.head;
              next_step(at);
            },
            nq, wd);
      }
    } else if (lane == 0) {
      bwd_producer<L>(sbase, &p.tm_k, &p.tm_v, kt, &p.tm_q, &p.tm_do, i0, nq, bh, wd,
                      tok ? bh % p.H : -1, hd.k0, hd.q0, p.width_qk / 64, p.width_v / 64);
    }
    __syncwarp();
  } else if (warp == W::kMmaWarp) {
    if (kWin || lane == 0) {
      const uint32_t tmem = bwd_uniform<kWin>(tmem_base);
      const int n = bwd_uniform<kWin>(nq);
      constexpr int fmt = kBf16 ? 1 : 0;
      constexpr uint32_t idesc_s = ptx::idesc_f16(kBwdTile, kBwdTile, fmt, 0);
      // dV has width_v columns, dK width_qk
      const uint32_t idesc_dv = ptx::idesc_f16(kBwdTile, kWin ? D : p.width_v, fmt, 1);
      const uint32_t idesc_dk = ptx::idesc_f16(kBwdTile, kWin ? D : p.width_qk, fmt, 1);
      const int steps_s = kWin ? D / 16 : p.width_qk / 16;
      const int steps_dp = kWin ? D / 16 : p.width_v / 16;
      constexpr uint32_t kSlotLo = L::kTile >> 4;
      const uint32_t k_lo = ptx::desc_lo(sbase + L::kRes, 16);
      const uint32_t v_lo = ptx::desc_lo(sbase + L::kRes + L::kTile, 16);
      const uint32_t q_lo0 = ptx::desc_lo(sbase + L::kRingA, 16);                  // K-major use
      const uint32_t do_lo0 = ptx::desc_lo(sbase + L::kRingB, 16);
      const uint32_t q_mn0 = ptx::desc_lo(sbase + L::kRingA, L::kChunkBytes);      // MN-major use
      const uint32_t do_mn0 = ptx::desc_lo(sbase + L::kRingB, L::kChunkBytes);
      const uint32_t tS = tmem + kColS, tDp = tmem + kColDp;
      const uint32_t tDv = tmem + kColAcc, tDk = tmem + kColAcc + D;
      auto full_a = [&](int it) {
        return ptx::wait_bounded(bar(L::bFullA + it % L::kStagesA), (it / L::kStagesA) & 1, wd,
                                 kSiteBwdFull);
      };
      auto full_b = [&](int it) {
        return ptx::wait_bounded(bar(L::bFullB + it % L::kStagesB), (it / L::kStagesB) & 1, wd,
                                 kSiteBwdFull);
      };
      // S^T = K_j Q_i^T and dP^T = V_j dO_i^T (keys on the TMEM lanes)
      auto issue_s = [&](int it) {
        if (!bwd_elected<kWin>()) return;
        issue_kmajor<D, L::kChunkBytes>(tS, k_lo, q_lo0 + (it % L::kStagesA) * kSlotLo, idesc_s,
                                        steps_s);
        ptx::mma_commit(xbar(X::kSFull));
      };
      auto issue_dp = [&](int it) {
        if (!bwd_elected<kWin>()) return;
        issue_kmajor<D, L::kChunkBytes>(tDp, v_lo, do_lo0 + (it % L::kStagesB) * kSlotLo, idesc_s,
                                        steps_dp);
        ptx::mma_commit(xbar(X::kDpFull));
      };
      bool alive = bwd_warp_ok<kWin>(ptx::wait_bounded(bar(L::bRes), 0, wd, kSiteBwdRes) &&
                                     full_a(0) && full_b(0));
      ptx::tc_fence_after();
      if (alive) {
        issue_s(0);
        issue_dp(0);
      }
      for (int it = 0; alive && it < n; ++it) {
        const bool more = it + 1 < n;
        alive = bwd_warp_ok<kWin>(
            ptx::wait_bounded(xbar(X::kPReady), it & 1, wd, kSiteBwdPFull));
        ptx::tc_fence_after();
        if (!alive) break;
        // dV_j += P^T dO_i; P^T sits in the first half of each group's columns of S^T
        if (bwd_elected<kWin>()) {
          issue_tmem_a<W::kGroups>(tDv, tS, do_mn0 + (it % L::kStagesB) * kSlotLo, idesc_dv,
                                   it > 0 ? 1u : 0u);
          ptx::mma_commit(bar(L::bEmptyB + it % L::kStagesB));
        }
        if (more) {
          alive = bwd_warp_ok<kWin>(full_a(it + 1));
          ptx::tc_fence_after();
          if (!alive) break;
          issue_s(it + 1);   // after dV in this thread's order: P^T has been read
        }
        alive = bwd_warp_ok<kWin>(
            ptx::wait_bounded(xbar(X::kDsReady), it & 1, wd, kSiteBwdDsReady));
        ptx::tc_fence_after();
        if (!alive) break;
        // dK_j += dS^T Q_i (scale applied at the end); dS^T likewise over dP^T
        if (bwd_elected<kWin>()) {
          issue_tmem_a<W::kGroups>(tDk, tDp, q_mn0 + (it % L::kStagesA) * kSlotLo, idesc_dk,
                                   it > 0 ? 1u : 0u);
          ptx::mma_commit(bar(L::bEmptyA + it % L::kStagesA));
        }
        if (more) {
          alive = bwd_warp_ok<kWin>(full_b(it + 1));
          ptx::tc_fence_after();
          if (!alive) break;
          issue_dp(it + 1);  // after dK: dS^T has been read
        }
      }
      if (bwd_elected<kWin>()) ptx::mma_commit(xbar(X::kDone));
      ptx::wait_drain(xbar(X::kDone), 0, 200000000ull);
    }
    __syncwarp();
  } else {
    // ============================================================ element-wise
    ptx::griddep_wait();   // D of the pass launched just before this grid
    const int quarter = warp & 3, group = warp >> 2;
    const int t = quarter * 32 + lane;                    // key row within the tile
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    // this thread's query columns of S^T and dP^T
    const uint32_t tS = tmem_base + lane_off + kColS + group * W::kCols;
    const uint32_t tDp = tmem_base + lane_off + kColDp + group * W::kCols;
    const long long key = static_cast<long long>(kt) * kBwdTile + t;
    const uint64_t c2 = ptx::f2_pack(p.scale_log2, p.scale_log2);

    // LSE and D of query row t of tile i, fetched one tile ahead by the
    // first group of the warps.  The loads are unconditional (a row past the
    // queries reads row 0) and nothing uses their values until the tile is
    // staged, so the warps do not wait for them; a query past N then gets
    // -LSE = -inf, so its P is 0, and D = 0.
    bool in_next = false;
    Step cur = first_step(), nxt = cur;   // the step at work and the one fetched
    auto fetch = [&](const Step& x, float& lse, float& dd) {
      const int qrow = x.tile * kBwdTile + t, qh = x.head;
      in_next = qrow < q_rows;
      const int qr = in_next ? qrow : 0;
      const long long qi = bwd_lse_at(p, tok, hd, qh, qr);
      lse = p.lse[qi];
      dd = p.delta[tok ? bwd_qrow(p, tok, hd, qh, qr) : qi];
    };
    float lse_next = 0.f, d_next = 0.f;
    if (group == 0) fetch(nxt, lse_next, d_next);
    int win_lo = 0, win_hi = W::kCols;   // kWin: this key's queries of the thread's, phases 1 to 2
    float pf[W::kCols];          // P^T of the current tile, from phase 1 to phase 2
    // dropout: keep bits of this key against the thread's 64 queries, from
    // the quad's words (zw[2 k2 + m]: word m of lane k2, blocks 8m + 4h + k2
    // of 4 queries each), from phase 1 to phase 2
    uint32_t zw[8] = {};
    const uint32_t csel = 0x4440u + (static_cast<uint32_t>(lane) & 3u);   // this key's byte
    // query bits of block b (queries 4b .. 4b + 3 of the thread's 64)
    auto zq = [&](int b) -> uint32_t {
      return col_query_bits(zw[2 * (b & 3) + (b >> 3)], csel, (b >> 2) & 1);
    };
    // vectors of query tile i0 + it: [0,128) -LSE, [128,256) D
    auto vec_of = [&](int it) {
      return reinterpret_cast<float*>(sgen + L::kVec) + (it % DkdvVec<D>::kBufs) * 256;
    };
    auto stage_vec = [&](int it) {
      float* vec = vec_of(it);
      // with one buffer, every thread must be done with the previous tile's
      if (DkdvVec<D>::kBufs == 1 && it > 0) ptx::named_bar_sync(1, W::kEwThreads);
      if (group == 0) {
        vec[t] = in_next ? -lse_next * 1.4426950408889634f : -INFINITY;   // -LSE, log2 units
        vec[128 + t] = in_next ? d_next : 0.f;
      }
      cur = nxt;
      next_step(nxt);
      if (group == 0 && it + 1 < nq) fetch(nxt, lse_next, d_next);
      ptx::named_bar_sync(2, W::kEwThreads);
    };

    // ---- phase 1: P^T = 2^(S^T c - LSE) over this thread's 64 queries
    auto phase1 = [&](int it) {
      const int i = cur.tile;
      const float4* nl4 = reinterpret_cast<const float4*>(vec_of(it)) + group * (W::kCols / 4);
      ptx::wait_bounded(xbar(X::kSFull), it & 1, wd, kSiteBwdSFull);
      __syncwarp();
      ptx::tc_fence_after();
      {
        uint32_t sr[W::kCols];
#pragma unroll
        for (int c = 0; c < W::kCols; c += 32) ptx::tmem_ld32(tS + c, sr + c);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < W::kCols; e += 4) {
          const float4 nl = nl4[e / 4];
          float x0, x1, x2, x3;
          ptx::f2_unpack(ptx::ffma2(ptx::f2_pack(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])),
                                    c2, ptx::f2_pack(nl.x, nl.y)), x0, x1);
          ptx::f2_unpack(ptx::ffma2(ptx::f2_pack(__uint_as_float(sr[e + 2]), __uint_as_float(sr[e + 3])),
                                    c2, ptx::f2_pack(nl.z, nl.w)), x2, x3);
          pf[e] = ptx::ex2(x0);
          pf[e + 1] = ptx::ex2(x1);
          pf[e + 2] = ptx::ex2(x2);
          pf[e + 3] = ptx::ex2(x3);
        }
      }
      if constexpr (kWin) {
        // queries q with key <= q + off < key + win (sinks: no upper bound);
        // padding keys see none, and rows past the queries are none (their
        // weights are 0, unless the score with a key that nobody sees is NaN)
        const int qb = i * kBwdTile + group * W::kCols;
        win_lo = key >= len ? W::kCols : static_cast<int>(key) - off - qb;
        win_hi = min(key < p.sinks ? q_rows : static_cast<int>(key) + p.win - off, q_rows) - qb;
        // (one compare and one select a query and end; no short circuits)
        if (win_lo > 0) {
#pragma unroll
          for (int e = 0; e < W::kCols; ++e) pf[e] = e < win_lo ? 0.f : pf[e];
        }
        if (win_hi < W::kCols) {
#pragma unroll
          for (int e = 0; e < W::kCols; ++e) pf[e] = e >= win_hi ? 0.f : pf[e];
        }
        // Rows at negative positions see no key, nor (without sinks) do rows
        // whose window starts past the batch's keys.  Whatever their Q and dO
        // hold, the weights 0 that they meet in dV and dK must give 0, so
        // these rows are cleared once S^T and dP^T have read them.
        const int pos0 = i * kBwdTile + off;
        const int r_lo = min(max(-pos0, 0), kBwdTile);
        const int r_hi = p.sinks > 0 ? kBwdTile : min(max(len + p.win - 1 - pos0, r_lo), kBwdTile);
        if (r_lo > 0 || r_hi < kBwdTile) {
          ptx::wait_bounded(xbar(X::kDpFull), it & 1, wd, kSiteBwdDpFull);
          __syncwarp();
          uint8_t* qt = sgen + L::kRingA + (it % L::kStagesA) * L::kTile;
          uint8_t* dt = sgen + L::kRingB + (it % L::kStagesB) * L::kTile;
          zero_rows(qt, L::kChunks, 0, r_lo, threadIdx.x, W::kEwThreads);
          zero_rows(qt, L::kChunks, r_hi, kBwdTile, threadIdx.x, W::kEwThreads);
          zero_rows(dt, L::kChunks, 0, r_lo, threadIdx.x, W::kEwThreads);
          zero_rows(dt, L::kChunks, r_hi, kBwdTile, threadIdx.x, W::kEwThreads);
          ptx::fence_proxy_async_smem();
        }
      } else if constexpr (kKv) {
        // padding keys see nothing; with causal masking query q sees this
        // key once q + off >= key
        const int qb = i * kBwdTile + group * W::kCols;
        const int lo = key >= len ? W::kCols : (kCausal ? static_cast<int>(key) - off - qb : 0);
#pragma unroll
        for (int e = 0; e < W::kCols; ++e)
          if (e < lo) pf[e] = 0.f;
      } else if (kCausal && i == kt) {   // diagonal tile: a key after the query is masked
#pragma unroll
        for (int e = 0; e < W::kCols; ++e)
          if (i * kBwdTile + group * W::kCols + e < key) pf[e] = 0.f;
      }
      // dropout: keep bits of this key against the thread's 64 queries, from
      // the quad's words (zw[2 k2 + m]: word m of lane k2, blocks 8m + 4h + k2
      // of 4 queries each); the dV product reads P with the dropped weights
      // zeroed
      if constexpr (kDrop) {
        const uint2 mine = drop_words16<true>(static_cast<uint32_t>(key >> 2),
                                              static_cast<uint32_t>(i * kBwdTile + group * W::kCols) >> 2,
                                              static_cast<uint32_t>(lane) & 3u,
                                              static_cast<uint32_t>(bh), p.drop_off, p.drop_k0,
                                              p.drop_k1, p.drop_t);
#pragma unroll
        for (int k2 = 0; k2 < 4; ++k2) {
          const int src = (lane & ~3) | k2;
          zw[2 * k2] = __shfl_sync(0xffffffffu, mine.x, src);
          zw[2 * k2 + 1] = __shfl_sync(0xffffffffu, mine.y, src);
        }
      }
      {
        // P and dS are rounded to the storage dtype, the tensor core's operand
        // type; what they sum up to (dV, dK, dQ) is fp32
        uint32_t pk[W::kCols / 2];
#pragma unroll
        for (int e = 0; e < W::kCols / 2; ++e) {
          pk[e] = ptx::pack2<kBf16>(pf[2 * e], pf[2 * e + 1]);
          if constexpr (kDrop) pk[e] &= prmt(zq(e >> 1), 0u, (e & 1) ? 0xBBAAu : 0x9988u);
        }
#pragma unroll
        for (int c = 0; c < W::kCols / 2; c += 16)
          ptx::tmem_st16(tS + c, pk + c);   // over S^T columns this warp has read
      }
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      ptx::mbar_arrive(xbar(X::kPReady));
    };

    // ---- phase 2: dS^T = P^T * (dP^T - D)
    auto phase2 = [&](int it) {
      const float4* dl4 = reinterpret_cast<const float4*>(vec_of(it) + 128) + group * (W::kCols / 4);
      ptx::wait_bounded(xbar(X::kDpFull), it & 1, wd, kSiteBwdDpFull);
      __syncwarp();
      ptx::tc_fence_after();
      uint32_t dk[W::kCols / 2];
#pragma unroll
      for (int ch = 0; ch < W::kCols / 32; ++ch) {
        uint32_t dpr[32];
        ptx::tmem_ld32(tDp + ch * 32, dpr);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 dd = dl4[(ch * 32 + e) / 4];
          const int f = ch * 32 + e;
          // dP^T, with dropout Z dP^T (the 256 / t joins in the subtraction of D)
          uint32_t zx = 0;
          if constexpr (kDrop) zx = zq(f >> 2);   // f is a multiple of 4: one block
          auto dpv = [&](int x) -> float {
            if constexpr (kDrop)
              return __uint_as_float(dpr[e + x] & prmt(zx, 0u, 0x8888u + 0x1111u * x));
            return __uint_as_float(dpr[e + x]);
          };
          auto dmd = [&](float a, float b, float da, float db) -> uint64_t {
            if constexpr (kDrop)
              return ptx::ffma2(ptx::f2_pack(a, b), ptx::f2_pack(p.drop_scale, p.drop_scale),
                                ptx::f2_pack(-da, -db));
            return ptx::fadd2(ptx::f2_pack(a, b), ptx::f2_pack(-da, -db));
          };
          float d0, d1, d2, d3;
          ptx::f2_unpack(ptx::fmul2(ptx::f2_pack(pf[f], pf[f + 1]), dmd(dpv(0), dpv(1), dd.x, dd.y)),
                         d0, d1);
          ptx::f2_unpack(ptx::fmul2(ptx::f2_pack(pf[f + 2], pf[f + 3]),
                                    dmd(dpv(2), dpv(3), dd.z, dd.w)), d2, d3);
          dk[f / 2] = ptx::pack2<kBf16>(d0, d1);
          dk[f / 2 + 1] = ptx::pack2<kBf16>(d2, d3);
        }
      }
      if constexpr (kWin) {
        // a select, not a product with the masked P: dP - D of a key outside
        // its batch's count need not be finite
        if (win_lo > 0) {
#pragma unroll
          for (int e = 0; e < W::kCols / 2; ++e)
            dk[e] &= (2 * e < win_lo ? 0u : 0xffffu) | (2 * e + 1 < win_lo ? 0u : 0xffff0000u);
        }
        if (win_hi < W::kCols) {
#pragma unroll
          for (int e = 0; e < W::kCols / 2; ++e)
            dk[e] &= (2 * e >= win_hi ? 0u : 0xffffu) | (2 * e + 1 >= win_hi ? 0u : 0xffff0000u);
        }
      }
#pragma unroll
      for (int c = 0; c < W::kCols / 2; c += 16)
        ptx::tmem_st16(tDp + c, dk + c);   // over dP^T columns this warp has read
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      ptx::mbar_arrive(xbar(X::kDsReady));
    };

    for (int it = 0; it < nq; ++it) {
      stage_vec(it);
      phase1(it);
      phase2(it);
    }
    // dV_j rows (the first half of the groups) and dK_j = scale * (dS^T Q)
    // rows (the second), each warp a part of the columns
    ptx::wait_bounded(xbar(X::kDone), 0, wd, kSiteBwdDone);
    __syncwarp();
    ptx::tc_fence_after();
    const long long row = bwd_krow(p, tok, hd, bh, key);
    constexpr int kShare = W::kGroups / 2;
    const bool is_dk = group >= kShare;
    const uint32_t acc = tmem_base + lane_off + kColAcc + (is_dk ? D : 0);
    const int width = kWin ? D : (is_dk ? p.width_qk : p.width_v);
    const int c0 = group % kShare * (width / kShare);
    const float mul = is_dk ? p.scale : (kDrop ? p.drop_scale : 1.f);
    if (part_ws != nullptr)
      store_acc_f32(acc, c0, width / kShare, mul,
                    part_ws + static_cast<size_t>(t) * 2 * D + (is_dk ? 0 : D));
    else
      store_acc_cols<kBf16>(acc, c0, width / kShare, width, mul, is_dk ? p.dk : p.dv, row,
                            key < key_rows);
  }
  bwd_teardown<L>(sbase);
}

// ---------------------------------------------------------------- dQ
// TMEM columns of the two dS buffers (16-bit, 64 packed columns each), after dQ.
template <int D>
__device__ __forceinline__ uint32_t dq_ds_col(int b) {
  return kColAcc + D + 64u * b;
}

// One CTA of the dQ pass: block `blk` of BH * n_tiles.
template <int D, bool kBf16, bool kCausal, bool kDrop, bool kKv, bool kWin = false>
__device__ __forceinline__ void bwd_dq_cta(const BwdParams& p, int blk, uint32_t tmem_base) {
  using L = BwdSmem<D, 0>;
  using X = DqBars;
  using W = BwdRoles<kWin>;
  static_assert(kColAcc + D + 128 <= kBwdTmemCols, "dS buffers fit in TMEM");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = ptx::smem_u32(smem_raw);
  const uint32_t sbase = (raw_base + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - raw_base);
  const int warp = bwd_uniform<kWin>(threadIdx.x >> 5), lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return sbase + L::kBar + 8u * i; };
  auto xbar = [&](int i) -> uint32_t { return bar(L::bX + i); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sgen + L::kMisc + 4);

  // Query tile qt of head bh; for causal runs the last query tiles (the most
  // key tiles to visit) are dealt first.
  int r, bh;
  bwd_item(p, blk, p.n_tiles, r, bh);
  const int qt = kCausal ? p.n_tiles - 1 - r : r;
  int nk = kCausal ? qt + 1 : p.n_tiles;   // key tiles j <= qt are visible
  int len = p.N, off = 0;                  // keys of this head, query offset (kKv)
  const bool tok = kKv && p.varlen;        // packed batch: token-major rows
  BwdHead hd{p.N, 0, p.N, 0, 0};
  if constexpr (kKv) {
    // key tiles up to the position of the tile's last query row
    hd = bwd_kv_head(p, bh, kCausal);
    len = hd.len;
    off = hd.off;
    if (qt * kBwdTile >= hd.lenq) return;   // past this sequence's queries: no rows
    const int nkv = (len + kBwdTile - 1) / kBwdTile;
    const int last = min(qt * kBwdTile + kBwdTile, hd.lenq) - 1 + off;
    nk = !kCausal ? nkv : (last < 0 ? 0 : min(last / kBwdTile + 1, nkv));
  }
  // kWin: of the key tiles 0 .. nk - 1 only the sink tiles and those from the
  // first row's window on are walked
  BwdWinKeys wk{};
  if constexpr (kWin) {
    wk = bwd_win_keys(qt * kBwdTile, min(qt * kBwdTile + kBwdTile, hd.lenq), len, off, nk, p.win,
                      p.sinks);
    nk = wk.count;
  }
  // kWin: of the first tile's keys any row sees only the sinks, in the first
  // column group; the products take that many keys, the other groups nothing
  const bool narrow0 = kWin && wk.ns == 1 && p.sinks <= kBwdNarrow && wk.lo >= kBwdTile;
  static_assert(!kWin || W::kCols == kBwdNarrow, "the first column group");
  auto k_tile = [&](int j) { return kWin && j >= wk.ns ? wk.wa + (j - wk.ns) : j; };
  const int q_rows = tok ? hd.lenq : p.N;
  if (kKv && nk <= 0) {
    // no query of this tile sees a key: its dQ rows are zero
    if (threadIdx.x < 256) {
      const int t = threadIdx.x & 127, hf = threadIdx.x >> 7;
      const long long qrow = static_cast<long long>(qt) * kBwdTile + t;
      if (qrow < q_rows) {
        // each half of the threads clears half of the row's width_qk columns
        uint4* row = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.dq) +
                                              bwd_qrow(p, tok, hd, bh, qrow) * (p.width_qk * 2) +
                                              hf * p.width_qk);
        for (int c = 0; c < p.width_qk / 16; ++c) row[c] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    return;
  }

  bwd_setup<L>(sbase, sgen, [&](auto b) {
    ptx::mbar_init(b(L::bX + X::kSFull), 1);
    ptx::mbar_init(b(L::bX + X::kSFree), W::kEwThreads);
    for (int k = 0; k < 2; ++k) {
      ptx::mbar_init(b(L::bX + X::kPFull + k), W::kEwThreads);
      ptx::mbar_init(b(L::bX + X::kDsFree + k), 1);
    }
    ptx::mbar_init(b(L::bX + X::kDone), 1);
  });
  const ptx::Watchdog wd{p.watchdog_cycles, abort_flag, p.status};

  if (warp == W::kLoadWarp) {
    if constexpr (kWin) {
      if (lane == 0) {
        const int kvh = bh / p.H * p.Hk + bh % p.H / p.G;
        bwd_producer_map<L>(
            sbase, &p.tm_q, &p.tm_do, [&](int& y, int& z) { y = qt * kBwdTile; z = bh; }, &p.tm_k,
            &p.tm_v, [&](int it, int& y, int& z) { y = k_tile(it) * kBwdTile; z = kvh; }, nk, wd);
      }
    } else if (lane == 0) {
      bwd_producer<L>(sbase, &p.tm_q, &p.tm_do, qt, &p.tm_k, &p.tm_v, 0, nk, bh, wd,
                      tok ? bh % p.H : -1, hd.q0, hd.k0, p.width_qk / 64, p.width_v / 64);
    }
    __syncwarp();
  } else if (warp == W::kMmaWarp) {
    if (kWin || lane == 0) {
      const uint32_t tmem = bwd_uniform<kWin>(tmem_base);
      const int n = bwd_uniform<kWin>(nk);
      const bool narrow = kWin && ptx::warp_all(narrow0);
      constexpr int fmt = kBf16 ? 1 : 0;
      constexpr uint32_t idesc_s = ptx::idesc_f16(kBwdTile, kBwdTile, fmt, 0);
      const uint32_t idesc_dq = ptx::idesc_f16(kBwdTile, kWin ? D : p.width_qk, fmt, 1);   // dQ: width_qk columns
      const int steps_s = kWin ? D / 16 : p.width_qk / 16;
      const int steps_dp = kWin ? D / 16 : p.width_v / 16;
      constexpr uint32_t kSlotLo = L::kTile >> 4;
      const uint32_t q_lo = ptx::desc_lo(sbase + L::kRes, 16);
      const uint32_t do_lo = ptx::desc_lo(sbase + L::kRes + L::kTile, 16);
      const uint32_t k_lo0 = ptx::desc_lo(sbase + L::kRingA, 16);                 // K-major use
      const uint32_t v_lo0 = ptx::desc_lo(sbase + L::kRingB, 16);
      const uint32_t k_mn0 = ptx::desc_lo(sbase + L::kRingA, L::kChunkBytes);     // MN-major use
      const uint32_t tS = tmem + kColS, tDp = tmem + kColDp;
      const uint32_t tDq = tmem + kColAcc;
      // dQ_i += dS_j K_j for key tile j (scale applied at the end)
      auto issue_dq = [&](int j) -> bool {
        const bool ok = bwd_warp_ok<kWin>(
            ptx::wait_bounded(xbar(X::kPFull + (j & 1)), (j >> 1) & 1, wd, kSiteBwdPFull));
        ptx::tc_fence_after();
        if (!ok) return false;
        const int slot = j % L::kStagesA;
        if (!bwd_elected<kWin>()) return true;
        issue_tmem_a<1>(tDq, tmem + dq_ds_col<D>(j & 1), k_mn0 + slot * kSlotLo, idesc_dq,
                        j > 0 ? 1u : 0u, kWin && narrow && j == 0);
        ptx::mma_commit(bar(L::bEmptyA + slot));
        ptx::mma_commit(xbar(X::kDsFree + (j & 1)));
        return true;
      };
      bool alive = bwd_warp_ok<kWin>(ptx::wait_bounded(bar(L::bRes), 0, wd, kSiteBwdRes));
      for (int it = 0; alive && it < n; ++it) {
        const int sa = it % L::kStagesA, sb = it % L::kStagesB;
        alive = ptx::wait_bounded(bar(L::bFullA + sa), (it / L::kStagesA) & 1, wd, kSiteBwdFull);
        alive = alive && ptx::wait_bounded(bar(L::bFullB + sb), (it / L::kStagesB) & 1, wd, kSiteBwdFull);
        // the element-wise warps have read S and dP of the previous key tile
        if (it > 0) alive = alive && ptx::wait_bounded(xbar(X::kSFree), (it - 1) & 1, wd, kSiteBwdSFree);
        alive = bwd_warp_ok<kWin>(alive);
        ptx::tc_fence_after();
        if (!alive) break;
        // S = Q_i K_j^T and dP = dO_i V_j^T (queries on the TMEM lanes)
        if (bwd_elected<kWin>()) {
          constexpr uint32_t idesc_narrow = ptx::idesc_f16(kBwdTile, kBwdNarrow, fmt, 0);
          const uint32_t idesc = kWin && narrow && it == 0 ? idesc_narrow : idesc_s;
          issue_kmajor<D, L::kChunkBytes>(tS, q_lo, k_lo0 + sa * kSlotLo, idesc, steps_s);
          issue_kmajor<D, L::kChunkBytes>(tDp, do_lo, v_lo0 + sb * kSlotLo, idesc, steps_dp);
          ptx::mma_commit(xbar(X::kSFull));
          ptx::mma_commit(bar(L::bEmptyB + sb));   // V_j is not read again
        }
        if (it > 0) alive = issue_dq(it - 1);
      }
      if (alive) issue_dq(nk - 1);
      if (bwd_elected<kWin>()) ptx::mma_commit(xbar(X::kDone));
      ptx::wait_drain(xbar(X::kDone), 0, 200000000ull);
    }
    __syncwarp();
  } else {
    // ============================================================ element-wise
    ptx::griddep_wait();   // D of the pass launched just before this grid
    const int quarter = warp & 3, group = warp >> 2;
    const int t = quarter * 32 + lane;                    // query row within the tile
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    // this thread's key columns of S and dP
    const uint32_t tS = tmem_base + lane_off + kColS + group * W::kCols;
    const uint32_t tDp = tmem_base + lane_off + kColDp + group * W::kCols;
    const long long qrow = static_cast<long long>(qt) * kBwdTile + t;
    const bool q_in = qrow < q_rows;
    const long long grow = bwd_qrow(p, tok, hd, bh, qrow);
    const long long li = bwd_lse_at(p, tok, hd, bh, qrow);
    const float nl = q_in ? -p.lse[li] * 1.4426950408889634f : -INFINITY;
    const float dl = q_in ? p.delta[tok ? grow : li] : 0.f;
    const uint64_t c2 = ptx::f2_pack(p.scale_log2, p.scale_log2);
    const uint64_t nl2 = ptx::f2_pack(nl, nl);
    const uint64_t ndl2 = ptx::f2_pack(-dl, -dl);
    for (int j = 0; j < nk; ++j) {
      ptx::wait_bounded(xbar(X::kSFull), j & 1, wd, kSiteBwdSFull);
      __syncwarp();
      ptx::tc_fence_after();
      // keys past N, and on the diagonal tile keys after this query, are
      // masked (limits relative to this thread's first key column)
      int lim = p.N - j * kBwdTile - group * W::kCols;
      int lo = 0;              // kWin: keys of the thread's before the window, sinks aside
      if constexpr (kWin) {
        const int key0 = k_tile(j) * kBwdTile, pos = static_cast<int>(qrow) + off;
        lim = min(len, pos + 1) - key0 - group * W::kCols;
        lo = pos - p.win + 1 - key0 - group * W::kCols;
        // Keys of this tile that no row sees get dS = 0; their rows of K are
        // cleared so that the product with them is 0 whatever they hold (S
        // and dP have read the tile).
        const int rows_k = narrow0 && j == 0 ? kBwdNarrow : kBwdTile;   // rows that are read
        const int r_hi = min(max(wk.hi - key0, 0), rows_k);
        const int r_lo = min(max(wk.lo - key0, 0), r_hi);
        const int r_sink = min(max(p.sinks - key0, 0), r_lo);
        if (r_sink < r_lo || r_hi < rows_k) {
          uint8_t* kt = sgen + L::kRingA + (j % L::kStagesA) * L::kTile;
          zero_rows(kt, L::kChunks, r_sink, r_lo, threadIdx.x, W::kEwThreads);
          zero_rows(kt, L::kChunks, r_hi, rows_k, threadIdx.x, W::kEwThreads);
          ptx::fence_proxy_async_smem();
        }
        if (narrow0 && j == 0 && group > 0) {
          ptx::mbar_arrive(xbar(X::kSFree));
          ptx::mbar_arrive(xbar(X::kPFull));   // of buffer 0
          continue;
        }
      } else if constexpr (kKv) {
        // keys past this head's count, and with causal masking keys after
        // this query's position
        lim = len - j * kBwdTile - group * W::kCols;
        if (kCausal) lim = min(lim, static_cast<int>(qrow) + off + 1 - j * kBwdTile - group * W::kCols);
      } else if (kCausal && j == qt) {
        lim = min(lim, t + 1 - group * W::kCols);
      }
      // all of S and dP into registers first: the next products wait for this
      uint32_t sr[W::kCols], dpr[W::kCols];
#pragma unroll
      for (int c = 0; c < W::kCols; c += 32) ptx::tmem_ld32(tS + c, sr + c);
#pragma unroll
      for (int c = 0; c < W::kCols; c += 32) ptx::tmem_ld32(tDp + c, dpr + c);
      ptx::tmem_wait_ld();
      ptx::tc_fence_before();
      ptx::mbar_arrive(xbar(X::kSFree));     // S and dP may be overwritten now
      // dropout: keep bits of this query against the thread's 64 keys, from
      // the quad's words (zw[2 k2 + m]: word m of lane k2, blocks 8m + 4h + k2
      // of 4 keys each)
      uint32_t zw[8] = {};
      if constexpr (kDrop) {
        const uint2 mine = drop_words16<false>(static_cast<uint32_t>(j * kBwdTile + group * W::kCols) >> 2,
                                               static_cast<uint32_t>(qrow >> 2),
                                               static_cast<uint32_t>(lane) & 3u,
                                               static_cast<uint32_t>(bh), p.drop_off, p.drop_k0,
                                               p.drop_k1, p.drop_t);
#pragma unroll
        for (int k2 = 0; k2 < 4; ++k2) {
          const int src = (lane & ~3) | k2;
          zw[2 * k2] = __shfl_sync(0xffffffffu, mine.x, src);
          zw[2 * k2 + 1] = __shfl_sync(0xffffffffu, mine.y, src);
        }
      }
      uint32_t dk[W::kCols / 2];
#pragma unroll
      for (int kc = 0; kc < W::kCols; kc += 2) {
        float x0, x1;
        ptx::f2_unpack(ptx::ffma2(ptx::f2_pack(__uint_as_float(sr[kc]), __uint_as_float(sr[kc + 1])),
                                  c2, nl2), x0, x1);
        float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1);
        if constexpr (!kWin) {
          if (kc >= lim) p0 = 0.f;
          if (kc + 1 >= lim) p1 = 0.f;
        }
        float g0 = __uint_as_float(dpr[kc]), g1 = __uint_as_float(dpr[kc + 1]);
        uint64_t gd;
        if constexpr (kDrop) {   // Z dP 256 / t - D
          const int b = kc >> 2;                       // block of keys 4b .. 4b + 3
          const uint32_t y = zw[2 * (b & 3) + (b >> 3)], r = static_cast<uint32_t>(qrow) & 3u;
          g0 = __uint_as_float(dpr[kc] & row_key_mask(y, r, (b >> 2) & 1, kc & 3));
          g1 = __uint_as_float(dpr[kc + 1] & row_key_mask(y, r, (b >> 2) & 1, (kc + 1) & 3));
          gd = ptx::ffma2(ptx::f2_pack(g0, g1), ptx::f2_pack(p.drop_scale, p.drop_scale), ndl2);
        } else {
          gd = ptx::fadd2(ptx::f2_pack(g0, g1), ndl2);
        }
        float d0, d1;
        ptx::f2_unpack(ptx::fmul2(ptx::f2_pack(p0, p1), gd), d0, d1);
        dk[kc / 2] = ptx::pack2<kBf16>(d0, d1);
      }
      if constexpr (kWin) {
        // masked keys by selection (dP of a key outside its batch's count
        // need not be finite): past the position, or before the window and
        // not a sink
        const int sink = p.sinks - k_tile(j) * kBwdTile - group * W::kCols;
        if (lo >= W::kCols) lim = min(lim, sink);
        if (lim < W::kCols) {
#pragma unroll
          for (int e = 0; e < W::kCols / 2; ++e)
            dk[e] &= (2 * e >= lim ? 0u : 0xffffu) | (2 * e + 1 >= lim ? 0u : 0xffff0000u);
        }
        if (lo > 0 && lo < W::kCols) {
#pragma unroll
          for (int e = 0; e < W::kCols / 2; ++e)
            dk[e] &= ((2 * e < lo) & (2 * e >= sink) ? 0u : 0xffffu) |
                     ((2 * e + 1 < lo) & (2 * e + 1 >= sink) ? 0u : 0xffff0000u);
        }
      }
      // dS to its TMEM buffer once the tensor core has read what it held
      // (dQ of key tile j - 2)
      const int b = j & 1;
      if (j >= 2) ptx::wait_bounded(xbar(X::kDsFree + b), ((j >> 1) - 1) & 1, wd, kSiteBwdDsFree);
      __syncwarp();
      ptx::tc_fence_after();
      const uint32_t tDs = tmem_base + lane_off + dq_ds_col<D>(b) + group * (W::kCols / 2);
#pragma unroll
      for (int c = 0; c < W::kCols / 2; c += 16) ptx::tmem_st16(tDs + c, dk + c);
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      ptx::mbar_arrive(xbar(X::kPFull + b));
    }
    // dQ = scale * (dS K): each group of the warps writes a part of the
    // columns, 32 at least
    ptx::wait_bounded(xbar(X::kDone), 0, wd, kSiteBwdDone);
    __syncwarp();
    ptx::tc_fence_after();
    const int cols = max(p.width_qk / W::kGroups, 32);
    if (group * cols < p.width_qk)
      store_acc_cols<kBf16>(tmem_base + lane_off + kColAcc, group * cols, cols, p.width_qk, p.scale,
                            p.dq, grow, q_in);
  }
  bwd_teardown<L>(sbase);
}

// ---------------------------------------------------------------- entry point
// Both tensor-core passes in one persistent grid of at most one CTA per SM.
// The work items are [0, BH * n_ktiles) dK/dV items (the ones with the most
// query tiles first), then the dQ items (most key tiles first); CTA c takes
// items c, c + grid, c + 2 grid, ...  (A snake order, c then grid - 1 - c,
// measured no better.)  One grid lets SMs that finish their dK/dV items
// take dQ items at once, so the two passes share one partial last round,
// and a CTA that stays resident across items skips the relaunch and the
// TMEM allocation of every item after its first.  Shared memory is sized
// for the larger layout.
template <int D, bool kBf16, bool kCausal, bool kDrop = false, bool kKv = false, bool kWin = false>
__global__ void __launch_bounds__(BwdRoles<kWin>::kThreads, 1)
    fa_bwd_kernel(const __grid_constant__ BwdParams p) {
  using W = BwdRoles<kWin>;
  __shared__ uint32_t s_tmem_base;
  const int warp = threadIdx.x >> 5;
  if (warp == W::kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_u32(&s_tmem_base), kBwdTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = s_tmem_base;
  // dK/dV items, one per key tile (kWin: more for the cut sink tiles)
  const int per_pass =
      kWin ? p.BHk * (p.n_ktiles + p.split_tiles * (p.split_parts - 1)) : p.BH * p.n_ktiles;
  const int total = per_pass + p.BH * p.n_tiles;
  for (int item = blockIdx.x; item < total; item += gridDim.x) {
    if (item < per_pass)
      bwd_dkdv_cta<D, kBf16, kCausal, kDrop, kKv, kWin>(p, item, tmem_base);
    else
      bwd_dq_cta<D, kBf16, kCausal, kDrop, kKv, kWin>(p, item - per_pass, tmem_base);
  }
  // A call in which no query sees a key (all counts 0, no keys, every position
  // negative) has only items without steps, none of which waits for the D
  // pass: without this wait the grid, and with it the call, could end while
  // that pass still writes `delta`.
  if constexpr (kKv) ptx::griddep_wait();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == W::kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, kBwdTmemCols);
  }
}

}  // namespace fa
