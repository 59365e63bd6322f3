// fa_decode_paged.cu — the entry point fa_decode_paged of the C ABI declared
// in include/fa.h: argument checks, TMA descriptors and the launches of the
// decoding kernels over a paged 8-bit cache.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "fa.h"
#include "fa_decode_paged_kernel.cuh"
#include "fa_decode_paged_tc_kernel.cuh"
#include "fa_host.cuh"

using namespace fa::host;

namespace fa {
namespace {

template <int D, bool kBf16, bool kInt8, int kTiles>
cudaError_t launch_main(const DecPagedParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};   // devices on which the smem limit was raised
  auto kernel = fa_decode_paged_kernel<D, kBf16, kInt8, kTiles>;
  constexpr int kAlloc = DpLayout<D, kTiles>::kAlloc;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done.load() & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kAlloc);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit);
  }
  kernel<<<p.grid, DpLayout<D, kTiles>::kThreads, kAlloc, stream>>>(p);
  return cudaGetLastError();
}

constexpr int kManyTiles = kDtRows / 8;   // row tiles of a unit of the kernel for many rows

template <int D, bool kBf16, bool kInt8>
cudaError_t launch_tc(const DecPagedParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  auto kernel = fa_decode_paged_tc_kernel<D, kBf16, kInt8>;
  constexpr int kAlloc = DtLayout<D>::kAlloc;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done.load() & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kAlloc);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit);
  }
  kernel<<<p.grid, kDtThreads, kAlloc, stream>>>(p);
  return cudaGetLastError();
}

template <int D, bool kBf16, bool kInt8>
cudaError_t launch_variant(const DecPagedParams& p, int tiles, int sms, cudaStream_t stream) {
  cudaError_t e = tiles == 1   ? launch_main<D, kBf16, kInt8, 1>(p, stream)
                  : tiles == 2 ? launch_main<D, kBf16, kInt8, 2>(p, stream)
                               : launch_tc<D, kBf16, kInt8>(p, stream);
  if (e != cudaSuccess) return e;
  // Programmatic dependent launch: the combine grid is set up while the main
  // kernel runs its last CTAs, and waits on the device for the parts.  Blocks
  // take several units where those are many, since most are whole then, and
  // more threads where a unit may have many parts.
  const int units = p.B * p.Hk * p.row_blocks, per_block = (units + 4 * sms - 1) / (4 * sms);
  constexpr int kMany = 2048 / D;                     // groups of D / 4 threads
  const bool many = p.runs > 16 * units;              // more than two batches of parts
  const int rows = many ? 1 : kDpCombineThreads / (D / 4);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((units + per_block - 1) / per_block, (p.slot_rows + rows - 1) / rows);
  cfg.blockDim = dim3(many ? kMany * (D / 4) : kDpCombineThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return many ? cudaLaunchKernelEx(&cfg, fa_decode_paged_combine_kernel<D, kBf16, kMany>, p, units,
                                   per_block)
              : cudaLaunchKernelEx(&cfg, fa_decode_paged_combine_kernel<D, kBf16, 1>, p, units,
                                   per_block);
}

constexpr int kMaxTokens = 16;

// Row tiles of a unit (8 rows each), runs (one per warp of a CTA per SM, or one
// per CTA for many rows, or fewer) and the workspace: two parts per run, and the units' table.
struct Plan {
  int tiles, row_blocks, slot_rows, grid, runs;
  size_t o_bytes, ml_bytes, bytes;
};
// Up to 16 rows the warps' own products win, from 17 on the other kernel (8 caches to
// 32768, 4 heads; the first kernel in blocks of 16 rows, us):
//     rows            9    16   17   32   64  128  129   d = 64: 16   32   64
//     by warps       50    56   82   88  135  248  277           42   64   85
//     through TMEM   62    63   63   63   64   73  121           59   58   60
// (16 rows of int8 57 and 63; 129 rows are two units, the second nearly empty.)
int row_tiles(int R) { return R <= 8 ? 1 : R <= 16 ? 2 : kManyTiles; }
int tile_keys(int tiles, int d) { return tiles == kManyTiles ? kDtKeys : dp_keys(d); }
// Tiles of all units at most: whole capacities, and one of each sequence's own.
long long max_tiles(int B, int Hk, int row_blocks, int keys, int capacity) {
  const long long tiles = (static_cast<long long>(capacity) + keys - 1) / keys + 1;
  return static_cast<long long>(B) * Hk * row_blocks * tiles;
}
int check_sizes(int B, int H, int Hk, int Nq, int d, int page_size, int pages_per_seq) {
  if (H < 0 || (H > 0 ? (Hk <= 0 || H % Hk != 0) : Hk != 0)) return FA_ERR_SHAPE;
  if (Nq < 1 || Nq > kMaxTokens) return FA_ERR_SHAPE;
  if (static_cast<long long>(B) * H * Nq > (1 << 30)) return FA_ERR_SHAPE;
  if (B == 0 || H == 0) return FA_OK;
  const int R = H / Hk * Nq, span = 8 * row_tiles(R);
  // the numbers of all tiles fit in int
  if (max_tiles(B, Hk, (R + span - 1) / span, tile_keys(span / 8, d),
                pages_per_seq * page_size) >= (1ll << 31))
    return FA_ERR_SHAPE;
  return FA_OK;
}
Plan make_plan(int B, int H, int Hk, int Nq, int d, int capacity, int sms) {
  Plan pl{};
  const int R = H / Hk * Nq;
  pl.tiles = row_tiles(R);
  pl.row_blocks = (R + 8 * pl.tiles - 1) / (8 * pl.tiles);
  pl.slot_rows = std::min(R, 8 * pl.tiles);
  const bool many = pl.tiles == kManyTiles;
  const long long min_tiles = many ? 1 : dp_min_tiles(pl.tiles);
  const long long warps = many ? 1 : dp_warps(pl.tiles);
  const long long most = max_tiles(B, Hk, pl.row_blocks, tile_keys(pl.tiles, d), capacity);
  const long long all = (most + min_tiles - 1) / min_tiles;
  pl.runs = static_cast<int>(std::min(all, sms * warps));
  pl.grid = std::min(pl.runs, sms);
  const size_t rows = 2 * static_cast<size_t>(pl.runs) * pl.slot_rows;
  pl.o_bytes = (rows * d * sizeof(float) + 255) / 256 * 256;
  pl.ml_bytes = (rows * sizeof(float2) + 255) / 256 * 256;
  const size_t units = static_cast<size_t>(B) * Hk * pl.row_blocks;
  pl.bytes = pl.o_bytes + pl.ml_bytes + (units * sizeof(int2) + 255) / 256 * 256;
  return pl;
}

}  // namespace
}  // namespace fa

extern "C" {

int fa_decode_paged_workspace_size(int B, int H, int Hk, int Nq, int d, int page_size,
                                   int pages_per_seq, size_t* bytes) {
  if (!bytes) return FA_ERR_NULLPTR;
  int rc = check_paged(B, Hk, d, 1, page_size, pages_per_seq, FA_E4M3);
  if (rc == FA_OK) rc = fa::check_sizes(B, H, Hk, Nq, d, page_size, pages_per_seq);
  if (rc != FA_OK) return rc;
  *bytes = 0;
  if (B == 0 || H == 0) return FA_OK;
  int dev = 0;
  const DeviceInfo* info = device_info(&dev);
  if (!info || !info->supported) return FA_ERR_DEVICE;
  *bytes = fa::make_plan(B, H, Hk, Nq, d, pages_per_seq * page_size, info->sms).bytes;
  return FA_OK;
}

int fa_decode_paged(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                    const float* v_scale, void* o, float* lse, int B, int H, int Hk, int Nq, int d,
                    int pages, int page_size, const int* page_table, int pages_per_seq,
                    const int* seqlens, int window, int sinks, float scale, int dtype,
                    int cache_dtype, void* workspace, size_t workspace_bytes,
                    cudaStream_t stream) {
  int rc = check_paged(B, Hk, d, pages, page_size, pages_per_seq, cache_dtype);
  if (rc == FA_OK) rc = fa::check_sizes(B, H, Hk, Nq, d, page_size, pages_per_seq);
  if (rc != FA_OK) return rc;
  if (window < 0 || sinks < 0) return FA_ERR_SHAPE;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_DTYPE;
  if (!std::isfinite(scale) || !(scale > 0.0f)) return FA_ERR_SCALE;
  if (B == 0 || H == 0) return FA_OK;
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !o || !lse || !page_table || !seqlens)
    return FA_ERR_NULLPTR;
  auto misaligned = [](const void* p, uintptr_t n) {
    return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0;
  };
  if (misaligned(q, 16) || misaligned(k_cache, 16) || misaligned(v_cache, 16) ||
      misaligned(o, 16) || misaligned(lse, 4) || misaligned(k_scale, 4) ||
      misaligned(v_scale, 4) || misaligned(page_table, 4) || misaligned(seqlens, 4))
    return FA_ERR_ALIGN;

  int dev = 0;
  const DeviceInfo* info = device_info(&dev);
  if (!info || !info->supported) return FA_ERR_DEVICE;
  if (info->err != FA_OK) return info->err;
  const int capacity = pages_per_seq * page_size;
  const fa::Plan pl = fa::make_plan(B, H, Hk, Nq, d, capacity, info->sms);
  const int keys = fa::tile_keys(pl.tiles, d);
  if (!workspace || workspace_bytes < pl.bytes) return FA_ERR_WORKSPACE;
  if (misaligned(workspace, 256)) return FA_ERR_ALIGN;

  fa::DecPagedParams p{};
  // the largest boxes that pages and tiles are both made of
  int box = keys;
  while (page_size % box != 0) box /= 2;
  p.boxes = keys / box;
  const long long rows = static_cast<long long>(pages) * Hk * page_size;
  if (!make_tmap_codes(&p.tm_k, k_cache, rows, d, box) ||
      !make_tmap_codes(&p.tm_v, v_cache, rows, d, box))
    return FA_ERR_TENSORMAP;
  p.q = q;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.table = page_table;
  p.per_seq = pages_per_seq;
  p.pages = pages;
  p.page = page_size;
  p.page_magic = page_size == fa::kPageRows
                     ? 0
                     : static_cast<uint32_t>(((1ull << 32) + page_size / fa::kPageRows - 1) /
                                             (page_size / fa::kPageRows));
  p.o = o;
  p.lse = lse;
  p.part_o = static_cast<float4*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + pl.o_bytes);
  p.cut = reinterpret_cast<int2*>(static_cast<uint8_t*>(workspace) + pl.o_bytes + pl.ml_bytes);
  p.status = info->status;
  const unsigned long long wd = g_watchdog_ns.load();
  p.watchdog_cycles = (wd ? wd : kDefaultWatchdogNs) * 21ull / 10ull;
  p.seqlens = seqlens;
  p.B = B;
  p.Hk = Hk;
  p.Nq = Nq;
  p.R = H / Hk * Nq;
  p.row_blocks = pl.row_blocks;
  p.slot_rows = pl.slot_rows;
  p.runs = pl.runs;
  p.grid = pl.grid;
  const int all = capacity + Nq + 1;
  p.win = window == 0 ? all : std::min(window, all);
  p.sinks = std::min(sinks, capacity);
  p.scale_log2 = scale * 1.4426950408889634f;
  const bool bf16 = dtype == FA_BF16;
  cudaError_t e;
  if (cache_dtype == FA_INT8) {
    if (d == 64)
      e = bf16 ? fa::launch_variant<64, true, true>(p, pl.tiles, info->sms, stream)
               : fa::launch_variant<64, false, true>(p, pl.tiles, info->sms, stream);
    else
      e = bf16 ? fa::launch_variant<128, true, true>(p, pl.tiles, info->sms, stream)
               : fa::launch_variant<128, false, true>(p, pl.tiles, info->sms, stream);
  } else {
    if (d == 64)
      e = bf16 ? fa::launch_variant<64, true, false>(p, pl.tiles, info->sms, stream)
               : fa::launch_variant<64, false, false>(p, pl.tiles, info->sms, stream);
    else
      e = bf16 ? fa::launch_variant<128, true, false>(p, pl.tiles, info->sms, stream)
               : fa::launch_variant<128, false, false>(p, pl.tiles, info->sms, stream);
  }
  return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

}  // extern "C"
