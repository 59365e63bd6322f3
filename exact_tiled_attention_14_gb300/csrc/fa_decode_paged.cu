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
  kernel<<<p.out.grid, DpLayout<D, kTiles>::kThreads, kAlloc, stream>>>(p);
  return cudaGetLastError();
}

template <int D, bool kBf16, bool kInt8>
cudaError_t launch_variant(const DecPagedParams& p, cudaStream_t stream) {
  cudaError_t e = p.out.row_span == 8    ? launch_main<D, kBf16, kInt8, 1>(p, stream)
                  : p.out.row_span == 16 ? launch_main<D, kBf16, kInt8, 2>(p, stream)
                                         : launch_main<D, kBf16, kInt8, 4>(p, stream);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int rows = 1 << p.out.combine_rows;
  const int groups = std::max(D / 4 * rows / kDwCombineThreads, 1);
  cfg.gridDim = dim3(p.out.grid, (p.out.slot_rows + rows - 1) / rows * groups);
  cfg.blockDim = dim3(kDwCombineThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_decode_win_combine_kernel<D, kBf16, 8>, p.out);
}

constexpr int kMaxTokens = 16;

// Rows of a unit (8, 16 or 32), grid (one CTA per SM, or one per key tile where
// there are fewer) and the workspace: two parts per CTA, and the run table.
struct Plan {
  int row_span, row_blocks, slot_rows, grid;
  size_t o_bytes, ml_bytes, bytes;
};
// Tiles of all units at most: whole capacities, and one of each sequence's own.
long long max_tiles(int B, int Hk, int row_blocks, int d, int capacity) {
  const long long tiles = (static_cast<long long>(capacity) + dp_keys(d) - 1) / dp_keys(d) + 1;
  return static_cast<long long>(B) * Hk * row_blocks * tiles;
}
int row_span_of(int R) { return R <= 8 ? 8 : R <= 16 ? 16 : 32; }
int check_sizes(int B, int H, int Hk, int Nq, int d, int page_size, int pages_per_seq) {
  if (H < 0 || (H > 0 ? (Hk <= 0 || H % Hk != 0) : Hk != 0)) return FA_ERR_SHAPE;
  if (Nq < 1 || Nq > kMaxTokens) return FA_ERR_SHAPE;
  if (static_cast<long long>(B) * H * Nq > (1 << 30)) return FA_ERR_SHAPE;
  if (B == 0 || H == 0) return FA_OK;
  const int R = H / Hk * Nq, span = row_span_of(R);
  // the numbers of all tiles fit in int
  if (max_tiles(B, Hk, (R + span - 1) / span, d, pages_per_seq * page_size) >= (1ll << 31))
    return FA_ERR_SHAPE;
  return FA_OK;
}
Plan make_plan(int B, int H, int Hk, int Nq, int d, int capacity, int sms) {
  Plan pl{};
  const int R = H / Hk * Nq;
  pl.row_span = row_span_of(R);
  pl.row_blocks = (R + pl.row_span - 1) / pl.row_span;
  pl.slot_rows = std::min(R, pl.row_span);
  pl.grid = static_cast<int>(
      std::min<long long>(max_tiles(B, Hk, pl.row_blocks, d, capacity), sms));
  const size_t rows = 2 * static_cast<size_t>(pl.grid) * pl.slot_rows;
  pl.o_bytes = (rows * d * sizeof(float) + 255) / 256 * 256;
  pl.ml_bytes = (rows * sizeof(float2) + 255) / 256 * 256;
  pl.bytes = pl.o_bytes + pl.ml_bytes + (pl.grid * sizeof(int4) + 255) / 256 * 256;
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
  const int capacity = pages_per_seq * page_size, keys = fa::dp_keys(d);
  const fa::Plan pl = fa::make_plan(B, H, Hk, Nq, d, capacity, info->sms);
  if (!workspace || workspace_bytes < pl.bytes) return FA_ERR_WORKSPACE;
  if (misaligned(workspace, 256)) return FA_ERR_ALIGN;

  fa::DecPagedParams p{};
  // one box a tile where a page holds whole tiles, else one per 16 keys
  p.boxes = page_size % keys == 0 ? 1 : keys / fa::kPageRows;
  const long long rows = static_cast<long long>(pages) * Hk * page_size;
  if (!make_tmap_codes(&p.tm_k, k_cache, rows, d, keys / p.boxes) ||
      !make_tmap_codes(&p.tm_v, v_cache, rows, d, keys / p.boxes))
    return FA_ERR_TENSORMAP;
  p.q = q;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.table = page_table;
  p.per_seq = pages_per_seq;
  p.pages = pages;
  p.page = page_size;
  fa::DecWinParams& out = p.out;
  out.o = o;
  out.lse = lse;
  out.part_o = static_cast<float4*>(workspace);
  out.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + pl.o_bytes);
  out.cut = reinterpret_cast<int4*>(static_cast<uint8_t*>(workspace) + pl.o_bytes + pl.ml_bytes);
  out.status = info->status;
  const unsigned long long wd = g_watchdog_ns.load();
  out.watchdog_cycles = (wd ? wd : kDefaultWatchdogNs) * 21ull / 10ull;
  out.seqlens = seqlens;
  out.B = B;
  out.Hk = Hk;
  out.Nq = Nq;
  out.R = H / Hk * Nq;
  out.row_span = pl.row_span;
  out.row_blocks = pl.row_blocks;
  out.slot_rows = pl.slot_rows;
  while (out.combine_rows < 5 && (1 << out.combine_rows) < pl.slot_rows) ++out.combine_rows;
  out.grid = pl.grid;
  const int all = capacity + Nq + 1;
  out.win = window == 0 ? all : std::min(window, all);
  out.sinks = std::min(sinks, capacity);
  out.scale_log2 = scale * 1.4426950408889634f;
  const bool bf16 = dtype == FA_BF16;
  cudaError_t e;
  if (cache_dtype == FA_INT8) {
    if (d == 64)
      e = bf16 ? fa::launch_variant<64, true, true>(p, stream)
               : fa::launch_variant<64, false, true>(p, stream);
    else
      e = bf16 ? fa::launch_variant<128, true, true>(p, stream)
               : fa::launch_variant<128, false, true>(p, stream);
  } else {
    if (d == 64)
      e = bf16 ? fa::launch_variant<64, true, false>(p, stream)
               : fa::launch_variant<64, false, false>(p, stream);
    else
      e = bf16 ? fa::launch_variant<128, true, false>(p, stream)
               : fa::launch_variant<128, false, false>(p, stream);
  }
  return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

}  // extern "C"
