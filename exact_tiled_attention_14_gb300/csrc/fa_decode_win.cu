// fa_decode_win.cu — the entry points fa_decode_window and fa_decode_tree of
// the C ABI declared in include/fa.h: argument checks, TMA descriptors and
// the launches of the tensor-core decoding kernels.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "fa.h"
#include "fa_decode_win_kernel.cuh"
#include "fa_host.cuh"

using namespace fa::host;

namespace fa {
namespace {

// Copies of the rows in the query tile (see the kernel's header).
int copies_of(int R) { return R <= kDwTile / 4 ? 4 : (R <= kDwTile / 2 ? 2 : 1); }

template <int D, bool kBf16, int kTiles, int kCopies>
cudaError_t launch_main(const DecWinParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};   // devices on which the smem limit was raised
  auto kernel = fa_decode_win_kernel<D, kBf16, kTiles, kCopies>;
  constexpr int kAlloc = DwLayout<D, kTiles>::kAlloc;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done.load() & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kAlloc);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit);
  }
  kernel<<<p.grid, kDwThreads, kAlloc, stream>>>(p);
  return cudaGetLastError();
}

template <int D, bool kBf16>
cudaError_t launch_variant(const DecWinParams& p, cudaStream_t stream) {
  const int copies = copies_of(p.R);
  cudaError_t e = p.row_span > kDwTile ? launch_main<D, kBf16, 2, 1>(p, stream)
                  : copies == 4        ? launch_main<D, kBf16, 1, 4>(p, stream)
                  : copies == 2        ? launch_main<D, kBf16, 1, 2>(p, stream)
                                       : launch_main<D, kBf16, 1, 1>(p, stream);
  if (e != cudaSuccess) return e;
  // Programmatic dependent launch: the combine grid is set up while the main
  // kernel runs its last CTAs, and waits on the device for the parts.
  cudaLaunchConfig_t cfg = {};
  const int rows = 1 << p.combine_rows;
  const int groups = std::max(D / 4 * rows / kDwCombineThreads, 1);
  cfg.gridDim = dim3(p.grid, (p.slot_rows + rows - 1) / rows * groups);
  cfg.blockDim = dim3(kDwCombineThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // Where units are cut into two or three parts, a thread with registers for
  // three lets more of them run at a time (40 against 72 registers; 128 rows
  // of 16 caches, 128 units: the call 72.5 us, 77.5 with eight); many parts
  // are loaded eight at a time, one wait for each eight.
  const bool few = p.grid <= 2ll * p.B * p.Hk * p.row_blocks;
  return few ? cudaLaunchKernelEx(&cfg, fa_decode_win_combine_kernel<D, kBf16, 3>, p)
             : cudaLaunchKernelEx(&cfg, fa_decode_win_combine_kernel<D, kBf16, 8>, p);
}

constexpr long long kMaxCount = 1ll << 30;
constexpr long long kMaxRowTiles = (1ll << 31) - 1;

// Sizes and widths, in the documented order.
int check_sizes(int B, int H, int Hk, int Nq, int Nk, int d, int max_q) {
  if (B < 0 || H < 0 || Hk < 0 || Nk < 0 || d <= 0) return FA_ERR_SHAPE;
  if (H > 0 ? (Hk <= 0 || H % Hk != 0) : Hk != 0) return FA_ERR_SHAPE;
  if (Nq < 1 || Nq > max_q) return FA_ERR_SHAPE;
  const long long heads = static_cast<long long>(B) * H;
  if (Nk > kMaxCount || heads > kMaxCount || heads * Nq > kMaxCount) return FA_ERR_SHAPE;
  // rows times the key tiles of a whole cache: the tiles of all units fit in int
  if (heads * Nq * ((Nk + kDwTile - 1ll) / kDwTile + 1) > kMaxRowTiles) return FA_ERR_SHAPE;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED_D;
  return FA_OK;
}

// Grid (one CTA per SM, or one per key tile where there are fewer) and the
// workspace: two parts per CTA, each the rows of a unit, and the run table.
struct Plan {
  int row_span, row_blocks, slot_rows, grid;
  size_t o_bytes, ml_bytes, bytes;
};
Plan make_plan(int B, int H, int Hk, int Nq, int Nk, int d, int sms) {
  Plan pl{};
  const int R = H / Hk * Nq;
  pl.row_span = R <= kDwTile ? kDwTile : 2 * kDwTile;
  pl.row_blocks = (R + pl.row_span - 1) / pl.row_span;
  pl.slot_rows = std::min(R, pl.row_span);
  // no unit has more tiles than its whole cache and one more of padding
  const long long tiles = (static_cast<long long>(Nk) + kDwTile - 1) / kDwTile + 1;
  const long long units = static_cast<long long>(B) * Hk * pl.row_blocks;
  pl.grid = static_cast<int>(std::min<long long>(units * tiles, sms));
  const size_t rows = 2 * static_cast<size_t>(pl.grid) * pl.slot_rows;
  pl.o_bytes = (rows * d * sizeof(float) + 255) / 256 * 256;
  pl.ml_bytes = (rows * sizeof(float2) + 255) / 256 * 256;
  pl.bytes = pl.o_bytes + pl.ml_bytes + (pl.grid * sizeof(int4) + 255) / 256 * 256;
  return pl;
}

int decode(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int Hk,
           int Nq, int Nk, int d, bool is_tree, const unsigned long long* tree, int window,
           int sinks, const int* seqlens, float scale, int dtype, void* workspace,
           size_t workspace_bytes, cudaStream_t stream) {
  const int rc = check_sizes(B, H, Hk, Nq, Nk, d, is_tree ? kDwMaxTree : kDwMaxTokens);
  if (rc != FA_OK) return rc;
  if (window < (is_tree ? 0 : 1) || sinks < 0) return FA_ERR_SHAPE;
  if (is_tree && Nk < Nq) return FA_ERR_SHAPE;   // the drafted tokens' keys are in the cache
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_DTYPE;
  if (!std::isfinite(scale) || !(scale > 0.0f)) return FA_ERR_SCALE;
  if (B == 0 || H == 0) return FA_OK;            // nothing to write
  if (!q || !o || !lse || (Nk > 0 && (!k || !v)) || (is_tree && !tree)) return FA_ERR_NULLPTR;
  auto misaligned = [](const void* p, uintptr_t n) {
    return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0;
  };
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(o, 16) ||
      misaligned(lse, 4) || misaligned(seqlens, 4) || misaligned(tree, 8))
    return FA_ERR_ALIGN;

  int dev = 0;
  const DeviceInfo* info = device_info(&dev);
  if (!info || !info->supported) return FA_ERR_DEVICE;
  if (info->err != FA_OK) return info->err;
  const Plan pl = make_plan(B, H, Hk, Nq, Nk, d, info->sms);
  if (!workspace || workspace_bytes < pl.bytes) return FA_ERR_WORKSPACE;
  if (misaligned(workspace, 256)) return FA_ERR_ALIGN;

  const bool bf16 = dtype == FA_BF16;
  const int bhk = B * Hk, R = H / Hk * Nq;
  DecWinParams p{};
  // without keys one box of the queries stands in; its rows are masked
  const bool has_k = Nk > 0;
  const void* kp = has_k ? k : q;
  const void* vp = has_k ? v : q;
  const int kh = has_k ? bhk : 1, kn = has_k ? Nk : 1;
  const int q_box = R <= kDwTile ? kDwTile / copies_of(R) : kDwTile;
  const int kv_box = dec_big_box(R > kDwTile ? 2 : 1);
  if (!make_tmap(&p.tm_q, q, bhk, R, d, bf16, q_box) ||
      !make_tmap(&p.tm_k, kp, kh, kn, d, bf16, kv_box) ||
      !make_tmap(&p.tm_v, vp, kh, kn, d, bf16, kv_box) ||
      !make_tmap(&p.tm_k16, kp, kh, kn, d, bf16, kDwBox) ||
      !make_tmap(&p.tm_v16, vp, kh, kn, d, bf16, kDwBox))
    return FA_ERR_TENSORMAP;
  p.o = o;
  p.lse = lse;
  p.part_o = static_cast<float4*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + pl.o_bytes);
  p.cut = reinterpret_cast<int4*>(static_cast<uint8_t*>(workspace) + pl.o_bytes + pl.ml_bytes);
  p.status = info->status;
  const unsigned long long wd = g_watchdog_ns.load();
  p.watchdog_cycles = (wd ? wd : kDefaultWatchdogNs) * 21ull / 10ull;
  p.seqlens = seqlens;
  p.tree = is_tree ? tree : nullptr;
  p.len_all = is_tree ? Nk - Nq : Nk;
  p.B = B;
  p.Hk = Hk;
  p.Nq = Nq;
  p.Nk = Nk;
  p.R = R;
  p.row_span = pl.row_span;
  p.row_blocks = pl.row_blocks;
  p.slot_rows = pl.slot_rows;
  while (p.combine_rows < 5 && (1 << p.combine_rows) < pl.slot_rows) ++p.combine_rows;
  p.grid = pl.grid;
  // a window past every position hides nothing, as none (0, tree) does
  const int all = Nk + Nq + 1;
  p.win = window == 0 ? all : std::min(window, all);
  p.sinks = std::min(sinks, Nk);
  p.scale_log2 = scale * 1.4426950408889634f;
  cudaError_t e;
  if (d == 64)
    e = bf16 ? launch_variant<64, true>(p, stream) : launch_variant<64, false>(p, stream);
  else
    e = bf16 ? launch_variant<128, true>(p, stream) : launch_variant<128, false>(p, stream);
  return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

}  // namespace
}  // namespace fa

extern "C" {

int fa_decode_window_workspace_size(int B, int H, int Hk, int Nq, int Nk, int d, size_t* bytes) {
  if (!bytes) return FA_ERR_NULLPTR;
  const int rc = fa::check_sizes(B, H, Hk, Nq, Nk, d, fa::kDwMaxTree);
  if (rc != FA_OK) return rc;
  *bytes = 0;
  if (B == 0 || H == 0) return FA_OK;
  int dev = 0;
  const DeviceInfo* info = device_info(&dev);
  if (!info || !info->supported) return FA_ERR_DEVICE;
  *bytes = fa::make_plan(B, H, Hk, Nq, Nk, d, info->sms).bytes;
  return FA_OK;
}

int fa_decode_window(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                     int Hk, int Nq, int Nk, int d, int window, int sinks, const int* seqlens_k,
                     float scale, int dtype, void* workspace, size_t workspace_bytes,
                     cudaStream_t stream) {
  return fa::decode(q, k, v, o, lse, B, H, Hk, Nq, Nk, d, false, nullptr, window, sinks, seqlens_k,
                    scale, dtype, workspace, workspace_bytes, stream);
}

int fa_decode_tree(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                   int Hk, int Nq, int Nk, int d, const unsigned long long* tree, int window,
                   int sinks, const int* seqlens_k, float scale, int dtype, void* workspace,
                   size_t workspace_bytes, cudaStream_t stream) {
  return fa::decode(q, k, v, o, lse, B, H, Hk, Nq, Nk, d, true, tree, window, sinks, seqlens_k,
                    scale, dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
