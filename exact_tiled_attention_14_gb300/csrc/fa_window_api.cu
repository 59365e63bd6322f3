// fa_window_api.cu — the sliding-window entry points fa_fwd_window and
// fa_bwd_window of the C ABI declared in include/fa.h: argument checks, TMA
// descriptors and the launches of the kernels' window variants.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "fa.h"
#include "fa_bwd_launch.cuh"
#include "fa_host.cuh"
#include "fa_launch.cuh"

using namespace fa::host;

namespace {

constexpr long long kMaxLen = 1ll << 30;   // queries plus keys: positions fit in int

// Sizes, widths, dtype and scale of a window call, in the documented order.
int check_window_sizes(int B, int H, int Hk, int Nq, int Nk, int d, int causal, int window,
                       int sinks, float scale, int dtype) {
  if (B < 0 || H < 0 || Hk < 0 || Nq < 0 || Nk < 0 || d <= 0) return FA_ERR_SHAPE;
  if (H > 0 ? (Hk <= 0 || H % Hk != 0) : Hk != 0) return FA_ERR_SHAPE;
  if (causal != 1 && causal != 2) return FA_ERR_SHAPE;
  if (window < 1 || sinks < 0) return FA_ERR_SHAPE;
  if (static_cast<long long>(Nq) + Nk > kMaxLen) return FA_ERR_SHAPE;
  const long long bh = static_cast<long long>(B) * H;
  const long long tiles = (static_cast<long long>(Nq) + fa::kBM - 1) / fa::kBM +
                          (static_cast<long long>(Nk) + fa::kBN - 1) / fa::kBN;
  // (a sink tile is cut into at most 64 parts, each a work item)
  if (bh > kMaxLen || bh * tiles > kMaxLen / 64) return FA_ERR_SHAPE;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED_D;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_DTYPE;
  if (!std::isfinite(scale) || !(scale > 0.0f)) return FA_ERR_SCALE;
  return FA_OK;
}

// Cut of the sink tiles of the backward pass: every query tile after a sink
// tile visits it, where a window's tile is visited by about window / 128 + 2,
// and the CTAs' work is dealt by items.  So a sink tile is cut into as many
// parts as give each the steps of a window's tile (a training step of B1
// H32/8 N16384 d128 window 2048 with 64 sinks: 2150 us, against 3015 with
// whole tiles, of which 8 of 152 CTAs hold one with half of a CTA's whole
// share each).  kMaxParts parts in all, four for each of 152 SMs, even the
// work out and bound the workspace (80 MB at d = 128); more sink tiles than
// that are dealt whole.  (A constant of GB300's 152 SMs, not the device's count:
// the size call is host-only and answers the same on every machine.)
constexpr long long kMaxParts = 608;
struct SinkSplit {
  int tiles = 0, parts = 1;
};
SinkSplit sink_split(int BHk, int Nq, int Nk, int window, int sinks) {
  SinkSplit s;
  const int used = std::min(sinks, Nk);
  if (used == 0 || BHk == 0) return s;
  const int tiles = (used + fa::kBwdTile - 1) / fa::kBwdTile;
  const long long q_tiles = (static_cast<long long>(Nq) + fa::kBwdTile - 1) / fa::kBwdTile;
  const long long per = static_cast<long long>(window) / fa::kBwdTile + 2;
  const long long parts = std::min<long long>((q_tiles + per - 1) / per,
                                              kMaxParts / (static_cast<long long>(BHk) * tiles));
  if (parts < 2) return s;
  s.tiles = tiles;
  s.parts = static_cast<int>(parts);
  return s;
}

bool misaligned(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

unsigned long long watchdog_cycles() {
  // counted in SM cycles, converted at the part's highest clock (2.1 GHz)
  const unsigned long long wd = g_watchdog_ns.load();
  return (wd ? wd : kDefaultWatchdogNs) * 21ull / 10ull;
}

}  // namespace

extern "C" {

int fa_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                  int Hk, int Nq, int Nk, int d, int causal, int window, int sinks,
                  const int* seqlens_k, float scale, int dtype, cudaStream_t stream) {
  const int rc = check_window_sizes(B, H, Hk, Nq, Nk, d, causal, window, sinks, scale, dtype);
  if (rc != FA_OK) return rc;
  if (B == 0 || H == 0 || Nq == 0) return FA_OK;   // nothing to write
  if (!q || !o || !lse || (Nk > 0 && (!k || !v))) return FA_ERR_NULLPTR;
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(o, 16) ||
      misaligned(lse, 4) || misaligned(seqlens_k, 4))
    return FA_ERR_ALIGN;

  int dev = 0;
  const DeviceInfo* info = device_info(&dev);
  if (!info || !info->supported) return FA_ERR_DEVICE;
  if (info->err != FA_OK) return info->err;

  const bool bf16 = dtype == FA_BF16;
  const int bh = B * H, bhk = B * Hk;
  fa::FwdParams p{};
  // With no keys no key tile is ever loaded; the maps still need a row and
  // an address (k, v may then be NULL: q stands in).
  const int nk_rows = Nk > 0 ? Nk : 1;
  const void* kp = Nk > 0 ? k : q;
  const void* vp = Nk > 0 ? v : q;
  if (!make_tmap(&p.tm_q, q, bh, Nq, d, bf16) ||
      !make_tmap(&p.tm_k, kp, Nk > 0 ? bhk : 1, nk_rows, d, bf16) ||
      !make_tmap(&p.tm_v, vp, Nk > 0 ? bhk : 1, nk_rows, d, bf16) ||
      !make_tmap(&p.tm_o, o, bh, Nq, d, bf16))
    return FA_ERR_TENSORMAP;
  p.o = o;
  p.lse = lse;
  p.trace = g_trace.load();
  p.status = info->status;
  p.watchdog_cycles = watchdog_cycles();
  p.BH = bh;
  p.N = Nq;
  p.n_qblk = (Nq + 2 * fa::kBM - 1) / (2 * fa::kBM);
  p.n_kv = (Nk + fa::kBN - 1) / fa::kBN;
  p.num_units = bh * p.n_qblk;
  // The query heads that read one key/value head are dealt together, block
  // by block, so the CTAs at work share that head's windows in L2.
  p.hgroup = H / Hk;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.Nk = Nk;
  p.H = H;
  p.seqlens_k = seqlens_k;
  p.align_br = causal == 2 ? 1 : 0;
  p.dqk = d;
  p.dv = d;
  set_dropout(&p, 256, 0, 0);
  // a window or sink count past every length hides nothing more
  p.win = std::min(window, std::max(Nq, Nk) + 1);
  p.sinks = std::min(sinks, Nk);
  p.Hk = Hk;
  const int grid = p.num_units < info->sms ? p.num_units : info->sms;
  return fa::launch_fwd_win(p, grid, d, bf16, stream) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

int fa_bwd_window_workspace_size(int B, int H, int Hk, int Nq, int Nk, int d, int window, int sinks,
                                 size_t* bytes) {
  if (!bytes) return FA_ERR_NULLPTR;
  const int rc = check_window_sizes(B, H, Hk, Nq, Nk, d, 1, window, sinks, 1.0f, FA_BF16);
  if (rc != FA_OK) return rc;
  const SinkSplit sp = sink_split(B * Hk, Nq, Nk, window, sinks);
  *bytes = static_cast<size_t>(B) * Hk * sp.tiles * sp.parts * fa::kBwdTile * 2 * d * sizeof(float);
  return FA_OK;
}

int fa_bwd_window(const void* q, const void* k, const void* v, const void* o, const float* lse,
                  const void* dout, void* dq, void* dk, void* dv, float* delta, int B, int H,
                  int Hk, int Nq, int Nk, int d, int causal, int window, int sinks,
                  const int* seqlens_k, float scale, int dtype, void* workspace,
                  size_t workspace_bytes, cudaStream_t stream) {
  const int rc = check_window_sizes(B, H, Hk, Nq, Nk, d, causal, window, sinks, scale, dtype);
  if (rc != FA_OK) return rc;
  if (B == 0 || H == 0 || (Nq == 0 && Nk == 0)) return FA_OK;   // nothing to write
  if (Nq > 0 && (!q || !o || !lse || !dout || !dq || !delta)) return FA_ERR_NULLPTR;
  if (Nk > 0 && (!k || !v || !dk || !dv)) return FA_ERR_NULLPTR;
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(o, 16) ||
      misaligned(dout, 16) || misaligned(dq, 16) || misaligned(dk, 16) || misaligned(dv, 16) ||
      misaligned(lse, 4) || misaligned(delta, 4) || misaligned(seqlens_k, 4))
    return FA_ERR_ALIGN;
  size_t need = 0;
  fa_bwd_window_workspace_size(B, H, Hk, Nq, Nk, d, window, sinks, &need);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return FA_ERR_WORKSPACE;
    if (misaligned(workspace, 256)) return FA_ERR_ALIGN;
  }

  int dev = 0;
  const DeviceInfo* info = device_info(&dev);
  if (!info || !info->supported) return FA_ERR_DEVICE;
  if (info->err != FA_OK) return info->err;

  const bool bf16 = dtype == FA_BF16;
  const int bh = B * H, bhk = B * Hk;
  fa::BwdParams p{};
  // Without queries or keys no tile of them is ever loaded; the maps still
  // need a row and an address.
  const bool has_q = Nq > 0, has_k = Nk > 0;
  if (!make_tmap(&p.tm_q, has_q ? q : k, has_q ? bh : 1, has_q ? Nq : 1, d, bf16) ||
      !make_tmap(&p.tm_do, has_q ? dout : k, has_q ? bh : 1, has_q ? Nq : 1, d, bf16) ||
      !make_tmap(&p.tm_k, has_k ? k : q, has_k ? bhk : 1, has_k ? Nk : 1, d, bf16) ||
      !make_tmap(&p.tm_v, has_k ? v : q, has_k ? bhk : 1, has_k ? Nk : 1, d, bf16))
    return FA_ERR_TENSORMAP;
  p.width_qk = d;
  p.width_v = d;
  p.lse = lse;
  p.delta = delta;
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  p.status = info->status;
  p.watchdog_cycles = watchdog_cycles();
  p.BH = bh;
  p.N = Nq;
  p.n_tiles = (Nq + fa::kBwdTile - 1) / fa::kBwdTile;
  p.Nk = Nk;
  p.n_ktiles = (Nk + fa::kBwdTile - 1) / fa::kBwdTile;
  p.H = H;
  p.seqlens_k = seqlens_k;
  p.align_br = causal == 2 ? 1 : 0;
  p.scale = scale;
  p.scale_log2 = scale * 1.4426950408889634f;
  set_dropout(&p, 256, 0, 0);
  p.item_group = H / Hk;   // dQ items: the heads that read one key/value head together
  p.win = std::min(window, std::max(Nq, Nk) + 1);
  p.sinks = std::min(sinks, Nk);
  p.Hk = Hk;
  p.G = H / Hk;
  p.BHk = bhk;
  const SinkSplit sp = sink_split(B * Hk, Nq, Nk, window, sinks);
  p.split_tiles = sp.tiles;
  p.split_parts = sp.parts;
  p.split_ws = static_cast<float*>(workspace);
  return fa::launch_bwd_win(p, o, dout, delta, d, bf16, info->sms, stream) == cudaSuccess
             ? FA_OK
             : FA_ERR_LAUNCH;
}

}  // extern "C"
