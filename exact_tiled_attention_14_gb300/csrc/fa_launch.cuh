// fa_launch.cuh — host-side launch of one compiled variant of the forward kernel.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "fa_fwd_kernel.cuh"

namespace fa {

// The parameters of a windowed launch at width D: the order of its units'
// tiles, which decode_unit reads from them, is the kernel's own.
template <int D>
FwdParams win_launch_params(FwdParams p) {
  p.gap_first = win_gap_first(D);
  return p;
}

// Launch fa_fwd_kernel<D, kBf16, kCausal, kSplit, kKv, kDrop, kWin> with `grid` persistent CTAs.
template <int D, bool kBf16, bool kCausal, bool kSplit, bool kKv = false, bool kDrop = false,
          bool kWin = false>
cudaError_t launch_variant(const FwdParams& p, int grid, cudaStream_t stream) {
  static std::atomic<uint64_t> attr_done{0};  // devices on which the smem limit was raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load() & bit)) {
    e = cudaFuncSetAttribute(fa_fwd_kernel<D, kBf16, kCausal, kSplit, kKv, kDrop, kWin>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D, kDrop, kWin>::kAlloc);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit);
  }
  auto kernel = fa_fwd_kernel<D, kBf16, kCausal, kSplit, kKv, kDrop, kWin>;
  constexpr int kThreads = threads_of<D, kDrop>(), kAlloc = Smem<D, kDrop, kWin>::kAlloc;
  if constexpr (kWin)
    kernel<<<grid, kThreads, kAlloc, stream>>>(win_launch_params<D>(p));
  else
    kernel<<<grid, kThreads, kAlloc, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_fwd_d64(const FwdParams& p, int grid, bool bf16, bool causal,
                           cudaStream_t stream);
cudaError_t launch_fwd_d128(const FwdParams& p, int grid, bool bf16, bool causal,
                            cudaStream_t stream);
// Queries against a key set of their own length (the kKv variants).
cudaError_t launch_fwd_kv_d64(const FwdParams& p, int grid, bool bf16, bool causal,
                              cudaStream_t stream);
cudaError_t launch_fwd_kv_d128(const FwdParams& p, int grid, bool bf16, bool causal,
                               cudaStream_t stream);
// Square calls with dropout on the attention weights (the kKv, kDrop variants).
cudaError_t launch_fwd_drop_d64(const FwdParams& p, int grid, bool bf16, bool causal,
                                cudaStream_t stream);
cudaError_t launch_fwd_drop_d128(const FwdParams& p, int grid, bool bf16, bool causal,
                                 cudaStream_t stream);
// Sliding-window calls with sinks and shared key/value heads (the kKv,
// kCausal, kWin variants).
cudaError_t launch_fwd_win(const FwdParams& p, int grid, int d, bool bf16, cudaStream_t stream);

}  // namespace fa
