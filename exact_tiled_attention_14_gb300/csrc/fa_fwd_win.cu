// fa_fwd_win.cu — the forward variants for sliding windows with sinks and
// shared key/value heads: widths 64 and 128 x bf16/fp16.
#include "fa_launch.cuh"

namespace fa {

cudaError_t launch_fwd_win(const FwdParams& p, int grid, int d, bool bf16, cudaStream_t stream) {
  if (d == 64)
    return bf16 ? launch_variant<64, true, true, false, true, false, true>(p, grid, stream)
                : launch_variant<64, false, true, false, true, false, true>(p, grid, stream);
  return bf16 ? launch_variant<128, true, true, false, true, false, true>(p, grid, stream)
              : launch_variant<128, false, true, false, true, false, true>(p, grid, stream);
}

}  // namespace fa
