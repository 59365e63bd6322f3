// fa_bwd_win.cu — the backward variants for sliding windows with sinks and
// shared key/value heads: widths 64 and 128 x bf16/fp16.
#include "fa_bwd_launch.cuh"

namespace fa {

cudaError_t launch_bwd_win(const BwdParams& p, const void* o, const void* dout, float* delta, int d,
                           bool bf16, int sms, cudaStream_t stream) {
  if (d == 64)
    return bf16
               ? launch_bwd_variant<64, true, true, false, true, true>(p, o, dout, delta, sms,
                                                                       stream)
               : launch_bwd_variant<64, false, true, false, true, true>(p, o, dout, delta, sms,
                                                                        stream);
  return bf16
             ? launch_bwd_variant<128, true, true, false, true, true>(p, o, dout, delta, sms, stream)
             : launch_bwd_variant<128, false, true, false, true, true>(p, o, dout, delta, sms,
                                                                       stream);
}

}  // namespace fa
