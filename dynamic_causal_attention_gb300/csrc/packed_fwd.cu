// packed_fwd.cu — the forward of the hybrid layer on sequences of different lengths laid
// end to end, and the frozen heads' dV: the fused kernel of attn_fwd_kernel.cuh on
// the items of a plan that packed_prep.cu makes on the device, handed out as CTAs come
// free.  Measured: 4 prompts of up to 8192 tokens (16 heads of 128 over 4, 4 frozen) 421 us,
// 1240 TFLOP/s or 63 % of the burst rate, in series of 60 calls; 436 in one of 2.6 s, over which the
// power cap takes the clock from 2.07 to 1.94 GHz.  16 of up to 4096 (12 heads of 64, 3 frozen)
// 145 us, 617 TFLOP/s.  With equal lengths it takes up to 3 % longer than the kernel for those: an item
// is claimed and passed on before it begins.
// The frozen heads' dV takes 49 us of the latter's documents; 63 with a tile for one sequence.
#include "attn_fwd_kernel.cuh"

namespace saf {

cudaError_t launch_packed_fwd(const PackedFwdLaunch& L, bool transposed, cudaStream_t s) {
  switch (L.d_h) {
    case 32:
      return transposed ? launch_fused<32, true, true>(L, s) : launch_fused<32, false, true>(L, s);
    case 64:
      return transposed ? launch_fused<64, true, true>(L, s) : launch_fused<64, false, true>(L, s);
    case 128:
      return transposed ? launch_fused<128, true, true>(L, s)
                        : launch_fused<128, false, true>(L, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace saf
