// packed_fwd.cu — the forward of the hybrid layer on sequences of different lengths laid
// end to end, and the frozen heads' dV: the fused kernel of attn_fwd_kernel.cuh on
// the items of a plan that packed_prep.cu makes on the device.
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
