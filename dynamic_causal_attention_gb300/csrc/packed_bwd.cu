// packed_bwd.cu — the dynamic heads' backward on sequences of different lengths laid end
// to end: the kernel of attn_bwd_kernel.cuh on the items of a plan that packed_prep.cu
// makes on the device.
#include "attn_bwd_kernel.cuh"

namespace saf {

cudaError_t launch_packed_bwd(const PackedBwdLaunch& L, cudaStream_t s) {
  switch (L.d_h) {
    case 32: return launch_dyn<32, true>(L, s);
    case 64: return launch_dyn<64, true>(L, s);
    case 128: return launch_dyn<128, true>(L, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace saf
