// packed_bwd.cu — the dynamic heads' backward on sequences of different lengths laid end
// to end: the kernel of attn_bwd_kernel.cuh on the items of a plan that packed_prep.cu
// makes on the device, shared out by cost (share_out in packed_prep.cu).  Measured: 16
// documents of up to 4096 tokens (9 dynamic heads of 64) 336 us, 640 TFLOP/s or 33 % of the
// burst rate; 3 of up to 8192 (12 dynamic heads of 128 over 8) 692 us, 860 TFLOP/s.  With equal
// lengths as fast as the kernel for those or 2 % faster.  Shorter sequences make shorter items,
// and K_J and V_J of an item cannot come before the last products of the one before have read
// theirs (its beginning and end cost about 3 steps).
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
