// gemm_w4_bf16_e2m1.hip — instantiations of the 4-bit-weight product: bf16 activations, e2m1 weights.
#include "gemm_w4_kernel.hpp"

namespace mswz {

hipError_t launch_w4_bf16_e2m1(const W4Args &a, hipStream_t stream) { return launch_w4_kind<true, true>(a, stream); }

}  // namespace mswz
