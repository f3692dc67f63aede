// gemm_w4_f16_u4.hip — instantiations of the 4-bit-weight product: f16 activations, u4 weights.
#include "gemm_w4_kernel.hpp"

namespace mswz {

hipError_t launch_w4_f16_u4(const W4Args &a, hipStream_t stream) { return launch_w4_kind<false, false>(a, stream); }

}  // namespace mswz
