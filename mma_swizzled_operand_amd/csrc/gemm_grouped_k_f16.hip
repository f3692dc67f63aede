// gemm_grouped_k_f16.hip — instantiations of the grouped product for f16 operands, grouped along K
// (both operands MN-major).
#include "gemm_grouped_kernel.hpp"

namespace mswz {

hipError_t launch_grouped_k_f16(const GroupedArgs &a, hipStream_t stream)
{
    return launch_grouped_kind<false, true, true>(a, stream);
}

}  // namespace mswz
