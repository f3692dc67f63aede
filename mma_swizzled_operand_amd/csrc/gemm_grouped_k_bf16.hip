// gemm_grouped_k_bf16.hip — instantiations of the grouped product for bf16 operands, grouped along K
// (both operands MN-major).
#include "gemm_grouped_kernel.hpp"

namespace mswz {

hipError_t launch_grouped_k_bf16(const GroupedArgs &a, hipStream_t stream)
{
    return launch_grouped_kind<true, true, true>(a, stream);
}

}  // namespace mswz
