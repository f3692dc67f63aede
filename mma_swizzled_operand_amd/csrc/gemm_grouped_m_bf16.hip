// gemm_grouped_m_bf16.hip — instantiations of the grouped product for bf16 operands, rows grouped along M.
#include "gemm_grouped_kernel.hpp"

namespace mswz {

hipError_t launch_grouped_m_bf16(const GroupedArgs &a, hipStream_t stream)
{
    return a.b_mn ? launch_grouped_kind<true, false, true>(a, stream) : launch_grouped_kind<true, false, false>(a, stream);
}

}  // namespace mswz
