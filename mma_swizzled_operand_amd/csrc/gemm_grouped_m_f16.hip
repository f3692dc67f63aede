// gemm_grouped_m_f16.hip — instantiations of the grouped product for f16 operands, rows grouped along M.
#include "gemm_grouped_kernel.hpp"

namespace mswz {

hipError_t launch_grouped_m_f16(const GroupedArgs &a, hipStream_t stream)
{
    return a.b_mn ? launch_grouped_kind<false, false, true>(a, stream) : launch_grouped_kind<false, false, false>(a, stream);
}

}  // namespace mswz
