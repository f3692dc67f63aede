// gemm_fp8.hip — choice of tile and K split of the E4M3 product with a scale
// per block of 128 (gemm_fp8_kernel.hpp), and the sum over the parts of a
// split K.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gemm_fp8_kernel.hpp"

namespace mswz {
namespace {

template <int BM, int BN, int WM, int WN, bool ROWB, int OUT>
hipError_t launch_tile(const Fp8Args &a, hipStream_t stream)
{
    const int tiles_m = (a.M + BM - 1) / BM, tiles_n = (a.N + BN - 1) / BN;
    const dim3 grid(uint32_t(tiles_m) * uint32_t(tiles_n), 1);
    hipLaunchKernelGGL((gemm_fp8_kernel<BM, BN, WM, WN, ROWB, OUT == kOutF32, OUT>), grid,
                       dim3(64 * (BM / WM) * (BN / WN)), 0, stream, a, tiles_m, tiles_n, -4, a.kb, fp8_whole_stores(a));
    return hipGetLastError();
}

template <bool ROWB, int OUT>
hipError_t launch_out(const Fp8Args &a, hipStream_t stream)
{
    if (int64_t((a.M + 255) / 256) * ((a.N + 255) / 256) >= 256)
        return launch_tile<256, 256, 128, 64, ROWB, OUT>(a, stream);
    return launch_tile<128, 128, 64, 64, ROWB, OUT>(a, stream);
}

template <bool ROWB>
hipError_t launch_rows(const Fp8Args &a, hipStream_t stream)
{
    return a.out == kOutF32 ? launch_out<ROWB, kOutF32>(a, stream)
         : a.out == kOutBf16 ? launch_out<ROWB, kOutBf16>(a, stream) : launch_out<ROWB, kOutF16>(a, stream);
}

}  // namespace

int64_t fp8_workspace_bytes(const Fp8Args &) { return 0; }

hipError_t launch_fp8(const Fp8Args &a, hipStream_t stream)
{
    if (a.M <= 64)
        return launch_fp8_skinny(a, stream);
    return a.tile ? launch_rows<false>(a, stream) : launch_rows<true>(a, stream);
}

}  // namespace mswz
