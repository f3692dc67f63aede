// gemm_fp8.hip — launches of the E4M3 product with a scale per block of 128
// (gemm_fp8_kernel.hpp) by the kernel that fp8_choice.hpp names, and the sum over
// the parts of a split K.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fp8_choice.hpp"
#include "gemm_fp8_kernel.hpp"

namespace mswz {
namespace {

// D = beta*D + the parts' sums, in part order; four columns a thread.
__global__ void __launch_bounds__(256)
fp8_reduce_kernel(Fp8Args a, int parts, bool vec)
{
    const int64_t pitch = fp8_part_pitch(a.N), pieces = pitch / 4, all = pieces * a.M;
    const int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (id >= all)
        return;
    const int m = int(id / pieces), n = int(id % pieces) * 4;
    f32x4 v = f32x4{};
    for (int p = 0; p < parts; ++p)
        v += *reinterpret_cast<const f32x4 *>(a.ws + (int64_t(p) * a.M + m) * pitch + n);
    fp8_store(a, m, n, v, vec);
}

template <int BM, int BN, int WM, int WN, int S, int P, bool ROWB, int OUT>
hipError_t launch_tile(const Fp8Args &a, hipStream_t stream, int parts = 1)
{
    const int tiles_m = (a.M + BM - 1) / BM, tiles_n = (a.N + BN - 1) / BN, per = (a.kb + parts - 1) / parts;
    parts = (a.kb + per - 1) / per;
    hipLaunchKernelGGL((gemm_fp8_kernel<BM, BN, WM, WN, S, P, ROWB, OUT == kOutF32, OUT>),
                       dim3(uint32_t(tiles_m) * uint32_t(tiles_n), parts), dim3(64 * (BM / WM) * (BN / WN)), 0, stream, a,
                       tiles_m, tiles_n, -4, per, parts == 1 && fp8_whole_lines(a) ? 2 : int(fp8_whole_stores(a)));
    if (parts > 1)
        hipLaunchKernelGGL(fp8_reduce_kernel, dim3(uint32_t((fp8_part_pitch(a.N) / 4 * a.M + 255) / 256)), dim3(256), 0,
                           stream, a, parts, fp8_whole_stores(a));
    return hipGetLastError();
}

template <bool ROWB, int OUT>
hipError_t launch_out(const Fp8Args &a, hipStream_t stream)
{
    constexpr bool F32 = OUT == kOutF32;
    switch (fp8_kernel(a)) {
    case kFp8Few: return launch_fp8_skinny(a, stream);
    case kFp8Split: return launch_tile<64, 64, 32, 32, 6, 2, ROWB, OUT>(a, stream, fp8_parts(a));
    case kFp8Tile32x64: return launch_tile<32, 64, 16, 32, 6, 2, ROWB, OUT>(a, stream);
    case kFp8Tile64x64: return launch_tile<64, 64, 16, 64, 4, 1, ROWB, OUT>(a, stream);
    case kFp8Tile128x64: return launch_tile<128, 64, 16, 64, 4, 1, ROWB, OUT>(a, stream);
    case kFp8Tile128x128: return launch_tile<128, 128, 32, 64, 4, 1, ROWB, OUT>(a, stream);
    case kFp8Tile128x128Twice: return launch_tile<128, 128, ROWB || F32 ? 64 : 32, 64, 2, 1, ROWB, OUT>(a, stream);
    case kFp8Tile256x256:
        if constexpr (!F32)
            return launch_tile<256, 256, 128, 64, 2, 1, ROWB, OUT>(a, stream);
    }
    return hipErrorUnknown;
}

template <bool ROWB>
hipError_t launch_rows(const Fp8Args &a, hipStream_t stream)
{
    return a.out == kOutF32 ? launch_out<ROWB, kOutF32>(a, stream)
         : a.out == kOutBf16 ? launch_out<ROWB, kOutBf16>(a, stream) : launch_out<ROWB, kOutF16>(a, stream);
}

}  // namespace

int64_t fp8_workspace_bytes(const Fp8Args &a)
{
    const int parts = fp8_parts(a);
    return parts > 1 ? parts * a.M * fp8_part_pitch(a.N) * 4 : 0;
}

hipError_t launch_fp8(const Fp8Args &a, hipStream_t stream)
{
    return a.tile ? launch_rows<false>(a, stream) : launch_rows<true>(a, stream);
}

}  // namespace mswz
