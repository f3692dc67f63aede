// gemm_w4.hip — choice of tile and K split of the 4-bit-weight product
// (gemm_w4_kernel.hpp, instantiated by gemm_w4_{bf16,f16}_{u4,e2m1}.hip), and
// the sum over the parts of a split K.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.hpp"
#include "experts.hpp"
#include "kernels.hpp"

namespace mswz {
namespace {

// D = beta*D + the parts' fp32 sums, in part order; one row piece of 256 columns per workgroup.
template <int OUT>
__global__ void __launch_bounds__(256)
w4_reduce_kernel(const float *__restrict__ ws, void *__restrict__ D, int M, int N, int ldd, int parts, int beta)
{
    const int n = blockIdx.x * 256 + threadIdx.x, m = blockIdx.y;
    if (n >= N)
        return;
    using T = std::conditional_t<OUT == kOutF32, float, std::conditional_t<OUT == kOutBf16, __bf16, _Float16>>;
    T *d = static_cast<T *>(D) + size_t(m) * ldd + n;
    float sum = beta ? float(*d) : 0.0f;
    for (int i = 0; i < parts; ++i)
        sum += ws[(size_t(i) * M + m) * N + n];
    *d = T(sum);
}

}  // namespace

int w4_rows(const W4Args &a)
{
    // rows that a tile is expected to hold: experts share them
    const int64_t rows = a.E ? (int64_t(a.M) + a.E - 1) / a.E : a.M;
    return rows > 16 ? 64 : rows > 4 ? 16 : 4;
}

// K parts of a product: 64-row tiles of 128 columns leave compute units idle
// below 256 of them, so K is split until there are as many, each part keeping
// at least four steps of 256.
static int parts_of(const W4Args &a)
{
    if (a.E || w4_rows(a) < 64)
        return 1;
    const int64_t tiles = int64_t((a.N + 127) / 128) * ((a.M + 63) / 64), steps = (a.K + 255) / 256;
    int parts = 1;
    while (parts < 8 && tiles * parts < 256 && steps / (2 * parts) >= 4)
        parts *= 2;
    return parts;
}

int64_t w4_workspace_bytes(const W4Args &a)
{
    const int parts = parts_of(a);
    return parts > 1 ? int64_t(parts) * a.M * a.N * 4 : 0;
}

hipError_t launch_w4(const W4Args &args, hipStream_t stream)
{
    W4Args a = args;
    a.parts = parts_of(a);
    const hipError_t e = a.bf16 ? (a.e2m1 ? launch_w4_bf16_e2m1(a, stream) : launch_w4_bf16_u4(a, stream))
                                : (a.e2m1 ? launch_w4_f16_e2m1(a, stream) : launch_w4_f16_u4(a, stream));
    if (a.parts == 1 || e != hipSuccess)
        return e;
    const int steps = (a.K + 255) / 256, per = (steps + a.parts - 1) / a.parts, parts = (steps + per - 1) / per;
    const dim3 grid((a.N + 255) / 256, a.M);
    if (a.out == kOutF32)
        hipLaunchKernelGGL((w4_reduce_kernel<kOutF32>), grid, dim3(256), 0, stream, a.ws, a.D, a.M, a.N, a.ldd, parts, a.beta);
    else if (a.bf16)
        hipLaunchKernelGGL((w4_reduce_kernel<kOutBf16>), grid, dim3(256), 0, stream, a.ws, a.D, a.M, a.N, a.ldd, parts, a.beta);
    else
        hipLaunchKernelGGL((w4_reduce_kernel<kOutF16>), grid, dim3(256), 0, stream, a.ws, a.D, a.M, a.N, a.ldd, parts, a.beta);
    return hipGetLastError();
}

}  // namespace mswz
