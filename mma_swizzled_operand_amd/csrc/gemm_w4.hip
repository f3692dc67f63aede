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

// D = beta*D + the parts' fp32 sums, in part order; 1024 columns of a row per
// workgroup, a thread's four columns loaded together.
template <int OUT>
__global__ void __launch_bounds__(256)
w4_reduce_kernel(const float *__restrict__ ws, void *__restrict__ D, int M, int N, int ldd, int parts, int beta)
{
    using T = std::conditional_t<OUT == kOutF32, float, std::conditional_t<OUT == kOutBf16, __bf16, _Float16>>;
    const int n0 = blockIdx.x * 1024 + threadIdx.x, m = blockIdx.y;
    T *const d = static_cast<T *>(D) + size_t(m) * ldd;
    float sum[4];
#pragma unroll
    for (int c = 0; c < 4; ++c)
        sum[c] = beta ? float(d[min(n0 + 256 * c, N - 1)]) : 0.0f;
    for (int i = 0; i < parts; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            sum[c] += ws[(size_t(i) * M + m) * N + min(n0 + 256 * c, N - 1)];
#pragma unroll
    for (int c = 0; c < 4; ++c)
        if (n0 + 256 * c < N)
            d[n0 + 256 * c] = T(sum[c]);
}

}  // namespace

int w4_rows(const W4Args &a)
{
    // rows that a tile is expected to hold: experts share them (16384 x 8192, u4:
    // one row in tiles of 4 takes 13.5 us, 16 in tiles of 16 15.9, 64 in tiles
    // of 64 31.4).  An expert with more has more tiles, whose weights come from
    // the L2: 128 rows and 32 experts of 4096 x 2048 take 46 us spread evenly,
    // 27 if all of them go to one expert.
    const int64_t rows = a.E ? (int64_t(a.M) + a.E - 1) / a.E : a.M;
    return rows > 16 ? 64 : rows > 4 ? 16 : 4;
}

int64_t w4_tiles64(const W4Args &a) { return a.E ? (a.E < a.M ? a.E : a.M) : (a.M + 63) / 64; }

// K parts of a product: where tiles of 64 rows by 64 columns leave half of the
// compute units idle, K is split between those of 64 x 128 until there are as
// many, each part keeping at least four steps of 256.  (64 rows by K 8192, 64
// columns unsplit / split and added up: N 4096, U4 29.8 / 17.8 us, 8192: 30.7 /
// 23.3, 10240: 30.7 / 37.3, 14336: 31.3 / 40.2; FP4 23.9 / 15.9, 23.8 / 19.4,
// 24.1 / 29.9, 24.7 / 33.9.)
static int parts_of(const W4Args &a)
{
    if (a.E || w4_rows(a) < 64 || w4_tiles64(a) * ((a.N + 63) / 64) > 128)
        return 1;
    const int64_t tiles = w4_tiles64(a) * ((a.N + 127) / 128), steps = (a.K + 255) / 256;
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
    const dim3 grid((a.N + 1023) / 1024, a.M);
    if (a.out == kOutF32)
        hipLaunchKernelGGL((w4_reduce_kernel<kOutF32>), grid, dim3(256), 0, stream, a.ws, a.D, a.M, a.N, a.ldd, parts, a.beta);
    else if (a.bf16)
        hipLaunchKernelGGL((w4_reduce_kernel<kOutBf16>), grid, dim3(256), 0, stream, a.ws, a.D, a.M, a.N, a.ldd, parts, a.beta);
    else
        hipLaunchKernelGGL((w4_reduce_kernel<kOutF16>), grid, dim3(256), 0, stream, a.ws, a.D, a.M, a.N, a.ldd, parts, a.beta);
    return hipGetLastError();
}

}  // namespace mswz
