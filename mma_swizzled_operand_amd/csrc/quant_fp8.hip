// quant_fp8.hip — rows of 16- or 32-bit values to E4M3 with an fp32 scale per
// block of 128 values along a row, or per 128 x 128 tile, as they lie (Q, S)
// and transposed (QT, ST; blocks along the transposed rows), in one pass:
//     s = max(largest |x| of the block, 2^-90) / 448   (or the next power of two)
//     q = the E4M3 value nearest to x / s, ties to the even code
//
// One workgroup of 256 threads owns a 128 x 128 tile of X: both block forms
// lie inside it, so X is read once for both outputs.  A thread holds 8
// consecutive rows x 8 consecutive columns: its 16-byte loads are whole
// 256-byte row pieces over 16 lanes, a block along a row is reduced over those
// 16 lanes, and the 8 rows of a column are 8 consecutive bytes of QT, which go
// through LDS into whole 128-byte lines.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.hpp"
#include "fp8.hpp"
#include "kernels.hpp"

namespace mswz {
namespace {

// Largest of v over each row of 16 lanes, in all of them.
__device__ __forceinline__ float max16(float v)
{
    auto ror = [](float x, auto n) {
        const int i = __builtin_bit_cast(int, x);
        return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(i, i, 0x120 + decltype(n)::value, 0xF, 0xF, false));
    };
    v = fmaxf(v, ror(v, std::integral_constant<int, 8>{}));
    v = fmaxf(v, ror(v, std::integral_constant<int, 4>{}));
    v = fmaxf(v, ror(v, std::integral_constant<int, 2>{}));
    return fmaxf(v, ror(v, std::integral_constant<int, 1>{}));
}

// The scale of a block whose largest magnitude is `most` (infinite if a value
// is): most / 448, or the smallest power of two that is not below it.  A block
// of zeros, or of values below 2^-90, takes 2^-90 as its largest.
__device__ __forceinline__ float scale_of(float most, bool pow2)
{
    most = fmaxf(most, 0x1p-90f);
    if (!pow2)
        return most / 448.0f;
    // 448 = 1.75 * 2^8: a mantissa up to 1.75 needs exponent - 8, above - 7
    const uint32_t bits = __builtin_bit_cast(uint32_t, most);
    if (bits >= 0x7f800000u)
        return most;
    return __builtin_bit_cast(float, ((bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u)) << 23);
}

// What a block's values are divided with: 1 / s in two parts, so that the
// quotient comes out within (1/2 + 2^-20) ulp.
struct Divisor {
    float s, hi, lo;
    __device__ explicit Divisor(float scale) : s(scale)
    {
        hi = 1.0f / s;
        // an infinite scale: finite values give 0, infinite ones NaN
        lo = hi == 0.0f ? 0.0f : fmaf(-s, hi, 1.0f) * hi;
    }
    // A value that rounds to E4M3 as x / s does.  E4M3's values and the
    // midpoints between them have at most five significant bits; te, the
    // quotient with its last bit cleared, is within 1.5 ulp of x / s, so it
    // lies on the same side of every midpoint or on it.  The sign of the
    // exact remainder x - te s then moves it one ulp towards x / s, off the
    // midpoint and not as far as the next one.
    __device__ float operator()(float x) const
    {
        const float t = fmaf(x, hi, x * lo);
        const float te = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, t) & ~1u);
        const float r = fmaf(-te, s, x);
        const float step = te * 0x1.8p-24f;
        return te + __builtin_amdgcn_fmed3f(r * (hi * 0x1p25f), -step, step);
    }
};

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d)
{
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true));
}

template <int IN, bool TILE>
__global__ void __launch_bounds__(256)
quant_fp8_kernel(const void *__restrict__ X, uint8_t *__restrict__ Q, float *__restrict__ S, uint8_t *__restrict__ QT,
                 float *__restrict__ ST, int M, int K, int64_t ldx, int tiles_k, bool pow2)
{
    using T = std::conditional_t<IN == kOutF32, float, std::conditional_t<IN == kOutBf16, __bf16, _Float16>>;
    typedef T t8 __attribute__((ext_vector_type(8)));
    __shared__ float most[4][128];
    __shared__ __attribute__((aligned(16))) uint8_t turned[128 * 144];   // [column][row], rows of 144 bytes

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int tm = blockIdx.x / tiles_k, tk = blockIdx.x - tm * tiles_k;
    const int m0 = tm * 128, k0 = tk * 128;
    const int rg = tid >> 4, cg = tid & 15;         // this thread's 8 rows and 8 columns
    const int m = m0 + 8 * rg, k = k0 + 8 * cg;
    const bool in_k = k < K;                         // (K % 16 == 0: the 8 columns are inside together)
    t8 x[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        x[r] = t8{};
        if (in_k && m + r < M)
            x[r] = *reinterpret_cast<const t8 *>(static_cast<const T *>(X) + int64_t(m + r) * ldx + k);
    }
    // (fmaxf passes the other operand over a NaN: a NaN takes no part)
    float row_most[8], col_most[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        row_most[i] = col_most[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            row_most[i] = fmaxf(row_most[i], fabsf(float(x[i][j])));
            col_most[i] = fmaxf(col_most[i], fabsf(float(x[j][i])));
        }
    }
    const int Mp = (M + 15) & ~15, blocks_m = (M + 127) / 128;
    if constexpr (TILE) {
        float all = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            all = fmaxf(all, row_most[i]);
        all = max16(all);
        if (cg == 0)
            most[0][rg] = all;
        __syncthreads();
        all = max16(most[0][lane & 15]);
        const float s = scale_of(all, pow2);
        if (tid == 0) {
            if (Q)
                S[int64_t(tm) * tiles_k + tk] = s;
            if (QT)
                ST[int64_t(tk) * blocks_m + tm] = s;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            row_most[i] = col_most[i] = s;   // the scales, below
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            row_most[i] = scale_of(max16(row_most[i]), pow2);
            if (Q && cg == 0 && m + i < M)
                S[int64_t(tk) * M + m + i] = row_most[i];
        }
        if (QT) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float v = col_most[j];
                v = fmaxf(v, __shfl_xor(v, 16));
                v = fmaxf(v, __shfl_xor(v, 32));
                if (lane < 16)
                    most[wave][8 * cg + j] = v;
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = 8 * cg + j;
                col_most[j] = scale_of(fmaxf(fmaxf(most[0][c], most[1][c]), fmaxf(most[2][c], most[3][c])), pow2);
                if (rg == 0 && in_k)
                    ST[int64_t(tm) * K + k + j] = col_most[j];
            }
        }
    }
    if (Q) {
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const Divisor by(row_most[r]);
            u32x2 q;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                q[h] = pack4(by(float(x[r][4 * h])), by(float(x[r][4 * h + 1])), by(float(x[r][4 * h + 2])),
                             by(float(x[r][4 * h + 3])));
            if (in_k && m + r < M)
                *reinterpret_cast<u32x2 *>(Q + int64_t(m + r) * K + k) = q;
        }
    }
    if (QT) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const Divisor by(col_most[j]);
            u32x2 q;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                q[h] = pack4(by(float(x[4 * h][j])), by(float(x[4 * h + 1][j])), by(float(x[4 * h + 2][j])),
                             by(float(x[4 * h + 3][j])));
            *reinterpret_cast<u32x2 *>(turned + (8 * cg + j) * 144 + 8 * rg) = q;
        }
        __syncthreads();
        // 16 bytes a thread, 8 threads a column
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = 32 * i + (tid >> 3), piece = 16 * (tid & 7);
            if (k0 + c < K && m0 + piece < Mp)
                *reinterpret_cast<u32x4 *>(QT + int64_t(k0 + c) * Mp + m0 + piece) =
                    *reinterpret_cast<const u32x4 *>(turned + c * 144 + piece);
        }
    }
}

template <int IN>
hipError_t launch(const QuantArgs &a, hipStream_t stream)
{
    const int tiles_k = (a.K + 127) / 128;
    const dim3 grid(uint32_t((a.M + 127) / 128) * uint32_t(tiles_k));
    if (a.tile)
        hipLaunchKernelGGL((quant_fp8_kernel<IN, true>), grid, dim3(256), 0, stream, a.X, a.Q, a.S, a.QT, a.ST, a.M, a.K,
                           a.ldx, tiles_k, a.pow2);
    else
        hipLaunchKernelGGL((quant_fp8_kernel<IN, false>), grid, dim3(256), 0, stream, a.X, a.Q, a.S, a.QT, a.ST, a.M, a.K,
                           a.ldx, tiles_k, a.pow2);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_fp8(const QuantArgs &a, hipStream_t stream)
{
    return a.dt == kOutF32 ? launch<kOutF32>(a, stream)
         : a.dt == kOutBf16 ? launch<kOutBf16>(a, stream) : launch<kOutF16>(a, stream);
}

}  // namespace mswz
