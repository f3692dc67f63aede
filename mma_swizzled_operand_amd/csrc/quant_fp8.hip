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
//
// Bound by the memory: 16384 x 4096 bf16 by rows, both ways, 58.4 us; 8192 x 8192
// by tiles, both ways, 57.2; 4.7 TB/s (a copy: 4.9); as they lie alone 41.6 and
// 38.1, transposed alone 45.4 and 44.4.  fp32: both ways 81.0 and 82.2 (5.0 TB/s),
// alone 61.8 and 61.4, 69.3 and 69.2.
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

// What a block counts as its largest magnitude.
__device__ __forceinline__ float largest(float most) { return fmaxf(most, 0x1p-90f); }

// The scale of a block of that largest magnitude (infinite if a value is):
// most / 448, or the smallest power of two that is not below it.
__device__ __forceinline__ float scale_of(float most, bool pow2)
{
    if (!pow2)
        return most / 448.0f;
    // 448 = 1.75 * 2^8: a mantissa up to 1.75 needs exponent - 8, above - 7
    const uint32_t bits = __builtin_bit_cast(uint32_t, most);
    if (bits >= 0x7f800000u)
        return most;
    return __builtin_bit_cast(float, ((bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u)) << 23);
}

// What the values of a block are divided with: 1 / s in two parts, so that
// x hi + x lo is within (1/2 + 2^-6) ulp of x / s (the lower part is subnormal, with
// an error of 2^-31 of the upper one, where s is near fp32's largest) and x / s
// itself where that is a value of fp32.  The result need not be the quotient: it has to lie on the
// quotient's side of every midpoint between two E4M3 values (five significant
// bits at most), or on it.
//
// 16-bit x (p = 8 or 11 bits).  x, the block's largest A and a midpoint m are
// integers X < 2^p, A < 2^p, u < 2^5 times powers of two, so x / (A / 448) either
// is m, or 7 X 2^i and u A 2^j differ by one at least, i.e. by 2^-16 of
// themselves.  s is A / 448 within 2^-24, so only in the first case can x / s be
// close to m, and then it lies above or below as s was rounded down or up: the
// same way for all of a block, which the lower part of 1 / s takes in with a
// step of 2^-20.  (s exact, or a power of two: no step, and the quotient comes
// out exactly.)  The upper part is 2^-19 of itself below 1 / s, so that the lower
// one is above zero with either step: with parts of opposite signs -0 would
// become 0.
//
// fp32 x.  te, the sum with its last bit cleared, is within 1.5 ulp of x / s, so
// it lies on the same side of every midpoint or on it.  The sign of the exact
// remainder x - te s then moves it one ulp towards x / s, off the midpoint and
// not as far as the next one; a zero gets its sign back at the end.
template <int IN>
struct Divisor {
    float hi, lo, s;   // (s: fp32 x only)

    __device__ Divisor() {}
    __device__ Divisor(float scale, float most, bool pow2) : s(scale)
    {
        const float inverse = 1.0f / s;
        // an infinite scale: finite values give 0, infinite ones NaN
        hi = lo = 0.0f;
        if (inverse == 0.0f)
            return;
        hi = IN == kOutF32 ? inverse : inverse * (1.0f - 0x1p-19f);
        float rest = fmaf(-s, hi, 1.0f);
        if (IN != kOutF32 && !pow2) {
            const float over = fmaf(s, 448.0f, -most);   // (the sign is exact)
            rest += over > 0.0f ? -0x1p-20f : over < 0.0f ? 0x1p-20f : 0.0f;
        }
        lo = rest * inverse;
    }
    __device__ float operator()(float x) const
    {
        const float t = fmaf(x, hi, x * lo);
        if constexpr (IN != kOutF32)
            return t;
        const float te = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, t) & ~1u);
        const float r = fmaf(-te, s, x);
        const float step = te * 0x1.8p-24f;
        return copysignf(te + __builtin_amdgcn_fmed3f(r * (hi * 0x1p25f), -step, step), x);
    }
};

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d)
{
    // (what the first conversion leaves of its old value, the second replaces)
    const int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, __builtin_bit_cast(int, a), false);
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true));
}

// PAST: the values go past the caches.
template <bool PAST, typename V>
__device__ __forceinline__ void store(V *to, V v)
{
    if constexpr (PAST)
        __builtin_nontemporal_store(v, to);
    else
        *to = v;
}

template <int IN, bool TILE, bool PAST>
__global__ void __launch_bounds__(256)
quant_fp8_kernel(const void *__restrict__ X, uint8_t *__restrict__ Q, float *__restrict__ S, uint8_t *__restrict__ QT,
                 float *__restrict__ ST, int M, int K, int64_t ldx, int tiles_k, bool pow2)
{
    using T = std::conditional_t<IN == kOutF32, float, std::conditional_t<IN == kOutBf16, __bf16, _Float16>>;
    typedef T t8 __attribute__((ext_vector_type(8)));
    // the largest of each row, and of each column by wave; then the rows' and the
    // columns' divisors
    __shared__ float most[5][128];
    __shared__ Divisor<IN> divisors[2][128];
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
    Divisor<IN> by_row[8], by_col[8];
    if constexpr (TILE) {
        float all = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            all = fmaxf(all, row_most[i]);
        all = max16(all);
        if (cg == 0)
            most[0][rg] = all;
        __syncthreads();
        all = largest(max16(most[0][lane & 15]));
        const float s = scale_of(all, pow2);
        if (tid == 0) {
            if (Q)
                S[int64_t(tm) * tiles_k + tk] = s;
            if (QT)
                ST[int64_t(tk) * blocks_m + tm] = s;
        }
        by_row[0] = Divisor<IN>(s, all, pow2);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            by_row[i] = by_col[i] = by_row[0];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = max16(row_most[i]);
            if (cg == 0)
                most[4][8 * rg + i] = v;
            float c = col_most[i];
            c = fmaxf(c, __shfl_xor(c, 16));
            c = fmaxf(c, __shfl_xor(c, 32));
            if (lane < 16)
                most[wave][8 * cg + i] = c;
        }
        __syncthreads();
        // one row or column a thread
        const int at = tid & 127;
        const bool col = tid >= 128;
        const float v = largest(col ? fmaxf(fmaxf(most[0][at], most[1][at]), fmaxf(most[2][at], most[3][at])) : most[4][at]);
        const float s = scale_of(v, pow2);
        divisors[col][at] = Divisor<IN>(s, v, pow2);
        if (!col && Q && m0 + at < M)
            S[int64_t(tk) * M + m0 + at] = s;
        if (col && QT && k0 + at < K)
            ST[int64_t(tm) * K + k0 + at] = s;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            by_row[i] = divisors[0][8 * rg + i];
            by_col[i] = divisors[1][8 * cg + i];
        }
    }
    if (Q) {
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const Divisor<IN> by = by_row[r];
            u32x2 q;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                q[h] = pack4(by(float(x[r][4 * h])), by(float(x[r][4 * h + 1])), by(float(x[r][4 * h + 2])),
                             by(float(x[r][4 * h + 3])));
            if (in_k && m + r < M)
                store<PAST>(reinterpret_cast<u32x2 *>(Q + int64_t(m + r) * K + k), q);
        }
    }
    if (QT) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const Divisor<IN> by = by_col[j];
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
                store<PAST>(reinterpret_cast<u32x4 *>(QT + int64_t(k0 + c) * Mp + m0 + piece),
                            *reinterpret_cast<const u32x4 *>(turned + c * 144 + piece));
        }
    }
}

template <int IN, bool TILE, bool PAST>
hipError_t launch_as(const QuantArgs &a, hipStream_t stream)
{
    const int tiles_k = (a.K + 127) / 128;
    hipLaunchKernelGGL((quant_fp8_kernel<IN, TILE, PAST>), dim3(uint32_t((a.M + 127) / 128) * uint32_t(tiles_k)), dim3(256),
                       0, stream, a.X, a.Q, a.S, a.QT, a.ST, a.M, a.K, a.ldx, tiles_k, a.pow2);
    return hipGetLastError();
}

template <int IN>
hipError_t launch(const QuantArgs &a, hipStream_t stream)
{
    // what the L2s do not hold is stored past them (16384 x 4096 bf16 both ways:
    // 62.9 us through them, 58.5 past them)
    if (int64_t(a.M) * a.K > int64_t(32) << 20)
        return a.tile ? launch_as<IN, true, true>(a, stream) : launch_as<IN, false, true>(a, stream);
    return a.tile ? launch_as<IN, true, false>(a, stream) : launch_as<IN, false, false>(a, stream);
}

}  // namespace

hipError_t launch_quant_fp8(const QuantArgs &a, hipStream_t stream)
{
    return a.dt == kOutF32 ? launch<kOutF32>(a, stream)
         : a.dt == kOutBf16 ? launch<kOutBf16>(a, stream) : launch<kOutF16>(a, stream);
}

}  // namespace mswz
