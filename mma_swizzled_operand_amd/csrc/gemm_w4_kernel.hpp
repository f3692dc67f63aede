// gemm_w4_kernel.hpp — products of a few rows of 16-bit activations with 4-bit
// weights, included by the units that instantiate it (gemm_w4_*.hip):
//     D[m][n] = beta*D + sum_g s[n][g] sum_{k in g} A[m][k] (w[n][k] - z[n][g])
//
// The weights are streamed once from memory straight into registers, turned
// into 16-bit MFMA operands there (exactly: 4-bit values have few significant
// bits) and multiplied against the activations with 16x16x32 MFMAs; a scale
// multiplies the fp32 sum of its group, so no weight is rounded.
//
// One workgroup of eight waves owns 16*NB columns of D and 16*MB rows; its
// waves split K in chunks of 128 (64 bytes of every weight row per wave and
// load, 512 bytes of a row by the workgroup's eight neighbours), each keeps
// fp32 sums of its own, and the sums meet in LDS at the end, added in wave
// order.
//
// Lane l = (r, q) = (l % 16, l / 16) loads 16 bytes of weight row r, K block q
// (32 values) of the chunk.  MFMA j multiplies dword j of every lane.  The K
// order inside the chunk is free as long as A follows it, but a scale group
// must not be shared by one MFMA with another one: for groups shorter than the
// chunk the lanes' dwords are exchanged first (two or four lane swaps per 16
// bytes) so that each MFMA's 32 K values lie in one group.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.hpp"
#include "experts.hpp"
#include "kernels.hpp"

namespace mswz {
namespace {

constexpr int kW4Waves = 8;
constexpr int kChunk = 128;     // K values of one 16-byte load of all four lane groups

typedef uint32_t u32v2 __attribute__((ext_vector_type(2)));

// Four 4-bit integers at bits 0-3, 4-7, 8-11, 12-15 of both halves of a dword
// become four pairs of 16-bit floats: pair i holds the values at bits 4i and
// 16 + 4i, i.e. elements i and i + 4 of the dword's eight.
//   fp16: 1024 + q has q in the last bits of its significand; subtracting
//         1024 + z is exact, and so is q - z;
//   bf16: 1 + q/16 has q in the upper four of its seven significand bits; the
//         product sum is corrected by (1 + z/16) times the sum of A and
//         multiplied by 16 s.
template <bool BF16>
__device__ __forceinline__ u32x4 u4_values(uint32_t w, uint32_t zz)
{
    u32x4 v;
    if constexpr (BF16) {
        v[0] = ((w << 3) & 0x00780078u) | 0x3f803f80u;
        v[1] = ((w >> 1) & 0x00780078u) | 0x3f803f80u;
        v[2] = ((w >> 5) & 0x00780078u) | 0x3f803f80u;
        v[3] = ((w >> 9) & 0x00780078u) | 0x3f803f80u;
    } else {
        typedef _Float16 h2 __attribute__((ext_vector_type(2)));
        const h2 z = __builtin_bit_cast(h2, zz);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t b = ((w >> (4 * i)) & 0x000f000fu) | 0x64006400u;
            v[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2, b) - z);
        }
    }
    return v;
}

// Eight E2M1 values, in element order.
template <bool BF16>
__device__ __forceinline__ u32x4 e2m1_values(uint32_t w)
{
    u32x4 v;
    if constexpr (BF16) {
        v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0));
        v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1));
        v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2));
        v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3));
    } else {
        v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0));
        v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1));
        v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2));
        v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3));
    }
    return v;
}

// A's eight values in the order u4_values gives the weights: (0,4)(1,5)(2,6)(3,7).
__device__ __forceinline__ u32x4 u4_order(u32x4 a)
{
    return u32x4{__builtin_amdgcn_perm(a[2], a[0], 0x05040100u), __builtin_amdgcn_perm(a[2], a[0], 0x07060302u),
                 __builtin_amdgcn_perm(a[3], a[1], 0x05040100u), __builtin_amdgcn_perm(a[3], a[1], 0x07060302u)};
}

__device__ __forceinline__ void swap32(uint32_t &a, uint32_t &b)
{
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t &a, uint32_t &b)
{
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

// SPAN: K values that share a scale inside a chunk, 32, 64 or 128.  After
// w4_arrange dword j of lane group q holds K block kb, dword kw of the chunk,
// so that MFMA j's values lie in one span.
template <int SPAN>
__device__ __forceinline__ void w4_arrange(u32x4 &w)
{
    if constexpr (SPAN < 128) {
        uint32_t a = w[0], b = w[1], c = w[2], d = w[3];
        swap32(a, c);   // c of lane groups 0, 1 <-> a of groups 2, 3
        swap32(b, d);
        if constexpr (SPAN == 32) {
            swap16(a, b);
            swap16(c, d);
        }
        w = u32x4{a, b, c, d};
    }
}
template <int SPAN>
__device__ __forceinline__ int w4_koff(int j, int q)
{
    if constexpr (SPAN == 128)
        return 32 * q + 8 * j;
    else if constexpr (SPAN == 64)
        return 32 * ((q & 1) + 2 * (j >> 1)) + 8 * ((j & 1) + 2 * (q >> 1));
    else
        return 32 * j + 8 * q;
}

// 2^(e - 127), e = 255 NaN
__device__ __forceinline__ float e8m0_value(uint32_t e)
{
    return __builtin_bit_cast(float, e == 0 ? 0x00400000u : e == 255 ? 0x7fc00000u : e << 23);
}

template <bool BF16>
__device__ __forceinline__ float scale16(uint16_t b)
{
    if constexpr (BF16)
        return __builtin_bit_cast(float, uint32_t(b) << 16);
    else
        return float(__builtin_bit_cast(_Float16, b));
}

struct W4Kernel {
    const uint8_t *A;
    const uint8_t *B;
    const uint8_t *S;
    const uint8_t *Z;
    const int32_t *offsets;
    void *D;
    int M, N, K, E;
    int group, groups;
    int lda, ldd;
    int beta;
};

template <bool BF16, bool E2M1, int SPAN, int MB, int NB, int OUT>
__global__ void __launch_bounds__(64 * kW4Waves)
w4_kernel(W4Kernel p)
{
    constexpr int kTiles = MB * NB;
    __shared__ __attribute__((aligned(16))) float red[kW4Waves][kTiles][64][4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int n0 = blockIdx.x * (16 * NB);
    int e = 0, tile = blockIdx.y, lo = 0, hi = p.M;
    if (p.offsets && !group_of_tile(p.offsets, p.E, p.M, 16 * MB, blockIdx.y, lane, e, tile, lo, hi))
        return;
    const int m0 = lo + 16 * MB * tile, rows = min(hi - m0, 16 * MB);

    const uint32_t row_bytes = uint32_t(p.K) / 2;
    const uint32_t w_bytes = uint32_t(p.N) * row_bytes;
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.B + size_t(e) * w_bytes, w_bytes);
    const uint32_t a_bytes = uint32_t(rows - 1) * uint32_t(p.lda) * 2 + uint32_t(p.K) * 2;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.A + size_t(m0) * p.lda * 2, a_bytes);
    // scales of this lane's weight rows (rows beyond N repeat the last one)
    const size_t sbase = size_t(e) * p.N * p.groups;

    f32x4 acc[NB][MB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
            acc[nb][mb] = f32x4{};
    const uint32_t one = BF16 ? 0x3f803f80u : 0x3c003c00u;
    const u32x4 ones = {one, one, one, one};

    const int chunks = (p.K + kChunk - 1) / kChunk;
    for (int c = wave; c < chunks; c += kW4Waves) {
        const int k0 = c * kChunk;
        u32x4 w[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const uint32_t row = n0 + 16 * nb + r;
            const uint32_t off = row * row_bytes + uint32_t(k0 / 2 + 16 * q);
            w[nb] = buffer_load16(rw, int(row) < p.N && k0 + 32 * q < p.K ? off : w_bytes, 0);
            w4_arrange<SPAN>(w[nb]);
        }
        u32x4 a[MB][4];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = k0 + w4_koff<SPAN>(j, q), m = 16 * mb + r;
                const u32x4 v = buffer_load16(ra, m < rows && k < p.K ? uint32_t(m * p.lda + k) * 2 : a_bytes, 0);
                a[mb][j] = E2M1 ? v : u4_order(v);
            }
        // the chunk's spans: MFMAs 4 s / spans ..
        constexpr int kSpans = 128 / SPAN, kPer = 4 / kSpans;
#pragma unroll
        for (int s = 0; s < kSpans; ++s) {
            if (k0 + SPAN * s >= p.K)
                break;
            const int g = (k0 + SPAN * s) / p.group;
            f32x4 asum[MB];
            if constexpr (BF16 && !E2M1) {
#pragma unroll
                for (int mb = 0; mb < MB; ++mb) {
                    asum[mb] = f32x4{};
#pragma unroll
                    for (int j = 0; j < kPer; ++j)
                        asum[mb] = mfma_16x16x32<BF16>(a[mb][kPer * s + j], ones, asum[mb]);
                }
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const size_t si = sbase + size_t(min(n0 + 16 * nb + r, p.N - 1)) * p.groups + g;
                float scale;
                uint32_t z = 8;
                if constexpr (E2M1) {
                    scale = e8m0_value(p.S[si]);
                } else {
                    scale = scale16<BF16>(reinterpret_cast<const uint16_t *>(p.S)[si]);
                    if (p.Z)
                        z = p.Z[si];
                }
                const uint32_t zz = (0x6400u + z) * 0x10001u;   // 1024 + z, twice (z below 256: no carry)
                f32x4 part[MB];
#pragma unroll
                for (int mb = 0; mb < MB; ++mb)
                    part[mb] = f32x4{};
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const uint32_t d = w[nb][kPer * s + j];
                    u32x4 v;
                    if constexpr (E2M1)
                        v = e2m1_values<BF16>(d);
                    else
                        v = u4_values<BF16>(d, zz);
#pragma unroll
                    for (int mb = 0; mb < MB; ++mb)
                        part[mb] = mfma_16x16x32<BF16>(a[mb][kPer * s + j], v, part[mb]);
                }
#pragma unroll
                for (int mb = 0; mb < MB; ++mb) {
                    if constexpr (BF16 && !E2M1) {
                        const float zs = 1.0f + float(z) * 0.0625f;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[nb][mb][i] = __builtin_fmaf(scale * 16.0f, __builtin_fmaf(-zs, asum[mb][i], part[mb][i]),
                                                            acc[nb][mb][i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[nb][mb][i] = __builtin_fmaf(scale, part[mb][i], acc[nb][mb][i]);
                    }
                }
            }
        }
    }

    // sums over waves: tile (nb, mb) is added up and stored by wave tile % 8;
    // lane holds column r of the 16, rows 4q .. 4q+3
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
            *reinterpret_cast<f32x4 *>(red[wave][nb * MB + mb][lane]) = acc[nb][mb];
    __syncthreads();
    for (int tl = wave; tl < kTiles; tl += kW4Waves) {
        f32x4 sum = *reinterpret_cast<const f32x4 *>(red[0][tl][lane]);
#pragma unroll
        for (int w = 1; w < kW4Waves; ++w)
            sum += *reinterpret_cast<const f32x4 *>(red[w][tl][lane]);
        const int n = n0 + 16 * (tl / MB) + r, mb = tl % MB;
        if (n >= p.N)
            continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = 16 * mb + 4 * q + i;
            if (m >= rows)
                continue;
            const size_t at = size_t(m0 + m) * p.ldd + n;
            using T = std::conditional_t<OUT == kOutF32, float, std::conditional_t<OUT == kOutBf16, __bf16, _Float16>>;
            T *d = static_cast<T *>(p.D) + at;
            *d = T(p.beta ? sum[i] + float(*d) : sum[i]);
        }
    }
}

template <bool BF16, bool E2M1, int SPAN, int MB, int NB>
hipError_t launch_w4_tile(const W4Args &a, hipStream_t stream)
{
    const W4Kernel p{static_cast<const uint8_t *>(a.A), a.B, static_cast<const uint8_t *>(a.S), a.Z, a.offsets, a.D,
                     a.M, a.N, a.K, a.E, a.group, a.groups, a.lda, a.ldd, a.beta};
    const int64_t tiles = a.offsets ? most_tiles(a.E, a.M, 16 * MB) : (a.M + 16 * MB - 1) / (16 * MB);
    const dim3 grid((a.N + 16 * NB - 1) / (16 * NB), unsigned(tiles));
    if (a.out == kOutF32)
        hipLaunchKernelGGL((w4_kernel<BF16, E2M1, SPAN, MB, NB, kOutF32>), grid, dim3(64 * kW4Waves), 0, stream, p);
    else
        hipLaunchKernelGGL((w4_kernel<BF16, E2M1, SPAN, MB, NB, BF16 ? kOutBf16 : kOutF16>), grid, dim3(64 * kW4Waves), 0,
                           stream, p);
    return hipGetLastError();
}

template <bool BF16, bool E2M1, int SPAN>
hipError_t launch_w4_span(const W4Args &a, hipStream_t stream)
{
    return a.M <= 16 || (a.offsets && a.M <= 16 * int64_t(a.E)) ? launch_w4_tile<BF16, E2M1, SPAN, 1, 2>(a, stream)
                                                               : launch_w4_tile<BF16, E2M1, SPAN, 4, 2>(a, stream);
}

template <bool BF16, bool E2M1>
hipError_t launch_w4_kind(const W4Args &a, hipStream_t stream)
{
    if constexpr (!E2M1) {
        if (a.group % 128 == 0)
            return launch_w4_span<BF16, E2M1, 128>(a, stream);
        if (a.group == 64)
            return launch_w4_span<BF16, E2M1, 64>(a, stream);
    }
    return launch_w4_span<BF16, E2M1, 32>(a, stream);
}

}  // namespace
}  // namespace mswz
