// gemm_fp8_skinny.hip — the E4M3 product with a scale per block of 128 for up
// to 32 rows of A (decoding): B is streamed once from memory straight into
// registers.
//
// One workgroup of eight waves owns all rows of A and 16 rows of B; its waves
// share out the K blocks, so there is no barrier until their sums meet in
// LDS.  A lane holds 32 bytes of a block of its row (chunks g and g + 4 of 16
// bytes, g = l/16; the order of K inside a block is free), for A's rows as for
// B's, kept kDepth blocks ahead in registers.  One 16x16x128 MFMA onto zero
// gives a block's sums (bf16 MFMAs for an fp32 D, see gemm_fp8_kernel.hpp), B's
// fragment first: a lane's four results are columns 4g .. 4g+3 of row l % 16.
//
// Bound by the memory and the time a launch takes: 1 x 4096 x 4096 6.6 us a call,
// of which the kernel is 5.9; 1 x 8192 x 8192 fp32 16.4 us, 4.1 TB/s.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gemm_fp8_kernel.hpp"

namespace mswz {
namespace {

constexpr int kSkinnyWaves = 8;

template <int NT, bool ROWB, bool EXACT>
__global__ void __launch_bounds__(64 * kSkinnyWaves)
gemm_fp8_skinny_kernel(Fp8Args a, bool vec)
{
    constexpr int W = kSkinnyWaves;
    constexpr int kRegs = 8 * (1 + NT) + NT + (ROWB ? 4 : 1);
    constexpr int kDepth = 4 * kRegs <= 120 ? 4 : 3 * kRegs <= 120 ? 3 : 2;
    __shared__ __attribute__((aligned(16))) f32x4 sums[W][NT][64];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int x16 = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const int u0 = a.kb * wave / W, u1 = a.kb * (wave + 1) / W;

    const uint32_t a_bytes = uint32_t(a.M - 1) * uint32_t(a.lda) + uint32_t(a.K);
    const uint32_t b_bytes = uint32_t(min(16, a.N - n0) - 1) * uint32_t(a.ldb) + uint32_t(a.K);
    const uint32_t sa_bytes = uint32_t(a.kb) * uint32_t(a.M) * 4;
    const uint32_t sb_bytes = uint32_t(a.kb) * uint32_t(ROWB ? a.N : (a.N + 127) / 128) * 4;
    const __amdgpu_buffer_rsrc_t a_rsrc = make_rsrc(a.A, a_bytes), b_rsrc = make_rsrc(a.B + int64_t(n0) * a.ldb, b_bytes);
    const __amdgpu_buffer_rsrc_t sa_rsrc = make_rsrc(a.SA, sa_bytes), sb_rsrc = make_rsrc(a.SB, sb_bytes);
    // a partial last block: whether this lane's chunk g (g + 4) lies beyond K
    const int rest = a.K % 128 ? a.K % 128 : 128;
    const bool beyond[2] = {16 * g >= rest, 16 * (g + 4) >= rest};

    struct Block {
        u32x4 b[2], x[NT][2];
        float sa[NT], sb[ROWB ? 4 : 1];
    };
    // the i-th block of this wave, zeros behind its last (what lies behind an
    // operand is asked for at the end of the buffer's range, which reads zeros)
    // (workgroups start at different blocks: rows a power of two apart lie in
    // the same channel of the L2; 2 to 5 %)
    const int n = u1 - u0, rot = n ? int(blockIdx.x / 8) % n : 0;
    auto load = [&](Block &d, int i) {
        const bool none = i >= n;
        // (behind the last from where the first is: the scalar offset stays inside
        // the buffers)
        const int u = none ? u0 : u0 + i + rot - (i + rot >= n ? n : 0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool out = none || (u == a.kb - 1 && beyond[h]);
            d.b[h] = buffer_load16(b_rsrc, out || n0 + x16 >= a.N ? b_bytes : uint32_t(x16) * uint32_t(a.ldb) + 16 * (g + 4 * h),
                                   uint32_t(u) * 128);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int row = 16 * t + x16;
                d.x[t][h] = buffer_load16(a_rsrc, out || row >= a.M ? a_bytes : uint32_t(row) * uint32_t(a.lda) + 16 * (g + 4 * h),
                                          uint32_t(u) * 128);
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int row = 16 * t + x16;
            d.sa[t] = __builtin_bit_cast(float, buffer_load4(sa_rsrc, none || row >= a.M ? sa_bytes : 4u * uint32_t(row),
                                                             uint32_t(u) * uint32_t(a.M) * 4));
        }
        if constexpr (ROWB) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int n = n0 + 4 * g + e;
                d.sb[e] = __builtin_bit_cast(float, buffer_load4(sb_rsrc, none || n >= a.N ? sb_bytes : 4u * uint32_t(n),
                                                                 uint32_t(u) * uint32_t(a.N) * 4));
            }
        } else {
            d.sb[0] = __builtin_bit_cast(float, buffer_load4(sb_rsrc, none ? sb_bytes : 4u * uint32_t(n0 / 128) * uint32_t(a.kb),
                                                             uint32_t(u) * 4));
        }
    };

    f32x4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
        acc[t] = f32x4{};
    auto compute = [&](const Block &d) {
        auto whole = [](const u32x4 *v) {
            return __builtin_bit_cast(i32x8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
        };
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            f32x4 p = f32x4{};
            if constexpr (EXACT) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    p = mfma_16x16x32<true>(e4m3_to_bf16(d.b[q / 2][2 * (q % 2)], d.b[q / 2][2 * (q % 2) + 1]),
                                            e4m3_to_bf16(d.x[t][q / 2][2 * (q % 2)], d.x[t][q / 2][2 * (q % 2) + 1]), p);
            } else {
                p = mfma_e4m3(whole(d.b), whole(d.x[t]));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[t][e] = fmaf(p[e], d.sa[t] * d.sb[ROWB ? e : 0], acc[t][e]);
        }
    };

    Block d[kDepth];
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
        load(d[i], i);
        __builtin_amdgcn_sched_barrier(0);   // (the loads stay in the order of their use)
    }
    for (int u = 0; u < n; u += kDepth) {
#pragma unroll
        for (int i = 0; i < kDepth; ++i) {
            compute(d[i]);
            load(d[i], u + i + kDepth);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
        sums[wave][t][lane] = acc[t];
    __syncthreads();
    // four columns a thread, a row's 16 columns side by side
    if (threadIdx.x < NT * 64) {
        const int m = threadIdx.x / 4, n4 = threadIdx.x % 4, col = n0 + 4 * n4;
        f32x4 v = f32x4{};
#pragma unroll
        for (int w = 0; w < W; ++w)
            v += sums[w][m / 16][n4 * 16 + m % 16];
        if (m < a.M && col < a.N)
            fp8_store(a, m, col, v, vec);
    }
}

template <int NT>
hipError_t launch(const Fp8Args &a, hipStream_t stream)
{
    const dim3 grid((a.N + 15) / 16), block(64 * kSkinnyWaves);
    const bool vec = fp8_whole_stores(a);
    if (a.tile) {
        if (a.out == kOutF32)
            hipLaunchKernelGGL((gemm_fp8_skinny_kernel<NT, false, true>), grid, block, 0, stream, a, vec);
        else
            hipLaunchKernelGGL((gemm_fp8_skinny_kernel<NT, false, false>), grid, block, 0, stream, a, vec);
    } else {
        if (a.out == kOutF32)
            hipLaunchKernelGGL((gemm_fp8_skinny_kernel<NT, true, true>), grid, block, 0, stream, a, vec);
        else
            hipLaunchKernelGGL((gemm_fp8_skinny_kernel<NT, true, false>), grid, block, 0, stream, a, vec);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_skinny(const Fp8Args &a, hipStream_t stream)
{
    return a.M > 16 ? launch<2>(a, stream) : launch<1>(a, stream);
}

}  // namespace mswz
