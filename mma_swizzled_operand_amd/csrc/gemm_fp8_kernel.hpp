// gemm_fp8_kernel.hpp — products of E4M3 operands with an fp32 scale per
// block of 128, included by the units that instantiate it (gemm_fp8_*.hip):
//     D[m][n] = beta*D + sum_b sa[b][m] sb(b, n) sum_{k in block b} A[m][k] B[n][k]
//
// A block of 128 values is one step of the K loop: 128 bytes of every operand
// row, staged by direct copies into an LDS tile with the layout of layout.hpp
// (fragments in the order of the 16-bit kinds: 16 consecutive rows, chunks
// kblk16(g) and that + 4, free of bank conflicts).  One 16x16x128 MFMA onto
// zero gives a block's sum for 16 x 16 outputs; four fp32 multiply-adds a lane
// then add it, times its scale, to the accumulators, on the vector unit while
// the matrix unit works on the next.  The scales of a step ride in the same
// stage.
//
// The E4M3 MFMA aligns the products of eight values before it adds them and
// drops what lies 13 bits below the largest (1.5e-5 of a result in all), which
// a 16-bit D does not show.  For an fp32 D (EXACT) the values are turned into
// bf16, which holds them exactly, and multiplied with the bf16 MFMA at half
// the rate.
#pragma once
#include <hip/hip_runtime.h>

#include <type_traits>

#include "device_common.hpp"
#include "fp8.hpp"
#include "kernels.hpp"

namespace mswz {
namespace {

// 16x16x128 MFMA of unscaled E4M3 operands onto zero.
__device__ __forceinline__ f32x4 mfma_e4m3(i32x8 a, i32x8 b)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{}, 0, 0, 0, 0, 0, 0);
}

// Eight E4M3 values as bf16 (exact).
__device__ __forceinline__ u32x4 e4m3_to_bf16(uint32_t lo, uint32_t hi)
{
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true))};
}

// Direct-to-LDS copy of one operand tile, ROWS rows x 128 bytes a step, by W
// waves: instruction q (wave q % W's) fills 1 KiB, tile rows 8q .. 8q+7, lane l
// the chunk that the layout puts at its place (dma_chunk).  Rows beyond the
// operand and chunks beyond K lie at the end of the buffer's range and read
// as zeros.
template <int ROWS, int W>
struct Fp8Copy {
    static constexpr int kInstr = ROWS / 8 / W;
    static_assert(kInstr * 8 * W == ROWS, "whole instructions a wave");
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t voff[kInstr], lds_off, nbytes;

    __device__ void init(const uint8_t *X, int64_t ld, int row0, int rows, int K, int wave, int lane, uint32_t tile_off)
    {
        nbytes = uint32_t(rows - 1) * uint32_t(ld) + uint32_t(K);
        rsrc = make_rsrc(X + int64_t(row0) * ld, nbytes);
#pragma unroll
        for (int i = 0; i < kInstr; ++i) {
            const int r = int(dma_row(wave + W * i, lane));
            voff[i] = r < rows ? uint32_t(r) * uint32_t(ld) + dma_chunk(wave + W * i, lane) * 16 : nbytes;
        }
        lds_off = tile_off + 8 * wave * kTileRowBytes;
    }
    // lim: bytes of a row's 128-byte slice inside K (128 but for a last, partial block)
    __device__ void issue(uint8_t *stage, int step, int lim, int wave, int lane) const
    {
#pragma unroll
        for (int i = 0; i < kInstr; ++i) {
            uint32_t off = voff[i] + uint32_t(step) * 128;
            if (lim < 128 && int(16 * dma_chunk(wave + W * i, lane)) >= lim)
                off = nbytes;
            buffer_load_lds16(rsrc, stage + lds_off + i * 8 * W * kTileRowBytes, off, 0);
        }
    }
};

// BM x BN outputs a workgroup, WM x WN a wave.  ROWB: B's scales belong to
// rows (else to 128 x 128 tiles).  EXACT: by way of bf16.  OUT, BETA: D.
template <int BM, int BN, int WM, int WN, bool ROWB, bool EXACT, int OUT>
__global__ void __launch_bounds__(64 * (BM / WM) * (BN / WN))
gemm_fp8_kernel(Fp8Args a, int tiles_m, int tiles_n, int group_m, int steps_per_part, bool vec)
{
    constexpr int W = (BM / WM) * (BN / WN), TI = WM / 16, TJ = WN / 16;
    constexpr int kAB = (BM + BN) * 128;
    // scale words of a step: wave w copies 64 of them into slot w of the stage
    constexpr int kSlotsA = BM / 64, kSlotsB = ROWB ? BN / 64 : 1;
    static_assert(kSlotsA + kSlotsB <= W, "one instruction a wave");
    __shared__ __attribute__((aligned(1024))) uint8_t lds0[kAB];
    __shared__ __attribute__((aligned(1024))) uint8_t lds1[kAB];
    __shared__ __attribute__((aligned(256))) uint8_t scl0[256 * W];
    __shared__ __attribute__((aligned(256))) uint8_t scl1[256 * W];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int tm, tn;
    tile_of_block(blockIdx.x, tiles_m, tiles_n, group_m, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int wm = (wave / (BN / WN)) * WM, wn = (wave % (BN / WN)) * WN;
    const int step0 = int(blockIdx.y) * steps_per_part, step1 = min(step0 + steps_per_part, a.kb);

    Fp8Copy<BM, W> ca;
    Fp8Copy<BN, W> cb;
    ca.init(a.A, a.lda, m0, min(BM, a.M - m0), a.K, wave, lane, 0);
    cb.init(a.B, a.ldb, n0, min(BN, a.N - n0), a.K, wave, lane, BM * 128);
    // this lane's scale: base offset and what a step adds (words beyond the
    // operand, and waves without a slot, read zeros at the end of the range)
    const bool for_a = wave < kSlotsA;
    const uint32_t s_rows = for_a ? a.M : ROWB ? a.N : (a.N + 127) / 128;
    const uint32_t s_bytes = s_rows * uint32_t(a.kb) * 4;
    const __amdgpu_buffer_rsrc_t s_rsrc = make_rsrc(for_a ? a.SA : a.SB, s_bytes);
    uint32_t s_row = for_a ? m0 + 64 * wave + lane
                     : ROWB ? n0 + 64 * (wave - kSlotsA) + lane : n0 / 128 + lane;
    const bool s_in = wave < kSlotsA + kSlotsB && s_row < s_rows;
    const uint32_t s_base = s_in ? ((for_a || ROWB) ? s_row : s_row * uint32_t(a.kb)) * 4 : s_bytes;
    const uint32_t s_step = s_in ? ((for_a || ROWB) ? s_rows * 4 : 4u) : 0u;

    auto issue = [&](uint8_t *stage, uint8_t *scales, int step) {
        const int lim = a.K - step * 128;
        ca.issue(stage, step, lim, wave, lane);
        cb.issue(stage, step, lim, wave, lane);
        buffer_load_lds4(s_rsrc, scales + 256 * wave, s_base + s_step * uint32_t(step), 0);
    };

    const int x16 = lane & 15, g = lane >> 4;
    uint32_t abase[TI], bbase[TJ];
#pragma unroll
    for (int i = 0; i < TI; ++i)
        abase[i] = tile_offset(uint32_t(wm + 16 * i + x16), uint32_t(kblk16(g)));
#pragma unroll
    for (int j = 0; j < TJ; ++j)
        bbase[j] = BM * 128 + tile_offset(uint32_t(wn + 16 * j + x16), uint32_t(kblk16(g)));

    // register r of a lane: column 16j + 4g + r of B's rows, row 16i + x16 of A's
    f32x4 acc[TJ][TI];
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
        for (int i = 0; i < TI; ++i)
            acc[j][i] = f32x4{};

    auto frag = [&](const uint8_t *s, uint32_t base) {
        const u32x4 lo = lds_read16(s, base), hi = lds_read16(s, base ^ 64);
        return i32x8{int(lo[0]), int(lo[1]), int(lo[2]), int(lo[3]), int(hi[0]), int(hi[1]), int(hi[2]), int(hi[3])};
    };
    auto compute = [&](const uint8_t *s, const uint8_t *scales) {
        const float *const sa = reinterpret_cast<const float *>(scales) + wm + x16;
        const float *const sb = reinterpret_cast<const float *>(scales) + 64 * kSlotsA;
        f32x4 sbv[ROWB ? TJ : 1];
        float sb_tile = 0.0f;
        if constexpr (ROWB) {
#pragma unroll
            for (int j = 0; j < TJ; ++j)
                sbv[j] = *reinterpret_cast<const f32x4 *>(sb + wn + 16 * j + 4 * g);
        } else {
            sb_tile = sb[BN > 128 ? wn / 128 : 0];
        }
        i32x8 bf[TJ];
#pragma unroll
        for (int j = 0; j < TJ; ++j)
            bf[j] = frag(s, bbase[j]);
#pragma unroll
        for (int i = 0; i < TI; ++i) {
            const i32x8 af = frag(s, abase[i]);
            const float scale = ROWB ? sa[16 * i] : sa[16 * i] * sb_tile;
#pragma unroll
            for (int j = 0; j < TJ; ++j) {
                f32x4 p;
                if constexpr (EXACT) {
                    p = f32x4{};
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        p = mfma_16x16x32<true>(e4m3_to_bf16(bf[j][2 * q], bf[j][2 * q + 1]),
                                                e4m3_to_bf16(af[2 * q], af[2 * q + 1]), p);
                } else {
                    p = mfma_e4m3(bf[j], af);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[j][i][r] = fmaf(p[r], ROWB ? scale * sbv[j][r] : scale, acc[j][i][r]);
            }
        }
    };

    if (step0 < step1) {
        issue(lds0, scl0, step0);
        lds_barrier_keep_vm<0>();
        for (int k = step0; k < step1; k += 2) {
            if (k + 1 < step1)
                issue(lds1, scl1, k + 1);
            compute(lds0, scl0);
            lds_barrier_keep_vm<0>();
            if (k + 1 < step1) {
                if (k + 2 < step1)
                    issue(lds0, scl0, k + 2);
                compute(lds1, scl1);
                lds_barrier_keep_vm<0>();
            }
        }
    }

    using T = std::conditional_t<OUT == kOutF32, float, std::conditional_t<OUT == kOutBf16, __bf16, _Float16>>;
    typedef T t4 __attribute__((ext_vector_type(4)));
    const bool split = gridDim.y > 1;
    const int64_t ld = split ? a.N : a.ldd;
    T *const D = static_cast<T *>(a.D);
    float *const part = a.ws + int64_t(blockIdx.y) * a.M * a.N;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
        const int m = m0 + wm + 16 * i + x16;
        if (m >= a.M)
            continue;
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            const int n = n0 + wn + 16 * j + 4 * g;
            const int64_t at = int64_t(m) * ld + n;
            f32x4 v = acc[j][i];
            if (split) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (n + r < a.N)
                        part[at + r] = v[r];
            } else if (vec && n + 4 <= a.N) {
                t4 *const p = reinterpret_cast<t4 *>(D + at);
                if (a.beta) {
                    const t4 old = *p;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        v[r] += float(old[r]);
                }
                *p = t4{T(v[0]), T(v[1]), T(v[2]), T(v[3])};
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (n + r < a.N)
                        D[at + r] = T(a.beta ? v[r] + float(D[at + r]) : v[r]);
            }
        }
    }
}

}  // namespace
}  // namespace mswz
