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
//
// What bounds it (a copy: 4.9 TB/s; a library product of this type with one
// scale a matrix: 2.71 PFLOP/s): 8192 x 8192 x 8192 with tile scales 449 us, 2.45
// PFLOP/s; MFMAs busy 61 %, the rest of a step is copies into LDS, fragment
// reads and the barrier.  Both gradients of 8192 x 4096 x 4096 257 us, 2.14
// PFLOP/s (MFMAs busy 51 % with tile scales; 45 % with row scales, which take a
// second multiplication a value).  64 x 16384 x 8192 31.8 us, 4.3 TB/s: as many
// bytes again come from the L2, A for every workgroup.
#pragma once
#include <hip/hip_runtime.h>

#include <tuple>
#include <type_traits>

#include "device_common.hpp"
#include "fp8.hpp"
#include "gemm256_kernel.hpp"
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

// Four consecutive outputs of row m, columns n .. n+3 (those inside D), rounded
// into D's kind.  vec: whole pieces are aligned (fp8_whole_stores).
template <int OUT>
__device__ __forceinline__ void fp8_store_as(const Fp8Args &a, int m, int n, f32x4 v, bool vec)
{
    using T = std::conditional_t<OUT == kOutF32, float, std::conditional_t<OUT == kOutBf16, __bf16, _Float16>>;
    typedef T t4 __attribute__((ext_vector_type(4)));
    T *const d = static_cast<T *>(a.D) + int64_t(m) * a.ldd + n;
    if (vec && n + 4 <= a.N) {
        t4 *const p = reinterpret_cast<t4 *>(d);
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
                d[r] = T(a.beta ? v[r] + float(d[r]) : v[r]);
    }
}

__device__ __forceinline__ void fp8_store(const Fp8Args &a, int m, int n, f32x4 v, bool vec)
{
    if (a.out == kOutF32)
        fp8_store_as<kOutF32>(a, m, n, v, vec);
    else if (a.out == kOutBf16)
        fp8_store_as<kOutBf16>(a, m, n, v, vec);
    else
        fp8_store_as<kOutF16>(a, m, n, v, vec);
}

// Whether four columns of D from a multiple of four on are one aligned piece.
inline bool fp8_whole_stores(const Fp8Args &a)
{
    return a.ldd % 4 == 0 && (reinterpret_cast<uintptr_t>(a.D) & (a.out == kOutF32 ? 15 : 7)) == 0;
}

// Whether a 16-bit D without an old one is made of whole, aligned pieces of 16
// bytes.
inline bool fp8_whole_lines(const Fp8Args &a)
{
    return a.out != kOutF32 && !a.beta && a.N % 8 == 0 && a.ldd % 8 == 0 && (reinterpret_cast<uintptr_t>(a.D) & 15) == 0;
}

// The LDS tile's layout: rows of 128 bytes, 16-byte chunk c of row r at place
// c ^ fp8_key(r).  As layout.hpp's tile_key for the rows of one fragment, but
// the same for every 16 rows: all fragments of an operand are read from two
// addresses (the chunk and that ^ 4) plus constants.
MSWZ_HD constexpr uint32_t fp8_key(uint32_t row) { return (row ^ ((row >> 3) & 1u)) & 7u; }
// Copy instruction q fills rows 8q .. 8q+7: the chunk that lane l fetches.
MSWZ_HD constexpr uint32_t fp8_dma_chunk(int q, int lane) { return uint32_t(lane & 7) ^ fp8_key(dma_row(q, lane)); }

// Direct-to-LDS copy of one operand tile, ROWS rows x 128 bytes a step, by W
// waves: instruction q (wave q % W's) fills 1 KiB, tile rows 8q .. 8q+7, lane l
// the chunk that the layout puts at its place (fp8_dma_chunk).  Rows beyond the
// operand, and in the last, partial block chunks beyond K, lie at the end of
// the buffer's range and read as zeros.
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
            voff[i] = r < rows ? uint32_t(r) * uint32_t(ld) + fp8_dma_chunk(wave + W * i, lane) * 16 : nbytes;
        }
        lds_off = tile_off + 8 * wave * kTileRowBytes;
    }
    // out: lanes whose chunk does not exist in this step
    __device__ void issue(uint8_t *stage, int step, bool out) const
    {
#pragma unroll
        for (int i = 0; i < kInstr; ++i)
            buffer_load_lds16(rsrc, stage + lds_off + i * 8 * W * kTileRowBytes, out ? nbytes : voff[i], uint32_t(step) * 128);
    }
};

// PAST: past the caches.
template <bool PAST, typename V>
__device__ __forceinline__ void store(V *to, V v)
{
    if constexpr (PAST)
        __builtin_nontemporal_store(v, to);
    else
        *to = v;
}

// BM x BN outputs a workgroup, WM x WN a wave, S stages in LDS, P blocks from one
// barrier to the next.  ROWB: B's scales belong to
// rows (else to 128 x 128 tiles).  EXACT: by way of bf16.  OUT: D's kind.
template <int BM, int BN, int WM, int WN, int S, int P, bool ROWB, bool EXACT, int OUT>
__global__ void __launch_bounds__(64 * (BM / WM) * (BN / WN))
gemm_fp8_kernel(Fp8Args a, int tiles_m, int tiles_n, int group_m, int steps_per_part, int vec)
{
    constexpr int W = (BM / WM) * (BN / WN), TI = WM / 16, TJ = WN / 16;
    constexpr int kAB = (BM + BN) * 128;
    // scale words of a step: wave w copies 64 of them into slot w of the stage
    constexpr int kSlotsA = (BM + 63) / 64, kSlotsB = ROWB ? (BN + 63) / 64 : 1;
    static_assert(kSlotsA + kSlotsB <= W, "one instruction a wave");
    // (arrays of their own: reads of one stage do not wait for copies into another)
    __shared__ __attribute__((aligned(1024))) uint8_t lds0[kAB];
    __shared__ __attribute__((aligned(1024))) uint8_t lds1[kAB];
    __shared__ __attribute__((aligned(1024))) uint8_t lds2[S > 2 ? kAB : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t lds3[S > 3 ? kAB : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t lds4[S > 4 ? kAB : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t lds5[S > 5 ? kAB : 16];
    __shared__ __attribute__((aligned(256))) uint8_t scl0[256 * W];
    __shared__ __attribute__((aligned(256))) uint8_t scl1[256 * W];
    __shared__ __attribute__((aligned(256))) uint8_t scl2[S > 2 ? 256 * W : 16];
    __shared__ __attribute__((aligned(256))) uint8_t scl3[S > 3 ? 256 * W : 16];
    __shared__ __attribute__((aligned(256))) uint8_t scl4[S > 4 ? 256 * W : 16];
    __shared__ __attribute__((aligned(256))) uint8_t scl5[S > 5 ? 256 * W : 16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    auto stage = [&](auto n) { return std::get<decltype(n)::value>(std::make_tuple(lds0, lds1, lds2, lds3, lds4, lds5)); };
    auto scales_of = [&](auto n) { return std::get<decltype(n)::value>(std::make_tuple(scl0, scl1, scl2, scl3, scl4, scl5)); };
    int tm, tn;
    tile_of_block(blockIdx.x, tiles_m, tiles_n, group_m, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int wm = (wave / (BN / WN)) * WM, wn = (wave % (BN / WN)) * WN;

    Fp8Copy<BM, W> ca;
    Fp8Copy<BN, W> cb;
    ca.init(a.A, a.lda, m0, min(BM, a.M - m0), a.K, wave, lane, 0);
    cb.init(a.B, a.ldb, n0, min(BN, a.N - n0), a.K, wave, lane, BM * 128);
    // this lane's scale word at step 0, and the bytes from one step's to the
    // next (words beyond the operand, and waves without a slot, read zeros at
    // the end of the range)
    const bool for_a = wave < kSlotsA;
    const uint32_t s_rows = for_a ? a.M : ROWB ? a.N : (a.N + 127) / 128;
    const uint32_t s_bytes = s_rows * uint32_t(a.kb) * 4;
    const __amdgpu_buffer_rsrc_t s_rsrc = make_rsrc(for_a ? a.SA : a.SB, s_bytes);
    const uint32_t s_row = for_a ? m0 + 64 * wave + lane
                           : ROWB ? n0 + 64 * (wave - kSlotsA) + lane : n0 / 128 + lane;
    const bool s_in = wave < kSlotsA + kSlotsB && s_row < s_rows;
    const uint32_t s_voff = s_in ? ((for_a || ROWB) ? s_row : s_row * uint32_t(a.kb)) * 4 : s_bytes;
    const uint32_t s_step = (for_a || ROWB) ? s_rows * 4 : 4u;

    const int step0 = int(blockIdx.y) * steps_per_part, step1 = min(step0 + steps_per_part, a.kb);
    // the tiles of one round start at different blocks: rows a power of two apart
    // lie in the same channels of the L2 and of the memory (64 x 16384 x 8192 35.2
    // us without, 33.1, 32.1, 32.3 and 32.0 with 1, 2, 4 and 8 neighbours that
    // start together; 48 x 8192 x 8192 21.6, 20.0, 18.8, 18.9, 19.5; with K 4096
    // within 3 %).  Tiles of later rounds find in the L2 what their neighbours read.
    const int rot = gridDim.x <= 256 ? tn / 4 % (step1 - step0) : 0;
    // a partial last block: the lanes whose chunk lies beyond K (the chunk is
    // the same in all of a wave's instructions, which are an even number of
    // eight-row groups apart)
    static_assert(W % 2 == 0, "fp8_dma_chunk does not depend on the instruction");
    const bool beyond = int(16 * fp8_dma_chunk(wave, lane)) >= a.K % 128 && a.K % 128 != 0;
    auto issue = [&](uint8_t *stage, uint8_t *scales, int step) {
        // (a step behind the last asks for nothing, from where the last one is:
        // the scalar offset stays inside the buffers)
        const int turned = min(step, step1 - 1) + rot, from = turned - (turned >= step1 ? step1 - step0 : 0);
        const bool out = step >= step1 || (from == a.kb - 1 && beyond);
        ca.issue(stage, from, out);
        cb.issue(stage, from, out);
        buffer_load_lds4(s_rsrc, scales + 256 * wave, step < step1 ? s_voff : s_bytes, s_step * uint32_t(from));
    };

    const int x16 = lane & 15, g = lane >> 4;
    const uint32_t at = uint32_t(x16) * kTileRowBytes + ((uint32_t(kblk16(g)) ^ fp8_key(x16)) << 4);
    const uint32_t a_at = uint32_t(wm) * kTileRowBytes + at, b_at = uint32_t(BM + wn) * kTileRowBytes + at;
    const uint32_t a_at64 = a_at ^ 64, b_at64 = b_at ^ 64;
    const uint32_t sa_at = 4 * uint32_t(wm + x16), sb_at = 256 * kSlotsA + 4 * uint32_t(ROWB ? wn + 4 * g : wn / 128);

    // register r of a lane: column 16j + 4g + r of B's rows, row 16i + x16 of A's
    f32x4 acc[TJ][TI];
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
        for (int i = 0; i < TI; ++i)
            acc[j][i] = f32x4{};

    // One block.  MFMA m = TJ i + j; a fragment, with its rows' scales, is read
    // kAhead MFMAs before its first use, and an MFMA's result is added kLag MFMAs
    // later, when it has left the matrix unit: the order is pinned, so that few
    // fragments are live beside the accumulators and the vector unit's work
    // lies between MFMAs.
    auto compute = [&](const uint8_t *s, const uint8_t *scales) {
        constexpr int kAhead = 2, kLag = 3, n = TI * TJ;
        using Sched = FragSchedule<TI, TJ, kAhead>;
        auto frag = [&](uint32_t lo_at, uint32_t hi_at) {
            const u32x4 lo = lds_read16(s, lo_at), hi = lds_read16(s, hi_at);
            return __builtin_bit_cast(i32x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        };
        auto word = [&](uint32_t off) { return *reinterpret_cast<const float *>(scales + off); };
        f32x4 sbv[ROWB ? TJ : 1], p[kLag + 1];
        float sav[TI];
        const float sb_tile = ROWB ? 1.0f : word(sb_at);
        i32x8 af[TI], bf[TJ];
        static_for<0, n + kLag>([&](auto mc) {
            constexpr int m = decltype(mc)::value;
            if constexpr (m < n) {
                constexpr int i = m / TJ, j = m % TJ, c0 = m == 0 ? 0 : Sched::issued(m - 1), c1 = Sched::issued(m);
                static_for<c0, c1>([&](auto rc) {
                    constexpr int it = Sched::item(decltype(rc)::value);
                    if constexpr (it > 0) {
                        af[it - 1] = frag(a_at + 2048 * (it - 1), a_at64 + 2048 * (it - 1));
                        sav[it - 1] = word(sa_at + 64 * (it - 1));
                    } else {
                        bf[-it - 1] = frag(b_at + 2048 * (-it - 1), b_at64 + 2048 * (-it - 1));
                        if constexpr (ROWB)
                            sbv[-it - 1] = *reinterpret_cast<const f32x4 *>(scales + sb_at + 64 * (-it - 1));
                    }
                });
                if constexpr (EXACT) {
                    f32x4 v = f32x4{};
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        v = mfma_16x16x32<true>(e4m3_to_bf16(bf[j][2 * q], bf[j][2 * q + 1]),
                                                e4m3_to_bf16(af[i][2 * q], af[i][2 * q + 1]), v);
                    p[m % (kLag + 1)] = v;
                } else {
                    p[m % (kLag + 1)] = mfma_e4m3(bf[j], af[i]);
                }
            }
            if constexpr (m >= kLag) {
                constexpr int l = m - kLag, i = l / TJ, j = l % TJ;
                const f32x4 v = p[l % (kLag + 1)];
                if constexpr (!ROWB && j == 0)
                    sav[i] *= sb_tile;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[j][i][r] = fmaf(v[r], ROWB ? sav[i] * sbv[ROWB ? j : 0][r] : sav[i], acc[j][i][r]);
            }
            if constexpr (P == 1)
                __builtin_amdgcn_sched_barrier(0);
        });
    };
    // P steps end when the next ones' copies are in LDS; those of the steps after
    // them stay in flight.  (Six stages of 64 x 64 in place of four: 64 x 16384 x 8192
    // 33.4 and 32.2 us.  Two steps a barrier where latency counts, of six stages: 333 x
    // 1003 x 2064 fp32 11.2 -> 10.4 us, bf16 8.8 -> 8.3, 100 x 1000 x 4096 9.9 -> 8.9;
    // of four, whose copies have less time: 10.5, 10.1, 12.0.  Where the memory counts,
    // 64 x 16384 x 8192, 32.5 -> 32.9.)
    constexpr int kCopies = decltype(ca)::kInstr + decltype(cb)::kInstr + 1;
    auto step_end = [] {
        __builtin_amdgcn_sched_barrier(0);
        lds_barrier_keep_vm<(S - 2 * P) * kCopies>();
        __builtin_amdgcn_sched_barrier(0);
    };

    static_for<0, S - P>([&](auto n) { issue(stage(n), scales_of(n), step0 + n); });
    step_end();
    // (steps behind the last are of zeros)
    for (int k = step0; k < step1; k += S)
        static_for<0, S / P>([&](auto n) {
            if (P > 1 && n > 0 && k + P * n >= step1)   // (few tiles, short K: none of zeros alone)
                return;
            static_for<0, P>([&](auto i) {
                constexpr int next = (P * n + S - P + i) % S;
                issue(stage(std::integral_constant<int, next>{}), scales_of(std::integral_constant<int, next>{}), k + P * n + S - P + i);
            });
            static_for<0, P>([&](auto i) {
                constexpr int now = P * n + i;
                compute(stage(std::integral_constant<int, now>{}), scales_of(std::integral_constant<int, now>{}));
            });
            step_end();
        });
    lds_barrier_keep_vm<0>();   // no copy may still be writing LDS when the workgroup ends

    // 16-bit D without an old one, 64 columns a wave: the tile goes through LDS
    // (16-byte chunk c of row r at place c ^ (r % 8) of its 128 bytes) and out row by
    // row: as whole lines past the caches where N is whole pieces of 16 bytes and
    // every one is aligned, else in pieces of four values or one (a lane's four columns at once:
    // 5432 x 3691 x 1712 104 us, 79 this way; 8192 x 8191 x 8192 514 and 461).  With an
    // old D a lane's four columns go out at once, as they were read: 4096 x 4096 x
    // 4096 bf16 71 us, 60 without; 8192 x 8192 x 8192 490 and 450
    if constexpr (OUT != kOutF32 && WN == 64) {
        static_assert(BM * BN * 2 <= 2 * kAB && (BM * BN * 2 <= kAB || W % 2 == 0), "in two stages");
        if (!a.beta && gridDim.y == 1) {
            using T = std::conditional_t<OUT == kOutBf16, __bf16, _Float16>;
            typedef T t4 __attribute__((ext_vector_type(4)));
            constexpr int kMine = WM * 128, kFit = kAB / kMine;   // waves whose tiles one stage holds
            uint8_t *const mine = (wave < kFit ? lds0 : lds1) + wave % kFit * kMine;
#pragma unroll
            for (int i = 0; i < TI; ++i)
#pragma unroll
                for (int j = 0; j < TJ; ++j) {
                    const uint32_t r = 16 * i + x16, c = 2 * j + (g >> 1);
                    *reinterpret_cast<t4 *>(mine + r * 128 + ((c ^ (r & 7)) << 4) + 8 * (g & 1)) =
                        t4{T(acc[j][i][0]), T(acc[j][i][1]), T(acc[j][i][2]), T(acc[j][i][3])};
                }
            wave_lds_sync();
            T *const d = static_cast<T *>(a.D);
            // WIDE values a lane, 64 / WIDE lanes a row
            auto rows = [&](auto wide, auto past) {
                constexpr int WIDE = decltype(wide)::value, LANES = 64 / WIDE;
                typedef T piece __attribute__((ext_vector_type(WIDE)));
                const int c = lane % LANES, n = n0 + wn + WIDE * c;
#pragma unroll 4
                for (int k = 0; k < WM * LANES / 64; ++k) {
                    const uint32_t r = 64 / LANES * k + lane / LANES;
                    const int m = m0 + wm + int(r);
                    if (m < a.M && n + WIDE <= a.N)
                        store<decltype(past)::value>(reinterpret_cast<piece *>(d + int64_t(m) * a.ldd + n),
                                                     *reinterpret_cast<const piece *>(mine + r * 128 + (((WIDE * c / 8) ^ (r & 7)) << 4) +
                                                                                      2 * (WIDE * c % 8)));
                }
            };
            if (vec == 2) {
                rows(std::integral_constant<int, 8>{}, std::true_type{});
            } else if (vec == 1) {
                rows(std::integral_constant<int, 4>{}, std::false_type{});
                // the up to three columns behind the last whole piece, a row a lane
                // (5432 x 3691 x 1712 with a pitch of 3692 57.5 us, 3696 columns with one of
                // 3700 57.5; as a branch in the loop above both 58.2)
                const int n = a.N & ~3, c = n - n0 - wn;
                if (n < a.N && c >= 0 && c < 64)
                    for (int r = lane; r < WM && m0 + wm + r < a.M; r += 64)
                        for (int e = 0; n + e < a.N; ++e)
                            d[int64_t(m0 + wm + r) * a.ldd + n + e] =
                                *reinterpret_cast<const T *>(mine + r * 128 + (((c / 8) ^ (r & 7)) << 4) + 2 * (c % 8 + e));
            } else {
                rows(std::integral_constant<int, 1>{}, std::false_type{});
            }
            return;
        }
    }
    // a part of K leaves its sums in the workspace, in rows of whole 16-byte pieces
    const bool split = gridDim.y > 1;
    const int64_t pitch = fp8_part_pitch(a.N);
    float *const part = a.ws + int64_t(blockIdx.y) * a.M * pitch;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
        const int m = m0 + wm + 16 * i + x16;
        if (m >= a.M)
            continue;
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            const int n = n0 + wn + 16 * j + 4 * g;
            if (split) {
                if (n < a.N)
                    *reinterpret_cast<f32x4 *>(part + m * pitch + n) = acc[j][i];
            } else {
                fp8_store_as<OUT>(a, m, n, acc[j][i], vec != 0);
            }
        }
    }
}

}  // namespace
}  // namespace mswz
