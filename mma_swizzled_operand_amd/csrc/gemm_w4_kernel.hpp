// gemm_w4_kernel.hpp — products of a few rows of 16-bit activations with 4-bit
// weights, included by the units that instantiate it (gemm_w4_*.hip):
//     D[m][n] = beta*D + sum_g s[n][g] sum_{k in g} A[m][k] (w[n][k] - z[n][g])
//
// The weights are streamed once from memory straight into registers, turned
// into 16-bit MFMA operands there (exactly: 4-bit values have few significant
// bits) and multiplied against the activations with 16x16x32 MFMAs, for one
// row as for sixteen: the MFMA takes 16 cycles per 512 weights, less than the
// conversions, which a dot product on the vector unit would come on top of.
// A scale multiplies fp32 sums of at most 128 values of its group, so no weight
// is rounded.
//
// One workgroup of eight waves owns up to ROWS rows and 16*NB*NG columns of D.
// Its waves split the columns NG ways and K KQ ways (NG * KQ = 8): a step is
// 128*KQ values of K, of which each wave takes 128 (64 bytes of each of its
// weight rows).  A large KQ asks for long pieces of each weight row, many
// columns let a copy of A, which every workgroup reads from L2, serve more
// weights; the grid decides (launch_w4_cols, launch_w4_span).
// Weights are loaded into registers, A and the scales into an LDS stage by
// direct copies, kAhead steps early; a step's barrier waits for its own copies
// and leaves the later steps' loads in flight.  (Scales and zero points loaded
// by the lanes that use them, two or three bytes each from sixteen rows, took
// longer than the weights: one row by 16384 x 8192 in 33 us, 18 us without.)
//
// Now, inputs changed from call to call: one row by 16384 x 8192, U4 in groups
// of 128, 13.7 us (70 MB at 5.1 TB/s, memory bound); 64 rows, FP4, 24.7 to 29.4
// us by card (74 MB, and 256 MB of A from L2, which is the longer part), U4
// 31.4; 32 experts of 4096 x 2048 and two rows each, U4 in groups of 64, 33.0 us
// (125 MB at 3.8 TB/s, the scales' short pieces and many short workgroups); 512
// rows by 16384 x 8192, U4 214, FP4 157 (the weights converted once per 64
// rows, matrix units 38 and 35 % busy).
//
// Lane l = (r, q) = (l % 16, l / 16) loads 16 bytes of weight row r, K block q
// (32 values) of the wave's 128.  MFMA j multiplies dword j of every lane.  The
// K order inside the 128 is free as long as A follows it, but a scale group
// must not be shared by one MFMA with another one: for shorter groups the
// lanes' dwords are exchanged first (two or four lane swaps per 16 bytes) so
// that each MFMA's 32 K values lie in one group.  FP4 weights with bf16
// activations skip that: the conversion itself multiplies by the block's
// power of two, exactly.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.hpp"
#include "experts.hpp"
#include "kernels.hpp"

namespace mswz {
namespace {

constexpr int kW4Threads = 512;
constexpr int kChunk = 128;               // K values of one 16-byte load of all four lane groups

// Compile-time loop: fn(std::integral_constant<int, F>), ..., up to L - 1.
template <int F, int L, class Fn>
__device__ __forceinline__ void static_for(Fn &&fn)
{
    if constexpr (F < L) {
        fn(std::integral_constant<int, F>{});
        static_for<F + 1, L>(fn);
    }
}

// Eight 4-bit integers of a dword as 16-bit floats, in element order.  A byte
// 0..15 read as E4M3 is that many times 2^-9 (subnormal up to 7, the first
// normal binade from 8), so the conversion with the factor 2^9 gives the
// integer; both 16-bit formats hold it exactly, and fp16 its difference to the
// zero point z (twice in zz) as well.
template <bool BF16>
__device__ __forceinline__ u32x4 u4_values(uint32_t w, uint32_t zz)
{
    const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
    const uint32_t lo = __builtin_amdgcn_perm(odd, even, 0x05010400u), hi = __builtin_amdgcn_perm(odd, even, 0x07030602u);
    if constexpr (BF16) {
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true))};
    } else {
        typedef _Float16 h2 __attribute__((ext_vector_type(2)));
        const h2 z = __builtin_bit_cast(h2, zz);
        auto sub = [&](auto v) { return __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2, v) - z); };
        return u32x4{sub(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.0f, false)),
                     sub(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.0f, true)),
                     sub(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.0f, false)),
                     sub(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.0f, true))};
    }
}

// Eight E2M1 values times a power of two, in element order.
template <bool BF16>
__device__ __forceinline__ u32x4 e2m1_values(uint32_t w, float scale)
{
    if constexpr (BF16)
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3))};
    else
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 0)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 1)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 2)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 3))};
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
// w4_arrange dword j of lane group q holds eight-value piece w4_piece of the
// chunk, so that MFMA j's values lie in one span.
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
__device__ __forceinline__ int w4_piece(int j, int q)
{
    if constexpr (SPAN == 128)
        return 4 * q + j;
    else if constexpr (SPAN == 64)
        return 4 * ((q & 1) + 2 * (j >> 1)) + (j & 1) + 2 * (q >> 1);
    else
        return 4 * j + q;
}

// A's stage holds a row's pieces next to each other (a copy instruction then
// reads 512 bytes or more of one row: rows of a power-of-two pitch lie in the
// same L2 channel, and 64 bytes of each of 16 rows took twice as long), piece c
// of row m at place c ^ row_key(m).  A 16-byte LDS read serves the lanes
// together that agree in lane bits 1 and 5: eight rows that share bit 1, and
// two lane groups' pieces, whose numbers differ in bit 2 (bit 0 for 32-value
// spans).  The key takes the other three bits from the eight rows, so that the
// sixteen reads fall into different banks.
// (Four rows: two lane groups and four rows, plain keys.)
template <int SPAN, int ROWS>
__host__ __device__ constexpr int row_key(int m)
{
    if (ROWS == 4)
        return SPAN == 32 ? m << 1 : m;
    return SPAN == 32 ? (m & 1) << 1 | (m & 2) >> 1 | (m & 12) : (m & 1) | (m & 4) >> 1 | (m & 2) << 1 | (m & 8);
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
    float *ws;            // SPLIT: fp32 partials [part][M][N]
    int M, N, K, E;
    uint64_t group_magic; // floor(c * group_magic / 2^32) = c / (chunks that share a scale)
    int groups;
    int lda, ldd;
    int beta;
    int part_steps;       // steps of one part of K
};

template <bool BF16, bool E2M1, int SPAN, int ROWS, int NB, int NG, int STAGES, int OUT, bool SPLIT>
__global__ void __launch_bounds__(kW4Threads)
w4_kernel(W4Kernel p)
{
    constexpr int KQ = 8 / NG, MB = ROWS < 16 ? 1 : ROWS / 16;
    constexpr bool kPre = E2M1 && BF16;             // scales folded into the conversion
    constexpr bool kSums = BF16 && !E2M1;           // zero points applied to sums of A
    static_assert(!kPre || SPAN == 128, "folded scales need no lane swaps");
    constexpr int kSpans = 128 / SPAN, kPer = 4 / kSpans;   // scale groups of a chunk, MFMAs of one
    constexpr int kCols = 16 * NB * NG;
    // A's part of a stage, in whole copies by all waves (what lies behind the
    // rows is written as zeros and not read); two of them take the waves' sums
    constexpr int kCopies = (ROWS * KQ * 16 + kW4Threads - 1) / kW4Threads;
    constexpr int kABytes = kCopies * kW4Threads * 16 > 4 * NB * MB * 1024 ? kCopies * kW4Threads * 16 : 4 * NB * MB * 1024;
    // A step's scales of one column lie next to each other in memory, at any
    // byte; they are copied as the aligned words that hold them.  Scales are
    // copied by waves 0-3 and zero points by 4-7 (FP4: scales by all).
    constexpr int kSize = E2M1 ? 1 : 2;                       // bytes of a scale
    constexpr int kPerCol = KQ * (kPre ? 4 : kSpans);         // scales of a column and step
    constexpr int kSWords = (kPerCol * kSize + 4 - kSize + 3) / 4, kZWords = E2M1 ? 0 : (kPerCol + 3 + 3) / 4;
    constexpr int kSThreads = E2M1 ? kW4Threads : kW4Threads / 2;
    constexpr int kSCopies = (kCols * kSWords + kSThreads - 1) / kSThreads;
    constexpr int kSBytes = kSCopies * kSThreads * 4;         // (whole copies: what lies behind is not read)
    constexpr int kStageBytes = kABytes + (E2M1 ? 1 : 2) * kSBytes;
    // LDS stages and register slots; steps in flight.  (Three stages leave room
    // for a second or third workgroup: one row by 16384 x 8192 with two, three,
    // four: 18.4, 14.1, 14.6 us)
    constexpr int kStages = STAGES, kAhead = STAGES - 1;
    static_assert(STAGES == 2 || STAGES == 3, "named stages");
    // one named array per stage: the compiler then knows which stage a copy
    // writes, and waits for no other one
    __shared__ __attribute__((aligned(1024))) uint8_t st0[kStageBytes], st1[kStageBytes], st2[STAGES == 3 ? kStageBytes : 4];
    auto stage = [&](int u) { return u == 0 ? st0 : u == 1 ? st1 : st2; };

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, q = lane >> 4, ng = wave % NG, kq = wave / NG;
    const int n0 = blockIdx.x * kCols;
    int e = 0, tile = blockIdx.y, lo = 0, hi = p.M;
    if (p.offsets && !group_of_tile(p.offsets, p.E, p.M, ROWS, blockIdx.y, lane, e, tile, lo, hi))
        return;
    const int m0 = lo + ROWS * tile, rows = min(hi - m0, ROWS);
    const int all_steps = (p.K + kChunk * KQ - 1) / (kChunk * KQ);
    const int first = SPLIT ? int(blockIdx.z) * p.part_steps : 0;
    const int steps = SPLIT ? min(p.part_steps, all_steps - first) : all_steps;

    // ---- per-lane offsets of the loads.  Rows beyond N or the tile, and A's
    // values beyond K, lie outside the buffers' ranges and read as zeros (the
    // latter by selects: with a branch for the last step a register might be the
    // target of either side's load, and every load in flight was waited for).
    // Weights beyond K, the next row's or zeros, meet those zeros.
    const uint32_t row_bytes = uint32_t(p.K) / 2;
    const uint32_t w_bytes = uint32_t(p.N) * row_bytes;
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.B + size_t(e) * w_bytes, w_bytes);
    const uint32_t a_bytes = uint32_t(rows - 1) * uint32_t(p.lda) * 2 + uint32_t(p.K) * 2;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.A + size_t(m0) * p.lda * 2, a_bytes);
    const uint32_t count = uint32_t(p.N) * uint32_t(p.groups);
    // aligned start of this matrix's scales (or zero points), the bytes to their
    // first one, and the range in whole words
    const bool zeros = !E2M1 && wave >= 4;
    const uint64_t s_start = reinterpret_cast<uint64_t>(p.S) + uint64_t(e) * count * kSize;
    const uint64_t z_start = reinterpret_cast<uint64_t>(p.Z) + uint64_t(e) * count;
    const uint32_t s_skip = uint32_t(s_start) & 3, z_skip = uint32_t(z_start) & 3;
    const uint32_t s_bytes = zeros ? (p.Z ? (z_skip + count + 3) & ~3u : 0) : (s_skip + count * kSize + 3) & ~3u;
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(reinterpret_cast<const void *>((zeros ? z_start : s_start) & ~uint64_t(3)), s_bytes);
    uint32_t w_off[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int n = n0 + 16 * (NB * ng + nb) + r;
        w_off[nb] = n < p.N ? uint32_t(n) * row_bytes + uint32_t(64 * kq + 16 * q) : w_bytes;
    }
    // word copies: word u % words of column u / words
    uint32_t s_off[kSCopies], s_word[kSCopies];
#pragma unroll
    for (int i = 0; i < kSCopies; ++i) {
        const uint32_t u = uint32_t(tid % kSThreads + kSThreads * i), words = zeros ? kZWords : kSWords;
        const uint32_t col = u / words, n = n0 + col;
        s_word[i] = 4 * (u - col * words);
        s_off[i] = col < kCols && n < uint32_t(p.N) ? (zeros ? z_skip : s_skip) + n * uint32_t(p.groups) * (zeros ? 1 : kSize) : 0x80000000u;   // (beyond any range, with any scale's offset)
    }
    auto group_of = [&](int c) {   // first scale of chunk c
        return kPre ? 4 * c : SPAN < 128 ? kSpans * c : int((uint64_t(c) * p.group_magic) >> 32);
    };
    uint32_t a_off[kCopies];
    int a_k[kCopies];
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
        // unit u of the stage: [row][piece's place]
        const int u = tid + kW4Threads * i, m = u / (16 * KQ);
        a_k[i] = 8 * (u % (16 * KQ) ^ row_key<SPAN, ROWS>(m));
        a_off[i] = m < rows ? uint32_t(m * p.lda + a_k[i]) * 2 : a_bytes;
    }

    // Step t's place along K.  Workgroups that share an XCD's L2 start at
    // different places, as they all read the same rows of A, whose pieces at one
    // place lie in few channels of the L2 if the pitch is a power of two (64
    // rows by 16384 x 8192, FP4: 26.5 us without, 25.6).
    const int turn = ROWS > 4 ? int(blockIdx.x >> 3) % steps : 0;
    auto chunk_of = [&](int t) __attribute__((always_inline)) {   // first chunk of the step
        const int at = t + turn;
        return (first + (ROWS > 4 && at >= steps ? at - steps : at)) * KQ;
    };
    // Two stages leave a step's weights, which come from memory, little time:
    // they are loaded one step earlier than A and the scales, before those of
    // the step between (28.0 -> 26.5 us; with three stages no gain).
    constexpr int kEarly = STAGES == 2, kSlots = kEarly ? 2 * kStages : kStages;
    u32x4 w[kSlots][NB];
    // the loads of step t (beyond the last they lie outside the buffers' ranges:
    // repeating the last step's cost its traffic once more per stage)
    auto load_w = [&](int slot, int t) __attribute__((always_inline)) {
        const uint32_t kb = uint32_t(chunk_of(t)) * 64;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
            w[slot][nb] = buffer_load16(rw, t < steps ? w_off[nb] + kb : w_bytes, 0);
    };
    auto load_as = [&](uint8_t *st, int t) __attribute__((always_inline)) {
        const int c0 = chunk_of(min(t, steps - 1));
        const bool past = t >= steps;
        const uint32_t kb = uint32_t(c0) * 64;
        const int left = past ? 0 : p.K - c0 * kChunk;     // K values from the step's first on
#pragma unroll
        for (int i = 0; i < kCopies; ++i)
            buffer_load_lds16(ra, st + 16 * (kW4Threads * i + 64 * wave), a_k[i] < left ? a_off[i] + kb * 4 : a_bytes, 0);
        const uint32_t g0 = uint32_t(group_of(c0)) * (zeros ? 1 : kSize);
#pragma unroll
        for (int i = 0; i < kSCopies; ++i)
            buffer_load_lds4(rs, st + kABytes + (zeros ? kSBytes : 0) + 4 * (kSThreads * i + 64 * (wave % (kSThreads / 64))),
                             past ? 0x80000000u : ((s_off[i] + g0) & ~3u) + s_word[i], 0);
    };
    auto load = [&](int u, int t) __attribute__((always_inline)) {   // (u = t modulo the stages and the slots)
        load_as(stage(u % kStages), t);
        if constexpr (kEarly)
            sched_fence();
        load_w((u + kEarly) % kSlots, t + kEarly);
    };
    constexpr int kLoads = kCopies + kSCopies + NB;   // vector-memory operations of one step

    // Lane (r, q) gets rows 4q .. 4q + 3 of the MFMA's result.  A tile of four
    // rows gives the MFMA each of them four times, row q in rows 4q .. 4q + 3,
    // so that a lane has one sum to scale instead of four (32 experts of 4096
    // x 2048, groups of 32: 46.7 -> 43.8 us; one row by 16384 x 8192: 14.0 ->
    // 13.5).
    constexpr int kSame = ROWS == 4 ? 4 : 1, kRegs = ROWS == 4 && !kPre ? 1 : 4;
    using Acc = std::conditional_t<kRegs == 1, float, f32x4>;
    Acc acc[NB][MB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
            acc[nb][mb] = Acc{};
    const u32x4 ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};

    // A's fragments: the lane's piece of row r for MFMA j and row block mb, i.e.
    // one base, XOR a constant of j, plus one of mb (opaque: else every sum of
    // them is kept in a register of its own through the loop)
    const int a_row = ROWS == 4 ? r >> 2 : r;
    const uint32_t a_base = 16u * uint32_t((a_row * KQ + kq) * 16 + (w4_piece<SPAN>(0, q) ^ row_key<SPAN, ROWS>(a_row)));
    auto pieces = [&](const uint8_t *st, int j, u32x4 *av) __attribute__((always_inline)) {
        const uint32_t at = opaque(a_base ^ uint32_t(16 * w4_piece<SPAN>(j, 0)));
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
            av[mb] = lds_read16(st, at + uint32_t(mb * 16 * KQ * 256));
    };
    // This lane's scales and zero points (absent ones are copied as zeros) of
    // column block nb, step t in the stage: spans 0 .. kSpans - 1 of the wave's
    // chunk (folded scales: the lane group's own).  A span that starts at or
    // behind K has no value of A, but its scale, the next row's or, in groups
    // longer than a chunk, the last group's, would still count if it was not
    // finite.
    const uint32_t no_z = p.Z ? 0u : 8u;
    const uint32_t s_col = uint32_t(n0 + 16 * NB * ng + r) * uint32_t(p.groups);   // first scale of block 0's column
    // bytes of block nb's first scale and zero point past a word, and their words' places
    uint32_t s_mod[NB], z_mod[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        s_mod[nb] = s_skip + (s_col + uint32_t(16 * nb * p.groups)) * kSize;
        z_mod[nb] = z_skip + s_col + uint32_t(16 * nb * p.groups);
    }
    const uint32_t s_place = uint32_t(kABytes + 4 * kSWords * (16 * NB * ng + r) + (kPre ? q : 0));
    const uint32_t z_place = uint32_t(kABytes + kSBytes + 4 * kZWords * (16 * NB * ng + r));
    auto scales = [&](const uint8_t *st, int t, int nb, uint32_t *sv, uint32_t *zv) __attribute__((always_inline)) {
        const int c0 = chunk_of(t), g0 = group_of(c0), g1 = group_of(c0 + kq);
        const uint32_t s_at = ((s_mod[nb] + uint32_t(g0) * kSize) & 3) + (s_place + uint32_t(g1 - g0) * kSize);
#pragma unroll
        for (int g = 0; g < kSpans; ++g) {
            const uint8_t *b = st + s_at + 64 * kSWords * nb + kSize * g;
            sv[g] = kSize == 2 ? *reinterpret_cast<const uint16_t *>(b) : *b;
        }
        if constexpr (!E2M1) {
            const uint32_t z_at = ((z_mod[nb] + uint32_t(g0)) & 3) + (z_place + uint32_t(g1 - g0));
#pragma unroll
            for (int g = 0; g < kSpans; ++g)
                zv[g] = *(st + z_at + 64 * kZWords * nb + g);
        }
        // chunk c0 + kq's values from K on have a scale of zero
        const int k0 = (c0 + kq) * kChunk - p.K;
#pragma unroll
        for (int g = 0; g < kSpans; ++g)   // (no branch: it would cost the loop its registers)
            sv[g] &= uint32_t((k0 + (kPre ? 32 * q : SPAN * g)) >> 31);
    };
    // A step's LDS reads all come before the work on them (64 rows: one MFMA's
    // rows ahead), since two waves a SIMD cannot hide one read's latency after
    // the other.
    constexpr int kReads = MB > 1 ? 2 : 4;
    auto compute = [&](const uint8_t *st, int slot, int t) __attribute__((always_inline)) {
        uint32_t sv[NB][kSpans], zv[NB][kSpans];
        u32x4 av[kReads][MB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
            scales(st, t, nb, sv[nb], zv[nb]);
#pragma unroll
        for (int j = 0; j < kReads; ++j)
            pieces(st, j, av[j]);
        if constexpr (kPre) {
            float scale[NB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                // 2^(ex - 127), ex = 255 converting to NaN.  Weights above 2 times
                // the largest two would pass bf16's range: those blocks are
                // multiplied unscaled, one lane group at a time, and their sums
                // scaled afterwards (what they add here, 2^-253 of that, is lost
                // in the rounding).
                const uint32_t ex = sv[nb][0];
                const bool big = ex == 253 || ex == 254;
                scale[nb] = __builtin_bit_cast(float, big ? 0 : ex << 23);
                if (__any(big)) {
                    for (int g = 0; g < 4; ++g) {
                        const uint32_t exg = __shfl(ex, 16 * g + r);
                        const bool bigg = exg == 253 || exg == 254;
                        f32x4 part[MB];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const u32x4 v = e2m1_values<BF16>(w[slot][nb][j], 1.0f);
                            u32x4 x[MB];
                            pieces(st, j, x);
                            // (A's other lane groups are zeroed, not their weights: an infinity
                            // of A times a zero weight would be NaN)
#pragma unroll
                            for (int mb = 0; mb < MB; ++mb)
                                part[mb] = mfma_16x16x32<BF16>(q == g ? x[mb] : u32x4{}, v, j ? part[mb] : f32x4{});
                        }
#pragma unroll
                        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                acc[nb][mb][i] += bigg ? e8m0_value(exg) * part[mb][i] : 0.0f;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    const u32x4 v = e2m1_values<BF16>(w[slot][nb][j], scale[nb]);
#pragma unroll
                    for (int mb = 0; mb < MB; ++mb)
                        acc[nb][mb] = mfma_16x16x32<BF16>(av[j % kReads][mb], v, acc[nb][mb]);
                }
                if (j + kReads < 4)
                    pieces(st, j + kReads, av[j % kReads]);
            }
            return;
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
            w4_arrange<SPAN>(w[slot][nb]);
#pragma unroll
        for (int s = 0; s < kSpans; ++s) {
            f32x4 part[NB][MB], sum[MB];
            uint32_t zz[NB];
            float scale[NB], zero[NB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                if constexpr (E2M1) {
                    scale[nb] = e8m0_value(sv[nb][s]);
                } else {
                    scale[nb] = scale16<BF16>(uint16_t(sv[nb][s]));
                    zero[nb] = float(zv[nb][s] | no_z);
                    zz[nb] = 0;
                    if constexpr (!BF16)
                        zz[nb] = __builtin_bit_cast(uint16_t, _Float16(zero[nb])) * 0x10001u;
                }
            }
#pragma unroll
            for (int jj = 0; jj < kPer; ++jj) {
                const int j = kPer * s + jj;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    u32x4 v;
                    if constexpr (E2M1)
                        v = e2m1_values<BF16>(w[slot][nb][j], 1.0f);
                    else
                        v = u4_values<BF16>(w[slot][nb][j], zz[nb]);
#pragma unroll
                    for (int mb = 0; mb < MB; ++mb)
                        part[nb][mb] = mfma_16x16x32<BF16>(av[j % kReads][mb], v, jj ? part[nb][mb] : f32x4{});
                }
                // the rows' sums over the span, the same in every column
                if constexpr (kSums)
#pragma unroll
                    for (int mb = 0; mb < MB; ++mb)
                        sum[mb] = mfma_16x16x32<BF16>(av[j % kReads][mb], ones, jj ? sum[mb] : f32x4{});
                if (j + kReads < 4)
                    pieces(st, j + kReads, av[j % kReads]);
                // (one MFMA row's conversions at a time: all of them spill)
                if constexpr (MB > 1)
                    __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                    for (int i = 0; i < kRegs; ++i) {
                        const float v = kSums ? __builtin_fmaf(-zero[nb], sum[mb][i], part[nb][mb][i]) : part[nb][mb][i];
                        if constexpr (kRegs == 1)
                            acc[nb][mb] = __builtin_fmaf(scale[nb], v, acc[nb][mb]);
                        else
                            acc[nb][mb][i] = __builtin_fmaf(scale[nb], v, acc[nb][mb][i]);
                    }
        }
    };

    // Step t: wait until its own loads have landed (the kAhead - 1 later steps',
    // and weights that are loaded early, may stay in flight), barrier (every wave's copies are in LDS, and all
    // have read the stage that is filled next), compute, load step t + kAhead.
    if constexpr (kEarly) {
        load_w(0, 0);
        sched_fence();
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
        load(u, u);
        sched_fence();
    }
    // (Whole rounds of slots without a branch, then the rest: with an exit in
    // every step the loop's registers had to be copied on the way round, which
    // waited for all loads in flight.)
    auto step = [&](auto uc, int t) __attribute__((always_inline)) {
        constexpr int u = decltype(uc)::value;
        lds_barrier_keep_vm<(kAhead - 1) * kLoads + kEarly * NB>();
        sched_fence();
        load(u + kAhead, t + kAhead);
        sched_fence();
        compute(stage(u % kStages), u, t);
        // (the sums are finished here: left open, several steps' products were
        // kept in registers until the last one's scales came)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
                acc[nb][mb] = opaque(acc[nb][mb]);
        sched_fence();
    };
    int t = 0;
    for (; t + kSlots <= steps; t += kSlots)
        static_for<0, kSlots>([&](auto uc) __attribute__((always_inline)) { step(uc, t + decltype(uc)::value); });
    static_for<0, kSlots - 1>([&](auto uc) __attribute__((always_inline)) {
        if (t + decltype(uc)::value < steps)
            step(uc, t + decltype(uc)::value);
    });
    lds_barrier_keep_vm<0>();   // no copy may still be writing LDS below, or when the workgroup ends

    // sums over the KQ waves of a column block: tile tl of column block ng is
    // added up, in wave order, by one of them (waves 0-3 leave theirs in stage
    // 0, 4-7 in stage 1); lane holds column r of the 16, rows 4q .. 4q+3 (of
    // four rows, row q)
    using Out = std::conditional_t<kSame == 4, float, f32x4>;
    auto sums = [&](int wv, int tl) {
        return reinterpret_cast<Out *>((wv < 4 ? st0 : st1) + (((wv & 3) * NB * MB + tl) * 64 + lane) * sizeof(Out));
    };
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            if constexpr (kSame == 4 && kRegs == 4)
                *sums(wave, nb * MB + mb) = acc[nb][mb][0];
            else
                *sums(wave, nb * MB + mb) = acc[nb][mb];
        }
    __syncthreads();
    for (int tl = kq; tl < NB * MB; tl += KQ) {
        Out sum = *sums(ng, tl);
#pragma unroll
        for (int x = 1; x < KQ; ++x)
            sum += *sums(NG * x + ng, tl);
        const int n = n0 + 16 * (NB * ng + tl / MB) + r, mb = tl % MB;
        if (n >= p.N)
            continue;
#pragma unroll
        for (int i = 0; i < 4 / kSame; ++i) {
            const int m = 16 * mb + 4 / kSame * q + i;
            if (m >= rows)
                continue;
            float v;
            if constexpr (kSame == 4)
                v = sum;
            else
                v = sum[i];
            if constexpr (SPLIT) {
                p.ws[(size_t(blockIdx.z) * p.M + m0 + m) * p.N + n] = v;
            } else {
                const size_t at = size_t(m0 + m) * p.ldd + n;
                using T = std::conditional_t<OUT == kOutF32, float, std::conditional_t<OUT == kOutBf16, __bf16, _Float16>>;
                T *d = static_cast<T *>(p.D) + at;
                *d = T(p.beta ? v + float(*d) : v);
            }
        }
    }
}

template <bool BF16, bool E2M1, int SPAN, int ROWS, int NB, int NG, int STAGES, bool SPLIT = false>
hipError_t launch_w4_tile(const W4Args &a, hipStream_t stream)
{
    constexpr int KQ = 8 / NG, kCols = 16 * NB * NG;
    const int steps = (a.K + kChunk * KQ - 1) / (kChunk * KQ), part_steps = (steps + a.parts - 1) / a.parts;
    const W4Kernel p{static_cast<const uint8_t *>(a.A), a.B, static_cast<const uint8_t *>(a.S), a.Z, a.offsets, a.D, a.ws,
                     a.M, a.N, a.K, a.E, (uint64_t(1) << 32) / unsigned(a.group < kChunk ? 1 : a.group / kChunk) + 1,
                     a.groups, a.lda, a.ldd, a.beta, part_steps};
    const int64_t tiles = a.offsets ? most_tiles(a.E, a.M, ROWS) : (a.M + ROWS - 1) / ROWS;
    const dim3 grid((a.N + kCols - 1) / kCols, unsigned(tiles), SPLIT ? (steps + part_steps - 1) / part_steps : 1);
    constexpr int kNarrow = BF16 ? kOutBf16 : kOutF16;
    if constexpr (SPLIT) {
        hipLaunchKernelGGL((w4_kernel<BF16, E2M1, SPAN, ROWS, NB, NG, STAGES, kOutF32, true>), grid, dim3(kW4Threads), 0, stream, p);
    } else if (a.out == kOutF32) {
        hipLaunchKernelGGL((w4_kernel<BF16, E2M1, SPAN, ROWS, NB, NG, STAGES, kOutF32, false>), grid, dim3(kW4Threads), 0, stream, p);
    } else {
        hipLaunchKernelGGL((w4_kernel<BF16, E2M1, SPAN, ROWS, NB, NG, STAGES, kNarrow, false>), grid, dim3(kW4Threads), 0, stream, p);
    }
    return hipGetLastError();
}

// Columns of a workgroup.  More columns share a copy of A and a step's
// addresses, and make a wave's part of K and with it its run of steps longer;
// fewer make more workgroups.  Time goes by rounds of 256 workgroups, one a
// compute unit, so a width is taken from where half as many columns would need
// a second round (16 rows), a little later for tiles of four rows, of which two
// workgroups share a compute unit.  U4 in groups of 128, us by the number of
// workgroups:
//   64 columns / 32, K 8192: one row 128: 12.8 / 9.6, 144: 12.9 / 14.6, 192:
//   13.2 / 14.6, 256: 13.6 / 14.9; 16 rows 128: 15.3 / 11.5, 144: 15.4 / 17.8;
//   32 experts of K 4096, two rows each, 160: 10.0 / 8.3, 192: 10.2 / 10.2;
//   32 / 16, K 8192: one row 128: 9.0 / 7.0, 192: 9.2 / 9.2, 256: 9.5 / 11.1;
//   16 rows 128: 10.9 / 8.3, 160: 10.9 / 14.6.
// FP4 falls the same way (64 / 32, one row 128: 11.9 / 9.2, 144: 11.9 / 13.9).
// 128 columns pay while K is short: half as many workgroups start and end (512
// of them / 1024, one row by K 1024 9.5 / 9.9, 2048 14.7 / 14.5, 3584 28.7 /
// 25.0, 8192 77 / 59; 32 experts of 2048 x 2048 16.2 / 17.5, x 4096 38.0 /
// 32.6).
template <bool BF16, bool E2M1, int SPAN, int ROWS>
hipError_t launch_w4_cols(const W4Args &a, hipStream_t stream)
{
    const int64_t tiles = a.E ? (a.E < a.M ? a.E : a.M) : 1;
    auto enough = [&](int cols, int wgs) { return tiles * ((a.N + cols - 1) / cols) >= wgs; };
    constexpr int kWgs = ROWS == 16 ? 129 : 192;
    return a.K <= 2048 && enough(128, 512) ? launch_w4_tile<BF16, E2M1, SPAN, ROWS, 2, 4, 3>(a, stream)
           : enough(64, kWgs)              ? launch_w4_tile<BF16, E2M1, SPAN, ROWS, 2, 2, 3>(a, stream)
           : enough(32, kWgs)              ? launch_w4_tile<BF16, E2M1, SPAN, ROWS, 1, 2, 3>(a, stream)
                                           : launch_w4_tile<BF16, E2M1, SPAN, ROWS, 1, 1, 3>(a, stream);
}

template <bool BF16, bool E2M1, int SPAN>
hipError_t launch_w4_span(const W4Args &a, hipStream_t stream)
{
    const int rows = w4_rows(a);
    // 64 rows by 128 columns where K is split (gemm_w4.hip) and where
    // workgroups of 64 columns would be a second round (64 rows by K 8192, U4,
    // 257 of those / 129 of 128: 58.4 / 52.6 us, 512: 67.6 / 62.9, 640: 95 /
    // 107; FP4 45.9 / 37.6, 61.1 / 49.4, 87.1 / 83.9), by 64 up to one round
    // (600 rows of 32 experts of 512 x 4096, 256 of those / 128: 22.2 / 33.3)
    if (rows == 64)
        return a.parts > 1                                 ? launch_w4_tile<BF16, E2M1, SPAN, 64, 2, 4, 3, true>(a, stream)
               : w4_tiles64(a) * ((a.N + 63) / 64) > 256 ? launch_w4_tile<BF16, E2M1, SPAN, 64, 2, 4, 3>(a, stream)
                                                           : launch_w4_tile<BF16, E2M1, SPAN, 64, 2, 2, 2>(a, stream);
    return rows == 16 ? launch_w4_cols<BF16, E2M1, SPAN, 16>(a, stream) : launch_w4_cols<BF16, E2M1, SPAN, 4>(a, stream);
}

template <bool BF16, bool E2M1>
hipError_t launch_w4_kind(const W4Args &a, hipStream_t stream)
{
    if constexpr (E2M1) {
        return launch_w4_span<BF16, E2M1, BF16 ? 128 : 32>(a, stream);
    } else {
        if (a.group % 128 == 0)
            return launch_w4_span<BF16, E2M1, 128>(a, stream);
        return a.group == 64 ? launch_w4_span<BF16, E2M1, 64>(a, stream) : launch_w4_span<BF16, E2M1, 32>(a, stream);
    }
}

}  // namespace
}  // namespace mswz
