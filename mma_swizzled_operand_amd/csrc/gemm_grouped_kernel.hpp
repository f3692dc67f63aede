// gemm_grouped_kernel.hpp — products over groups of rows, included by the
// units that instantiate it (gemm_grouped_*.hip):
//     D[p] = beta*D[p] + A[p] . B[e]^T          for the rows p of group e (rows grouped along M)
//     D[e] = beta*D[e] + sum_p A[p]^T B[p]      over the rows p of group e (grouped along K)
// fp16 / bf16 operands, fp32 sums.
//
// The 256 x 256 tile, its LDS stages, its direct global-to-LDS copies and its
// fragment reads are those of gemm256_kernel.hpp.  What a group adds is where
// a workgroup's tile lies: groups along M are cut into row tiles of their own
// (no tile spans two groups, since their B differs), numbered group by group,
// and a workgroup finds its group by a wave-wide count over the bounds; along
// K a group is the K range of its own output matrix.  The buffer ranges end
// with the group, so rows of the next one read as zeros.
#pragma once
#include "experts.hpp"
#include "gemm256_kernel.hpp"

namespace mswz {
namespace {

constexpr int kRaster = 4;   // row tiles whose column tiles are walked together

template <bool BF16, bool A_MN, bool B_MN, int OUT, bool BETA>
__global__ void __launch_bounds__(64 * W)
grouped_kernel(const uint8_t *__restrict__ A, const uint8_t *__restrict__ B, const int32_t *__restrict__ offsets,
               void *__restrict__ D, int E, int M, int N, int K, int tiles_m, int tiles_n)
{
    static_assert(!A_MN || B_MN, "along K both operands are MN-major");
    constexpr bool kMf16 = !A_MN;   // both MN-major: 32x32x16 MFMAs, as in gemm256_kernel
    __shared__ __attribute__((aligned(1024))) uint8_t lds0[kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t lds1[kStage];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // workgroup -> tile: each XCD (workgroup number % 8) takes one contiguous
    // run of the tiles that exist
    int e = 0, tm = 0, tn = 0, lo = 0, hi = 0;
    const int mt = A_MN ? E * tiles_m : group_tiles(offsets, E, M, kBM, lane);
    const int total = mt * tiles_n, per = (total + 7) / 8;
    const int id = int(blockIdx.x & 7u) * per + int(blockIdx.x >> 3);
    if (int(blockIdx.x >> 3) >= per || id >= total)
        return;
    {
        const int span = kRaster * tiles_n, first = id / span * kRaster, in = id % span;
        const int rows = min(kRaster, mt - first);
        tm = first + in % rows;
        tn = in / rows;
    }
    if constexpr (A_MN) {
        e = tm / tiles_m;
        tm -= e * tiles_m;
        group_bounds(offsets, e, K, lo, hi);
    } else {
        int t;
        group_of_tile(offsets, E, M, kBM, tm, lane, e, t, lo, hi);
        tm = t;
    }
    const int Kg = A_MN ? hi - lo : K;          // K values of this tile
    const int Mg = A_MN ? M : hi - lo;          // rows of this tile's matrix
    const int m0 = tm * kBM, n0 = tn * kBN;
    const int rows_a = min(kBM, Mg - m0), rows_b = min(kBN, N - n0);
    constexpr int kWavesN = 4;
    const int wm = (wave / kWavesN) * 128, wn = (wave % kWavesN) * 64;

    const uint8_t *Ag = A + (A_MN ? size_t(lo) * M : size_t(lo) * K) * 2;
    const uint8_t *Bg = B + (A_MN ? size_t(lo) * N : size_t(e) * N * K) * 2;
    DmaOperand<W> da, db;
    DmaMnOperand<W> dma, dmb;
    if constexpr (A_MN)
        dma.init(Ag, M, M, m0, Kg, wave, lane, 0);
    else
        da.init(Ag, m0, rows_a, uint32_t(K) * 2, wave, lane, 0);
    if constexpr (B_MN)
        dmb.init(Bg, N, N, n0, Kg, wave, lane, kATile);
    else
        db.init(Bg, n0, rows_b, uint32_t(K) * 2, wave, lane, kATile);
    auto issue = [&](uint8_t *stage, int kt) {
        if constexpr (A_MN)
            dma.issue(stage, kt);
        else
            da.issue(stage, kt);
        if constexpr (B_MN)
            dmb.issue(stage, kt);
        else
            db.issue(stage, kt);
    };

    constexpr int TM = kMf16 ? 8 : 4, TN = kMf16 ? 4 : 2;
    using Acc = std::conditional_t<kMf16, f32x4, f32x16>;
    uint32_t abase[TM], bbase[TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
        abase[i] = kMf16 ? kfrag_base<false>(0, wm, i, kblk16(lane >> 4), lane) : mn_frag_base(0, wm + 32 * i, lane);
#pragma unroll
    for (int j = 0; j < TN; ++j)
        bbase[j] = !kMf16  ? mn_frag_base(kATile, wn + 32 * j, lane)
                   : B_MN ? mn_frag_base16(kATile, wn + 16 * j, lane)
                          : kfrag_base<false>(kATile, wn, j, kblk16(lane >> 4), lane);
    Acc acc[TN][TM];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i)
            acc[j][i] = Acc{};

    auto compute = [&](const uint8_t *s) {
        uint32_t ab[TM], bb[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i)
            ab[i] = opaque(abase[i]);
#pragma unroll
        for (int j = 0; j < TN; ++j)
            bb[j] = opaque(bbase[j]);
        if constexpr (kMf16) {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                u32x4 af[TM], bf[TN];
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    af[i] = lds_read16(s, ab[i] ^ uint32_t(ks << 6));
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    if constexpr (B_MN) {
                        const u32x2 x = lds_read_tr16(s, bb[j] + uint32_t(32 * ks) * kMnRowBytes);
                        const u32x2 y = lds_read_tr16(s, bb[j] + uint32_t(32 * ks + 4) * kMnRowBytes);
                        bf[j] = u32x4{x[0], x[1], y[0], y[1]};
                    } else {
                        bf[j] = lds_read16(s, bb[j] ^ uint32_t(ks << 6));
                    }
                }
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int i = 0; i < TM; ++i)
                        acc[j][i] = mfma_16x16x32<BF16>(bf[j], af[i], acc[j][i]);
            }
        } else {
            auto frag = [&](uint32_t base, int ks) {
                const uint32_t b = base ^ uint32_t((ks & 1) << 5);
                const u32x2 x = lds_read_tr16(s, b + uint32_t(16 * ks) * kMnRowBytes);
                const u32x2 y = lds_read_tr16(s, b + uint32_t(16 * ks + 4) * kMnRowBytes);
                return u32x4{x[0], x[1], y[0], y[1]};
            };
            u32x4 af[2][TM], bf[2][TN];
            auto rd = [&](int ks) {
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    af[ks & 1][i] = frag(ab[i], ks);
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    bf[ks & 1][j] = frag(bb[j], ks);
            };
            rd(0);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                if (ks + 1 < 4)
                    rd(ks + 1);
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int i = 0; i < TM; ++i)
                        acc[j][i] = mfma_32x32x16<BF16>(bf[ks & 1][j], af[ks & 1][i], acc[j][i]);
            }
        }
    };

    // two K steps per iteration, one stage each (gemm256_kernel's main loop)
    const int KT = Kg / 64;
    if (KT > 0) {
        issue(lds0, 0);
        __syncthreads();
        int kt = 0;
        for (; kt + 1 < KT; kt += 2) {
            issue(lds1, kt + 1);
            compute(lds0);
            lds_barrier_keep_vm<0>();
            issue(lds0, min(kt + 2, KT - 1));
            compute(lds1);
            lds_barrier_keep_vm<0>();
        }
        if (kt < KT)
            compute(lds0);
        __syncthreads();   // no copy may still be writing LDS when the workgroup ends
    }
    if (Kg % 64) {
        // the partial last step: K values beyond the group read as zeros
        lds_barrier_keep_vm<0>();
        if constexpr (A_MN)
            dma.issue_tail(lds0, KT, Kg, wave, lane);
        else
            da.issue_tail(lds0, KT, uint32_t(Kg % 64) * 2, wave, lane);
        if constexpr (B_MN)
            dmb.issue_tail(lds0, KT, Kg, wave, lane);
        else
            db.issue_tail(lds0, KT, uint32_t(Kg % 64) * 2, wave, lane);
        lds_barrier_keep_vm<0>();
        compute(lds0);
    }

    // D's rows start at the group's (along M) or at the group's matrix (along K)
    const size_t d0 = (A_MN ? size_t(e) * M + m0 : size_t(lo) + m0) * N;
    if constexpr (kMf16) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const int m = wm + 16 * i + (lane & 15), n = n0 + wn + 16 * j + 4 * (lane >> 4);
                if (m < rows_a && n < N)
                    store_d4<OUT, BETA, OUT == kOutF32>(D, d0 + size_t(m) * N + n, acc[j][i]);
            }
    } else {
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int m = wm + 32 * i + (lane & 31), n = n0 + wn + 32 * j + 8 * h + 4 * (lane >> 5);
                    if (m < rows_a && n < N)
                        store_d4<OUT, BETA>(D, d0 + size_t(m) * N + n,
                                            f32x4{acc[j][i][4 * h], acc[j][i][4 * h + 1], acc[j][i][4 * h + 2],
                                                  acc[j][i][4 * h + 3]});
                }
    }
}

template <bool BF16, bool A_MN, bool B_MN, int OUT>
hipError_t launch_grouped_out(const GroupedArgs &a, hipStream_t stream)
{
    const int64_t tiles_m = A_MN ? (a.M + kBM - 1) / kBM : most_tiles(a.E, a.M, kBM);
    const int64_t tiles_n = (a.N + kBN - 1) / kBN;
    const int64_t tiles = tiles_m * tiles_n * (A_MN ? a.E : 1);
    const dim3 grid(unsigned((tiles + 7) / 8 * 8));   // each XCD the same number
    const uint8_t *A = static_cast<const uint8_t *>(a.A), *B = static_cast<const uint8_t *>(a.B);
    if (a.beta)
        hipLaunchKernelGGL((grouped_kernel<BF16, A_MN, B_MN, OUT, true>), grid, dim3(64 * W), 0, stream, A, B, a.offsets,
                           a.D, a.E, a.M, a.N, a.K, int(tiles_m), int(tiles_n));
    else
        hipLaunchKernelGGL((grouped_kernel<BF16, A_MN, B_MN, OUT, false>), grid, dim3(64 * W), 0, stream, A, B, a.offsets,
                           a.D, a.E, a.M, a.N, a.K, int(tiles_m), int(tiles_n));
    return hipGetLastError();
}

template <bool BF16, bool A_MN, bool B_MN>
hipError_t launch_grouped_kind(const GroupedArgs &a, hipStream_t stream)
{
    return a.out == kOutF32 ? launch_grouped_out<BF16, A_MN, B_MN, kOutF32>(a, stream)
                            : launch_grouped_out<BF16, A_MN, B_MN, BF16 ? kOutBf16 : kOutF16>(a, stream);
}

}  // namespace
}  // namespace mswz
