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
//
// 16384 rows of 16 equal groups by 4096 x 2048, bf16: 241 to 256 us by card,
// 1140 to 1070 TFLOP/s (a library product of those sizes without groups: 189 to
// 218); uneven groups, whose last tiles are partly filled, 267 to 287.  A step takes 1.9 us, in which the
// copies bring 64 KiB into each compute unit and the matrix units are busy for
// 0.9: it is bound by the copies' way through the L2 and by waiting for the
// slowest of them at each barrier.  One workgroup per compute unit that goes
// from tile to tile and starts the next one's copies before it stores the last
// took 4 % longer, since tiles were then dealt out beforehand; K tails checked in
// every copy, instead of in a step of their own, 6 %.
#pragma once
#include "experts.hpp"
#include "gemm256_kernel.hpp"

namespace mswz {
namespace {

constexpr int kRaster = 4;   // row tiles whose column tiles are walked together
constexpr int kCusPerXcd = 32;

template <bool BF16, bool A_MN, bool B_MN, int OUT, bool BETA>
__global__ void __launch_bounds__(64 * W)
grouped_kernel(const uint8_t *__restrict__ A, const uint8_t *__restrict__ B, const int32_t *__restrict__ offsets,
               void *__restrict__ D, int E, int M, int N, int K, int tiles_m, int tiles_n)
{
    static_assert(!A_MN || B_MN, "along K both operands are MN-major");
    constexpr bool kMf16 = !A_MN;   // both MN-major: 32x32x16 MFMAs, as in gemm256_kernel
    // Two stages of A and three of B, all of the LDS.  A group's B is its own,
    // so unlike one large product's it is fetched from memory by the one XCD
    // that works on the group, and memory's latency is longer than a step.
    __shared__ __attribute__((aligned(1024))) uint8_t a0[kATile], a1[kATile], b0[kBTile], b1[kBTile], b2[kBTile];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int e = 0, tm = 0, tn = 0, lo = 0, hi = 0, height = kBM;
    bool second = false;   // the lower half of a tile that two workgroups share
    if constexpr (A_MN) {
        // Every group has the same tiles; the longest groups go first, and each
        // is spread over all XCDs, so that the workgroups that start last are
        // the short ones.
        const int tiles = tiles_m * tiles_n, rank = int(blockIdx.x) / tiles;
        if (rank >= E)
            return;
        e = group_by_length(offsets, E, K, rank, lane);
        tile_of_block(int(blockIdx.x) - rank * tiles, tiles_m, tiles_n, -kRaster, tm, tn);
        group_bounds(offsets, e, K, lo, hi);
    } else {
        // Each XCD (workgroup number % 8) takes one contiguous run of the row
        // tiles x column tiles that exist.  Its last round of 32 workgroups, if
        // at most half full, is cut into tiles of half the rows.
        const int mt = group_tiles(offsets, E, M, kBM, lane), total = mt * tiles_n, per = (total + 7) / 8;
        const int xcd = int(blockIdx.x & 7u), at = int(blockIdx.x >> 3);
        const int left = per % kCusPerXcd, halves = left <= kCusPerXcd / 2 ? left : 0;
        int id = at;
        if (at >= per - halves) {
            id = per - halves + (at - (per - halves)) / 2;
            height = kBM / 2;
            second = (at - (per - halves)) % 2;
        }
        if (id >= per || xcd * per + id >= total)
            return;
        id += xcd * per;
        const int span = kRaster * tiles_n, first = id / span * kRaster, in = id % span;
        const int rows = min(kRaster, mt - first);
        int t;
        group_of_tile(offsets, E, M, kBM, first + in % rows, lane, e, t, lo, hi);
        tm = t;
        tn = in / rows;
    }
    const int Kg = A_MN ? hi - lo : K;          // K values of this tile
    const int Mg = A_MN ? M : hi - lo;          // rows of this tile's matrix
    const int m0 = tm * kBM + (second ? kBM / 2 : 0), n0 = tn * kBN;
    const int rows_a = min(height, Mg - m0), rows_b = min(kBN, N - n0);
    if (rows_a <= 0)
        return;
    constexpr int kWavesN = 4;
    const int wm = (wave / kWavesN) * 128, wn = (wave % kWavesN) * 64;
    // a wave whose part lies outside D copies and waits with the others, and
    // leaves the matrix units to the wave that shares its SIMD
    const bool idle = wm >= rows_a || n0 + wn >= N;

    const uint8_t *Ag = A + (A_MN ? size_t(lo) * M : size_t(lo) * K) * 2;
    const uint8_t *Bg = B + (A_MN ? size_t(lo) * N : size_t(e) * N * K) * 2;
    DmaOperand<W> da, db;
    DmaMnOperand<W> dma, dmb;
    if constexpr (A_MN)
        dma.init(Ag, M, M, m0, Kg, wave, lane, 0);
    else
        da.init(Ag, m0, rows_a, uint32_t(K) * 2, wave, lane, 0);
    if constexpr (B_MN)
        dmb.init(Bg, N, N, n0, Kg, wave, lane, 0);
    else
        db.init(Bg, n0, rows_b, uint32_t(K) * 2, wave, lane, 0);
    auto issue_a = [&](uint8_t *stage, int kt) {
        if constexpr (A_MN)
            dma.issue(stage, kt);
        else
            da.issue(stage, kt);
    };
    auto issue_b = [&](uint8_t *stage, int kt) {
        if constexpr (B_MN)
            dmb.issue(stage, kt);
        else
            db.issue(stage, kt);
    };
    constexpr int kCopies = DmaOperand<W>::kInstr;   // copy instructions of one operand and step
    static_assert(kCopies == DmaMnOperand<W>::kInstr, "either layout");

    constexpr int TM = kMf16 ? 8 : 4, TN = kMf16 ? 4 : 2;
    using Acc = std::conditional_t<kMf16, f32x4, f32x16>;
    uint32_t abase[TM], bbase[TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
        abase[i] = kMf16 ? kfrag_base<false>(0, wm, i, kblk16(lane >> 4), lane) : mn_frag_base(0, wm + 32 * i, lane);
#pragma unroll
    for (int j = 0; j < TN; ++j)
        bbase[j] = !kMf16  ? mn_frag_base(0, wn + 32 * j, lane)
                   : B_MN ? mn_frag_base16(0, wn + 16 * j, lane)
                          : kfrag_base<false>(0, wn, j, kblk16(lane >> 4), lane);
    Acc acc[TN][TM];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i)
            acc[j][i] = Acc{};

    auto compute = [&](const uint8_t *sa, const uint8_t *sb) {
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
                    af[i] = lds_read16(sa, ab[i] ^ uint32_t(ks << 6));
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    if constexpr (B_MN) {
                        const u32x2 x = lds_read_tr16(sb, bb[j] + uint32_t(32 * ks) * kMnRowBytes);
                        const u32x2 y = lds_read_tr16(sb, bb[j] + uint32_t(32 * ks + 4) * kMnRowBytes);
                        bf[j] = u32x4{x[0], x[1], y[0], y[1]};
                    } else {
                        bf[j] = lds_read16(sb, bb[j] ^ uint32_t(ks << 6));
                    }
                }
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int i = 0; i < TM; ++i)
                        acc[j][i] = mfma_16x16x32<BF16>(bf[j], af[i], acc[j][i]);
            }
        } else {
            auto frag = [&](const uint8_t *s, uint32_t base, int ks) {
                const uint32_t b = base ^ uint32_t((ks & 1) << 5);
                const u32x2 x = lds_read_tr16(s, b + uint32_t(16 * ks) * kMnRowBytes);
                const u32x2 y = lds_read_tr16(s, b + uint32_t(16 * ks + 4) * kMnRowBytes);
                return u32x4{x[0], x[1], y[0], y[1]};
            };
            u32x4 af[2][TM], bf[2][TN];
            auto rd = [&](int ks) {
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    af[ks & 1][i] = frag(sa, ab[i], ks);
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    bf[ks & 1][j] = frag(sb, bb[j], ks);
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

    // Step t computes from A's stage t % 2 and B's stage t % 3 while A's copies
    // of step t + 1 and B's of step t + 2 are on their way; the barrier that
    // ends it leaves B's in flight.  Copies beyond the last step repeat it into
    // stages that nobody reads again.
    const int KT = Kg / 64;
    auto stage_a = [&](int u) { return u % 2 == 0 ? a0 : a1; };
    auto stage_b = [&](int u) { return u % 3 == 0 ? b0 : u % 3 == 1 ? b1 : b2; };
    if (KT > 0) {
        issue_a(a0, 0);
        issue_b(b0, 0);
        issue_b(b1, min(1, KT - 1));
        lds_barrier_keep_vm<kCopies>();
        auto step = [&](auto uc, int t) {
            constexpr int u = decltype(uc)::value;
            issue_a(stage_a(u + 1), min(t + 1, KT - 1));
            issue_b(stage_b(u + 2), min(t + 2, KT - 1));
            if (!idle)
                compute(stage_a(u), stage_b(u));
            lds_barrier_keep_vm<kCopies>();
        };
        int t = 0;
        for (; t + 6 <= KT; t += 6)
            static_for<0, 6>([&](auto uc) { step(uc, t + decltype(uc)::value); });
        static_for<0, 5>([&](auto uc) {
            if (t + decltype(uc)::value < KT)
                step(uc, t + decltype(uc)::value);
        });
        lds_barrier_keep_vm<0>();   // no copy may still be writing LDS when the workgroup ends
    }
    if (Kg % 64) {
        // the partial last step: K values beyond the group read as zeros
        if constexpr (A_MN)
            dma.issue_tail(a0, KT, Kg, wave, lane);
        else
            da.issue_tail(a0, KT, uint32_t(Kg % 64) * 2, wave, lane);
        if constexpr (B_MN)
            dmb.issue_tail(b0, KT, Kg, wave, lane);
        else
            db.issue_tail(b0, KT, uint32_t(Kg % 64) * 2, wave, lane);
        lds_barrier_keep_vm<0>();
        compute(a0, b0);
    }

    // D's rows start at the group's (along M) or at the group's matrix (along K).
    // The tile goes to memory through the (now idle) stages, each wave's part
    // through 16 KiB of its own, so that stores cover whole 128-byte lines of
    // D's rows and can pass the caches: the MFMA's layout gives a row 32 or 64
    // bytes per store.
    const size_t d0 = (A_MN ? size_t(e) * M + m0 : size_t(lo) + m0) * N;
    __syncthreads();
    uint8_t *const area = (wave < 2 ? a0 : wave < 4 ? a1 : wave < 6 ? b0 : b1) + (wave & 1) * (kATile / 2);
    // MFMA block (i, j), register group h: row and 4-column piece in the wave's part
    constexpr int kPieces = kMf16 ? 1 : 4, kBlockRows = kMf16 ? 16 : 32;
    const int row0 = lane % kBlockRows, piece0 = kMf16 ? lane >> 4 : lane >> 5;
    auto values = [&](int i, int j, int h) {
        return f32x4{acc[j][i][4 * h], acc[j][i][4 * h + 1], acc[j][i][4 * h + 2], acc[j][i][4 * h + 3]};
    };
    if constexpr (OUT == kOutF32) {
        // 32 rows of 256 bytes at a time, 16-byte chunks XOR-keyed by row
        // (layout.hpp, epi_key)
        static_for<0, 4>([&](auto qc) {
            constexpr int qr = decltype(qc)::value, kI = 32 / kBlockRows;
#pragma unroll
            for (int ii = 0; ii < kI; ++ii)
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int h = 0; h < kPieces; ++h) {
                        const uint32_t row = kBlockRows * ii + row0, c = kMf16 ? 4 * j + piece0 : 8 * j + 2 * h + piece0;
                        *reinterpret_cast<f32x4 *>(area + row * kEpiPitch + ((c ^ epi_key(row)) << 4)) =
                            values(kI * qr + ii, j, h);
                    }
            wave_lds_sync();
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const f32x4 v = *reinterpret_cast<const f32x4 *>(area + epi_read_offset(k, lane));
                const int m = wm + 32 * qr + 4 * k + (lane >> 4), n = n0 + wn + 4 * (lane & 15);
                if (m < rows_a && n < N)
                    store_d4<OUT, BETA, true>(D, d0 + size_t(m) * N + n, v);
            }
            wave_lds_sync();   // the next quarter's writes come after these reads
        });
    } else if constexpr (!BETA) {
        // all 128 rows of 128 bytes, 16-byte chunk c of row m at c ^ (m % 8)
        using T = std::conditional_t<OUT == kOutBf16, __bf16, _Float16>;
        typedef T t4 __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int h = 0; h < kPieces; ++h) {
                    const f32x4 v = values(i, j, h);
                    const t4 t = {T(v[0]), T(v[1]), T(v[2]), T(v[3])};
                    const uint32_t row = kBlockRows * i + row0, p = kMf16 ? 4 * j + piece0 : 8 * j + 2 * h + piece0;
                    *reinterpret_cast<t4 *>(area + row * 128 + (((p >> 1) ^ (row & 7)) << 4) + 8 * (p & 1)) = t;
                }
        wave_lds_sync();
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const uint32_t row = 8 * k + (lane >> 3), c = lane & 7;
            const u32x4 v = lds_read16(area, row * 128 + ((c ^ (row & 7)) << 4));
            const int m = wm + int(row), n = n0 + wn + 8 * int(c);
            if (m < rows_a && n < N)
                __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(static_cast<T *>(D) + d0 + size_t(m) * N + n));
        }
    } else {
        // D's old value is added before the one rounding
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int h = 0; h < kPieces; ++h) {
                    const int m = wm + kBlockRows * i + row0;
                    const int n = n0 + wn + 4 * (kMf16 ? 4 * j + piece0 : 8 * j + 2 * h + piece0);
                    if (m < rows_a && n < N)
                        store_d4<OUT, true>(D, d0 + size_t(m) * N + n, values(i, j, h));
                }
    }
}

template <bool BF16, bool A_MN, bool B_MN, int OUT>
hipError_t launch_grouped_out(const GroupedArgs &a, hipStream_t stream)
{
    const int64_t tiles_m = A_MN ? (a.M + kBM - 1) / kBM : most_tiles(a.E, a.M, kBM);
    const int64_t tiles_n = (a.N + kBN - 1) / kBN;
    const int64_t tiles = tiles_m * tiles_n * (A_MN ? a.E : 1);
    // along M each XCD the same number, and room for its halved last round
    const dim3 grid(unsigned(A_MN ? tiles : ((tiles + 7) / 8 + kCusPerXcd / 2) * 8));
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
