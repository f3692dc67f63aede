// moe_layer.hip — a gated layer of experts for a few tokens, in two kernels (three
// for more than 16 choices):
//     h[c]  = act(W1[e][:I] x) * (W1[e][I:] x)        for each choice c = (t, j), e = ids[t][j]
//     y[t]  = sum_j w[t][j] W2[e] h[c]
//
// With a few tokens the time is that of reading the chosen experts' weights
// once.  A workgroup of the first kernel owns 16 columns of h for one expert,
// its eight waves split the inner size between them, and each lane loads its
// weight rows' pieces straight into registers, several units ahead, without a
// barrier until the waves' sums meet.  The rows of an expert are found from
// the ids by the workgroups themselves.  The second kernel owns 16 columns of y
// for all experts, whose sums meet in LDS; with more than 16 choices it owns
// columns for one expert, and a third one adds up a token's choices.  With two
// choices an expert or more, both products take the tokens' values from LDS
// (Staged).
//
// 16 tokens, 4 of 32 experts of 4096 x 2048 bf16, by the experts in use: 16 of them
// 150 us, 20 to 24 204 to 218, 25 to 32 263 to 286 (4.8 to 5.6 TB/s of weights; a
// copy: 4.9): both products have 32 workgroups an expert, so 2, 3 or 4 for a compute
// unit; of 215 the three kernels take 144, 70 and 5.  64 tokens, 8 of 64 of 2048 x
// 1024 E4M3: 91 to 95 us with 59 to 61 in use, kernels 56, 33 and 5, 4.4 TB/s while
// the products run: their starts and ends are a larger share.  One token, 2 of 8 of
// 1024 x 512: 12 us, two launches of three dependent reads each.
//
// 16x16x32 MFMAs, the weights first: lane l holds 8 values of weight row
// l % 16 (of token l % 16 as the second operand), and its four results are
// columns 4 (l/16) .. + 3 of token l % 16.
//
// h passes to the second kernel as two bf16 parts, its upper 8 bits and the
// next 8 (relative error 2^-16), so that the layer's result does not show the
// step between; the second part costs MFMAs, of which there are plenty.  fp16
// weights then enter as two bf16 parts as well (exactly): an h beyond fp16's
// range stays what it is.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.hpp"
#include "experts.hpp"
#include "gemm256_kernel.hpp"
#include "kernels.hpp"

namespace mswz {
namespace {

constexpr int kFewWaves = 8, kWaves = 4, kThreads = 64 * kWaves, kPerWave = kLayerChoices / kWaves;
constexpr int kSumThreads = 64;
constexpr int kCols = 16;         // columns of h or y a workgroup
constexpr int kFewChoices = 16;   // choices whose sums meet in LDS (one tile of tokens)

enum Weights { kW16 = 0, kWE4m3 = 1 };

// Where the second kernel finds the choices (written by the first kernel): the
// experts in use, one after the other, and all choices sorted by expert; one
// read deep.
struct LayerTable {
    struct {
        int32_t expert, start, count, pad;   // expert -1: no more in use
    } slot[1024];
    int32_t few[kFewChoices][kFewChoices];   // up to 16 choices: those of each slot, -1 behind the last
    int32_t order[kLayerChoices];            // more: from the slot's start on
};

__device__ __forceinline__ float activation(float v, int act)
{
    if (act == kActSilu)
        return v / (1.0f + __expf(-v));
    // (1 + tanh(u)) / 2 = 1 / (1 + e^-2u)
    const float u = 0.7978845608028654f * (v + 0.044715f * v * v * v);
    return v / (1.0f + __expf(-2.0f * u));
}

// The two bf16 parts of v: its upper half, and what is left of it (nothing
// of an infinity or a NaN).
__device__ __forceinline__ void split_bf16(float v, uint32_t &hi, uint32_t &lo)
{
    uint32_t bits = __builtin_bit_cast(uint32_t, v) & 0xffff0000u;
    float rest = v - __builtin_bit_cast(float, bits);
    if (!(fabsf(v) < __builtin_inff())) {
        rest = 0.0f;
        if (v != v)
            bits = 0x7fc00000u;
    }
    hi = bits >> 16;
    lo = __builtin_bit_cast(uint16_t, __bf16(rest));
}

// 8 E4M3 values (two words) as 16-bit ones, exactly.
template <bool BF16>
__device__ __forceinline__ u32x4 from_e4m3(uint32_t a, uint32_t b)
{
    if constexpr (BF16)
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true))};
    else
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true))};
}

// Eight fp16 values as bf16 parts whose sum they are.
__device__ __forceinline__ void split_f16x8(u32x4 v, u32x4 &hi, u32x4 &lo)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h[2], l[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
            split_bf16(float(__builtin_bit_cast(_Float16, uint16_t(v[i] >> (16 * e)))), h[e], l[e]);
        hi[i] = h[0] | (h[1] << 16);
        lo[i] = l[0] | (l[1] << 16);
    }
}

// Tiles of 16 weight rows a wave, and units that it keeps in flight: E4M3 rows
// are half as long, so more of them share a token's values.
template <int WK>
constexpr int tiles_of() { return WK == kWE4m3 ? 4 : 2; }
template <int WK>
constexpr int depth_of(int NT) { return WK == kW16 && NT == 1 ? 4 : 2; }

// A wave's share of a product of weight rows (TILES tiles of 16) with rows of
// tokens (NT tiles of 16).  A unit is 64 bytes of every weight row, 32 values of
// 16 bits or 64 of E4M3; lane l holds 16 bytes of it, at 16 (l/16), and the
// values of its token's row that meet them.  kDepth units are in flight.  DOWN:
// the rows are h's two parts, 8 values of the upper part next to the same of the
// lower; else X's.
template <bool BF16, int WK, bool DOWN, int TILES, int NT, int kDepth>
struct Stream {
    static constexpr int NX = (WK == kWE4m3 ? 2 : 1) * (DOWN ? 2 : 1);   // 16-byte pieces of a token's row a unit
    // scales of a block: the gate's tiles (even) and the others of h, or one for
    // all columns of y, which lie in one tile of 128
    static constexpr int NS = DOWN ? 1 : 2;
    static_assert(WK == kW16 || kDepth % 2 == 0, "a scale's block is two units");
    struct Unit {
        u32x4 w[TILES], x[NT][NX];
        float s[NS];
    };
    __amdgpu_buffer_rsrc_t w_rsrc, x_rsrc, s_rsrc;
    uint32_t w_row[TILES], s_row[NS], x_row[NT];   // byte offsets of this lane's rows, the end of the range for none
    uint32_t w_end, x_end, s_end, row_bytes;
    f32x4 acc[NT][TILES];

    __device__ void load(Unit &d, int u, bool none, int g, bool last) const
    {
        const uint32_t at = 64u * uint32_t(u) + 16u * uint32_t(g);
        const bool out = none || at >= row_bytes;
#pragma unroll
        for (int t = 0; t < TILES; ++t)
            d.w[t] = buffer_load16(w_rsrc, out ? w_end : w_row[t] + at, 0);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < NX; ++i)
                d.x[t][i] = buffer_load16(x_rsrc, out || x_row[t] == x_end ? x_end : x_row[t] + NX * at + 16 * i, 0);
        if constexpr (WK == kWE4m3)
            if (last)
#pragma unroll
                for (int t = 0; t < NS; ++t)
                    d.s[t] = __builtin_bit_cast(float, buffer_load4(s_rsrc, none ? s_end : s_row[t] + 4u * uint32_t(u / 2), 0));
    }

    // one MFMA step: 8 values a lane of the weights with those of a token
    static __device__ __forceinline__ f32x4 step(u32x4 w, const u32x4 *x, f32x4 c)
    {
        if constexpr (!DOWN)
            return mfma_16x16x32<BF16>(w, x[0], c);
        else
            return mfma_16x16x32<true>(w, x[1], mfma_16x16x32<true>(w, x[0], c));
    }

    // the same for all tiles of tokens (fp16 weights are split once for them)
    template <int N>
    static __device__ __forceinline__ void steps(u32x4 w, const u32x4 (*x)[NX], f32x4 (*sum)[TILES], int tile)
    {
        if constexpr (DOWN && !BF16) {
            u32x4 hi, lo;
            split_f16x8(w, hi, lo);
#pragma unroll
            for (int t = 0; t < N; ++t) {
                sum[t][tile] = mfma_16x16x32<true>(hi, x[t][1], mfma_16x16x32<true>(hi, x[t][0], sum[t][tile]));
                sum[t][tile] = mfma_16x16x32<true>(lo, x[t][1], mfma_16x16x32<true>(lo, x[t][0], sum[t][tile]));
            }
        } else {
#pragma unroll
            for (int t = 0; t < N; ++t)
                sum[t][tile] = step(w, x[t], sum[t][tile]);
        }
    }

    // units u0 .. u1 - 1 (E4M3: both even), the turn-th and the ones after it
    // first: waves that start at different places do not ask the same channels
    // of the L2 for the tokens' rows at the same time
    __device__ void run(int u0, int u1, int turn, int g)
    {
        constexpr int per = WK == kWE4m3 ? 2 : 1;
        const int n = u1 - u0, rot = n > 0 ? turn % (n / per) * per : 0;
        auto unit = [&](int i) { return u0 + i + rot - (i + rot >= n ? n : 0); };
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < TILES; ++i)
                acc[t][i] = f32x4{};
        Unit d[kDepth];
        static_for<0, kDepth>([&](auto i) {
            load(d[i], unit(i), i >= n, g, i % 2 == 1);
            __builtin_amdgcn_sched_barrier(0);   // (the loads stay in the order of their use)
        });
        f32x4 part[NT][TILES];
        for (int u = 0; u < n; u += kDepth)
            static_for<0, kDepth>([&](auto ic) {
                constexpr int i = decltype(ic)::value;
#pragma unroll
                for (int w = 0; w < TILES; ++w) {
                    if constexpr (WK == kW16) {
                        steps<NT>(d[i].w[w], d[i].x, acc, w);
                    } else {
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const u32x4 v = from_e4m3<BF16 || DOWN>(d[i].w[w][2 * q], d[i].w[w][2 * q + 1]);
#pragma unroll
                            for (int t = 0; t < NT; ++t)
                                part[t][w] = step(v, d[i].x[t] + q * (NX / 2), i % 2 == 0 && q == 0 ? f32x4{} : part[t][w]);
                        }
                        if (i % 2 == 1)
#pragma unroll
                            for (int t = 0; t < NT; ++t)
#pragma unroll
                                for (int r = 0; r < 4; ++r)
                                    acc[t][w][r] = fmaf(d[i].s[w % NS], part[t][w][r], acc[t][w][r]);
                    }
                }
                load(d[i], unit(u + i + kDepth), u + i + kDepth >= n, g, i % 2 == 1);
                __builtin_amdgcn_sched_barrier(0);
            });
    }
};

// Calls fn with up to MOST (2 or 4) tiles of 16 rows at a time, rows r0 .. of n.
template <int MOST, class Fn>
__device__ __forceinline__ void by_rows(int n, Fn &&fn)
{
    for (int r0 = 0; r0 < n; r0 += 16 * MOST)
        if (n - r0 <= 16)
            fn(r0, std::integral_constant<int, 1>{});
        else if (MOST == 2 || n - r0 <= 32)
            fn(r0, std::integral_constant<int, 2>{});
        else
            fn(r0, std::integral_constant<int, MOST>{});
}

// The sums of the `parts` waves that share a product, one tile of tokens: the
// first of them gets them, in their order.
template <int TILES>
__device__ __forceinline__ void add_parts(f32x4 (*sums)[TILES][64], f32x4 *v, int wave, int parts, int lane)
{
    if (parts == 1)
        return;
#pragma unroll
    for (int i = 0; i < TILES; ++i)
        sums[wave][i][lane] = v[i];
    __syncthreads();
    if (wave % parts == 0)
        for (int w = 1; w < parts; ++w)
#pragma unroll
            for (int i = 0; i < TILES; ++i)
                v[i] += sums[wave + w][i][lane];
    __syncthreads();
}

// The part of a wave among `parts`: units of 64 bytes, whole blocks of a scale.
template <int WK>
__device__ __forceinline__ void share(uint32_t row_bytes, int part, int parts, int &u0, int &u1)
{
    constexpr int per = WK == kWE4m3 ? 2 : 1;
    const int units = int((row_bytes + 64 * per - 1) / (64 * per));
    u0 = per * (units * part / parts);
    u1 = per * (units * (part + 1) / parts);
}

// The blockIdx.y-th of the experts in use (-1: there are fewer) and its n
// choices, in ascending order, in LDS; the first workgroup of an expert writes
// them down for the second kernel.
struct ExpertRows {
    uint32_t used[32];
    int before[2][kWaves];
    uint16_t rows[kLayerChoices];
};

__device__ __forceinline__ int find_expert(const LayerArgs &a, ExpertRows &lds, int &n)
{
    uint32_t *const used = lds.used;
    int(*const before)[kWaves] = lds.before;
    uint16_t *const rows = lds.rows;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int choices = a.T * a.topk;
    if (tid < 32)
        used[tid] = 0;
    __syncthreads();
    int id[kPerWave / 64];
#pragma unroll
    for (int i = 0; i < kPerWave / 64; ++i) {
        const int c = wave * kPerWave + 64 * i + lane;
        id[i] = c < choices ? a.ids[c] : -1;
        if (uint32_t(id[i]) < uint32_t(a.E))
            atomicOr(&used[id[i] >> 5], 1u << (id[i] & 31));
    }
    __syncthreads();
    int expert = -1;
    {
        const uint32_t word = lane < 32 ? used[lane] : 0u;
        const int n = __builtin_popcount(word), sum = wave_scan(n, lane);
        const int want = blockIdx.y;
        const uint64_t past = __ballot(sum > want);
        if (past) {
            const int who = __builtin_ctzll(past);
            uint32_t w = __builtin_amdgcn_readlane(int(word), who);
            for (int skip = want - (__builtin_amdgcn_readlane(sum, who) - __builtin_amdgcn_readlane(n, who)); skip > 0; --skip)
                w &= w - 1;
            expert = 32 * who + __builtin_ctz(w);
        }
    }
    LayerTable *const table = static_cast<LayerTable *>(a.table);
    if (expert < 0) {
        if (blockIdx.x == 0 && tid == 0)
            table->slot[blockIdx.y].expert = -1;
        return -1;
    }
    int mine = 0, below = 0;
#pragma unroll
    for (int i = 0; i < kPerWave / 64; ++i) {
        mine += __builtin_popcountll(__ballot(id[i] == expert));
        below += __builtin_popcountll(__ballot(id[i] >= 0 && id[i] < expert));
    }
    if (lane == 0) {
        before[0][wave] = mine;
        before[1][wave] = below;
    }
    __syncthreads();
    int start = 0, at = 0;
    n = 0;
    for (int w = 0; w < kWaves; ++w) {
        at += w < wave ? before[0][w] : 0;
        n += before[0][w];
        start += before[1][w];
    }
#pragma unroll
    for (int i = 0; i < kPerWave / 64; ++i) {
        const uint64_t hit = __ballot(id[i] == expert);
        if (id[i] == expert)
            rows[at + __builtin_popcountll(hit & ((uint64_t(1) << lane) - 1))] = uint16_t(wave * kPerWave + 64 * i + lane);
        at += __builtin_popcountll(hit);
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        if (choices <= kFewChoices) {
            if (tid < kFewChoices)
                table->few[blockIdx.y][tid] = tid < n ? rows[tid] : -1;
        } else {
            for (int r = tid; r < n; r += kThreads)
                table->order[start + r] = rows[r];
        }
        if (tid == 0) {
            table->slot[blockIdx.y].expert = expert;
            table->slot[blockIdx.y].start = start;
            table->slot[blockIdx.y].count = n;
        }
    }
    return expert;
}

// Four columns i .. i + 3 of a choice's h from the two sums.
__device__ __forceinline__ void store_h(const LayerArgs &a, int choice, int i, f32x4 gate, f32x4 up)
{
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        split_bf16(activation(gate[e], a.act) * up[e], hi[e], lo[e]);
    // of every 8 columns the upper parts, then the lower ones
    uint8_t *const to = static_cast<uint8_t *>(a.h) + (int64_t(choice) * a.I + (i & ~7)) * 4 + 2 * (i & 7);
    *reinterpret_cast<u32x2 *>(to) = u32x2{hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16)};
    *reinterpret_cast<u32x2 *>(to + 16) = u32x2{lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16)};
}

// What the first kernels share: TILES / 2 tiles of 16 columns of h from i0 on, the
// gate's rows and the others in turn.
template <bool BF16, int WK, int TILES, int NT, int kDepth>
__device__ __forceinline__ Stream<BF16, WK, false, TILES, NT, kDepth>
up_stream(const LayerArgs &a, int expert, int i0, int x16)
{
    const uint32_t row_bytes = uint32_t(a.H) * (WK == kWE4m3 ? 1 : 2);
    const int ib = (a.I + 127) / 128, hb = (a.H + 127) / 128;
    Stream<BF16, WK, false, TILES, NT, kDepth> s;
    s.row_bytes = row_bytes;
    s.w_end = 2u * uint32_t(a.I) * row_bytes;
    s.w_rsrc = make_rsrc(static_cast<const uint8_t *>(a.W1) + uint64_t(expert) * s.w_end, s.w_end);
    s.x_end = uint32_t(a.T - 1) * uint32_t(a.ldx) * 2 + uint32_t(a.H) * 2;
    s.x_rsrc = make_rsrc(a.X, s.x_end);
#pragma unroll
    for (int c = 0; c < TILES / 2; ++c) {
        s.w_row[2 * c] = uint32_t(min(i0 + 16 * c + x16, a.I - 1)) * row_bytes;
        s.w_row[2 * c + 1] = s.w_row[2 * c] + uint32_t(a.I) * row_bytes;
    }
    if constexpr (WK == kWE4m3) {
        s.s_end = 2u * uint32_t(ib) * uint32_t(hb) * 4;
        s.s_rsrc = make_rsrc(a.S1 + int64_t(expert) * 2 * ib * hb, s.s_end);
        s.s_row[0] = uint32_t(min(i0, a.I - 1) / 128) * uint32_t(hb) * 4;
        s.s_row[1] = s.s_row[0] + uint32_t(ib) * uint32_t(hb) * 4;
    }
    return s;
}

// The first kernel: the choices of one expert, the blockIdx.y-th of those in
// use; 8 * TILES columns of h for every `parts` waves.
template <bool BF16, int WK>
__global__ void __launch_bounds__(kThreads)
moe_layer_up_kernel(LayerArgs a, int parts)
{
    __shared__ ExpertRows found;
    __shared__ __attribute__((aligned(16))) f32x4 sums[kWaves][tiles_of<WK>()][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int n;
    const int expert = find_expert(a, found, n);
    if (expert < 0)
        return;
    const uint16_t *const rows = found.rows;
    constexpr int kSize = WK == kWE4m3 ? 1 : 2;
    constexpr int TILES = tiles_of<WK>();
    const int i0 = (int(blockIdx.x) * (kWaves / parts) + wave / parts) * (8 * TILES), x16 = lane & 15, g = lane >> 4;
    const uint32_t row_bytes = uint32_t(a.H) * kSize, x_pitch = uint32_t(a.ldx) * 2;
    int u0, u1;
    share<WK>(row_bytes, wave % parts, parts, u0, u1);
    if (i0 >= a.I)
        u1 = u0;   // (this wave's columns lie behind the last)
    by_rows<2>(n, [&](int r0, auto tiles) {
        constexpr int NT = decltype(tiles)::value;
        auto s = up_stream<BF16, WK, TILES, NT, depth_of<WK>(NT)>(a, expert, i0, x16);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int r = r0 + 16 * t + x16;
            s.x_row[t] = r < n ? uint32_t(rows[r] / uint32_t(a.topk)) * x_pitch : s.x_end;
        }
        s.run(u0, u1, i0 / (8 * TILES), g);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            f32x4 *const v = s.acc[t];
            add_parts<TILES>(sums, v, wave, parts, lane);
            const int r = r0 + 16 * t + x16;
#pragma unroll
            for (int c = 0; c < TILES / 2; ++c) {
                const int i = i0 + 16 * c + 4 * g;
                if (wave % parts != 0 || r >= n || i >= a.I)
                    continue;
                store_h(a, rows[r], i, v[2 * c], v[2 * c + 1]);
            }
        }
    });
}

// What the second kernels share: TILES tiles of 16 columns of y from h0 on, for
// the rows r0 .. of an expert's n.
template <bool BF16, int WK, int TILES, int NT, int kDepth>
__device__ __forceinline__ Stream<BF16, WK, true, TILES, NT, kDepth>
down_stream(const LayerArgs &a, int expert, int h0, const int *choice, int x16)
{
    const uint32_t row_bytes = uint32_t(a.I) * (WK == kWE4m3 ? 1 : 2);
    const int ib = (a.I + 127) / 128, hb = (a.H + 127) / 128;
    Stream<BF16, WK, true, TILES, NT, kDepth> s;
    s.row_bytes = row_bytes;
    s.w_end = uint32_t(a.H) * row_bytes;
    s.w_rsrc = make_rsrc(static_cast<const uint8_t *>(a.W2) + uint64_t(expert) * s.w_end, s.w_end);
    s.x_end = uint32_t(a.T * a.topk) * uint32_t(a.I) * 4;
    s.x_rsrc = make_rsrc(a.h, s.x_end);
    if constexpr (WK == kWE4m3) {
        s.s_end = uint32_t(hb) * uint32_t(ib) * 4;
        s.s_rsrc = make_rsrc(a.S2 + int64_t(expert) * hb * ib, s.s_end);
        s.s_row[0] = uint32_t(min(h0, a.H - 1) / 128) * uint32_t(ib) * 4;
    }
#pragma unroll
    for (int i = 0; i < TILES; ++i)
        s.w_row[i] = uint32_t(min(h0 + 16 * i + x16, a.H - 1)) * row_bytes;
#pragma unroll
    for (int t = 0; t < NT; ++t)
        s.x_row[t] = choice[t] >= 0 ? uint32_t(choice[t]) * uint32_t(a.I) * 4 : s.x_end;
    return s;
}

// The second kernel for a few choices: 16 columns of y for all tokens.  Its
// waves share out the experts in use and, `splits` ways, the inner size; each
// choice's sums go to LDS and a token's are added up in the order of its
// choices.
template <bool BF16, int WK>
__global__ void __launch_bounds__(64 * kFewWaves)
moe_layer_down_kernel(LayerArgs a, int slots, int splits)
{
    __shared__ __attribute__((aligned(16))) float of_choice[kFewWaves * kFewChoices * kCols];   // [splits][choices][16]
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int choices = a.T * a.topk, h0 = blockIdx.x * kCols, x16 = lane & 15, g = lane >> 4, split = wave % splits;
    const LayerTable *const table = static_cast<const LayerTable *>(a.table);
    // lane c: choice c's expert and weight, for the sums below
    const int id = lane < choices ? a.ids[lane] : -1;
    const float weight = lane < choices ? a.w[lane] : 0.0f;
    int u0, u1;
    share<WK>(uint32_t(a.I) * (WK == kWE4m3 ? 1 : 2), split, splits, u0, u1);
    for (int slot = wave / splits; slot < slots; slot += kFewWaves / splits) {
        const int choice = table->few[slot][x16], expert = table->slot[slot].expert;
        if (expert < 0)
            break;
        auto s = down_stream<BF16, WK, 1, 1, 4>(a, expert, h0, &choice, x16);
        s.run(u0, u1, blockIdx.x, g);
        if (choice >= 0)
            *reinterpret_cast<f32x4 *>(of_choice + (split * choices + choice) * kCols + 4 * g) = s.acc[0][0];
    }
    __syncthreads();
    using T = std::conditional_t<BF16, __bf16, _Float16>;
    const int t = tid / kCols, col = tid % kCols;   // (at most 16 tokens of 16 columns)
    if (wave >= (kFewChoices * kCols) / 64)
        return;
    float y = 0.0f;
    for (int j = 0; j < a.topk; ++j) {
        const int c = min(t, a.T - 1) * a.topk + j;
        const float w = __shfl(weight, c);
        const bool in = uint32_t(__shfl(id, c)) < uint32_t(a.E);
        float v = 0.0f;
        for (int s = 0; s < splits; ++s)
            v += in ? of_choice[(s * choices + c) * kCols + col] : 0.0f;
        y = in ? fmaf(w, v, y) : y;
    }
    if (t < a.T && h0 + col < a.H)
        static_cast<T *>(a.Y)[int64_t(t) * a.ldx + h0 + col] = T(y);
}

// The second kernel for more choices: those of one expert, in fp32 rows of the
// workspace; 16 * TILES columns of y for every `parts` waves.
template <bool BF16, int WK>
__global__ void __launch_bounds__(kThreads)
moe_layer_rows_kernel(LayerArgs a, int parts)
{
    constexpr int TILES = tiles_of<WK>();
    __shared__ __attribute__((aligned(16))) f32x4 sums[kWaves][TILES][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const LayerTable *const table = static_cast<const LayerTable *>(a.table);
    const int expert = table->slot[blockIdx.y].expert, start = table->slot[blockIdx.y].start, n = table->slot[blockIdx.y].count;
    if (expert < 0)
        return;
    const int h0 = (int(blockIdx.x) * (kWaves / parts) + wave / parts) * TILES * kCols, x16 = lane & 15, g = lane >> 4;
    int u0, u1;
    share<WK>(uint32_t(a.I) * (WK == kWE4m3 ? 1 : 2), wave % parts, parts, u0, u1);
    if (h0 >= a.H)
        u1 = u0;   // (this wave's columns lie behind the last)
    by_rows<2>(n, [&](int r0, auto tiles) {
        constexpr int NT = decltype(tiles)::value;
        int choice[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
            choice[t] = r0 + 16 * t + x16 < n ? table->order[start + r0 + 16 * t + x16] : -1;
        auto s = down_stream<BF16, WK, TILES, NT, depth_of<WK>(NT)>(a, expert, h0, choice, x16);
        s.run(u0, u1, h0 / (TILES * kCols), g);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            f32x4 *const v = s.acc[t];
            add_parts<TILES>(sums, v, wave, parts, lane);
            if (wave % parts == 0 && choice[t] >= 0)
#pragma unroll
                for (int i = 0; i < TILES; ++i)
                    if (h0 + 16 * i + 4 * g < a.H)
                        *reinterpret_cast<f32x4 *>(a.rows + int64_t(choice[t]) * a.H + h0 + 16 * i + 4 * g) = v[i];
        }
    });
}

// As Stream, for many rows of tokens: a workgroup's four waves have weight rows
// of their own and take the tokens' values from LDS, which direct copies fill a
// chunk of kUnits units ahead, so that a token's row is read from the L2 once for
// 128 weight rows.  Row r of a chunk has kChunk bytes, its 16-byte piece c at place
// c ^ (r % 16).  The weights' loads are a chunk ahead in registers; a chunk's
// barrier waits for the copies and leaves the loads behind them in flight.
template <bool BF16, int WK, bool DOWN, int NT>
struct Staged {
    using One = Stream<BF16, WK, DOWN, 2, NT, 2>;
    static constexpr int NX = One::NX, NS = One::NS, kUnits = NX == 4 ? 2 : 4, kChunk = 64 * NX * kUnits;
    static constexpr int kInstr = NT * 16 * kChunk / 1024 / kWaves;
    static constexpr int kLoads = 2 * kUnits + (WK == kWE4m3 ? NS * kUnits / 2 : 0);
    struct Unit {
        u32x4 w[2];
        float s[NS];
    };
    uint32_t from[kInstr], at[kInstr];   // this lane's token row in each copy, and its place in a chunk

    // row_of(r): byte offset of row r's values, x_end for none
    template <class RowOf>
    __device__ void init(RowOf &&row_of, int wave, int lane)
    {
#pragma unroll
        for (int q = 0; q < kInstr; ++q) {
            const int byte = 1024 * (wave + kWaves * q) + 16 * lane, r = byte / kChunk;
            at[q] = 16 * uint32_t((byte % kChunk / 16) ^ (r & 15));
            from[q] = row_of(r);
        }
    }
    __device__ void copy(const One &o, uint8_t *stage, int chunk, uint32_t token_bytes, int wave) const
    {
#pragma unroll
        for (int q = 0; q < kInstr; ++q) {
            const uint32_t off = uint32_t(chunk) * kChunk + at[q];
            buffer_load_lds16(o.x_rsrc, stage + 1024 * (wave + kWaves * q),
                              off < token_bytes && from[q] != o.x_end ? from[q] + off : o.x_end, 0);
        }
    }
    __device__ void load(const One &o, Unit &d, int u, int units, int g, bool last) const
    {
        const uint32_t off = 64u * uint32_t(u) + 16u * uint32_t(g);
        const bool out = u >= units || off >= o.row_bytes;
#pragma unroll
        for (int t = 0; t < 2; ++t)
            d.w[t] = buffer_load16(o.w_rsrc, out ? o.w_end : o.w_row[t] + off, 0);
        if constexpr (WK == kWE4m3)
            if (last)
#pragma unroll
                for (int t = 0; t < NS; ++t)
                    d.s[t] = __builtin_bit_cast(float, buffer_load4(o.s_rsrc, u >= units ? o.s_end : o.s_row[t] + 4u * uint32_t(u / 2), 0));
    }
    // o: rows and ranges; its sums are the result.  The turn-th chunk is the first:
    // workgroups and experts that start at different places keep all channels of
    // the memory busy (us for the layer, all from the first chunk, neighbours'
    // workgroups apart, and the experts too: 16 tokens, 4 of 32 experts of 4096 x
    // 2048 bf16 228, 219, 216; 64, 4 of 4 of 4096 x 4096 131, 121, 119; 32, 4 of 16
    // of 4096 x 2048 181, 189, 154; 64, 8 of 64 of 2048 x 1024 E4M3 96, 96, 96)
    __device__ void run(One &o, uint8_t *stage0, uint8_t *stage1, uint32_t token_bytes, int turn, int wave, int lane) const
    {
        const int x16 = lane & 15, g = lane >> 4;
        const int units = int((o.row_bytes + 63) / 64), whole = WK == kWE4m3 ? (units + 1) & ~1 : units;
        const int chunks = (whole + kUnits - 1) / kUnits, rot = turn % chunks;
        auto place = [&](int c) { return c >= chunks ? chunks : c + rot - (c + rot >= chunks ? chunks : 0); };
#pragma unroll
        for (int t = 0; t < NT; ++t)
            o.acc[t][0] = o.acc[t][1] = f32x4{};
        Unit d[kUnits];
        copy(o, stage0, place(0), token_bytes, wave);
        __builtin_amdgcn_sched_barrier(0);   // (the wait below counts the loads behind the copies)
        static_for<0, kUnits>([&](auto i) {
            load(o, d[i], place(0) * kUnits + i, whole, g, i % 2 == 1);
            __builtin_amdgcn_sched_barrier(0);
        });
        lds_barrier_keep_vm<kLoads>();
        __builtin_amdgcn_sched_barrier(0);
        f32x4 part[NT][2];
        auto chunk = [&](const uint8_t *stage, uint8_t *next, int c) {
            const int then = place(c + 1);
            copy(o, next, then, token_bytes, wave);
            __builtin_amdgcn_sched_barrier(0);
            static_for<0, kUnits>([&](auto ic) {
                constexpr int i = decltype(ic)::value;
                u32x4 x[NT][NX];
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int p = 0; p < NX; ++p)
                        x[t][p] = lds_read16(stage, (16 * t + x16) * kChunk + (((NX * (4 * i + g) + p) ^ x16) << 4));
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    if constexpr (WK == kW16) {
                        One::template steps<NT>(d[i].w[w], x, o.acc, w);
                    } else {
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const u32x4 v = from_e4m3<BF16 || DOWN>(d[i].w[w][2 * q], d[i].w[w][2 * q + 1]);
#pragma unroll
                            for (int t = 0; t < NT; ++t)
                                part[t][w] = One::step(v, x[t] + q * (NX / 2), i % 2 == 0 && q == 0 ? f32x4{} : part[t][w]);
                        }
                        if (i % 2 == 1)
#pragma unroll
                            for (int t = 0; t < NT; ++t)
#pragma unroll
                                for (int r = 0; r < 4; ++r)
                                    o.acc[t][w][r] = fmaf(d[i].s[w % NS], part[t][w][r], o.acc[t][w][r]);
                    }
                }
                load(o, d[i], then * kUnits + i, whole, g, i % 2 == 1);
                __builtin_amdgcn_sched_barrier(0);
            });
            lds_barrier_keep_vm<kLoads>();
            __builtin_amdgcn_sched_barrier(0);
        };
        for (int c = 0; c < chunks; c += 2) {
            chunk(stage0, stage1, c);
            if (c + 1 < chunks)
                chunk(stage1, stage0, c + 1);
        }
        lds_barrier_keep_vm<0>();   // no copy may still be writing LDS
    }
};

// The kernels of a layer with many choices for an expert: as moe_layer_up_kernel
// and moe_layer_rows_kernel, 64 columns of h and 128 of y a workgroup.
template <bool BF16, int WK>
__global__ void __launch_bounds__(kThreads)
moe_layer_up_staged_kernel(LayerArgs a)
{
    __shared__ ExpertRows found;
    __shared__ __attribute__((aligned(1024))) uint8_t stage0[Staged<BF16, WK, false, 4>::kInstr * kWaves * 1024];
    __shared__ __attribute__((aligned(1024))) uint8_t stage1[Staged<BF16, WK, false, 4>::kInstr * kWaves * 1024];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int n;
    const int expert = find_expert(a, found, n);
    if (expert < 0)
        return;
    const uint16_t *const rows = found.rows;
    const int i0 = (int(blockIdx.x) * kWaves + wave) * kCols;
    by_rows<4>(n, [&](int r0, auto tiles) {
        constexpr int NT = decltype(tiles)::value;
        auto o = up_stream<BF16, WK, 2, NT, 2>(a, expert, i0, lane & 15);
        Staged<BF16, WK, false, NT> s;
        s.init([&](int r) { return r0 + r < n ? uint32_t(rows[r0 + r] / uint32_t(a.topk)) * uint32_t(a.ldx) * 2 : o.x_end; },
               wave, lane);
        s.run(o, stage0, stage1, uint32_t(a.H) * 2, blockIdx.x / 4 + 3 * blockIdx.y, wave, lane);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int r = r0 + 16 * t + (lane & 15), i = i0 + 4 * (lane >> 4);
            if (r < n && i < a.I)
                store_h(a, rows[r], i, o.acc[t][0], o.acc[t][1]);
        }
    });
}

template <bool BF16, int WK>
__global__ void __launch_bounds__(kThreads)
moe_layer_rows_staged_kernel(LayerArgs a)
{
    __shared__ __attribute__((aligned(1024))) uint8_t stage0[Staged<BF16, WK, true, 4>::kInstr * kWaves * 1024];
    __shared__ __attribute__((aligned(1024))) uint8_t stage1[Staged<BF16, WK, true, 4>::kInstr * kWaves * 1024];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const LayerTable *const table = static_cast<const LayerTable *>(a.table);
    const int expert = table->slot[blockIdx.y].expert, start = table->slot[blockIdx.y].start, n = table->slot[blockIdx.y].count;
    if (expert < 0)
        return;
    const int h0 = (int(blockIdx.x) * kWaves + wave) * 2 * kCols;
    by_rows<4>(n, [&](int r0, auto tiles) {
        constexpr int NT = decltype(tiles)::value;
        int none[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
            none[t] = -1;
        auto o = down_stream<BF16, WK, 2, NT, 2>(a, expert, h0, none, lane & 15);
        Staged<BF16, WK, true, NT> s;
        s.init([&](int r) { return r0 + r < n ? uint32_t(table->order[start + r0 + r]) * uint32_t(a.I) * 4 : o.x_end; }, wave, lane);
        s.run(o, stage0, stage1, uint32_t(a.I) * 4, blockIdx.x / 2 + 3 * blockIdx.y, wave, lane);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int r = r0 + 16 * t + (lane & 15);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int h = h0 + 16 * i + 4 * (lane >> 4);
                if (r < n && h < a.H)
                    *reinterpret_cast<f32x4 *>(a.rows + int64_t(table->order[start + r]) * a.H + h) = o.acc[t][i];
            }
        }
    });
}

// y[t] = sum_j w[t][j] rows[t][j], in the order of j; four columns a thread,
// the ids and weights of eight choices read at once (whatever lies where a choice
// is left out is not used): one choice after the other the layer of 64 tokens, 8
// of 64 experts of 2048 x 1024 E4M3 took 96.1 us, this way 94.2, that of 8 tokens,
// 8 of 64 of 512 x 256 19.3 and 17.9; the rows' reads pinned before the first sum:
// no more.
template <bool BF16>
__global__ void __launch_bounds__(kSumThreads)
moe_layer_sum_kernel(LayerArgs a)
{
    constexpr int kAtOnce = 8;
    const int t = blockIdx.y, h = (blockIdx.x * kSumThreads + threadIdx.x) * 4;
    if (h >= a.H)
        return;
    f32x4 y = f32x4{};
    for (int j0 = 0; j0 < a.topk; j0 += kAtOnce) {
        f32x4 v[kAtOnce];
        int id[kAtOnce];
        float w[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int c = t * a.topk + min(j0 + i, a.topk - 1);
            v[i] = *reinterpret_cast<const f32x4 *>(a.rows + int64_t(c) * a.H + h);
            id[i] = a.ids[c];
            w[i] = a.w[c];
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            if (j0 + i < a.topk && uint32_t(id[i]) < uint32_t(a.E))
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y[e] = fmaf(w[i], v[i][e], y[e]);
    }
    using T = std::conditional_t<BF16, __bf16, _Float16>;
    typedef T t4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<t4 *>(static_cast<T *>(a.Y) + int64_t(t) * a.ldx + h) = t4{T(y[0]), T(y[1]), T(y[2]), T(y[3])};
}

template <bool BF16, int WK>
hipError_t launch(const LayerArgs &a, hipStream_t stream)
{
    const int choices = a.T * a.topk, experts = a.E < choices ? a.E : choices;
    const dim3 block(kThreads);
    // waves that share a product, until there are enough of them for the chip
    // (28 experts in use of 4096 x 2048 bf16, 16 tokens: 175 and 85 us for the two
    // kernels with 4096 waves, 155 and 85 with 8192, 146 and 86 with 16384; 64
    // experts of 2048 x 1024 E4M3, 64 tokens: 72 and 52, 71 and 47, 74 and 45)
    constexpr int64_t kEnough = WK == kWE4m3 ? 8192 : 16384;
    auto parts_for = [&](int64_t slabs) {
        int parts = 1;
        while (parts < kWaves && experts * slabs * parts < kEnough)
            parts *= 2;
        return parts;
    };
    auto groups = [](int slabs, int parts) { return uint32_t((slabs + kWaves / parts - 1) / (kWaves / parts)); };
    // With two rows an expert or more, the tokens' values by way of LDS, as long
    // as that makes workgroups for half of the chip (us for the whole layer, with
    // neither kernel, the first, the second, both: 64 tokens, 4 of 4 experts of
    // 4096 x 4096 bf16 247, 161, 205, 119; E4M3 139, 99, 124, 85; 8 of 64 of 2048 x
    // 1024 E4M3 119, 106, 110, 96; 32 tokens, 4 of 16 of 4096 x 2048 bf16 186, 171,
    // 170, 154; 8 tokens, 4 of 16 of 2048 x 2048 bf16 81, -, 75.2, 75.0; E4M3 54.5,
    // -, 52.7, 47.6; the other way 10 tokens, 5 of 10 of 2048 x 2048 -, 74, 65, 72,
    // whose 320 and 160 workgroups fill the chip badly; too few workgroups: 30
    // tokens, 2 of 4 of 1024 x 1024 20, 23, -, 27)
    auto staged = [&](int groups) { return choices >= 2 * experts && int64_t(groups) * experts >= 128; };
    constexpr int TILES = tiles_of<WK>();
    const int staged_up = (a.I + kWaves * kCols - 1) / (kWaves * kCols);
    if (choices > kFewChoices && staged(staged_up)) {
        hipLaunchKernelGGL((moe_layer_up_staged_kernel<BF16, WK>), dim3(staged_up, experts), block, 0, stream, a);
    } else {
        const int slabs = (a.I + 8 * TILES - 1) / (8 * TILES), parts = parts_for(slabs);
        hipLaunchKernelGGL((moe_layer_up_kernel<BF16, WK>), dim3(groups(slabs, parts), experts), block, 0, stream, a, parts);
    }
    if (choices <= kFewChoices) {
        // waves that share an expert, as long as there is one for each
        int splits = 1;
        while (2 * splits * experts <= kFewWaves)
            splits *= 2;
        hipLaunchKernelGGL((moe_layer_down_kernel<BF16, WK>), dim3((a.H + kCols - 1) / kCols), dim3(64 * kFewWaves), 0, stream,
                           a, experts, splits);
        return hipGetLastError();
    }
    const int staged_down = (a.H + 2 * kWaves * kCols - 1) / (2 * kWaves * kCols);
    if (staged(staged_down)) {
        hipLaunchKernelGGL((moe_layer_rows_staged_kernel<BF16, WK>), dim3(staged_down, experts), block, 0, stream, a);
    } else {
        const int wide = (a.H + TILES * kCols - 1) / (TILES * kCols), parts = parts_for(wide);
        hipLaunchKernelGGL((moe_layer_rows_kernel<BF16, WK>), dim3(groups(wide, parts), experts), block, 0, stream, a, parts);
    }
    hipLaunchKernelGGL(moe_layer_sum_kernel<BF16>, dim3((a.H + 4 * kSumThreads - 1) / (4 * kSumThreads), a.T),
                       dim3(kSumThreads), 0, stream, a);
    return hipGetLastError();
}

// bytes of h, whole 16-byte pieces
int64_t h_bytes(const LayerArgs &a) { return int64_t(a.T) * a.topk * a.I * 4; }

}  // namespace

int64_t layer_workspace_bytes(const LayerArgs &a)
{
    const int64_t choices = int64_t(a.T) * a.topk;
    return int64_t(sizeof(LayerTable)) + h_bytes(a) + (choices > kFewChoices ? choices * a.H * 4 : 0);
}

hipError_t launch_moe_layer(const LayerArgs &args, void *workspace, hipStream_t stream)
{
    LayerArgs a = args;
    a.table = workspace;
    a.h = static_cast<uint8_t *>(workspace) + sizeof(LayerTable);
    a.rows = reinterpret_cast<float *>(static_cast<uint8_t *>(a.h) + h_bytes(a));
    if (a.e4m3)
        return a.bf16 ? launch<true, kWE4m3>(a, stream) : launch<false, kWE4m3>(a, stream);
    return a.bf16 ? launch<true, kW16>(a, stream) : launch<false, kW16>(a, stream);
}

}  // namespace mswz
