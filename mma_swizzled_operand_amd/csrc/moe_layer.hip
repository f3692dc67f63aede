// moe_layer.hip — a gated layer of experts for a few tokens, in two kernels:
//     h[c]  = act(W1[e][:I] x) * (W1[e][I:] x)        for each choice c = (t, j), e = ids[t][j]
//     y[t]  = sum_j w[t][j] W2[e] h[c]
//
// With a few tokens the time is that of reading the chosen experts' weights
// once.  A workgroup owns 16 columns of h (or of y), its eight waves split
// the inner size between them, and each lane loads its weight rows' pieces
// straight into registers, without a barrier until the waves' sums meet.  The
// rows of an expert are found from the ids by the workgroups themselves.
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
#include "kernels.hpp"

namespace mswz {
namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves, kPerWave = kLayerChoices / kWaves;
constexpr int kCols = 16;   // columns of h or y a workgroup

enum Weights { kW16 = 0, kWE4m3 = 1 };

// Where the second kernel finds the choices: experts in use, and all choices
// sorted by expert (written by the first kernel).
struct LayerTable {
    int32_t active;                      // experts with a choice
    int32_t pad[3];
    int32_t expert[1024], start[1024], count[1024];
    int32_t order[kLayerChoices];
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

// K elements of a unit, the piece of the inner size that waves share out:
// one MFMA's for 16-bit weights, a scale's block for E4M3.
template <int WK>
constexpr int unit_k() { return WK == kWE4m3 ? 128 : 32; }

// The first kernel: 16 columns of h for the choices of one expert, the
// blockIdx.y-th of those in use.
template <bool BF16, int WK>
__global__ void __launch_bounds__(kThreads)
moe_layer_up_kernel(LayerArgs a)
{
    __shared__ uint32_t used[32];
    __shared__ int before[2][kWaves];
    __shared__ uint16_t rows[kLayerChoices];
    __shared__ __attribute__((aligned(16))) f32x4 sums[kWaves][4][2][64];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int choices = a.T * a.topk;
    // ---- the expert and its choices, in ascending order ----
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
    int expert = -1, active = 0;
    {
        const uint32_t word = lane < 32 ? used[lane] : 0u;
        const int n = __builtin_popcount(word), sum = wave_scan(n, lane);
        active = __builtin_amdgcn_readlane(sum, 63);
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
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0)
        table->active = active;
    if (expert < 0)
        return;
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
    int n = 0, start = 0, at = 0;
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
        for (int r = tid; r < n; r += kThreads)
            table->order[start + r] = rows[r];
        if (tid == 0) {
            table->expert[blockIdx.y] = expert;
            table->start[blockIdx.y] = start;
            table->count[blockIdx.y] = n;
        }
    }

    // ---- the products ----
    constexpr int UK = unit_k<WK>(), kSize = WK == kWE4m3 ? 1 : 2;
    const int i0 = blockIdx.x * kCols, x16 = lane & 15, g = lane >> 4;
    const uint32_t row_bytes = uint32_t(a.H) * kSize, w_bytes = 2u * uint32_t(a.I) * row_bytes;
    const __amdgpu_buffer_rsrc_t w_rsrc = make_rsrc(static_cast<const uint8_t *>(a.W1) + uint64_t(expert) * w_bytes, w_bytes);
    const uint32_t x_pitch = uint32_t(a.ldx) * 2, x_bytes = uint32_t(a.T - 1) * x_pitch + uint32_t(a.H) * 2;
    const __amdgpu_buffer_rsrc_t x_rsrc = make_rsrc(a.X, x_bytes);
    const uint32_t gate = uint32_t(min(i0 + x16, a.I - 1)) * row_bytes, up = gate + uint32_t(a.I) * row_bytes;
    const int units = (a.H + UK - 1) / UK, u0 = units * wave / kWaves, u1 = units * (wave + 1) / kWaves;
    const int ib = (a.I + 127) / 128, hb = (a.H + 127) / 128;
    const float *const s_gate = WK == kWE4m3 ? a.S1 + (int64_t(expert) * 2 * ib + i0 / 128) * hb : nullptr;
    const float *const s_up = WK == kWE4m3 ? s_gate + int64_t(ib) * hb : nullptr;

    auto some = [&](int r0, auto tiles) {
        constexpr int NT = decltype(tiles)::value;
        uint32_t xrow[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int r = r0 + 16 * t + x16;
            xrow[t] = r < n ? uint32_t(rows[r] / a.topk) * x_pitch : x_bytes;
        }
        f32x4 acc[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t)
            acc[t][0] = acc[t][1] = f32x4{};
        // (a piece beyond the inner size reads zeros, and so does a token beyond the last)
        auto x_at = [&](int t, int k) { return buffer_load16(x_rsrc, k < a.H ? xrow[t] + 2 * uint32_t(k) : x_bytes, 0); };
        if constexpr (WK == kW16) {
#pragma unroll 4
            for (int u = u0; u < u1; ++u) {
                const int k = UK * u + 8 * g;
                const u32x4 wg = buffer_load16(w_rsrc, k < a.H ? gate + 2 * uint32_t(k) : w_bytes, 0);
                const u32x4 wu = buffer_load16(w_rsrc, k < a.H ? up + 2 * uint32_t(k) : w_bytes, 0);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const u32x4 x = x_at(t, k);
                    acc[t][0] = mfma_16x16x32<BF16>(wg, x, acc[t][0]);
                    acc[t][1] = mfma_16x16x32<BF16>(wu, x, acc[t][1]);
                }
            }
        } else {
            for (int u = u0; u < u1; ++u) {
                const float sg = s_gate[u], su = s_up[u];
                f32x4 part[NT][2];
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    part[t][0] = part[t][1] = f32x4{};
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int k = UK * u + 64 * half + 16 * g;
                    const u32x4 wg = buffer_load16(w_rsrc, k < a.H ? gate + uint32_t(k) : w_bytes, 0);
                    const u32x4 wu = buffer_load16(w_rsrc, k < a.H ? up + uint32_t(k) : w_bytes, 0);
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const u32x4 x = x_at(t, k + 8 * q);
                            part[t][0] = mfma_16x16x32<BF16>(from_e4m3<BF16>(wg[2 * q], wg[2 * q + 1]), x, part[t][0]);
                            part[t][1] = mfma_16x16x32<BF16>(from_e4m3<BF16>(wu[2 * q], wu[2 * q + 1]), x, part[t][1]);
                        }
                }
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        acc[t][0][r] = fmaf(sg, part[t][0][r], acc[t][0][r]);
                        acc[t][1][r] = fmaf(su, part[t][1][r], acc[t][1][r]);
                    }
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            sums[wave][t][0][lane] = acc[t][0];
            sums[wave][t][1][lane] = acc[t][1];
        }
        __syncthreads();
        if (wave < NT) {
            f32x4 vg = f32x4{}, vu = f32x4{};
            for (int w = 0; w < kWaves; ++w) {
                vg += sums[w][wave][0][lane];
                vu += sums[w][wave][1][lane];
            }
            const int r = r0 + 16 * wave + x16, i = i0 + 4 * g;
            if (r < n && i < a.I) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    split_bf16(activation(vg[e], a.act) * vu[e], hi[e], lo[e]);
                // of every 8 columns the upper parts, then the lower ones
                uint8_t *const to = static_cast<uint8_t *>(a.h) + (int64_t(rows[r]) * a.I + (i & ~7)) * 4 + 2 * (i & 7);
                *reinterpret_cast<u32x2 *>(to) = u32x2{hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16)};
                *reinterpret_cast<u32x2 *>(to + 16) = u32x2{lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16)};
            }
        }
        __syncthreads();
    };
    for (int r0 = 0; r0 < n; r0 += 64) {
        if (n - r0 <= 16)
            some(r0, std::integral_constant<int, 1>{});
        else if (n - r0 <= 32)
            some(r0, std::integral_constant<int, 2>{});
        else
            some(r0, std::integral_constant<int, 4>{});
    }
}

// The second kernel: 16 columns of y for all tokens.  Its waves share out the
// experts in use and, `splits` ways, the inner size; each choice's sums go to
// LDS and a token's are added up in the order of its choices.
template <bool BF16, int WK>
__global__ void __launch_bounds__(kThreads)
moe_layer_down_kernel(LayerArgs a, int splits)
{
    extern __shared__ __attribute__((aligned(16))) float of_choice[];   // [splits][choices][16]
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int choices = a.T * a.topk;
    const LayerTable *const table = static_cast<const LayerTable *>(a.table);
    const int active = table->active;

    constexpr int UK = unit_k<WK>(), kSize = WK == kWE4m3 ? 1 : 2;
    const int h0 = blockIdx.x * kCols, x16 = lane & 15, g = lane >> 4;
    const uint32_t row_bytes = uint32_t(a.I) * kSize, w_bytes = uint32_t(a.H) * row_bytes;
    const uint32_t wrow = uint32_t(min(h0 + x16, a.H - 1)) * row_bytes;
    const uint32_t h_bytes = uint32_t(choices) * uint32_t(a.I) * 4;
    const __amdgpu_buffer_rsrc_t h_rsrc = make_rsrc(a.h, h_bytes);
    const int split = wave % splits;
    const int units = (a.I + UK - 1) / UK, u0 = units * split / splits, u1 = units * (split + 1) / splits;
    const int ib = (a.I + 127) / 128, hb = (a.H + 127) / 128;

    for (int slot = wave / splits; slot < active; slot += kWaves / splits) {
        const int expert = table->expert[slot], start = table->start[slot], n = table->count[slot];
        const __amdgpu_buffer_rsrc_t w_rsrc =
            make_rsrc(static_cast<const uint8_t *>(a.W2) + uint64_t(expert) * w_bytes, w_bytes);
        const float *const s_row = WK == kWE4m3 ? a.S2 + (int64_t(expert) * hb + h0 / 128) * ib : nullptr;
        auto some = [&](int r0, auto tiles) {
            constexpr int NT = decltype(tiles)::value;
            int choice[NT];
            uint32_t hrow[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int r = r0 + 16 * t + x16;
                choice[t] = r < n ? table->order[start + r] : -1;
                hrow[t] = r < n ? uint32_t(choice[t]) * uint32_t(a.I) * 4 : h_bytes;
            }
            f32x4 acc[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t)
                acc[t] = f32x4{};
            // the parts of h at columns k .. k + 7
            auto h_at = [&](int t, int k, int part) {
                return buffer_load16(h_rsrc, k < a.I ? hrow[t] + 4 * uint32_t(k) + 16 * part : h_bytes, 0);
            };
            if constexpr (WK == kW16) {
#pragma unroll 4
                for (int u = u0; u < u1; ++u) {
                    const int k = UK * u + 8 * g;
                    const u32x4 w = buffer_load16(w_rsrc, k < a.I ? wrow + 2 * uint32_t(k) : w_bytes, 0);
                    u32x4 whi = w, wlo;
                    if constexpr (!BF16)
                        split_f16x8(w, whi, wlo);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const u32x4 hi = h_at(t, k, 0), lo = h_at(t, k, 1);
                        acc[t] = mfma_16x16x32<true>(whi, hi, acc[t]);
                        acc[t] = mfma_16x16x32<true>(whi, lo, acc[t]);
                        if constexpr (!BF16) {
                            acc[t] = mfma_16x16x32<true>(wlo, hi, acc[t]);
                            acc[t] = mfma_16x16x32<true>(wlo, lo, acc[t]);
                        }
                    }
                }
            } else {
                for (int u = u0; u < u1; ++u) {
                    const float s = s_row[u];
                    f32x4 part[NT];
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        part[t] = f32x4{};
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int k = UK * u + 64 * half + 16 * g;
                        const u32x4 w = buffer_load16(w_rsrc, k < a.I ? wrow + uint32_t(k) : w_bytes, 0);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const u32x4 wq = from_e4m3<true>(w[2 * q], w[2 * q + 1]);
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                part[t] = mfma_16x16x32<true>(wq, h_at(t, k + 8 * q, 0), part[t]);
                                part[t] = mfma_16x16x32<true>(wq, h_at(t, k + 8 * q, 1), part[t]);
                            }
                        }
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[t][r] = fmaf(s, part[t][r], acc[t][r]);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
                if (choice[t] >= 0)
                    *reinterpret_cast<f32x4 *>(of_choice + (split * choices + choice[t]) * kCols + 4 * g) = acc[t];
        };
        for (int r0 = 0; r0 < n; r0 += 64) {
            if (n - r0 <= 16)
                some(r0, std::integral_constant<int, 1>{});
            else if (n - r0 <= 32)
                some(r0, std::integral_constant<int, 2>{});
            else
                some(r0, std::integral_constant<int, 4>{});
        }
    }
    __syncthreads();
    using T = std::conditional_t<BF16, __bf16, _Float16>;
    for (int o = tid; o < a.T * kCols; o += kThreads) {
        const int t = o / kCols, col = o % kCols;
        float y = 0.0f;
        for (int j = 0; j < a.topk; ++j) {
            const int c = t * a.topk + j;
            if (uint32_t(a.ids[c]) >= uint32_t(a.E))
                continue;
            float v = 0.0f;
            for (int s = 0; s < splits; ++s)
                v += of_choice[(s * choices + c) * kCols + col];
            y = fmaf(a.w[c], v, y);
        }
        if (h0 + col < a.H)
            static_cast<T *>(a.Y)[int64_t(t) * a.ldx + h0 + col] = T(y);
    }
}

template <bool BF16, int WK>
hipError_t launch(const LayerArgs &a, hipStream_t stream)
{
    const int choices = a.T * a.topk, experts = a.E < choices ? a.E : choices;
    hipLaunchKernelGGL((moe_layer_up_kernel<BF16, WK>), dim3((a.I + kCols - 1) / kCols, experts), dim3(kThreads), 0, stream, a);
    // waves that share an expert, until the experts in use can be as many as waves
    int splits = 1;
    while (splits < kWaves && experts * splits < 2 * kWaves && 2 * splits * choices <= kLayerChoices)
        splits *= 2;
    const size_t lds = size_t(splits) * choices * kCols * 4;
    hipLaunchKernelGGL((moe_layer_down_kernel<BF16, WK>), dim3((a.H + kCols - 1) / kCols), dim3(kThreads), lds, stream, a, splits);
    return hipGetLastError();
}

}  // namespace

int64_t layer_workspace_bytes(const LayerArgs &a)
{
    return int64_t(sizeof(LayerTable)) + int64_t(a.T) * a.topk * a.I * 4;
}

hipError_t launch_moe_layer(const LayerArgs &args, void *workspace, hipStream_t stream)
{
    LayerArgs a = args;
    a.table = workspace;
    a.h = static_cast<uint8_t *>(workspace) + sizeof(LayerTable);
    if (a.e4m3)
        return a.bf16 ? launch<true, kWE4m3>(a, stream) : launch<false, kWE4m3>(a, stream);
    return a.bf16 ? launch<true, kW16>(a, stream) : launch<false, kW16>(a, stream);
}

}  // namespace mswz
