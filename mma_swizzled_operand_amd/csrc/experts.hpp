// experts.hpp — internal interface between the C ABI of the expert operators
// (experts_abi.hip) and their kernels (moe.hip, gemm_w4*.hip,
// gemm_grouped*.hip), and what those kernels share.  Not installed.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mswz {

// element kinds of rows and scales, as in OutKind (kernels.hpp)
struct MoeArgs {
    int T, topk, E;
    int vecs;                // 16-byte pieces of one row
    int64_t ldx16;           // 16-byte pieces from one token's row to the next
    int dt;                  // OutKind
};

int64_t moe_workspace_bytes(const MoeArgs &a);
hipError_t launch_moe_dispatch(const MoeArgs &a, const int32_t *ids, const void *X, void *Xs, int32_t *offsets,
                               int32_t *order, int32_t *pos, void *workspace, hipStream_t stream);
hipError_t launch_moe_combine(const MoeArgs &a, const void *Ys, const int32_t *pos, const float *w, void *Y,
                              hipStream_t stream);
hipError_t launch_moe_combine_grad(const MoeArgs &a, const void *dY, const void *Ys, const int32_t *pos,
                                   const float *w, void *dYs, float *dw, hipStream_t stream);

struct W4Args {
    const void *A;
    const uint8_t *B;
    const void *S;
    const uint8_t *Z;
    const int32_t *offsets;  // NULL: one weight matrix
    void *D;
    float *ws;               // partials of the split form
    int M, N, K, E;
    int group, groups;       // K elements per scale, scales per row
    int lda, ldd;
    int beta;
    int out;                 // OutKind
    bool bf16, e2m1;
    int parts = 1;           // K parts of the split form (set by launch_w4)
};

int w4_rows(const W4Args &a);         // rows of the tile that the launch takes
int64_t w4_tiles64(const W4Args &a);  // tiles of 64 rows that hold some
int64_t w4_workspace_bytes(const W4Args &a);
hipError_t launch_w4(const W4Args &a, hipStream_t stream);
// one unit per activation and weight kind
hipError_t launch_w4_bf16_u4(const W4Args &a, hipStream_t stream);
hipError_t launch_w4_bf16_e2m1(const W4Args &a, hipStream_t stream);
hipError_t launch_w4_f16_u4(const W4Args &a, hipStream_t stream);
hipError_t launch_w4_f16_e2m1(const W4Args &a, hipStream_t stream);

struct GroupedArgs {
    const void *A;
    const void *B;
    const int32_t *offsets;
    void *D;
    int E, M, N, K;
    int beta;
    int out;                 // OutKind
    bool bf16, k_axis, b_mn;
};

hipError_t launch_grouped(const GroupedArgs &a, hipStream_t stream);
hipError_t launch_grouped_m_bf16(const GroupedArgs &a, hipStream_t stream);
hipError_t launch_grouped_m_f16(const GroupedArgs &a, hipStream_t stream);
hipError_t launch_grouped_k_bf16(const GroupedArgs &a, hipStream_t stream);
hipError_t launch_grouped_k_f16(const GroupedArgs &a, hipStream_t stream);

// choices (tokens times choices of each) that a layer takes
constexpr int kLayerChoices = 1024;
enum LayerAct { kActSilu = 0, kActGelu = 1 };

struct LayerArgs {
    const void *X;           // [T][ldx]
    const int32_t *ids;      // [T][topk]
    const float *w;          // [T][topk]
    const void *W1;          // [E][2I][H]
    const float *S1;         // e4m3: [E][2][ceil(I/128)][ceil(H/128)]
    const void *W2;          // [E][H][I]
    const float *S2;         // e4m3: [E][ceil(H/128)][ceil(I/128)]
    void *Y;                 // [T][ldx]
    void *table, *h;         // parts of the workspace
    float *rows;             // [T * topk][H]
    int T, topk, E, H, I;
    int64_t ldx;
    int act;                 // LayerAct
    bool bf16, e4m3;
};

int64_t layer_workspace_bytes(const LayerArgs &a);
hipError_t launch_moe_layer(const LayerArgs &a, void *workspace, hipStream_t stream);

// Bounds of group e in 0 .. rows, whatever the array holds: an expert's rows
// are [lo, hi), empty where the bounds do not ascend.
__device__ __forceinline__ void group_bounds(const int32_t *offsets, int e, int rows, int &lo, int &hi)
{
    lo = min(max(offsets[e], 0), rows);
    hi = min(max(offsets[e + 1], lo), rows);
}

// Sum of v over the lanes up to and including this one.
__device__ __forceinline__ int wave_scan(int v, int lane)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int up = __shfl_up(v, d);
        v += lane >= d ? up : 0;
    }
    return v;
}

// Row tiles of all groups, tile_rows rows each (every lane takes part).
__device__ __forceinline__ int group_tiles(const int32_t *offsets, int E, int rows, int tile_rows, int lane)
{
    int sum = 0;
    for (int c = 0; c < E; c += 64) {
        int lo = 0, hi = 0;
        if (c + lane < E)
            group_bounds(offsets, c + lane, rows, lo, hi);
        sum += (hi - lo + tile_rows - 1) / tile_rows;
    }
    return __builtin_amdgcn_readlane(wave_scan(sum, lane), 63);
}

// The group and row tile of tile number t, counted group by group; false
// beyond the last.  Every lane takes part and gets the same answer: lane l
// counts the tiles of group c + l, and the running sum shows the group that
// tile t falls into.
__device__ __forceinline__ bool group_of_tile(const int32_t *offsets, int E, int rows, int tile_rows, int t, int lane,
                                              int &e, int &tile, int &lo, int &hi)
{
    int before = 0;
    for (int c = 0; c < E; c += 64) {
        int l0 = 0, h0 = 0;
        if (c + lane < E)
            group_bounds(offsets, c + lane, rows, l0, h0);
        const int mine = (h0 - l0 + tile_rows - 1) / tile_rows;
        const int sum = wave_scan(mine, lane);
        const uint64_t past = __ballot(before + sum > t);
        if (past) {
            const int who = __builtin_ctzll(past);
            e = c + who;
            tile = t - before - __builtin_amdgcn_readlane(sum - mine, who);
            lo = __builtin_amdgcn_readlane(l0, who);
            hi = __builtin_amdgcn_readlane(h0, who);
            return true;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
    }
    return false;
}

// The group that comes at place `rank` when groups are ordered by length, the
// longest first (equal ones in their own order); up to 64 groups, more keep
// their own order.  Every lane takes part.
__device__ __forceinline__ int group_by_length(const int32_t *offsets, int E, int rows, int rank, int lane)
{
    if (E > 64)
        return rank;
    int lo = 0, hi = -1;
    if (lane < E)
        group_bounds(offsets, lane, rows, lo, hi);
    const int mine = hi - lo;
    int before = 0;
    for (int i = 0; i < E; ++i) {
        const int other = __builtin_amdgcn_readlane(mine, i);
        before += other > mine || (other == mine && i < lane);
    }
    return __builtin_ctzll(__ballot(lane < E && before == rank));
}

// Most row tiles that E groups of together at most `rows` rows can make.
inline int64_t most_tiles(int64_t E, int64_t rows, int64_t tile_rows)
{
    return (E < rows ? E : rows) + rows / tile_rows;
}

}  // namespace mswz
