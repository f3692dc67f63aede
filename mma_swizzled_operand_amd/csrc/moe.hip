// moe.hip — tokens to their experts' rows and back: a stable counting sort of
// the T x topk choices by expert, the copy of the token rows in that order, the
// weighted sum back, and its gradient.  All of it is bound by memory: each
// row is read and written once, in 16-byte pieces, 1 KiB per wave and
// instruction, one wave per (token, 1 KiB column piece) so that neither few
// long rows nor many short ones leave the chip idle.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.hpp"
#include "experts.hpp"
#include "kernels.hpp"

namespace mswz {
namespace {

constexpr int kSortThreads = 256, kSortWaves = kSortThreads / 64;
constexpr int kRounds = 8;                                  // choices per lane
constexpr int kSlots = kSortThreads * kRounds;              // choices per workgroup of the sort
constexpr int kMaxE = 1024;

// Lanes that hold the same key, as a mask: one ballot per key bit.
__device__ __forceinline__ uint64_t same_key(uint32_t key, int bits)
{
    uint64_t m = ~uint64_t(0);
    for (int b = 0; b < bits; ++b) {
        const uint64_t v = __ballot((key >> b) & 1u);
        m &= (key >> b) & 1u ? v : ~v;
    }
    return m;
}

// The sort's common part.  Wave w of workgroup g owns choices
// kSlots g + 512 w .. +511, 64 per round in choice order.  rank[r] is the
// number of the wave's earlier choices of the same expert, hist[w][e] the
// wave's count.  Choices left out and places beyond n count as expert E,
// which has no row of hist.
__device__ __forceinline__ void wave_ranks(const int32_t *__restrict__ ids, int n, int E, int bits, int first,
                                           int32_t *hist, int lane, uint32_t *key, int *rank)
{
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int slot = first + 64 * r + lane;
        const uint32_t id = slot < n ? uint32_t(ids[slot]) : uint32_t(E);
        key[r] = id < uint32_t(E) ? id : uint32_t(E);
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const uint64_t same = same_key(key[r], bits);
        const uint64_t below = same & ((uint64_t(1) << lane) - 1);
        rank[r] = __builtin_popcountll(below);
        if (key[r] < uint32_t(E)) {
            rank[r] += hist[key[r]];
        }
        wave_lds_sync();   // every lane has read the count before its group's first lane raises it
        if (key[r] < uint32_t(E) && below == 0)
            hist[key[r]] += __builtin_popcountll(same);
        wave_lds_sync();
    }
}

// Counts of each workgroup's choices, [workgroup][E].
__global__ void __launch_bounds__(kSortThreads)
moe_count_kernel(const int32_t *__restrict__ ids, int n, int E, int32_t *__restrict__ counts)
{
    __shared__ int32_t hist[kMaxE];
    for (int e = threadIdx.x; e < E; e += kSortThreads)
        hist[e] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int slot = blockIdx.x * kSlots + r * kSortThreads + threadIdx.x;
        const uint32_t id = slot < n ? uint32_t(ids[slot]) : uint32_t(E);
        if (id < uint32_t(E))
            atomicAdd(&hist[id], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kSortThreads)
        counts[int64_t(blockIdx.x) * E + e] = hist[e];
}

// Places of a workgroup's choices: the counts of all workgroups give each
// expert's first row and what earlier workgroups put before this one's
// choices, the waves' own counts the rest.
__global__ void __launch_bounds__(kSortThreads)
moe_place_kernel(const int32_t *__restrict__ ids, int n, int E, int bits, const int32_t *__restrict__ counts,
                 int32_t *__restrict__ offsets, int32_t *__restrict__ order, int32_t *__restrict__ pos)
{
    __shared__ int32_t hist[kSortWaves][kMaxE];
    __shared__ int32_t base[kMaxE];
    __shared__ int32_t wave_sum[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, groups = gridDim.x;
    for (int e = tid; e < kSortWaves * kMaxE; e += kSortThreads)
        (&hist[0][0])[e] = 0;
    __syncthreads();
    uint32_t key[kRounds];
    int rank[kRounds];
    const int first = blockIdx.x * kSlots + wave * 64 * kRounds;
    wave_ranks(ids, n, E, bits, first, hist[wave], lane, key, rank);

    // each thread: up to four consecutive experts' totals, then a scan over threads
    constexpr int kPer = kMaxE / kSortThreads;
    int total[kPer], before[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = tid * kPer + i;
        total[i] = before[i] = 0;
        if (e < E)
            for (int g = 0; g < groups; ++g) {
                const int c = counts[int64_t(g) * E + e];
                total[i] += c;
                before[i] += g < int(blockIdx.x) ? c : 0;
            }
        sum += total[i];
    }
    const int scan = wave_scan(sum, lane);
    if (lane == 63)
        wave_sum[wave] = scan;
    __syncthreads();
    int start = scan - sum, used = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
        start += w < wave ? wave_sum[w] : 0;
        used += wave_sum[w];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = tid * kPer + i;
        if (e < E) {
            base[e] = start + before[i];
            if (blockIdx.x == 0) {
                offsets[e] = start;
                if (e == E - 1)
                    offsets[E] = start + total[i];
            }
        }
        start += total[i];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int slot = first + 64 * r + lane;
        if (slot >= n)
            continue;
        int p = -1;
        if (key[r] < uint32_t(E)) {
            p = base[key[r]] + rank[r];
            for (int w = 0; w < wave; ++w)
                p += hist[w][key[r]];
            order[p] = slot;
        }
        pos[slot] = p;
        // places behind the last group hold no choice
        if (slot >= used)
            order[slot] = -1;
    }
}

// Xs[pos[t][j]] = X[t]: one wave per token and 1 KiB column piece.
__global__ void __launch_bounds__(256)
moe_gather_kernel(const u32x4 *__restrict__ X, const int32_t *__restrict__ pos, u32x4 *__restrict__ Xs, int T, int topk,
                  int vecs, int pieces, int64_t ldx16)
{
    const int lane = threadIdx.x & 63;
    const int64_t id = int64_t(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = int(id / pieces), v = int(id % pieces) * 64 + lane;
    if (t >= T || v >= vecs)
        return;
    const u32x4 x = X[t * ldx16 + v];
    for (int j = 0; j < topk; ++j) {
        const int p = pos[int64_t(t) * topk + j];
        if (p >= 0)
            Xs[int64_t(p) * vecs + v] = x;
    }
}

// 16 bytes of row elements as floats, and back (rounded to nearest even).
template <int DT>
struct Row16 {
    static constexpr int kElems = DT == kOutF32 ? 4 : 8;
    using T = std::conditional_t<DT == kOutF32, float, std::conditional_t<DT == kOutBf16, __bf16, _Float16>>;
    typedef T vec __attribute__((ext_vector_type(kElems)));
    __device__ static void get(u32x4 r, float *f)
    {
        const vec v = __builtin_bit_cast(vec, r);
#pragma unroll
        for (int i = 0; i < kElems; ++i)
            f[i] = float(v[i]);
    }
    __device__ static u32x4 put(const float *f)
    {
        vec v;
#pragma unroll
        for (int i = 0; i < kElems; ++i)
            v[i] = T(f[i]);
        return __builtin_bit_cast(u32x4, v);
    }
};

// Y[t] = sum_j w Ys[pos]: one wave per token and 1 KiB column piece; the sum is
// held in fp32 and rounded once.
template <int DT, bool WEIGHTS>
__global__ void __launch_bounds__(256)
moe_combine_kernel(const u32x4 *__restrict__ Ys, const int32_t *__restrict__ pos, const float *__restrict__ w,
                   u32x4 *__restrict__ Y, int T, int topk, int vecs, int pieces, int64_t ldx16)
{
    using R = Row16<DT>;
    const int lane = threadIdx.x & 63;
    const int64_t id = int64_t(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = int(id / pieces), v = int(id % pieces) * 64 + lane;
    if (t >= T || v >= vecs)
        return;
    const uint32_t rows = uint32_t(T) * uint32_t(topk);
    float acc[R::kElems] = {};
    for (int j = 0; j < topk; ++j) {
        const uint32_t p = uint32_t(pos[int64_t(t) * topk + j]);
        if (p >= rows)
            continue;
        float y[R::kElems];
        R::get(Ys[int64_t(p) * vecs + v], y);
        const float wj = WEIGHTS ? w[int64_t(t) * topk + j] : 1.0f;
#pragma unroll
        for (int i = 0; i < R::kElems; ++i)
            acc[i] = WEIGHTS ? __builtin_fmaf(wj, y[i], acc[i]) : acc[i] + y[i];
    }
    Y[t * ldx16 + v] = R::put(acc);
}

// dYs[pos] = w dY[t], dw = <dY[t], Ys[pos]>: one workgroup per token, its four
// waves taking the row's 1 KiB pieces in turn; choices in groups of kJ, whose
// dot products stay in registers and are summed over lanes, then waves, in a
// fixed order.
template <int DT>
__global__ void __launch_bounds__(256)
moe_combine_grad_kernel(const u32x4 *__restrict__ dY, const u32x4 *__restrict__ Ys, const int32_t *__restrict__ pos,
                        const float *__restrict__ w, u32x4 *__restrict__ dYs, float *__restrict__ dw, int T, int topk,
                        int vecs, int64_t ldx16)
{
    using R = Row16<DT>;
    constexpr int kJ = 8;
    __shared__ float part[4][kJ];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = blockIdx.x;
    const uint32_t rows = uint32_t(T) * uint32_t(topk);
    for (int j0 = 0; j0 < topk; j0 += kJ) {
        float dot[kJ] = {};
        for (int v = threadIdx.x; v < vecs; v += 256) {
            float dy[R::kElems];
            R::get(dY[t * ldx16 + v], dy);
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                if (j0 + j >= topk)
                    break;
                const uint32_t p = uint32_t(pos[t * topk + j0 + j]);
                if (p >= rows)
                    continue;
                float y[R::kElems], g[R::kElems];
                R::get(Ys[int64_t(p) * vecs + v], y);
                const float wj = w[t * topk + j0 + j];
#pragma unroll
                for (int i = 0; i < R::kElems; ++i) {
                    dot[j] = __builtin_fmaf(dy[i], y[i], dot[j]);
                    g[i] = wj * dy[i];
                }
                dYs[int64_t(p) * vecs + v] = R::put(g);
            }
        }
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
#pragma unroll
            for (int d = 32; d; d /= 2)
                dot[j] += __shfl_xor(dot[j], d);
            if (lane == 0)
                part[wave][j] = dot[j];
        }
        __syncthreads();
        if (int(threadIdx.x) < kJ && j0 + int(threadIdx.x) < topk)
            dw[t * topk + j0 + threadIdx.x] =
                (part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]);
        __syncthreads();
    }
}

int bits_for(int E)
{
    int b = 1;
    while ((1 << b) <= E)   // keys 0 .. E
        ++b;
    return b;
}

}  // namespace

int64_t moe_workspace_bytes(const MoeArgs &a)
{
    const int64_t n = int64_t(a.T) * a.topk;
    return (n + kSlots - 1) / kSlots * a.E * 4;
}

hipError_t launch_moe_dispatch(const MoeArgs &a, const int32_t *ids, const void *X, void *Xs, int32_t *offsets,
                               int32_t *order, int32_t *pos, void *workspace, hipStream_t stream)
{
    const int n = a.T * a.topk, groups = (n + kSlots - 1) / kSlots;
    int32_t *counts = static_cast<int32_t *>(workspace);
    hipLaunchKernelGGL(moe_count_kernel, dim3(groups), dim3(kSortThreads), 0, stream, ids, n, a.E, counts);
    hipLaunchKernelGGL(moe_place_kernel, dim3(groups), dim3(kSortThreads), 0, stream, ids, n, a.E, bits_for(a.E), counts,
                       offsets, order, pos);
    if (X) {
        const int pieces = (a.vecs + 63) / 64;
        const int64_t blocks = (int64_t(a.T) * pieces + 3) / 4;
        hipLaunchKernelGGL(moe_gather_kernel, dim3(unsigned(blocks)), dim3(256), 0, stream, static_cast<const u32x4 *>(X),
                           pos, static_cast<u32x4 *>(Xs), a.T, a.topk, a.vecs, pieces, a.ldx16);
    }
    return hipGetLastError();
}

namespace {

template <int DT>
hipError_t combine_dt(const MoeArgs &a, const void *Ys, const int32_t *pos, const float *w, void *Y, hipStream_t stream)
{
    const int pieces = (a.vecs + 63) / 64;
    const int64_t blocks = (int64_t(a.T) * pieces + 3) / 4;
    auto *y = static_cast<u32x4 *>(Y);
    auto *ys = static_cast<const u32x4 *>(Ys);
    if (w)
        hipLaunchKernelGGL((moe_combine_kernel<DT, true>), dim3(unsigned(blocks)), dim3(256), 0, stream, ys, pos, w, y, a.T,
                           a.topk, a.vecs, pieces, a.ldx16);
    else
        hipLaunchKernelGGL((moe_combine_kernel<DT, false>), dim3(unsigned(blocks)), dim3(256), 0, stream, ys, pos, w, y,
                           a.T, a.topk, a.vecs, pieces, a.ldx16);
    return hipGetLastError();
}

template <int DT>
hipError_t grad_dt(const MoeArgs &a, const void *dY, const void *Ys, const int32_t *pos, const float *w, void *dYs,
                   float *dw, hipStream_t stream)
{
    hipLaunchKernelGGL((moe_combine_grad_kernel<DT>), dim3(a.T), dim3(256), 0, stream, static_cast<const u32x4 *>(dY),
                       static_cast<const u32x4 *>(Ys), pos, w, static_cast<u32x4 *>(dYs), dw, a.T, a.topk, a.vecs, a.ldx16);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_combine(const MoeArgs &a, const void *Ys, const int32_t *pos, const float *w, void *Y,
                              hipStream_t stream)
{
    switch (a.dt) {
    case kOutBf16: return combine_dt<kOutBf16>(a, Ys, pos, w, Y, stream);
    case kOutF16: return combine_dt<kOutF16>(a, Ys, pos, w, Y, stream);
    default: return combine_dt<kOutF32>(a, Ys, pos, w, Y, stream);
    }
}

hipError_t launch_moe_combine_grad(const MoeArgs &a, const void *dY, const void *Ys, const int32_t *pos, const float *w,
                                   void *dYs, float *dw, hipStream_t stream)
{
    switch (a.dt) {
    case kOutBf16: return grad_dt<kOutBf16>(a, dY, Ys, pos, w, dYs, dw, stream);
    case kOutF16: return grad_dt<kOutF16>(a, dY, Ys, pos, w, dYs, dw, stream);
    default: return grad_dt<kOutF32>(a, dY, Ys, pos, w, dYs, dw, stream);
    }
}

}  // namespace mswz
