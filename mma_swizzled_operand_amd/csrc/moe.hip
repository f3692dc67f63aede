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
constexpr int kRounds = 4;                                  // choices per lane
constexpr int kSlots = kSortThreads * kRounds;              // choices per workgroup of the sort
constexpr int kMaxE = 1024;
constexpr int kFew = 1024;                                  // choices that one launch sorts and copies
constexpr int kUncountedMost = 8192;                        // choices that each workgroup of the sort counts itself
constexpr int kCountedMost = 16384, kCountedGroups = 256;   // counts, of so many workgroups, that each one adds up itself

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
// kSlots g + 64 kRounds w .., 64 per round in choice order.  rank[r] is the
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

// Each expert's counts of the workgroups, in place, become what the workgroups
// before it hold, and row `groups` the expert's total.  A workgroup takes
// `width` experts (a power of two); its threads of one expert take a run of
// rows each: one pass adds up the run, a scan over the runs gives each its
// start, a second pass writes.  Eight loads in flight, as in the sort.
constexpr int kScanThreads = 1024, kScanWidth = 16;
__global__ void __launch_bounds__(kScanThreads)
moe_scan_kernel(int32_t *__restrict__ counts, int groups, int E, int width)
{
    __shared__ int32_t sums[kScanThreads];
    const int tid = threadIdx.x, parts = kScanThreads / width, part = tid / width, e = blockIdx.x * width + tid % width;
    const int run = (groups + parts - 1) / parts, g0 = min(part * run, groups), g1 = min(g0 + run, groups);
    int32_t *const c = counts + min(e, E - 1);
    int sum = 0;
    for (int g = g0; g < g1; g += 8) {
        int v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = c[int64_t(min(g + i, g1 - 1)) * E];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum += g + i < g1 ? v[i] : 0;
    }
    // (runs of one expert lie `width` apart)
    sums[tid] = sum;
    __syncthreads();
    for (int d = width; d < kScanThreads; d *= 2) {
        const int before = tid >= d ? sums[tid - d] : 0;
        __syncthreads();
        sums[tid] += before;
        __syncthreads();
    }
    if (e >= E)
        return;
    int before = sums[tid] - sum;
    for (int g = g0; g < g1; g += 8) {
        int v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = c[int64_t(min(g + i, g1 - 1)) * E];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (g + i < g1) {
                c[int64_t(g + i) * E] = before;
                before += v[i];
            }
    }
    if (part == parts - 1)
        c[int64_t(groups) * E] = before;
}

// Places of a workgroup's choices: the counts of all workgroups give each
// expert's first row and what earlier workgroups put before this one's
// choices, the waves' own counts the rest.  kCounted: each workgroup adds up
// moe_count_kernel's counts (from L2), several threads an expert, eight loads
// of each in flight: one load at a time took 20 us at 32 workgroups.
// kUncounted: it counts all choices itself, which saves the other kernel's
// launch while there are few: sort and copy of 2048 / 8192 / 16384 choices with
// it 10.5 / 12.4 / 15.1 us, without 8.4 / 11.7 / 16.8.  kScanned: it finds its
// sums in moe_scan_kernel's table, since adding up all counts in every
// workgroup grows with the square of the choices.
enum Sort { kUncounted, kCounted, kScanned };
template <Sort SORT>
__global__ void __launch_bounds__(kSortThreads)
moe_place_kernel(const int32_t *__restrict__ ids, int n, int E, int bits, const int32_t *__restrict__ counts,
                 int32_t *__restrict__ offsets, int32_t *__restrict__ order, int32_t *__restrict__ pos)
{
    __shared__ int32_t hist[kSortWaves][kMaxE];
    __shared__ int32_t total[kMaxE], base[kMaxE];
    __shared__ int32_t wave_sum[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, groups = gridDim.x;
    for (int e = tid; e < E; e += kSortThreads) {
        total[e] = base[e] = 0;
        for (int w = 0; w < kSortWaves; ++w)
            hist[w][e] = 0;
    }
    __syncthreads();
    if constexpr (SORT == kScanned) {
        for (int e = tid; e < E; e += kSortThreads) {
            total[e] = counts[int64_t(groups) * E + e];
            base[e] = counts[int64_t(blockIdx.x) * E + e];
        }
    } else if constexpr (SORT == kCounted) {
        // experts in columns of `width` threads, groups dealt to the rows of threads
        int width = 64;
        while (width < E && width < kSortThreads)
            width *= 2;
        const int parts = kSortThreads / width, part = tid / width;
        for (int e = tid % width; e < E; e += width) {
            int sum = 0, before = 0;
            for (int g0 = part; g0 < groups; g0 += 8 * parts) {
                int c[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    c[i] = counts[int64_t(min(g0 + i * parts, groups - 1)) * E + e];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int g = g0 + i * parts;
                    sum += g < groups ? c[i] : 0;
                    before += g < int(blockIdx.x) ? c[i] : 0;
                }
            }
            atomicAdd(&total[e], sum);
            atomicAdd(&base[e], before);
        }
    } else {
        const int mine = blockIdx.x * kSlots;
        for (int s0 = tid; s0 < n; s0 += 8 * kSortThreads) {
            uint32_t id[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                id[i] = uint32_t(ids[min(s0 + i * kSortThreads, n - 1)]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int s = s0 + i * kSortThreads;
                if (s < n && id[i] < uint32_t(E)) {
                    atomicAdd(&total[id[i]], 1);
                    if (s < mine)
                        atomicAdd(&base[id[i]], 1);
                }
            }
        }
    }
    uint32_t key[kRounds];
    int rank[kRounds];
    const int first = blockIdx.x * kSlots + wave * 64 * kRounds;
    wave_ranks(ids, n, E, bits, first, hist[wave], lane, key, rank);
    __syncthreads();

    // each thread: consecutive experts' totals, then a scan over threads
    constexpr int kPer = kMaxE / kSortThreads;
    const int per = (E + kSortThreads - 1) / kSortThreads;
    int mine[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        mine[i] = i < per && tid * per + i < E ? total[tid * per + i] : 0;
        sum += mine[i];
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
        const int e = tid * per + i;
        if (i < per && e < E) {
            base[e] += start;
            if (blockIdx.x == 0)
                offsets[e] = start;
        }
        start += mine[i];
    }
    if (blockIdx.x == 0 && tid == 0)
        offsets[E] = used;
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

// Few choices: the sort and the copy in one launch.  Workgroup (t, piece)
// finds the rows of token t's choices by counting the choices before them
// (smaller expert, or the same expert earlier), all of them from one read of
// ids, and copies its piece of the row; workgroup T writes offsets and the
// places behind the last group, from a histogram.  (1024 choices 5.0 us in a
// graph; in two launches 2048 take 8.4.)
__global__ void __launch_bounds__(256)
moe_few_kernel(const int32_t *__restrict__ ids, const u32x4 *__restrict__ X, u32x4 *__restrict__ Xs, int T, int topk,
               int E, int vecs, int64_t ldx16, int32_t *__restrict__ offsets, int32_t *__restrict__ order,
               int32_t *__restrict__ pos)
{
    __shared__ int32_t cnt[kMaxE];
    __shared__ int32_t wave_sum[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = T * topk;
    const int t = blockIdx.x;
    if (t < T) {
        for (int j = tid; j < topk; j += 256)
            cnt[j] = 0;
        __syncthreads();
        constexpr int kPer = kFew / 256;
        uint32_t id[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int s = tid + 256 * i;
            id[i] = s < n ? uint32_t(ids[s]) : ~0u;
        }
        for (int j = 0; j < topk; ++j) {
            const int slot = t * topk + j;
            const uint32_t mine = uint32_t(ids[slot]);
            int before = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                before += __builtin_popcountll(__ballot(id[i] < mine || (id[i] == mine && tid + 256 * i < slot)));
            if (lane == 0 && before)
                atomicAdd(&cnt[j], before);
        }
        __syncthreads();
        if (blockIdx.y == 0)
            for (int j = tid; j < topk; j += 256) {
                const int slot = t * topk + j;
                const bool in = uint32_t(ids[slot]) < uint32_t(E);
                pos[slot] = in ? cnt[j] : -1;
                if (in)
                    order[cnt[j]] = slot;
            }
        const int v = blockIdx.y * 256 + tid;
        if (X && v < vecs) {
            const u32x4 x = X[t * ldx16 + v];
            for (int j = 0; j < topk; ++j)
                if (uint32_t(ids[t * topk + j]) < uint32_t(E))
                    Xs[int64_t(cnt[j]) * vecs + v] = x;
        }
        return;
    }
    if (blockIdx.y)
        return;
    for (int e = tid; e < E; e += 256)
        cnt[e] = 0;
    __syncthreads();
    for (int s = tid; s < n; s += 256) {
        const uint32_t id = uint32_t(ids[s]);
        if (id < uint32_t(E))
            atomicAdd(&cnt[id], 1);
    }
    __syncthreads();
    const int per = (E + 255) / 256;
    int sum = 0;
    for (int i = 0; i < per; ++i)
        sum += tid * per + i < E ? cnt[tid * per + i] : 0;
    const int scan = wave_scan(sum, lane);
    if (lane == 63)
        wave_sum[wave] = scan;
    __syncthreads();
    int start = scan - sum, used = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        start += w < wave ? wave_sum[w] : 0;
        used += wave_sum[w];
    }
    for (int i = 0; i < per; ++i)
        if (tid * per + i < E) {
            offsets[tid * per + i] = start;
            start += cnt[tid * per + i];
        }
    if (tid == 0)
        offsets[E] = used;
    for (int s = used + tid; s < n; s += 256)
        order[s] = -1;
}

// The values of choices j0 .. j0 + J - 1 of token t, J scalar loads at once
// (behind the last choice its value again).
template <int J, typename T>
__device__ __forceinline__ void choices(const T *__restrict__ x, int64_t t, int topk, int j0, T *v)
{
    const T *const p = x + t * topk + j0;
    if (j0 + J <= topk) {
#pragma unroll
        for (int j = 0; j < J; ++j)
            v[j] = p[j];
    } else {
#pragma unroll
        for (int j = 0; j < J; ++j)
            v[j] = p[min(j, topk - 1 - j0)];
    }
}

// A wave's token and first 16-byte piece: a workgroup's four waves share a row
// of four or more 1 KiB pieces, shorter rows go one or two waves a token.
// (Dividing a wave number by the row's pieces, in 64 bits, took more
// instructions than the copy itself.)
struct WaveRow {
    int t, v;
};
__device__ __forceinline__ WaveRow wave_row(int lg)
{
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int t = int((blockIdx.x * 4u + unsigned(wave)) >> lg);
    return {t, (int(blockIdx.y) * 4 + (wave & ((1 << lg) - 1))) * 64 + (int(threadIdx.x) & 63)};
}

// Xs[pos[t][j]] = X[t]: one wave per token and 1 KiB column piece.  Stored past
// the caches: with plain stores the rows' lines had to leave the memory-side
// cache again while the copy (or the sum that follows it) read
// (8192 tokens to 8 experts each, 2048 bf16: 59.4 -> 51.9 us; the sum of 4096
// such tokens after its gradient 40.2 -> 27.6 us, of which the stores in the
// gradient 10 and the sum's own 2.6).
template <int J>
__global__ void __launch_bounds__(256)
moe_gather_kernel(const u32x4 *__restrict__ X, const int32_t *__restrict__ pos, u32x4 *__restrict__ Xs, int T, int topk,
                  int vecs, int lg, int64_t ldx16)
{
    const auto [t, v] = wave_row(lg);
    if (t >= T || v >= vecs)
        return;
    const u32x4 x = X[t * ldx16 + v];
    for (int j0 = 0; j0 < topk; j0 += J) {
        int p[J];
        choices<J>(pos, t, topk, j0, p);
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (p[j] >= 0 && j0 + j < topk)
                __builtin_nontemporal_store(x, &Xs[int64_t(p[j]) * vecs + v]);
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
// held in fp32 and rounded once.  The rows of J choices are loaded before any
// is added, so that their latencies run together; a choice left out loads row
// 0 and is masked, as a branch around a load made each wait for the one before
// (4096 tokens of 8 x 2048 bf16 take 27.6 us, 150 MB at 5.4 TB/s).
template <int DT, bool WEIGHTS, int J>
__global__ void __launch_bounds__(256)
moe_combine_kernel(const u32x4 *__restrict__ Ys, const int32_t *__restrict__ pos, const float *__restrict__ w,
                   u32x4 *__restrict__ Y, int T, int topk, int vecs, int lg, int64_t ldx16)
{
    using R = Row16<DT>;
    const auto [t, v] = wave_row(lg);
    if (t >= T || v >= vecs)
        return;
    const uint32_t rows = uint32_t(T) * uint32_t(topk);
    float acc[R::kElems] = {};
    for (int j0 = 0; j0 < topk; j0 += J) {
        u32x4 y[J];
        int p[J];
        float wj[J];
        choices<J>(pos, t, topk, j0, p);
        if constexpr (WEIGHTS)
            choices<J>(w, t, topk, j0, wj);
#pragma unroll
        for (int j = 0; j < J; ++j)
            y[j] = Ys[int64_t(uint32_t(p[j]) < rows ? p[j] : 0) * vecs + v];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const bool in = uint32_t(p[j]) < rows && j0 + j < topk;
            float f[R::kElems];
            R::get(in ? y[j] : u32x4{}, f);
            const float wi = !WEIGHTS ? 1.0f : in ? wj[j] : 0.0f;
#pragma unroll
            for (int i = 0; i < R::kElems; ++i)
                acc[i] = __builtin_fmaf(wi, f[i], acc[i]);
        }
    }
    __builtin_nontemporal_store(R::put(acc), &Y[t * ldx16 + v]);
}

// dYs[pos] = w dY[t], dw = <dY[t], Ys[pos]>: one workgroup per token, its four
// waves taking the row's 1 KiB pieces in turn; choices in groups of J, loaded
// as in the sum, whose dot products stay in registers and are summed over
// lanes, then waves, in a fixed order.  (4096 tokens of 8 x 2048 bf16: 45.6 us,
// 285 MB at 6.3 TB/s.)
template <int DT, int J>
__global__ void __launch_bounds__(256)
moe_combine_grad_kernel(const u32x4 *__restrict__ dY, const u32x4 *__restrict__ Ys, const int32_t *__restrict__ pos,
                        const float *__restrict__ w, u32x4 *__restrict__ dYs, float *__restrict__ dw, int T, int topk,
                        int vecs, int64_t ldx16)
{
    using R = Row16<DT>;
    __shared__ float part[4][J];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t t = blockIdx.x;
    const uint32_t rows = uint32_t(T) * uint32_t(topk);
    for (int j0 = 0; j0 < topk; j0 += J) {
        float dot[J] = {}, wj[J];
        int p[J];
        choices<J>(pos, t, topk, j0, p);
        choices<J>(w, t, topk, j0, wj);
#pragma unroll
        for (int j = 0; j < J; ++j)
            p[j] = uint32_t(p[j]) < rows && j0 + j < topk ? p[j] : -1;
        for (int v = tid; v < vecs; v += 256) {
            float dy[R::kElems];
            u32x4 y[J];
            const u32x4 d = dY[t * ldx16 + v];
#pragma unroll
            for (int j = 0; j < J; ++j)
                y[j] = __builtin_nontemporal_load(&Ys[int64_t(max(p[j], 0)) * vecs + v]);
            R::get(d, dy);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float f[R::kElems], g[R::kElems];
                R::get(y[j], f);
#pragma unroll
                for (int i = 0; i < R::kElems; ++i) {
                    dot[j] = __builtin_fmaf(dy[i], f[i], dot[j]);
                    g[i] = wj[j] * dy[i];
                }
                if (p[j] >= 0)
                    __builtin_nontemporal_store(R::put(g), &dYs[int64_t(p[j]) * vecs + v]);
            }
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
#pragma unroll
            for (int d = 32; d; d /= 2)
                dot[j] += __shfl_xor(dot[j], d);
            if (lane == 0)
                part[wave][j] = p[j] >= 0 ? dot[j] : 0.0f;
        }
        __syncthreads();
        if (tid < J && j0 + tid < topk)
            dw[t * topk + j0 + tid] = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
        __syncthreads();
    }
}

// waves that share a token's row (log2), and the grid of wave_row
int waves_log2(const MoeArgs &a) { return a.vecs <= 64 ? 0 : a.vecs <= 128 ? 1 : 2; }
dim3 row_grid(const MoeArgs &a, int lg)
{
    return dim3(unsigned(((int64_t(a.T) << lg) + 3) / 4), unsigned((a.vecs + 255) / 256));
}

int bits_for(int E)
{
    int b = 1;
    while ((1 << b) <= E)   // keys 0 .. E
        ++b;
    return b;
}

}  // namespace

static bool few(const MoeArgs &a) { return a.T * a.topk <= kFew; }

static int64_t sort_groups(const MoeArgs &a) { return (int64_t(a.T) * a.topk + kSlots - 1) / kSlots; }

// How the sort finds its sums.  The scan costs a launch and saves every
// workgroup the reading of all counts; the sort alone in a graph, counted /
// scanned, in us: 16 workgroups and 1024 experts 14.2 / 14.8, 32: 18.2 / 15.1;
// 128 and 128 12.9 / 14.0, 256: 16.8 / 14.6; 256 and 64 13.1 / 14.1, 512: 17.8
// / 15.7; 256 and 8 13.5 / 13.3, 512: 17.0 / 14.1; 1024 and 1024 414 / 30.
static Sort sort_of(const MoeArgs &a)
{
    const int64_t groups = sort_groups(a);
    if (int64_t(a.T) * a.topk <= kUncountedMost)
        return kUncounted;
    return groups <= kCountedGroups && groups * a.E <= kCountedMost ? kCounted : kScanned;
}

int64_t moe_workspace_bytes(const MoeArgs &a)
{
    const Sort sort = sort_of(a);
    return sort == kUncounted ? 0 : (sort_groups(a) + (sort == kScanned)) * a.E * 4;
}

hipError_t launch_moe_dispatch(const MoeArgs &a, const int32_t *ids, const void *X, void *Xs, int32_t *offsets,
                               int32_t *order, int32_t *pos, void *workspace, hipStream_t stream)
{
    if (few(a)) {
        hipLaunchKernelGGL(moe_few_kernel, dim3(a.T + 1, X ? (a.vecs + 255) / 256 : 1), dim3(256), 0, stream, ids,
                           static_cast<const u32x4 *>(X), static_cast<u32x4 *>(Xs), a.T, a.topk, a.E, a.vecs, a.ldx16,
                           offsets, order, pos);
        return hipGetLastError();
    }
    const int n = a.T * a.topk, groups = int(sort_groups(a));
    const int bits = bits_for(a.E);
    int32_t *counts = static_cast<int32_t *>(workspace);
    const Sort sort = sort_of(a);
    if (sort == kUncounted) {
        hipLaunchKernelGGL(moe_place_kernel<kUncounted>, dim3(groups), dim3(kSortThreads), 0, stream, ids, n, a.E, bits,
                           static_cast<const int32_t *>(nullptr), offsets, order, pos);
    } else {
        hipLaunchKernelGGL(moe_count_kernel, dim3(groups), dim3(kSortThreads), 0, stream, ids, n, a.E, counts);
        if (sort == kCounted) {
            hipLaunchKernelGGL(moe_place_kernel<kCounted>, dim3(groups), dim3(kSortThreads), 0, stream, ids, n, a.E, bits,
                               counts, offsets, order, pos);
        } else {
            int width = 1;
            while (width < kScanWidth && width < a.E)
                width *= 2;
            hipLaunchKernelGGL(moe_scan_kernel, dim3((a.E + width - 1) / width), dim3(kScanThreads), 0, stream, counts, groups,
                               a.E, width);
            hipLaunchKernelGGL(moe_place_kernel<kScanned>, dim3(groups), dim3(kSortThreads), 0, stream, ids, n, a.E, bits,
                               counts, offsets, order, pos);
        }
    }
    if (X) {
        const int lg = waves_log2(a);
        const dim3 grid = row_grid(a, lg);
        const auto *x = static_cast<const u32x4 *>(X);
        auto *xs = static_cast<u32x4 *>(Xs);
        if (a.topk <= 2)
            hipLaunchKernelGGL(moe_gather_kernel<2>, grid, dim3(256), 0, stream, x, pos, xs, a.T, a.topk, a.vecs, lg, a.ldx16);
        else
            hipLaunchKernelGGL(moe_gather_kernel<8>, grid, dim3(256), 0, stream, x, pos, xs, a.T, a.topk, a.vecs, lg, a.ldx16);
    }
    return hipGetLastError();
}

namespace {

template <int DT, int J>
hipError_t combine_j(const MoeArgs &a, const void *Ys, const int32_t *pos, const float *w, void *Y, hipStream_t stream)
{
    const int lg = waves_log2(a);
    const dim3 grid = row_grid(a, lg);
    auto *y = static_cast<u32x4 *>(Y);
    auto *ys = static_cast<const u32x4 *>(Ys);
    if (w)
        hipLaunchKernelGGL((moe_combine_kernel<DT, true, J>), grid, dim3(256), 0, stream, ys, pos, w, y, a.T, a.topk, a.vecs, lg,
                           a.ldx16);
    else
        hipLaunchKernelGGL((moe_combine_kernel<DT, false, J>), grid, dim3(256), 0, stream, ys, pos, w, y, a.T, a.topk,
                           a.vecs, lg, a.ldx16);
    return hipGetLastError();
}

// choices loaded together: no more than a token has, up to eight
template <int DT>
hipError_t combine_dt(const MoeArgs &a, const void *Ys, const int32_t *pos, const float *w, void *Y, hipStream_t stream)
{
    return a.topk <= 2   ? combine_j<DT, 2>(a, Ys, pos, w, Y, stream)
           : a.topk <= 4 ? combine_j<DT, 4>(a, Ys, pos, w, Y, stream)
                         : combine_j<DT, 8>(a, Ys, pos, w, Y, stream);
}

template <int DT, int J>
hipError_t grad_j(const MoeArgs &a, const void *dY, const void *Ys, const int32_t *pos, const float *w, void *dYs,
                  float *dw, hipStream_t stream)
{
    hipLaunchKernelGGL((moe_combine_grad_kernel<DT, J>), dim3(a.T), dim3(256), 0, stream, static_cast<const u32x4 *>(dY),
                       static_cast<const u32x4 *>(Ys), pos, w, static_cast<u32x4 *>(dYs), dw, a.T, a.topk, a.vecs, a.ldx16);
    return hipGetLastError();
}

template <int DT>
hipError_t grad_dt(const MoeArgs &a, const void *dY, const void *Ys, const int32_t *pos, const float *w, void *dYs,
                   float *dw, hipStream_t stream)
{
    return a.topk <= 2   ? grad_j<DT, 2>(a, dY, Ys, pos, w, dYs, dw, stream)
           : a.topk <= 4 ? grad_j<DT, 4>(a, dY, Ys, pos, w, dYs, dw, stream)
                         : grad_j<DT, 8>(a, dY, Ys, pos, w, dYs, dw, stream);
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
