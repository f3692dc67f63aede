// fp8_choice.hpp — which kernel a product of E4M3 operands takes, by sizes, type
// of D and pitches.  Host code without HIP calls, so that tests can ask for the
// choice too (tests/probes).
#pragma once
#include <stdint.h>

#include "fp8.hpp"
#include "kernels.hpp"

namespace mswz {

// In the order of fp8_tile's table from kFp8Tile32x64 on.
enum Fp8Kernel {
    kFp8Few,            // up to 32 rows of A, no barriers (gemm_fp8_skinny.hip)
    kFp8Split,          // tiles of 64 x 64, K split over workgroups
    kFp8Tile32x64,
    kFp8Tile64x64,
    kFp8Tile128x64,
    kFp8Tile128x128,
    kFp8Tile128x128Twice,   // two workgroups a compute unit
    kFp8Tile256x256
};

inline int64_t fp8_tiles(const Fp8Args &a, int bm, int bn) { return int64_t((a.M + bm - 1) / bm) * ((a.N + bn - 1) / bn); }

// Whether a few rows of A take the kernel without barriers
// (gemm_fp8_skinny.hip): up to 32, as long as there are few columns; with more, the
// tiles fetch whole lines.  us, without barriers and by tiles, 16-bit D: 2 rows of
// 4096 by 4096 columns 7.4 and 10.1, of 8192 by 4096 9.5 and 12.0, of 4096 by 6144
// 11.5 and 11.6, of 8192 by 12288 23.6 and 22.8; 16 rows 8.0 and 10.2, 11.7 and
// 12.3, 12.8 and 11.9, 34.7 and 23.9; 32 rows 9.4 and 10.3, 16.7 and 13.1 (tiles
// with K split), 18.6 and 12.5, 43 and 26.  K 2048: within 10 %.  An fp32 D's tiles
// have two to four times the work at a step: 8 rows of 8192 by 8192 18.2 and 21.5,
// by 16384 36 and 26; 16 rows of 4096 by 8192 12.9 and 13.8, of 8192 by 5120 20.3
// and 18.3.
inline bool fp8_is_few(const Fp8Args &a)
{
    if (a.M <= 16)
        return fp8_tiles(a, 64, 64) <= (a.out == kOutF32 ? 128 : 64);
    return a.M <= 32 && fp8_tiles(a, 64, 64) <= 64 && a.kb < 48;
}

// K parts of a product: where tiles of 64 x 64 leave half of the compute units
// idle and K is long, it is split until there are as many, each part keeping
// eight blocks at least (four and twelve: within 3 %).  Unsplit, with tiles of 32
// x 64, and split: 64 x 2048 x 8192 16.6 and 12.2 us, 512 x 512 x 8192 16.4 and
// 13.4, 128 x 4096 x 8192 19.7 and 18.8; 64 x 4096 x 4096 10.2 and 11.8, 100 x 1000
// x 4096 9.8 and 10.9: with few blocks the second launch takes what the split
// gives.
inline int fp8_parts(const Fp8Args &a)
{
    const int64_t t = fp8_tiles(a, 64, 64);
    if (fp8_is_few(a) || t > 128 || a.kb < 48)
        return 1;
    const int64_t most = a.kb / 8;
    return int(256 / t < most ? 256 / t : most);
}

// The tile whose rounds over the chip take the least time.  A round takes
// `start` and `step` for each block of K, `uneven` more where rows are not whole
// lines of 128 bytes (a copied row then costs two), in units of 10 ns, fitted to
// the times below; the compute units hold one workgroup each but for the second
// form of 128 x 128, of which they hold two.  us in the order of the table, tile
// scales, bf16 D: 64 x 4096 x 4096 9.7, 12.6, 14.3, 18.3, 24.8, 44.2; 256 x 4096 x
// 4096 17.1, 13.0, 15.4, 19.0, 25.7, 46.7; 512 x 4096 x 4096 28.7, 21.3, 17.7, 22.3,
// 31.3, 49.5; 1024 x 4096 x 4096 51.0, 36.6, 32.8, 23.3, 31.6, 50.0; 2048 x 4096 x
// 4096 95, 66, 60, 43.6, 39.2, 51.3; 2048 x 4096 x 1024 35.2, 21.0, 20.7, 14.9,
// 11.7, 17.3; 4096 x 4096 x 4096 186, 129, 116, 85, 76, 61; 5432 x 3696 x 1712 -, 86,
// 86, 73, 61, 60.  The largest does not leave the bf16 form registers, so an fp32
// D stops at 128 x 128 (4096 x 4096 x 4096 128 us, 238 with it).
// Waves of 64 columns store whole lines (waves of 32 rows by 64 columns and of 64
// by 32 in the first form of 128 x 128: 1024 x 4096 x 4096 23.3 and 26.5 us).  In
// the second form eight waves of 32 x 64 hide more than four of 64 x 64, if both
// workgroups' registers fit (2048 x 4096 x 4096 39.1 and 41.0 us; row scales 63.6
// and 50.0, fp32 D 79.8 and 71.6).
inline Fp8Kernel fp8_tile(const Fp8Args &a)
{
    const bool f32 = a.out == kOutF32;
    const struct {
        int64_t tiles, slots, step, uneven, start;
    } all[6] = {{fp8_tiles(a, 32, 64), 256, f32 ? 24 : 16, 4, 40},
                {fp8_tiles(a, 64, 64), 256, f32 ? 39 : 25, 6, 30},
                {fp8_tiles(a, 128, 64), 256, f32 ? 77 : 41, 10, 140},
                {fp8_tiles(a, 128, 128), 256, f32 ? 119 : 64, 16, 130},
                {fp8_tiles(a, 128, 128), 512, f32 ? 205 : 115, 17, 150},
                {fp8_tiles(a, 256, 256), 256, 165, 12, 400}};
    const bool uneven = a.lda % 128 != 0 || a.ldb % 128 != 0;
    int best = 0;
    int64_t least = INT64_MAX;
    for (int i = 0; i < (f32 ? 5 : 6); ++i) {
        const int64_t time = (all[i].tiles + all[i].slots - 1) / all[i].slots *
                             ((all[i].step + (uneven ? all[i].uneven : 0)) * a.kb + all[i].start);
        if (time <= least) {
            least = time;
            best = i;
        }
    }
    return Fp8Kernel(kFp8Tile32x64 + best);
}

inline Fp8Kernel fp8_kernel(const Fp8Args &a)
{
    return fp8_is_few(a) ? kFp8Few : fp8_parts(a) > 1 ? kFp8Split : fp8_tile(a);
}

}  // namespace mswz
