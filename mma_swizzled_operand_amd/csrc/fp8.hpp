// fp8.hpp — internal interface between the C ABI of the E4M3 operators with
// a scale per block of 128 (fp8_abi.hip) and their kernels (gemm_fp8*.hip,
// quant_fp8.hip).  Not installed.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mswz {

constexpr int kFp8Block = 128;   // values per scale

struct Fp8Args {
    const uint8_t *A;        // [M][lda] E4M3
    const float *SA;         // [kb][M]
    const uint8_t *B;        // [N][ldb] E4M3
    const float *SB;         // tile: [ceil(N/128)][kb], row: [kb][N]
    void *D;
    float *ws;               // partials of the split form
    int M, N, K, kb;         // kb: K blocks
    int64_t lda, ldb, ldd;
    int beta;
    int out;                 // OutKind
    bool tile;               // B's scales belong to 128 x 128 tiles
};

// floats from one row of a part's sums to the next
__host__ __device__ constexpr int64_t fp8_part_pitch(int64_t N) { return (N + 3) & ~int64_t(3); }

int64_t fp8_workspace_bytes(const Fp8Args &a);
hipError_t launch_fp8(const Fp8Args &a, hipStream_t stream);
hipError_t launch_fp8_skinny(const Fp8Args &a, hipStream_t stream);   // up to 32 rows of A

struct QuantArgs {
    const void *X;           // [M][ldx]
    uint8_t *Q;              // [M][K] or NULL
    float *S;
    uint8_t *QT;             // [K][Mp], Mp = M rounded up to 16, or NULL
    float *ST;
    int M, K;
    int64_t ldx;
    int dt;                  // OutKind
    bool tile, pow2;
};

hipError_t launch_quant_fp8(const QuantArgs &a, hipStream_t stream);

}  // namespace mswz
