// fp8_abi.hip — the C ABI declared in include/mswz_fp8.h: plan creation,
// argument checks and dispatch, in abi.hip's manner: everything the library
// cannot run is rejected with a status before any GPU work.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <new>

#include "../../include/mswz_fp8.h"
#include "fp8.hpp"
#include "kernels.hpp"

struct gemm_fp8_plan {
    mswz::Fp8Args a;
};
struct quant_fp8_plan {
    mswz::QuantArgs a;
};

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 20, kMaxLd = int64_t(1) << 22;
// (256 bytes short of 4 GiB, as in abi.hip: a masked access points at the end
// of the buffer's range, which must not wrap around)
constexpr int64_t kMaxBytes = (int64_t(1) << 32) - 256;

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool in_range(int64_t v) { return v > 0 && v <= kMaxDim; }
bool known_dt(int d) { return d >= MSWZ_DT_F16 && d <= MSWZ_DT_E2M1_P64; }
int64_t up(int64_t v, int64_t n) { return (v + n - 1) / n; }

// F32, BF16 or F16 as an OutKind, -1 for other formats
int value_kind(int dt)
{
    return dt == MSWZ_DT_F32 ? mswz::kOutF32 : dt == MSWZ_DT_BF16 ? mswz::kOutBf16 : dt == MSWZ_DT_F16 ? mswz::kOutF16 : -1;
}

int status(hipError_t e) { return e == hipSuccess ? MSWZ_OK : MSWZ_ERR_HIP; }

}  // namespace

extern "C" {

int gemm_fp8_plan_create(gemm_fp8_plan **out, int64_t M, int64_t N, int64_t K, int d_dt, int b_block, int64_t lda,
                         int64_t ldb, int64_t ldd)
{
    if (!out)
        return MSWZ_ERR_INVALID;
    *out = nullptr;
    if (!in_range(M) || !in_range(N) || !in_range(K) || !known_dt(d_dt) ||
        (b_block != MSWZ_FP8_ROW && b_block != MSWZ_FP8_TILE) || lda < 0 || ldb < 0 || ldd < 0 || (lda && lda < K) ||
        (ldb && ldb < K) || (ldd && ldd < N))
        return MSWZ_ERR_INVALID;
    const int64_t kb = up(K, mswz::kFp8Block);
    if (value_kind(d_dt) < 0 || K % 16 != 0 || lda % 16 != 0 || ldb % 16 != 0 || lda > kMaxLd || ldb > kMaxLd ||
        ldd > kMaxLd)
        return MSWZ_ERR_UNSUPPORTED;
    if (4 * kb * M >= kMaxBytes || 4 * kb * N >= kMaxBytes || up(M, 64) * up(N, 64) >= int64_t(1) << 22)
        return MSWZ_ERR_UNSUPPORTED;
    gemm_fp8_plan *p = new (std::nothrow) gemm_fp8_plan{};
    if (!p)
        return MSWZ_ERR_INVALID;
    mswz::Fp8Args &a = p->a;
    a.M = int(M);
    a.N = int(N);
    a.K = int(K);
    a.kb = int(kb);
    a.lda = lda ? lda : K;
    a.ldb = ldb ? ldb : K;
    a.ldd = ldd ? ldd : N;
    a.out = value_kind(d_dt);
    a.tile = b_block == MSWZ_FP8_TILE;
    *out = p;
    return MSWZ_OK;
}

void gemm_fp8_plan_destroy(gemm_fp8_plan *p) { delete p; }

int64_t gemm_fp8_plan_workspace_size(const gemm_fp8_plan *p)
{
    return p ? mswz::fp8_workspace_bytes(p->a) : int64_t(MSWZ_ERR_INVALID);
}

int gemm_run_fp8(const gemm_fp8_plan *p, const void *A, const float *SA, const void *B, const float *SB, void *D, int beta,
                 void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!p || !A || !SA || !B || !SB || !D || (beta != 0 && beta != 1))
        return MSWZ_ERR_INVALID;
    const int64_t need = mswz::fp8_workspace_bytes(p->a);
    if (need && (!workspace || workspace_bytes < need))
        return MSWZ_ERR_INVALID;
    if (!aligned(A, 16) || !aligned(B, 16) || !aligned(SA, 4) || !aligned(SB, 4) ||
        !aligned(D, p->a.out == mswz::kOutF32 ? 4 : 2) || (need && !aligned(workspace, 16)))
        return MSWZ_ERR_ALIGN;
    mswz::Fp8Args a = p->a;
    a.A = static_cast<const uint8_t *>(A);
    a.SA = SA;
    a.B = static_cast<const uint8_t *>(B);
    a.SB = SB;
    a.D = D;
    a.ws = need ? static_cast<float *>(workspace) : nullptr;
    a.beta = beta;
    return status(mswz::launch_fp8(a, static_cast<hipStream_t>(stream)));
}

int quant_fp8_plan_create(quant_fp8_plan **out, int64_t M, int64_t K, int dt, int block, int scales, int64_t ldx)
{
    if (!out)
        return MSWZ_ERR_INVALID;
    *out = nullptr;
    if (!in_range(M) || !in_range(K) || !known_dt(dt) || (block != MSWZ_FP8_ROW && block != MSWZ_FP8_TILE) ||
        (scales != MSWZ_SCALE_F32 && scales != MSWZ_SCALE_POW2) || ldx < 0 || (ldx && ldx < K))
        return MSWZ_ERR_INVALID;
    if (value_kind(dt) < 0 || K % 16 != 0 || ldx % 8 != 0 || ldx > kMaxLd ||
        up(M, 128) * up(K, 128) >= int64_t(1) << 23)
        return MSWZ_ERR_UNSUPPORTED;
    quant_fp8_plan *p = new (std::nothrow) quant_fp8_plan{};
    if (!p)
        return MSWZ_ERR_INVALID;
    p->a.M = int(M);
    p->a.K = int(K);
    p->a.ldx = ldx ? ldx : K;
    p->a.dt = value_kind(dt);
    p->a.tile = block == MSWZ_FP8_TILE;
    p->a.pow2 = scales == MSWZ_SCALE_POW2;
    *out = p;
    return MSWZ_OK;
}

void quant_fp8_plan_destroy(quant_fp8_plan *p) { delete p; }

int quant_fp8(const quant_fp8_plan *p, const void *X, void *Q, float *S, void *QT, float *ST, void *stream)
{
    if (!p || !X || (Q == nullptr) != (S == nullptr) || (QT == nullptr) != (ST == nullptr) || (!Q && !QT))
        return MSWZ_ERR_INVALID;
    if (!aligned(X, 16) || !aligned(Q, 16) || !aligned(S, 4) || !aligned(QT, 16) || !aligned(ST, 4))
        return MSWZ_ERR_ALIGN;
    mswz::QuantArgs a = p->a;
    a.X = X;
    a.Q = static_cast<uint8_t *>(Q);
    a.S = S;
    a.QT = static_cast<uint8_t *>(QT);
    a.ST = ST;
    return status(mswz::launch_quant_fp8(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
