// experts_abi.hip — the C ABI declared in include/mswz_experts.h: plan
// creation, argument checks and dispatch of the expert operators, in abi.hip's
// manner: everything the library cannot run is rejected with a status before
// any GPU work.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <new>

#include "../../include/mswz_experts.h"
#include "experts.hpp"
#include "kernels.hpp"

struct gemm_w4_plan {
    mswz::W4Args a;
};
struct gemm_grouped_plan {
    mswz::GroupedArgs a;
};
struct moe_plan {
    mswz::MoeArgs a;
};

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 20, kMaxLd = int64_t(1) << 22, kMaxExperts = 1024;
// (256 bytes short of 4 GiB, as in abi.hip: a masked access points at the
// end of the buffer's range, which must not wrap around)
constexpr int64_t kMaxBytes = (int64_t(1) << 32) - 256;

// row tiles are the launch's second dimension
constexpr int64_t kMaxW4Rows = int64_t(1) << 16;

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool in_range(int64_t v) { return v > 0 && v <= kMaxDim; }

bool known_dt(int d) { return d >= MSWZ_DT_F16 && d <= MSWZ_DT_U4; }
bool is16(int d) { return d == MSWZ_DT_F16 || d == MSWZ_DT_BF16; }

int out_kind(int d_dt)
{
    return d_dt == MSWZ_DT_BF16 ? mswz::kOutBf16 : d_dt == MSWZ_DT_F16 ? mswz::kOutF16 : mswz::kOutF32;
}

int status(hipError_t e) { return e == hipSuccess ? MSWZ_OK : MSWZ_ERR_HIP; }

}  // namespace

extern "C" {

int gemm_w4_plan_create(gemm_w4_plan **out, int64_t M, int64_t N, int64_t K, int64_t E, int a_dt, int w_dt, int d_dt,
                        int32_t group, int64_t lda, int64_t ldd)
{
    if (!out)
        return MSWZ_ERR_INVALID;
    *out = nullptr;
    if (!in_range(M) || !in_range(N) || !in_range(K) || E < 0 || !known_dt(a_dt) || !known_dt(w_dt) || !known_dt(d_dt) ||
        group <= 0)
        return MSWZ_ERR_INVALID;
    if (lda < 0 || ldd < 0 || (lda && lda < K) || (ldd && ldd < N))
        return MSWZ_ERR_INVALID;
    const bool e2m1 = w_dt == MSWZ_DT_E2M1;
    if (E > kMaxExperts || !is16(a_dt) || (w_dt != MSWZ_DT_U4 && !e2m1) || (d_dt != MSWZ_DT_F32 && d_dt != a_dt))
        return MSWZ_ERR_UNSUPPORTED;
    if (group != 32 && (e2m1 || (group != 64 && group % 128 != 0)))
        return MSWZ_ERR_UNSUPPORTED;
    // rows of B are whole 16-byte pieces, and so are rows of A
    if (M > kMaxW4Rows || K % 32 != 0 || lda % 8 != 0 || lda > kMaxLd || ldd > kMaxLd || N * (K / 2) >= kMaxBytes)
        return MSWZ_ERR_UNSUPPORTED;
    gemm_w4_plan *p = new (std::nothrow) gemm_w4_plan{};
    if (!p)
        return MSWZ_ERR_INVALID;
    mswz::W4Args &a = p->a;
    a.M = int(M);
    a.N = int(N);
    a.K = int(K);
    a.E = int(E);
    a.group = group;
    a.groups = int((K + group - 1) / group);
    a.lda = int(lda ? lda : K);
    a.ldd = int(ldd ? ldd : N);
    a.out = out_kind(d_dt);
    a.bf16 = a_dt == MSWZ_DT_BF16;
    a.e2m1 = e2m1;
    *out = p;
    return MSWZ_OK;
}

void gemm_w4_plan_destroy(gemm_w4_plan *p) { delete p; }

int64_t gemm_w4_plan_workspace_size(const gemm_w4_plan *p)
{
    return p ? mswz::w4_workspace_bytes(p->a) : int64_t(MSWZ_ERR_INVALID);
}

int gemm_run_w4(const gemm_w4_plan *p, const void *A, const void *B, const void *S, const uint8_t *Z,
                const int32_t *offsets, void *D, int beta, void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!p || !A || !B || !S || !D || (beta != 0 && beta != 1))
        return MSWZ_ERR_INVALID;
    if ((p->a.E > 0) != (offsets != nullptr) || (p->a.e2m1 && Z))
        return MSWZ_ERR_INVALID;
    const int64_t need = mswz::w4_workspace_bytes(p->a);
    if (need && (!workspace || workspace_bytes < need))
        return MSWZ_ERR_INVALID;
    if (!aligned(A, 16) || !aligned(B, 16) || !aligned(D, p->a.out == mswz::kOutF32 ? 4 : 2) ||
        !aligned(S, p->a.e2m1 ? 1 : 2) || !aligned(offsets, 4) || (need && !aligned(workspace, 16)))
        return MSWZ_ERR_ALIGN;
    mswz::W4Args a = p->a;
    a.A = A;
    a.B = static_cast<const uint8_t *>(B);
    a.S = S;
    a.Z = Z;
    a.offsets = offsets;
    a.D = D;
    a.ws = need ? static_cast<float *>(workspace) : nullptr;
    a.beta = beta;
    return status(mswz::launch_w4(a, static_cast<hipStream_t>(stream)));
}

int gemm_grouped_plan_create(gemm_grouped_plan **out, int64_t E, int64_t M, int64_t N, int64_t K, int dt, int d_dt,
                             int axis, int b_major)
{
    if (!out)
        return MSWZ_ERR_INVALID;
    *out = nullptr;
    if (!in_range(M) || !in_range(N) || !in_range(K) || E <= 0 || !known_dt(dt) || !known_dt(d_dt) ||
        (axis != MSWZ_GROUP_M && axis != MSWZ_GROUP_K) || (b_major != MSWZ_MAJOR_K && b_major != MSWZ_MAJOR_MN))
        return MSWZ_ERR_INVALID;
    const bool k_axis = axis == MSWZ_GROUP_K, b_mn = b_major == MSWZ_MAJOR_MN;
    if (E > kMaxExperts || !is16(dt) || (d_dt != MSWZ_DT_F32 && d_dt != dt) || (k_axis && !b_mn))
        return MSWZ_ERR_UNSUPPORTED;
    // 16-byte rows: K-major operands along K, MN-major ones along M or N, D along N
    if (N % 8 != 0 || (k_axis && M % 8 != 0) || (!k_axis && K % 8 != 0))
        return MSWZ_ERR_UNSUPPORTED;
    if ((b_mn && K * N * 2 >= kMaxBytes) || (k_axis && K * M * 2 >= kMaxBytes))
        return MSWZ_ERR_UNSUPPORTED;
    // a launch has fewer than 2^32 threads: 512 for each tile of 256 x 256 and
    // for at most 135 workgroups that find none
    const int64_t tiles_n = (N + 255) / 256, tiles_m = k_axis ? E * ((M + 255) / 256) : mswz::most_tiles(E, M, 256);
    if (tiles_m * tiles_n > (int64_t(1) << 23) - 256)
        return MSWZ_ERR_UNSUPPORTED;
    gemm_grouped_plan *p = new (std::nothrow) gemm_grouped_plan{};
    if (!p)
        return MSWZ_ERR_INVALID;
    p->a.E = int(E);
    p->a.M = int(M);
    p->a.N = int(N);
    p->a.K = int(K);
    p->a.out = out_kind(d_dt);
    p->a.bf16 = dt == MSWZ_DT_BF16;
    p->a.k_axis = k_axis;
    p->a.b_mn = b_mn;
    *out = p;
    return MSWZ_OK;
}

void gemm_grouped_plan_destroy(gemm_grouped_plan *p) { delete p; }

int gemm_run_grouped(const gemm_grouped_plan *p, const void *A, const void *B, const int32_t *offsets, void *D, int beta,
                     void *stream)
{
    if (!p || !A || !B || !offsets || !D || (beta != 0 && beta != 1))
        return MSWZ_ERR_INVALID;
    if (!aligned(A, 16) || !aligned(B, 16) || !aligned(D, 16) || !aligned(offsets, 4))
        return MSWZ_ERR_ALIGN;
    mswz::GroupedArgs a = p->a;
    a.A = A;
    a.B = B;
    a.offsets = offsets;
    a.D = D;
    a.beta = beta;
    return status(mswz::launch_grouped(a, static_cast<hipStream_t>(stream)));
}

int moe_plan_create(moe_plan **out, int64_t T, int64_t topk, int64_t E, int64_t H, int dt, int64_t ldx)
{
    if (!out)
        return MSWZ_ERR_INVALID;
    *out = nullptr;
    if (T <= 0 || topk <= 0 || E <= 0 || !in_range(H) || !known_dt(dt) || ldx < 0 || (ldx && ldx < H))
        return MSWZ_ERR_INVALID;
    constexpr int64_t kMaxChoices = int64_t(1) << 24;
    if (T >= kMaxChoices || topk >= kMaxChoices || T * topk >= kMaxChoices || E > kMaxExperts ||
        (!is16(dt) && dt != MSWZ_DT_F32))
        return MSWZ_ERR_UNSUPPORTED;
    const int64_t per16 = dt == MSWZ_DT_F32 ? 4 : 8;   // elements in 16 bytes
    if (H % per16 != 0 || ldx % per16 != 0 || ldx > kMaxLd)
        return MSWZ_ERR_UNSUPPORTED;
    moe_plan *p = new (std::nothrow) moe_plan{};
    if (!p)
        return MSWZ_ERR_INVALID;
    p->a.T = int(T);
    p->a.topk = int(topk);
    p->a.E = int(E);
    p->a.vecs = int(H / per16);
    p->a.ldx16 = (ldx ? ldx : H) / per16;
    p->a.dt = out_kind(dt);
    *out = p;
    return MSWZ_OK;
}

void moe_plan_destroy(moe_plan *p) { delete p; }

int64_t moe_plan_workspace_size(const moe_plan *p)
{
    return p ? mswz::moe_workspace_bytes(p->a) : int64_t(MSWZ_ERR_INVALID);
}

int moe_dispatch(const moe_plan *p, const int32_t *ids, const void *X, void *Xs, int32_t *offsets, int32_t *order,
                 int32_t *pos, void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!p || !ids || !offsets || !order || !pos || (X == nullptr) != (Xs == nullptr))
        return MSWZ_ERR_INVALID;
    const int64_t need = mswz::moe_workspace_bytes(p->a);
    if (need && (!workspace || workspace_bytes < need))
        return MSWZ_ERR_INVALID;
    if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(order, 4) || !aligned(pos, 4) || !aligned(X, 16) ||
        !aligned(Xs, 16) || (need && !aligned(workspace, 16)))
        return MSWZ_ERR_ALIGN;
    return status(mswz::launch_moe_dispatch(p->a, ids, X, Xs, offsets, order, pos, workspace,
                                            static_cast<hipStream_t>(stream)));
}

int moe_combine(const moe_plan *p, const void *Ys, const int32_t *pos, const float *w, void *Y, void *stream)
{
    if (!p || !Ys || !pos || !Y)
        return MSWZ_ERR_INVALID;
    if (!aligned(Ys, 16) || !aligned(pos, 4) || !aligned(w, 4) || !aligned(Y, 16))
        return MSWZ_ERR_ALIGN;
    return status(mswz::launch_moe_combine(p->a, Ys, pos, w, Y, static_cast<hipStream_t>(stream)));
}

int moe_combine_grad(const moe_plan *p, const void *dY, const void *Ys, const int32_t *pos, const float *w, void *dYs,
                     float *dw, void *stream)
{
    if (!p || !dY || !Ys || !pos || !w || !dYs || !dw)
        return MSWZ_ERR_INVALID;
    if (!aligned(dY, 16) || !aligned(Ys, 16) || !aligned(pos, 4) || !aligned(w, 4) || !aligned(dYs, 16) ||
        !aligned(dw, 4))
        return MSWZ_ERR_ALIGN;
    return status(mswz::launch_moe_combine_grad(p->a, dY, Ys, pos, w, dYs, dw, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace mswz {

hipError_t launch_grouped(const GroupedArgs &a, hipStream_t stream)
{
    if (a.k_axis)
        return a.bf16 ? launch_grouped_k_bf16(a, stream) : launch_grouped_k_f16(a, stream);
    return a.bf16 ? launch_grouped_m_bf16(a, stream) : launch_grouped_m_f16(a, stream);
}

}  // namespace mswz
