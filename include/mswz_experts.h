/*
 * mswz_experts.h — C ABI of libmswz.so's products with 4-bit weights, of its
 * products over rows grouped by expert, and of the token movement around them
 * (gfx950).  Statuses, dtypes and majors are those of mswz_gemm.h, and so are
 * the rules: the caller owns every device buffer and the stream; a plan holds
 * host metadata only, is immutable and may be used from several host threads
 * and streams at once; a run call checks its arguments, enqueues its kernels
 * on `stream` (which must belong to the current device) and returns; it
 * allocates nothing, does not synchronise, keeps no pointer and can be
 * captured into a graph; results are bit-identical run to run.  Matrices are
 * row-major, device memory; what a call writes must not overlap what it reads
 * or writes elsewhere (D itself is read where beta is 1).
 *
 * A layer of experts is moe_dispatch (tokens to sorted rows), products over
 * the sorted rows (gemm_run_grouped, or gemm_run_w4 with 4-bit weights) and
 * moe_combine (rows back to tokens); training adds gemm_run_grouped's two
 * gradient forms, moe_combine_grad, and moe_combine without weights, which is
 * moe_dispatch's gradient.
 *
 * Sorted rows.  `offsets`, int32 [E+1] in device memory, bounds the groups:
 * rows offsets[e] .. offsets[e+1] - 1 belong to expert e.  Row counts are
 * known on the device only; the plan's M is the capacity.  Bounds are clamped
 * to 0 .. M (K for MSWZ_GROUP_K) and a group whose bounds descend is empty, so
 * no value of them reads or writes outside the buffers; what groups that
 * overlap leave in D is not defined.  Rows outside every group are neither read
 * nor written.
 */
#ifndef MSWZ_EXPERTS_H
#define MSWZ_EXPERTS_H

#include <stdint.h>

#include "mswz_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Weight formats of gemm_w4_plan_create (MSWZ_DT_E2M1 is the other one). */
enum {
    MSWZ_DT_U4 = 9              /* unsigned 4-bit integers, two per byte, element 2j in the low nibble of byte j */
};

typedef struct gemm_w4_plan gemm_w4_plan;
typedef struct gemm_grouped_plan gemm_grouped_plan;
typedef struct moe_plan moe_plan;

/*
 * Plan of a product with 4-bit weights and 16-bit activations:
 *
 *   D[m][n] = beta*D[m][n] + sum_g s[e][n][g] * sum_{k in group g} A[m][k] (w[e][n][k] - z[e][n][g])
 *
 *   M, N, K   rows of A and D, columns of D, inner size; M at most 65536,
 *             K % 32 == 0, N * K / 2 below 4 GiB
 *   E         0: one weight matrix for all rows; > 0 (at most 1024): one per
 *             expert, rows sorted by expert
 *   a_dt      MSWZ_DT_F16 or MSWZ_DT_BF16
 *   w_dt      MSWZ_DT_U4: w = 0..15, s in a_dt, z uint8 or absent (then 8);
 *             MSWZ_DT_E2M1: w the FP4 value, s = 2^(byte - 127) (OCP E8M0, 255
 *             is NaN), no z
 *   d_dt      MSWZ_DT_F32, or a_dt (the fp32 result rounded to nearest even)
 *   group     K elements per scale: 32, 64 or a multiple of 128 (E2M1: 32);
 *             the last group may be shorter, ceil(K / group) scales per row
 *   lda, ldd  elements from one row of A (D) to the next, 0 for K (N);
 *             lda % 8 == 0, both at most 2^22
 * Storage: A [M][K]; B uint8 [E][N][K/2] (two elements a byte); S and Z
 * [E][N][ceil(K/group)]; without experts one matrix, E = 1 in these shapes.
 * The 4-bit integers, z and the products enter exactly; sums are fp32.  A
 * scale multiplies the fp32 sums of a group's runs of 128 values (of a shorter
 * group's values); with bf16 A and E2M1 weights it multiplies the weights,
 * exactly.  So an infinite scale of a long group gives NaN if its runs' sums
 * differ in sign or one is zero.  With bf16 A and U4 weights a run's sum is
 * that of A w less z times that of A: a row of A holding an infinity, or values
 * whose sums leave fp32's range, gives NaN.
 * Returns MSWZ_OK, MSWZ_ERR_INVALID or MSWZ_ERR_UNSUPPORTED.
 */
int gemm_w4_plan_create(gemm_w4_plan **out, int64_t M, int64_t N, int64_t K, int64_t E, int a_dt,
                        int w_dt, int d_dt, int32_t group, int64_t lda, int64_t ldd);
void gemm_w4_plan_destroy(gemm_w4_plan *plan);

/* Device workspace gemm_run_w4 needs for this plan, in bytes (0: none). */
int64_t gemm_w4_plan_workspace_size(const gemm_w4_plan *plan);

/*
 * Enqueue the product.  A, B and workspace are 16-byte aligned, S and D
 * aligned to their elements (the whole 4-byte words that hold their first and
 * last bytes are read); Z may be NULL (U4) and is NULL for E2M1; offsets is
 * NULL exactly for a plan without experts; beta is 0 or 1.  The workspace (NULL
 * where none is needed) is the caller's, its contents before the call do not
 * matter, and calls that may overlap must not share it, replays of two captured
 * graphs among them.
 * Returns MSWZ_OK, MSWZ_ERR_INVALID, MSWZ_ERR_ALIGN or MSWZ_ERR_HIP.
 */
int gemm_run_w4(const gemm_w4_plan *plan, const void *A, const void *B, const void *S,
                const uint8_t *Z, const int32_t *offsets, void *D, int beta, void *workspace,
                int64_t workspace_bytes, void *stream);

/* What a group spans in gemm_grouped_plan_create. */
enum { MSWZ_GROUP_M = 0, MSWZ_GROUP_K = 1 };

/*
 * Plan of a product over E groups of rows (E at most 1024).
 *   MSWZ_GROUP_M  D[p] = beta*D[p] + A[p] . B[e]^T for the rows p of expert e:
 *                 A [M][K] K-major, B K-major [E][N][K] or MN-major [E][K][N],
 *                 D [M][N]; M is the capacity.  With an MN-major B this is the
 *                 row gradient of the K-major product.
 *   MSWZ_GROUP_K  D[e] = beta*D[e] + sum_p A[p]^T B[p] over the rows p of
 *                 expert e: A [K][M], B [K][N] (both MN-major), D [E][M][N]; K
 *                 is the capacity.  The weight gradient.  An expert without
 *                 rows gets beta*D.
 *   dt    MSWZ_DT_F16 or MSWZ_DT_BF16, of A and B
 *   d_dt  MSWZ_DT_F32 or dt
 * Rows are 16-byte aligned: K % 8 == 0 for K-major operands, N % 8 == 0, and
 * M % 8 == 0 for MSWZ_GROUP_K; an operand's [K][N] or [K][M] matrix is below
 * 4 GiB, and D has fewer than 2^23 - 256 tiles of 256 x 256, counted for
 * MSWZ_GROUP_M as if every expert's last tile were partly filled.
 * Returns MSWZ_OK, MSWZ_ERR_INVALID or MSWZ_ERR_UNSUPPORTED.
 */
int gemm_grouped_plan_create(gemm_grouped_plan **out, int64_t E, int64_t M, int64_t N, int64_t K,
                             int dt, int d_dt, int axis, int b_major);
void gemm_grouped_plan_destroy(gemm_grouped_plan *plan);

/*
 * Enqueue the grouped product.  A, B and D are 16-byte aligned, offsets 4-byte;
 * beta is 0 or 1.
 * Returns MSWZ_OK, MSWZ_ERR_INVALID, MSWZ_ERR_ALIGN or MSWZ_ERR_HIP.
 */
int gemm_run_grouped(const gemm_grouped_plan *plan, const void *A, const void *B,
                     const int32_t *offsets, void *D, int beta, void *stream);

/*
 * Plan of the token movement: T tokens of H elements, `topk` expert choices
 * each, E experts (at most 1024).  The product T * topk is below 2^24.
 *   dt    MSWZ_DT_F16, MSWZ_DT_BF16 or MSWZ_DT_F32, of the rows; rows are whole
 *         16-byte pieces (H % 8 == 0, H % 4 == 0 for F32), H at most 2^20
 *   ldx   elements from one token's row to the next (X, Y and dY), 0 for H;
 *         a multiple of 8 (4 for F32), at most 2^22.  Sorted rows are packed.
 * Returns MSWZ_OK, MSWZ_ERR_INVALID or MSWZ_ERR_UNSUPPORTED.
 */
int moe_plan_create(moe_plan **out, int64_t T, int64_t topk, int64_t E, int64_t H, int dt,
                    int64_t ldx);
void moe_plan_destroy(moe_plan *plan);

/* Device workspace moe_dispatch needs for this plan, in bytes (0: none). */
int64_t moe_plan_workspace_size(const moe_plan *plan);

/*
 * Sort the tokens' choices by expert and copy the tokens' rows in that order.
 *   ids      int32 [T][topk]; a choice outside 0 .. E-1 is left out
 *   offsets  int32 [E+1], written: the groups' bounds (offsets[0] = 0)
 *   order    int32 [T*topk], written: t*topk + j of each sorted row, in
 *            ascending order inside a group; -1 behind the last group
 *   pos      int32 [T][topk], written: the sorted row of choice j of token t,
 *            -1 if it is left out
 *   X, Xs    [T][H] and [T*topk][H]: Xs[pos[t][j]] = X[t]; rows behind the last
 *            group are left as they were.  Both NULL: the sort alone.
 * Integers are 4-byte aligned, rows and workspace 16-byte.  The workspace
 * rules are gemm_run_w4's.
 * Returns MSWZ_OK, MSWZ_ERR_INVALID, MSWZ_ERR_ALIGN or MSWZ_ERR_HIP.
 */
int moe_dispatch(const moe_plan *plan, const int32_t *ids, const void *X, void *Xs,
                 int32_t *offsets, int32_t *order, int32_t *pos, void *workspace,
                 int64_t workspace_bytes, void *stream);

/*
 * Y[t] = sum_j w[t][j] Ys[pos[t][j]], summed in fp32 in the order of j and
 * rounded once; a choice whose pos is outside 0 .. T*topk-1 adds nothing (its
 * weight is not read into the sum).  w fp32 [T][topk], or NULL for ones: the
 * gradient of moe_dispatch (dX from dXs).  Statuses as moe_dispatch.
 */
int moe_combine(const moe_plan *plan, const void *Ys, const int32_t *pos, const float *w, void *Y,
                void *stream);

/*
 * The gradients of moe_combine with weights:
 *   dYs[pos[t][j]] = w[t][j] dY[t]      (rows that no pos names are left as they were)
 *   dw[t][j] = sum_h dY[t][h] Ys[pos[t][j]][h]   (fp32; 0 for a choice left out)
 * Two choices must not share a row (moe_dispatch gives each its own).
 * Statuses as moe_dispatch.
 */
int moe_combine_grad(const moe_plan *plan, const void *dY, const void *Ys, const int32_t *pos,
                     const float *w, void *dYs, float *dw, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MSWZ_EXPERTS_H */
