/*
 * mswz_moe_layer.h — C ABI of libmswz.so's whole gated layer of experts for a
 * few tokens (gfx950): what mswz_experts.h gives in parts for many.  Statuses
 * and dtypes are those of mswz_gemm.h, and so are the rules: the caller owns
 * every device buffer and the stream; a plan holds host metadata only, is
 * immutable and may be used from several host threads and streams at once; the
 * run call checks its arguments, enqueues its kernels on `stream` (which must
 * belong to the current device) and returns; it allocates nothing, does not
 * synchronise, keeps no pointer and can be captured into a graph; results are
 * bit-identical run to run.  Matrices are row-major, device memory; what the
 * call writes must not overlap what it reads.
 */
#ifndef MSWZ_MOE_LAYER_H
#define MSWZ_MOE_LAYER_H

#include <stdint.h>

#include "mswz_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The gate's activation in moe_layer_plan_create. */
enum {
    MSWZ_ACT_SILU = 0,          /* v / (1 + e^-v) */
    MSWZ_ACT_GELU = 1           /* v/2 (1 + tanh(sqrt(2/pi) (v + 0.044715 v^3))) */
};

typedef struct moe_layer_plan moe_layer_plan;

/*
 * Plan of a whole gated layer of experts for a few tokens (decoding):
 *
 *   Y[t] = sum_j w[t][j] W2[e] (act(W1[e][0:I] X[t]) * (W1[e][I:2I] X[t])),  e = ids[t][j]
 *
 *   T, topk, E  tokens, choices of each, experts (at most 1024); T * topk at
 *               most 1024
 *   H, I        elements of a token, and of an expert's inner row
 *   dt          MSWZ_DT_F16 or MSWZ_DT_BF16, of X and Y
 *   w_dt        of W1 and W2: dt, or MSWZ_DT_E4M3 with an fp32 scale for each
 *               128 x 128 tile of a matrix
 *   act         MSWZ_ACT_*
 *   ldx         elements from one token's row to the next (X and Y), 0 for H;
 *               a multiple of 8, at most 2^22
 * H and I are multiples of 8 (16 for E4M3); an expert's W1, T * topk * I * 4
 * bytes and X are below 4 GiB.
 * Storage: W1 [E][2I][H], the gate's rows first; W2 [E][H][I]; S1 [E][2]
 * [ceil(I/128)][ceil(H/128)], the gate's tiles and the other half's, counted
 * from the first row of each; S2 [E][ceil(H/128)][ceil(I/128)].  With I a
 * multiple of 128, S1 is quant_fp8's tile scales of the whole W1.
 * E4M3 weights have this call only: gemm_run_grouped takes 16-bit ones, so more
 * choices than it allows are a gemm_run_fp8 for each expert and matrix, with the
 * experts' row counts on the host.
 * Sums are fp32; between the two products a value keeps 16 significant bits
 * and fp32's range; Y is rounded once to nearest even.  A weight or value that
 * is not finite makes the outputs that it enters infinite or NaN.
 * Returns MSWZ_OK, MSWZ_ERR_INVALID or MSWZ_ERR_UNSUPPORTED.
 */
int moe_layer_plan_create(moe_layer_plan **out, int64_t T, int64_t topk, int64_t E, int64_t H,
                          int64_t I, int dt, int w_dt, int act, int64_t ldx);
void moe_layer_plan_destroy(moe_layer_plan *plan);

/* Device workspace moe_layer needs for this plan, in bytes. */
int64_t moe_layer_plan_workspace_size(const moe_layer_plan *plan);

/*
 * Enqueue the layer: two kernels for up to 16 choices, three for more.  ids
 * int32 [T][topk], a choice outside 0 .. E-1 is left out (a token without any
 * gives zeros); an expert may be chosen twice; w fp32 [T][topk].  S1 and S2 are
 * given exactly for E4M3 weights.  X, W1, W2, Y and workspace are 16-byte
 * aligned, the others 4-byte.  The workspace is the caller's, its contents
 * before the call do not matter, and calls that may overlap must not share it,
 * replays of two captured graphs among them.
 * Returns MSWZ_OK, MSWZ_ERR_INVALID, MSWZ_ERR_ALIGN or MSWZ_ERR_HIP.
 */
int moe_layer(const moe_layer_plan *plan, const void *X, const int32_t *ids, const float *w,
              const void *W1, const float *S1, const void *W2, const float *S2, void *Y,
              void *workspace, int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MSWZ_MOE_LAYER_H */
