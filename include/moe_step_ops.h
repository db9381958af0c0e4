/*
 * moe_step_ops.h -- operators for what surrounds a layer's products in a
 * training step, and for the weights that the step leaves:
 *
 *   moe_balance, moe_balance_bwd: the router's balance loss and z loss with
 *     the experts' counts, and the gradient of the router's logits;
 *   moe_orthogonalize: an update (a weight gradient or its momentum)
 *     orthogonalised by Newton-Schulz products, for a stack of matrices;
 *   moe_mxfp4_quant_weights, moe_mxfp4_mm: weights in OCP MXFP4 (4 bits, a
 *     scale per 32) and products of bf16 rows with them, grouped or dense.
 *
 * The conventions of moe.h and moe_ops.h hold: device pointers owned by the
 * caller, no allocation, no host synchronisation, stream-ordered calls that can
 * be captured into a graph, arguments checked on the host before anything is
 * launched, results bit-identical from run to run.  The current device must be
 * the one the buffers and the stream belong to.  Calls share no state: two calls
 * may overlap when neither writes what the other one uses (a workspace is
 * written by its call).  An output overlaps no input of its call.
 */
#ifndef MOE_STEP_OPS_H
#define MOE_STEP_OPS_H

#include "moe_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* kernel ids reported in moe_profile.kernel, after those of moe_ops.h */
#define MOE_STEP_K_BALANCE       41
#define MOE_STEP_K_BALANCE_BWD   42
#define MOE_STEP_K_ORTHOGONALIZE 43
#define MOE_STEP_K_MXFP4_WEIGHTS 44
#define MOE_STEP_K_MXFP4_MM      45

/*
 * Balance loss and z loss of a router.  logits z [T,E] (dtype MOE_F32 or
 * MOE_BF16), expert_idx [T,K] int32 the experts chosen, valid [T] bytes or NULL
 * (all valid).  A token counts when it is valid and one of its logits is above
 * -inf (masked experts have logits of -inf, and any value in a token that does
 * not count is without effect).  With n counting tokens, p_t = softmax(z_t):
 *     counts[e]  choices of expert e by counting tokens (an id outside 0..E-1
 *                is no choice; an expert chosen twice by a token counts twice)
 *     tokens[0]  n
 *     load[e]    (1/n) sum_t p_te
 *     lse[t]     log sum_e exp z_te, -inf for a token that does not count
 *     loss[0]    E / (n K) sum_e counts[e] load[e]     (1 when balanced)
 *     loss[1]    (1/n) sum_t lse_t^2
 * All zeros (lse -inf) for n = 0.  Sums run in fp32 or wider.
 *   0 <= T < 2^24, 1 <= K <= 1024, 1 <= E <= 1024, T * K <= 2^30.
 */
typedef struct moe_balance_desc {
    int32_t  T, E, K;
    int32_t  dtype;         /* of the logits and their gradient */
    uint32_t flags;         /* must be 0 */
    uint32_t reserved;      /* must be 0 */
    moe_profile* profile;   /* NULL, or launch timing (see moe.h) */
} moe_balance_desc;

/* Workspace of moe_balance in bytes; 0 for an invalid descriptor.  Host only. */
size_t moe_balance_workspace_bytes(const moe_balance_desc* desc);

int moe_balance(const moe_balance_desc* desc, const void* logits, const int32_t* expert_idx, const uint8_t* valid,
                int32_t* counts, int32_t* tokens, float* load, float* lse, float* loss, void* ws, size_t ws_bytes,
                void* stream);

/*
 * Gradient of the logits.  counts, tokens, lse: of moe_balance on the same
 * logits; d_loss [2] fp32 on the device, the gradients of the two losses (their
 * weights in the total loss):
 *     dz[t,e] = p_te ( d_loss[0] E / (n^2 K) (counts[e] - sum_j counts[j] p_tj)
 *                      + d_loss[1] 2/n lse_t )             (0 for a token that does not count)
 * and, when gate and d_gate [T,K] fp32 are given, the gradient of gates that
 * are a softmax over the token's chosen logits (moe_route's):
 *     dz[t, expert_idx[t,k]] += gate[t,k] (d_gate[t,k] - sum_j gate[t,j] d_gate[t,j])
 * for the choices inside 0..E-1, of every token (what a dropped choice holds is
 * without effect).  expert_idx, gate and d_gate: all three or none.  dz [T,E] in
 * the logits' type, rounded once.
 */
int moe_balance_bwd(const moe_balance_desc* desc, const void* logits, const int32_t* counts, const int32_t* tokens,
                    const float* lse, const float* d_loss, const int32_t* expert_idx, const float* gate,
                    const float* d_gate, void* dz, void* stream);

/*
 * Orthogonalised update.  For each matrix G of g [E,M,N] (dtype MOE_F32 or
 * MOE_BF16, dense), with X_0 = G / (|G| + eps), |G| the Frobenius norm, and A = X X^T
 * (X transposed first where M > N):
 *     X <- coef[3i] X + coef[3i+1] A X + coef[3i+2] A^2 X      for the steps i in turn
 *     o = scale * X                                            (o as g, rounded once)
 * coef [steps][3] is a host array, read before the call returns.  With (3.4445,
 * -4.7750, 2.0315) in five steps the singular values of X come to lie within about 0.7 ..
 * 1.2, those of a matrix of zeros stay zeros.  A matrix that holds a NaN or an infinity gives NaNs,
 * and changes no other one.  Any M and N, any finite G (the norm is taken in 64 bits).
 *   Precision.  With fp32 matrices every product is taken to about 2^-22 of its
 * factors and summed in fp32, as fp32 products are: results are as far from the
 * definition as those of fp32 products step by step (1.3e-6 to 3.2e-6 of the result's norm
 * for the coefficients above and sides of thousands, up to 2.6e-5 where one direction is far above all others, and
 * fp32 products 4e-5 there; sums over millions may add as much again).  With bf16 matrices
 * several steps share one product with X, as many as are expected to add at most 1.5e-3 of the result's norm to its
 * rounding's 1.7e-3 when one direction is far above all others: measured 2e-4 to 5e-4 then for 100 rows (of the
 * smaller side, rows of zeros not counted) or more, up to 1.2e-3 for two, and 2e-4 or less for singular values that
 * fall like 1/i.  The
 * polynomials' values on singular values 0 .. 1 have to stay below 2^40; a step sequence that
 * grows past that gives results that are not finite.
 *   Limits: 1 <= E <= 1024, 1 <= steps <= 64, min(M, N) <= 16384, a padded matrix
 * (M and N rounded up to 64) below 2^29 elements (MOE_ESHAPE); coef, eps and scale
 * finite, eps >= 0 (MOE_EINVAL).  g and o aligned to their element.
 *   Workspace: moe_orthogonalize_workspace_bytes, 256-byte aligned, not shared with
 * a call that may overlap.  (It covers as many matrices at a time as fill the card.)
 */
typedef struct moe_ortho_desc {
    int32_t  E, M, N;
    int32_t  dtype;
    int32_t  steps;
    float    eps, scale;
    uint32_t flags;         /* must be 0 */
    uint32_t reserved;      /* must be 0 */
    const float* coef;      /* host, [steps][3] */
    moe_profile* profile;   /* NULL, or launch timing (see moe.h) */
} moe_ortho_desc;

size_t moe_orthogonalize_workspace_bytes(const moe_ortho_desc* desc);
int moe_orthogonalize(const moe_ortho_desc* desc, const void* g, void* o, void* ws, size_t ws_bytes, void* stream);

/*
 * Weights in OCP MXFP4.  32 values along the reduction share an E8M0 scale code,
 * 2^(code - 127) (255: NaN, and every product with the block is NaN); a value is an
 * E2M1 code times it: 0, 0.5, 1, 1.5, 2, 3, 4, 6 for codes 0..7, their negatives for
 * 8..15.  A byte holds two codes, the lower index in its lower half.
 *   moe_mxfp4_quant_weights  w [E,K,N] (dtype MOE_F32 or MOE_BF16, 16-byte aligned)
 *       -> q [E,N,K/2] bytes, s [E,N,K/32] bytes: the reduction contiguous.  Scale
 *       exponent floor(log2(largest magnitude)) - 2, at least -127; values to nearest, ties
 *       to the even code, at most 6; a block with a NaN or an infinity gets code 255.
 *       K a multiple of 32, N of 16, each at most 2^20, 1 <= E <= 1024.
 */
int moe_mxfp4_quant_weights(int dtype, int E, int K, int N, const void* w, void* q, void* s, moe_profile* profile,
                            void* stream);

/*
 * Product of bf16 rows with MXFP4 weights:  c[r,j] = sum_i a[r,i] w[e,j,i] for the rows r of expert
 * e's segment, w the values of q and s.  desc (moe_mm_desc) and plan as in moe_fp8_mm:
 * a [a_rows, K] bf16; rows = the plan's capacity, a_rows = rows or with MOE_MM_GATHER T
 * (row r reads a's row row_token[r]; a token outside 0..a_rows-1 counts as zeros); plan
 * NULL: dense, E = 1.  c [rows, N] in desc->out, rounded once; rows of no segment are left as they were.
 *   Precision: every product is exact and sums run in fp32 (a value past the largest bf16
 * number, which scale codes 253 and 254 allow, counts as an infinity).  Calls of few rows
 * per expert add up in another order, so a row's result may depend, within fp32's rounding,
 * on the sizes of the call.  The same call gives the same bits.
 *   Limits: K a multiple of 32, N of 16, each at most 2^20, E <= 1024, N * K below 2^31, with
 * MOE_MM_GATHER a_rows * K below 2^30 (MOE_ESHAPE; larger ones go through moe_permute),
 * (ceil(rows / 128) + E) ceil(N / 256) below 2^24 - 8 (rows_used in place of rows where given).
 * a, q and c 16-byte aligned.
 */
int moe_mxfp4_mm(const moe_mm_desc* desc, const void* a, const void* q, const void* s, const moe_plan* plan, void* c,
                 void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_STEP_OPS_H */
