/*
 * moe_ops.h -- the operators around the experts' products, one by one, for
 * callers whose router, experts or precision differ from the layer of moe.h:
 *
 *   moe_sort, moe_permute, moe_unpermute and their gradients: tokens sorted by
 *     expert and back, from any expert choice, with the weights applied;
 *   moe_fp8_mm, moe_fp8_wgrad and the quantizers: matrix products of E4M3
 *     operands with a scale for each block of 128, grouped by expert or dense;
 *   moe_swiglu_fp8, moe_swiglu_bwd: the activation between the two products,
 *     quantized for the second one, and its gradient.
 *
 * The conventions of moe.h hold: device pointers owned by the caller, no
 * allocation, no host synchronisation, stream-ordered calls that can be
 * captured into a graph, arguments checked on the host before anything is
 * launched, the status codes and element types of moe.h, results bit-identical
 * from run to run.  The current device must be the one the buffers and the
 * stream belong to.  Calls share no state: two calls may overlap when neither
 * writes what the other one uses.  An output overlaps no input of its call.
 *
 * E4M3 blocks.  Codes are OCP FP8 E4M3 bytes (largest value 448, no infinity).
 * A block of 128 values has one fp32 scale
 *     s = max(amax / 448, 2^-126),    code = E4M3(x * (1 / s)),
 * with s, 1 / s and the product rounded to fp32 and the code to nearest, ties
 * to even; the value it stands for is code * s.  A block that holds a NaN or
 * an infinity gets a NaN scale, so every product with it is NaN.  Where 128
 * does not divide a length, the last block is shorter.
 */
#ifndef MOE_OPS_H
#define MOE_OPS_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* kernel ids reported in moe_profile.kernel, after those of moe.h */
#define MOE_OPS_K_SORT          29  /* expert choices -> plan                      */
#define MOE_OPS_K_PERMUTE       30  /* token rows to the plan's rows               */
#define MOE_OPS_K_PERMUTE_FP8   31  /* the same, quantized on the way              */
#define MOE_OPS_K_UNPERMUTE     32  /* weighted sum of a token's rows              */
#define MOE_OPS_K_UNPERMUTE_BWD 33  /* its row and weight gradients                */
#define MOE_OPS_K_QUANT_ROWS    34  /* 1 x 128 blocks along the rows               */
#define MOE_OPS_K_QUANT_WEIGHTS 35  /* 128 x 128 blocks, both layouts              */
#define MOE_OPS_K_QUANT_COLS    36  /* 128 x 1 blocks along a segment              */
#define MOE_OPS_K_FP8_MM        37  /* product of rows with their expert's weights */
#define MOE_OPS_K_FP8_WGRAD     38  /* product over a segment's rows               */
#define MOE_OPS_K_SWIGLU_FP8    39
#define MOE_OPS_K_SWIGLU_BWD    40

/*
 * Plan: which rows belong to which expert.
 *   T, K, E: tokens, choices per token, experts.  0 <= T < 2^24,
 *     1 <= K <= 1024, T*K <= 2^30, 1 <= E <= 1024; K may exceed E and a token
 *     may choose an expert twice.
 *   align: every expert's segment starts at a multiple of it, 1..256
 *     (moe_fp8_quant_cols and moe_fp8_wgrad need a multiple of 128).
 */
typedef struct moe_plan_desc {
    int32_t  T, K, E, align;
    uint32_t flags;         /* must be 0 */
    uint32_t reserved;      /* must be 0 */
    moe_profile* profile;   /* NULL, or launch timing (see moe.h) */
} moe_plan_desc;

/*
 * Device buffers of a plan, written by moe_sort; cap = moe_plan_rows(desc).
 *   offsets   [E+1] first row of each segment; offsets[E] ends the last one
 *   counts    [E]   rows of each segment: offsets[e] .. offsets[e]+counts[e]-1
 *   row_token [cap] token of each row; -1 for the rows between a segment's
 *                   last row and the next segment; from offsets[E] on as it was
 *   slot_row  [T*K] row of each choice, -1 when it was dropped
 */
typedef struct moe_plan {
    int32_t* offsets;
    int32_t* counts;
    int32_t* row_token;
    int32_t* slot_row;
} moe_plan;

/* Rows a plan can have: T*K + min(E, T*K) * (align - 1).  0 for an invalid
 * descriptor (and for T = 0).  Host only. */
size_t moe_plan_rows(const moe_plan_desc* desc);

/* Workspace of moe_sort in bytes; 0 for an invalid descriptor.  Host only. */
size_t moe_sort_workspace_bytes(const moe_plan_desc* desc);

/*
 * Sorts the T*K choices by expert, those of one expert in ascending slot
 * number t*K + k.  expert_idx [T*K] int32; an id outside 0..E-1 drops its
 * choice.  ws: 256-byte aligned, not shared with a call that may overlap.
 */
int moe_sort(const moe_plan_desc* desc, const int32_t* expert_idx, const moe_plan* plan, void* ws,
             size_t ws_bytes, void* stream);

/*
 * Rows to their experts and back.  dtype MOE_F32 or MOE_BF16; d a multiple of
 * 16; matrices dense and 16-byte aligned (else MOE_EINVAL).  Rows of xp, q, s
 * and dy that belong to no choice are left as they were.
 *   moe_permute        xp[slot_row[t,k]] = x[t]               x [T,d], xp [cap,d]
 *   moe_permute_fp8    the same rows as codes q [cap,d] and scales
 *                      s [cap, ceil(d/128)], blocks along d
 *   moe_permute_bwd    dx[t] = sum_k dxp[slot_row[t,k]]       dxp [cap,d], dx [T,d]
 *   moe_unpermute      o[t] = sum_k w[t,k] y[slot_row[t,k]]   y [cap,d], w [T,K]
 *                      fp32, o [T,d]
 *   moe_unpermute_bwd  dy[slot_row[t,k]] = w[t,k] d_o[t],
 *                      dw[t,k] = <d_o[t], y[slot_row[t,k]]>   dw [T,K] fp32
 * Sums run in fp32 over ascending k; dropped choices add nothing (whatever
 * their weight holds), their dw is 0, and a token without choices gets zeros.
 * dw may be NULL, and then y too; dy may be NULL, and then w too.
 */
int moe_permute(const moe_plan_desc* desc, const moe_plan* plan, int dtype, int d, const void* x, void* xp,
                void* stream);
int moe_permute_fp8(const moe_plan_desc* desc, const moe_plan* plan, int dtype, int d, const void* x, void* q,
                    float* s, void* stream);
int moe_permute_bwd(const moe_plan_desc* desc, const moe_plan* plan, int dtype, int d, const void* dxp, void* dx,
                    void* stream);
int moe_unpermute(const moe_plan_desc* desc, const moe_plan* plan, int dtype, int d, const void* y, const float* w,
                  void* o, void* stream);
int moe_unpermute_bwd(const moe_plan_desc* desc, const moe_plan* plan, int dtype, int d, const void* d_o,
                      const void* y, const float* w, void* dy, float* dw, void* stream);

/*
 * Quantizers.  src dtype MOE_F32 or MOE_BF16, C (K, N) multiples of 16,
 * matrices 16-byte aligned.
 *   moe_fp8_quant_rows     src [R,C] -> q [R,C], s [R, ceil(C/128)]; with a
 *                          plan (desc and plan non-NULL, R = moe_plan_rows)
 *                          only the plan's rows are read and written.  R >= 0.
 *   moe_fp8_quant_weights  w [E,K,N] -> q [E,K,N] and qt [E,N,K] (either may be
 *                          NULL), s [E, ceil(K/128), ceil(N/128)], blocks 128 x 128
 *   moe_fp8_quant_cols     per segment and column, blocks of 128 rows from the
 *                          segment's first row on: q [cap/128, C, 128] (block,
 *                          column, row in the block), s [cap/128, C]; the rows
 *                          that fill up a segment's last block count as zeros.
 *                          align must be a multiple of 128; blocks from
 *                          offsets[E] on are left as they were.  src is [cap,C],
 *                          or with gather != 0 [T,C], read through row_token.
 */
int moe_fp8_quant_rows(const moe_plan_desc* desc, const moe_plan* plan, int dtype, int64_t R, int C,
                       const void* src, void* q, float* s, moe_profile* profile, void* stream);
int moe_fp8_quant_weights(int dtype, int E, int K, int N, const void* w, void* q, void* qt, float* s,
                          moe_profile* profile, void* stream);
int moe_fp8_quant_cols(const moe_plan_desc* desc, const moe_plan* plan, int dtype, int C, int gather,
                       const void* src, void* q, float* s, void* stream);

/* moe_mm_desc.flags */
#define MOE_MM_GATHER       1u  /* row r of the product reads a's row row_token[r] */
#define MOE_MM_SB_OUT_MAJOR 2u  /* sb is [E, ceil(N/128), ceil(K/128)]             */

/*
 * Product of E4M3 operands with a scale per block of 128 along the reduction:
 *     c[r,j] = sum over blocks B of  sa[r,B] * sb[e,B,j/128] * sum_{i in B} a[r,i] b[e,j,i]
 * for the rows r of expert e's segment.  Precision: with an fp32 result every
 * product is exact and all sums run in fp32.  With a bf16 result the 8-bit matrix
 * cores may form a block's inner sums: they add eight neighbouring products at a
 * time and cut those off 13 bits below the largest one's leading power of two, which
 * is an error below 7 * 2^-13 of sum |a b| (times the scales); all further sums run
 * in fp32.  On normally distributed values that is 1.4e-5 of the result in the mean
 * square, beside 1.7e-3 for its rounding to bf16; where large products cancel it may
 * be more than the rounding.  Calls of few rows per expert sum in fp32 throughout, so
 * a row's bf16 result may depend, within this error, on the sizes of the call it is
 * part of.  The same call gives the same bits.
 * Scales: an fp32 result takes any two, zero and subnormal ones too, whose product is
 * below 2^228.  A bf16 result may be formed with their product sa * sb rounded to fp32
 * first: where that is below 2^-126 a block's share is off by up to 2^-125 more, and
 * where it passes the largest number the result is not finite.
 *   a  [a_rows, K] codes, sa [a_rows, ceil(K/128)]
 *   b  [E, N, K] codes (the reduction contiguous), sb [E, ceil(K/128), ceil(N/128)]
 *      (or out-major, MOE_MM_SB_OUT_MAJOR)
 *   c  [rows, N] (dtype `out`); rows of no segment are left as they were.
 * With a plan, rows = the plan's capacity and a_rows = rows, or T with
 * MOE_MM_GATHER.  Without one (plan NULL) the product is dense: E = 1 and
 * a_rows = rows.  rows = 0 does nothing.  rows_used: at most so many of the rows
 * belong to segments, T*K for a plan (all segments' rows together; results of
 * further ones are not computed); 0: rows.
 *
 * For weights w [E,K,N] quantized by moe_fp8_quant_weights: x w takes b = qt,
 * sb = s; its input gradient, dy w^T, takes b = q (a product with K and N
 * changed over), sb = s and MOE_MM_SB_OUT_MAJOR.  Weights kept as [N,K] with
 * scales [N/128, K/128] are b and an out-major sb as they are.
 *   Limits: K and N multiples of 16 and at most 2^20, E <= 1024, N * K below
 *   2^31, with MOE_MM_GATHER a_rows * K below 2^31 (MOE_ESHAPE; larger ones go
 *   through moe_permute_fp8).
 */
typedef struct moe_mm_desc {
    int32_t  a_rows, rows, rows_used, E, K, N;
    int32_t  out;           /* MOE_F32 or MOE_BF16 */
    uint32_t flags;         /* MOE_MM_* */
    uint32_t reserved;      /* must be 0 */
    moe_profile* profile;
} moe_mm_desc;

int moe_fp8_mm(const moe_mm_desc* desc, const void* a, const float* sa, const void* b, const float* sb,
               const moe_plan* plan, void* c, void* stream);

/*
 * Weight gradient: per expert, over the blocks B of 128 rows of its segment,
 *     dw[e,i,j] = sum_B sa[B,i] * sb[B,j] * sum_{r in B} a[B,i,r] b[B,j,r]
 *   a [cap/128, M, 128], sa [cap/128, M] and b [cap/128, N, 128], sb [cap/128, N]
 *   from moe_fp8_quant_cols with this plan; dw [E,M,N] (dtype `out`), zeros for
 *   an expert without rows.  M and N multiples of 16 and at most 2^20.  Precision
 *   and scales as in moe_fp8_mm.
 */
int moe_fp8_wgrad(const moe_plan_desc* desc, const moe_plan* plan, int M, int N, int out, const void* a,
                  const float* sa, const void* b, const float* sb, void* dw, void* stream);

/*
 * SwiGLU between the two products.  h [R,2n]: columns 0..n-1 (G) feed SiLU,
 * n..2n-1 (U) are the up half, as in moe.h; n a multiple of 16.  With a plan
 * (R = moe_plan_rows) only the plan's rows are read and written.
 * The sigmoid is off by at most 5 * 2^-24 of itself; below 2^-126 (gates under -87.3)
 * it may count as 0.
 *   moe_swiglu_fp8   A = silu(G) U in fp32 -> codes q [R,n], scales
 *                    s [R, ceil(n/128)], and when `a` is non-NULL A itself
 *                    [R,n] in h's type
 *   moe_swiglu_bwd   dh [R,2n] = ( da U s (1 + G (1 - s)), da silu(G) ),
 *                    s = sigmoid(G); da [R,n] and dh in h's type
 */
int moe_swiglu_fp8(const moe_plan_desc* desc, const moe_plan* plan, int dtype, int64_t R, int n, const void* h,
                   void* q, float* s, void* a, moe_profile* profile, void* stream);
int moe_swiglu_bwd(const moe_plan_desc* desc, const moe_plan* plan, int dtype, int64_t R, int n, const void* da,
                   const void* h, void* dh, moe_profile* profile, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_OPS_H */
