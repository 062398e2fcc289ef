/*
 * liblp, the LM head in 8-bit integers: what a rollout engine that serves its
 * head with 8-bit weights and activations computes, for AMD Instinct MI355X
 * (gfx950). The quantiser, the rows of logits (for lp_sample, lp_verify and
 * lp_top_logprobs), and the score of given tokens without the logits (beside
 * lp_score, whose head is bf16): the same weights scored both ways separate
 * what quantisation changes from what the rest of the engine does.
 *
 * The conventions are liblp.h's: C ABI, every pointer argument device memory
 * owned by the caller unless stated otherwise, work enqueued on `stream`,
 * argument errors returned before anything is enqueued, no allocation and no
 * state in the library. The functions live in the same shared library.
 *
 * A matrix in 8 bits is [rows, H] int8 codes (element stride 1, row stride ld
 * elements) with one fp32 scale per row: it stands for scale[r] * code[r, k].
 * Hidden states have a scale per token, the head one per vocabulary row.
 *
 * Batch invariance: each row's outputs are a fixed function of that row, the
 * head, H and the dtype; they do not depend on the number of rows, the row's
 * place in the batch, the stream or the occupancy. Sums of products are exact
 * (32-bit integers); no floating-point atomics.
 */
#ifndef LIBLP_INT8_H
#define LIBLP_INT8_H

#include "liblp_logits.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most hidden elements of a product: 2^17 - 1, so that sums of products of
 * codes (at most 2^14 each) stay below 2^31. */
#define LP_INT8_MAX_HIDDEN 131071

/* ------------------------------------------------------------------------
 * Rows in 8 bits
 *
 * For every row r of x (LP_F32, LP_BF16 or LP_F16, row stride ldx, any
 * alignment of the element type):
 *
 *   scale[r] = max_k |x[r, k]| times the fp32 number nearest to 1/127, rounded
 *              to fp32 (that number is off by 2^-28, so that the scale of a row
 *              that is not tiny is max / 127 to 1.07 2^-24, where the rounded
 *              quotient would be to 2^-24)
 *   q[r, k]  = the integer nearest to x[r, k] / scale[r] (the quotient of the
 *              real numbers, ties to even), within [-127, 127]
 *
 * A row whose scale is 0 (zeros; or values so small that the scale rounds to
 * 0) has codes 0. A row with a NaN or an infinity has scale NaN and codes 0 and
 * is counted in bad_rows (one int32, may be NULL; the library ADDS).
 *
 * Layout: q [R, H] with row stride ldq, a multiple of 16, and 16-byte aligned,
 * as the products below take it; the codes behind H up to the next multiple of
 * 16 are written as zeros; q and scale lie apart from x and from each other.
 * Errors: LP_EINVAL for R < 0, H < 1, ldx < H, ldq < H or not a multiple of 16,
 * an unknown dtype, NULL or misaligned pointers; LP_EUNSUPPORTED for R or H above
 * 2^31 - 1 or more rows than one dispatch holds (16 777 215). R == 0 does nothing.
 * ------------------------------------------------------------------------ */
lp_status lp_quantize_int8(const void* x, int64_t ldx, int32_t dtype, int64_t R,
                           int64_t H, int8_t* q, int64_t ldq, float* scale,
                           int32_t* bad_rows, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Rows of logits from an 8-bit head
 *
 *   z[t, v] = (S x_scale[t]) w_scale[v],  S = sum_k x[t, k] w[v, k]
 *
 * S is exact; it is rounded to fp32 (exact below 2^24) and each product is
 * rounded to fp32, then z to `dtype`: an error of at most 3 2^-24 relative
 * (where neither product is subnormal) and, for bf16 and fp16, one rounding
 * more. fp16 overflows to infinity from |z| = 65 520 on. A NaN scale gives NaN.
 *
 * Layout: x [T, H], row stride ldx, any alignment; w [V, H] 16-byte aligned
 * with row stride ldw, a multiple of 16 (what lies behind H up to the next
 * multiple of 16 may be read and counts for nothing); out [T, V] in `dtype`,
 * row stride ld_out >= V elements, any alignment of the element type, apart from
 * the inputs; columns from V on are left as they are.
 *
 * Workspace: lp_logits_int8_workspace_bytes(T, H), 256-byte aligned (hidden
 * states whose rows are not multiples of 128 elements at 16-byte aligned
 * addresses are laid out there first). Its contents on entry are ignored;
 * calls that may overlap need one each.
 *
 * Errors: LP_EINVAL for T < 0, H < 1, V < 1, ldx < H, ldw < H, ld_out < V, an
 * unknown dtype, NULL or misaligned pointers, a small workspace;
 * LP_EUNSUPPORTED for H above LP_INT8_MAX_HIDDEN, ldw not a multiple of 16, ldw
 * or ld_out above 2^22, T above 4 194 240, V above 2^31 - 256, or more tiles of 256
 * rows of w by 256 rows of x than 2^31 - 513. T == 0 does nothing.
 * ------------------------------------------------------------------------ */
size_t lp_logits_int8_workspace_bytes(int64_t T, int64_t H);

lp_status lp_logits_int8(const int8_t* x, int64_t ldx, const float* x_scale,
                         const int8_t* w, int64_t ldw, const float* w_scale,
                         int64_t T, int64_t H, int64_t V, void* out,
                         int64_t ld_out, int32_t dtype, void* workspace,
                         size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Scores under an 8-bit head
 *
 *   logprob[t] = z[t, target] / temperature - ln sum_v exp(z[t, v] / temperature)
 *
 * with z in fp32 as above, or with LP_SCORE_BF16_LOGITS rounded to bf16
 * first, as an engine that stores its logits in bf16 has them. out_lse (may
 * be NULL): the log-sum-exp. A target id outside [0, V_true) gives NaN and is
 * counted in bad_rows (one int32, may be NULL). A row with a NaN or +inf logit
 * (of a NaN or infinite scale) gives NaN; -inf is a token of probability 0.
 *
 * Precision: exponentials and sums are fp32, per 128 vocabulary rows and
 * joined in a fixed order, the score is taken from them in fp64 and is at most
 * 0; as lp_score, within about 1e-5 nats at logits of ordinary size. Logits in fp32 are taken as (S w_scale) x_scale here, so
 * |S w_scale| has to stay below fp32's largest number and
 * w_scale above its smallest normal one. Logits over the temperature are fp32
 * numbers too, in units of ln 2: |z| / temperature has to stay below 2.3e38.
 *
 * Layout and errors as for lp_logits_int8, target_ids [T] int64, out_logprob
 * and out_lse [T] fp32, apart from the inputs; LP_EINVAL for a temperature that is not a positive
 * normal number or an unknown flag. Workspace: lp_score_int8_workspace_bytes(T, H,
 * V_true).
 * ------------------------------------------------------------------------ */
size_t lp_score_int8_workspace_bytes(int64_t T, int64_t H, int64_t V_true);

lp_status lp_score_int8(const int8_t* x, int64_t ldx, const float* x_scale,
                        const int8_t* w, int64_t ldw, const float* w_scale,
                        const int64_t* target_ids, int64_t T, int64_t H,
                        int64_t V_true, float temperature, uint32_t flags,
                        float* out_logprob, float* out_lse, int32_t* bad_rows,
                        void* workspace, size_t workspace_bytes,
                        hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBLP_INT8_H */
