/*
 * liblp, operators on rows of logits: the token draw of a rollout, the
 * verification of drafted tokens, the top logits of a scored position, and the distillation loss against a teacher's
 * top logits with its gradient, for AMD Instinct MI355X (gfx950).
 *
 * The conventions are liblp.h's: C ABI, every pointer argument device memory
 * owned by the caller unless stated otherwise, work enqueued on `stream`,
 * argument errors returned before anything is enqueued, no allocation and no
 * state in the library. The functions live in the same shared library.
 *
 * Logits: [rows, columns] in `dtype` (LP_F32, LP_BF16 or LP_F16), element
 * stride 1, row stride ld elements, any alignment of the element type.
 * V_true is the true vocabulary: columns from V_true on are never read. -inf
 * is a masked token (probability 0).
 *
 * Batch invariance: each row's outputs are a fixed function of that row's
 * logits and settings, V_true and the dtype; they do not depend on the number
 * of rows, the row's place in the batch, its alignment, the stream or the
 * occupancy. No floating-point atomics.
 *
 * Scratch memory: where a call takes a workspace, its contents on entry are
 * ignored, and calls that may overlap need one each (two captured graphs that
 * replay side by side too). The *_workspace_bytes of a number of rows and a V_true
 * serve every call of the same dtype with fewer of either, too.
 */
#ifndef LIBLP_LOGITS_H
#define LIBLP_LOGITS_H

#include "liblp.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LP_F32 0
#define LP_BF16 1
#define LP_F16 2

/* ------------------------------------------------------------------------
 * Token draw: temperature, top-k, top-p and min-p from given random numbers
 *
 * For every row n with temperature tau, top_k, top_p, min_p and the random
 * number u of the row:
 *
 *   s_v  = z_v / tau,   w_v = exp(s_v - max s)       (z: the row's logits)
 *   The tokens are ordered by (z descending, index ascending); C(m) is the
 *   sum of the first m weights of that order.
 *   k'   = the finite logits' count, at most top_k where top_k > 0
 *   m_p  = the least m >= 1 with C(m) >= top_p C(k')   (k' where top_p >= 1)
 *   m_m  = the number of w_v >= min_p, at least 1      (no limit: min_p <= 0)
 *   kept = min(k', m_p, m_m): the kept tokens are the first `kept`
 *   rank = the least r with C(r + 1) > u C(kept)
 *
 *   token      the token at that rank
 *   logprob    s_token - ln sum_{v < V_true} exp s_v: the score of the token
 *              under the full vocabulary, comparable with lp_score's at the
 *              same temperature
 *   processed  ln(w_token / C(kept)): the score under the distribution that
 *              the token was drawn from
 *
 * The raw and the processed score answer different questions, and a comparison
 * needs the same one on both sides ([AMD] "Make Sure Both Scores Answer the
 * Same Question": k = 2 turns (0.5, 0.3, 0.2) into (0.625, 0.375, 0)).
 *
 * tau == 0 is the greedy draw: token = the lowest index of the largest logit,
 * logprob at temperature 1, processed 0, kept 1. u is clamped to
 * [0, 1 - 2^-24]. top_p <= 0 keeps one token. A row that has a NaN or +inf
 * logit, no finite logit, a temperature other than 0 or a positive normal
 * number (finite, at least 2^-126), or a NaN u, top_p or min_p gives token -1,
 * NaN scores and kept 0, and is counted in bad_rows.
 *
 * Precision: what is kept and drawn is decided in fp64. Rows with top_k in
 * [1, 420], greedy ones and rows with min_p alone (at most 1 024 tokens kept)
 * go by a short list: fp64 weights and sums. The others go by buckets of 1/32
 * nat: weights in fp64 (8e-14 relative), summed as 64-bit integers per bucket,
 * so sums do not depend on an order; tokens more than 39.9 nats below the
 * maximum may weigh 0 there (they still count for top_k and kept). The raw
 * score's sum over the vocabulary is, for short lists, fp64 for the listed
 * tokens and the 16-byte groups that they lie in, and of fp32 exponentials
 * joined in fp64 for the rest: an error of at most 210 * 2^-24, usually 1e-7, of
 * the probability outside the list, so that the scores of near-certain tokens
 * keep their digits. Else it is the buckets': 1e-12, and the probability of the
 * tokens more than 39.9 nats below the maximum (at most V_true e^-39.9, 5e-12).
 * Scores are rounded to fp32 once.
 *
 * Layout: u [N] fp32; temperatures, top_ps, min_ps [N] fp32 and top_ks [N]
 * int32 give each row's settings, where NULL the scalar beside it holds for
 * every row. out_token [N] int64, out_logprob [N] fp32; out_processed [N]
 * fp32 and out_kept [N] int32 may be NULL. bad_rows: one int32, may be NULL;
 * the library ADDS the number of bad rows. Workspace: at least
 * lp_sample_workspace_bytes(N, V_true, dtype) bytes, 256-byte aligned.
 *
 * Errors: LP_EINVAL for N < 0, V_true < 1, ld < V_true, an unknown dtype, a
 * NULL required pointer, logits or another array not aligned to its element
 * type, a workspace that is too small or misaligned, and for a scalar
 * setting that is used: temperature neither 0 nor a positive normal number,
 * top_p or min_p NaN. LP_EUNSUPPORTED for V_true above LP_SELECT_MAX_VOCAB or
 * N above 4 194 303. N == 0 does nothing.
 * ------------------------------------------------------------------------ */
#define LP_SELECT_MAX_VOCAB 1048576

size_t lp_sample_workspace_bytes(int64_t N, int64_t V_true, int32_t dtype);

lp_status lp_sample(const void* logits, int64_t ld, int32_t dtype, int64_t N,
                    int64_t V_true, const float* u, const float* temperatures,
                    float temperature, const int32_t* top_ks, int32_t top_k,
                    const float* top_ps, float top_p, const float* min_ps,
                    float min_p, int64_t* out_token, float* out_logprob,
                    float* out_processed, int32_t* out_kept, int32_t* bad_rows,
                    void* workspace, size_t workspace_bytes,
                    hipStream_t stream);

/* ------------------------------------------------------------------------
 * Verification of drafted tokens
 *
 * Speculative decoding: a draft (a smaller model, or text copied from the
 * prompt) proposes D tokens at most for each of B sequences, the target model
 * scores all of them at once, and from given random numbers a prefix of them is
 * accepted and one token more is drawn, so that every token that comes out is
 * distributed as lp_sample's would be.
 *
 * Sequence b has n = counts[b] drafted tokens x_0 .. x_{n-1} (D where counts is
 * NULL), the target's rows b (D + 1) + j, j <= n, and the draft model's rows
 * b D + j, j < n, under one setting of temperature, top_k, top_p and min_p.
 *
 *   p_j(v)   the probability with which lp_sample draws v from the target's row
 *            j: w_v / C(kept) for the kept tokens, 0 for the others
 *   q_j(v)   the same of the draft's row j; without draft logits (NULL) 1 for
 *            v = x_j: the draft proposes that token alone
 *   x_j is accepted if all before it are and u[b, j] q_j(x_j) < p_j(x_j)
 *   a        the number of accepted tokens
 *   token a  the least v with  sum_{i <= v} r_i > u[b, D] sum_i r_i,  where
 *            r_v = max(p_a(v) - q_a(v), 0) if a < n (p_a(v) where no r is
 *            positive), and r_v = p_n(v) if a = n
 *
 * out_tokens [B, D + 1]: x_0 .. x_{a-1}, token a, then -1. out_accepted [B]: a.
 * out_logprob, out_processed [B, D + 1]: ln of the token's probability under the
 * target's full vocabulary at the temperature (as lp_sample's logprob,
 * comparable with lp_score) and under p_j (as its processed score); 0 behind
 * token a. Temperature 0 (greedy) has p and q concentrated on the lowest index
 * of the largest logit, logprob at temperature 1 and processed 0. The random
 * numbers are clamped to [0, 1 - 2^-24].
 *
 * A sequence whose count lies outside [0, D], whose drafted tokens (j < n) lie
 * outside [0, V_true), whose rows (target j <= n, draft j < n) or settings have
 * no valid draw (see lp_sample), or whose random numbers (j < n, and D) are NaN
 * gives tokens -1, NaN scores and accepted -1, and is counted in bad_rows.
 * Rows, ids and random numbers behind a sequence's drafts are not read.
 *
 * Precision: p and q in fp64, each weight, and the sum of a row that is kept whole, to
 * 1.1e-12 relative, with C and the borders as lp_sample has them otherwise;
 * acceptances, the sums over r and the last token are decided in fp64, sums in
 * an order fixed by V_true and the dtype. Scores are rounded to fp32 once.
 *
 * Layout: draft_logits has the logits' dtype, row stride ld_draft; draft_ids
 * [B, D] int64; u [B, D + 1] fp32; counts [B] int32 or NULL; settings as for
 * lp_sample, arrays [B]; out_processed may be NULL. D may be 0 (draft_ids NULL).
 * Workspace: at least lp_verify_workspace_bytes(B, D, V_true, dtype) bytes,
 * 256-byte aligned.
 *
 * Errors: as for lp_sample, with D < 0 and ld_draft < V_true; LP_EUNSUPPORTED
 * for D above LP_VERIFY_MAX_DRAFTS or B (2 D + 1) above 4 194 303. B == 0 does
 * nothing.
 * ------------------------------------------------------------------------ */
#define LP_VERIFY_MAX_DRAFTS 63

size_t lp_verify_workspace_bytes(int64_t B, int64_t D, int64_t V_true, int32_t dtype);

lp_status lp_verify(const void* logits, int64_t ld, int32_t dtype, int64_t B,
                    int64_t D, int64_t V_true, const void* draft_logits,
                    int64_t ld_draft, const int64_t* draft_ids,
                    const int32_t* counts, const float* u,
                    const float* temperatures, float temperature,
                    const int32_t* top_ks, int32_t top_k, const float* top_ps,
                    float top_p, const float* min_ps, float min_p,
                    int64_t* out_tokens, int32_t* out_accepted,
                    float* out_logprob, float* out_processed,
                    int32_t* bad_rows, void* workspace, size_t workspace_bytes,
                    hipStream_t stream);

/* ------------------------------------------------------------------------
 * Top logits of every row
 *
 * The first k tokens of the order (z descending, index ascending):
 *   out_ids     [N, k] int64
 *   out_logits  [N, k] fp32, the logits themselves (exact)
 *   out_logprob [N, k] fp32, z / temperature - lse
 *   out_lse     [N] fp32, may be NULL: ln sum_{v < V_true} exp(z_v / temperature)
 * A row with fewer than k finite logits ends in id -1, logit -inf, logprob
 * -inf. A row with a NaN or +inf logit, or without a finite one, is id -1 and
 * NaN throughout (lse NaN) and counted in bad_rows (one int32, may be NULL).
 *
 * The teacher's side of lp_distill_*: out_ids with out_logits (renormalised
 * there) or with out_logprob (taken as they are).
 *
 * Logprobs and lse have the precision of the token draw's raw score by short
 * lists. Errors as for lp_sample, plus LP_EINVAL for k < 1 or k > V_true and a
 * temperature that is not a positive normal number, LP_EUNSUPPORTED for k above
 * LP_TOP_MAX. Workspace: lp_top_logprobs_workspace_bytes(N, V_true, dtype).
 * ------------------------------------------------------------------------ */
#define LP_TOP_MAX 1024

size_t lp_top_logprobs_workspace_bytes(int64_t N, int64_t V_true, int32_t dtype);

lp_status lp_top_logprobs(const void* logits, int64_t ld, int32_t dtype,
                          int64_t N, int64_t V_true, int32_t k,
                          float temperature, int64_t* out_ids,
                          float* out_logits, float* out_logprob,
                          float* out_lse, int32_t* bad_rows, void* workspace,
                          size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Distillation from a teacher's top logits: loss and gradient
 *
 * For every row t with student logits z, the teacher's entries (i_k, x_k),
 * k < K, and temperature tau; an entry with id -1 is absent:
 *
 *   p    = softmax(z / tau) over v < V_true
 *   q_k  = softmax over the row's entries of x_k / tau, or with
 *          LP_DISTILL_LOGPROBS exp(x_k): x_k is a logprob already (at the
 *          temperature the caller wants), and Q = sum_k q_k is what it is
 *   loss = sum_{k: q_k > 0} q_k (ln q_k - ln p[i_k])
 *   d loss / d z_v = (Q p_v - sum_{k: i_k = v} q_k) / tau
 *
 * (the forward Kullback-Leibler divergence KL(q || p) where Q = 1). An id
 * that occurs twice in a row counts with the sum of its entries.
 *
 * A row whose entries are all absent, or weigh 0, has loss 0 and gradient 0,
 * whatever its logits are. An id outside [0, V_true) other than -1 makes the
 * row's loss and gradient NaN and is counted in bad_rows (one int32, may be
 * NULL). NaN or +inf logits, and rows without a finite logit, give NaN; a
 * teacher entry on a masked token (z = -inf) gives loss +inf and the
 * formula's gradient (p = 0).
 *
 * lp_distill_forward   loss [T] fp32 and row_state [T][4] fp64 (8-byte
 *                      aligned; may be NULL), what the backward pass needs of
 *                      a row: maximum, sum, teacher's normaliser, Q.
 * lp_distill_backward  grad_logits[t, v] = grad_loss[t] * d loss / d z_v
 *                      from the forward's row_state and the same inputs, in
 *                      the logits' dtype, rounded once. Columns [V_true,
 *                      V_columns) are written as zeros. A row with
 *                      grad_loss 0 is written as zeros and its logits are
 *                      not read.
 * lp_distill_step      both in one call, with the row weights known
 *                      beforehand: loss [T] (unweighted) and grad_logits =
 *                      weight[t] * d loss / d z. The same bits as the two calls.
 *
 * grad_logits [T, V_columns], row stride ld_grad elements; it may be the
 * logits' own buffer (same base, ld_grad = ld): every logit is read before
 * its place is written. Any other overlap is not allowed.
 *
 * Precision: the sums over the vocabulary are fp32 per thread (at most 32
 * terms) and fp64 from there on, in an order fixed by V_true and the dtype;
 * teacher terms and the loss are fp64. grad_loss[t] / temperature has to be in
 * fp32's range: a row where it is not has infinities and NaN in its gradient.
 *
 * Layout: teacher_ids [T, K] int64 and teacher [T, K] fp32, contiguous.
 * Workspace: lp_distill_workspace_bytes(T, V_true, dtype) for forward and
 * step, 256-byte aligned.
 *
 * Errors: LP_EINVAL for T < 0, V_true < 1, ld < V_true, V_columns < V_true,
 * ld_grad < V_columns, K < 1, an unknown dtype or flag, a temperature that is
 * not a positive normal number, NULL required or misaligned pointers, a small or misaligned workspace;
 * LP_EUNSUPPORTED for K above LP_DISTILL_MAX_K, T above 2^31 - 1 or
 * V_columns above 2^31 - 1. T == 0 does nothing.
 * ------------------------------------------------------------------------ */
#define LP_DISTILL_MAX_K 1024
#define LP_DISTILL_LOGPROBS 1u

size_t lp_distill_workspace_bytes(int64_t T, int64_t V_true, int32_t dtype);

lp_status lp_distill_forward(const void* logits, int64_t ld, int32_t dtype,
                             int64_t T, int64_t V_true,
                             const int64_t* teacher_ids, const float* teacher,
                             int64_t K, float temperature, uint32_t flags,
                             float* out_loss, double* row_state,
                             int32_t* bad_rows, void* workspace,
                             size_t workspace_bytes, hipStream_t stream);

lp_status lp_distill_backward(const void* logits, int64_t ld, int32_t dtype,
                              int64_t T, int64_t V_true, int64_t V_columns,
                              const int64_t* teacher_ids, const float* teacher,
                              int64_t K, float temperature, uint32_t flags,
                              const double* row_state, const float* grad_loss,
                              void* grad_logits, int64_t ld_grad,
                              hipStream_t stream);

lp_status lp_distill_step(const void* logits, int64_t ld, int32_t dtype,
                          int64_t T, int64_t V_true, int64_t V_columns,
                          const int64_t* teacher_ids, const float* teacher,
                          int64_t K, float temperature, uint32_t flags,
                          const float* weight, float* out_loss,
                          void* grad_logits, int64_t ld_grad,
                          int32_t* bad_rows, void* workspace,
                          size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBLP_LOGITS_H */
