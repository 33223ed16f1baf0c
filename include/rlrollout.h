/*
 * rlrollout.h — C ABI of the rollout's operators: the half of a training step
 * that draws the tokens whose loss rlloss.h computes (GB300, sm_103a).
 *
 * The rollout buffer of the RL.cu article (ainews.cool, section
 * "技术深度解析", bullet "滚动缓冲区") holds actions and their
 * log-probabilities.  The calls below make them: 8-bit codes of hidden states
 * and of the LM head, the logits of that 8-bit head, and the verification of
 * drafted tokens against those logits, which without drafts is the sampling of
 * a decode step.  The source pages have no formula for them; each declaration
 * states the definition it computes.
 *
 * Conventions are rlloss.h's: every array is DEVICE memory owned by the
 * caller on the current device, nothing is allocated, calls are stream-ordered
 * and capturable, argument errors are found on the host before anything is
 * launched, device-detected errors set RL_DEVERR_* bits and never trap.
 */
#ifndef RLROLLOUT_H
#define RLROLLOUT_H

#include "rlloss.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most columns of an 8-bit product: the sum of so many products of two 8-bit
 * codes stays inside 32 bits. */
#define RL_INT8_MAX_D 131071

/* Most drafted tokens of a sequence. */
#define RL_VERIFY_MAX_DRAFT 128

/*
 * 8-bit codes of each row of a matrix and the scale they stand for, x ~
 * scale codes: hidden states token by token, or a weight channel by channel.
 *   a         = max_d |x[r, d]|
 *   scale[r]  = a / 127, rounded to fp32
 *   codes[r, d] = x[r, d] / scale[r] rounded to the nearest integer (the exact
 *               quotient, ties to even), at most 127 in size
 * A row whose scale is 0 (all zeros, or a below 2^-143) has codes 0; a row
 * that holds NaN or an infinity has scale NaN and codes 0, so that a product
 * with it is NaN.
 *   x     : [R, ld_x] of `dtype` (RL_F32, RL_BF16, RL_F16), 16-byte aligned,
 *           ld_x * sizeof(dtype) a multiple of 16, ld_x >= D.
 *   codes : int8 [R, ld_c], 16-byte aligned, ld_c >= D a multiple of 16, no
 *           byte of it in x; columns D .. ld_c-1 are not written.
 *   scale : float [R].
 * Errors: RL_ERR_DTYPE, RL_ERR_SHAPE (R < 0, R >= 2^31, D < 1, D >= 2^31, a stride below
 * D or so large that 64 bits do not address the rows), RL_ERR_NULL, RL_ERR_ALIGN, RL_ERR_ALIAS (an
 * output in x or in the other), RL_ERR_CUDA.  R =
 * 0 launches nothing.
 */
rl_status rl_quantize_rows_int8(const void* x, rl_dtype dtype, long long R, long long D, long long ld_x,
                                signed char* codes, long long ld_c, float* scale, void* stream);

/*
 * Logits of an 8-bit LM head, from codes with a scale for each token and each
 * channel (what rl_quantize_rows_int8 gives of hidden states and weight):
 *   logits[r, v] = scale_h[r] scale_w[v] sum_d hidden[r, d] weight[v, d]
 * The sum is exact: a row's logits are the same bits in any batch.  It is
 * rounded to fp32, multiplied by scale_h, then by scale_w in fp32, and rounded
 * to `dtype`.
 *   hidden, weight : int8 [R, ld_h] and [V, ld_w], 16-byte aligned, strides
 *                    multiples of 16 and >= D; all 256 codes are allowed.
 *   scale_h, scale_w : float [R] and [V].
 *   logits    : [R, ld] of `dtype` (RL_F32, RL_BF16, RL_F16), 16-byte aligned,
 *               ld * sizeof(dtype) a multiple of 16, ld >= V; columns V ..
 *               ld-1 are not written.
 *   status_dev: one unsigned int or NULL; RL_DEVERR_* bits are ORed into it.
 *   workspace : rl_lmhead_int8_workspace_size(R, D) bytes, 16-byte aligned; it
 *               need not be initialised; calls that may overlap take one each.
 *   1 <= D <= RL_INT8_MAX_D.
 * Errors: RL_ERR_DTYPE, RL_ERR_SHAPE (R < 0, R >= 2^31, V < 1, V >= 2^31, D out of
 * range, a stride too small or so large that 64 bits do not address the rows, more than
 * 2^30 tiles of 128 channels and 128 tokens), RL_ERR_NULL, RL_ERR_ALIGN, RL_ERR_ALIAS (logits
 * or workspace in an input or in one another), RL_ERR_WORKSPACE, RL_ERR_CUDA.  R = 0
 * launches nothing.
 */
rl_status rl_lmhead_logits_int8(const signed char* hidden, long long ld_h, const float* scale_h,
                                const signed char* weight, long long ld_w, const float* scale_w, long long R,
                                long long D, long long V, rl_dtype dtype, void* logits, long long ld,
                                unsigned int* status_dev, void* workspace, size_t workspace_bytes,
                                void* stream);

/* Bytes of device workspace rl_lmhead_logits_int8 needs (0 for sizes it refuses). */
size_t rl_lmhead_int8_workspace_size(long long R, long long D);

/*
 * Verification of drafted tokens, and the token drawn after those that stay.
 * Sequence b has n = n_draft[b] drafted tokens and n + 1 rows of target
 * logits: row i follows its first i drafts.  With p_i = softmax(target row i /
 * temperature) and q_i the distribution draft i was drawn from,
 *   q_i(v) = exp(draft_logits[b, i, v] / temperature - draft_lse[b, i]),
 * or, without draft_logits, 1 at draft_ids[b, i] and 0 elsewhere:
 *   draft i stays, if all before it did, iff
 *       uniforms[b, i] q_i(d) < p_i(d),        d = draft_ids[b, i]
 *   a = the number that stay
 *   one more token is drawn, from p_n if a = n, else from
 *       max(p_a - q_a, 0) (from p_a where that is 0 everywhere, to 2^-38 of what q_a has where they are equal):
 *       the first token at which the sum of weights in token order exceeds
 *       uniforms[b, G] times their total
 *   tokens[b]     = the a drafts that stay, the drawn token, then -1
 *   n_accepted[b] = a
 *   logp_out[b, i] = log p_i(tokens[b, i]),   lse_out[b, i] = the log-sum-exp
 *       of target row i / temperature, for i <= a; 0 behind
 * So tokens are drawn as from p alone, whatever the drafts.  With G = 0 the
 * call draws one token for each row; lse_out is then what a later call takes
 * as draft_lse.  Rows behind the first draft that does not stay decide
 * nothing.  The drawn token's border is resolved to 2^-34 of the total (for
 * max(p - q, 0) of p's total; to V 2^-52, or 2^-52 |draft_lse|, where that is more) or better, a
 * draft's own test to 2^-34 of p_i(d) (likewise), so that what stays and what is drawn are the same in
 * any batch.  (fp32 sums decide what lies further than 2^-19 of the total from a border, or 2^-17 of p_i(d); that
 * they are never off by so much rests on rows built to add up their roundings, of which none was off by
 * more than 2^-20.3, not on a proof.)
 * Log-probabilities are fp32, with relative precision next to 0.
 *
 * n_draft[b] = -1 leaves a sequence out: its tokens are -1, the rest 0, nothing
 * of it is read.  A logit of -inf is a token of probability 0.  A row without a
 * distribution (all -inf, or NaN or +inf in it; a draft's row or draft_lse with
 * NaN or infinite, where it is needed) ends its sequence: token -1 and
 * logp NaN there.  A draft id outside [0, V) or an n_draft outside [-1, G] sets
 * RL_DEVERR_ID_RANGE and gives tokens -1, n_accepted 0 and logp and lse NaN for the
 * whole sequence.  A uniform outside [0, 1) or NaN counts as the nearest number
 * inside (NaN as 0) for the draw.
 */
typedef struct {
  const void* target_logits;      /* [B, G + 1, ld] of dtype, 16-byte aligned, ld * sizeof a multiple of 16 */
  rl_dtype dtype;                 /* default RL_BF16; RL_F32, RL_F16 */
  long long B, G, V, ld;          /* 0 <= G <= RL_VERIFY_MAX_DRAFT, 1 <= V <= 2^26 */
  const void* draft_logits;       /* nullable: [B, G, ld_draft] of dtype, aligned alike */
  long long ld_draft;
  const float* draft_lse;         /* [B, G]; with draft_logits */
  const long long* draft_ids;     /* [B, G]; NULL iff G = 0 */
  const int* n_draft;             /* nullable: [B], G each */
  const double* uniforms;         /* [B, G + 1] in [0, 1) */
  double temperature;             /* default 1; in [0.01, 100] */
  long long* tokens;              /* [B, G + 1] */
  long long* n_accepted;          /* nullable: [B] */
  float* logp_out;                /* nullable: [B, G + 1] */
  float* lse_out;                 /* nullable: [B, G + 1] */
  unsigned int* status_dev;       /* nullable: RL_DEVERR_* bits are ORed into it */
} rl_verify_drafts_desc;

/* Fill *desc with the defaults above (all pointers NULL, sizes 0). */
void rl_verify_drafts_desc_init(rl_verify_drafts_desc* desc);

/*
 * Errors: RL_ERR_NULL (desc, target_logits, draft_ids, draft_lse beside
 * draft_logits, uniforms, tokens), RL_ERR_DTYPE, RL_ERR_SHAPE (B < 0, G, V or a
 * stride out of range, B (G + 1) >= 2^31, rows that 64 bits do not address), RL_ERR_ARG
 * (temperature), RL_ERR_ALIGN, RL_ERR_ALIAS (an output in an input or in another output),
 * RL_ERR_CUDA.  B = 0 launches nothing.
 */
rl_status rl_verify_drafts(const rl_verify_drafts_desc* desc, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* RLROLLOUT_H */
