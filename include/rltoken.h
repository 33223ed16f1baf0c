/*
 * rltoken.h — C ABI of the token log-probability and distillation operators
 * that stand beside the fused policy loss (rlloss.h; GB300, sm_103a).
 *
 * The policy loss consumes log-probabilities of sampled tokens (the rollout
 * buffer of the RL.cu article, ainews.cool, section "技术深度解析", bullet
 * "滚动缓冲区", holds them) and returns one fixed objective's gradient.  The
 * calls below give the pieces around it for logits that are in memory: the
 * log-probabilities of any given tokens with the entropy and the top
 * alternatives of each row, their gradient, and the loss and gradient of
 * distillation from a teacher's top log-probabilities.  The source pages have
 * no formula for them; each declaration states the definition it computes.
 *
 * Conventions are rlloss.h's: every array is DEVICE memory owned by the
 * caller on the current device, nothing is allocated, calls are stream-ordered
 * and capturable, argument errors are found on the host before anything is
 * launched, device-detected errors set RL_DEVERR_* bits, make the affected
 * outputs NaN and never trap.  A bounded wait that gives up (RL_DEVERR_TIMEOUT)
 * may affect any row: the call's loss and every row that is not known to be
 * right become NaN, right ones among them.
 *
 * Common arguments:
 *   logits      : [R, ld] of `dtype` (RL_F32, RL_BF16, RL_F16), row-major,
 *                 16-byte aligned, ld * sizeof(dtype) a multiple of 16,
 *                 ld >= V; the columns V .. ld-1 are ignored.
 *   V           : 1 <= V <= 2^26.
 *   mask        : uint8[R], nonzero = valid row; NULL = every row is valid.
 *                 The logits, ids and teacher of a masked row are not read.
 *                 With a mask the forward pass and the distillation take R <=
 *                 2^28 (the way to the next valid row stays far below the
 *                 limit of their waits).
 *   temperature : z = logits / temperature enters every formula;
 *                 0.01 <= temperature <= 100.
 *   status_dev  : one unsigned int or NULL; RL_DEVERR_* bits are ORed into it.
 * A logit of -inf is a token that cannot occur (probability 0, log-probability
 * -inf, nothing in the entropy).  A valid row whose logits are all -inf has no
 * distribution: its log-probabilities and entropy are NaN.  NaN or +inf in a
 * valid row makes that row's results NaN.  A log-probability below fp32's range
 * is -inf, a probability below 2^-126 counts as 0.
 */
#ifndef RLTOKEN_H
#define RLTOKEN_H

#include "rlloss.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most alternatives, given ids or teacher entries a row may have. */
#define RL_TOKEN_MAX_K 128

/* (device) the same teacher id twice in one row (rl_topk_distill_fwd_bwd). */
#define RL_DEVERR_ID_REPEAT 4u

/*
 * Log-probabilities of given tokens, with entropy and top alternatives.
 * For each valid row r, with z = logits[r] / temperature:
 *   lse_out[r]        = log sum_v exp z_v
 *   logp_out[r, j]    = z[ids[r, j]] - lse_out[r]            j < n_ids
 *   entropy_out[r]    = -sum_v p_v log p_v,  p = softmax(z)
 *   topk_ids[r, i]    = the i-th most likely token, ties to the lower id (a
 *                       NaN logit comes before every number)   i < k
 *   topk_logp[r, i]   = its log-probability
 * Masked rows get logp, entropy, lse and topk_logp 0 and topk_ids -1.
 *   ids      : int64 [R, n_ids] contiguous; an id outside [0, V) makes its
 *              logp NaN and sets RL_DEVERR_ID_RANGE.  NULL iff n_ids = 0.
 *   logp_out : float [R, n_ids]; NULL iff n_ids = 0.
 *   entropy_out, lse_out : float [R], each may be NULL.
 *   topk_ids, topk_logp  : int64 and float [R, k], both NULL iff k = 0.
 *   0 <= n_ids, k <= RL_TOKEN_MAX_K, k <= V, with k > 0 a row may have at
 *   most 4 MB (2^21 16-bit or 2^20 fp32 logits).
 * fp32 arithmetic on the exact differences to the row's maximum; the maximum
 * itself stays out of the running sum, so that a log-probability next to 0
 * keeps its relative precision.  A row's sum is rounded at most V / 256 + 64
 * times (V / 64 + 64 where the row's maximum is at or below -16384, fp16 -32768,
 * or above 2^24 temperature ln 2).  Deterministic: a row's results depend on its
 * logits and on the launch's shape, not on other rows.  One launch.
 * Errors: RL_ERR_DTYPE, RL_ERR_SHAPE (R < 0, R >= 2^31, R > 2^28 with a mask, V
 * or ld out of range, k > V, a row too long for k > 0), RL_ERR_ARG (n_ids or k out of range,
 * temperature), RL_ERR_NULL, RL_ERR_ALIGN, RL_ERR_CUDA.  R = 0 launches
 * nothing.
 */
rl_status rl_token_logprobs(const void* logits, rl_dtype dtype, long long R, long long V, long long ld,
                            const long long* ids, int n_ids, const unsigned char* mask, float temperature,
                            int k, float* logp_out, float* entropy_out, float* lse_out,
                            long long* topk_ids, float* topk_logp, unsigned int* status_dev, void* stream);

/*
 * Gradient of the log-probabilities and the entropy of rl_token_logprobs with
 * respect to the logits.  For each valid row, with p_v = exp(z_v - lse):
 *   dlogits_v = (1 / temperature) [ sum_j dlogp_j ([v = ids_j] - p_v)
 *                                   - dentropy p_v (z_v - lse + entropy) ]
 * rounded once to `dtype`; masked rows get an all-zero row.
 *   lse      : float [R], as rl_token_logprobs wrote it.  Its rounding is a
 *              relative error of up to |lse| 2^-24 in every p_v, which counts
 *              for logits of many thousands, and for those alone.
 *   dlogp    : float [R, n_ids]; NULL iff n_ids = 0.  An id that a row names
 *              several times collects the sum of its gradients; an id outside
 *              [0, V) makes the row NaN and sets RL_DEVERR_ID_RANGE.
 *   entropy, dentropy : float [R] each, or both NULL (no entropy gradient).
 *   dlogits  : [R, ld] of `dtype`, written (columns >= V untouched); may be
 *              the same pointer as logits; sharing other elements with it is
 *              RL_ERR_ALIAS (columns beside the logits' own are none of theirs).
 * One launch.  Errors as rl_token_logprobs, and RL_ERR_NULL when neither
 * dlogp nor dentropy is given.
 */
rl_status rl_token_logprobs_bwd(const void* logits, rl_dtype dtype, long long R, long long V, long long ld,
                                const long long* ids, int n_ids, const unsigned char* mask,
                                float temperature, const float* lse, const float* entropy,
                                const float* dlogp, const float* dentropy, void* dlogits,
                                unsigned int* status_dev, void* stream);

/* Where the teacher's mass outside its given entries goes. */
typedef enum {
  RL_DISTILL_TAIL_BUCKET = 0,   /* one more outcome: any token that is not given */
  RL_DISTILL_TAIL_RENORM = 1    /* nowhere: the given entries are normalised to 1 */
} rl_distill_tail;

/* Scalar results of rl_topk_distill_fwd_bwd (device memory, written at the
 * end): the loss, and means over the N valid rows of the two divergences and
 * of the tail's probability under the teacher and the student (RENORM: only
 * the forward divergence; the others are 0). */
typedef struct {
  double loss;
  double forward_kl;
  double reverse_kl;
  double teacher_tail;
  double student_tail;
  long long n_rows;      /* N */
  int device_error;      /* RL_DEVERR_* bits seen during this call */
  int reserved;
} rl_distill_stats;

/*
 * Distillation from a teacher's top log-probabilities: the loss and its
 * gradient with respect to the student's logits, in one launch.  On-policy
 * distillation puts this objective in the place of, or beside, the policy
 * loss on the same [R, V] logits; the teacher's side is what rl_token_logprobs
 * returns (topk_ids, topk_logp).
 *
 * For each valid row, the teacher gives K entries (id_j, l_j); an id of -1 is
 * an empty entry.  p = softmax(logits / temperature).
 *   BUCKET: q_j = exp(l_j); the tokens that are not given form one outcome
 *     with q_t = max(1 - sum_j q_j, 2^-24) and p_t = max(sum of their p,
 *     2^-126) (no such outcome when all V tokens are given).
 *   RENORM: q = softmax over the row's l_j (they may be logits then); there is
 *     no further outcome, and reverse must be 0.
 *   F = sum_b q_b (ln q_b - ln p_b)     G = sum_b p_b (ln p_b - max(ln q_b, ln 2^-126))
 *   L_r = weight_r [ (1 - reverse) F + reverse G ]
 *   loss = (1/N) sum_r L_r,  N = norm if norm > 0, else the number of valid rows
 * and, with Q = sum_b q_b and s = grad_scale weight_r / (N temperature),
 *   dlogits_v = s [ (1 - reverse) (p_v Q - q_v) + reverse p_v (ln p_v - ln q_v - G) ]   v given
 *   dlogits_v = s p_v [ (1 - reverse) (Q - q_t/p_t) + reverse (ln p_t - ln q_t - G) ]   v not given
 * rounded once to `dtype`.  Masked rows get loss 0 and an all-zero gradient;
 * so does a RENORM row with no entry.  The tail's mass is summed by itself,
 * never taken as 1 - sum p_j.
 * An id outside [-1, V) or named twice in a row sets RL_DEVERR_ID_RANGE or
 * RL_DEVERR_ID_REPEAT and makes the row's loss and gradient NaN.
 * Deterministic: fixed-order fp64 reductions.
 */
typedef struct {
  const void* logits;
  rl_dtype dtype;
  long long R, V, ld;
  const long long* teacher_ids;   /* int64 [R, K] */
  const float* teacher_logp;      /* float [R, K] */
  int K;                          /* 1 .. RL_TOKEN_MAX_K */
  const unsigned char* mask;      /* nullable: every row is valid */
  const float* weight;            /* nullable: float [R], 1 */
  rl_distill_tail tail;           /* default RL_DISTILL_TAIL_BUCKET */
  float reverse;                  /* default 0; in [0, 1] */
  float temperature;              /* default 1 */
  float grad_scale;               /* default 1 */
  double norm;                    /* default 0 (= the number of valid rows) */
  void* dlogits;                  /* nullable: forward only; may be logits itself */
  float* row_loss_out;            /* nullable: float [R], L_r */
  float* loss_out;                /* nullable: float [1], the loss */
  rl_distill_stats* stats_dev;
  void* workspace;                /* rl_topk_distill_workspace_size(); zero-filled once, left ready */
  size_t workspace_bytes;
} rl_topk_distill_desc;

/* Fill *desc with the defaults above (all pointers NULL, sizes 0). */
void rl_topk_distill_desc_init(rl_topk_distill_desc* desc);

/* Bytes of device workspace rl_topk_distill_fwd_bwd needs (zero-filled before
 * its first use; every call leaves it ready for the next; one call at a time). */
size_t rl_topk_distill_workspace_size(void);

/*
 * Errors: RL_ERR_NULL (desc, stats_dev, logits or teacher), RL_ERR_DTYPE
 * (dtype, tail), RL_ERR_SHAPE, RL_ERR_ARG (K, reverse, temperature,
 * grad_scale, norm out of range; reverse != 0 with RENORM), RL_ERR_ALIGN (as
 * above; workspace on 16, stats_dev on 8 bytes),
 * RL_ERR_ALIAS (dlogits shares elements with logits and is not logits),
 * RL_ERR_WORKSPACE, RL_ERR_CUDA.
 */
rl_status rl_topk_distill_fwd_bwd(const rl_topk_distill_desc* desc, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* RLTOKEN_H */
