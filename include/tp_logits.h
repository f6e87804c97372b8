/*
 * libtp, stored score rows: consumers of scores that a model has already written (its logits [N, M], one
 * row per position, one column per vocabulary entry), beside the lazy consumers of tp.h.
 *
 *   token log probabilities   of one given token per row, with the row's entropy and its top alternatives
 *   top-k distillation        KL divergence of a student's row from a teacher's list of top values
 *
 * Notation of a row: x_v its scores, T the temperature, p_v = exp(x_v / T) / sum_u exp(x_u / T).
 *
 * Conventions: those of tp.h (caller-owned device memory, nothing allocated, nothing synchronised, status
 * codes only, every argument validated before anything is launched, tp_last_error, launch hook and timer,
 * TP_FAULT_INJECT with the entry's name), and
 *   - No entry here needs a workspace.
 *   - Rows are read where they lie (tp_rows): any row stride, one level of grouping, any alignment that the
 *     element type has. Everything else is dense and row-major: [N], [N, k], [N, K], stats [N, 8].
 *   - Scores are fp32, fp16 or bf16; probabilities, sums and statistics are fp32 or wider; gradients have
 *     the scores' type (one rounding at the end).
 *   - A score of -inf is a masked column: probability 0, gradient 0, never an alternative. A row of -inf
 *     alone has log probability -inf, entropy 0, no alternatives and gradient 0. The type's lowest value is a
 *     score like any other, at any temperature: its probability is 0 beside an ordinary one, its distance
 *     finite. NaN or +inf in a row that is read gives NaN in its results; nothing else is promised for them.
 *   - Rows left out (a token, or a whole list, that does not count) are not looked at: zeros, (-inf, -1), and
 *     a zero gradient, whatever the row holds. (Their memory must be there all the same: a row's first scores
 *     may be on their way to the cache before its token or list is seen.)
 *   - Results do not depend on the run: no atomics on floating data, the same call gives the same bits. Another
 *     number of rows or alternatives, or another alignment, may split a row over other threads, and its sums
 *     then round otherwise in the last bits.
 */
#ifndef TP_LOGITS_H_
#define TP_LOGITS_H_

#include "tp.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { TP_ROWS_F32 = 0, TP_ROWS_F16 = 1, TP_ROWS_BF16 = 2 } tp_rows_dtype;

/* N rows of M scores. Row i starts at element (i / group) * group_stride + (i % group) * row_stride of
 * data; the M scores of a row are adjacent. A plain matrix has group = N (group_stride is then not read);
 * a shifted batch such as logits[:, :-1] of [B, S, M] has group = S - 1, row_stride = M,
 * group_stride = S * M. 1 <= N < 2^31, 1 <= M <= 2^30; N is a multiple of group; strides are >= 0 elements. Rows that
 * are written must not overlap one another. */
typedef struct {
    tp_rows_dtype dtype;
    int64_t N, M;
    int64_t group, row_stride, group_stride;
    void* data;
} tp_rows;

/* Log probability of tokens[i] in row i, the row's entropy, and its `top` likeliest columns:
 *     logprobs[i] = log p_t,   entropy[i] = - sum_v p_v log p_v   (natural logarithms)
 *     top_logprobs [N, top], top_ids [N, top]: the largest x_v, descending, ties to the lower column; fewer
 *     than `top` columns above -inf leave (-inf, -1) at the end (the rule of tp_pairwise_topk).
 * tokens [N] int64: a token outside [0, M) leaves its row out. tokens and logprobs are both NULL when no
 * tokens are given; every row then counts. 0 <= top <= min(M, 128); the two top arrays are NULL when top
 * is 0. stats [N, 8] receives what the backward takes back; NULL when no backward follows.
 * temperature in [1e-3, 1e3]. */
TP_API tp_status tp_token_logprobs(const tp_rows* logits, const int64_t* tokens, double temperature, int top,
                                   float* logprobs, float* entropy, float* stats, float* top_logprobs,
                                   int64_t* top_ids, void* stream);

/* Gradient of L = sum_i grad_logprobs_i logprobs_i + grad_entropy_i entropy_i:
 *     dL/dx_v = (grad_logprobs_i ([v = t] - p_v) - grad_entropy_i p_v (log p_v + entropy_i)) / T
 * logits, tokens, temperature as in the forward, stats as it wrote them; either upstream gradient [N] may
 * be NULL (zero), not both; masked columns get 0 as long as their values over T stay below 2^120. grad may be
 * the logits themselves (same data, type and strides: overwritten), or lie between their rows at the same
 * strides (two halves of one buffer's rows); otherwise it must lie outside the span of every input. */
TP_API tp_status tp_token_logprobs_backward(const tp_rows* logits, const int64_t* tokens, double temperature,
                                            const float* stats, const float* grad_logprobs,
                                            const float* grad_entropy, const tp_rows* grad, void* stream);

/* Divergence of each row from a teacher's list of K columns and values (1 <= K <= 128, any order):
 * ids [N, K] int64, values [N, K] float. An entry counts when its id is in [0, M) and its value is above
 * -inf; a row without one is left out. A column listed twice holds both shares.
 *   rest = 0: values are the teacher's scores; q = softmax(values / T) over the entries that count,
 *             loss_i = sum_k q_k (log q_k - log p_{id_k})
 *   rest = 1: values are the teacher's log probabilities (tp_token_logprobs' top_logprobs, taken at the same
 *             temperature); q_k = exp(value_k), and the columns not listed form one more class with
 *             q_r = 1 - sum_k q_k against p_r = their probability:
 *             loss_i = sum_k q_k (log q_k - log p_{id_k}) + q_r (log q_r - log p_r)
 *             q_r below 2^-20 counts as 0: the rounding of fp32 log probabilities can leave as much of a full
 *             list. The last term is also left out when no unlisted column is above -inf.
 * A listed column with q_k > 0 and a score of -inf gives +inf. stats [N, 8]: as above. */
TP_API tp_status tp_topk_distillation(const tp_rows* logits, int K, const int64_t* ids, const float* values,
                                      double temperature, int rest, float* loss, float* stats, void* stream);

/* Gradient of L = sum_i grad_loss_i loss_i with respect to the scores (the teacher's list is constant):
 *     listed columns    grad_loss_i (Z p_v - sum of their q_k) / T,   Z = sum_k q_k (+ q_r)
 *     other columns     grad_loss_i (Z p_r - q_r) (p_v / p_r) / T     (rest = 0: grad_loss_i p_v / T)
 * grad as in tp_token_logprobs_backward. */
TP_API tp_status tp_topk_distillation_backward(const tp_rows* logits, int K, const int64_t* ids,
                                               const float* values, double temperature, int rest,
                                               const float* stats, const float* grad_loss, const tp_rows* grad,
                                               void* stream);

/* Loss and gradient in one call, for row weights known beforehand: loss as tp_topk_distillation (not
 * weighted), grad the gradient of sum_i weights_i loss_i; weights [N] may be NULL (all ones). stats [N, 8]
 * is written as by the forward and must not be NULL. */
TP_API tp_status tp_topk_distillation_grad(const tp_rows* logits, int K, const int64_t* ids, const float* values,
                                           const float* weights, double temperature, int rest, float* loss,
                                           float* stats, const tp_rows* grad, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TP_LOGITS_H_ */
