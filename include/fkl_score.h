/*
 * fkl_score.h - C ABI of the scoring operators: the log-probability of given tokens, the
 * entropy of the distribution they are scored under, and its most likely alternatives.
 *
 * On-policy distillation draws text (fkl_generate.h) and then scores it: a server returns the
 * log-probabilities of its tokens with a few alternatives, and a training step needs them, with
 * an entropy term, as a differentiable function of the logits or of the hidden states.  For a
 * row of logits x, a token v* and a temperature T,
 *
 *     z_v = x_v / T,  lse = log sum_v exp(z_v),  q_v = exp(z_v - lse)
 *     logprob = z_{v*} - lse,   entropy = -sum_v q_v log q_v
 *     d/dx_v (a logprob + b entropy) = ( a (1[v = v*] - q_v) - b q_v (log q_v + entropy) ) / T
 *
 * fkl_token_logprobs reads logits in memory; fkl_logprob_forward projects hidden states through
 * the LM head, x = H W^T, and never writes the T x V logits, as the loss of fkl.h does.
 *
 * Conventions (device pointers, streams, errors, ownership) are those of fkl.h: the library
 * allocates no device memory, never synchronises, refuses bad arguments on the host before
 * anything is enqueued, and gives the same bits for the same inputs.
 *
 * Rows.  `mask` (uint8, 1 = valid; NULL = all valid) leaves rows out: their logprob and entropy
 * are 0, their gradient is 0, and neither their token nor what their logits or hidden states hold (NaN, say)
 * reaches anything else.  In the others a token outside [0, V) gives logprob NaN.
 *
 * NaN.  The two forms differ.  Over logits in memory it counts as -inf, as in the sampler whose tokens are scored: a row's
 * score stays finite, and what a token outside [0, V) spoils is its own row of the gradient.  From hidden
 * states, where a NaN is a fault of the product's operands, it makes its row's scores NaN, and a token outside [0, V) or
 * a NaN row spoils the whole gradient of the head, into which all rows go (the former that of the hidden states too).
 */
#ifndef FKL_SCORE_H_
#define FKL_SCORE_H_

#include <stddef.h>
#include <stdint.h>

#include "fkl_generate.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Scores the rows of logits in memory.
 *   logits   [B][V] of `type` (FKL_TYPE_*), rows `ld` elements apart (ld >= V), aligned to the type.
 *            As in fkl_sample, -inf bans an id, NaN counts as -inf, and +inf ids share all the
 *            probability
 *   tokens   int32 or int64 [B] (token_bytes 4 or 8)
 *   mask     uint8 [B] or NULL
 *   temperature       T > 0 for all rows, or, where temperature_rows (float [B]) is not NULL, one per
 *                     row; a row whose T is not a finite number above 0 is NaN.  From 4.25e-39 down log2(e) / T
 *                     is no float: such a T is refused, or makes its row NaN
 *   top_n    0 <= top_n <= min(V, 128): the row's top_n largest logits, largest first, ties by the lower id
 *   logprob, entropy  float [B]
 *   stats    float [B][2] or NULL: the row's largest logit m and log sum_v exp((x_v - m) / T), for the
 *            backward (with these two the gradient loses nothing when the logits are large)
 *   top_ids  int32 [B][top_n], top_logprobs float [B][top_n]; both may be NULL when top_n is 0.  A row with
 *            fewer ids that can be produced, or a row left out, ends in id -1 and -inf
 * A row with nothing to produce (every logit -inf or NaN) is NaN, with ids -1 and top_logprobs NaN; the other
 * rows are unaffected.  0 <= B <= 2^31 - 1, 1 <= V <= 2^22.
 */
fkl_status fkl_token_logprobs(const void* logits, int32_t type, int64_t B, int64_t V, int64_t ld, const void* tokens,
                              int32_t token_bytes, const uint8_t* mask, float temperature,
                              const float* temperature_rows, int32_t top_n, float* logprob, float* entropy,
                              float* stats, int32_t* top_ids, float* top_logprobs, void* stream);

/*
 * The gradient of sum_b (a_b logprob_b + b_b entropy_b) in the logits: dlogits [B][V] of the logits' type,
 * rows `ldd` elements apart, each value computed in fp32 and rounded once.  Every element of the B x V is
 * written (what lies between rows is not).
 *   grad_logprob, grad_entropy   float [B]; NULL = 0
 *   stats, entropy               the forward's
 * The row of a token outside [0, V), and a row that the forward found NaN, is NaN.  dlogits may be the logits
 * themselves when the strides agree; other overlaps are not allowed.
 */
fkl_status fkl_token_logprobs_backward(const void* logits, int32_t type, int64_t B, int64_t V, int64_t ld,
                                       const void* tokens, int32_t token_bytes, const uint8_t* mask,
                                       float temperature, const float* temperature_rows, const float* stats,
                                       const float* entropy, const float* grad_logprob, const float* grad_entropy,
                                       void* dlogits, int64_t ldd, void* stream);

/*
 * Scores tokens from hidden states: logits x = H W^T (bf16 inputs, fp32 accumulation) with temperature tau
 * (finite, and above 4.25e-39, from where log2(e) / tau is a float), in one pass of the tensor-core product whose
 * tiles are reduced where they are accumulated.
 *   H  bf16 [T][d], W bf16 [V][d], 16-byte aligned, d a multiple of 8
 *   tokens  int32 or int64 [T] (token_bytes 4 or 8);  mask uint8 [T] or NULL
 *   logprob, entropy, lse   float [T]; lse (natural log of sum_v exp(x_v / tau)) is written for every row,
 *           those left out included
 *   workspace   fkl_logprob_workspace_size bytes, 256-byte aligned
 * A logit that overflows to -inf has no weight; NaN or +inf among a row's logits makes its outputs NaN.  A token
 * outside [0, V) is recorded for fkl_read_status (FKL_ERR_BAD_TOPK_ID) beside its NaN; a wait that runs out
 * (FKL_ERR_TIMEOUT) makes every output NaN.
 *
 * fkl_logprob_forward_ex also writes `stats` (float [T][2], or NULL) for the backward: a reference logit m (one that is
 * at most 10 tau ln 2 below the row's largest) and log sum_v exp((x_v - m) / tau).  Its lse may be NULL.
 */
size_t fkl_logprob_workspace_size(int64_t T, int64_t d, int64_t V);
fkl_status fkl_logprob_forward(const uint16_t* H, const uint16_t* W, const void* tokens, int32_t token_bytes,
                               const uint8_t* mask, int64_t T, int64_t d, int64_t V, float tau, float* logprob,
                               float* entropy, float* lse, void* workspace, size_t ws_bytes, void* stream);
fkl_status fkl_logprob_forward_ex(const uint16_t* H, const uint16_t* W, const void* tokens, int32_t token_bytes,
                                  const uint8_t* mask, int64_t T, int64_t d, int64_t V, float tau, float* logprob,
                                  float* entropy, float* lse, float* stats, void* workspace, size_t ws_bytes,
                                  void* stream);

/*
 * The gradient of sum_t (a_t logprob_t + b_t entropy_t): dH [T][d] and dW [V][d], as float or, with
 * grad_bf16 = 1, as bfloat16 bit patterns (fp32 sums rounded once), 16-byte aligned.  One of them may be NULL:
 * its product is left out (a frozen head, say).  The logits are recomputed block by block as in fkl_backward, and
 * `chunk` bounds the buffer of their gradient: at most max(chunk * V, 256 * T) bfloat16 values, as a block is at least
 * one tile of 256 columns wide and may take all tokens (where chunk >= T: T * V, V rounded up to whole tiles).
 * Beside it the workspace holds 42 MB for partial tiles of dH, a bfloat16 copy of a block's hidden states, 24 bytes
 * for each row of the head and, for bfloat16 gradients, fp32 sums of dH and of dW where several blocks add to them and
 * of T / 5 rows of dW; it is sized for both gradients and a mask whether they are there or not.
 *   grad_logprob, grad_entropy   float [T]; NULL = 0
 *   logprob, entropy   the forward's
 *   lse, stats   the forward's; one of them may be NULL in fkl_logprob_backward_ex.  With `stats` q is right at any
 *           tau.  Without, it is taken from lse, whose rounding is 2^-24 |lse| of it: a row whose |lse| is above 2^15,
 *           where that passes the rounding of the logits' gradient to bf16 (logits of 30 below tau = 1e-3), has NaN
 *           gradients, unless it is left out or its a_t and b_t are 0
 *   accumulate   FKL_ACCUMULATE_DH and/or FKL_ACCUMULATE_DW add into float gradients (0 with grad_bf16)
 *   workspace    fkl_logprob_backward_workspace_size bytes, 256-byte aligned
 * A token outside [0, V) in a valid row (FKL_ERR_BAD_TOPK_ID) and a wait that runs out (FKL_ERR_TIMEOUT) fill
 * both gradients with NaN.
 */
size_t fkl_logprob_backward_workspace_size(int64_t T, int64_t d, int64_t V, int64_t chunk, int32_t grad_bf16);
fkl_status fkl_logprob_backward(const uint16_t* H, const uint16_t* W, const void* tokens, int32_t token_bytes,
                                const uint8_t* mask, const float* logprob, const float* entropy, const float* lse,
                                const float* grad_logprob, const float* grad_entropy, int64_t T, int64_t d, int64_t V,
                                float tau, int64_t chunk, int32_t grad_bf16, int32_t accumulate, void* dH, void* dW,
                                void* workspace, size_t ws_bytes, void* stream);
fkl_status fkl_logprob_backward_ex(const uint16_t* H, const uint16_t* W, const void* tokens, int32_t token_bytes,
                                   const uint8_t* mask, const float* logprob, const float* entropy, const float* lse,
                                   const float* stats, const float* grad_logprob, const float* grad_entropy, int64_t T,
                                   int64_t d, int64_t V, float tau, int64_t chunk, int32_t grad_bf16, int32_t accumulate,
                                   void* dH, void* dW, void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FKL_SCORE_H_ */
