/*
 * fkl_generate.h - C ABI of the generation operators: the LM head (or any projection) in
 * 8-bit integers, and the sampler that draws a token from its logits.
 *
 * On-policy distillation trains a student on text that it (or its teacher) has drawn.  One
 * generation step projects a few hidden states through the LM head and draws a token per
 * row; the weights, which such a step does little more than read, are held in 8-bit integers
 * with one scale per output channel, and the hidden states are brought to 8 bits with one
 * scale per token.
 *
 *     quantise   s_m = max_k |x_mk| * fl(1/127) (fp32),  q_mk = round(x_mk / s_m) to nearest even
 *     product    y_mn = (sum_k q_mk w_nk) * s_m * t_n
 *     sample     see fkl_sample
 *
 * Conventions (device pointers, streams, errors, ownership) are those of fkl.h: the library
 * allocates no device memory, never synchronises, refuses bad arguments on the host before
 * anything is enqueued, and gives the same bits for the same inputs.  None of the operators
 * has a gradient: the weights are fixed while text is drawn, and a draw has none.
 */
#ifndef FKL_GENERATE_H_
#define FKL_GENERATE_H_

#include <stddef.h>
#include <stdint.h>

#include "fkl.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of hidden states, outputs and logits. */
enum { FKL_TYPE_F32 = 0, FKL_TYPE_BF16 = 1, FKL_TYPE_F16 = 2 };

/*
 * Brings each row of x to 8-bit integers: with a_m the largest magnitude of row m,
 *     scale[m] = a_m * fl(1/127),   q[m][k] = round(x[m][k] / scale[m]) in [-127, 127]
 * (IEEE division and rounding to nearest even, so the integers are reproducible).  A row of
 * zeros has scale 0 and zeros; a row that holds a NaN or an infinity has scale NaN and zeros,
 * which makes every output of the product in that row NaN.
 *   x      [rows][cols] of type x_type, rows `ldx` elements apart (ldx >= cols)
 *   q      int8 [rows][cols], contiguous
 *   scale  float [rows]
 * x is aligned to its element size, q has no alignment rule (16-byte aligned rows of both are
 * read and written with vectors).  0 <= rows < 2^31, 1 <= cols < 2^31.
 * Used for the tokens of a call and, once, for a weight: a row is then an output channel.
 */
fkl_status fkl_quantize_int8(const void* x, int32_t x_type, int64_t rows, int64_t cols, int64_t ldx, int8_t* q,
                             float* scale, void* stream);

/*
 * Product of 8-bit integers with a scale per token and per channel:
 *     out[m][n] = (sum_k xq[m][k] * wq[n][k]) * x_scale[m] * w_scale[n]
 * rounded once to out_type.  The sum is exact while its partial sums stay below 2^24 in
 * magnitude (always for K <= 1024), and for up to 4 tokens with K <= 24576.  Beyond, each 16-deep step
 * of the tensor cores' fp32 accumulation loses at most 2^-23 of the partial sum.
 *   xq int8 [M][K], x_scale float [M]; wq int8 [N][K], w_scale float [N]; all contiguous
 *   out [M][N] of type out_type, rows `ldo` elements apart (ldo >= N), aligned to its type
 * xq and wq are 16-byte aligned and K is a multiple of 16 (rows are whole 16-byte units).
 * 0 <= M <= 2^31 - 512, 1 <= N <= 2^31 - 512, 16 <= K <= 131072.  Any value of int8, -128 included.
 * The kernel's waits are limited (5 s each).  Should one run out, the outputs that are not finished are
 * NaN and fkl_read_status(workspace, stream) returns FKL_ERR_TIMEOUT until the workspace's next
 * call; fkl_sample draws -1 from such a row when all of it is NaN.
 */
/* Bytes for this shape on the current device.  Not monotone: partial sums are kept only for shapes
 * whose tiles are cut along K, so a buffer for several shapes takes the largest of their sizes. */
size_t fkl_int8_matmul_workspace_size(int64_t M, int64_t N, int64_t K);
fkl_status fkl_int8_matmul(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale, int64_t M,
                           int64_t N, int64_t K, int32_t out_type, void* out, int64_t ldo, void* workspace,
                           size_t ws_bytes, void* stream);

/*
 * fkl_quantize_int8 of the hidden states followed by fkl_int8_matmul, the call of a
 * generation step: x [M][K] of type x_type, rows `ldx` elements apart (ldx >= K).
 */
size_t fkl_int8_linear_workspace_size(int64_t M, int64_t N, int64_t K);
fkl_status fkl_int8_linear(const void* x, int32_t x_type, int64_t ldx, const int8_t* wq, const float* w_scale,
                           int64_t M, int64_t N, int64_t K, int32_t out_type, void* out, int64_t ldo, void* workspace,
                           size_t ws_bytes, void* stream);

/*
 * Settings of fkl_sample: each as one value for all rows, or (where the pointer is not
 * NULL) as a device array with a value per row.
 *   temperature   T > 0; any other value (0, negative, NaN) takes the largest logit
 *   top_k         keep the k largest logits; k <= 0 or k > V keeps all
 *   top_p         of those, keep the smallest set of largest logits that holds at least this
 *                 share of their probability (always the largest one); >= 1 keeps all
 *   min_p         of those, keep the ones at least min_p times as probable as the largest
 *                 (always the largest); <= 0 keeps all
 */
typedef struct fkl_sample_params {
  float temperature;
  int32_t top_k;
  float top_p;
  float min_p;
  const float* temperature_rows;
  const int32_t* top_k_rows;
  const float* top_p_rows;
  const float* min_p_rows;
} fkl_sample_params;

/*
 * Draws one token per row from given uniform random numbers.  For row b, with m its largest
 * logit,
 *     z_v = (x_v - m) * fl(1/T)  (0 where x_v = m),  w_v = floor(2^40 exp(z_v))
 * The weights are whole numbers, so every sum of them is exact and independent of its order.
 * Logits are ranked by value, ties by the lower id; the three filters of fkl_sample_params
 * are applied in their order (top_p: id v stays if the weight ranked before it is below
 * ceil(top_p * total), in double).  With W the kept weight and r = floor(u * W) (in double,
 * limited to [0, W - 1]) the token is the first id, in the order of ids, at which the running
 * kept weight exceeds r, and logprob = z_token - log(2^-40 W), its log-probability among the
 * kept ids.
 *   logits   [B][V] of `type`, rows `ld` elements apart (ld >= V), aligned to the type; -inf
 *            bans an id, NaN counts as -inf, +inf ids share all the probability
 *   u        float [B] in [0, 1)
 *   token    int32 [B];  logprob  float [B] or NULL
 * A row with nothing to draw (every logit -inf or NaN) gets token -1 and logprob NaN; the
 * other rows are unaffected.  0 <= B < 2^31, 1 <= V <= 2^22.
 */
fkl_status fkl_sample(const void* logits, int32_t type, int64_t B, int64_t V, int64_t ld, const float* u,
                      const fkl_sample_params* params, int32_t* token, float* logprob, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FKL_GENERATE_H_ */
