/*
 * scape_layers.h -- C ABI of the training-layer operators on one GB300 (sm_103a).
 *
 * A sharded optimizer step reads W workers' gradients; these operators produce
 * them on the same GPU: the residual RMS norm, activation checkpoints in
 * 8 bits, and the linear layer with its gradients; at the two ends of a language
 * model the embedding and the log probabilities of tokens, with theirs; and before
 * the step the gradients' norm and clipping.  What the backward pass
 * keeps of a layer is 8 bits a value, because the workers' residuals
 * (scape_bind()) take most of the device's memory; weight gradients are written
 * where the caller wants them, e.g. into the flat vector scape_step() reads.
 *
 * Conventions for every entry point
 *   - Return value: SCAPE_OK or a negative scape_status (scape.h).  Nothing
 *     throws across the ABI.  scape_layer_last_error() gives the message of the
 *     calling thread's last failure.
 *   - Pointers are device pointers; the caller owns every buffer.  Nothing is
 *     allocated.  Where an entry point takes a workspace, its *_workspace
 *     function gives the bytes (0: NULL will do); the workspace is 256-byte
 *     aligned, is free for other use once the call's work is done, and holds
 *     nothing between calls.
 *   - `stream` is a cudaStream_t passed as void*; all work is enqueued on it.
 *     Calls can be captured into a CUDA graph.
 *   - Matrices are row-major with unit column stride and a row stride (ld*,
 *     in elements, at least the number of columns).  Any alignment and any
 *     stride is accepted.  Outputs that share memory with an input or with each
 *     other are refused, but where one "may be" an input: the same address and
 *     stride then.  (Slices of a wider buffer may lie between each other.)
 *     Rows or columns of zero length are valid and do nothing (a weight
 *     gradient of no rows is zero).
 *   - dtype arguments are scape_dtype (SCAPE_F32, SCAPE_BF16).  Sums, norms and
 *     products are held in 32 bits and rounded once, when they are stored.  The
 *     32-bit sums of a product (more than a few rows) are the tensor cores', which
 *     cut what does not fit instead of rounding it: sums come out too near 0, by
 *     1e-6 of themselves for a contraction of 1024 and 2e-5 for 65536 (normally
 *     distributed operands; a chain of rounded 32-bit sums: 3e-7 and 6e-7, to
 *     either side).  Results of an activation or its slope below 2^-110 may be 0.
 *   - Results do not depend on timing: equal calls give equal bits.
 *
 * 8-bit format.  Each row is cut into blocks of 32 consecutive columns (the
 * last may be shorter).  A block holds one scale byte `code`, meaning
 * 2^(code - 127), and e4m3 values q (4 exponent bits, 3 fraction bits, largest
 * 448), x ~ q 2^(code - 127): code is the smallest value >= 1 for which the
 * block's largest finite magnitude is at most 448 2^(code - 127); q is rounded
 * to nearest even.  Infinities and NaN become NaN and do not affect the rest of
 * their block.  Scales are uint8, ceil(cols / 32) contiguous bytes a row; codes
 * written are 1 to 247, and 0 and 255 are not read as powers of two.
 * A power-of-two scale makes every q 2^(code - 127) exact in bfloat16 and float32
 * but for the ends of their range.  At code 247 a magnitude of 248 2^120 (3.3e38) on
 * rounds to q = 256, which stands for 2^128 and is read as infinity; at codes 1 and
 * 2 the least values, odd multiples of 2^-135 and 2^-134, are read in bfloat16 as
 * the nearest multiple of 2^-133, its smallest step.
 */
#ifndef SCAPE_LAYERS_H
#define SCAPE_LAYERS_H

#include "scape.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SCAPE_PACK_BLOCK 32

/* Activations: identity; max(z, 0); 0.5 z (1 + tanh(sqrt(2/pi) (z + 0.044715
 * z^3))); z / (1 + exp(-z)).  The slope of relu at 0 is 0. */
enum scape_activation {
    SCAPE_ACT_NONE = 0,
    SCAPE_ACT_RELU = 1,
    SCAPE_ACT_GELU = 2,
    SCAPE_ACT_SILU = 3
};

/* Message of the calling thread's last failed scape_layer_* call ("" if none). */
const char *scape_layer_last_error(void);

/*
 * Waits that kernels on the current device have given up since the last call, by
 * any thread (every wait inside the matrix-product kernels ends after a time
 * limit; a kernel that gave up leaves its output incomplete, and the call that
 * launched it returned SCAPE_OK).  0 = none, for all work before it on `stream`,
 * which it synchronises.
 */
int scape_layer_status(int *host_status, void *stream);

/*
 * Launches a kernel that waits limit_ns (1 ns to 2 s) for something that does not
 * come, then gives up as a product kernel does.  It writes nothing else.  For
 * tests of a program's handling of scape_layer_status().
 */
int scape_layer_probe_wait(int64_t limit_ns, void *stream);

/* x[rows, cols] -> q[rows, cols], scale[rows, ceil(cols / 32)]. */
int scape_layer_pack8(const void *x, int64_t ldx, int dtype, int64_t rows, int64_t cols,
                      uint8_t *q, int64_t ldq, uint8_t *scale, void *stream);

/* y = act(values of (q, scale)), in dtype. */
int scape_layer_unpack8(const uint8_t *q, int64_t ldq, const uint8_t *scale, int64_t rows,
                        int64_t cols, int activation, void *y, int64_t ldy, int dtype,
                        void *stream);

/* dz = dy * act'(values of (q, scale)): the gradient through an activation
 * whose input was kept in 8 bits.  dz may be dy. */
int scape_layer_act_grad(const void *dy, int64_t lddy, const uint8_t *q, int64_t ldq,
                         const uint8_t *scale, int64_t rows, int64_t cols, int activation,
                         void *dz, int64_t lddz, int dtype, void *stream);

/*
 * h = x + residual (h = x when residual is NULL);  rstd = (mean h^2 + eps)^-1/2
 * y = h * rstd * weight.  x, residual, h and y are of dtype; weight (cols) is of
 * weight_dtype; rstd is float32, one a row.  h, rstd, and the 8-bit form of y
 * (q, scale; rounded from the 32-bit y) may be NULL; h may be x or residual.
 */
int scape_layer_add_rmsnorm(const void *x, int64_t ldx, const void *residual, int64_t ldres,
                            const void *weight, int weight_dtype, int64_t rows, int64_t cols,
                            float eps, int dtype, void *y, int64_t ldy, void *h, int64_t ldh,
                            float *rstd, uint8_t *q, int64_t ldq, uint8_t *scale, void *stream);

/*
 * Its gradient, from h and rstd: n = h * rstd, d = dy * weight,
 *   dx = rstd * (d - n * mean(d * n)) + dh,   dweight = sum over rows of dy * n.
 * dh is the gradient that reaches h from elsewhere (NULL: none); dx is the
 * gradient of x and of residual alike.  dweight (cols, of dweight_dtype) may be
 * NULL.  dx may be dy or dh.
 */
int scape_layer_add_rmsnorm_bwd_workspace(int64_t rows, int64_t cols, size_t *bytes);
int scape_layer_add_rmsnorm_bwd(const void *dy, int64_t lddy, const void *h, int64_t ldh,
                                const void *weight, int weight_dtype, const float *rstd,
                                const void *dh, int64_t lddh, int64_t rows, int64_t cols,
                                int dtype, void *dx, int64_t lddx, void *dweight,
                                int dweight_dtype, void *workspace, size_t ws_bytes,
                                void *stream);

/*
 * z = x weight^T + bias;  y = act(z) + residual;  all bfloat16.
 * x[rows, k], weight[n, k], bias[n] or NULL, residual[rows, n] or NULL,
 * y[rows, n]; q, scale (the 8-bit form of z, rounded from 32 bits) may be NULL.
 * y may be residual.  k >= 1.
 */
int scape_layer_linear_workspace(const void *x, int64_t ldx, const void *weight, int64_t ldw,
                                 int64_t rows, int64_t k, int64_t n, size_t *bytes);
int scape_layer_linear(const void *x, int64_t ldx, const void *weight, int64_t ldw,
                       const void *bias, const void *residual, int64_t ldres, int64_t rows,
                       int64_t k, int64_t n, int activation, void *y, int64_t ldy, uint8_t *q,
                       int64_t ldq, uint8_t *scale, void *workspace, size_t ws_bytes,
                       void *stream);

/*
 * dx = (dy weight) * act'(values of (q, scale)): the gradient of a linear
 * layer's input, taken on through the activation that made that input, whose
 * own input was kept in 8 bits (activation SCAPE_ACT_NONE: q, scale unused).
 * dy[rows, n], weight[n, k], q[rows, k], dx[rows, k]; bfloat16.  n >= 1.
 */
int scape_layer_linear_bwd_input_workspace(const void *dy, int64_t lddy, const void *weight,
                                           int64_t ldw, int64_t rows, int64_t k, int64_t n,
                                           size_t *bytes);
int scape_layer_linear_bwd_input(const void *dy, int64_t lddy, const void *weight, int64_t ldw,
                                 const uint8_t *q, int64_t ldq, const uint8_t *scale,
                                 int activation, int64_t rows, int64_t k, int64_t n, void *dx,
                                 int64_t lddx, void *workspace, size_t ws_bytes, void *stream);

/*
 * dweight = dy^T a, dbias = sum over rows of dy, for the layer input
 * a[rows, k]: either x (bfloat16; q NULL), or act(values of (q, scale)) (x
 * NULL).  a is rounded to bfloat16, as the forward pass used it.
 * dweight[n, k] and dbias[n] (or NULL) are of grad_dtype.
 */
int scape_layer_linear_bwd_weight_workspace(const void *dy, int64_t lddy, const void *x,
                                            int64_t ldx, int64_t rows, int64_t k, int64_t n,
                                            size_t *bytes);
int scape_layer_linear_bwd_weight(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                                  const uint8_t *q, int64_t ldq, const uint8_t *scale,
                                  int activation, int64_t rows, int64_t k, int64_t n,
                                  void *dweight, int64_t lddw, void *dbias, int grad_dtype,
                                  void *workspace, size_t ws_bytes, void *stream);

/*
 * Which kernels the current device runs for a product of these sizes (an answer for
 * profiling and tests; nothing is launched).  kernel: one of scape_linear_kernel;
 * columns: of a tile (0: no tiles); cluster: blocks that share a tile's
 * contraction (0: one each).  keeps_8bit: the forward product also stores z in 8 bits.
 */
enum scape_linear_product {
    SCAPE_LINEAR_FORWARD = 0,
    SCAPE_LINEAR_INPUT_GRAD = 1,
    SCAPE_LINEAR_WEIGHT_GRAD = 2
};
enum scape_linear_kernel {
    SCAPE_PLAN_FEW_ROWS = 0,       /* without tensor cores */
    SCAPE_PLAN_SPLIT = 1,          /* tiles of 128 rows */
    SCAPE_PLAN_PAIRS = 2,          /* tiles of 256 rows by pairs of blocks */
    SCAPE_PLAN_PAIRS_AND_SPLIT = 3 /* whole rounds of those, the tiles left over split */
};
int scape_layer_linear_plan(int product, int64_t rows, int64_t k, int64_t n, int keeps_8bit,
                            int *kernel, int *columns, int *cluster);

/* ---------------------------------------------------------------- tokens
 * Tokens (and targets) are int32 or int64 (token_bytes 4 or 8).  One below 0 stands
 * for none; one that is not below vocab is never used as an index, and what is
 * computed for it is NaN.  A row has at most 2^30 columns.
 */

/*
 * y[i] = scale * weight[tokens[i]], zeros where the token is none.  weight[vocab, cols]
 * is of weight_dtype, y[count, cols] of dtype.  vocab >= 1.
 */
int scape_layer_embedding(const void *tokens, int token_bytes, int64_t count, const void *weight,
                          int64_t ldw, int weight_dtype, int64_t vocab, int64_t cols, float scale,
                          void *y, int64_t ldy, int dtype, void *stream);

/*
 * dweight[v] = scale * sum of dy[i] over the i with tokens[i] = v, in an order fixed
 * by the tokens alone.  accumulate 0: rows without a token become zeros; else the
 * sum is added to dweight (in 32 bits, rounded once) and rows without a token are
 * left alone, for a table that is also the output layer's weight.  Tokens that are
 * none or out of range contribute nothing.
 */
int scape_layer_embedding_bwd_workspace(int64_t count, int64_t vocab, int64_t cols, size_t *bytes);
int scape_layer_embedding_bwd(const void *dy, int64_t lddy, int dtype, const void *tokens,
                              int token_bytes, int64_t count, int64_t vocab, int64_t cols,
                              float scale, int accumulate, void *dweight, int64_t lddw,
                              int dweight_dtype, void *workspace, size_t ws_bytes, void *stream);

/*
 * Of logits x[rows, vocab] (dtype), a row at a time:
 *   lse = log sum_j exp x_j;  logprob = x_target - lse (0 where the target is none);
 *   entropy = -sum_j p_j log p_j with p_j = exp(x_j - lse);
 *   the `top` (0 to SCAPE_TOP_MAX, at most vocab) largest logits in falling order,
 *   of equal ones the lowest column first: their columns and log probabilities.
 * A logit of -infinity has p = 0 and adds nothing; in a row of nothing else lse is
 * -infinity, the entropy 0 and every log probability -infinity.  NaN or +infinity in
 * a row makes its results NaN (NaN is last among the alternatives, whose columns
 * are still distinct).  entropy, top_logprob and top_token [rows, top] may be NULL
 * (the last two together).
 */
#define SCAPE_TOP_MAX 32
#define SCAPE_TOP_VOCAB_MAX 4194304 /* columns, where alternatives are asked for */
int scape_layer_token_logprobs(const void *logits, int64_t ldx, int dtype, const void *targets,
                               int token_bytes, int64_t rows, int64_t vocab, int top,
                               float *logprob, float *lse, float *entropy, float *top_logprob,
                               int64_t *top_token, void *stream);
/*
 * The same with the log-sum-exp in two numbers, lse + lse_rest [rows]: lse_rest is what
 * lse's rounding to 32 bits leaves (0 where lse is not finite).  NULL: not wanted.
 */
int scape_layer_token_logprobs_rest(const void *logits, int64_t ldx, int dtype, const void *targets,
                                    int token_bytes, int64_t rows, int64_t vocab, int top,
                                    float *logprob, float *lse, float *lse_rest, float *entropy,
                                    float *top_logprob, int64_t *top_token, void *stream);

/*
 * dlogits_j = dlogprob (1[j = target] - p_j) - dentropy p_j (log p_j + entropy), from
 * what the forward call gave.  dentropy NULL: its term is left out (entropy is then
 * not read); a row whose target is none is then zeros, whatever its logits.  dlogits
 * may be logits.
 */
int scape_layer_token_logprobs_bwd(const void *logits, int64_t ldx, int dtype, const void *targets,
                                   int token_bytes, int64_t rows, int64_t vocab, const float *lse,
                                   const float *dlogprob, const float *entropy,
                                   const float *dentropy, void *dlogits, int64_t lddx,
                                   void *stream);
/*
 * The same from a log-sum-exp of two numbers.  From lse alone p_j = exp(x_j - lse) is off
 * by lse's rounding, 2^-24 |lse| of itself, and 1 - p_target, where it is that small, is
 * lost (from |lse| = 4096 on the sums of a row are formed again, and it is slower).  With
 * lse_rest it is the softmax's wherever the logits lie.  NULL: lse alone.
 */
int scape_layer_token_logprobs_rest_bwd(const void *logits, int64_t ldx, int dtype,
                                        const void *targets, int token_bytes, int64_t rows,
                                        int64_t vocab, const float *lse, const float *lse_rest,
                                        const float *dlogprob, const float *entropy,
                                        const float *dentropy, void *dlogits, int64_t lddx,
                                        void *stream);

/*
 * A row's loss and its gradient in one pass over the logits:
 *   loss = -w logprob;  dlogits_j = w (p_j - 1[j = target]),
 * w = weight[row], or weight_all for every row where weight is NULL.  Both are 0 where
 * the target is none, whatever the logits.  dlogits may be logits.
 */
int scape_layer_token_loss_workspace(const void *logits, int64_t ldx, int dtype, int64_t rows,
                                     int64_t vocab, const void *dlogits, int64_t lddx,
                                     size_t *bytes);
int scape_layer_token_loss(const void *logits, int64_t ldx, int dtype, const void *targets,
                           int token_bytes, int64_t rows, int64_t vocab, const float *weight,
                           float weight_all, float *loss, void *dlogits, int64_t lddx,
                           void *workspace, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------- gradients
 * n tensors of host_numel[i] contiguous elements of host_dtype[i].  The host arrays
 * are read during the call only.
 */

/*
 * norm = sqrt(sum over all tensors of the elements' squares), one float32.  The sum
 * is held in 64 bits above short 32-bit ones, and squares outside float32's range are
 * scaled, so it neither overflows nor loses small gradients (a norm past float32's
 * largest is infinity).  NaN or an infinity among the elements makes it NaN or infinite.
 */
int scape_layer_grad_norm_workspace(int n, const int64_t *host_numel, size_t *bytes);
int scape_layer_grad_norm(int n, const void *const *host_grads, const int64_t *host_numel,
                          const int *host_dtype, float *norm, void *workspace, size_t ws_bytes,
                          void *stream);

/*
 * The norm, and out[i] = grads[i] * min(1, max_norm / (norm + eps)), each of
 * host_out_dtype[i].  host_out NULL: in place; out[i] may be grads[i] (same type).
 * max_norm >= 0, eps >= 0.  The factor is used as it comes out of the norm in 64 bits:
 * NaN where an element is, 0 where one is infinite, and NaN for 0 / 0 (max_norm, the
 * norm and eps all 0) or infinity / infinity.
 */
int scape_layer_clip_grads(int n, const void *const *host_grads, const int64_t *host_numel,
                           const int *host_dtype, void *const *host_out,
                           const int *host_out_dtype, float max_norm, float eps, float *norm,
                           void *workspace, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SCAPE_LAYERS_H */
