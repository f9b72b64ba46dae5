/*
 * scape_layers.h -- C ABI of the training-layer operators on one GB300 (sm_103a).
 *
 * A sharded optimizer step reads W workers' gradients; these operators produce
 * them on the same GPU: the residual RMS norm, activation checkpoints in
 * 8 bits, and the linear layer with its gradients.  What the backward pass
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

#ifdef __cplusplus
}
#endif

#endif /* SCAPE_LAYERS_H */
