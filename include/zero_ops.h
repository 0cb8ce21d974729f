/*
 * zero_ops.h -- C ABI of libzeroops.so: operators of a training step next to the
 * owner's step of zero_shard.h, on one gfx950 GPU:
 *  - layer norm, forward and backward with the weight's and bias's gradients;
 *  - root-mean-square norm with the residual's addition, forward (into storage or into
 *    8 bits with scales) and backward;
 *  - packing to 8 bits with a power of two for every 128 elements, and back; the matrix product
 *    of what is packed so;
 *  - softmax cross entropy over a vocabulary, from hidden states and the output
 *    weight, with both gradients under the loss scale and no logits in memory;
 *  - log probabilities of given tokens with entropy and top alternatives, from hidden states
 *    and the output weight, and their gradients;
 *  - AdamW over the tensors of a model at once, with moments in 32 or in 8 bits.
 * The gradients that they write are what a rank contributes to
 * zero_bucket_reduce (in the storage format, carrying the loss scale), or what
 * zero_adamw_step applies where a model's tensors are not one flat shard.
 *
 * Conventions, as in zero_shard.h:
 *  - Every function returns a zero_status.  Arguments are validated before
 *    anything is launched; on an error nothing is launched and no state changes.
 *    zero_ops_last_error() then holds a one-line explanation (thread-local).
 *  - No exceptions, aborts or prints cross this boundary.
 *  - Arrays are caller-owned memory of the current device, at any address
 *    aligned to their element; a written array must not overlap another array of
 *    the call unless the function says so.  Before a launch the library asks the
 *    HIP runtime about every array and refuses pageable host memory, another
 *    device's memory and ranges past the end of an allocation (best effort: the
 *    runtime sees allocations, not the tensors inside them).
 *  - Calls enqueue on `stream` (a hipStream_t as void*, NULL: the default stream),
 *    which must be of the current device, and do not synchronise unless they say
 *    so.  They launch kernels only and may be captured in a HIP graph.  A
 *    workspace belongs to one call at a time: calls that may overlap on the GPU
 *    need one each.  Its contents between calls mean nothing.
 *  - The same inputs give the same bits: no sum depends on an order of arrival.
 */
#ifndef ZERO_OPS_H
#define ZERO_OPS_H

#include "zero_shard.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ZERO_OPS_ABI_VERSION 1

/* ------------------------------------------------------------------ layer norm
 *
 * Over the last dimension of `rows` rows of `width` elements; row r of an array
 * begins at element r * stride (stride >= width).  type is the storage of x, y,
 * dy and dx; affine that of weight, bias and their gradients: type, or ZERO_FP32.
 *     mean = sum(x) / width ;  rstd = 1 / sqrt(sum((x - mean)^2) / width + eps)
 *     y = (x - mean) * rstd * weight + bias
 * in fp32, rounded to type once.  weight and bias may be NULL (1 and 0); mean and
 * rstd (fp32, one a row) may be NULL where no backward pass follows.  y may be x
 * (same address and stride).  rows = 0 does nothing.
 * Errors: INVALID_ARG (NULL x or y, unknown types, rows < 0, width < 1, stride <
 * width, eps < 0 or not finite, misaligned or overlapping arrays), UNSUPPORTED
 * (width > 2^24 or rows > 2^31 - 1), HIP.
 */
zero_status zero_layernorm_forward(const void* x, int64_t x_stride, const void* weight,
                                   const void* bias, int64_t rows, int64_t width,
                                   zero_lp_dtype type, zero_lp_dtype affine, double eps, void* y,
                                   int64_t y_stride, float* mean, float* rstd, void* stream);

/* Bytes of workspace zero_layernorm_backward needs for these sizes. */
zero_status zero_layernorm_workspace(int64_t rows, int64_t width, int64_t* bytes);

/*
 * The gradients for dy, with the forward pass's x, mean and rstd:
 *     xhat = (x - mean) * rstd ;  g = dy * weight
 *     dx = rstd * (g - mean(g) - xhat * mean(g * xhat))
 *     dweight = sum over rows of dy * xhat ;  dbias = sum over rows of dy
 * in fp32, rounded once.  dweight and dbias may each be NULL; with both NULL no
 * workspace is needed.  Both are written, not added to; with rows = 0 they are
 * zeros.  workspace is 16-byte aligned.
 * Errors: as zero_layernorm_forward; INVALID_ARG also for a workspace too small.
 */
zero_status zero_layernorm_backward(const void* dy, int64_t dy_stride, const void* x,
                                    int64_t x_stride, const void* weight, const float* mean,
                                    const float* rstd, int64_t rows, int64_t width,
                                    zero_lp_dtype type, zero_lp_dtype affine, void* dx,
                                    int64_t dx_stride, void* dweight, void* dbias, void* workspace,
                                    int64_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------ root-mean-square norm
 *
 * Over the last dimension, with the residual's addition in front of it:
 *     h = x + residual, rounded to type            (residual NULL: h is x, and the
 *                                                   argument h NULL)
 *     rstd = 1 / sqrt(sum(h^2) / width + eps) ;  y = h * rstd * weight
 * The sum, rstd and y are taken in 64 bits.  The result is y, rounded to fp32 and that to type; or
 * codes and exps, y in 8 bits as zero_scaled_pack holds numbers, rounded to them once; or both.  At least
 * one is given.
 * Row r of an array begins at element r * its stride; exps has a byte for every 128
 * elements of a row, ceil(width / 128) in all.  affine is the storage of weight: type or
 * ZERO_FP32; weight NULL is 1.  rstd (fp32, one a row) may be NULL.  h may be x or residual,
 * and y may be x (same address and stride).  rows = 0 does nothing.
 * Errors: INVALID_ARG (as zero_layernorm_forward, and eps above fp32's range; codes without exps
 * or the reverse, h without residual or the reverse, neither y nor codes), UNSUPPORTED (width >
 * 2^24 or rows > 2^31 - 1), HIP.
 */
typedef struct {
    int64_t rows, width;
    zero_lp_dtype type, affine;
    double eps;
    int64_t x_stride, residual_stride, h_stride, y_stride, codes_stride, exps_stride;
} zero_rmsnorm_desc;

zero_status zero_rmsnorm_forward(const zero_rmsnorm_desc* desc, const void* x, const void* residual,
                                 const void* weight, void* h, void* y, float* rstd, uint8_t* codes,
                                 uint8_t* exps, void* stream);

/* Bytes of workspace zero_rmsnorm_backward needs for these sizes. */
zero_status zero_rmsnorm_workspace(int64_t rows, int64_t width, int64_t* bytes);

/*
 * The gradients for dy, with the forward pass's h and rstd, and dh, what has come down to
 * h by other ways (NULL: nothing):
 *     xhat = h * rstd ;  g = dy * weight
 *     dx = rstd * (g - xhat * mean(g * xhat)) + dh ;  dweight = sum over rows of dy * xhat
 * in fp32, rounded once.  dx is the gradient of x and of residual alike; it may be dh.
 * dweight may be NULL (then no workspace is needed); it is written, not added to, and
 * zeros with rows = 0.  workspace is 16-byte aligned.
 * Errors: as zero_layernorm_backward.
 */
typedef struct {
    int64_t rows, width;
    zero_lp_dtype type, affine;
    int64_t dy_stride, h_stride, dh_stride, dx_stride;
} zero_rmsnorm_grad_desc;

zero_status zero_rmsnorm_backward(const zero_rmsnorm_grad_desc* desc, const void* dy, const void* h,
                                  const void* weight, const float* rstd, const void* dh, void* dx,
                                  void* dweight, void* workspace, int64_t workspace_bytes,
                                  void* stream);

/* ------------------------------------------------------------------ 8 bits with scales
 *
 * An element is an e4m3 number (a sign, 4 bits of exponent with bias 7, 3 of mantissa; largest
 * 448, 0x7f and 0xff NaN, no infinity) times 2^(E - 127), E a byte that 128 elements side by
 * side in a row have in common (the last block of a row may be shorter), or, square, 128
 * x 128 elements.  E = 255 is NaN.
 *
 * zero_scaled_pack takes x [rows][width] to codes [rows][width] and exps
 * [rows][ceil(width / 128)] (square: [ceil(rows / 128)][ceil(width / 128)]), to codes_t
 * [width][rows] and exps_t [width][ceil(rows / 128)] (square: [ceil(width / 128)][ceil(rows /
 * 128)]) of the transpose, or to both.  E is the least for which the block's largest finite
 * element is at most 448 * 2^(E - 127), but 27 at least; elements are rounded to the nearest,
 * ties to even, those that are not finite to NaN (and those above 1.875 * 2^127 to that, so that
 * none becomes infinite).  Square blocks have the same numbers in
 * both; others are rounded in each by its own scales.
 * rows = 0 or width = 0 does nothing.
 * Errors: INVALID_ARG (NULL x, codes without exps or the reverse, neither codes nor codes_t,
 * unknown type, sizes < 0, strides too small, square not 0 or 1, misaligned or overlapping
 * arrays), UNSUPPORTED (rows or width > 2^31 - 1, or more than 2^46 elements), HIP.
 */
zero_status zero_scaled_pack(const void* x, int64_t x_stride, int64_t rows, int64_t width,
                             zero_lp_dtype type, int32_t square, uint8_t* codes,
                             int64_t codes_stride, uint8_t* exps, int64_t exps_stride,
                             uint8_t* codes_t, int64_t codes_t_stride, uint8_t* exps_t,
                             int64_t exps_t_stride, void* stream);

/* What codes and exps stand for, rounded to type (exact in fp32 and bf16 for what
 * zero_scaled_pack writes).  Errors: as zero_scaled_pack. */
zero_status zero_scaled_unpack(const uint8_t* codes, int64_t codes_stride, const uint8_t* exps,
                               int64_t exps_stride, int64_t rows, int64_t width, int32_t square,
                               zero_lp_dtype type, void* out, int64_t out_stride, void* stream);

/*
 * The product of packed arrays, both with the depth along their rows:
 *     out[i][j] = sum over l of A[i][l] * B[j][l]  (+ bias[j])
 * for a [m][k] with a_exps [m][ceil(k / 128)] and b [n][k] with b_exps of either form, in fp32,
 * rounded to type (of out and bias) once; bias may be NULL.  For 2-byte results the products
 * are the card's 8-bit ones, which add 8 side by side to within 2^-13 of the largest of them (some
 * 1.5e-5 of a result, a tenth of fp16's rounding) and their sums in fp32; for fp32 results the
 * operands are taken as bf16, which holds their values exactly where scales are what zero_scaled_pack
 * writes (27 to 247; an element beyond fp32's range is infinite, one below bf16's normal
 * range may be 0), at half that rate.  With x packed along its rows
 * and w in squares, y = x w^T is (x, w); dx = dy w is (dy, codes_t of w); dw = dy^T x is
 * (codes_t of dy, codes_t of x), those two packed in blocks along their transposes' rows.
 * m = 0 or n = 0 does nothing; k = 0 gives bias, or zeros.
 * Performance: with more than 32 rows of a, an operand whose address or stride is no multiple of 4
 * bytes (or its stride above 2^22) is copied into the workspace first; for fp32 results both
 * are, as bf16.
 */
typedef struct {
    int64_t m, n, k;
    zero_lp_dtype type;
    int32_t b_square;            /* the form of b_exps */
    int64_t a_stride, a_exps_stride, b_stride, b_exps_stride, out_stride; /* elements a row */
} zero_scaled_product_desc;

/* Bytes of workspace (256-byte aligned) for these sizes and type of out.  Fewer rows may need
 * more: a workspace for several sizes is as large as the largest of their answers. */
zero_status zero_scaled_product_workspace(int64_t m, int64_t n, int64_t k, zero_lp_dtype type,
                                          int64_t* bytes);

/* Errors: INVALID_ARG (NULL or misaligned arrays, unknown type, sizes < 0, strides too small,
 * b_square not 0 or 1, workspace too small, overlaps), UNSUPPORTED (m or n > 2^31 - 1, m * n >
 * 2^40, k > 2^22, strides of exponents > 2^22), HIP. */
zero_status zero_scaled_product(const zero_scaled_product_desc* desc, const uint8_t* a,
                                const uint8_t* a_exps, const uint8_t* b, const uint8_t* b_exps,
                                const void* bias, void* out, void* workspace,
                                int64_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------ vocabulary loss
 *
 * hidden [tokens][width] and weight [vocab][width] of one 2-byte type, targets
 * int64, `counted` the number of targets that are not ignore_index:
 *     z = hidden weight^T ;  lse_n = log(sum_v exp(z_nv))
 *     losses_n = lse_n - z_n,target  (0 where the target is ignore_index)
 *     loss = sum(losses) / counted                      (0 where none counts)
 *     G_nv = (exp(z_nv - lse_n) - [v = target_n]) * grad_scale / counted
 *            (0 where the target is ignore_index)
 *     dhidden = G weight ;  dweight = G^T hidden
 * z, its sums and the results in fp32; G is held in 2 bytes between the products,
 * the gradients are rounded to type once.  grad_scale is the loss scale the
 * gradients carry (and 1 / Nd, or a weight of the micro-batch, where wanted).
 * dhidden and dweight are given both or neither (NULL: the loss alone); they
 * are written, not added to.  A token that is left out enters nothing but its own lse: its
 * hidden state need not be finite.  losses, lse and targets hold `tokens` elements;
 * lse may be NULL.  A target outside [0, vocab) that is not ignore_index gives
 * loss NaN and NaN gradients, which a checked step skips.
 * tokens = 0: loss 0, dweight zeros.
 * Tokens are taken max_tokens at a time (0: 8192), with the workspace's size in
 * proportion; the gradient of the weight is then summed in fp32 in the workspace.
 * Performance: both operands are copied into the workspace first where the width is
 * no multiple of 8, and either where its address is no multiple of 4 bytes or its
 * stride is odd.
 */
typedef struct {
    int64_t tokens, vocab, width;
    zero_lp_dtype type;          /* ZERO_FP16 or ZERO_BF16 */
    int64_t max_tokens;
    int64_t ignore_index;
    int64_t hidden_stride, weight_stride, dhidden_stride, dweight_stride; /* elements a row */
    double grad_scale;
} zero_vocab_loss_desc;

/* Bytes of workspace (256-byte aligned) for these sizes, without (gradient = 0)
 * or with the gradients.  Fewer tokens may need more (their products go in more parts): a
 * workspace for several counts is as large as the largest of their answers.  It has room for a
 * copy of both operands, also where none is made. */
zero_status zero_vocab_loss_workspace(int64_t tokens, int64_t vocab, int64_t width,
                                      int64_t max_tokens, int32_t gradient, int64_t* bytes);

/* Errors: INVALID_ARG (NULL or misaligned arrays, one gradient without the other,
 * sizes < 0, vocab or width < 1, strides < width, max_tokens outside [0, 65535],
 * grad_scale not finite in fp32, workspace too small, overlaps), UNSUPPORTED (ZERO_FP32;
 * width > 2^20, vocab > 2^21 - 64, tokens > 2^31 - 1), HIP. */
zero_status zero_vocab_loss(const zero_vocab_loss_desc* desc, const void* hidden, const void* weight,
                            const int64_t* targets, float* losses, float* lse, float* loss,
                            void* dhidden, void* dweight, void* workspace, int64_t workspace_bytes,
                            void* stream);

/* ------------------------------------------------------------------ log probabilities
 *
 * hidden [tokens][width] and weight [vocab][width] of one 2-byte type, ids int64, one a row:
 *     z = hidden weight^T ;  lse_n = log(sum_v exp(z_nv)) ;  p = exp(z - lse)
 *     logprobs_n = z_n,id - lse_n         (0 where the id is ignore_index, NaN where it is
 *                                          another outside [0, vocab))
 *     entropy_n = -sum_v p_nv log(p_nv)
 *     top_ids, top_logprobs [tokens][top]: the ids of the `top` largest z of a row in their
 *         order, of equal ones the lower id first, and z - lse of each; NaN ranks last
 * in fp32.  ids and logprobs are both given or both NULL, top_ids and top_logprobs where top > 0;
 * entropy may be NULL.  lse, entropy and alternatives are every row's, whatever its id.
 * tokens = 0 does nothing.  A row whose logits are all -infinity has lse -infinity and
 * NaN for the rest; one with a logit of +infinity or NaN has NaN.
 * Tokens are taken max_tokens at a time (0: 8192), with the workspace's size in proportion
 * (with alternatives: 4 bytes for each of a chunk's logits).
 * Performance: as zero_vocab_loss's operands.
 */
typedef struct {
    int64_t tokens, vocab, width;
    zero_lp_dtype type;          /* ZERO_FP16 or ZERO_BF16 */
    int32_t top;                 /* 0 to 64, and at most vocab */
    int64_t max_tokens;
    int64_t ignore_index;
    int64_t hidden_stride, weight_stride; /* elements a row */
} zero_token_logprobs_desc;

/* Bytes of workspace (256-byte aligned) for these sizes, of zero_token_logprobs (gradient = 0)
 * or of zero_token_logprobs_backward (1: top is not looked at).  A workspace for several counts
 * of tokens is as large as the largest of their answers. */
zero_status zero_token_logprobs_workspace(int64_t tokens, int64_t vocab, int64_t width,
                                          int64_t max_tokens, int32_t top, int32_t gradient,
                                          int64_t* bytes);

/* Errors: INVALID_ARG (NULL or misaligned arrays, one of a pair without the other, sizes < 0,
 * vocab or width < 1, strides < width, max_tokens outside [0, 65535], top outside [0, 64] or above
 * vocab, workspace too small, overlaps), UNSUPPORTED (ZERO_FP32; width > 2^20, vocab > 2^21 -
 * 64, tokens > 2^31 - 1), HIP. */
zero_status zero_token_logprobs(const zero_token_logprobs_desc* desc, const void* hidden,
                                const void* weight, const int64_t* ids, float* logprobs, float* lse,
                                float* entropy, int64_t* top_ids, float* top_logprobs,
                                void* workspace, int64_t workspace_bytes, void* stream);

/*
 * The gradients of sum(dlogprobs * logprobs) + sum(dentropy * entropy), with the forward pass's
 * lse and entropy:
 *     G_nv = dlogprobs_n * ([v = id_n] - p_nv) - dentropy_n * p_nv * (log(p_nv) + entropy_n)
 *     dhidden = G weight ;  dweight = G^T hidden
 * dentropy may be NULL (then entropy may be too).  dlogprobs of a row whose id is ignore_index is not
 * used; a row with neither gradient enters nothing, whatever its hidden state holds.  A row
 * whose id is another outside [0, vocab) has NaN gradients, and makes all of dweight NaN.  Both
 * results are written, not added to, and carry what scale dlogprobs and dentropy carry; dweight is
 * zeros with tokens = 0.
 * G is held in 2 bytes between the products, with the power of two that brings the largest row's
 * |dlogprobs| + |dentropy| (1 + log vocab) to the top of the range: in fp16 entries below 2^-39 of
 * that are lost.
 * Errors: as zero_token_logprobs.
 */
typedef struct {
    int64_t tokens, vocab, width;
    zero_lp_dtype type;
    int64_t max_tokens;
    int64_t ignore_index;
    int64_t hidden_stride, weight_stride, dhidden_stride, dweight_stride;
} zero_token_logprobs_grad_desc;

zero_status zero_token_logprobs_backward(const zero_token_logprobs_grad_desc* desc,
                                         const void* hidden, const void* weight, const int64_t* ids,
                                         const float* lse, const float* entropy,
                                         const float* dlogprobs, const float* dentropy,
                                         void* dhidden, void* dweight, void* workspace,
                                         int64_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------ AdamW over tensors
 *
 * One tensor: numel elements of gradient and parameter in the storage format `type`
 * (a param copy beside the fp32 master with the 2-byte formats; NULL, the master
 * being the parameter, with ZERO_FP32), and its moments:
 *  - state_bits 32: exp_avg and exp_avg_sq fp32, the _exp pointers NULL;
 *  - state_bits 8: exp_avg and exp_avg_sq one byte an element, and one int8 exponent
 *    for every block of 256 elements (the last may be shorter): an element stands
 *    for c * 2^e, c a small float: for exp_avg a sign, 4 bits of exponent and 3 of
 *    mantissa, for exp_avg_sq 5 and 3 bits.  With field f and mantissa k, c is
 *    (1 + k/8) * 2^(f - 15) or (f = 0) k * 2^-17 for exp_avg, and
 *    (1 + k/8) * 2^(f - 31) or k * 2^-33 for exp_avg_sq.  e = 127 marks a block
 *    that held a value not finite (or above 1.875 * 2^126): it stands for NaN.  No
 *    exponent is below -100: less is read as -100.  An exp_avg_sq below 2^-33 of its block's
 *    largest may be held as 0, and its element's next updates are then too large: gradients
 *    that differ by more than 2^15 within 256 elements want 32 bits.
 *    All bytes 0 are all zeros.
 * weight_decay < 0 takes the hyper-parameters'; the learning rate is lr * lr_scale.
 * Arrays must not overlap and must outlive the handle.
 */
typedef struct {
    int64_t numel;
    zero_lp_dtype type;
    const void* grad;
    float* master;
    void* param;
    void* exp_avg;
    void* exp_avg_sq;
    int8_t* exp_avg_exp;
    int8_t* exp_avg_sq_exp;
    double weight_decay;
    double lr_scale;
} zero_adamw_tensor;

typedef struct {
    int32_t state_bits;      /* 32 or 8 */
    int32_t checked;         /* 1: unscaled gradients are checked first; 0: applied as they are */
    double max_grad_norm;    /* > 0: clip to this global norm (needs checked); 0: off */
    uint64_t seed;           /* of the random rounding of 8-bit moments */
} zero_adamw_cfg;

typedef struct zero_adamw_s* zero_adamw_t; /* opaque */

/*
 * A handle over n tensors.  Allocates a table of them (device memory) and a few
 * KB; copies the table, synchronously.  hp and ls as for zero_shard_init: the step
 * counter and the loss scale live in device memory.
 * Errors: INVALID_ARG (NULL, n < 1, numel < 0, a tensor's arrays NULL, misaligned
 * or not those of its state_bits and type, overlaps, values out of range,
 * max_grad_norm without checked), UNSUPPORTED (n > 2^20, more than 2^38 elements),
 * OOM, HIP.
 */
zero_status zero_adamw_init(const zero_adamw_tensor* tensors, int32_t n, const zero_adam_hparams* hp,
                            const zero_loss_scale_cfg* ls, const zero_adamw_cfg* cfg,
                            zero_adamw_t* out);

/* Other gradient arrays, one for each tensor of the handle, from the next step on
 * `stream` on (an enqueue, 256 pointers a launch).  As at init, they must not overlap an
 * array that the step writes; the old ones must outlive the steps that read them.
 * Errors: STATE, INVALID_ARG (NULL, n not the handle's, misaligned, overlaps), HIP. */
zero_status zero_adamw_set_grads(zero_adamw_t h, const void* const* grads, int32_t n, void* stream);

/*
 * Enqueue one step of every tensor.  checked: the squared norm of the unscaled
 * gradients g = f32(grad) * fp32(1/scale) over all tensors (fp64, fixed order)
 * decides as in the device-resident flow of zero_shard.h: one that is not finite
 * skips the step and, with dynamic scaling, halves the scale; clean steps advance
 * t, and coef = min(1, max_grad_norm / (norm + 1e-6)) multiplies g.  Then, per
 * element, the update of zero_adam_step, bit for bit.  With 8-bit moments the
 * update uses m and v before they are held; what is held are they, rounded up or
 * down at random in proportion (16 random bits each, a hash of seed, t, the
 * tensor's index and the element's).
 * hp = NULL: the init values; otherwise *hp is this step's (its betas must be the
 * init's, its initial_step is ignored).  Not with hp = NULL or otherwise is anything
 * read back: see zero_adamw_result.  A captured step replays with its hp.
 * Errors: STATE (dead handle, another device current), INVALID_ARG, HIP.
 */
zero_status zero_adamw_step(zero_adamw_t h, const zero_adam_hparams* hp, void* stream);

/* The last step's result (grad_norm 0 for a step that was not checked).
 * Synchronises `stream`. */
zero_status zero_adamw_result(zero_adamw_t h, void* stream, zero_step_info* out);

/* Step counter, loss scale and clean steps (synchronises `stream`); and back. */
zero_status zero_adamw_get_counters(zero_adamw_t h, void* stream, int64_t* step_t, double* scale,
                                    int64_t* good_steps);
zero_status zero_adamw_set_counters(zero_adamw_t h, void* stream, int64_t step_t, double scale,
                                    int64_t good_steps);

/* Release the handle's memory, after its work has ended (synchronises the device).
 * The caller's arrays are untouched.  A second destroy returns ZERO_ERR_STATE. */
zero_status zero_adamw_destroy(zero_adamw_t h);

/*
 * Between fp32 (or, out, bf16: it holds every such value exactly) and 8-bit moments
 * as above: n elements in blocks of 256, is_signed 1 for exp_avg's format and 0 for
 * exp_avg_sq's (whose negative inputs become 0).  pack rounds to the nearest (a value within
 * 2^-17 of a step above the middle goes down).
 * Errors: INVALID_ARG (NULL with n > 0, n < 0, is_signed not 0 or 1, out_type neither
 * ZERO_FP32 nor ZERO_BF16, misaligned or overlapping arrays), HIP.
 */
zero_status zero_moments_pack(const float* x, int64_t n, int32_t is_signed, uint8_t* codes,
                              int8_t* exps, void* stream);
zero_status zero_moments_unpack(const uint8_t* codes, const int8_t* exps, int64_t n,
                                int32_t is_signed, zero_lp_dtype out_type, void* out, void* stream);

const char* zero_ops_last_error(void);
int zero_ops_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* ZERO_OPS_H */
