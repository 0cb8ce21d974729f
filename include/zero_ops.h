/*
 * zero_ops.h -- C ABI of libzeroops.so: operators of a training step next to the
 * owner's step of zero_shard.h, on one gfx950 GPU:
 *  - layer norm, forward and backward with the weight's and bias's gradients;
 *  - softmax cross entropy over a vocabulary, from hidden states and the output
 *    weight, with both gradients under the loss scale and no logits in memory;
 *  - AdamW over the tensors of a model at once, with moments in 32 or in 8 bits.
 * The gradients that the first two write are what a rank contributes to
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
