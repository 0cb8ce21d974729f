// Launch interface between the operators' C ABI (zero_ops.cpp) and their kernels.
// Arguments are checked by the caller.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace zo {

// Storage codes are the public header's: 1 fp16, 2 bf16, 3 fp32.

// ------------------------------------------------------------------ layer norm

struct NormForward {
    const void* x;
    const void* weight;
    const void* bias;
    void* y;
    float* mean;
    float* rstd;
    int64_t rows, width, x_stride, y_stride;
    float eps;
};

struct NormBackward {
    const void* dy;
    const void* x;
    const void* weight;
    const float* mean;
    const float* rstd;
    void* dx;
    void* dweight;
    void* dbias;
    float* partial;       // norm_partial_rows() rows of 2 * width
    int64_t rows, width, dy_stride, x_stride, dx_stride;
};

int64_t norm_partial_rows(int64_t rows, int64_t width);
hipError_t norm_forward(const NormForward& a, int type, int affine, hipStream_t s);
hipError_t norm_backward(const NormBackward& a, int type, int affine, hipStream_t s);

// ------------------------------------------------------------------ vocabulary loss

struct TileChoice {            // of the products: 32 ni x 64 nj results a workgroup
    int ni, nj;
};

struct LossPlan {              // what a call's sizes settle
    int64_t tokens, vocab, width;
    int64_t chunk;             // tokens whose exponentials are held at once
    int64_t vocab_ld;          // their row stride
    int64_t pieces;            // of a token's ids, with statistics each
    int64_t width_ld;          // the width in whole chunks of 8
    TileChoice logits_tile, hidden_tile, weight_tile;
    int hidden_splits, weight_splits;      // parts of the gradients' products
    bool pairs;                // an entry of G is held as two numbers
    // byte offsets into the workspace
    int64_t off_alpha, off_target, off_lse, off_stats, off_exp, off_split, off_sum, off_hidden, off_weight;
    int64_t bytes;
};

struct Loss {
    const void* hidden;
    const void* weight;
    const int64_t* targets;
    float* losses;
    float* lse;
    float* loss;
    void* dhidden;
    void* dweight;
    char* space;
    int64_t hidden_stride, weight_stride, dhidden_stride, dweight_stride;
    int64_t ignore_index;
    double grad_scale;
};

LossPlan loss_plan(int64_t tokens, int64_t vocab, int64_t width, int64_t max_chunk, bool gradient);
hipError_t vocab_loss(const Loss& a, const LossPlan& p, int type, hipStream_t s);

// ------------------------------------------------------------------ AdamW over tensors

constexpr int kStateBlock = 256;       // elements that share an exponent (8-bit states)

struct TensorEntry {           // device table, one a tensor
    const void* grad;
    float* master;
    void* param;
    void* m;
    void* v;
    int8_t* m_exp;
    int8_t* v_exp;
    int64_t numel;
    float weight_decay;
    float lr_scale;
    int32_t type;              // storage code
    int32_t pad;
};

struct ChunkEntry {            // device table, one a workgroup of the update
    int32_t tensor;
    int32_t pad;
    int64_t begin;             // first element of the tensor
};

struct AdamwState {            // in device memory
    double sumsq;              // of the last checked step (not finite: overflow)
    double scale, last_scale;
    double pw1, pw2;           // betas to the power t
    int64_t t, good;
    float inv_scale;           // of the gradients the next check reads
    float upd_inv_scale, bc1, bc2, clip;    // the decided step's
    int32_t skip;
};

struct AdamwScalars {
    float b1, omb1, b2, omb2, eps, lr, wd;
    double b1d, b2d;
    double min_scale, max_norm;
    int32_t bias_correction, dynamic, growth_interval, l2;
    uint64_t seed;
};

// Elements of a workgroup of the update: 4 blocks of 256 a wave; or one, where the
// elements are few and more workgroups finish sooner.
constexpr int64_t kAdamwChunk = 4096, kAdamwSmallChunk = 1024;
constexpr int64_t kAdamwLarge = 8 << 20;  // elements from which on chunks are large
constexpr int64_t kAdamwPartials = 2048;  // of the check, at most
constexpr int64_t kAdamwInline = 512;     // that the update adds itself

struct AdamwLaunch {
    const TensorEntry* tensors;
    const ChunkEntry* chunks;
    int64_t nchunks, chunk;
    AdamwState* state;         // and a copy beside it
    double* partial;           // kAdamwPartials
    AdamwScalars s;
};

hipError_t adamw_step(const AdamwLaunch& a, int bits, bool checked, hipStream_t s);
int64_t adamw_chunk(int64_t elements);
hipError_t adamw_set_state(AdamwState* state, const AdamwState& to, hipStream_t s);
constexpr int kGradsPerLaunch = 256;
hipError_t adamw_set_grads(TensorEntry* tensors, const void* const* grads, int64_t first, int count, hipStream_t s);
hipError_t moments_pack(const float* x, uint8_t* codes, int8_t* exps, int64_t n, bool is_signed, hipStream_t s);
hipError_t moments_unpack(const uint8_t* codes, const int8_t* exps, void* out, int64_t n, int type, bool is_signed, hipStream_t s);

}  // namespace zo
