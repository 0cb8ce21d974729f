// Softmax cross entropy over a vocabulary, from hidden states H [tokens][width] and
// the output weight W [vocab][width], with both gradients:
//     z = H W^T ;  lse_n = log sum_v exp z_nv ;  loss_n = lse_n - z_n,target
//     G_nv = (exp(z_nv - lse_n) - [v is n's target]) * grad_scale / counted
//     dH = G W ;  dW = G^T H
// for the tokens that count (target != ignore_index); the others have loss 0 and a
// row of zeros in G.
//
// The logits never reach memory.  The first product's epilogue takes each 64 ids
// of a token (a piece) to their maximum m and the sum of exp(z - m), both in fp32,
// and, where gradients are wanted, leaves exp(z - m) in the 2-byte type.  When every
// piece is done, a token's pieces join to its lse, and one pass multiplies each
// piece by exp(m - lse): those are the probabilities.  So the gradients cost
// three matrix products in all (6 tokens vocab width operations); computing the
// logits again would make it four.  The exponentials of a chunk of tokens, 2 bytes
// each, are what is held: 0.8 GB at 8192 tokens and 50257 ids, of 288.
//
// Rounding to 2 bytes twice (the exponential, then its product with exp(m - lse))
// costs G a relative error of at most two half steps an entry, random in sign over
// the sums that follow.  The target's entry, where p - 1 would cancel, is computed
// from the fp32 logit as expm1(z - lse).  What is held is G times 2^15 (fp16) or 2^32
// (bf16), taken back in the products' epilogues: entries down to 2^-29 and 2^-158
// stay normal numbers.

#include "ops_common.h"
#include "ops_gemm.h"
#include "ops_internal.h"

namespace zo {
namespace {

constexpr int kPiece = 64;
constexpr int64_t kVocabPad = 64;

constexpr float kLog2e = 1.44269504088896340736f;

template <typename T> constexpr float kHoldLog2 = 32.0f;        // factor of what is held
template <> constexpr float kHoldLog2<_Float16> = 15.0f;
template <typename T> constexpr float kHold = (float)(1ull << (int)kHoldLog2<T>);

// Workgroup -> tile.  Workgroups go round the 8 dies; each die gets a run of tiles
// that lie together (kGroup tiles of i by all of j, column by column), so that its
// L2 serves the operands' pieces to the tiles that share them.
__device__ __forceinline__ void tile_of(int64_t id, int64_t ti, int64_t tj, int64_t& i, int64_t& j)
{
    constexpr int64_t kDies = 8, kGroup = 8;
    const int64_t all = ti * tj, die = id % kDies, at = id / kDies;
    const int64_t q = all / kDies, r = all % kDies;
    const int64_t n = die * q + (die < r ? die : r) + at;
    const int64_t per = kGroup * tj, g = n / per;
    const int64_t first = g * kGroup;
    const int64_t high = ti - first < kGroup ? ti - first : kGroup;
    i = first + (n - g * per) % high;
    j = (n - g * per) / high;
}

template <typename T>
__device__ __forceinline__ T to_type(float x)
{
    return static_cast<T>(x);
}

// ------------------------------------------------------------------ the logits

struct LogitsArgs {
    Operand h, w;
    const int64_t* targets;     // of the chunk's tokens
    float* target_logit;
    float2* stats;              // [tokens][pieces]
    void* exps;                 // [tokens][vocab_ld], or NULL: the loss alone
    int64_t tokens, vocab, vocab_ld, pieces;
    int64_t ti, tj;
};

template <typename T>
__global__ __launch_bounds__(kGemmThreads, 2) void logits_kernel(LogitsArgs a)
{
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    int64_t bi, bj;
    tile_of(blockIdx.x, a.ti, a.tj, bi, bj);
    f4 acc[8][4];
    const int steps = (int)ceil_div(a.h.depth, kDeep);
    gemm_tile<T, kInner, kInner>(a.h, a.w, bi * kTile, bj * kTile, 0, steps,
                                 (uint32_t)(uintptr_t)(ZO_LDS char*)smem, acc);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t v0 = bj * kTile + (wave & 3) * kWaveJ;       // the wave's piece of 64 ids
    if (v0 >= a.vocab_ld) return;
    const int64_t v = v0 + (lane >> 4) * 16;                   // the lane's 16 ids
#pragma unroll
    for (int ti = 0; ti < 8; ++ti) {
        const int64_t n = bi * kTile + (wave >> 2) * kWaveI + ti * 16 + (lane & 15);
        float m = -INFINITY;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            if (v + k >= a.vocab) acc[ti][k >> 2][k & 3] = -INFINITY;
            m = fmaxf(m, acc[ti][k >> 2][k & 3]);
        }
        m = fmaxf(m, __shfl_xor(m, 16, kWave));
        m = fmaxf(m, __shfl_xor(m, 32, kWave));
        const int64_t target = n < a.tokens ? a.targets[n] - v : -1;
        // a piece of -infinities has no exponentials: 0, not exp(-inf + inf)
        const float base = m == -INFINITY ? 0.0f : m;
        float sum = 0.0f;
        vec_t<T, 8> held[2];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float z = acc[ti][k >> 2][k & 3];
            if (target == k && v + k < a.vocab) a.target_logit[n] = z;
            // (the factor in the exponent: nothing is lost below fp32's normal range)
            const float e = __builtin_amdgcn_exp2f(fmaf(z - base, kLog2e, kHoldLog2<T>));
            sum += e;
            held[k >> 3][k & 7] = to_type<T>(e);
        }
        sum *= 1.0f / kHold<T>;
        sum += __shfl_xor(sum, 16, kWave);
        sum += __shfl_xor(sum, 32, kWave);
        if (n < a.tokens) {
            if (lane < 16) a.stats[n * a.pieces + v0 / kPiece] = make_float2(m, sum);
            if (a.exps != nullptr) {
                auto* to = reinterpret_cast<vec_t<T, 8>*>(static_cast<T*>(a.exps) + n * a.vocab_ld + v);
                to[0] = held[0];
                to[1] = held[1];
            }
        }
    }
}

// ------------------------------------------------------------------ statistics

__device__ __forceinline__ float block_max(float x, float* sh)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor(x, off, kWave));
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = x;
    __syncthreads();
    x = fmaxf(fmaxf(sh[0], sh[1]), fmaxf(sh[2], sh[3]));
    __syncthreads();
    return x;
}

__device__ __forceinline__ double block_sum(double x, double* sh)
{
    x = wave_sum(x);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = x;
    __syncthreads();
    x = (sh[0] + sh[1]) + (sh[2] + sh[3]);
    __syncthreads();
    return x;
}

// One workgroup a token: its pieces join to lse, its loss, and (in place) each
// piece's factor exp(m - lse).  A target outside the vocabulary that is not
// ignore_index has loss NaN and factors NaN: the gradients then carry NaN, and a
// checked step is skipped.
__global__ __launch_bounds__(256) void join_kernel(float2* stats, const float* target_logit,
                                                   const int64_t* targets, float* losses, float* lse_out,
                                                   int64_t pieces, int64_t vocab, int64_t ignore)
{
    __shared__ float shm[4];
    __shared__ double shs[4];
    const int64_t n = blockIdx.x;
    float2* row = stats + n * pieces;
    float m = -INFINITY;
    for (int64_t p = threadIdx.x; p < pieces; p += 256) m = fmaxf(m, row[p].x);
    m = block_max(m, shm);
    const float base = m == -INFINITY ? 0.0f : m;
    double sum = 0.0;
    for (int64_t p = threadIdx.x; p < pieces; p += 256) {
        const float2 s = row[p];
        sum += (double)(s.y * expf(s.x - base));
    }
    sum = block_sum(sum, shs);
    const float lse = base + (float)log(sum);
    const int64_t t = targets[n];
    const bool counts = t != ignore, known = t >= 0 && t < vocab;
    if (threadIdx.x == 0) {
        lse_out[n] = lse;
        losses[n] = !counts ? 0.0f : known ? lse - target_logit[n] : __builtin_nanf("");
    }
    for (int64_t p = threadIdx.x; p < pieces; p += 256) {
        const float f = expf(row[p].x - lse);
        row[p].y = !counts ? 0.0f : known ? f : __builtin_nanf("");
    }
}

// How many tokens count, and the factor of the products' results.
__global__ __launch_bounds__(1024) void count_kernel(const int64_t* targets, int64_t tokens, int64_t ignore,
                                                     double grad_scale, float hold, float* alpha)
{
    __shared__ int sh[16];
    int n = 0;
    for (int64_t i = threadIdx.x; i < tokens; i += 1024) n += targets[i] != ignore;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) n += __shfl_xor(n, off, kWave);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = n;
    __syncthreads();
    if (threadIdx.x == 0) {
        int all = 0;
        for (int k = 0; k < 16; ++k) all += sh[k];
        alpha[0] = (float)(grad_scale / (all > 0 ? all : 1) / hold);
        alpha[1] = (float)(all > 0 ? all : 1);
    }
}

// The mean loss: fp64, in a fixed order.
__global__ __launch_bounds__(1024) void mean_kernel(const float* losses, int64_t tokens, const float* alpha,
                                                    float* loss)
{
    __shared__ double sh[16];
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < tokens; i += 1024) s += losses[i];
    s = wave_sum(s);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        double all = 0.0;
        for (int k = 0; k < 16; ++k) all += sh[k];
        *loss = (float)(all / (double)alpha[1]);
    }
}

// ------------------------------------------------------------------ G

// In place: what a piece holds times its factor, the target's entry by itself.
// A lane has 8 ids; a workgroup 2048 of one token.
template <typename T>
__global__ __launch_bounds__(256) void scale_kernel(T* exps, const float2* stats, const float* target_logit,
                                                    const float* lse, const int64_t* targets,
                                                    int64_t vocab, int64_t vocab_ld, int64_t pieces,
                                                    int64_t ignore)
{
    const int64_t n = blockIdx.y;
    const int64_t v = (int64_t)blockIdx.x * 2048 + threadIdx.x * 8;
    if (v >= vocab_ld) return;
    auto* at = reinterpret_cast<vec_t<T, 8>*>(exps + n * vocab_ld + v);
    const int64_t t = targets[n];
    const float f = stats[n * pieces + v / kPiece].y;
    vec_t<T, 8> x = *at;
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = t == ignore ? to_type<T>(0.0f) : to_type<T>((float)x[k] * f);
    if (t != ignore && t >= v && t < v + 8 && t < vocab) {
        const T own = to_type<T>(expm1f(target_logit[n] - lse[n]) * kHold<T>);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (t - v == k) x[k] = own;
    }
    *at = x;
}

// ------------------------------------------------------------------ the gradients

struct GradArgs {
    Operand p, q;
    const float* alpha;
    void* out;                // 2-byte results, row stride out_ld
    float* part;              // splits: fp32 parts [split][rows][cols], else NULL
    float* sum;               // running fp32 sum over chunks of tokens [rows][cols], or NULL
    int64_t rows, cols, out_ld;
    int64_t ti, tj;
    int64_t steps;            // of the whole depth
    int splits;
    int vector_out;           // 4 results can be stored at once
    int sum_in, sum_out;      // the sum is added / is where the result goes
};

template <typename T, Layout LP>
__global__ __launch_bounds__(kGemmThreads, 2) void grad_kernel(GradArgs a)
{
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    const int64_t tiles = a.ti * a.tj;
    const int64_t split = blockIdx.x / tiles;
    int64_t bi, bj;
    tile_of(blockIdx.x % tiles, a.ti, a.tj, bi, bj);
    const int64_t s0 = a.steps * split / a.splits, s1 = a.steps * (split + 1) / a.splits;
    f4 acc[8][4];
    gemm_tile<T, LP, kOuter>(a.p, a.q, bi * kTile, bj * kTile, s0 * kDeep, (int)(s1 - s0),
                             (uint32_t)(uintptr_t)(ZO_LDS char*)smem, acc);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float alpha = a.alpha[0];
#pragma unroll
    for (int ti = 0; ti < 8; ++ti) {
        const int64_t i = bi * kTile + (wave >> 2) * kWaveI + ti * 16 + (lane & 15);
        if (i >= a.rows) continue;
#pragma unroll
        for (int tj = 0; tj < 4; ++tj) {
            const int64_t j = bj * kTile + (wave & 3) * kWaveJ + tj * 16 + (lane >> 4) * 4;
            const f4 c = acc[ti][tj];
            if (a.part != nullptr) {
                float* to = a.part + (split * a.rows + i) * a.cols + j;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (j + e < a.cols) to[e] = c[e];
                continue;
            }
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = c[e] * alpha;
                if (a.sum_in && j + e < a.cols) x[e] += a.sum[i * a.cols + j + e];
            }
            if (a.sum_out) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (j + e < a.cols) a.sum[i * a.cols + j + e] = x[e];
            } else {
                T* to = static_cast<T*>(a.out) + i * a.out_ld + j;
                if (a.vector_out && j + 4 <= a.cols) {
                    vec_t<T, 4> y;
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = to_type<T>(x[e]);
                    *reinterpret_cast<vec_t<T, 4>*>(to) = y;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (j + e < a.cols) to[e] = to_type<T>(x[e]);
                }
            }
        }
    }
}

// The parts of a split product, added in the order of the splits.
template <typename T>
__global__ __launch_bounds__(256) void join_splits_kernel(const float* part, int splits, int64_t rows,
                                                          int64_t cols, const float* alpha, T* out,
                                                          int64_t out_ld)
{
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at >= rows * cols) return;
    float s = 0.0f;
    for (int k = 0; k < splits; ++k) s += part[k * rows * cols + at];
    out[at / cols * out_ld + at % cols] = to_type<T>(s * alpha[0]);
}

// Rows of any stride and alignment to rows of ld, a multiple of 8, zeros behind the width.
template <typename T>
__global__ __launch_bounds__(256) void repack_kernel(const T* x, int64_t stride, int64_t rows, int64_t width,
                                                     T* out, int64_t ld)
{
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (at >= rows * ld) return;
    const int64_t r = at / ld, c = at % ld;
    vec_t<T, 8> y;
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = c + k < width ? x[r * stride + c + k] : to_type<T>(0.0f);
    *reinterpret_cast<vec_t<T, 8>*>(out + at) = y;
}

bool loads_as_it_is(const void* p, int64_t stride, int64_t width)
{
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 8 == 0 && width % 8 == 0 && stride <= (1 << 21);
}

template <typename K>
hipError_t allow_lds(K kernel)
{
    return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                               2 * kStageBytes);
}

template <typename T>
hipError_t run(const Loss& a, const LossPlan& p, hipStream_t s)
{
    static const hipError_t allowed = [] {
        hipError_t e = allow_lds(logits_kernel<T>);
        if (e == hipSuccess) e = allow_lds(grad_kernel<T, kInner>);
        if (e == hipSuccess) e = allow_lds(grad_kernel<T, kOuter>);
        return e;
    }();
    if (allowed != hipSuccess) return allowed;
    float* alpha = reinterpret_cast<float*>(a.space + p.off_alpha);
    float* target_logit = reinterpret_cast<float*>(a.space + p.off_target);
    float* lse = a.lse != nullptr ? a.lse : reinterpret_cast<float*>(a.space + p.off_lse);
    float2* stats = reinterpret_cast<float2*>(a.space + p.off_stats);
    const bool gradient = a.dweight != nullptr;
    T* exps = gradient ? reinterpret_cast<T*>(a.space + p.off_exp) : nullptr;
    const T* h = static_cast<const T*>(a.hidden);
    const T* w = static_cast<const T*>(a.weight);
    int64_t h_ld = a.hidden_stride, w_ld = a.weight_stride, depth = p.width;
    if (!loads_as_it_is(h, h_ld, p.width) || !loads_as_it_is(w, w_ld, p.width)) {
        T* hp = reinterpret_cast<T*>(a.space + p.off_hidden);
        T* wp = reinterpret_cast<T*>(a.space + p.off_weight);
        auto repack = [&](const T* x, int64_t stride, int64_t rows, T* out) {
            if (rows > 0)
                repack_kernel<T><<<dim3((unsigned)ceil_div(rows * p.width_ld, 2048)), 256, 0, s>>>(x, stride, rows, p.width, out, p.width_ld);
        };
        repack(h, h_ld, p.tokens, hp);
        repack(w, w_ld, p.vocab, wp);
        h = hp;
        w = wp;
        h_ld = w_ld = depth = p.width_ld;
    }
    count_kernel<<<1, 1024, 0, s>>>(a.targets, p.tokens, a.ignore_index, a.grad_scale, kHold<T>, alpha);
    const Operand ow{w, w_ld, p.vocab, depth};
    if (p.tokens == 0 && gradient) {       // a sum over no tokens
        GradArgs g{};
        g.p = Operand{w, p.vocab_ld, p.vocab_ld, 0};
        g.q = Operand{w, w_ld, depth, 0};
        g.alpha = alpha;
        g.rows = p.vocab;
        g.cols = p.width;
        g.ti = ceil_div(p.vocab, kTile);
        g.tj = ceil_div(p.width, kTile);
        g.splits = 1;
        g.out = a.dweight;
        g.out_ld = a.dweight_stride;
        grad_kernel<T, kOuter><<<dim3((unsigned)(g.ti * g.tj)), kGemmThreads, 2 * kStageBytes, s>>>(g);
    }
    for (int64_t n0 = 0; n0 < p.tokens; n0 += p.chunk) {
        const int64_t n = p.tokens - n0 < p.chunk ? p.tokens - n0 : p.chunk;
        const Operand oh{h + n0 * h_ld, h_ld, n, depth};
        LogitsArgs l{oh, ow, a.targets + n0, target_logit, stats, exps, n, p.vocab, p.vocab_ld, p.pieces,
                     ceil_div(n, kTile), ceil_div(p.vocab, kTile)};
        logits_kernel<T><<<dim3((unsigned)(l.ti * l.tj)), kGemmThreads, 2 * kStageBytes, s>>>(l);
        join_kernel<<<dim3((unsigned)n), 256, 0, s>>>(stats, target_logit, a.targets + n0, a.losses + n0,
                                                      lse + n0, p.pieces, p.vocab, a.ignore_index);
        if (!gradient) continue;
        scale_kernel<T><<<dim3((unsigned)ceil_div(p.vocab_ld, 2048), (unsigned)n), 256, 0, s>>>(
            exps, stats, target_logit, lse + n0, a.targets + n0, p.vocab, p.vocab_ld, p.pieces, a.ignore_index);
        GradArgs g{};
        g.alpha = alpha;
        g.cols = p.width;
        g.tj = ceil_div(p.width, kTile);
        // dH = G W: k runs over the vocabulary, in parts where there are few tiles
        g.p = Operand{exps, p.vocab_ld, n, p.vocab_ld};
        g.q = Operand{w, w_ld, depth, p.vocab};
        g.rows = n;
        g.ti = ceil_div(n, kTile);
        g.steps = p.vocab_ld / kDeep;
        g.splits = p.splits;
        g.out = static_cast<T*>(a.dhidden) + n0 * a.dhidden_stride;
        g.out_ld = a.dhidden_stride;
        g.vector_out = ((uintptr_t)g.out & 7) == 0 && g.out_ld % 4 == 0;
        g.part = p.splits > 1 ? reinterpret_cast<float*>(a.space + p.off_split) : nullptr;
        grad_kernel<T, kInner><<<dim3((unsigned)(g.ti * g.tj * g.splits)), kGemmThreads, 2 * kStageBytes, s>>>(g);
        if (p.splits > 1)
            join_splits_kernel<T><<<dim3((unsigned)ceil_div(n * p.width, 256)), 256, 0, s>>>(
                g.part, p.splits, n, p.width, alpha, static_cast<T*>(g.out), g.out_ld);
        // dW = G^T H: k runs over the chunk's tokens; with several chunks the sum
        // stays in fp32 until the last
        g.p = Operand{exps, p.vocab_ld, p.vocab_ld, n};
        g.q = Operand{oh.base, h_ld, depth, n};
        g.rows = p.vocab;
        g.ti = ceil_div(p.vocab, kTile);
        g.steps = ceil_div(n, kDeep);
        g.splits = 1;
        g.out = a.dweight;
        g.out_ld = a.dweight_stride;
        g.vector_out = ((uintptr_t)g.out & 7) == 0 && g.out_ld % 4 == 0;
        g.part = nullptr;
        g.sum = reinterpret_cast<float*>(a.space + p.off_sum);
        g.sum_in = n0 > 0;
        g.sum_out = n0 + n < p.tokens;
        grad_kernel<T, kOuter><<<dim3((unsigned)(g.ti * g.tj)), kGemmThreads, 2 * kStageBytes, s>>>(g);
    }
    mean_kernel<<<1, 1024, 0, s>>>(a.losses, p.tokens, alpha, a.loss);
    return hipGetLastError();
}

}  // namespace

LossPlan loss_plan(int64_t tokens, int64_t vocab, int64_t width, int64_t max_chunk, bool gradient)
{
    LossPlan p{};
    p.tokens = tokens;
    p.vocab = vocab;
    p.width = width;
    p.vocab_ld = round_up(vocab, kVocabPad);
    p.pieces = p.vocab_ld / kPiece;
    p.width_ld = round_up(width, 8);
    p.chunk = tokens < max_chunk ? tokens : max_chunk;
    if (p.chunk < 1) p.chunk = 1;
    // parts of the vocabulary: enough workgroups for every CU, none with less than
    // 8 steps
    const int64_t tiles = ceil_div(p.chunk, kTile) * ceil_div(width, kTile);
    const int64_t steps = p.vocab_ld / kDeep;
    int64_t splits = tiles < kCUs ? kCUs / tiles : 1;
    if (splits > steps / 8) splits = steps / 8;
    p.splits = splits < 1 ? 1 : (int)splits;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t off = at;
        at += round_up(bytes, 256);
        return off;
    };
    p.off_alpha = take(16);
    p.off_target = take(p.chunk * 4);
    p.off_lse = take(tokens * 4);
    p.off_stats = take(p.chunk * p.pieces * 8);
    p.off_exp = take(gradient ? p.chunk * p.vocab_ld * 2 : 0);
    p.off_split = take(gradient && p.splits > 1 ? p.splits * p.chunk * width * 4 : 0);
    p.off_sum = take(gradient && p.chunk < tokens ? vocab * width * 4 : 0);
    p.off_hidden = take(tokens * p.width_ld * 2);
    p.off_weight = take(vocab * p.width_ld * 2);
    p.bytes = at;
    return p;
}

hipError_t vocab_loss(const Loss& a, const LossPlan& p, int type, hipStream_t s)
{
    return type == 1 ? run<_Float16>(a, p, s) : run<__bf16>(a, p, s);
}

}  // namespace zo
