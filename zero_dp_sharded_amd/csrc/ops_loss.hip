// Softmax cross entropy over a vocabulary, from hidden states H [tokens][width] and
// the output weight W [vocab][width], with both gradients:
//     z = H W^T ;  lse_n = log sum_v exp z_nv ;  loss_n = lse_n - z_n,target
//     G_nv = (exp(z_nv - lse_n) - [v is n's target]) * grad_scale / counted
//     dH = G W ;  dW = G^T H
// for the tokens that count (target != ignore_index); the others have loss 0 and a
// row of zeros in G.
//
// The logits never reach memory.  The first product's epilogue takes each piece of a
// token (64 or 80 ids) to its maximum m and the sum of exp(z - m), both fp32, and, where
// gradients are wanted, leaves exp(z - m) in the 2-byte type.  A second kernel joins
// a token's pieces to lse and multiplies them by exp(m - lse), in place.  So the
// gradients cost three matrix products in all (6 tokens vocab width operations);
// computing the logits again would make it four.  What is held are the exponentials of a
// chunk of tokens, 2 bytes each: 0.8 GB at 8192 tokens and 50257 ids, of 288; the
// pass over them takes 330 us of 3710 (5.2 TB/s).  The three products take 1240, 1215 and
// 1130 us there in the mean, 1060 to 1170 TFLOP/s of the 1550 that a large library product
// reaches (at best 1157, 1122 and 1031; by the box's clock the whole takes 3710 to 3970):
// ops_gemm.h says what bounds them.  (bf16 could do without the pass, by
// exponentials without a maximum and the factors exp(-lse) in the second product's
// epilogue and in a copy of H; that took 7% less, and the copy's rounding made the
// weight's gradient 1.7 times less exact.)
//
// An entry of G is rounded to 2 bytes twice (as exp, and by its factor); up to 32 tokens it
// is held in two 2-byte numbers, as good as exact (see kPairs).  The target's entry, where p - 1 would cancel, is computed from the fp32 logit as expm1(z - lse).
// What is held is G times 2^15 (fp16) or 2^32 (bf16), taken back in the products'
// epilogues: entries far below the type's normal range stay.

#include <type_traits>

#include "ops_common.h"
#include "ops_gemm.h"
#include "ops_internal.h"

namespace zo {
namespace {

constexpr int64_t kLastCache = 256 << 20;
constexpr float kLog2e = 1.44269504088896340736f;
template <typename T> constexpr float kHoldLog2 = 32.0f;        // factor of what is held
template <> constexpr float kHoldLog2<_Float16> = 15.0f;
template <typename T> constexpr float kHold = (float)(1ull << (int)kHoldLog2<T>);

// The n-th tile of those that die `die` of 8 takes.  Workgroups go round the dies;
// each die gets a run of tiles that lie together (8 tiles of i by all of j, column by
// column), so that its L2 serves the operands' pieces to the tiles that share them.
constexpr uint32_t kDies = 8;

__device__ __forceinline__ uint32_t tiles_of(uint32_t die, uint32_t all)
{
    return all / kDies + (die < all % kDies ? 1 : 0);
}

__device__ __forceinline__ void tile_of(uint32_t die, uint32_t at, uint32_t ti, uint32_t tj, int64_t& i, int64_t& j)
{
    constexpr uint32_t kGroup = 8;
    const uint32_t q = ti * tj / kDies, r = ti * tj % kDies;
    const uint32_t n = die * q + (die < r ? die : r) + at;
    const uint32_t per = kGroup * tj, g = n / per;
    const uint32_t first = g * kGroup;
    const uint32_t high = ti - first < kGroup ? ti - first : kGroup;
    // (the same for all lanes: kept where that costs no vector register)
    i = __builtin_amdgcn_readfirstlane(first + (n - g * per) % high);
    j = __builtin_amdgcn_readfirstlane((n - g * per) / high);
}

template <typename T>
__device__ __forceinline__ T to_type(float x)
{
    return static_cast<T>(x);
}

__device__ __forceinline__ uint32_t lds_address(char* smem) { return (uint32_t)(uintptr_t)(ZO_LDS char*)smem; }

// ------------------------------------------------------------------ the logits

struct LogitsArgs {
    Operand h, w;
    const int64_t* targets;     // of the chunk's tokens
    float* target_logit;
    float2* stats;              // [tokens][pieces]: maximum and sum
    void* exps;                 // [tokens][vocab_ld], or NULL: the loss alone
    int pairs;                  // the exponentials are in pairs: beside each what its rounding takes away (NI = 2)
    int64_t tokens, vocab, vocab_ld, pieces;
    uint32_t ti, tj;          // tiles
};

// From a tile's logits to the pieces' statistics and the exponentials.
template <typename T, int NI, int NJ>
__device__ __forceinline__ void logits_out(const LogitsArgs& a, int64_t bi, int64_t bj, f4 (&acc)[NI][NJ])
{
    using G = Gemm<T, kInner, kInner, NI, NJ>;
    constexpr int R = 4 * NJ;                                  // a lane's ids
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));      // (addresses are made here, and not kept in registers over the products)
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // 16 from v on, and with NJ = 5 another 4 from `far` on
    const int64_t v = bj * G::kTileJ + G::column_of(0, wave, lane);
    const int64_t far = bj * G::kTileJ + G::column_of(4, wave, lane) - 16;       // (id of k >= 16: far + k)
    if (bj * G::kTileJ + (wave & 3) * 64 >= a.vocab_ld) return;                  // (NJ = 4: past the last piece)
    if ((bj + 1) * G::kTileJ > a.vocab) {                      // the tile that the vocabulary ends in
#pragma unroll
        for (int ti = 0; ti < NI; ++ti)
#pragma unroll
            for (int k = 0; k < R; ++k)
                if ((k < 16 ? v : far) + k >= a.vocab) acc[ti][k >> 2][k & 3] = -INFINITY;
    }
#pragma unroll
    for (int ti = 0; ti < NI; ++ti) {
        const int64_t n = bi * G::kTileI + G::row_of(ti, wave, lane);
        float m = acc[ti][0][0];
#pragma unroll
        for (int k = 1; k < R; ++k) m = fmaxf(m, acc[ti][k >> 2][k & 3]);
        m = fmaxf(m, __shfl_xor(m, 16, kWave));
        m = fmaxf(m, __shfl_xor(m, 32, kWave));
        const int64_t target = n < a.tokens ? a.targets[n] : -1;
        const bool near = target >= v && target < v + 16;
        if (near || (NJ == 5 && target >= far + 16 && target < far + 20)) {
            // (a chain of selections: an index into the registers would put them in memory)
            const int at = (int)(target - (near ? v : far));
            float z = 0.0f;
#pragma unroll
            for (int k = 0; k < R; ++k) z = at == k ? acc[ti][k >> 2][k & 3] : z;
            a.target_logit[n] = z;
        }
        // a piece of -infinities has no exponentials: 0, not exp(-inf + inf)
        const float base = m == -INFINITY ? 0.0f : m;
        float sum = 0.0f;
        vec_t<T, 4> held[NJ], low[NJ];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            // (the factor in the exponent: nothing is lost below fp32's normal range)
            const float e = __builtin_amdgcn_exp2f(fmaf(acc[ti][k >> 2][k & 3] - base, kLog2e, kHoldLog2<T>));
            sum += e;
            held[k >> 2][k & 3] = to_type<T>(e);
            if constexpr (NI == 2) low[k >> 2][k & 3] = to_type<T>(e - (float)held[k >> 2][k & 3]);
        }
        sum += __shfl_xor(sum, 16, kWave);
        sum += __shfl_xor(sum, 32, kWave);
        if (n < a.tokens) {
            if (lane < 16) a.stats[n * a.pieces + bj * 4 + (wave & 3)] = make_float2(m, sum * (1.0f / kHold<T>));
            if (a.exps != nullptr) {
                T* to = static_cast<T*>(a.exps) + (NI == 2 && a.pairs ? pair_row(n) : n) * a.vocab_ld;
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    reinterpret_cast<vec_t<T, 8>*>(to + v)[q] =
                        __builtin_shufflevector(held[2 * q], held[2 * q + 1], 0, 1, 2, 3, 4, 5, 6, 7);
                if constexpr (NJ == 5) *reinterpret_cast<vec_t<T, 4>*>(to + far + 16) = held[4];
                if constexpr (NI == 2) {
                    if (a.pairs) {
                        auto* under = reinterpret_cast<vec_t<T, 8>*>(to + 16 * a.vocab_ld + v);
#pragma unroll
                        for (int q = 0; q < 2; ++q)
                            under[q] = __builtin_shufflevector(low[2 * q], low[2 * q + 1], 0, 1, 2, 3, 4, 5, 6, 7);
                    }
                }
            }
        }
    }
}

// A die's workgroups walk its tiles, and load the next one while they are at a tile's
// exponentials (a tile of width 1600 is 25 steps of 2 us, its exponentials 7 us and its
// first loads 3).
template <typename T, int NI, int NJ>
__global__ __launch_bounds__(kGemmThreads, 2) void logits_kernel(LogitsArgs a)
{
    using G = Gemm<T, kInner, kInner, NI, NJ>;
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    const uint32_t die = blockIdx.x % kDies, mine = tiles_of(die, a.ti * a.tj);
    const uint32_t stride = (gridDim.x + kDies - 1 - die) / kDies;       // workgroups of the die
    const int steps = (int)ceil_div(a.h.depth, kDeep);
    G g(a.h, a.w, lds_address(smem));
    int64_t bi = 0, bj = 0;
    uint32_t at = blockIdx.x / kDies;
    if (at >= mine) return;
    tile_of(die, at, a.ti, a.tj, bi, bj);
    g.begin(a.h, a.w, bi * G::kTileI, bj * G::kTileJ, 0, steps);
    for (;;) {
        f4 acc[NI][NJ];
        const int64_t i = bi, j = bj;
        at += stride;
        g.run(steps, acc, [&] {
            if (at >= mine) return;
            tile_of(die, at, a.ti, a.tj, bi, bj);
            g.begin(a.h, a.w, bi * G::kTileI, bj * G::kTileJ, 0, steps);
        });
        logits_out<T, NI, NJ>(a, i, j, acc);
        if (at >= mine) return;
    }
}

// The piece that id v belongs to: waves take 64 ids of each 256, or 64 + 16 of each 320.
template <int NJ>
__device__ __forceinline__ int64_t piece_of(int64_t v)
{
    if constexpr (NJ == 4) return v / 64;
    const int64_t tile = v / 320, at = v % 320;
    return tile * 4 + (at < 256 ? at / 64 : (at - 256) / 16);
}

// ------------------------------------------------------------------ joining the pieces

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

struct JoinArgs {
    const float2* stats;
    const float* target_logit;
    const int64_t* targets;
    float* losses;
    float* lse;
    void* exps;               // NULL: the loss alone
    int pairs;                // they are in pairs
    int64_t pieces, vocab, vocab_ld, ignore;
    const void* hidden;       // rows of width_ld, hidden_ld apart
    void* kept;               // the same rows side by side (or where they are), of ignored tokens zeros
    int64_t hidden_ld, width_ld;
};

// A token: lse, its loss, and from its exponentials its row of G.  Where there are few
// tokens, several workgroups a token (blockIdx.y) share its row, and each finds lse.  A
// target outside the vocabulary that is not ignore_index has loss NaN and a row of NaN:
// the gradients then carry NaN, and a checked step is skipped.
//
// The hidden states go into the workspace for the weight's gradient, with zeros for the
// tokens that are left out: their rows of G are zeros, but 0 times what is not finite is NaN
// (8192 tokens of width 1600: 52 MB more in a pass of 1.7 GB).
//
// PAST: rows of more than the last cache's 256 MiB in all go past the caches (8192 tokens
// x 50257 bf16: the loss and its gradients 3823 -> 3777 us; of 2048 tokens, which the
// products then find there, 1052 -> 1064).
template <typename T, int NJ, bool PAST>
__global__ __launch_bounds__(256) void join_kernel(JoinArgs a)
{
    __shared__ float shm[4];
    __shared__ double shs[4];
    const int64_t n = blockIdx.x;
    const float2* row = a.stats + n * a.pieces;
    float m = -INFINITY;
    for (int64_t p = threadIdx.x; p < a.pieces; p += 256) m = fmaxf(m, row[p].x);
    m = block_max(m, shm);
    const float base = m == -INFINITY ? 0.0f : m;
    double sum = 0.0;
    for (int64_t p = threadIdx.x; p < a.pieces; p += 256) {
        const float2 s = row[p];
        sum += (double)(s.y * expf(s.x - base));
    }
    sum = block_sum(sum, shs);
    const float lse = base + (float)log(sum);
    const int64_t t = a.targets[n];
    const bool counts = t != a.ignore, known = t >= 0 && t < a.vocab;
    const float z = counts && known ? a.target_logit[n] : 0.0f;
    // what a token without a known target has instead
    const float nothing = counts ? __builtin_nanf("") : 0.0f;
    if (threadIdx.x == 0 && blockIdx.y == 0) {
        a.lse[n] = lse;
        a.losses[n] = counts && known ? lse - z : nothing;
    }
    if (a.exps == nullptr) return;
    const T* hidden = static_cast<const T*>(a.hidden) + n * a.hidden_ld;
    T* kept = static_cast<T*>(a.kept) + n * a.width_ld;
    if (hidden != kept || !counts) {
        for (int64_t c = (blockIdx.y * 256 + threadIdx.x) * 8; c < a.width_ld; c += gridDim.y * 2048) {
            vec_t<T, 8> x = {};
            if (counts) x = load_vec<T, 8>(hidden + c);
            *reinterpret_cast<vec_t<T, 8>*>(kept + c) = x;
        }
    }
    T* exps = static_cast<T*>(a.exps) + (a.pairs ? pair_row(n) : n) * a.vocab_ld;
    const float target = expm1f(z - lse) * kHold<T>;
    const T own = to_type<T>(target);
    if (a.pairs) {
        T* low = exps + 16 * a.vocab_ld;
        for (int64_t v = (blockIdx.y * 256 + threadIdx.x) * 8; v < a.vocab_ld; v += gridDim.y * 2048) {
            auto* at = reinterpret_cast<vec_t<T, 8>*>(exps + v);
            auto* under = reinterpret_cast<vec_t<T, 8>*>(low + v);
            const float f = expf(row[piece_of<NJ>(v)].x - lse);
            vec_t<T, 8> x = *at, y = *under;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float g = ((float)x[k] + (float)y[k]) * f;
                if (v + k == t) g = target;
                if (!(counts && known)) g = nothing;
                x[k] = to_type<T>(g);
                y[k] = to_type<T>(g - (float)x[k]);
            }
            *at = x;
            *under = y;
        }
        return;
    }
#pragma unroll 4
    for (int64_t v = (blockIdx.y * 256 + threadIdx.x) * 8; v < a.vocab_ld; v += gridDim.y * 2048) {
        const float f = expf(row[piece_of<NJ>(v)].x - lse);
        vec_t<T, 8> x = load_vec<T, 8, PAST>(exps + v);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            x[k] = counts && known ? to_type<T>((float)x[k] * f) : to_type<T>(nothing);
            if (counts && known && v + k == t) x[k] = own;
        }
        store_vec<T, 8, PAST>(exps + v, x);
    }
}

// Sums over all tokens, in a fixed order: how many count, which settles the factor of
// the products' results, and (the last time) the mean loss.
__global__ __launch_bounds__(1024) void total_kernel(const int64_t* targets, const float* losses, int64_t tokens,
                                                     int64_t ignore, double grad_scale, float hold, float* alpha,
                                                     float* loss)
{
    __shared__ int shn[16];
    __shared__ double shs[16];
    int n = 0;
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < tokens; i += 1024) {
        n += targets[i] != ignore;
        if (loss != nullptr) s += losses[i];
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) n += __shfl_xor(n, off, kWave);
    s = wave_sum(s);
    if ((threadIdx.x & 63) == 0) {
        shn[threadIdx.x >> 6] = n;
        shs[threadIdx.x >> 6] = s;
    }
    __syncthreads();
    if (threadIdx.x != 0) return;
    int all = 0;
    s = 0.0;
    for (int k = 0; k < 16; ++k) {
        all += shn[k];
        s += shs[k];
    }
    if (all < 1) all = 1;
    *alpha = (float)(grad_scale / all / hold);
    if (loss != nullptr) *loss = (float)(s / all);
}

// ------------------------------------------------------------------ the gradients

struct GradArgs {
    Operand p, q;
    const float* alpha;
    void* out;                // 2-byte results, row stride out_ld
    float* part;              // splits: fp32 parts [split][rows][cols], else NULL
    float* sum;               // running fp32 sum over chunks of tokens [rows][cols], or NULL
    int64_t rows, cols, out_ld;
    uint32_t ti, tj;          // tiles
    int64_t steps;            // of the whole depth
    int splits;
    int vector_out;           // results that can be stored at once: 8, 4, or 0
    int sum_in, sum_out;      // the sum is added / is where the result goes
    int pairs;                // p's rows are in pairs, and a result is the sum of a pair's (NI = 2)
};

template <typename T, Layout LP, int NI, int NJ>
__global__ __launch_bounds__(kGemmThreads, 2) void grad_kernel(GradArgs a)
{
    using G = Gemm<T, LP, kOuter, NI, NJ>;
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    const uint32_t tiles = a.ti * a.tj, id = blockIdx.x % tiles;
    const int64_t split = __builtin_amdgcn_readfirstlane(blockIdx.x / tiles);
    int64_t bi, bj;
    tile_of(id % kDies, id / kDies, a.ti, a.tj, bi, bj);
    const int64_t s0 = a.steps * split / a.splits, s1 = a.steps * (split + 1) / a.splits;
    f4 acc[NI][NJ];
    G g(a.p, a.q, lds_address(smem));
    g.begin(a.p, a.q, bi * G::kTileI, bj * G::kTileJ, s0 * kDeep, (int)(s1 - s0));
    g.run((int)(s1 - s0), acc, [] {});
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float alpha = a.alpha[0];
    if constexpr (NI == 2 && LP == kInner) {
        if (a.pairs) {
#pragma unroll
            for (int tj = 0; tj < NJ; ++tj) acc[0][tj] += acc[1][tj];
        }
    }
    auto row_at = [&](int ti) -> int64_t {
        const int row = G::row_of(ti, wave, lane);
        if constexpr (NI == 2 && LP == kInner)
            if (a.pairs) return ti == 0 ? pair_entry(row) : a.rows;        // (one tile)
        return bi * G::kTileI + row;
    };
    if (a.part == nullptr && !a.sum_in && !a.sum_out && a.vector_out) {       // as good as always
#pragma unroll
        for (int ti = 0; ti < NI; ++ti) {
            const int64_t i = row_at(ti);
            if (i >= a.rows) continue;
            T* to = static_cast<T*>(a.out) + i * a.out_ld;
            if constexpr (G::kRuns && NJ == 4) {
                const int64_t j = bj * G::kTileJ + G::column_of(0, wave, lane);
                if (a.vector_out == 8 && j + 16 <= a.cols) {
                    vec_t<T, 8> y[2];
#pragma unroll
                    for (int k = 0; k < 16; ++k) y[k >> 3][k & 7] = to_type<T>(acc[ti][k >> 2][k & 3] * alpha);
                    reinterpret_cast<vec_t<T, 8>*>(to + j)[0] = y[0];
                    reinterpret_cast<vec_t<T, 8>*>(to + j)[1] = y[1];
                    continue;
                }
            }
#pragma unroll
            for (int tj = 0; tj < NJ; ++tj) {
                const int64_t j = bj * G::kTileJ + G::column_of(tj, wave, lane);
                vec_t<T, 4> y;
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = to_type<T>(acc[ti][tj][e] * alpha);
                if (j + 4 <= a.cols) {
                    *reinterpret_cast<vec_t<T, 4>*>(to + j) = y;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (j + e < a.cols) to[j + e] = y[e];
                }
            }
        }
        return;
    }
#pragma unroll
    for (int ti = 0; ti < NI; ++ti) {
        const int64_t i = row_at(ti);
        if (i >= a.rows) continue;
#pragma unroll
        for (int tj = 0; tj < NJ; ++tj) {
            const int64_t j = bj * G::kTileJ + G::column_of(tj, wave, lane);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (j + e >= a.cols) continue;
                const float c = acc[ti][tj][e];
                if (a.part != nullptr) {
                    a.part[(split * a.rows + i) * a.cols + j + e] = c;
                    continue;
                }
                float* sum = a.sum + i * a.cols + j + e;
                const float x = a.sum_in ? *sum + c * alpha : c * alpha;
                if (a.sum_out) *sum = x;
                else static_cast<T*>(a.out)[i * a.out_ld + j + e] = to_type<T>(x);
            }
        }
    }
}

// The parts of a split product, added in the order of the splits: W results a lane.
template <typename T, int W>
__global__ __launch_bounds__(256) void join_splits_kernel(const float* part, int splits, int64_t rows,
                                                          int64_t cols, const float* alpha, T* out,
                                                          int64_t out_ld)
{
    const int64_t all = rows * cols, at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * W;
    if (at >= all) return;
    float s[W];
#pragma unroll
    for (int e = 0; e < W; ++e) s[e] = 0.0f;
#pragma unroll 8
    for (int k = 0; k < splits; ++k) {
        const vec_t<float, W> x = *reinterpret_cast<const vec_t<float, W>*>(part + k * all + at);
#pragma unroll
        for (int e = 0; e < W; ++e) s[e] += x[e];
    }
    vec_t<T, W> y;
#pragma unroll
    for (int e = 0; e < W; ++e) y[e] = to_type<T>(s[e] * alpha[0]);
    store_vec<T, W>(out + at / cols * out_ld + at % cols, y);
}

// Rows of any stride and alignment to rows of ld, a multiple of 8, zeros behind the
// width: of one array or, from workgroup `first` on, of another.
template <typename T>
struct Repack {
    const T* x;
    T* out;
    int64_t stride, rows;
};

template <typename T>
__global__ __launch_bounds__(256) void repack_kernel(Repack<T> a, Repack<T> b, int64_t base, int64_t first, int64_t width,
                                                     int64_t ld)
{
    const int64_t group = base + blockIdx.x;
    const bool second = group >= first;
    const Repack<T> r = second ? b : a;
    const int64_t at = ((group - (second ? first : 0)) * 256 + threadIdx.x) * 8;
    if (at >= r.rows * ld) return;
    const int64_t i = at / ld, c = at % ld;
    const T* x = r.x + i * r.stride + c;
    vec_t<T, 8> y;
    if (c + 8 <= width) {
        y = load_vec<T, 8>(x);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = c + k < width ? x[k] : to_type<T>(0.0f);
    }
    *reinterpret_cast<vec_t<T, 8>*>(r.out + at) = y;
}

// ------------------------------------------------------------------ launches
//
// (Of all of them only the copies could pass a launch's work-items: a product's tiles are
// fewer than 2^22, by what memory its operands take, and the rest goes by chunks of tokens.)

// What the products' loads need of an address and a stride.
bool loads_as_it_is(const void* p, int64_t stride)
{
    return (reinterpret_cast<uintptr_t>(p) & 3) == 0 && stride % 2 == 0 && stride <= (1 << 21);
}

// A kernel's LDS beyond 64 KiB is asked for once.
template <typename K>
hipError_t allow(K kernel, int lds)
{
    return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
}

template <typename T, int NI, int NJ>
hipError_t logits(LogitsArgs l, hipStream_t s)
{
    using G = Gemm<T, kInner, kInner, NI, NJ>;
    static const hipError_t allowed = allow(logits_kernel<T, NI, NJ>, G::kLds);
    if (allowed != hipSuccess) return allowed;
    l.ti = (uint32_t)ceil_div(l.tokens, G::kTileI);
    l.tj = (uint32_t)ceil_div(l.vocab, G::kTileJ);
    // as many workgroups as stand in the CUs at once: one, or two of the small tile's
    const uint32_t stand = kCUs * (NI == 2 ? 2 : 1), tiles = l.ti * l.tj;
    logits_kernel<T, NI, NJ><<<dim3(tiles < stand ? tiles : stand), kGemmThreads, G::kLds, s>>>(l);
    return hipSuccess;
}

template <typename T, Layout LP, int NI, int NJ>
hipError_t grad(GradArgs g, hipStream_t s)
{
    using G = Gemm<T, LP, kOuter, NI, NJ>;
    static const hipError_t allowed = allow(grad_kernel<T, LP, NI, NJ>, G::kLds);
    if (allowed != hipSuccess) return allowed;
    g.ti = (uint32_t)ceil_div(g.rows, G::kTileI);
    g.tj = (uint32_t)ceil_div(g.cols, G::kTileJ);
    g.vector_out = ((uintptr_t)g.out & 15) == 0 && g.out_ld % 8 == 0 ? 8 : ((uintptr_t)g.out & 7) == 0 && g.out_ld % 4 == 0 ? 4 : 0;
    // a single step has no second stage: more workgroups fit in a CU
    const int lds = g.steps <= 1 ? G::kStageBytes : G::kLds;
    grad_kernel<T, LP, NI, NJ><<<dim3(g.ti * g.tj * g.splits), kGemmThreads, lds, s>>>(g);
    return hipSuccess;
}

template <typename T, Layout LP>
hipError_t grad(const GradArgs& g, const TileChoice& c, hipStream_t s)
{
    if (c.ni == 2) return grad<T, LP, 2, 4>(g, s);
    return c.nj == 4 ? grad<T, LP, 8, 4>(g, s) : grad<T, LP, 8, 5>(g, s);
}

template <typename T>
hipError_t run(const Loss& a, const LossPlan& p, hipStream_t s)
{
    float* alpha = reinterpret_cast<float*>(a.space + p.off_alpha);
    float* target_logit = reinterpret_cast<float*>(a.space + p.off_target);
    float* lse = a.lse != nullptr ? a.lse : reinterpret_cast<float*>(a.space + p.off_lse);
    float2* stats = reinterpret_cast<float2*>(a.space + p.off_stats);
    const bool gradient = a.dweight != nullptr;
    T* exps = gradient ? reinterpret_cast<T*>(a.space + p.off_exp) : nullptr;
    const T* h = static_cast<const T*>(a.hidden);
    const T* w = static_cast<const T*>(a.weight);
    int64_t h_ld = a.hidden_stride, w_ld = a.weight_stride;
    // operands whose rows cannot be loaded as they lie, 8 elements at a time
    Repack<T> copies[2];
    int many = 0;
    if (!loads_as_it_is(h, h_ld) || p.width % 8 != 0) {
        T* to = reinterpret_cast<T*>(a.space + p.off_hidden);
        copies[many++] = Repack<T>{h, to, h_ld, p.tokens};
        h = to;
        h_ld = p.width_ld;
    }
    if (!loads_as_it_is(w, w_ld) || p.width % 8 != 0) {
        T* to = reinterpret_cast<T*>(a.space + p.off_weight);
        copies[many++] = Repack<T>{w, to, w_ld, p.vocab};
        w = to;
        w_ld = p.width_ld;
    }
    if (many > 0) {
        const int64_t first = ceil_div(copies[0].rows * p.width_ld, 2048);
        const int64_t all = first + (many > 1 ? ceil_div(copies[1].rows * p.width_ld, 2048) : 0);
        in_launches(all, 256, [&](int64_t base, int64_t count) {
            repack_kernel<T><<<dim3((unsigned)count), 256, 0, s>>>(copies[0], copies[many - 1], base, first, p.width, p.width_ld);
        });
    }
    auto total = [&](float* loss) {
        total_kernel<<<1, 1024, 0, s>>>(a.targets, a.losses, p.tokens, a.ignore_index, a.grad_scale, kHold<T>, alpha, loss);
    };
    hipError_t e = hipSuccess;
    if (p.tokens == 0) {
        total(a.loss);
        if (gradient) {                    // a sum over no tokens
            GradArgs g{};
            g.p = Operand{w, p.vocab_ld, p.vocab_ld, 0};
            g.q = Operand{w, w_ld, p.width, 0};
            g.alpha = alpha;
            g.rows = p.vocab;
            g.cols = p.width;
            g.splits = 1;
            g.out = a.dweight;
            g.out_ld = a.dweight_stride;
            e = grad<T, kOuter>(g, p.weight_tile, s);
        }
        return e != hipSuccess ? e : hipGetLastError();
    }
    const Operand ow{w, w_ld, p.vocab, p.width_ld};
    for (int64_t n0 = 0; n0 < p.tokens && e == hipSuccess; n0 += p.chunk) {
        const int64_t n = p.tokens - n0 < p.chunk ? p.tokens - n0 : p.chunk;
        const bool last = n0 + n == p.tokens;
        const Operand oh{h + n0 * h_ld, h_ld, n, p.width_ld};
        const int64_t held = p.pairs ? pair_rows(n) : n;        // rows of G
        const LogitsArgs l{oh, ow, a.targets + n0, target_logit, stats, exps, p.pairs, n, p.vocab, p.vocab_ld, p.pieces, 0, 0};
        if (p.logits_tile.ni == 2) e = logits<T, 2, 4>(l, s);
        else if (p.logits_tile.nj == 4) e = logits<T, 8, 4>(l, s);
        else e = logits<T, 8, 5>(l, s);
        if (e != hipSuccess) return e;
        T* kept = reinterpret_cast<T*>(a.space + p.off_hidden) + n0 * p.width_ld;
        const JoinArgs j{stats, target_logit, a.targets + n0, a.losses + n0, lse + n0, exps, p.pairs,
                         p.pieces, p.vocab, p.vocab_ld, a.ignore_index, oh.base, kept, h_ld, p.width_ld};
        // (a workgroup has 2048 ids at a time; 1024 workgroups fill the card)
        int64_t share = gradient && n < 1024 ? ceil_div(1024, n) : 1;
        if (share > ceil_div(p.vocab_ld, 2048)) share = ceil_div(p.vocab_ld, 2048);
        const dim3 joins((unsigned)n, (unsigned)share);
        const bool past = n * p.vocab_ld * 2 > kLastCache;
        if (p.logits_tile.nj == 4 && past) join_kernel<T, 4, true><<<joins, 256, 0, s>>>(j);
        else if (p.logits_tile.nj == 4) join_kernel<T, 4, false><<<joins, 256, 0, s>>>(j);
        else if (past) join_kernel<T, 5, true><<<joins, 256, 0, s>>>(j);
        else join_kernel<T, 5, false><<<joins, 256, 0, s>>>(j);
        if (n0 == 0 || last) total(last ? a.loss : nullptr);
        if (!gradient) continue;
        GradArgs g{};
        g.alpha = alpha;
        g.cols = p.width;
        // A product, in parts of its depth where that fills the card.
        auto product = [&](auto layout, int splits, const TileChoice& tile) {
            constexpr Layout LP = decltype(layout)::value;
            g.splits = splits;
            g.part = splits > 1 ? reinterpret_cast<float*>(a.space + p.off_split) : nullptr;
            const hipError_t err = grad<T, LP>(g, tile, s);
            if (err != hipSuccess || splits == 1) return err;
            T* out = static_cast<T*>(g.out);
            const int64_t all = g.rows * g.cols;
            if (g.cols % 4 == 0)
                join_splits_kernel<T, 4><<<dim3((unsigned)ceil_div(all, 1024)), 256, 0, s>>>(g.part, splits, g.rows, g.cols, alpha, out, g.out_ld);
            else
                join_splits_kernel<T, 1><<<dim3((unsigned)ceil_div(all, 256)), 256, 0, s>>>(g.part, splits, g.rows, g.cols, alpha, out, g.out_ld);
            return hipSuccess;
        };
        // dH = G W: k runs over the vocabulary
        g.p = Operand{exps, p.vocab_ld, held, p.vocab_ld};
        g.q = Operand{w, w_ld, p.width, p.vocab};
        g.rows = n;
        g.pairs = p.pairs;
        g.steps = p.vocab_ld / kDeep;
        g.out = static_cast<T*>(a.dhidden) + n0 * a.dhidden_stride;
        g.out_ld = a.dhidden_stride;
        e = product(std::integral_constant<Layout, kInner>{}, p.hidden_splits, p.hidden_tile);
        if (e != hipSuccess) return e;
        // dW = G^T H: k runs over the chunk's tokens; with several chunks the sum
        // stays in fp32 until the last
        g.p = Operand{exps, p.vocab_ld, p.vocab_ld, held, p.pairs ? n : 0};
        g.q = Operand{kept, p.width_ld, p.width_ld, n, p.pairs ? n : 0, true};
        g.rows = p.vocab;
        g.pairs = 0;
        g.steps = ceil_div(held, kDeep);
        g.out = a.dweight;
        g.out_ld = a.dweight_stride;
        g.sum = reinterpret_cast<float*>(a.space + p.off_sum);
        g.sum_in = n0 > 0;
        g.sum_out = !last;
        e = product(std::integral_constant<Layout, kOuter>{}, p.weight_splits, p.weight_tile);
    }
    return e != hipSuccess ? e : hipGetLastError();
}

// Rows up to which tiles of 64 are taken instead of 256.  At 16 tokens x 50257 x 1600
// they take 29, 30 and 44 us for the three products, against 38, 41 and 65.
constexpr int64_t kFewRows = 128;

// Tokens up to which an entry of G is held as two 2-byte numbers, the second what the
// first's rounding took away.  Of few tokens a single entry can make up most of a
// gradient, which is then off by that entry's rounding (4 tokens x 22719 x 57 fp16: the
// weight's gradient by 4.2e-4 of its norm, 2.2e-4 in pairs, as much as its own rounding).
// The second halves are rows of their own in the same tile of 64 and cost no product: 16
// tokens x 50257 x 1600 bf16 take 142 us, 138 without.
constexpr int64_t kPairs = 32;

// Rounds of tiles over the card.
int64_t rounds_of(int64_t rows, int64_t cols, const TileChoice& c, int64_t splits)
{
    return ceil_div(ceil_div(rows, 32 * c.ni) * ceil_div(cols, 64 * c.nj) * splits, kCUs * (c.ni == 2 ? 2 : 1));
}

// The tile of a gradient's product of `steps` steps, and into how many parts its depth
// goes, by what they should take: a step of 256 x 256 x 64 is 1.6 us, of 256 x 320
// 1.2 times that (at 8192 x 1600 x 50257 the weight's gradient takes 1124 us with it, in 4
// rounds, and 1350 without, in 6), of 64 x 256, two to a CU, 0.8; a round's beginning and
// end 4; and the parts go through memory at 4 TB/s, and through a launch.
TileChoice choose(int64_t rows, int64_t cols, int64_t steps, bool may_split, int* splits)
{
    const bool few = rows <= kFewRows;
    TileChoice tile{few ? 2 : 8, 4};
    double best = 0.0;
    *splits = 1;
    for (int nj = 4; nj <= (few ? 4 : 5); ++nj) {
        const TileChoice c{few ? 2 : 8, nj};
        // a part for every 8 steps at most (9 may go as 4 and 5), and no more than four rounds of them
        const int64_t tiles = ceil_div(rows, 32 * c.ni) * ceil_div(cols, 64 * c.nj);
        const int64_t most = may_split ? (steps + 7) / 8 : 1;
        for (int64_t k = 1; k <= most && (k == 1 || tiles * k <= 4 * kCUs); ++k) {
            const double step = few ? 0.8 : nj == 5 ? 1.92 : 1.6;
            const double t = rounds_of(rows, cols, c, k) * (ceil_div(steps, k) * step + 4.0) +
                             (k > 1 ? 2.0 * k * rows * cols * 4 / 4e6 + 5.0 : 0.0);
            if (best == 0.0 || t < best) {
                best = t;
                tile = c;
                *splits = (int)k;
            }
        }
    }
    return tile;
}

}  // namespace

LossPlan loss_plan(int64_t tokens, int64_t vocab, int64_t width, int64_t max_chunk, bool gradient)
{
    LossPlan p{};
    p.tokens = tokens;
    p.vocab = vocab;
    p.width = width;
    p.width_ld = round_up(width, 8);
    p.chunk = tokens < max_chunk ? tokens : max_chunk;
    if (p.chunk < 1) p.chunk = 1;
    // the logits: no parts; the larger tile where its rounds are fewer by enough
    const TileChoice narrow{8, 4}, wide{8, 5};
    p.logits_tile = p.chunk <= kFewRows ? TileChoice{2, 4}
                    : rounds_of(p.chunk, vocab, wide, 1) * 6 < rounds_of(p.chunk, vocab, narrow, 1) * 5 ? wide : narrow;
    p.vocab_ld = round_up(vocab, p.logits_tile.nj == 5 ? 320 : 64);      // whole pieces, whole steps
    p.pieces = p.vocab_ld / (16 * p.logits_tile.nj);
    p.pairs = gradient && p.chunk <= kPairs;
    p.hidden_tile = choose(p.chunk, width, p.vocab_ld / kDeep, true, &p.hidden_splits);
    p.weight_tile = choose(vocab, width, ceil_div(p.chunk, kDeep), p.chunk >= tokens, &p.weight_splits);
    if (p.chunk <= kFewRows) p.weight_tile = TileChoice{2, 4};           // one or two steps: storing is what takes the time
    const int64_t parts_hidden = p.hidden_splits > 1 ? p.hidden_splits * p.chunk * width : 0;
    const int64_t parts_weight = p.weight_splits > 1 ? p.weight_splits * vocab * width : 0;
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
    p.off_exp = take(gradient ? (p.pairs ? pair_rows(p.chunk) : p.chunk) * p.vocab_ld * 2 : 0);
    p.off_split = take(gradient ? (parts_hidden > parts_weight ? parts_hidden : parts_weight) * 4 : 0);
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
