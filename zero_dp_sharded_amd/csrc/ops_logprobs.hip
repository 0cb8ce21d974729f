// Log probabilities of given tokens, straight from hidden states H [tokens][width] and the output
// weight W [vocab][width], with each row's entropy and its largest alternatives:
//     z = H W^T ;  lse_n = log sum_v exp z_nv ;  logprob_n = z_n,token - lse_n
//     entropy_n = lse_n - sum_v p_nv z_nv ,  p = exp(z - lse)
//     the `top` largest z of a row, the lower id first where they are alike
// and the gradients of sum(d logprob) + sum(e entropy):
//     G_nv = d_n ([v is n's token] - p_nv) - e_n p_nv (z_nv - lse_n + entropy_n)
//     dH = G W ;  dW = G^T H
//
// Forward, a product whose epilogue takes each piece of a row (64 or 80 ids) to its maximum m, the sum
// of exp(z - m), and the sum of exp(z - m)(z - m), all fp32; a wave a token joins the pieces.
// entropy = log S - X / S of the joined sums about the row's maximum: both terms are
// positive, nothing cancels.  Where alternatives are asked for, the logits go to memory in fp32 for a
// chunk of tokens, and the wave reads only the pieces that can hold them: those whose
// maxima are the `top` largest (a piece below has as many elements before each of its own).  And only those
// are written: the first columns of tiles give each row a bound (columns_before), pieces below it stay
// where they are.  8192 x 50257 x 1600 bf16 with entropy and 5 alternatives 1270 us call after call; under a
// profiler, whose launches stand apart, 140 for the first columns, 1243 for the others (950 TFLOP/s with their
// epilogue), 7 for the bounds, 53 for the join.  Without alternatives, by tiles of 256 x 320, 1119, and 314 for 2048
// tokens.  16 tokens with 20 alternatives 61: 32 in the product, which reads W at 5 TB/s by 197 workgroups, and 19 in
// the join, a wave's chain of sums and rankings.
//
// Backward, the forward's lse and entropy make G in the epilogue of the same product: no pass over
// it lies between, as the loss has (ops_loss.hip), whose two other products follow.  What is held
// is G times a power of two that brings the largest |d| + |e| (1 + log vocab) to the top of the
// type's range (fp16: 2^15 of it), taken back in the products' epilogues.  2048 x 50257 x 1600 fp16 916 us: 343
// for G, 348 for each gradient.
//
// By the 4 waves to a tile of the 8-bit product, with 25 steps to a tile, 8192 tokens took 1222 us for 1277, and G of
// 2048 tokens, whose 256 x 320 tiles end better in rounds of the card, 380 for 335.  Both kernels have this one form: the
// forward's alone could have that.

#include <type_traits>

#include "ops_common.h"
#include "ops_gemm.h"
#include "ops_internal.h"
#include "ops_scaled.h"
#include "ops_vocab.h"

namespace zo {
namespace {

// A die's workgroups walk the tiles of H W^T, and load the next one while they are at a tile's
// results: out(i, j, acc).  Columns from tile j0 on.
template <typename T, int NI, int NJ, typename Out>
__device__ __forceinline__ void walk(const Operand& h, const Operand& w, uint32_t ti, uint32_t tj, uint32_t j0, char* smem, Out out)
{
    using G = Gemm<T, kInner, kInner, NI, NJ>;
    const uint32_t die = blockIdx.x % kDies, mine = tiles_of(die, ti * tj);
    const uint32_t stride = (gridDim.x + kDies - 1 - die) / kDies;       // workgroups of the die
    const int steps = (int)ceil_div(h.depth, kDeep);
    G g(h, w, lds_address(smem));
    int64_t bi = 0, bj = 0;
    uint32_t at = blockIdx.x / kDies;
    if (at >= mine) return;
    tile_of(die, at, ti, tj, bi, bj);
    bj += j0;
    g.begin(h, w, bi * G::kTileI, bj * G::kTileJ, 0, steps);
    for (;;) {
        f4 acc[NI][NJ];
        const int64_t i = bi, j = bj;
        at += stride;
        g.run(steps, acc, [&] {
            if (at >= mine) return;
            tile_of(die, at, ti, tj, bi, bj);
            bj += j0;
            g.begin(h, w, bi * G::kTileI, bj * G::kTileJ, 0, steps);
        });
        out(i, j, acc);
        if (at >= mine) return;
    }
}

// ------------------------------------------------------------------ forward

struct ScoreArgs {
    Operand h, w;
    const int64_t* tokens;      // of the chunk, or NULL
    float* given_logit;
    float2* stats;              // [tokens][pieces]: maximum and sum
    float* weighted;            // the sums of exp(z - m)(z - m), or NULL
    float* logits;              // [tokens][vocab_ld], or NULL
    const uint32_t* least;      // of a row, in order: pieces whose maxima are less are not written; or NULL
    int64_t count, vocab, vocab_ld, pieces;
    uint32_t ti, tj, j0;        // tiles, the first column of them
};

// Bits in the order of the values, NaN before all; -0 is 0.
__device__ __forceinline__ uint32_t in_order(float x)
{
    if (x != x) return 0;
    const uint32_t u = bits(x + 0.0f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}

// From a tile's logits to the pieces' statistics.
template <typename T, int NI, int NJ>
__device__ __forceinline__ void score_out(const ScoreArgs& a, int64_t bi, int64_t bj, f4 (&acc)[NI][NJ])
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
        if (NJ == 4 && (bj + 1) * G::kTileJ > a.vocab && m == -INFINITY) {
            // (what lies behind the vocabulary is no element: a piece with NaN alone before it has that for its largest)
            int some = 0;
#pragma unroll
            for (int k = 0; k < R; ++k) some |= v + k < a.vocab && acc[ti][k >> 2][k & 3] == acc[ti][k >> 2][k & 3];
            some |= __shfl_xor(some, 16, kWave);
            some |= __shfl_xor(some, 32, kWave);
            if (!some) m = __builtin_nanf("");
        }
        const int64_t token = a.tokens != nullptr && n < a.count ? a.tokens[n] : -1;
        const bool near = token >= v && token < v + 16;
        if (near || (NJ == 5 && token >= far + 16 && token < far + 20)) {
            // (a chain of selections: an index into the registers would put them in memory)
            const int at = (int)(token - (near ? v : far));
            float z = 0.0f;
#pragma unroll
            for (int k = 0; k < R; ++k) z = at == k ? acc[ti][k >> 2][k & 3] : z;
            a.given_logit[n] = z;
        }
        // a piece of -infinities has no exponentials: 0, not exp(-inf + inf)
        const float base = m == -INFINITY ? 0.0f : m;
        float sum = 0.0f, weighted = 0.0f;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const float d = acc[ti][k >> 2][k & 3] - base;
            const float e = __builtin_amdgcn_exp2f(d * kLog2e);
            sum += e;
            // (0 of -infinity is 0; NaN stays)
            weighted = fmaf(e, d == -INFINITY ? 0.0f : d, weighted);
        }
        sum += __shfl_xor(sum, 16, kWave);
        sum += __shfl_xor(sum, 32, kWave);
        weighted += __shfl_xor(weighted, 16, kWave);
        weighted += __shfl_xor(weighted, 32, kWave);
        if (n >= a.count) continue;
        if (lane < 16) {
            const int64_t piece = n * a.pieces + bj * 4 + (wave & 3);
            a.stats[piece] = make_float2(m, sum);
            if (a.weighted != nullptr) a.weighted[piece] = weighted;
        }
        if (NJ == 4 && a.logits != nullptr) {
            if (a.least != nullptr && in_order(m) < a.least[n]) continue;
            float* to = a.logits + n * a.vocab_ld + v;
#pragma unroll
            for (int q = 0; q < 4; ++q) store_vec<float, 4>(to + 4 * q, acc[ti][q]);
        }
    }
}

template <typename T, int NI, int NJ>
__global__ __launch_bounds__(kGemmThreads, 2) void score_kernel(ScoreArgs a)
{
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    walk<T, NI, NJ>(a.h, a.w, a.ti, a.tj, a.j0, smem, [&](int64_t i, int64_t j, f4 (&acc)[NI][NJ]) { score_out<T, NI, NJ>(a, i, j, acc); });
}

// ------------------------------------------------------------------ joining the pieces

struct ScoreJoin {
    const float2* stats;
    const float* weighted;      // NULL: no entropy
    const float* logits;        // NULL: no alternatives
    const float* given_logit;
    const int64_t* tokens;      // NULL: none given
    float* logprobs;
    float* lse;
    float* entropy;
    int64_t* top_ids;           // [tokens][top]
    float* top_logprobs;
    int64_t pieces, vocab, vocab_ld, ignore;
    int top;
};

// An element of an order by value, the lower id first where they are alike.
struct Ranked {
    uint32_t value;
    int32_t id;
    __device__ __forceinline__ bool before(const Ranked& o) const { return value > o.value || (value == o.value && id < o.id); }
};

constexpr int32_t kNoId = 0x7fffffff;

// The first of all lanes'.
__device__ __forceinline__ Ranked first_of(const Ranked& mine)
{
    const uint32_t value = lanes_max<64>(mine.value);
    const bool has = mine.value == value;
    const uint64_t who = __ballot(has);
    if (__popcll(who) == 1) return Ranked{value, __shfl(mine.id, __ffsll((unsigned long long)who) - 1, kWave)};
    return Ranked{value, (int32_t)~lanes_max<64>(has ? ~(uint32_t)mine.id : 0u)};
}

// The first `most` in order of what the lanes have, one after the other: next(e) is a lane's first behind
// e.  taken(r, e) is called by all lanes.
template <typename Next, typename Taken>
__device__ __forceinline__ void in_turn(int most, Next next, Taken taken)
{
    Ranked mine = next(Ranked{0xffffffffu, -1});
    for (int r = 0; r < most; ++r) {
        const Ranked e = first_of(mine);
        taken(r, e);
        // (the lane that had it has its next)
        if (mine.id == e.id && mine.value == e.value) mine = next(e);
    }
}

__device__ __forceinline__ void sooner(Ranked& best, const Ranked& last, const Ranked& e)
{
    if (last.before(e) && e.before(best)) best = e;
}

// The k-th largest of the 64 lanes' values (k from 1 to 64), by counting.
__device__ __forceinline__ uint32_t kth_of(uint32_t value, int k)
{
    const int lane = threadIdx.x & 63;
    int before = 0;
#pragma unroll
    for (int l = 0; l < 64; ++l) {
        const uint32_t other = __builtin_amdgcn_readlane(value, l);
        before += other > value || (other == value && l < lane);
    }
    const uint64_t who = __ballot(before == k - 1);
    return __builtin_amdgcn_readlane(value, __ffsll((unsigned long long)who) - 1);
}

// A bound for the `top` largest logits of a row from the maxima of its pieces: the top-th largest of what
// the lanes' shares of them (every 64th piece) reach.  So many elements are no less.
__device__ __forceinline__ uint32_t bound_of(uint32_t reach, int top, int pieces) { return pieces < top ? 0 : kth_of(reach, top); }

__global__ __launch_bounds__(64) void bound_kernel(const float2* stats, uint32_t* least, int64_t row_pieces, int pieces, int top)
{
    const float2* row = stats + (int64_t)blockIdx.x * row_pieces;
    uint32_t reach = 0;
    for (int p = threadIdx.x; p < pieces; p += 64) reach = larger(reach, in_order(row[p].x));
    reach = bound_of(reach, top, pieces);
    if (threadIdx.x == 0) least[blockIdx.x] = reach;
}

constexpr int kCandidates = 256;           // that are ranked by counting

// Adds the lanes' items that `is` says to a list in LDS.
__device__ __forceinline__ int append(int count, bool is, int lane)
{
    const uint64_t who = __ballot(is);
    return count + __popcll(who & ((1ull << lane) - 1));
}

// A token.  FEW: up to 1024 pieces, whose maxima stay in registers.
//
// The alternatives: of the pieces whose maxima reach the bound (as many as are asked for, and a few more) the
// logits that do are put into a list and ranked, each by how many are before it.  Where that
// would be more than the list holds (many logits alike) the pieces are taken one after the
// other in order, as many as are asked for, and then their logits.
template <bool FEW>
__global__ __launch_bounds__(64) void score_join_kernel(ScoreJoin a)
{
    extern __shared__ float held[];            // [top][64] logits
    __shared__ uint32_t values[kCandidates];
    __shared__ int32_t ids[kCandidates];
    constexpr int K = FEW ? 16 : 1;
    const int64_t n = blockIdx.x;
    const int lane = threadIdx.x;
    const float2* row = a.stats + n * a.pieces;
    const int pieces = (int)a.pieces;          // a lane has lane, lane + 64, ...
    float2 s[K];
    float m = -INFINITY;
    if constexpr (FEW) {
#pragma unroll
        for (int k = 0; k < K; ++k) s[k] = k * 64 + lane < pieces ? row[k * 64 + lane] : make_float2(-INFINITY, 0.0f);
#pragma unroll
        for (int k = 0; k < K; ++k) m = fmaxf(m, s[k].x);
    } else {
        for (int p = lane; p < pieces; p += 64) m = fmaxf(m, row[p].x);
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, kWave));
    const float base = m == -INFINITY ? 0.0f : m;
    double sum = 0.0, weighted = 0.0;
    auto add = [&](float2 part, float w) {
        // (a piece of -infinities adds nothing)
        const float d = part.x == -INFINITY ? 0.0f : part.x - base;
        const double f = part.x == -INFINITY ? 0.0 : (double)expf(d);
        sum += f * (double)part.y;
        weighted += f * ((double)w + (double)part.y * (double)d);
    };
    if constexpr (FEW) {
        float w[K];
#pragma unroll
        for (int k = 0; k < K; ++k) w[k] = a.weighted != nullptr && k * 64 + lane < pieces ? a.weighted[n * a.pieces + k * 64 + lane] : 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k * 64 + lane < pieces) add(s[k], w[k]);
    } else {
        for (int p = lane; p < pieces; p += 64) add(row[p], a.weighted != nullptr ? a.weighted[n * a.pieces + p] : 0.0f);
    }
    sum = lanes_sum(sum);
    weighted = lanes_sum(weighted);
    const double log_sum = log(sum), lse = (double)base + log_sum;
    if (lane == 0) {
        a.lse[n] = (float)lse;
        if (a.weighted != nullptr) a.entropy[n] = (float)(log_sum - weighted / sum);
        if (a.tokens != nullptr) {
            const int64_t t = a.tokens[n];
            const bool known = t >= 0 && t < a.vocab;
            a.logprobs[n] = t == a.ignore ? 0.0f : known ? (float)((double)a.given_logit[n] - lse) : __builtin_nanf("");
        }
    }
    if (a.top == 0) return;
    const float* z = a.logits + n * a.vocab_ld;
    auto piece = [&](int k) {                   // the lane's k-th
        const int p = k * 64 + lane;
        if (p >= pieces) return Ranked{0u, kNoId};
        if constexpr (FEW) return Ranked{in_order(s[k].x), p};
        else return Ranked{in_order(row[p].x), p};
    };
    const int rounds = (pieces + 63) / 64;
    uint32_t reach = 0;                         // (of NaN alone 0: a bound of 0, which all reach)
    if constexpr (FEW) {
#pragma unroll
        for (int k = 0; k < K; ++k) reach = larger(reach, piece(k).value);
    } else {
        for (int k = 0; k < rounds; ++k) reach = larger(reach, piece(k).value);
    }
    const uint32_t bound = bound_of(reach, a.top, pieces);
    int count = 0;
    auto collect = [&](int k) {
        const Ranked e = piece(k);
        const bool is = e.id != kNoId && e.value >= bound;
        const int at = append(count, is, lane);
        if (is && at < kCandidates) ids[at] = e.id;
        count += __popcll(__ballot(is));
    };
    if constexpr (FEW) {
#pragma unroll
        for (int k = 0; k < K; ++k) collect(k);
    } else {
        for (int k = 0; k < rounds; ++k) collect(k);
    }
    __syncthreads();
    if (count <= kCandidates) {
        // 16 pieces' logits at a time (their list is read before it is written over)
        const int chosen = count;
        int from[kCandidates / 64];
#pragma unroll
        for (int q = 0; q < kCandidates / 64; ++q) from[q] = q * 64 + lane < chosen ? ids[q * 64 + lane] : 0;
        __syncthreads();
        count = 0;
        for (int c = 0; c < chosen; c += 16) {
            float x[16];
            int32_t id[16];
            const int part = c >> 6;
            const int mine = part == 0 ? from[0] : part == 1 ? from[1] : part == 2 ? from[2] : from[3];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                id[k] = __builtin_amdgcn_readlane(mine, (c + k) & 63) * 64 + lane;
                x[k] = z[id[k]];
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const uint32_t value = in_order(x[k]);
                const bool is = c + k < chosen && id[k] < a.vocab && value >= bound;
                const int at = append(count, is, lane);
                if (is && at < kCandidates) {
                    values[at] = value;
                    ids[at] = id[k];
                }
                count += __popcll(__ballot(is));
            }
        }
        __syncthreads();
        if (count <= kCandidates) {
            for (int c = lane; c < count; c += 64) {
                const Ranked e{values[c], ids[c]};
                int before = 0;
#pragma unroll 8
                for (int k = 0; k < count; ++k) before += Ranked{values[k], ids[k]}.before(e);
                if (before < a.top) {
                    a.top_ids[n * a.top + before] = e.id;
                    a.top_logprobs[n * a.top + before] = (float)((double)z[e.id] - lse);
                }
            }
            return;
        }
    }
    __syncthreads();
    const int wanted = a.top < pieces ? a.top : pieces;
    in_turn(wanted, [&](const Ranked& last) {
        Ranked best{0, kNoId};
        if constexpr (FEW) {
#pragma unroll
            for (int k = 0; k < K; ++k) sooner(best, last, piece(k));
        } else {
            for (int k = 0; k < rounds; ++k) sooner(best, last, piece(k));
        }
        return best;
    }, [&](int r, const Ranked& e) {
        if (lane == 0) ids[r] = e.id * 64;
        held[r * 64 + lane] = z[(int64_t)e.id * 64 + lane];
    });
    __syncthreads();
    in_turn(a.top, [&](const Ranked& last) {
        Ranked best{0, kNoId};
        for (int k = 0; k < wanted; ++k) {
            const int32_t id = ids[k] + lane;
            if (id < a.vocab) sooner(best, last, Ranked{in_order(held[k * 64 + lane]), id});
        }
        return best;
    }, [&](int r, const Ranked& e) {
        if (lane != 0) return;
        a.top_ids[n * a.top + r] = e.id;
        a.top_logprobs[n * a.top + r] = (float)((double)z[e.id] - lse);
    });
}

// ------------------------------------------------------------------ backward

struct RowFactors {             // of a token
    float lse, d, e, entropy;   // d and e with the factor that G is held with
};

struct FactorArgs {
    const int64_t* tokens;
    const float* lse;
    const float* entropy;       // with dentropy
    const float* dlogprobs;
    const float* dentropy;      // or NULL
    float* alpha;               // the products' factor, and the inverse
    RowFactors* rows;
    const void* hidden;
    void* kept;                 // rows of width_ld, of tokens without any gradient zeros
    int64_t count, vocab, width, width_ld, hidden_ld, ignore;
    float spread;               // 1 + log vocab: what an entropy's entries reach
};

// d of a token: 0 where none is given, NaN where it is none of the vocabulary's.
__device__ __forceinline__ float given(const FactorArgs& a, int64_t n)
{
    const int64_t t = a.tokens[n];
    if (t == a.ignore) return 0.0f;
    return t >= 0 && t < a.vocab ? a.dlogprobs[n] : __builtin_nanf("");
}

// The factor: a power of two at least as large as any finite |d| + spread |e|, and what it makes of
// 2^kHoldLog2.
template <typename T>
__global__ __launch_bounds__(1024) void factor_kernel(FactorArgs a)
{
    __shared__ uint32_t sh[16];
    constexpr float kPart = 0x1p-8f;           // the sum passes fp32, not this part of it: spread is below 16
    uint32_t most = 0;
    for (int64_t n = threadIdx.x; n < a.count; n += 1024) {
        const float d = given(a, n), e = a.dentropy != nullptr ? a.dentropy[n] : 0.0f;
        most = with_size(most, kPart * fabsf(d) + kPart * a.spread * fabsf(e));
    }
    most = lanes_max<64>(most);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = most;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int k = 1; k < 16; ++k) most = larger(most, sh[k]);
    // (up to 133; not below what both factors can be in fp32)
    const int low = -126 + (int)kHoldLog2<T>;
    int up = low;
    if (most != 0) {
        (void)frexpf(from_bits(most), &up);
        up = up + 8 < low ? low : up + 8;
    }
    a.alpha[0] = ldexpf(1.0f, up - (int)kHoldLog2<T>);
    a.alpha[1] = ldexpf(1.0f, (int)kHoldLog2<T> - up);
}

// A wave a token: its factors and its hidden state (zeros where it has no gradient: 0 times what is
// not finite is NaN).
template <typename T>
__global__ __launch_bounds__(256) void rows_kernel(FactorArgs a, int64_t first)
{
    const int64_t n = (first + blockIdx.x) * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (n >= a.count) return;
    const float d = given(a, n), e = a.dentropy != nullptr ? a.dentropy[n] : 0.0f;
    const bool any = d != 0.0f || e != 0.0f;
    if (lane == 0) a.rows[n] = RowFactors{a.lse[n], d * a.alpha[1], e * a.alpha[1], e != 0.0f ? a.entropy[n] : 0.0f};
    const T* x = static_cast<const T*>(a.hidden) + n * a.hidden_ld;
    T* to = static_cast<T*>(a.kept) + n * a.width_ld;
    for (int64_t c = lane * 8; c < a.width_ld; c += 512) {
        vec_t<T, 8> y = {};
        if (any) {
            if (c + 8 <= a.width) {
                y = load_vec<T, 8>(x + c);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (c + k < a.width) y[k] = x[c + k];
            }
        }
        *reinterpret_cast<vec_t<T, 8>*>(to + c) = y;
    }
}

struct DScoreArgs {
    Operand h, w;
    const int64_t* tokens;      // of the chunk
    const RowFactors* rows;
    void* g;                    // [tokens][vocab_ld]
    int pairs;                  // entries in pairs: beside each what its rounding takes away (NI = 2)
    int64_t count, vocab, vocab_ld;
    uint32_t ti, tj;
};

// From a tile's logits to its entries of G.
template <typename T, int NI, int NJ>
__device__ __forceinline__ void dscore_out(const DScoreArgs& a, int64_t bi, int64_t bj, f4 (&acc)[NI][NJ])
{
    using G = Gemm<T, kInner, kInner, NI, NJ>;
    constexpr int R = 4 * NJ;
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));      // (addresses are made here, and not kept in registers over the products)
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t v = bj * G::kTileJ + G::column_of(0, wave, lane);
    const int64_t far = bj * G::kTileJ + G::column_of(4, wave, lane) - 16;
    if (bj * G::kTileJ + (wave & 3) * 64 >= a.vocab_ld) return;
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
        if (n >= a.count) continue;
        const RowFactors f = a.rows[n];
        const bool none = f.d == 0.0f && f.e == 0.0f;
        const int64_t token = a.tokens[n];
        const bool near = token >= v && token < v + 16;
        const int at = near ? (int)(token - v) : NJ == 5 && token >= far + 16 && token < far + 20 ? (int)(token - far) : -1;
        // the token's 1 - p by expm1, which does not cancel
        float rest = 0.0f;
        if (at >= 0) {
            float z = 0.0f;
#pragma unroll
            for (int k = 0; k < R; ++k) z = at == k ? acc[ti][k >> 2][k & 3] : z;
            rest = expm1f(z - f.lse);
        }
        vec_t<T, 4> high[NJ], low[NJ];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const float u = acc[ti][k >> 2][k & 3] - f.lse;
            const float p = __builtin_amdgcn_exp2f(u * kLog2e);
            const float own = -f.d * (at == k ? rest : p);
            // (p log p is 0 where p is, of -infinity too; d and e that are not finite stay so)
            float g = f.e != 0.0f ? fmaf(-f.e * p, p == 0.0f ? 0.0f : u + f.entropy, own) : own;
            if (none) g = 0.0f;
            high[k >> 2][k & 3] = static_cast<T>(g);
            if constexpr (NI == 2) low[k >> 2][k & 3] = static_cast<T>(g - (float)high[k >> 2][k & 3]);
        }
        T* to = static_cast<T*>(a.g) + (NI == 2 && a.pairs ? pair_row(n) : n) * a.vocab_ld;
#pragma unroll
        for (int q = 0; q < 2; ++q)
            reinterpret_cast<vec_t<T, 8>*>(to + v)[q] = __builtin_shufflevector(high[2 * q], high[2 * q + 1], 0, 1, 2, 3, 4, 5, 6, 7);
        if constexpr (NJ == 5) *reinterpret_cast<vec_t<T, 4>*>(to + far + 16) = high[4];
        if constexpr (NI == 2) {
            if (a.pairs) {
                auto* under = reinterpret_cast<vec_t<T, 8>*>(to + 16 * a.vocab_ld + v);
#pragma unroll
                for (int q = 0; q < 2; ++q) under[q] = __builtin_shufflevector(low[2 * q], low[2 * q + 1], 0, 1, 2, 3, 4, 5, 6, 7);
            }
        }
    }
}

template <typename T, int NI, int NJ>
__global__ __launch_bounds__(kGemmThreads, 2) void dscore_kernel(DScoreArgs a)
{
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    walk<T, NI, NJ>(a.h, a.w, a.ti, a.tj, 0, smem, [&](int64_t i, int64_t j, f4 (&acc)[NI][NJ]) { dscore_out<T, NI, NJ>(a, i, j, acc); });
}

// ------------------------------------------------------------------ launches

// Workgroups of a walk: as many as stand in the CUs at once: one, or two of the small tile's.
template <int NI>
unsigned standing(uint32_t tiles)
{
    const uint32_t stand = kCUs * (NI == 2 ? 2 : 1);
    return tiles < stand ? tiles : stand;
}

template <typename T, int NI, int NJ>
hipError_t score(ScoreArgs a, hipStream_t s)
{
    using G = Gemm<T, kInner, kInner, NI, NJ>;
    static const hipError_t allowed = allow(score_kernel<T, NI, NJ>, G::kLds);
    if (allowed != hipSuccess) return allowed;
    score_kernel<T, NI, NJ><<<dim3(standing<NI>(a.ti * a.tj)), kGemmThreads, G::kLds, s>>>(a);
    return hipSuccess;
}

template <typename T>
hipError_t score(const ScoreArgs& a, const TileChoice& tile, hipStream_t s)
{
    return tile.ni == 2 ? score<T, 2, 4>(a, s) : tile.nj == 5 ? score<T, 8, 5>(a, s) : score<T, 8, 4>(a, s);
}

template <typename T, int NI, int NJ>
hipError_t dscore(DScoreArgs a, hipStream_t s)
{
    using G = Gemm<T, kInner, kInner, NI, NJ>;
    static const hipError_t allowed = allow(dscore_kernel<T, NI, NJ>, G::kLds);
    if (allowed != hipSuccess) return allowed;
    a.ti = (uint32_t)ceil_div(a.count, G::kTileI);
    a.tj = (uint32_t)ceil_div(a.vocab, G::kTileJ);
    dscore_kernel<T, NI, NJ><<<dim3(standing<NI>(a.ti * a.tj)), kGemmThreads, G::kLds, s>>>(a);
    return hipSuccess;
}

// The operands as the products can load them: where they lie, or copies in the workspace.
template <typename T>
void lay_out(const void* hidden, int64_t hidden_stride, const void* weight, int64_t weight_stride, int64_t tokens, int64_t vocab, int64_t width,
             int64_t width_ld, void* hidden_room, void* weight_room, const T*& h, int64_t& h_ld, const T*& w, int64_t& w_ld, hipStream_t s)
{
    h = static_cast<const T*>(hidden);
    w = static_cast<const T*>(weight);
    h_ld = hidden_stride;
    w_ld = weight_stride;
    Repack<T> copies[2];
    int many = 0;
    if (hidden_room != nullptr && (!loads_as_it_is(h, h_ld) || width % 8 != 0)) {
        T* to = static_cast<T*>(hidden_room);
        copies[many++] = Repack<T>{h, to, h_ld, tokens};
        h = to;
        h_ld = width_ld;
    }
    if (!loads_as_it_is(w, w_ld) || width % 8 != 0) {
        T* to = static_cast<T*>(weight_room);
        copies[many++] = Repack<T>{w, to, w_ld, vocab};
        w = to;
        w_ld = width_ld;
    }
    if (many == 0) return;
    const int64_t first = ceil_div(copies[0].rows * width_ld, 2048);
    const int64_t all = first + (many > 1 ? ceil_div(copies[1].rows * width_ld, 2048) : 0);
    in_launches(all, 256, [&](int64_t base, int64_t count) {
        repack_kernel<T><<<dim3((unsigned)count), 256, 0, s>>>(copies[0], copies[many - 1], base, first, width, width_ld);
    });
}

// Tile columns whose logits are all written, so that their largest bound what has to be of the rest; 0: no
// such beginning.  With a share f of P pieces before, some top / f of the rest reach the bound: f is
// sqrt(top / P), in whole rounds of tiles over the card.
uint32_t columns_before(uint32_t ti, uint32_t tj, int top)
{
    const double share = sqrt((double)top / (4.0 * tj));
    const uint32_t rounds = (uint32_t)ceil(share * tj * ti / kCUs);
    const uint32_t columns = rounds * kCUs / ti;
    return ti < 4 || columns < 1 || columns > tj / 2 || columns * 4 < (uint32_t)top ? 0 : columns;
}

template <typename T>
hipError_t logprobs(const Logprobs& a, const LogprobPlan& p, hipStream_t s)
{
    const T *h, *w;
    int64_t h_ld, w_ld;
    lay_out<T>(a.hidden, a.hidden_stride, a.weight, a.weight_stride, p.tokens, p.vocab, p.width, p.width_ld, a.space + p.off_hidden,
               a.space + p.off_weight, h, h_ld, w, w_ld, s);
    float2* stats = reinterpret_cast<float2*>(a.space + p.off_stats);
    float* weighted = a.entropy != nullptr ? reinterpret_cast<float*>(a.space + p.off_weighted) : nullptr;
    float* logits = p.top > 0 ? reinterpret_cast<float*>(a.space + p.off_logits) : nullptr;
    float* given_logit = reinterpret_cast<float*>(a.space + p.off_given);
    for (int64_t n0 = 0; n0 < p.tokens; n0 += p.chunk) {
        const int64_t n = p.tokens - n0 < p.chunk ? p.tokens - n0 : p.chunk;
        const int64_t* tokens = a.tokens != nullptr ? a.tokens + n0 : nullptr;
        ScoreArgs sa{Operand{h + n0 * h_ld, h_ld, n, p.width_ld}, Operand{w, w_ld, p.vocab, p.width_ld}, tokens, given_logit, stats, weighted,
                     logits, nullptr, n, p.vocab, p.vocab_ld, p.pieces, 0, 0, 0};
        sa.ti = (uint32_t)ceil_div(n, 32 * p.tile.ni);
        sa.tj = (uint32_t)ceil_div(p.vocab, 64 * p.tile.nj);
        const uint32_t all = sa.tj, first = p.top > 0 ? columns_before(sa.ti, sa.tj, p.top) : 0;
        if (first > 0) {
            sa.tj = first;
            hipError_t e = score<T>(sa, p.tile, s);
            if (e != hipSuccess) return e;
            uint32_t* least = reinterpret_cast<uint32_t*>(a.space + p.off_least);
            bound_kernel<<<dim3((unsigned)n), 64, 0, s>>>(stats, least, p.pieces, (int)first * 4, p.top);
            sa.least = least;
            sa.j0 = first;
            sa.tj = all - first;
        }
        const hipError_t e = score<T>(sa, p.tile, s);
        if (e != hipSuccess) return e;
        const ScoreJoin j{stats, weighted, logits, given_logit, tokens, a.logprobs != nullptr ? a.logprobs + n0 : nullptr, a.lse + n0,
                          a.entropy != nullptr ? a.entropy + n0 : nullptr, a.top_ids != nullptr ? a.top_ids + n0 * p.top : nullptr,
                          a.top_logprobs != nullptr ? a.top_logprobs + n0 * p.top : nullptr, p.pieces, p.vocab, p.vocab_ld, a.ignore_index, p.top};
        const size_t lds = (size_t)p.top * 256;
        if (p.pieces <= 1024) score_join_kernel<true><<<dim3((unsigned)n), 64, lds, s>>>(j);
        else score_join_kernel<false><<<dim3((unsigned)n), 64, lds, s>>>(j);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t logprobs_backward(const LogprobsGrad& a, const LogprobGradPlan& p, hipStream_t s)
{
    const LossPlan& l = p.loss;
    const T *h, *w;
    int64_t h_ld, w_ld;
    lay_out<T>(a.hidden, a.hidden_stride, a.weight, a.weight_stride, l.tokens, l.vocab, l.width, l.width_ld, nullptr, a.space + l.off_weight, h, h_ld,
               w, w_ld, s);
    T* kept = reinterpret_cast<T*>(a.space + l.off_hidden);
    float* alpha = reinterpret_cast<float*>(a.space + l.off_alpha);
    RowFactors* rows = reinterpret_cast<RowFactors*>(a.space + p.off_rows);
    const FactorArgs f{a.tokens, a.lse, a.entropy, a.dlogprobs, a.dentropy, alpha, rows, h, kept, l.tokens, l.vocab, l.width, l.width_ld, h_ld,
                       a.ignore_index, 1.0f + logf((float)l.vocab)};
    factor_kernel<T><<<1, 1024, 0, s>>>(f);
    in_launches(ceil_div(l.tokens, 4), 256, [&](int64_t first, int64_t count) { rows_kernel<T><<<dim3((unsigned)count), 256, 0, s>>>(f, first); });
    T* g = reinterpret_cast<T*>(a.space + l.off_exp);
    constexpr int type = std::is_same<T, _Float16>::value ? 1 : 2;
    if (l.tokens == 0)                         // sums over no tokens
        return vocab_gradients(VocabChunk{g, kept, w, w_ld, nullptr, a.dweight, 0, a.dweight_stride, alpha, a.space, 0, true, true}, l, type, s);
    for (int64_t n0 = 0; n0 < l.tokens; n0 += l.chunk) {
        const int64_t n = l.tokens - n0 < l.chunk ? l.tokens - n0 : l.chunk;
        const DScoreArgs d{Operand{kept + n0 * l.width_ld, l.width_ld, n, l.width_ld}, Operand{w, w_ld, l.vocab, l.width_ld}, a.tokens + n0, rows + n0,
                           g, l.pairs, n, l.vocab, l.vocab_ld, 0, 0};
        hipError_t e = l.logits_tile.ni == 2 ? dscore<T, 2, 4>(d, s) : l.logits_tile.nj == 4 ? dscore<T, 8, 4>(d, s) : dscore<T, 8, 5>(d, s);
        if (e == hipSuccess)
            e = vocab_gradients(VocabChunk{g, kept + n0 * l.width_ld, w, w_ld, static_cast<T*>(a.dhidden) + n0 * a.dhidden_stride, a.dweight,
                                           a.dhidden_stride, a.dweight_stride, alpha, a.space, n, n0 == 0, n0 + n == l.tokens},
                                l, type, s);
        if (e != hipSuccess) return e;
    }
    return hipGetLastError();
}

}  // namespace

LogprobPlan logprob_plan(int64_t tokens, int64_t vocab, int64_t width, int64_t max_chunk, int top)
{
    LogprobPlan p{};
    const LossPlan l = loss_plan(tokens, vocab, width, max_chunk, false);       // the loss's tiles
    p.tokens = tokens;
    p.vocab = vocab;
    p.width = width;
    p.width_ld = l.width_ld;
    p.chunk = l.chunk;
    p.top = top;
    p.tile = l.logits_tile;
    // (pieces have to lie in the order of their ids where they are chosen by it)
    if (top > 0 && p.tile.nj == 5) p.tile.nj = 4;
    p.vocab_ld = round_up(vocab, p.tile.nj == 5 ? 320 : 64);
    p.pieces = p.vocab_ld / (16 * p.tile.nj);
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t off = at;
        at += round_up(bytes, 256);
        return off;
    };
    p.off_given = take(p.chunk * 4);
    p.off_stats = take(p.chunk * p.pieces * 8);
    p.off_weighted = take(p.chunk * p.pieces * 4);
    p.off_least = take(p.chunk * 4);
    p.off_logits = take(top > 0 ? p.chunk * p.vocab_ld * 4 : 0);
    p.off_hidden = take(tokens * p.width_ld * 2);
    p.off_weight = take(vocab * p.width_ld * 2);
    p.bytes = at;
    return p;
}

LogprobGradPlan logprob_grad_plan(int64_t tokens, int64_t vocab, int64_t width, int64_t max_chunk)
{
    LogprobGradPlan p{};
    p.loss = loss_plan(tokens, vocab, width, max_chunk, true);
    p.off_rows = p.loss.bytes;
    p.bytes = p.off_rows + round_up(tokens * (int64_t)sizeof(RowFactors), 256);
    return p;
}

hipError_t logprobs_forward(const Logprobs& a, const LogprobPlan& p, int type, hipStream_t s)
{
    return type == 1 ? logprobs<_Float16>(a, p, s) : logprobs<__bf16>(a, p, s);
}

hipError_t logprobs_backward(const LogprobsGrad& a, const LogprobGradPlan& p, int type, hipStream_t s)
{
    return type == 1 ? logprobs_backward<_Float16>(a, p, s) : logprobs_backward<__bf16>(a, p, s);
}

}  // namespace zo
