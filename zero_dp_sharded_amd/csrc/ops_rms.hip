// Root-mean-square norm over the last dimension, with the residual's addition in front:
//     h = round(x + r) ;  rstd = 1 / sqrt(sum h^2 / D + eps) ;  y = h rstd w
// y in storage, or in 8 bits with a power of two for every 128 elements (ops_scaled.h), or
// both; and backward, with the gradient dh that comes down the residual's way:
//     xhat = h rstd ;  g = dy w ;  dx = rstd (g - xhat mean(g xhat)) + dh
//     dw = sum_rows dy xhat
// Backward in fp32, forward in 64 bits; h, the codes and the gradients are rounded once, y by way of fp32.  The norm
// is of h as it is held: what the backward pass reads.
//
// Bound by memory where rows are whole vectors of its waves, as the layer norm (ops_norm.hip), and laid
// out as it is: a row in the registers of one to 16 waves between its sum and its results, rows of more
// than 16384 elements read again from cache.  Sums over a wave are moves within the vector unit.  8192 x 5120
// bf16 with a residual into 8 bits 58 us, 5.1 TB/s.
//
// Where a row ends within a vector of its waves, or before it (1600, 1601 elements of 2 bytes), load_raw's branch for single
// elements, which waits for every load before it, makes a chain of the loads: x's, then the residual's, then, behind
// the sum, the weight's.  4099 x 1601 fp16 13 us, of which its bytes are 8; a row of 1600 5.5.
//
// Backward, a workgroup walks rows and keeps its sums for dw, which a second kernel adds in
// order.  The next row is asked for before this one's sum; at widths as those the branch waits for it there, and
// the loads hide behind nothing but other waves.  16384 x 1600 bf16 with dh 40 us, 5.2 TB/s, and 4.5 for the sums.

#include "ops_common.h"
#include "ops_internal.h"
#include "ops_scaled.h"

namespace zo {
namespace {

// Results of more bytes than the L2s hold are written past them, as the layer norm's.
constexpr int64_t kCaches = 32 << 20;

// Sum of x over the NW waves of a row, the same in each.
template <int NW, typename F>
__device__ __forceinline__ F row_sum(F x, F* sh)
{
    x = lanes_sum(x);
    if constexpr (NW > 1) {
        __syncthreads();                       // the last sums have been read
        if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = x;
        __syncthreads();
        x = 0;
#pragma unroll
        for (int k = 0; k < NW; ++k) x += sh[k];
    }
    return x;
}

// The W elements from column c on, zeros past the width.
template <typename T, int W>
__device__ __forceinline__ vec_t<T, W> load_raw(const T* row, int64_t c, int64_t width)
{
    if (c + W <= width) return load_vec<T, W>(row + c);
    vec_t<T, W> v;
#pragma unroll
    for (int k = 0; k < W; ++k) v[k] = c + k < width ? row[c + k] : static_cast<T>(0.0f);
    return v;
}

template <typename T, int W>
__device__ __forceinline__ void load_part(const T* row, int64_t c, int64_t width, float (&x)[W])
{
    const vec_t<T, W> v = load_raw<T, W>(row, c, width);
#pragma unroll
    for (int k = 0; k < W; ++k) x[k] = (float)v[k];
}

template <bool PAST, typename T, int W>
__device__ __forceinline__ void store_raw(T* row, int64_t c, int64_t width, vec_t<T, W> v)
{
    if (c + W <= width) {
        store_vec<T, W, PAST>(row + c, v);
    } else {
#pragma unroll
        for (int k = 0; k < W; ++k)
            if (c + k < width) row[c + k] = v[k];
    }
}

template <bool PAST, typename T, int W>
__device__ __forceinline__ void store_part(T* row, int64_t c, int64_t width, const float (&x)[W])
{
    vec_t<T, W> v;
#pragma unroll
    for (int k = 0; k < W; ++k) v[k] = static_cast<T>(x[k]);
    store_raw<PAST, T, W>(row, c, width, v);
}

// x[0..W) of column c as codes; 128 / W lanes have a block.  All lanes of a block's group
// come here together (those past the width with zeros).
template <int W>
__device__ __forceinline__ void store_codes(uint8_t* row, uint8_t* exps, int64_t c, int64_t width, const float (&x)[W])
{
    uint32_t big = 0;
#pragma unroll
    for (int k = 0; k < W; ++k) big = larger(big, bits(x[k]) & 0x7fffffffu);
    if (big >= kNotFinite) {
        big = 0;
#pragma unroll
        for (int k = 0; k < W; ++k) big = with_size(big, x[k]);
    }
    const uint32_t E = scale_of(lanes_max<kScaleBlock / W>(big));
    if (c >= width) return;
    vec_t<uint32_t, W / 4> v;
#pragma unroll
    for (int q = 0; q < W / 4; ++q) v[q] = codes_of(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3], E);
    if (c + W <= width) {
        __builtin_memcpy(row + c, &v, W);
    } else {
#pragma unroll
        for (int k = 0; k < W; ++k)
            if (c + k < width) row[c + k] = (uint8_t)(v[k / 4] >> (8 * (k % 4)));
    }
    if (c % kScaleBlock == 0) exps[c / kScaleBlock] = (uint8_t)E;
}

// The sum of squares, rstd and y are in 64 bits before they are rounded: no square passes its range, and a
// result in 8 bits, which changes by a whole step where y lies next to a middle, is the
// definition's (the vector unit's 64-bit rate is its 32-bit one).
__device__ __forceinline__ double rstd_of(double q, int64_t width, double eps) { return 1.0 / sqrt(q / (double)width + eps); }

// y in fp32, which storage takes (2 bytes are rounded again: off by 2^-24 of y more than half a step at most).
// ODD: rounded to odd, for codes: 24 bits of which the last says whether any was lost, so that none comes to lie on a
// middle that is not there already, and the second rounding is of y itself.  (To the nearest twice, 15 to 23 of 8192 x
// 5120 codes were a step off; 56 us then, 58 so.  Done only where fp32 looks like a middle it keeps more in registers: 62.)
template <bool ODD>
__device__ __forceinline__ float scaled(float x, double rstd, float w)
{
    const double y = (double)x * (rstd * (double)w);
    if constexpr (!ODD) return (float)y;
    constexpr uint32_t kLost = (1u << 29) - 1;             // of the 52 bits of a mantissa the last 29
    const uint64_t u = __builtin_bit_cast(uint64_t, y);
    const uint32_t low = (uint32_t)u, kept = (low | ((low & kLost) + kLost)) & ~kLost;
    return (float)__builtin_bit_cast(double, (u >> 32) << 32 | kept);
}

// ------------------------------------------------------------------ forward

template <typename A, int W>
__device__ __forceinline__ void load_weight(const RmsForward& a, int64_t c, float (&w)[W])
{
#pragma unroll
    for (int e = 0; e < W; ++e) w[e] = 1.0f;
    if (a.weight != nullptr) load_part<A, W>(static_cast<const A*>(a.weight), c, a.width, w);
}

// x[0..W) of column c, normed: to y, or (CODED) as codes, and to y where that is given too.  All lanes of a block's group
// come here together.
template <bool PAST, bool CODED, typename A, typename T, int W>
__device__ __forceinline__ void put_results(const RmsForward& a, int64_t row, T* y, int64_t c, const float (&x)[W], double rstd)
{
    float r[W];
    if (!CODED || y != nullptr) {
        load_weight<A>(a, c, r);
#pragma unroll
        for (int e = 0; e < W; ++e) r[e] = scaled<false>(x[e], rstd, r[e]);
        if (c < a.width) store_part<PAST>(y, c, a.width, r);
    }
    if constexpr (CODED) {
        load_weight<A>(a, c, r);
#pragma unroll
        for (int e = 0; e < W; ++e) r[e] = scaled<true>(x[e], rstd, r[e]);
        // (past the width 0: inf or NaN as rstd make NaN of the zeros there)
#pragma unroll
        for (int e = 0; e < W; ++e)
            if (c + e >= a.width) r[e] = 0.0f;
        store_codes<W>(a.codes + row * a.codes_stride, a.exps + row * a.exps_stride, c, a.width, r);
    }
}

// NW waves a row, K vectors a lane; with NW == 1 a workgroup has 4 rows.
template <typename T, typename A, bool PAST, bool CODED, int NW, int K>
__global__ __launch_bounds__(NW == 1 ? 256 : NW * 64) void rms_forward_kernel(RmsForward a)
{
    constexpr int W = Vec<T>::W;
    __shared__ double sh[NW];
    const int lane = NW == 1 ? threadIdx.x & 63 : threadIdx.x;
    const int64_t row = NW == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
    if (row >= a.rows) return;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    float v[K][W];
    {
        vec_t<T, W> in[K];
#pragma unroll
        for (int k = 0; k < K; ++k) in[k] = load_raw<T, W>(x, (int64_t)(k * NW * 64 + lane) * W, a.width);
        if (a.residual != nullptr) {
            const T* r = static_cast<const T*>(a.residual) + row * a.residual_stride;
            T* h = static_cast<T*>(a.h) + row * a.h_stride;
            vec_t<T, W> add[K];
#pragma unroll
            for (int k = 0; k < K; ++k) add[k] = load_raw<T, W>(r, (int64_t)(k * NW * 64 + lane) * W, a.width);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int64_t c = (int64_t)(k * NW * 64 + lane) * W;
#pragma unroll
                for (int e = 0; e < W; ++e) in[k][e] = static_cast<T>((float)in[k][e] + (float)add[k][e]);
                if (c < a.width) store_raw<PAST, T, W>(h, c, a.width, in[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < W; ++e) v[k][e] = (float)in[k][e];
    }
    double q = 0.0;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < W; ++e) q = fma((double)v[k][e], (double)v[k][e], q);
    const double rstd = rstd_of(row_sum<NW>(q, sh), a.width, a.eps);
    if (lane == 0 && a.rstd != nullptr) a.rstd[row] = (float)rstd;
    T* y = a.y != nullptr ? static_cast<T*>(a.y) + row * a.y_stride : nullptr;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t c = (int64_t)(k * NW * 64 + lane) * W;
        put_results<PAST, CODED, A>(a, row, y, c, v[k], rstd);
    }
}

// Rows too long for registers: 16 waves walk the row twice.
template <typename T, typename A, bool PAST, bool CODED>
__global__ __launch_bounds__(1024) void rms_forward_long_kernel(RmsForward a)
{
    constexpr int W = Vec<T>::W;
    __shared__ double sh[16];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const int64_t c0 = (int64_t)threadIdx.x * W, step = 1024 * W;
    const T* from = x;                         // h: x, or the sum
    double q = 0.0;
    if (a.residual != nullptr) {
        const T* r = static_cast<const T*>(a.residual) + row * a.residual_stride;
        T* h = static_cast<T*>(a.h) + row * a.h_stride;
        from = h;
        for (int64_t c = c0; c < a.width; c += step) {
            vec_t<T, W> in = load_raw<T, W>(x, c, a.width), add = load_raw<T, W>(r, c, a.width);
#pragma unroll
            for (int e = 0; e < W; ++e) {
                in[e] = static_cast<T>((float)in[e] + (float)add[e]);
                q = fma((double)(float)in[e], (double)(float)in[e], q);
            }
            store_raw<false, T, W>(h, c, a.width, in);       // (a lane reads back what it wrote)
        }
    } else {
        for (int64_t c = c0; c < a.width; c += step) {
            float v[W];
            load_part<T, W>(x, c, a.width, v);
#pragma unroll
            for (int e = 0; e < W; ++e) q = fma((double)v[e], (double)v[e], q);
        }
    }
    const double rstd = rstd_of(row_sum<16>(q, sh), a.width, a.eps);
    if (threadIdx.x == 0 && a.rstd != nullptr) a.rstd[row] = (float)rstd;
    T* y = a.y != nullptr ? static_cast<T*>(a.y) + row * a.y_stride : nullptr;
    // (whole blocks: the lanes of one come to its codes together)
    for (int64_t c = c0; c < round_up(a.width, kScaleBlock); c += step) {
        float v[W];
        load_part<T, W>(from, c, a.width, v);
        put_results<PAST, CODED, A>(a, row, y, c, v, rstd);
    }
}

// ------------------------------------------------------------------ backward

// A workgroup of WAVES waves, NW to a row, walks rows blockIdx, blockIdx + grid, ... (in
// groups of WAVES / NW), asks for the next row before it is at one, and keeps its sums for dw.
// With one wave a row the weight is kept in LDS, to have the registers for that.
template <typename T, typename A, bool PAST, int NW, int WAVES, int K>
__global__ __launch_bounds__(WAVES * 64) void rms_backward_kernel(RmsBackward a)
{
    constexpr int W = Vec<T>::W;
    constexpr int ROWS = WAVES / NW;
    static_assert(ROWS == 1 || NW == 1, "several rows a workgroup: a wave each");
    constexpr bool AHEAD = NW <= 4;
    __shared__ float sh[NW];
    // the weight, 4 elements a lane side by side (AHEAD); at the end, with ROWS > 1, the
    // sums of the waves, [K * W][64]
    extern __shared__ __attribute__((aligned(16))) float fold[];
    const int lane = NW == 1 ? threadIdx.x & 63 : threadIdx.x;
    const int wave = threadIdx.x >> 6;
    const float inv = 1.0f / (float)a.width;
    float dw[K][W];
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int e = 0; e < W; ++e) dw[k][e] = 0.0f;
    }
    auto load_weight = [&](int k, float (&w)[W]) {
#pragma unroll
        for (int e = 0; e < W; ++e) w[e] = 1.0f;
        if (a.weight != nullptr)
            load_part<A, W>(static_cast<const A*>(a.weight), (int64_t)(k * NW * 64 + lane) * W, a.width, w);
    };
    if constexpr (AHEAD) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float w[W];
            load_weight(k, w);
#pragma unroll
            for (int e = 0; e < W; ++e) fold[((k * (W / 4) + e / 4) * NW * 64 + lane) * 4 + e % 4] = w[e];
        }
        __syncthreads();
    }
    auto weight = [&](int k, float (&w)[W]) {
        if constexpr (AHEAD) {
#pragma unroll
            for (int q = 0; q < W / 4; ++q) {
                const vec_t<float, 4> v =
                    *reinterpret_cast<const vec_t<float, 4>*>(fold + ((k * (W / 4) + q) * NW * 64 + lane) * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) w[q * 4 + e] = v[e];
            }
        } else {
            load_weight(k, w);
        }
    };
    const int64_t stride = (int64_t)gridDim.x * ROWS;
    int64_t row = (int64_t)blockIdx.x * ROWS + (NW == 1 ? wave : 0);
    vec_t<T, W> nx[K], ng[K], nd[K];           // the next row, as it lies in memory
    auto fetch = [&](int64_t r) {
        const T* hr = static_cast<const T*>(a.h) + r * a.h_stride;
        const T* dyr = static_cast<const T*>(a.dy) + r * a.dy_stride;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t c = (int64_t)(k * NW * 64 + lane) * W;
            nx[k] = load_raw<T, W>(hr, c, a.width);
            ng[k] = load_raw<T, W>(dyr, c, a.width);
        }
        if (a.dh != nullptr) {
            const T* dhr = static_cast<const T*>(a.dh) + r * a.dh_stride;
#pragma unroll
            for (int k = 0; k < K; ++k) nd[k] = load_raw<T, W>(dhr, (int64_t)(k * NW * 64 + lane) * W, a.width);
        }
    };
    float nrstd = 0.0f;
    if (a.dh == nullptr) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < W; ++e) nd[k][e] = static_cast<T>(0.0f);
    }
    if (AHEAD && row < a.rows) {
        fetch(row);
        nrstd = a.rstd[row];
    }
    // (rows of NW == 1 end wave by wave, the others' workgroups together: no barrier is
    // missed)
    for (; row < a.rows; row += stride) {
        if constexpr (!AHEAD) {
            fetch(row);
            nrstd = a.rstd[row];
        }
        float x[K][W], g[K][W];
        vec_t<T, W> d[K];
        const float rstd = nrstd;
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int e = 0; e < W; ++e) {
                x[k][e] = (float)nx[k][e] * rstd;
                g[k][e] = (float)ng[k][e];
            }
            d[k] = nd[k];
            // past the width h is 0, and 0 times an infinite rstd is none: both are 0 there
            const int left = (int)a.width - (k * NW * 64 + lane) * W;
            if (left < W) {
#pragma unroll
                for (int e = 0; e < W; ++e)
                    if (e >= left) x[k][e] = 0.0f;
            }
        }
        if (AHEAD && row + stride < a.rows) {
            fetch(row + stride);
            nrstd = a.rstd[row + stride];
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float w[W];
            weight(k, w);
#pragma unroll
            for (int e = 0; e < W; ++e) {
                dw[k][e] = fmaf(g[k][e], x[k][e], dw[k][e]);
                g[k][e] *= w[e];
                s = fmaf(g[k][e], x[k][e], s);
            }
        }
        s = row_sum<NW>(s, sh) * inv;
        T* dxr = static_cast<T*>(a.dx) + row * a.dx_stride;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t c = (int64_t)(k * NW * 64 + lane) * W;
            if (c >= a.width) continue;
#pragma unroll
            for (int e = 0; e < W; ++e) g[k][e] = fmaf(rstd, fmaf(-x[k][e], s, g[k][e]), (float)d[k][e]);
            store_part<PAST>(dxr, c, a.width, g[k]);
        }
    }
    if (a.partial == nullptr) return;
    float* out = a.partial + (int64_t)blockIdx.x * a.width;
    if constexpr (ROWS > 1) {
        // the waves' sums, one wave after the other, once all are done with the weight
        __syncthreads();
        for (int turn = 0; turn < ROWS; ++turn) {
            if (wave == turn) {
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int e = 0; e < W; ++e) {
                        const int at = (k * W + e) * 64 + lane;
                        if (turn > 0) dw[k][e] += fold[at];
                        fold[at] = dw[k][e];
                    }
            }
            __syncthreads();
        }
        if (wave != ROWS - 1) return;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t c = (int64_t)(k * NW * 64 + lane) * W;
        if (c < a.width) store_part<false>(out, c, a.width, dw[k]);
    }
}

// Rows too long for registers: dx row by row, and the sums for dw over slabs of rows, a
// lane W columns.
template <typename T, typename A, bool PAST>
__global__ __launch_bounds__(1024) void rms_backward_long_kernel(RmsBackward a)
{
    constexpr int W = Vec<T>::W;
    __shared__ float sh[16];
    const int64_t row = blockIdx.x;
    const T* hr = static_cast<const T*>(a.h) + row * a.h_stride;
    const T* dyr = static_cast<const T*>(a.dy) + row * a.dy_stride;
    const T* dhr = a.dh != nullptr ? static_cast<const T*>(a.dh) + row * a.dh_stride : nullptr;
    T* dxr = static_cast<T*>(a.dx) + row * a.dx_stride;
    const float rstd = a.rstd[row], inv = 1.0f / (float)a.width;
    const int64_t c0 = (int64_t)threadIdx.x * W, step = 1024 * W;
    float s = 0.0f;
    for (int turn = 0; turn < 2; ++turn) {
        for (int64_t c = c0; c < a.width; c += step) {
            float x[W], g[W], w[W];
            load_part<T, W>(hr, c, a.width, x);
            load_part<T, W>(dyr, c, a.width, g);
            if (a.weight != nullptr) {
                load_part<A, W>(static_cast<const A*>(a.weight), c, a.width, w);
#pragma unroll
                for (int e = 0; e < W; ++e) g[e] *= w[e];
            }
#pragma unroll
            for (int e = 0; e < W; ++e) x[e] = c + e < a.width ? x[e] * rstd : 0.0f;
            if (turn == 0) {
#pragma unroll
                for (int e = 0; e < W; ++e) s = fmaf(g[e], x[e], s);
                continue;
            }
            float d[W];
#pragma unroll
            for (int e = 0; e < W; ++e) d[e] = 0.0f;
            if (dhr != nullptr) load_part<T, W>(dhr, c, a.width, d);
#pragma unroll
            for (int e = 0; e < W; ++e) g[e] = fmaf(rstd, fmaf(-x[e], s, g[e]), d[e]);
            store_part<PAST>(dxr, c, a.width, g);
        }
        if (turn == 0) s = row_sum<16>(s, sh) * inv;
    }
}

template <typename T>
__global__ __launch_bounds__(256) void rms_columns_kernel(RmsBackward a, int64_t slab)
{
    constexpr int W = Vec<T>::W;
    const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * W;
    if (c >= a.width) return;
    float dw[W];
#pragma unroll
    for (int e = 0; e < W; ++e) dw[e] = 0.0f;
    const int64_t r0 = blockIdx.y * slab, r1 = r0 + slab < a.rows ? r0 + slab : a.rows;
    for (int64_t row = r0; row < r1; ++row) {
        float x[W], g[W];
        load_part<T, W>(static_cast<const T*>(a.h) + row * a.h_stride, c, a.width, x);
        load_part<T, W>(static_cast<const T*>(a.dy) + row * a.dy_stride, c, a.width, g);
        const float rstd = a.rstd[row];
#pragma unroll
        for (int e = 0; e < W; ++e) dw[e] = fmaf(g[e], x[e] * rstd, dw[e]);
    }
    store_part<false>(a.partial + (int64_t)blockIdx.y * a.width, c, a.width, dw);
}

// dw: the partial rows, added in 16 runs by 16 waves, the runs in order.
template <typename A>
__global__ __launch_bounds__(1024) void rms_fold_kernel(const float* partial, int64_t parts, int64_t width, A* dweight)
{
    __shared__ float sh[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    const int64_t p0 = parts * wave / 16, p1 = parts * (wave + 1) / 16;
    float s = 0.0f;
    if (c < width) {
#pragma unroll 16
        for (int64_t p = p0; p < p1; ++p) s += partial[p * width + c];
    }
    sh[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || c >= width) return;
#pragma unroll
    for (int k = 1; k < 16; ++k) s += sh[k][lane];
    dweight[c] = static_cast<A>(s);
}

// ------------------------------------------------------------------ launches

constexpr int64_t kLongRows = 64;      // workgroups over the rows of very long ones

// The arrays from row `first` on.
template <typename T>
RmsForward from_row(RmsForward a, int64_t first)
{
    a.x = static_cast<const T*>(a.x) + first * a.x_stride;
    if (a.residual != nullptr) {
        a.residual = static_cast<const T*>(a.residual) + first * a.residual_stride;
        a.h = static_cast<T*>(a.h) + first * a.h_stride;
    }
    if (a.y != nullptr) a.y = static_cast<T*>(a.y) + first * a.y_stride;
    if (a.rstd != nullptr) a.rstd += first;
    if (a.codes != nullptr) {
        a.codes += first * a.codes_stride;
        a.exps += first * a.exps_stride;
    }
    a.rows -= first;
    return a;
}

template <typename T>
RmsBackward from_row(RmsBackward a, int64_t first)
{
    a.dy = static_cast<const T*>(a.dy) + first * a.dy_stride;
    a.h = static_cast<const T*>(a.h) + first * a.h_stride;
    if (a.dh != nullptr) a.dh = static_cast<const T*>(a.dh) + first * a.dh_stride;
    a.dx = static_cast<T*>(a.dx) + first * a.dx_stride;
    a.rstd += first;
    a.rows -= first;
    return a;
}

template <typename T, typename A, bool PAST, bool CODED>
hipError_t forward_rows(const RmsForward& a, hipStream_t s)
{
    constexpr int W = Vec<T>::W;
    // lanes that a row keeps busy with one vector each; a wave keeps up to 64 elements of a
    // lane in registers
    const int64_t lanes = ceil_div(a.width, W);
    auto run = [&](auto kernel, int threads, int rows) {
        in_launches(ceil_div(a.rows, rows), threads, [&](int64_t first, int64_t count) {
            kernel<<<dim3((unsigned)count), threads, 0, s>>>(from_row<T>(a, first * rows));
        });
    };
    constexpr int M = 8 / W;               // vectors of a lane in 8 elements
    if (lanes <= 64 * M) run(rms_forward_kernel<T, A, PAST, CODED, 1, M>, 256, 4);
    else if (lanes <= 128 * M) run(rms_forward_kernel<T, A, PAST, CODED, 1, 2 * M>, 256, 4);
    else if (lanes <= 256 * M) run(rms_forward_kernel<T, A, PAST, CODED, 1, 4 * M>, 256, 4);
    else if (lanes <= 512 * M) run(rms_forward_kernel<T, A, PAST, CODED, 4, 2 * M>, 256, 1);
    else if (lanes <= 768 * M) run(rms_forward_kernel<T, A, PAST, CODED, 4, 3 * M>, 256, 1);
    else if (lanes <= 1024 * M) run(rms_forward_kernel<T, A, PAST, CODED, 4, 4 * M>, 256, 1);
    else if (lanes <= 2048 * M) run(rms_forward_kernel<T, A, PAST, CODED, 16, 2 * M>, 1024, 1);
    else run(rms_forward_long_kernel<T, A, PAST, CODED>, 1024, 1);
    return hipGetLastError();
}

template <typename T, typename A, bool PAST>
hipError_t backward_rows(const RmsBackward& a, hipStream_t s)
{
    constexpr int W = Vec<T>::W;
    const int64_t lanes = ceil_div(a.width, W);
    int64_t parts = 0;
    if (a.rows > 0) {
        // `most` workgroups walk the rows: what their registers let stand in the CUs
        auto run = [&](auto kernel, int waves, int rows, int k, int64_t most) {
            parts = ceil_div(a.rows, rows);
            if (parts > most) parts = most;
            const size_t lds = rows > 1 ? (size_t)k * W * 64 * sizeof(float) : waves == 4 ? (size_t)k * W * 256 * sizeof(float) : 0;
            kernel<<<dim3((unsigned)parts), waves * 64, lds, s>>>(a);
        };
        constexpr int M = 8 / W;           // vectors of a lane in 8 elements
        if (lanes <= 64 * M) run(rms_backward_kernel<T, A, PAST, 1, 16, M>, 16, 16, M, kCUs);
        else if (lanes <= 128 * M) run(rms_backward_kernel<T, A, PAST, 1, 8, 2 * M>, 8, 8, 2 * M, kCUs);
        else if (lanes <= 256 * M) {
            // (4-byte rows of this size do not fit a wave's registers twice)
            if constexpr (W == 8) run(rms_backward_kernel<T, A, PAST, 1, 8, 4>, 8, 8, 4, kCUs);
            else run(rms_backward_kernel<T, A, PAST, 4, 4, 2>, 4, 1, 2, 2 * kCUs);
        }
        else if (lanes <= 512 * M) run(rms_backward_kernel<T, A, PAST, 4, 4, 2 * M>, 4, 1, 2 * M, 2 * kCUs);
        else if (lanes <= 1024 * M) run(rms_backward_kernel<T, A, PAST, 4, 4, 4 * M>, 4, 1, 4 * M, 2 * kCUs);
        else if (lanes <= 2048 * M) run(rms_backward_kernel<T, A, PAST, 8, 8, 4 * M>, 8, 1, 4 * M, kCUs);
        else {
            in_launches(a.rows, 1024, [&](int64_t first, int64_t count) {
                rms_backward_long_kernel<T, A, PAST><<<dim3((unsigned)count), 1024, 0, s>>>(from_row<T>(a, first));
            });
            parts = a.rows < kLongRows ? a.rows : kLongRows;
            const int64_t slab = ceil_div(a.rows, parts);
            parts = ceil_div(a.rows, slab);
            if (a.partial != nullptr)
                rms_columns_kernel<T><<<dim3((unsigned)ceil_div(lanes, 256), (unsigned)parts), 256, 0, s>>>(a, slab);
        }
    }
    if (a.partial != nullptr)
        rms_fold_kernel<A><<<dim3((unsigned)ceil_div(a.width, 64)), 1024, 0, s>>>(a.partial, parts, a.width, static_cast<A*>(a.dweight));
    return hipGetLastError();
}

template <typename T, typename A>
hipError_t forward(const RmsForward& a, hipStream_t s)
{
    const bool past = a.rows * a.width * (int64_t)sizeof(T) > kCaches;
    if (a.codes != nullptr) return past ? forward_rows<T, A, true, true>(a, s) : forward_rows<T, A, false, true>(a, s);
    return past ? forward_rows<T, A, true, false>(a, s) : forward_rows<T, A, false, false>(a, s);
}

template <typename T, typename A>
hipError_t backward(const RmsBackward& a, hipStream_t s)
{
    return a.rows * a.width * (int64_t)sizeof(T) > kCaches ? backward_rows<T, A, true>(a, s) : backward_rows<T, A, false>(a, s);
}

}  // namespace

int64_t rms_partial_rows(int64_t rows) { return rows < 2 * kCUs ? (rows < 1 ? 1 : rows) : 2 * kCUs; }

hipError_t rms_forward(const RmsForward& a, int type, int affine, hipStream_t s)
{
    switch (type * 4 + affine) {
    case 1 * 4 + 1: return forward<_Float16, _Float16>(a, s);
    case 1 * 4 + 3: return forward<_Float16, float>(a, s);
    case 2 * 4 + 2: return forward<__bf16, __bf16>(a, s);
    case 2 * 4 + 3: return forward<__bf16, float>(a, s);
    default: return forward<float, float>(a, s);
    }
}

hipError_t rms_backward(const RmsBackward& a, int type, int affine, hipStream_t s)
{
    switch (type * 4 + affine) {
    case 1 * 4 + 1: return backward<_Float16, _Float16>(a, s);
    case 1 * 4 + 3: return backward<_Float16, float>(a, s);
    case 2 * 4 + 2: return backward<__bf16, __bf16>(a, s);
    case 2 * 4 + 3: return backward<__bf16, float>(a, s);
    default: return backward<float, float>(a, s);
    }
}

}  // namespace zo
