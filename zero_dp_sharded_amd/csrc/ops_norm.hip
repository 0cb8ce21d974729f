// Layer norm over the last dimension, forward and backward:
//     mean = sum x / D ;  rstd = 1 / sqrt(sum (x - mean)^2 / D + eps)
//     xhat = (x - mean) rstd ;  y = xhat w + b
//     g = dy w ;  dx = rstd (g - mean(g) - xhat mean(g xhat))
//     dw = sum_rows dy xhat ;  db = sum_rows dy
// All of it in fp32, rounded once at the end.
//
// Both directions are bound by memory: 2 (forward) or 3 (backward) rows of D
// elements, each moved once.  A row stays in registers between its sums and its
// results; it belongs to one wave where it fits (no barrier at all), else to 4, 8
// or 16 waves that join their sums through LDS; a row of more than 16384 elements is read
// again from cache instead.  The backward pass reads a row while it works on the one
// before.
//
// Measured: forward 8192 x 5120 fp16 27.5 us, 6.1 TB/s.  Backward 16384 x 1600 bf16 39 us
// and 4 for the fold, 4.0 TB/s: a wave holds its row twice and its sums, so that two
// stand in a SIMD, and the row's sums, two chains of shuffles, are waited for (its vector
// instructions alone would take 18 us; 4 waves a row instead of one 51).  One row of
// 1600: 4 us, 8.5 with the call.
//
// The weight's and bias's gradients are sums over all rows: each workgroup keeps
// the sums of the rows it walks in registers, adds its waves' in LDS, and writes
// one row of partial sums; a second kernel adds those in their order.  No atomics,
// so the same input gives the same bits.

#include "ops_common.h"
#include "ops_internal.h"

namespace zo {
namespace {

// PAST: results of more bytes than the L2s hold (4 MiB for each of 8 dies) are written past
// them, so that what is still to be read stays there: 8192 rows of 5120 fp16 forward
// 33.0 -> 27.8 us, 16384 rows of 1600 bf16 21.8 -> 20.9.  That is the norm by itself.  A reader
// right behind it would have found part of 50 to 200 MB in the last cache: with an elementwise
// one both take 63.0 and 39.4 us against 59.7 and 38.7 through the caches, with a matrix product
// the same within 3% either way.  Smaller results stay for their reader.
constexpr int64_t kCaches = 32 << 20;

// Sum of a and b over the NW waves of a row, the same in each.
template <int NW>
__device__ __forceinline__ void row_sum(float& a, float& b, float2* sh)
{
    a = wave_sum(a);
    b = wave_sum(b);
    if constexpr (NW > 1) {
        const int wave = threadIdx.x >> 6;
        __syncthreads();                       // the last sums have been read
        if ((threadIdx.x & 63) == 0) sh[wave] = make_float2(a, b);
        __syncthreads();
        a = b = 0.0f;
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            a += sh[k].x;
            b += sh[k].y;
        }
    }
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

template <bool PAST = false, typename T, int W>
__device__ __forceinline__ void store_part(T* row, int64_t c, int64_t width, const float (&x)[W])
{
    if (c + W <= width) {
        vec_t<T, W> v;
#pragma unroll
        for (int k = 0; k < W; ++k) v[k] = static_cast<T>(x[k]);
        store_vec<T, W, PAST>(row + c, v);
    } else {
#pragma unroll
        for (int k = 0; k < W; ++k)
            if (c + k < width) row[c + k] = static_cast<T>(x[k]);
    }
}

// ------------------------------------------------------------------ forward

// NW waves a row, K vectors a lane; with NW == 1 a workgroup has 4 rows.
template <typename T, typename A, bool PAST, int NW, int K>
__global__ __launch_bounds__(NW == 1 ? 256 : NW * 64) void forward_kernel(NormForward a)
{
    constexpr int W = Vec<T>::W;
    __shared__ float2 sh[NW];
    const int lane = NW == 1 ? threadIdx.x & 63 : threadIdx.x;
    const int64_t row = NW == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
    if (row >= a.rows) return;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    float v[K][W];
    float s = 0.0f, unused = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) load_part<T, W>(x, (int64_t)(k * NW * 64 + lane) * W, a.width, v[k]);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < W; ++e) s += v[k][e];
    row_sum<NW>(s, unused, sh);
    const float mean = s / (float)a.width;
    float q = 0.0f;
    unused = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t c = (int64_t)(k * NW * 64 + lane) * W;
#pragma unroll
        for (int e = 0; e < W; ++e) {
            v[k][e] = c + e < a.width ? v[k][e] - mean : 0.0f;
            q = fmaf(v[k][e], v[k][e], q);
        }
    }
    row_sum<NW>(q, unused, sh);
    const float rstd = 1.0f / sqrtf(q / (float)a.width + a.eps);
    if (lane == 0) {
        if (a.mean != nullptr) a.mean[row] = mean;
        if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(a.y) + row * a.y_stride;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t c = (int64_t)(k * NW * 64 + lane) * W;
        if (c >= a.width) continue;
        float w[W], b[W];
#pragma unroll
        for (int e = 0; e < W; ++e) {
            w[e] = 1.0f;
            b[e] = 0.0f;
        }
        if (a.weight != nullptr) load_part<A, W>(static_cast<const A*>(a.weight), c, a.width, w);
        if (a.bias != nullptr) load_part<A, W>(static_cast<const A*>(a.bias), c, a.width, b);
#pragma unroll
        for (int e = 0; e < W; ++e) w[e] = fmaf(v[k][e] * rstd, w[e], b[e]);
        store_part<PAST>(y, c, a.width, w);
    }
}

// Rows too long for registers: 16 waves walk the row three times.
template <typename T, typename A, bool PAST>
__global__ __launch_bounds__(1024) void forward_long_kernel(NormForward a)
{
    constexpr int W = Vec<T>::W;
    __shared__ float2 sh[16];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    T* y = static_cast<T*>(a.y) + row * a.y_stride;
    const int64_t c0 = (int64_t)threadIdx.x * W, step = 1024 * W;
    float s = 0.0f, q = 0.0f, unused = 0.0f;
    for (int64_t c = c0; c < a.width; c += step) {
        float v[W];
        load_part<T, W>(x, c, a.width, v);
#pragma unroll
        for (int e = 0; e < W; ++e) s += v[e];
    }
    row_sum<16>(s, unused, sh);
    const float mean = s / (float)a.width;
    for (int64_t c = c0; c < a.width; c += step) {
        float v[W];
        load_part<T, W>(x, c, a.width, v);
#pragma unroll
        for (int e = 0; e < W; ++e)
            if (c + e < a.width) q = fmaf(v[e] - mean, v[e] - mean, q);
    }
    unused = 0.0f;
    row_sum<16>(q, unused, sh);
    const float rstd = 1.0f / sqrtf(q / (float)a.width + a.eps);
    if (threadIdx.x == 0) {
        if (a.mean != nullptr) a.mean[row] = mean;
        if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    for (int64_t c = c0; c < a.width; c += step) {
        float v[W], w[W], b[W];
        load_part<T, W>(x, c, a.width, v);
#pragma unroll
        for (int e = 0; e < W; ++e) {
            w[e] = 1.0f;
            b[e] = 0.0f;
        }
        if (a.weight != nullptr) load_part<A, W>(static_cast<const A*>(a.weight), c, a.width, w);
        if (a.bias != nullptr) load_part<A, W>(static_cast<const A*>(a.bias), c, a.width, b);
#pragma unroll
        for (int e = 0; e < W; ++e) w[e] = fmaf((v[e] - mean) * rstd, w[e], b[e]);
        store_part<PAST>(y, c, a.width, w);
    }
}

// ------------------------------------------------------------------ backward

// A workgroup of WAVES waves, NW to a row, walks rows blockIdx, blockIdx + grid,
// ... (in groups of WAVES / NW) and keeps its sums for dw and db.  Up to 4 waves a row,
// the next row is read meanwhile, and the weight is kept in LDS to have the registers
// for that; with 8, LDS does not reach: the weight is read row by row from cache.
template <typename T, typename A, bool PAST, int NW, int WAVES, int K>
__global__ __launch_bounds__(WAVES * 64) void backward_kernel(NormBackward a)
{
    constexpr int W = Vec<T>::W;
    constexpr int ROWS = WAVES / NW;
    static_assert(ROWS == 1 || NW == 1, "several rows a workgroup: a wave each");
    constexpr bool AHEAD = NW <= 4;
    __shared__ float2 sh[NW];
    // the weight, 4 elements a lane side by side (AHEAD); at the end, with ROWS > 1, the
    // sums of the waves, [2][K * W][64]
    extern __shared__ __attribute__((aligned(16))) float fold[];
    const int lane = NW == 1 ? threadIdx.x & 63 : threadIdx.x;
    const int wave = threadIdx.x >> 6;
    const float inv = 1.0f / (float)a.width;
    float dw[K][W], db[K][W];
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int e = 0; e < W; ++e) dw[k][e] = db[k][e] = 0.0f;
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
    vec_t<T, W> nx[K], ng[K];                  // the next row, as it lies in memory
    auto fetch = [&](int64_t r) {
        const T* xr = static_cast<const T*>(a.x) + r * a.x_stride;
        const T* dyr = static_cast<const T*>(a.dy) + r * a.dy_stride;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t c = (int64_t)(k * NW * 64 + lane) * W;
            nx[k] = load_raw<T, W>(xr, c, a.width);
            ng[k] = load_raw<T, W>(dyr, c, a.width);
        }
    };
    float nmean = 0.0f, nrstd = 0.0f;
    if (AHEAD && row < a.rows) {
        fetch(row);
        nmean = a.mean[row];
        nrstd = a.rstd[row];
    }
    // (rows of NW == 1 end wave by wave, the others' workgroups together: no barrier is
    // missed)
    for (; row < a.rows; row += stride) {
        if constexpr (!AHEAD) {
            fetch(row);
            nmean = a.mean[row];
            nrstd = a.rstd[row];
        }
        float x[K][W], g[K][W];
        const float mean = nmean, rstd = nrstd;
        float sg = 0.0f, sgx = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int e = 0; e < W; ++e) {
                x[k][e] = ((float)nx[k][e] - mean) * rstd;
                g[k][e] = (float)ng[k][e];
            }
            // past the width g is 0, but -mean * rstd may be infinite: both are 0 there
            const int left = (int)a.width - (k * NW * 64 + lane) * W;
            if (left < W) {
#pragma unroll
                for (int e = 0; e < W; ++e)
                    if (e >= left) x[k][e] = 0.0f;
            }
        }
        if (AHEAD && row + stride < a.rows) {
            fetch(row + stride);
            nmean = a.mean[row + stride];
            nrstd = a.rstd[row + stride];
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float w[W];
            weight(k, w);
#pragma unroll
            for (int e = 0; e < W; ++e) {
                dw[k][e] = fmaf(g[k][e], x[k][e], dw[k][e]);
                db[k][e] += g[k][e];
                g[k][e] *= w[e];
                sg += g[k][e];
                sgx = fmaf(g[k][e], x[k][e], sgx);
            }
        }
        row_sum<NW>(sg, sgx, sh);
        sg *= inv;
        sgx *= inv;
        T* dxr = static_cast<T*>(a.dx) + row * a.dx_stride;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t c = (int64_t)(k * NW * 64 + lane) * W;
            if (c >= a.width) continue;
#pragma unroll
            for (int e = 0; e < W; ++e) g[k][e] = rstd * fmaf(-x[k][e], sgx, g[k][e] - sg);
            store_part<PAST>(dxr, c, a.width, g[k]);
        }
    }
    if (a.partial == nullptr) return;
    float* out = a.partial + (int64_t)blockIdx.x * 2 * a.width;
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
                        if (turn > 0) {
                            dw[k][e] += fold[at];
                            db[k][e] += fold[K * W * 64 + at];
                        }
                        fold[at] = dw[k][e];
                        fold[K * W * 64 + at] = db[k][e];
                    }
            }
            __syncthreads();
        }
        if (wave != ROWS - 1) return;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t c = (int64_t)(k * NW * 64 + lane) * W;
        if (c >= a.width) continue;
        store_part(out, c, a.width, dw[k]);
        store_part(out + a.width, c, a.width, db[k]);
    }
}

// Rows too long for registers: dx row by row, and the sums for dw and db over
// slabs of rows, a lane W columns.
template <typename T, typename A, bool PAST>
__global__ __launch_bounds__(1024) void backward_long_kernel(NormBackward a)
{
    constexpr int W = Vec<T>::W;
    __shared__ float2 sh[16];
    const int64_t row = blockIdx.x;
    const T* xr = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* dyr = static_cast<const T*>(a.dy) + row * a.dy_stride;
    T* dxr = static_cast<T*>(a.dx) + row * a.dx_stride;
    const float mean = a.mean[row], rstd = a.rstd[row], inv = 1.0f / (float)a.width;
    const int64_t c0 = (int64_t)threadIdx.x * W, step = 1024 * W;
    float sg = 0.0f, sgx = 0.0f;
    for (int turn = 0; turn < 2; ++turn) {
        for (int64_t c = c0; c < a.width; c += step) {
            float x[W], g[W], w[W];
            load_part<T, W>(xr, c, a.width, x);
            load_part<T, W>(dyr, c, a.width, g);
            if (a.weight != nullptr) {
                load_part<A, W>(static_cast<const A*>(a.weight), c, a.width, w);
#pragma unroll
                for (int e = 0; e < W; ++e) g[e] *= w[e];
            }
#pragma unroll
            for (int e = 0; e < W; ++e) {
                // (past the width: 0, as in backward_kernel)
                const float xhat = c + e < a.width ? (x[e] - mean) * rstd : 0.0f;
                if (turn == 0) {
                    sg += g[e];
                    sgx = fmaf(g[e], xhat, sgx);
                } else {
                    g[e] = rstd * fmaf(-xhat, sgx, g[e] - sg);
                }
            }
            if (turn == 1) store_part<PAST>(dxr, c, a.width, g);
        }
        if (turn == 0) {
            row_sum<16>(sg, sgx, sh);
            sg *= inv;
            sgx *= inv;
        }
    }
}

template <typename T>
__global__ __launch_bounds__(256) void columns_long_kernel(NormBackward a, int64_t slab)
{
    constexpr int W = Vec<T>::W;
    const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * W;
    if (c >= a.width) return;
    float dw[W], db[W];
#pragma unroll
    for (int e = 0; e < W; ++e) dw[e] = db[e] = 0.0f;
    const int64_t r0 = blockIdx.y * slab, r1 = r0 + slab < a.rows ? r0 + slab : a.rows;
    for (int64_t row = r0; row < r1; ++row) {
        float x[W], g[W];
        load_part<T, W>(static_cast<const T*>(a.x) + row * a.x_stride, c, a.width, x);
        load_part<T, W>(static_cast<const T*>(a.dy) + row * a.dy_stride, c, a.width, g);
        const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
        for (int e = 0; e < W; ++e) {
            dw[e] = fmaf(g[e], (x[e] - mean) * rstd, dw[e]);
            db[e] += g[e];
        }
    }
    float* out = a.partial + (int64_t)blockIdx.y * 2 * a.width;
    store_part(out, c, a.width, dw);
    store_part(out + a.width, c, a.width, db);
}

// dw and db: the partial rows, added in 16 runs by 16 waves, the runs in order.
template <typename A>
__global__ __launch_bounds__(1024) void fold_kernel(const float* partial, int64_t parts, int64_t width,
                                                    A* dweight, A* dbias)
{
    __shared__ float sh[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;       // of 2 * width columns
    const int64_t p0 = parts * wave / 16, p1 = parts * (wave + 1) / 16;
    float s = 0.0f;
    if (c < 2 * width) {
#pragma unroll 16
        for (int64_t p = p0; p < p1; ++p) s += partial[p * 2 * width + c];
    }
    sh[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || c >= 2 * width) return;
#pragma unroll
    for (int k = 1; k < 16; ++k) s += sh[k][lane];
    if (c < width) {
        if (dweight != nullptr) dweight[c] = static_cast<A>(s);
    } else if (dbias != nullptr) {
        dbias[c - width] = static_cast<A>(s);
    }
}

// ------------------------------------------------------------------ launches

constexpr int64_t kLongRows = 64;      // workgroups over the rows of very long ones

// The arrays from row `first` on.
template <typename T>
NormForward from_row(NormForward a, int64_t first)
{
    a.x = static_cast<const T*>(a.x) + first * a.x_stride;
    a.y = static_cast<T*>(a.y) + first * a.y_stride;
    if (a.mean != nullptr) a.mean += first;
    if (a.rstd != nullptr) a.rstd += first;
    a.rows -= first;
    return a;
}

template <typename T>
NormBackward from_row(NormBackward a, int64_t first)
{
    a.dy = static_cast<const T*>(a.dy) + first * a.dy_stride;
    a.x = static_cast<const T*>(a.x) + first * a.x_stride;
    a.dx = static_cast<T*>(a.dx) + first * a.dx_stride;
    a.mean += first;
    a.rstd += first;
    a.rows -= first;
    return a;
}

template <typename T, typename A, bool PAST>
hipError_t forward_rows(const NormForward& a, hipStream_t s)
{
    constexpr int W = Vec<T>::W;
    // lanes that a row keeps busy with one vector each; a wave keeps up to 64 elements
    // of a lane in registers
    const int64_t lanes = ceil_div(a.width, W);
    auto run = [&](auto kernel, int threads, int rows) {
        in_launches(ceil_div(a.rows, rows), threads, [&](int64_t first, int64_t count) {
            kernel<<<dim3((unsigned)count), threads, 0, s>>>(from_row<T>(a, first * rows));
        });
    };
    constexpr int M = 8 / W;               // vectors of a lane in 8 elements
    if (lanes <= 64 * M) run(forward_kernel<T, A, PAST, 1, M>, 256, 4);
    else if (lanes <= 128 * M) run(forward_kernel<T, A, PAST, 1, 2 * M>, 256, 4);
    else if (lanes <= 256 * M) run(forward_kernel<T, A, PAST, 1, 4 * M>, 256, 4);
    else if (lanes <= 384 * M) run(forward_kernel<T, A, PAST, 1, 6 * M>, 256, 4);
    else if (lanes <= 512 * M) run(forward_kernel<T, A, PAST, 4, 2 * M>, 256, 1);
    else if (lanes <= 768 * M) run(forward_kernel<T, A, PAST, 4, 3 * M>, 256, 1);
    else if (lanes <= 1024 * M) run(forward_kernel<T, A, PAST, 4, 4 * M>, 256, 1);
    else if (lanes <= 2048 * M) run(forward_kernel<T, A, PAST, 16, 2 * M>, 1024, 1);
    else run(forward_long_kernel<T, A, PAST>, 1024, 1);
    return hipGetLastError();
}

template <typename T, typename A, bool PAST>
hipError_t backward_rows(const NormBackward& a, hipStream_t s)
{
    constexpr int W = Vec<T>::W;
    const int64_t lanes = ceil_div(a.width, W);
    int64_t parts = 0;
    if (a.rows > 0) {
        // `most` workgroups walk the rows: what their registers let stand in the CUs
        auto run = [&](auto kernel, int waves, int rows, int k, int64_t most) {
            parts = ceil_div(a.rows, rows);
            if (parts > most) parts = most;
            const size_t lds = rows > 1 ? (size_t)2 * k * W * 64 * sizeof(float) : waves == 4 ? (size_t)k * W * 256 * sizeof(float) : 0;
            kernel<<<dim3((unsigned)parts), waves * 64, lds, s>>>(a);
        };
        constexpr int M = 8 / W;           // vectors of a lane in 8 elements
        if (lanes <= 64 * M) run(backward_kernel<T, A, PAST, 1, 16, M>, 16, 16, M, kCUs);
        else if (lanes <= 128 * M) run(backward_kernel<T, A, PAST, 1, 8, 2 * M>, 8, 8, 2 * M, kCUs);
        else if (lanes <= 256 * M) {
            // (4-byte rows of this size do not fit a wave's registers twice)
            if constexpr (W == 8) run(backward_kernel<T, A, PAST, 1, 8, 4>, 8, 8, 4, kCUs);
            else run(backward_kernel<T, A, PAST, 4, 4, 2>, 4, 1, 2, 2 * kCUs);
        }
        else if (lanes <= 512 * M) run(backward_kernel<T, A, PAST, 4, 4, 2 * M>, 4, 1, 2 * M, 2 * kCUs);
        else if (lanes <= 1024 * M) run(backward_kernel<T, A, PAST, 4, 4, 4 * M>, 4, 1, 4 * M, 2 * kCUs);
        else if (lanes <= 2048 * M) run(backward_kernel<T, A, PAST, 8, 8, 4 * M>, 8, 1, 4 * M, kCUs);
        else {
            in_launches(a.rows, 1024, [&](int64_t first, int64_t count) {
                backward_long_kernel<T, A, PAST><<<dim3((unsigned)count), 1024, 0, s>>>(from_row<T>(a, first));
            });
            parts = a.rows < kLongRows ? a.rows : kLongRows;
            const int64_t slab = ceil_div(a.rows, parts);
            parts = ceil_div(a.rows, slab);
            if (a.partial != nullptr)
                columns_long_kernel<T><<<dim3((unsigned)ceil_div(lanes, 256), (unsigned)parts), 256, 0, s>>>(a, slab);
        }
    }
    if (a.partial != nullptr)
        fold_kernel<A><<<dim3((unsigned)ceil_div(2 * a.width, 64)), 1024, 0, s>>>(
            a.partial, parts, a.width, static_cast<A*>(a.dweight), static_cast<A*>(a.dbias));
    return hipGetLastError();
}

template <typename T, typename A>
hipError_t forward(const NormForward& a, hipStream_t s)
{
    return a.rows * a.width * (int64_t)sizeof(T) > kCaches ? forward_rows<T, A, true>(a, s) : forward_rows<T, A, false>(a, s);
}

template <typename T, typename A>
hipError_t backward(const NormBackward& a, hipStream_t s)
{
    return a.rows * a.width * (int64_t)sizeof(T) > kCaches ? backward_rows<T, A, true>(a, s) : backward_rows<T, A, false>(a, s);
}

}  // namespace

int64_t norm_partial_rows(int64_t rows, int64_t) { return rows < 2 * kCUs ? (rows < 1 ? 1 : rows) : 2 * kCUs; }

hipError_t norm_forward(const NormForward& a, int type, int affine, hipStream_t s)
{
    switch (type * 4 + affine) {
    case 1 * 4 + 1: return forward<_Float16, _Float16>(a, s);
    case 1 * 4 + 3: return forward<_Float16, float>(a, s);
    case 2 * 4 + 2: return forward<__bf16, __bf16>(a, s);
    case 2 * 4 + 3: return forward<__bf16, float>(a, s);
    default: return forward<float, float>(a, s);
    }
}

hipError_t norm_backward(const NormBackward& a, int type, int affine, hipStream_t s)
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
