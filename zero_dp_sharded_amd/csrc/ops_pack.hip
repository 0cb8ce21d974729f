// Packing to 8 bits with a power of two for every 128 elements (ops_scaled.h), along
// the rows of an array, along the rows of its transpose, or both from one reading; and back.
//
// Bound by memory.  A workgroup takes 128 x 128 elements; a lane has 8 rows of 8
// columns, so that the largest of 128 elements along a row is one exchange among 16 lanes,
// along a column one in LDS, and 8 codes side by side are there in either
// direction.  The transposed codes go through LDS, to be written in runs of 128 bytes.
// 8192 x 6400 bf16 both ways 36 us call after call (5.8 TB/s, in part from the last cache) and 48 with
// its array in memory; 4801 x 1601 fp32 in squares 7.7 and 9.7.  A weight of 20480 x 5120 in squares, both
// ways, 85 us from bf16 (4.9 TB/s) and 122 from fp32; 6400 x 1600 11 and 17.  Back, 16 of a row to a lane: 8192 x 6400 to
// bf16 25 to 29 us, 6.3 TB/s.

#include <type_traits>

#include "ops_common.h"
#include "ops_internal.h"
#include "ops_scaled.h"

namespace zo {
namespace {

constexpr int kTile = kScaleBlock;

// Where 8 codes of a column lie in LDS, rows 8 band to + 7: a lane's 8 columns and its neighbours' are written
// at once, and the exclusive or takes them to different banks.
__device__ __forceinline__ int turned_at(int column, int band) { return column * kTile + ((band ^ (column >> 3)) & 15) * 8; }

// 8 x 8 elements of a lane, two side by side in a word where they are of 2 bytes, with what the largest and
// the codes are taken from: of a row the elements in turn, of a column the rows in turn.
template <typename T>
struct Block {
    typedef vec_t<T, 2> two;
    typedef vec_t<uint16_t, 2> word;
    static constexpr uint32_t kInfinite = std::is_same<T, _Float16>::value ? 0x7c00u : 0x7f80u;
    two v[8][4];

    __device__ __forceinline__ void load(const T* x, int64_t stride)
    {
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const vec_t<T, 8> r = load_vec<T, 8>(x + p * stride);
            __builtin_memcpy(v[p], &r, 16);
        }
    }
    __device__ __forceinline__ void set(int p, int k, T x) { v[p][k / 2][k % 2] = x; }
    __device__ __forceinline__ float at(int p, int k) const { return (float)v[p][k / 2][k % 2]; }
    static __device__ __forceinline__ word most(word a, word b) { return __builtin_elementwise_max(a, b); }
    __device__ __forceinline__ word size(int p, int w) const { return __builtin_bit_cast(word, __builtin_bit_cast(uint32_t, v[p][w]) & 0x7fff7fffu); }
    static __device__ __forceinline__ uint32_t as_float(uint32_t half)
    {
        if constexpr (std::is_same<T, _Float16>::value) return bits((float)__builtin_bit_cast(_Float16, (uint16_t)half));
        else return half << 16;
    }
    // The largest of the rows and of the columns, as bits of fp32; false: something is not finite.
    __device__ __forceinline__ bool largest(uint32_t (&along)[8], uint32_t (&down)[8]) const
    {
        word d[4], all = {0, 0};
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            word a = size(p, 0);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const word x = size(p, w);
                a = most(a, x);
                d[w] = p ? most(d[w], x) : x;
            }
            all = most(all, a);
            along[p] = as_float(larger(a[0], a[1]));
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            down[2 * w] = as_float(d[w][0]);
            down[2 * w + 1] = as_float(d[w][1]);
        }
        return larger(all[0], all[1]) < kInfinite;
    }
    __device__ __forceinline__ uint2 row_codes(int p, float scale) const
    {
        short2_t lo = {0, 0}, hi = {0, 0};
        lo = two_codes<false>(lo, v[p][0], scale);
        lo = two_codes<true>(lo, v[p][1], scale);
        hi = two_codes<false>(hi, v[p][2], scale);
        hi = two_codes<true>(hi, v[p][3], scale);
        return make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
    }
    __device__ __forceinline__ two pair(int p, int k) const { return two{v[p][k / 2][k % 2], v[p + 1][k / 2][k % 2]}; }
    __device__ __forceinline__ uint2 column_codes(int k, float scale) const
    {
        short2_t lo = {0, 0}, hi = {0, 0};
        lo = two_codes<false>(lo, pair(0, k), scale);
        lo = two_codes<true>(lo, pair(2, k), scale);
        hi = two_codes<false>(hi, pair(4, k), scale);
        hi = two_codes<true>(hi, pair(6, k), scale);
        return make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
    }
};

template <>
struct Block<float> {
    float v[8][8];

    __device__ __forceinline__ void load(const float* x, int64_t stride)
    {
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const vec_t<float, 4> lo = load_vec<float, 4>(x + p * stride), hi = load_vec<float, 4>(x + p * stride + 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[p][k] = lo[k];
                v[p][4 + k] = hi[k];
            }
        }
    }
    __device__ __forceinline__ void set(int p, int k, float x) { v[p][k] = x; }
    __device__ __forceinline__ float at(int p, int k) const { return v[p][k]; }
    __device__ __forceinline__ bool largest(uint32_t (&along)[8], uint32_t (&down)[8]) const
    {
        uint32_t all = 0;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            along[p] = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t u = bits(v[p][k]) & 0x7fffffffu;
                along[p] = larger(along[p], u);
                down[k] = p ? larger(down[k], u) : u;
            }
            all = larger(all, along[p]);
        }
        return all < kNotFinite;
    }
    __device__ __forceinline__ uint2 row_codes(int p, float scale) const
    {
        short2_t lo = {0, 0}, hi = {0, 0};
        lo = two_codes<false>(lo, v[p][0], v[p][1], scale);
        lo = two_codes<true>(lo, v[p][2], v[p][3], scale);
        hi = two_codes<false>(hi, v[p][4], v[p][5], scale);
        hi = two_codes<true>(hi, v[p][6], v[p][7], scale);
        return make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
    }
    __device__ __forceinline__ uint2 column_codes(int k, float scale) const
    {
        short2_t lo = {0, 0}, hi = {0, 0};
        lo = two_codes<false>(lo, v[0][k], v[1][k], scale);
        lo = two_codes<true>(lo, v[2][k], v[3][k], scale);
        hi = two_codes<false>(hi, v[4][k], v[5][k], scale);
        hi = two_codes<true>(hi, v[6][k], v[7][k], scale);
        return make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
    }
};

// 8 codes with their E.
__device__ __forceinline__ uint2 topped(uint2 codes, uint32_t E)
{
    if (E == kTopScale) codes = make_uint2(below_top(codes.x), below_top(codes.y));
    return codes;
}

// 8 codes to p, or as many of them as `left` says.
__device__ __forceinline__ void put8(uint8_t* p, uint2 v, int64_t left)
{
    if (left >= 8) {
        __builtin_memcpy(p, &v, 8);
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < left) p[k] = (uint8_t)((k < 4 ? v.x : v.y) >> (8 * (k % 4)));
}

template <typename T, bool SQUARE>
__global__ __launch_bounds__(256) void scaled_pack_kernel(ScaledPack a, int64_t first)
{
    __shared__ uint32_t big[4][kTile];
    __shared__ __attribute__((aligned(16))) uint8_t turned[kTile * kTile], scales[kTile];
    // (the dies, which workgroups go round, have runs of tiles: what tiles side by side share of a line, of the
    // exponents above all, is in one L2.  4801 x 1601 fp32 squares 10.1 -> 7.8 us)
    const uint32_t die = blockIdx.x % 8, per = gridDim.x / 8, rest = gridDim.x % 8;
    const int64_t id = first + die * per + (die < rest ? die : rest) + blockIdx.x / 8;
    const int64_t r0 = id / a.tiles * kTile, c0 = id % a.tiles * kTile;
    const int lane = threadIdx.x & 15, band = threadIdx.x >> 4;       // columns 8 lane .., rows 8 band ..
    const int64_t c = c0 + lane * 8, r = r0 + band * 8;
    const T* x = static_cast<const T*>(a.x) + r * a.x_stride + c;
    Block<T> b;
    if (c + 8 <= a.width && r + 8 <= a.rows) {
        b.load(x, a.x_stride);
    } else {
#pragma unroll
        for (int p = 0; p < 8; ++p)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                b.set(p, k, r + p < a.rows && c + k < a.width ? x[p * a.x_stride + k] : static_cast<T>(0.0f));
    }
    uint32_t along[8], down[8];            // the largest of the lane's rows, and of its columns
    if (!b.largest(along, down)) {
#pragma unroll
        for (int k = 0; k < 8; ++k) along[k] = down[k] = 0;
#pragma unroll
        for (int p = 0; p < 8; ++p)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                along[p] = with_size(along[p], b.at(p, k));
                down[k] = with_size(down[k], b.at(p, k));
            }
    }
    uint32_t E = 0;
    if constexpr (SQUARE) {
        uint32_t all = 0;
#pragma unroll
        for (int p = 0; p < 8; ++p) all = larger(all, along[p]);
        all = lanes_max<64>(all);
        if ((threadIdx.x & 63) == 0) big[0][threadIdx.x >> 6] = all;
        __syncthreads();
        E = scale_of(larger(larger(big[0][0], big[0][1]), larger(big[0][2], big[0][3])));
        if (threadIdx.x == 0) {
            if (a.codes != nullptr) a.exps[r0 / kTile * a.exps_stride + c0 / kTile] = (uint8_t)E;
            if (a.codes_t != nullptr) a.exps_t[c0 / kTile * a.exps_t_stride + r0 / kTile] = (uint8_t)E;
        }
    }
    if (a.codes != nullptr) {
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            uint32_t e = E;
            if constexpr (!SQUARE) e = scale_of(lanes_max<16>(along[p]));
            if (r + p >= a.rows) continue;
            if (!SQUARE && lane == 0) a.exps[(r + p) * a.exps_stride + c0 / kTile] = (uint8_t)e;
            if (c >= a.width) continue;
            const uint2 out = topped(b.row_codes(p, from_bits(e << 23)), e);
            put8(a.codes + (r + p) * a.codes_stride + c, out, a.width - c);
        }
    }
    if (a.codes_t == nullptr) return;
    uint2 es = make_uint2(0, 0);           // E of the lane's 8 columns
    if constexpr (!SQUARE) {
        // over a wave's 4 bands, then over the waves
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            auto r = __builtin_amdgcn_permlane16_swap(down[k], down[k], false, false);
            down[k] = larger(r[0], r[1]);
            r = __builtin_amdgcn_permlane32_swap(down[k], down[k], false, false);
            down[k] = larger(r[0], r[1]);
        }
        if ((threadIdx.x & 48) == 0) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                *reinterpret_cast<uint4*>(&big[threadIdx.x >> 6][lane * 8 + q * 4]) = make_uint4(down[4 * q], down[4 * q + 1], down[4 * q + 2], down[4 * q + 3]);
        }
        __syncthreads();
        if (threadIdx.x < kTile) {
            const int t = threadIdx.x;
            const uint32_t e = scale_of(larger(larger(big[0][t], big[1][t]), larger(big[2][t], big[3][t])));
            scales[t] = (uint8_t)e;
            if (c0 + t < a.width) a.exps_t[(c0 + t) * a.exps_t_stride + r0 / kTile] = (uint8_t)e;
        }
        __syncthreads();
        es = *reinterpret_cast<const uint2*>(scales + lane * 8);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t e = SQUARE ? E : ((k < 4 ? es.x : es.y) >> (8 * (k % 4))) & 0xff;
        *reinterpret_cast<uint2*>(turned + turned_at(lane * 8 + k, band)) = topped(b.column_codes(k, from_bits(e << 23)), e);
    }
    __syncthreads();
    // 8 lanes a column, 16 codes each
    const int64_t at = r0 + (threadIdx.x & 7) * 16;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int column = q * 32 + (threadIdx.x >> 3);
        if (c0 + column >= a.width || at >= a.rows) continue;
        // (a pair of 8 lies in one 16, its halves changed over where the column says so)
        const bool over = (column >> 3) & 1;
        const uint4 u = *reinterpret_cast<const uint4*>(turned + (turned_at(column, (threadIdx.x & 7) * 2) & ~15));
        const uint4 v = over ? make_uint4(u.z, u.w, u.x, u.y) : u;
        uint8_t* to = a.codes_t + (c0 + column) * a.codes_t_stride + at;
        if (at + 16 <= a.rows) {
            __builtin_memcpy(to, &v, 16);
        } else {
            put8(to, make_uint2(v.x, v.y), a.rows - at);
            put8(to + 8, make_uint2(v.z, v.w), a.rows - at - 8);
        }
    }
}

// What codes stand for, and zeros behind the width up to `fill`: a lane 16 of a row.
template <typename T>
__global__ __launch_bounds__(256) void scaled_unpack_kernel(ScaledUnpack a, int64_t first)
{
    const int64_t id = (first + blockIdx.x) * 256 + threadIdx.x;
    if (id >= a.rows * a.chunks) return;
    // (32 bits where they do: a 64-bit division is a hundred instructions)
    int64_t row, chunk;
    if (a.rows * a.chunks <= UINT32_MAX) {
        row = (uint32_t)id / (uint32_t)a.chunks;
        chunk = (uint32_t)id - (uint32_t)row * (uint32_t)a.chunks;
    } else {
        row = id / a.chunks;
        chunk = id - row * a.chunks;
    }
    const int64_t c = chunk * 16;
    const uint8_t* from = a.codes + row * a.codes_stride + c;
    T* to = static_cast<T*>(a.out) + row * a.out_stride + c;
    const float scale = c < a.width ? scale_value(a.exps[(a.square ? row / kTile : row) * a.exps_stride + c / kTile]) : 0.0f;
    uint32_t v[4] = {0, 0, 0, 0};
    const bool whole = c + 16 <= a.width;
    if (whole) {
        __builtin_memcpy(v, from, 16);
    } else {
#pragma unroll
        for (int k = 0; k < 16; ++k)
            if (c + k < a.width) v[k / 4] |= (uint32_t)from[k] << (8 * (k % 4));
    }
    float y[16];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        y[4 * q + 0] = __builtin_amdgcn_cvt_f32_fp8((int)v[q], 0) * scale;
        y[4 * q + 1] = __builtin_amdgcn_cvt_f32_fp8((int)v[q], 1) * scale;
        y[4 * q + 2] = __builtin_amdgcn_cvt_f32_fp8((int)v[q], 2) * scale;
        y[4 * q + 3] = __builtin_amdgcn_cvt_f32_fp8((int)v[q], 3) * scale;
    }
    constexpr int W = Vec<T>::W;
#pragma unroll
    for (int q = 0; q < 16 / W; ++q) {
        vec_t<T, W> o;
#pragma unroll
        for (int k = 0; k < W; ++k) o[k] = static_cast<T>(y[q * W + k]);
        if (whole) {
            store_vec<T, W>(to + q * W, o);
        } else {
#pragma unroll
            for (int k = 0; k < W; ++k)
                if (c + q * W + k < a.fill) to[q * W + k] = c + q * W + k < a.width ? o[k] : static_cast<T>(0.0f);
        }
    }
}

template <typename T>
hipError_t pack(ScaledPack a, hipStream_t s)
{
    a.tiles = ceil_div(a.width, kTile);
    in_launches(ceil_div(a.rows, kTile) * a.tiles, 256, [&](int64_t first, int64_t count) {
        if (a.square) scaled_pack_kernel<T, true><<<dim3((unsigned)count), 256, 0, s>>>(a, first);
        else scaled_pack_kernel<T, false><<<dim3((unsigned)count), 256, 0, s>>>(a, first);
    });
    return hipGetLastError();
}

template <typename T>
hipError_t unpack(ScaledUnpack a, hipStream_t s)
{
    if (a.fill < a.width) a.fill = a.width;
    a.chunks = ceil_div(a.fill, 16);
    in_launches(ceil_div(a.rows * a.chunks, 256), 256, [&](int64_t first, int64_t count) {
        scaled_unpack_kernel<T><<<dim3((unsigned)count), 256, 0, s>>>(a, first);
    });
    return hipGetLastError();
}

}  // namespace

hipError_t scaled_pack(const ScaledPack& a, int type, hipStream_t s)
{
    return type == 1 ? pack<_Float16>(a, s) : type == 2 ? pack<__bf16>(a, s) : pack<float>(a, s);
}

hipError_t scaled_unpack(const ScaledUnpack& a, int type, hipStream_t s)
{
    return type == 1 ? unpack<_Float16>(a, s) : type == 2 ? unpack<__bf16>(a, s) : unpack<float>(a, s);
}

}  // namespace zo
