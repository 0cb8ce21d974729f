// AdamW over the tensors of a model at once, with moments in 32 or in 8 bits.
//
// One launch updates every tensor: a table in device memory, made when the handle
// is, cuts the tensors into chunks of 4096 elements, a workgroup each.  A lane has 4
// elements side by side, so that every load and store of a wave is whole lines (512
// bytes of 2-byte gradients, 1 KiB of fp32), and a wave's 256 elements are a block
// of the 8-bit states.  Bound by memory: per element and step 28 bytes with fp32
// moments and 2-byte storage, 14 with 8-bit moments.
//
// The arithmetic is that of the shard's Adam (each operation rounded to fp32 in
// the order written, no fused multiply-adds), so that a tensor's update has the same bits
// as the same elements in a shard.
//
// 8-bit moments.  A block of 256 elements has one power of two 2^e (int8) and a
// small float an element; what is held is exact in fp32 and in bf16:
//     m: sign, 4 bits of exponent, 3 of mantissa;  v (never negative): 5 and 3
// with the largest code 1.875 * 2^e, the normal range down to 2^-14 (m) and 2^-30 (v)
// of 2^e, and gradual underflow below.  v has no square root taken before it is held:
// 5 bits of exponent cover gradients that differ by 2^16 within a block, and a v
// that falls to 0 beside an m that does not would make the update explode.
// Rounding is up or down at random, with the odds that keep the mean: v changes by
// a thousandth a step, less than half of a code, and rounding to the nearest would
// hold it where it is for ever.  The random bits are a hash of (seed, step, tensor,
// element), 16 for each moment, so a step can be repeated bit by bit.  The update
// itself uses the new moments before they are rounded.

#include "ops_common.h"
#include "ops_internal.h"

namespace zo {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr int kExpLeast = -100;       // the smallest power of two a block has
constexpr int kExpNaN = 127;          // a block that holds nothing finite
constexpr int kThreads = 256;
constexpr int kBlocksPerWave = (int)(kAdamwChunk / kThreads / 4);    // 4 elements a lane

template <int TYPE> struct Stored;
template <> struct Stored<1> { using T = _Float16; };
template <> struct Stored<2> { using T = __bf16; };
template <> struct Stored<3> { using T = float; };

__device__ __forceinline__ float pow2(int e) { return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23); }

// 32 bits of noise from 32 bits: shifts against multiplications by the fractions
// of the golden ratio and of the root of two.
__device__ __forceinline__ uint32_t mix(uint32_t x)
{
    x ^= x >> 16;
    x *= 0x9E3779B9u;
    x ^= x >> 15;
    x *= 0xB504F333u;
    return x ^ (x >> 16);
}

__device__ __forceinline__ uint32_t noise_key(uint64_t seed, int64_t t, int32_t tensor, int64_t element)
{
    uint32_t key = (uint32_t)seed;
    key = mix(mix(key) + (uint32_t)(seed >> 32));
    key = mix(mix(key) + (uint32_t)t);
    key = mix(mix(key) + (uint32_t)tensor);
    return mix(mix(key) + (uint32_t)(element >> 32));
}

// The largest of the wave's values, as bits of non-negative floats (so a NaN is
// the largest of all).
__device__ __forceinline__ uint32_t wave_max(uint32_t x)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        const uint32_t y = __shfl_xor(x, off, kWave);
        x = x > y ? x : y;
    }
    return x;
}

// The block's exponent for the largest magnitude's bits: the least e with
// largest <= 1.875 * 2^e.
__device__ __forceinline__ int block_exp(uint32_t bits)
{
    const int e = (int)(bits >> 23) - 127 + ((bits & 0x7fffffu) > 0x700000u ? 1 : 0);
    return e < kExpLeast ? kExpLeast : e > kExpNaN ? kExpNaN : e;
}

// Magnitude x >= 0 to a code: scaled so that the code's least normal exponent is
// fp32's, the code is the top bits of the float, and noise below them, added, rounds.
// LEAST: 14 (m) or 30 (v).
template <int LEAST>
__device__ __forceinline__ uint32_t encode(float x, float inv_block, uint32_t r16)
{
    const float z = (x * inv_block) * pow2(LEAST - 126);
    return (__builtin_bit_cast(uint32_t, z) + (r16 << 4) + 8) >> 20;
}

template <int LEAST>
__device__ __forceinline__ float decode(uint32_t code, float block)
{
    return (__builtin_bit_cast(float, code << 20) * pow2(126 - LEAST)) * block;
}

__device__ __forceinline__ float block_scale(int e)
{
    return e >= kExpNaN ? __builtin_nanf("") : pow2(e < kExpLeast ? kExpLeast : e);
}

// 4 elements from e on of an array of n, zeros past the end.
template <typename T>
__device__ __forceinline__ f4 load4(const T* p, int64_t e, int64_t n)
{
    f4 x;
    if (e + 4 <= n) {
        const vec_t<T, 4> v = load_vec<T, 4>(p + e);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = (float)v[k];
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = e + k < n ? (float)p[e + k] : 0.0f;
    }
    return x;
}

template <typename T>
__device__ __forceinline__ void store4(T* p, int64_t e, int64_t n, f4 x)
{
    if (e + 4 <= n) {
        vec_t<T, 4> v;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = static_cast<T>(x[k]);
        store_vec<T, 4>(p + e, v);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (e + k < n) p[e + k] = static_cast<T>(x[k]);
    }
}

__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int64_t e, int64_t n)
{
    if (e + 4 <= n) {
        const vec_t<uint8_t, 4> v = load_vec<uint8_t, 4>(p + e);
        return __builtin_bit_cast(uint32_t, v);
    }
    uint32_t x = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (e + k < n) x |= (uint32_t)p[e + k] << (8 * k);
    return x;
}

__device__ __forceinline__ void store_codes(uint8_t* p, int64_t e, int64_t n, uint32_t x)
{
    if (e + 4 <= n) {
        store_vec<uint8_t, 4>(p + e, __builtin_bit_cast(vec_t<uint8_t, 4>, x));
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (e + k < n) p[e + k] = (uint8_t)(x >> (8 * k));
    }
}

// ------------------------------------------------------------------ the check

template <int TYPE>
__device__ __forceinline__ void norm_chunk(const TensorEntry& t, int64_t begin, float inv_scale, double& ss,
                                           int& flag)
{
    using T = typename Stored<TYPE>::T;
    const T* g = static_cast<const T*>(t.grad);
    f4 x[kBlocksPerWave];
#pragma unroll
    for (int u = 0; u < kBlocksPerWave; ++u)
        x[u] = load4(g, begin + (u * kThreads + threadIdx.x) * 4, t.numel);
#pragma unroll
    for (int u = 0; u < kBlocksPerWave; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float y = x[u][k] * inv_scale;
            flag |= (__builtin_bit_cast(uint32_t, y) & 0x7f800000u) == 0x7f800000u;
            ss += (double)y * (double)y;
        }
}

// One fp64 partial sum of squares a chunk, NaN where an unscaled value is not finite.
__global__ __launch_bounds__(kThreads) void norm_kernel(AdamwLaunch a)
{
    __shared__ double sh[4];
    __shared__ int shf[4];
    const ChunkEntry c = a.chunks[blockIdx.x];
    const TensorEntry t = a.tensors[c.tensor];
    const float inv_scale = a.state->inv_scale;
    double ss = 0.0;
    int flag = 0;
    if (t.type == 1) norm_chunk<1>(t, c.begin, inv_scale, ss, flag);
    else if (t.type == 2) norm_chunk<2>(t, c.begin, inv_scale, ss, flag);
    else norm_chunk<3>(t, c.begin, inv_scale, ss, flag);
    ss = wave_sum(ss);
    flag = __any(flag);
    if ((threadIdx.x & 63) == 0) {
        sh[threadIdx.x >> 6] = ss;
        shf[threadIdx.x >> 6] = flag;
    }
    __syncthreads();
    if (threadIdx.x == 0)
        a.partial[blockIdx.x] = (shf[0] | shf[1] | shf[2] | shf[3]) ? __builtin_nan("")
                                                                    : (sh[0] + sh[1]) + (sh[2] + sh[3]);
}

// The partials in a fixed order, then the step's decision, as the shard's device-
// resident flow takes it; without a check every step is taken.
__global__ __launch_bounds__(1024) void decide_kernel(AdamwLaunch a, int checked)
{
    __shared__ double sh[16];
    double s = 0.0;
    if (checked) {
        for (int64_t i = threadIdx.x; i < a.nchunks; i += 1024) s += a.partial[i];
        s = wave_sum(s);
        if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = s;
        __syncthreads();
        s = 0.0;
        if (threadIdx.x == 0)
            for (int k = 0; k < 16; ++k) s += sh[k];
    }
    if (threadIdx.x != 0) return;
    AdamwState d = *a.state;
    const bool overflow = !__builtin_isfinite(s);
    d.sumsq = s;
    d.last_scale = d.scale;
    d.upd_inv_scale = d.inv_scale;
    d.skip = overflow;
    d.clip = 1.0f;
    if (!overflow) {
        d.t += 1;
        d.pw1 = d.pw1 * a.s.b1d;
        d.pw2 = d.pw2 * a.s.b2d;
        d.bc1 = a.s.bias_correction ? (float)(1.0 - d.pw1) : 1.0f;
        d.bc2 = a.s.bias_correction ? (float)(1.0 - d.pw2) : 1.0f;
        if (a.s.max_norm > 0.0) {
            const double c = a.s.max_norm / (sqrt(s) + 1e-6);
            if (c < 1.0) d.clip = (float)c;
        }
    }
    if (a.s.dynamic) {
        if (overflow) {
            const double sc = d.scale / 2.0;
            d.scale = sc < a.s.min_scale ? a.s.min_scale : sc;
            d.good = 0;
        } else if (++d.good == a.s.growth_interval) {
            d.scale = d.scale * 2.0;
            d.good = 0;
        }
    }
    d.inv_scale = (float)(1.0 / d.scale);
    *a.state = d;
}

// ------------------------------------------------------------------ the update

// Textbook Adam on one element, in the order of the public header.
__device__ __forceinline__ void adam(float g, float& p, float& m, float& v, const AdamwScalars& s,
                                     const AdamwState& d, float wd, float lr)
{
    g = g * d.upd_inv_scale;
    g = g * d.clip;
    if (s.l2) g = g + wd * p;
    m = s.b1 * m + s.omb1 * g;
    v = s.b2 * v + s.omb2 * (g * g);
    float u = (m / d.bc1) / (sqrtf(v / d.bc2) + s.eps);
    if (!s.l2) u = u + wd * p;
    p = p - lr * u;
}

template <int TYPE, int BITS>
__device__ __forceinline__ void update_chunk(const AdamwLaunch& a, const AdamwState& d, const TensorEntry& t,
                                             const ChunkEntry& c)
{
    using T = typename Stored<TYPE>::T;
    const int64_t n = t.numel;
    const int lane = threadIdx.x & 63;
    f4 g[kBlocksPerWave], p[kBlocksPerWave], m[kBlocksPerWave], v[kBlocksPerWave];
    uint32_t cm[kBlocksPerWave], cv[kBlocksPerWave];
    float bm[kBlocksPerWave], bv[kBlocksPerWave];
    const int64_t e0 = c.begin + threadIdx.x * 4;
#pragma unroll
    for (int u = 0; u < kBlocksPerWave; ++u) {
        const int64_t e = e0 + u * kThreads * 4;
        g[u] = load4(static_cast<const T*>(t.grad), e, n);
        p[u] = load4(t.master, e, n);
        if constexpr (BITS == 32) {
            m[u] = load4(static_cast<const float*>(t.m), e, n);
            v[u] = load4(static_cast<const float*>(t.v), e, n);
        } else {
            cm[u] = load_codes(static_cast<const uint8_t*>(t.m), e, n);
            cv[u] = load_codes(static_cast<const uint8_t*>(t.v), e, n);
            const int64_t b = e / kStateBlock, last = (n - 1) / kStateBlock;
            bm[u] = block_scale(t.m_exp[b < last ? b : last]);
            bv[u] = block_scale(t.v_exp[b < last ? b : last]);
        }
    }
    const float wd = t.weight_decay < 0.0f ? a.s.wd : t.weight_decay, lr = a.s.lr * t.lr_scale;
    uint32_t key = 0;
    if constexpr (BITS == 8) key = noise_key(a.s.seed, d.t, c.tensor, c.begin);
#pragma unroll
    for (int u = 0; u < kBlocksPerWave; ++u) {
        const int64_t e = e0 + u * kThreads * 4;
        if constexpr (BITS == 8) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t x = cm[u] >> (8 * k) & 255, y = cv[u] >> (8 * k) & 255;
                const float mag = decode<14>(x & 127, bm[u]);
                m[u][k] = x & 128 ? -mag : mag;
                v[u][k] = decode<30>(y, bv[u]);
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float pk = p[u][k], mk = m[u][k], vk = v[u][k];
            adam(g[u][k], pk, mk, vk, a.s, d, wd, lr);
            p[u][k] = pk;
            m[u][k] = mk;
            v[u][k] = vk;
        }
        store4(t.master, e, n, p[u]);
        if constexpr (TYPE != 3) store4(static_cast<T*>(t.param), e, n, p[u]);
        if constexpr (BITS == 32) {
            store4(static_cast<float*>(t.m), e, n, m[u]);
            store4(static_cast<float*>(t.v), e, n, v[u]);
        } else {
            uint32_t top_m = 0, top_v = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (e + k < n) {
                    const uint32_t x = __builtin_bit_cast(uint32_t, fabsf(m[u][k]));
                    const uint32_t y = __builtin_bit_cast(uint32_t, fabsf(v[u][k]));
                    top_m = x > top_m ? x : top_m;
                    top_v = y > top_v ? y : top_v;
                }
            const int em = block_exp(wave_max(top_m)), ev = block_exp(wave_max(top_v));
            const float im = pow2(em == kExpNaN ? 0 : -em), iv = pow2(ev == kExpNaN ? 0 : -ev);
            uint32_t xm = 0, xv = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t r = mix(key + (uint32_t)(e + k) * 0xDDB3D743u);
                const uint32_t x = encode<14>(fabsf(m[u][k]), im, r & 0xffffu);
                const uint32_t y = encode<30>(v[u][k], iv, r >> 16);
                xm |= ((x & 127) | (m[u][k] < 0.0f ? 128u : 0u)) << (8 * k);
                xv |= (y & 255) << (8 * k);
            }
            store_codes(static_cast<uint8_t*>(t.m), e, n, xm);
            store_codes(static_cast<uint8_t*>(t.v), e, n, xv);
            const int64_t first = e - lane * 4;       // the wave's block
            if (lane == 0 && first < n) {
                t.m_exp[first / kStateBlock] = (int8_t)em;
                t.v_exp[first / kStateBlock] = (int8_t)ev;
            }
        }
    }
}

template <int BITS>
__global__ __launch_bounds__(kThreads) void update_kernel(AdamwLaunch a)
{
    const ChunkEntry c = a.chunks[blockIdx.x];
    const TensorEntry t = a.tensors[c.tensor];
    const AdamwState d = *a.state;
    if (d.skip) return;
    if (t.type == 1) update_chunk<1, BITS>(a, d, t, c);
    else if (t.type == 2) update_chunk<2, BITS>(a, d, t, c);
    else update_chunk<3, BITS>(a, d, t, c);
}

// ------------------------------------------------------------------ tables and states

struct GradPointers {
    const void* p[kGradsPerLaunch];
};

__global__ __launch_bounds__(kGradsPerLaunch) void set_grads_kernel(TensorEntry* tensors, GradPointers g, int count)
{
    const int k = threadIdx.x;
    if (k < count) tensors[k].grad = g.p[k];
}

__global__ void set_state_kernel(AdamwState* state, AdamwState to) { *state = to; }

template <bool SIGNED>
__global__ __launch_bounds__(kThreads) void pack_kernel(const float* x, uint8_t* codes, int8_t* exps, int64_t n)
{
    const int64_t e = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4;
    const int lane = threadIdx.x & 63;
    const f4 v = load4(x, e, n);
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t b = __builtin_bit_cast(uint32_t, fabsf(v[k]));
        top = b > top ? b : top;
    }
    const int be = block_exp(wave_max(top));
    const float inv = pow2(be == kExpNaN ? 0 : -be);
    uint32_t c = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        // to the nearest: half a code, less half of the noise's last place
        if constexpr (SIGNED)
            c |= ((encode<14>(fabsf(v[k]), inv, 32767) & 127) | (v[k] < 0.0f ? 128u : 0u)) << (8 * k);
        else
            c |= (encode<30>(v[k] > 0.0f ? v[k] : 0.0f, inv, 32767) & 255) << (8 * k);
    }
    store_codes(codes, e, n, c);
    if (lane == 0 && e < n) exps[e / kStateBlock] = (int8_t)be;
}

template <typename T, bool SIGNED>
__global__ __launch_bounds__(kThreads) void unpack_kernel(const uint8_t* codes, const int8_t* exps, T* out, int64_t n)
{
    const int64_t e = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4;
    if (e >= n) return;
    const float b = block_scale(exps[e / kStateBlock]);
    const uint32_t c = load_codes(codes, e, n);
    f4 x;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t y = c >> (8 * k) & 255;
        if constexpr (SIGNED) {
            const float mag = decode<14>(y & 127, b);
            x[k] = y & 128 ? -mag : mag;
        } else {
            x[k] = decode<30>(y, b);
        }
    }
    store4(out, e, n, x);
}

}  // namespace

hipError_t adamw_step(const AdamwLaunch& a, int bits, bool checked, hipStream_t s)
{
    const dim3 grid((unsigned)a.nchunks);
    if (checked && a.nchunks > 0) norm_kernel<<<grid, kThreads, 0, s>>>(a);
    decide_kernel<<<1, 1024, 0, s>>>(a, checked);
    if (a.nchunks > 0) {
        if (bits == 32) update_kernel<32><<<grid, kThreads, 0, s>>>(a);
        else update_kernel<8><<<grid, kThreads, 0, s>>>(a);
    }
    return hipGetLastError();
}

hipError_t adamw_set_state(AdamwState* state, const AdamwState& to, hipStream_t s)
{
    set_state_kernel<<<1, 1, 0, s>>>(state, to);
    return hipGetLastError();
}

hipError_t adamw_set_grads(TensorEntry* tensors, const void* const* grads, int64_t first, int count, hipStream_t s)
{
    GradPointers g{};
    for (int k = 0; k < count; ++k) g.p[k] = grads[first + k];
    set_grads_kernel<<<1, kGradsPerLaunch, 0, s>>>(tensors + first, g, count);
    return hipGetLastError();
}

hipError_t moments_pack(const float* x, uint8_t* codes, int8_t* exps, int64_t n, bool is_signed, hipStream_t s)
{
    const dim3 grid((unsigned)ceil_div(n, kThreads * 4));
    if (n == 0) return hipSuccess;
    if (is_signed) pack_kernel<true><<<grid, kThreads, 0, s>>>(x, codes, exps, n);
    else pack_kernel<false><<<grid, kThreads, 0, s>>>(x, codes, exps, n);
    return hipGetLastError();
}

template <typename T>
static void unpack(const uint8_t* codes, const int8_t* exps, void* out, int64_t n, bool is_signed, hipStream_t s)
{
    const dim3 grid((unsigned)ceil_div(n, kThreads * 4));
    if (is_signed) unpack_kernel<T, true><<<grid, kThreads, 0, s>>>(codes, exps, static_cast<T*>(out), n);
    else unpack_kernel<T, false><<<grid, kThreads, 0, s>>>(codes, exps, static_cast<T*>(out), n);
}

hipError_t moments_unpack(const uint8_t* codes, const int8_t* exps, void* out, int64_t n, int type, bool is_signed,
                          hipStream_t s)
{
    if (n == 0) return hipSuccess;
    if (type == 2) unpack<__bf16>(codes, exps, out, n, is_signed, s);
    else unpack<float>(codes, exps, out, n, is_signed, s);
    return hipGetLastError();
}

}  // namespace zo
