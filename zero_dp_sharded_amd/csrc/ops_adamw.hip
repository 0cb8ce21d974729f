// AdamW over the tensors of a model at once, with moments in 32 or in 8 bits.
//
// One launch updates every tensor: a table in device memory, made when the handle
// is, cuts the tensors into chunks, a workgroup each.  A lane has 4 elements side by
// side, so that every load and store of a wave is whole lines (512 bytes of 2-byte
// gradients, 1 KiB of fp32), and a wave's 256 elements are a block of the 8-bit
// states.  Bound by memory: per element and step 28 bytes with fp32 moments and 2-byte
// storage, 16 with 8-bit moments; with the latter only because the arithmetic is
// spare (a division by a step's constant in 3 operations, one hash for both moments'
// noise, powers of two by ldexp): at 5 TB/s a wave has about 400 cycles for 256
// elements of 16 bytes.
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

template <int TYPE> struct Stored;
template <> struct Stored<1> { using T = _Float16; };
template <> struct Stored<2> { using T = __bf16; };
template <> struct Stored<3> { using T = float; };

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
// the largest of all): inside rows of 16 lanes by DPP (a rotation by 8 or 4 reaches the
// partner once those before agree), across rows by shuffles.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x)
{
    const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, false);
    return x > y ? x : y;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t x)
{
    x = dpp_max<0x128>(x);      // row_ror:8
    x = dpp_max<0x124>(x);      // row_ror:4
    x = dpp_max<0x4E>(x);       // quad_perm [2,3,0,1]
    x = dpp_max<0xB1>(x);       // quad_perm [1,0,3,2]
#pragma unroll
    for (int off = 16; off <= 32; off *= 2) {
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

// A value to a code: scaled so that the code's least normal exponent is fp32's, the
// code is the top bits of the float's magnitude, and noise below them, added, rounds.
// LEAST: 14 (m) or 30 (v).
template <int LEAST>
__device__ __forceinline__ uint32_t encode(float x, int block, uint32_t r16)
{
    const float z = __builtin_amdgcn_ldexpf(fabsf(x), LEAST - 126 - block);
    return (__builtin_bit_cast(uint32_t, z) + (r16 << 4) + 8) >> 20;
}

__device__ __forceinline__ uint32_t encode_m(float x, int block, uint32_t r16)
{
    return (encode<14>(x, block, r16) & 127) | (__builtin_bit_cast(uint32_t, x) >> 24 & 128);
}

__device__ __forceinline__ uint32_t encode_v(float x, int block, uint32_t r16)
{
    return encode<30>(x, block, r16) & 255;
}

// The code in bits 8 k to 8 k + 7, and what it stands for.
__device__ __forceinline__ float decode_m(uint32_t codes, int k, int block)
{
    const uint32_t c = codes << (24 - 8 * k);                       // at the top
    const uint32_t bits = (c & 0x7f000000u) >> 4 | (c & 0x80000000u);
    return __builtin_amdgcn_ldexpf(__builtin_bit_cast(float, bits), 126 - 14 + block);
}

__device__ __forceinline__ float decode_v(uint32_t codes, int k, int block)
{
    return __builtin_amdgcn_ldexpf(__builtin_bit_cast(float, (codes >> (8 * k) & 255) << 20), 126 - 30 + block);
}

// A stored exponent for the decoders; a block of nothing finite is multiplied by NaN.
__device__ __forceinline__ int block_of(int e) { return e < kExpLeast ? kExpLeast : e; }

// x / c for a constant c in (0, 1], r its reciprocal, rounded: the quotient's
// remainder is exact, and one step with it rounds as the division does (Markstein).
// Where the remainder could fall below fp32's range the division itself is taken.
__device__ __forceinline__ float divide_by(float x, float c, float r)
{
    const float q = x * r;
    const float exact = fmaf(fmaf(-q, c, x), r, q);
    const uint32_t b = __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
    if (__builtin_expect(b - 1 < 0x0d000000u - 1 || b >= 0x7e800000u, 0)) return x / c;    // below 2^-101, above 2^126
    return exact;
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
__device__ __forceinline__ void norm_part(const TensorEntry& t, int64_t begin, int64_t end, float inv_scale,
                                          double& ss)
{
    using T = typename Stored<TYPE>::T;
    constexpr int W = Vec<T>::W;
    const T* g = static_cast<const T*>(t.grad);
    auto add = [&](float x) {
        const double y = (double)(x * inv_scale);
        ss = __builtin_fma(y, y, ss);      // (the product is exact in 64 bits)
    };
    int64_t e = begin + threadIdx.x * W;
    constexpr int64_t step = kThreads * W;
    for (; e + 3 * step + W <= end; e += 4 * step) {
        vec_t<T, W> x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = load_vec<T, W>(g + e + u * step);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int k = 0; k < W; ++k) add((float)x[u][k]);
    }
    for (; e < end; e += step) {
        if (e + W <= end) {
            const vec_t<T, W> x = load_vec<T, W>(g + e);
#pragma unroll
            for (int k = 0; k < W; ++k) add((float)x[k]);
        } else {
            for (int64_t k = e; k < end; ++k) add((float)g[k]);
        }
    }
}

// The step's decision, as the shard's device-resident flow takes it, from the state
// before it and the sum of squares (0 without a check: every step is taken).
__device__ __forceinline__ AdamwState decide(const AdamwLaunch& a, AdamwState d, double s)
{
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
    return d;
}

__device__ __forceinline__ double block_sum(double x, double* sh)
{
    x = wave_sum(x);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = x;
    __syncthreads();
    return (sh[0] + sh[1]) + (sh[2] + sh[3]);
}

// Workgroup b sums the squares of chunks [b n / grid, (b + 1) n / grid), tensor by tensor,
// into an fp64 partial.  A value that is not finite makes its sum so, and no finite
// ones can: fp32 squares stay far below fp64's range.
__global__ __launch_bounds__(kThreads) void norm_kernel(AdamwLaunch a)
{
    __shared__ double sh[4];
    const float inv_scale = a.state->inv_scale;
    const int64_t last = a.nchunks * (blockIdx.x + 1) / gridDim.x;
    double ss = 0.0;
    for (int64_t c = a.nchunks * blockIdx.x / gridDim.x; c < last;) {
        const ChunkEntry first = a.chunks[c];
        const TensorEntry t = a.tensors[first.tensor];
        // as many chunks as are left of this tensor
        int64_t count = ceil_div(t.numel - first.begin, a.chunk);
        if (count > last - c) count = last - c;
        int64_t end = first.begin + count * a.chunk;
        if (end > t.numel) end = t.numel;
        if (t.type == 1) norm_part<1>(t, first.begin, end, inv_scale, ss);
        else if (t.type == 2) norm_part<2>(t, first.begin, end, inv_scale, ss);
        else norm_part<3>(t, first.begin, end, inv_scale, ss);
        c += count;
    }
    ss = block_sum(ss, sh);
    if (threadIdx.x == 0) {
        a.partial[blockIdx.x] = ss;
        // the state as the update finds it that decides for itself
        if (blockIdx.x == 0) a.state[1] = a.state[0];
    }
}

// The partials in a fixed order, and the decision.  (A launch of its own: left to the
// workgroup of the check that ends last, the fences that takes cost 100 us at 2048
// workgroups, against 5 for the launch.)
__device__ __forceinline__ double sum_partials(const double* partial, int64_t partials)
{
    __shared__ double sh[4];
    double s = 0.0;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < partials; i += kThreads) s += partial[i];
    return block_sum(s, sh);
}

__global__ __launch_bounds__(kThreads) void decide_kernel(AdamwLaunch a, int64_t partials)
{
    const double s = sum_partials(a.partial, partials);
    if (threadIdx.x == 0) *a.state = decide(a, *a.state, s);
}

// ------------------------------------------------------------------ the update

// Textbook Adam on one element, in the order of the public header.
__device__ __forceinline__ void adam(float g, float& p, float& m, float& v, const AdamwScalars& s,
                                     const AdamwState& d, float r1, float r2, float wd, float lr)
{
    g = g * d.upd_inv_scale;
    g = g * d.clip;
    if (s.l2) g = g + wd * p;
    m = s.b1 * m + s.omb1 * g;
    v = s.b2 * v + s.omb2 * (g * g);
    float u = divide_by(m, d.bc1, r1) / (sqrtf(divide_by(v, d.bc2, r2)) + s.eps);
    if (!s.l2) u = u + wd * p;
    p = p - lr * u;
}

// U: blocks of 256 elements a wave.  `decided` gives the step's state, once the loads
// are under way.
template <int TYPE, int BITS, int U, typename F>
__device__ __forceinline__ void update_chunk(const AdamwLaunch& a, const TensorEntry& t, const ChunkEntry& c,
                                             F decided)
{
    using T = typename Stored<TYPE>::T;
    const int64_t n = t.numel;
    const int lane = threadIdx.x & 63;
    f4 g[U], p[U], m[U], v[U];
    uint32_t cm[U], cv[U];
    int bm[U], bv[U];
    const int64_t e0 = c.begin + threadIdx.x * 4;
#pragma unroll
    for (int u = 0; u < U; ++u) {
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
            bm[u] = t.m_exp[b < last ? b : last];
            bv[u] = t.v_exp[b < last ? b : last];
        }
    }
    const AdamwState d = decided();
    if (d.skip) return;
    const float wd = t.weight_decay < 0.0f ? a.s.wd : t.weight_decay, lr = a.s.lr * t.lr_scale;
    const float r1 = 1.0f / d.bc1, r2 = 1.0f / d.bc2;
    uint32_t key = 0;
    if constexpr (BITS == 8) key = noise_key(a.s.seed, d.t, c.tensor, c.begin);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t e = e0 + u * kThreads * 4;
        if constexpr (BITS == 8) {
            const int em = block_of(bm[u]), ev = block_of(bv[u]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                m[u][k] = decode_m(cm[u], k, em);
                v[u][k] = decode_v(cv[u], k, ev);
            }
            if (em == kExpNaN || ev == kExpNaN) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    m[u][k] = em == kExpNaN ? __builtin_nanf("") : m[u][k];
                    v[u][k] = ev == kExpNaN ? __builtin_nanf("") : v[u][k];
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float pk = p[u][k], mk = m[u][k], vk = v[u][k];
            adam(g[u][k], pk, mk, vk, a.s, d, r1, r2, wd, lr);
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
            uint32_t xm = 0, xv = 0;
            const uint32_t at = key + (uint32_t)e * 0xDDB3D743u;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t r = mix(at + k * 0xDDB3D743u);
                xm |= encode_m(m[u][k], em, r & 0xffffu) << (8 * k);
                xv |= encode_v(v[u][k], ev, r >> 16) << (8 * k);
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

// PARTIALS: every workgroup adds the check's partials itself and takes the same
// decision from the state that the check left aside; the first writes it.  Up to 512
// partials (2M elements: 17.2 -> 16.3 us a step) that is faster than a launch for it.
template <int BITS, int U, bool PARTIALS>
__global__ __launch_bounds__(kThreads) void update_kernel(AdamwLaunch a, int64_t partials)
{
    const ChunkEntry c = a.chunks[blockIdx.x];
    const TensorEntry t = a.tensors[c.tensor];
    auto decided = [&]() -> AdamwState {
        if constexpr (!PARTIALS) {
            return *a.state;
        } else {
            __shared__ AdamwState sh;
            const double s = sum_partials(a.partial, partials);
            if (threadIdx.x == 0) {
                sh = decide(a, a.state[1], s);
                if (blockIdx.x == 0) a.state[0] = sh;
            }
            __syncthreads();
            return sh;
        }
    };
    if (t.type == 1) update_chunk<1, BITS, U>(a, t, c, decided);
    else if (t.type == 2) update_chunk<2, BITS, U>(a, t, c, decided);
    else update_chunk<3, BITS, U>(a, t, c, decided);
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
    uint32_t c = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        // to the nearest: half a code, less half of the noise's last place
        if constexpr (SIGNED) c |= encode_m(v[k], be, 32767) << (8 * k);
        else c |= encode_v(v[k] > 0.0f ? v[k] : 0.0f, be, 32767) << (8 * k);
    }
    store_codes(codes, e, n, c);
    if (lane == 0 && e < n) exps[e / kStateBlock] = (int8_t)be;
}

// 8 elements a lane: 512 bytes of codes a wave, and 1 or 2 KiB of values.
template <typename T, bool SIGNED>
__global__ __launch_bounds__(kThreads) void unpack_kernel(const uint8_t* codes, const int8_t* exps, T* out, int64_t n)
{
    const int64_t e = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 8;
    if (e >= n) return;
    const int b = block_of(exps[e / kStateBlock]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t c = load_codes(codes, e + 4 * h, n);
        f4 x;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[k] = SIGNED ? decode_m(c, k, b) : decode_v(c, k, b);
            if (b == kExpNaN) x[k] = __builtin_nanf("");
        }
        store4(out, e + 4 * h, n, x);
    }
}

}  // namespace

hipError_t adamw_step(const AdamwLaunch& a, int bits, bool checked, hipStream_t s)
{
    // the check: a workgroup for 4096 elements, and 8 a CU at most, whose loads fill the
    // memory's pipe
    int64_t sums = checked ? ceil_div(a.nchunks * a.chunk, kAdamwChunk) : 0;
    if (sums > kAdamwPartials) sums = kAdamwPartials;
    if (sums > 0) norm_kernel<<<dim3((unsigned)sums), kThreads, 0, s>>>(a);
    const dim3 grid((unsigned)a.nchunks);
    const bool small = a.chunk == kAdamwSmallChunk;
    if (small && sums > 0 && sums <= kAdamwInline) {
        if (bits == 32) update_kernel<32, 1, true><<<grid, kThreads, 0, s>>>(a, sums);
        else update_kernel<8, 1, true><<<grid, kThreads, 0, s>>>(a, sums);
        return hipGetLastError();
    }
    decide_kernel<<<1, kThreads, 0, s>>>(a, sums);
    if (a.nchunks > 0) {
        if (bits == 32 && small) update_kernel<32, 1, false><<<grid, kThreads, 0, s>>>(a, 0);
        else if (bits == 32) update_kernel<32, 4, false><<<grid, kThreads, 0, s>>>(a, 0);
        else if (small) update_kernel<8, 1, false><<<grid, kThreads, 0, s>>>(a, 0);
        else update_kernel<8, 4, false><<<grid, kThreads, 0, s>>>(a, 0);
    }
    return hipGetLastError();
}

int64_t adamw_chunk(int64_t elements) { return elements < kAdamwLarge ? kAdamwSmallChunk : kAdamwChunk; }

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
    const dim3 grid((unsigned)ceil_div(n, kThreads * 8));
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
