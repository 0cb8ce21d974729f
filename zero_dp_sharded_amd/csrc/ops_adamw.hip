// AdamW over the tensors of a model at once, with moments in 32 or in 8 bits.
//
// One launch updates every tensor: a table in device memory, made when the handle
// is, cuts the tensors into chunks, of one workgroup or several.  A lane has 4 elements side by
// side, so that every load and store of a wave is whole lines (512 bytes of 2-byte
// gradients, 1 KiB of fp32), and a wave's 256 elements are a block of the 8-bit
// states.  Bound by memory: per element and step 28 bytes with fp32 moments and 2-byte
// storage, 16 with 8-bit moments, and the check reads the gradient once more.  326M
// elements take 1476 us with the check, 6.6 TB/s, as a copy past the caches does.  With
// 8-bit moments the arithmetic binds as well, spare as it is (a division by a step's
// constant in 3 operations, one hash for both moments' noise, powers of two by ldexp):
// 120 vector instructions an element, 1040 us, 5.0 TB/s.  Up to 2M elements it is two
// launches and their latency: 1.8M in 16.5 us.
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
// 5 bits of exponent cover gradients that differ by 2^15 within a block (of constant ones no
// update is above twice Adam's).  Further down a v falls to 0 beside an m that does not, and
// single updates grow: 28 times Adam's at 2^16, 200 times at 2^20.
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
constexpr int kLds = 160 * 1024;      // of a CU

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

// Four values to codes, side by side: scaled so that the code's least normal exponent is
// fp32's, the code is the top bits of the float's magnitude, and 16 bits of noise below them,
// added, round.  LEAST: 14 (m) or 30 (v).  Below the least normal exponent the scaling would
// round by itself, to 2^-20 of a code's step, and could carry a value past the noise's border:
// there the bits are those of the value as an integer, cut off.  (They are the fewest: one
// test for four.)
template <int LEAST, bool SIGNED>
__device__ __forceinline__ uint32_t encode(f4 x, int block, const uint32_t (&noise)[4])
{
    uint32_t z[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) z[k] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_ldexpf(fabsf(x[k]), LEAST - 126 - block));
    const uint32_t a = z[0] < z[1] ? z[0] : z[1], b = z[2] < z[3] ? z[2] : z[3];
    if (__builtin_expect((a < b ? a : b) <= 0x800000u, 0)) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (z[k] <= 0x800000u) z[k] = (uint32_t)__builtin_amdgcn_ldexpf(fabsf(x[k]), LEAST + 23 - block);
    }
    uint32_t codes = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t c = (z[k] + (noise[k] << 4) + 8) >> 20;
        const float xk = x[k];      // (the bits of a vector's element itself come out as an older value's)
        if constexpr (SIGNED) codes |= ((c & 127) | (__builtin_bit_cast(uint32_t, xk) >> 24 & 128)) << (8 * k);
        else codes |= (c & 255) << (8 * k);
    }
    return codes;
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
// Where the remainder could fall below fp32's range, or the quotient pass it (then the
// remainder is infinite, and the step inf - inf), the division itself is taken.  (r is at
// least 1: a quotient below 2^126 has an x below it too.)
__device__ __forceinline__ float divide_by(float x, float c, float r)
{
    const float q = x * r;
    const float exact = fmaf(-fmaf(q, c, -x), r, q);      // (so, and not by x - q c: a -0 stays one)
    const uint32_t b = __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
    const uint32_t big = __builtin_bit_cast(uint32_t, q) & 0x7fffffffu;
    if (__builtin_expect(b - 1 < 0x0d000000u - 1 || big >= 0x7e800000u, 0)) return x / c;    // x below 2^-101, q above 2^126
    return exact;
}

// 4 elements from e on of an array of n, zeros past the end.
template <bool NT = false, typename T>
__device__ __forceinline__ f4 load4(const T* p, int64_t e, int64_t n)
{
    f4 x;
    if (e + 4 <= n) {
        const vec_t<T, 4> v = load_vec<T, 4, NT>(p + e);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = (float)v[k];
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = e + k < n ? (float)p[e + k] : 0.0f;
    }
    return x;
}

template <bool NT = false, typename T>
__device__ __forceinline__ void store4(T* p, int64_t e, int64_t n, f4 x)
{
    if (e + 4 <= n) {
        vec_t<T, 4> v;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = static_cast<T>(x[k]);
        store_vec<T, 4, NT>(p + e, v);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (e + k < n) p[e + k] = static_cast<T>(x[k]);
    }
}

template <bool NT = false>
__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int64_t e, int64_t n)
{
    if (e + 4 <= n) {
        const vec_t<uint8_t, 4> v = load_vec<uint8_t, 4, NT>(p + e);
        return __builtin_bit_cast(uint32_t, v);
    }
    uint32_t x = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (e + k < n) x |= (uint32_t)p[e + k] << (8 * k);
    return x;
}

template <bool NT = false>
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t e, int64_t n, uint32_t x)
{
    if (e + 4 <= n) {
        store_vec<uint8_t, 4, NT>(p + e, __builtin_bit_cast(vec_t<uint8_t, 4>, x));
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

// U: blocks of 256 elements a wave, those of a workgroup's waves side by side.
// `decided` gives the step's state, once the loads are under way.
template <int TYPE, int BITS, int WAVES, int U, bool NT, typename F>
__device__ __forceinline__ void update_part(const AdamwLaunch& a, const TensorEntry& t, int32_t tensor, int64_t begin,
                                            F decided)
{
    constexpr int kStep = WAVES * kStateBlock;
    using T = typename Stored<TYPE>::T;
    const int64_t n = t.numel;
    const int lane = threadIdx.x & 63;
    f4 g[U], p[U], m[U], v[U];
    uint32_t cm[U], cv[U];
    int bm[U], bv[U];
    const int64_t e0 = begin + threadIdx.x * 4;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t e = e0 + u * kStep;
        g[u] = load4<NT>(static_cast<const T*>(t.grad), e, n);
        p[u] = load4<NT>(t.master, e, n);
        if constexpr (BITS == 32) {
            m[u] = load4<NT>(static_cast<const float*>(t.m), e, n);
            v[u] = load4<NT>(static_cast<const float*>(t.v), e, n);
        } else {
            cm[u] = load_codes<NT>(static_cast<const uint8_t*>(t.m), e, n);
            cv[u] = load_codes<NT>(static_cast<const uint8_t*>(t.v), e, n);
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
    if constexpr (BITS == 8) key = noise_key(a.s.seed, d.t, tensor, begin);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t e = e0 + u * kStep;
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
        store4<NT>(t.master, e, n, p[u]);
        if constexpr (TYPE != 3) store4<NT>(static_cast<T*>(t.param), e, n, p[u]);
        if constexpr (BITS == 32) {
            store4<NT>(static_cast<float*>(t.m), e, n, m[u]);
            store4<NT>(static_cast<float*>(t.v), e, n, v[u]);
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
            uint32_t low[4], high[4];
            const uint32_t at = key + (uint32_t)e * 0xDDB3D743u;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t r = mix(at + k * 0xDDB3D743u);
                low[k] = r & 0xffffu;
                high[k] = r >> 16;
            }
            const uint32_t xm = encode<14, true>(m[u], em, low), xv = encode<30, false>(v[u], ev, high);
            store_codes<NT>(static_cast<uint8_t*>(t.m), e, n, xm);
            store_codes<NT>(static_cast<uint8_t*>(t.v), e, n, xv);
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
template <int BITS, int WAVES, int U, bool NT, bool PARTIALS>
__global__ __launch_bounds__(WAVES * 64) void update_kernel(AdamwLaunch a, int64_t partials)
{
    constexpr int kElements = WAVES * U * kStateBlock;
    const uint32_t parts = (uint32_t)(a.chunk / kElements);
    const ChunkEntry c = a.chunks[blockIdx.x / parts];
    const TensorEntry t = a.tensors[c.tensor];
    const int64_t begin = c.begin + blockIdx.x % parts * kElements;
    if (begin >= t.numel) return;              // (never the first workgroup)
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
    if (t.type == 1) update_part<1, BITS, WAVES, U, NT>(a, t, c.tensor, begin, decided);
    else if (t.type == 2) update_part<2, BITS, WAVES, U, NT>(a, t, c.tensor, begin, decided);
    else update_part<3, BITS, WAVES, U, NT>(a, t, c.tensor, begin, decided);
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

// NT: past the caches, for arrays of kAdamwLarge elements and more.
template <bool SIGNED, bool NT>
__global__ __launch_bounds__(kThreads) void pack_kernel(const float* x, uint8_t* codes, int8_t* exps, int64_t n)
{
    const int64_t e = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4;
    const int lane = threadIdx.x & 63;
    f4 v = load4<NT>(x, e, n);
    if constexpr (!SIGNED) {
        // negative inputs are 0, for the block's exponent too (a NaN stays one)
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = v[k] < 0.0f ? 0.0f : v[k];
    }
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t b = __builtin_bit_cast(uint32_t, fabsf(v[k]));
        top = b > top ? b : top;
    }
    const int be = block_exp(wave_max(top));
    // to the nearest: half a code's step, less half of the noise's last place
    const uint32_t half[4] = {32767, 32767, 32767, 32767};
    const uint32_t c = encode<SIGNED ? 14 : 30, SIGNED>(v, be, half);
    store_codes<NT>(codes, e, n, c);
    if (lane == 0 && e < n) exps[e / kStateBlock] = (int8_t)be;
}

// 16 bytes of values a lane and store, kUnpack of them: a wave's loads and stores are whole
// lines (326M values to bf16 161 us, 6.1 TB/s; 212 through the caches, and 430 past
// them with half lines).
constexpr int kUnpack = 4;

template <typename T, bool SIGNED, bool NT>
__global__ __launch_bounds__(kThreads) void unpack_kernel(const uint8_t* codes, const int8_t* exps, T* out, int64_t n)
{
    constexpr int W = Vec<T>::W;
    const int64_t e0 = ((int64_t)blockIdx.x * kUnpack * kThreads + threadIdx.x) * W, last = (n - 1) / kStateBlock;
    uint32_t c[kUnpack][W / 4];
    int b[kUnpack];
#pragma unroll
    for (int u = 0; u < kUnpack; ++u) {
        const int64_t e = e0 + u * kThreads * W, block = e / kStateBlock;
        if (e + W <= n) {
            const auto v = load_vec<uint8_t, W, NT>(codes + e);
            __builtin_memcpy(c[u], &v, W);
        } else {
#pragma unroll
            for (int q = 0; q < W / 4; ++q) c[u][q] = load_codes<false>(codes, e + 4 * q, n);
        }
        b[u] = block_of(exps[block < last ? block : last]);
    }
#pragma unroll
    for (int u = 0; u < kUnpack; ++u) {
        const int64_t e = e0 + u * kThreads * W;
        vec_t<T, W> x;
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const float y = SIGNED ? decode_m(c[u][k / 4], k % 4, b[u]) : decode_v(c[u][k / 4], k % 4, b[u]);
            x[k] = static_cast<T>(b[u] == kExpNaN ? __builtin_nanf("") : y);
        }
        if (e + W <= n) {
            store_vec<T, W, NT>(out + e, x);
        } else {
#pragma unroll
            for (int k = 0; k < W; ++k)
                if (e + k < n) out[e + k] = x[k];
        }
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
    const bool small = a.chunk == kAdamwSmallChunk;
    // `parts` workgroups of `threads` lanes a chunk
    auto update = [&](auto kernel, int threads, int64_t parts, int lds, int64_t partials) {
        in_launches(a.nchunks, threads * (int)parts, [&](int64_t first, int64_t count) {
            AdamwLaunch from = a;
            from.chunks += first;
            kernel<<<dim3((unsigned)(count * parts)), threads, lds, s>>>(from, partials);
        });
        return hipGetLastError();
    };
    if (small && sums > 0 && sums <= kAdamwInline)
        return bits == 32 ? update(update_kernel<32, 4, 1, false, true>, kThreads, 1, 0, sums)
                          : update(update_kernel<8, 4, 1, false, true>, kThreads, 1, 0, sums);
    decide_kernel<<<1, kThreads, 0, s>>>(a, sums);
    if (small)
        return bits == 32 ? update(update_kernel<32, 4, 1, false, false>, kThreads, 1, 0, 0)
                          : update(update_kernel<8, 4, 1, false, false>, kThreads, 1, 0, 0);
    // Past the caches, all of it.  With fp32 moments 8 streams share the memory, and a wave
    // of 256 elements a workgroup, 18 to a CU (held there by LDS that is asked for and
    // not used), is what it serves best: 326M elements in 1471 us with the check
    // (16 a CU: 1488, 14: 1542, 20: 1527; workgroups of 4 waves of 1024 elements: 1720,
    // and 1883 through the caches).  With 8-bit moments the arithmetic wants all the waves
    // there are: workgroups of 4 of 1024 elements and no limit 1010 us (through the caches
    // 1050; 16 waves of 256 elements 1550; timed before the smallest codes were rounded once,
    // which made it 1040).
    if (bits == 32) return update(update_kernel<32, 1, 1, true, false>, 64, a.chunk / kStateBlock, kLds / 18 - 1024, 0);
    return update(update_kernel<8, 4, 4, true, false>, kThreads, 1, 0, 0);
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

template <bool NT>
static void pack(const float* x, uint8_t* codes, int8_t* exps, int64_t n, bool is_signed, hipStream_t s)
{
    constexpr int64_t kGroup = kThreads * 4;       // elements of a workgroup
    auto run = [&](auto kernel) {
        in_launches(ceil_div(n, kGroup), kThreads, [&](int64_t first, int64_t count) {
            const int64_t e = first * kGroup;
            kernel<<<dim3((unsigned)count), kThreads, 0, s>>>(x + e, codes + e, exps + e / kStateBlock, n - e);
        });
    };
    if (is_signed) run(pack_kernel<true, NT>);
    else run(pack_kernel<false, NT>);
}

hipError_t moments_pack(const float* x, uint8_t* codes, int8_t* exps, int64_t n, bool is_signed, hipStream_t s)
{
    if (n == 0) return hipSuccess;
    if (n < kAdamwLarge) pack<false>(x, codes, exps, n, is_signed, s);
    else pack<true>(x, codes, exps, n, is_signed, s);
    return hipGetLastError();
}

template <typename T, bool NT>
static void unpack(const uint8_t* codes, const int8_t* exps, void* out, int64_t n, bool is_signed, hipStream_t s)
{
    constexpr int64_t kGroup = (int64_t)kUnpack * kThreads * Vec<T>::W;
    auto run = [&](auto kernel) {
        in_launches(ceil_div(n, kGroup), kThreads, [&](int64_t first, int64_t count) {
            const int64_t e = first * kGroup;
            kernel<<<dim3((unsigned)count), kThreads, 0, s>>>(codes + e, exps + e / kStateBlock, static_cast<T*>(out) + e, n - e);
        });
    };
    if (is_signed) run(unpack_kernel<T, true, NT>);
    else run(unpack_kernel<T, false, NT>);
}

hipError_t moments_unpack(const uint8_t* codes, const int8_t* exps, void* out, int64_t n, int type, bool is_signed,
                          hipStream_t s)
{
    if (n == 0) return hipSuccess;
    const bool large = n >= kAdamwLarge;
    if (type == 2 && large) unpack<__bf16, true>(codes, exps, out, n, is_signed, s);
    else if (type == 2) unpack<__bf16, false>(codes, exps, out, n, is_signed, s);
    else if (large) unpack<float, true>(codes, exps, out, n, is_signed, s);
    else unpack<float, false>(codes, exps, out, n, is_signed, s);
    return hipGetLastError();
}

}  // namespace zo
