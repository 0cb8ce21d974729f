// 8-bit numbers with a power of two for every 128 of them, as the norm's output and the
// packing write them and the product reads them: e4m3 (a sign, 4 bits of exponent, 3 of
// mantissa; largest 448, 0x7f NaN, no infinity), and a byte E for the factor 2^(E - 127),
// 255 NaN: what the matrix instructions take as operand and scale.
//
// A block's E is the least that brings its largest finite value within 448, so that
// nothing saturates; a number loses nothing by a power of two but what falls below the
// least step (2^-9 of the scale).  E is 27 (2^-100) at least: every value then is a bf16.
// An element that is not finite becomes NaN and does not enter the largest.  One above 1.875 *
// 2^127, which would round to 2^128, is held as that: none becomes infinite.
#pragma once

#include "ops_common.h"

namespace zo {

constexpr int kScaleBlock = 128;
constexpr uint32_t kLeastScale = 27;

// Sums and maxima over lanes by moves within the vector unit (a shuffle through LDS costs
// six times the latency).  DPP codes: quad_perm, row_half_mirror and row_mirror exchange
// lanes of 16; the rows of 16 and halves of 32 are exchanged by permlane swaps.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
}

constexpr int kXor1 = 0xb1, kXor2 = 0x4e, kHalfMirror = 0x141, kMirror = 0x140;

__device__ __forceinline__ uint32_t bits(float x) { return __builtin_bit_cast(uint32_t, x); }
__device__ __forceinline__ float from_bits(uint32_t x) { return __builtin_bit_cast(float, x); }

// Over the 64 lanes, the same in each (a swap of x with itself gives every lane both
// sides' values, in the same order).
__device__ __forceinline__ float lanes_sum(float x)
{
    x += from_bits(dpp<kXor1>(bits(x)));
    x += from_bits(dpp<kXor2>(bits(x)));
    x += from_bits(dpp<kHalfMirror>(bits(x)));
    x += from_bits(dpp<kMirror>(bits(x)));
    auto r = __builtin_amdgcn_permlane16_swap(bits(x), bits(x), false, false);
    x = from_bits(r[0]) + from_bits(r[1]);
    r = __builtin_amdgcn_permlane32_swap(bits(x), bits(x), false, false);
    return from_bits(r[0]) + from_bits(r[1]);
}

__device__ __forceinline__ double lanes_sum(double x)
{
    auto moved = [](double x, auto move) {
        const uint64_t u = __builtin_bit_cast(uint64_t, x);
        return __builtin_bit_cast(double, (uint64_t)move((uint32_t)(u >> 32)) << 32 | move((uint32_t)u));
    };
    x += moved(x, [](uint32_t u) { return dpp<kXor1>(u); });
    x += moved(x, [](uint32_t u) { return dpp<kXor2>(u); });
    x += moved(x, [](uint32_t u) { return dpp<kHalfMirror>(u); });
    x += moved(x, [](uint32_t u) { return dpp<kMirror>(u); });
    const double a = moved(x, [](uint32_t u) { return (uint32_t)__builtin_amdgcn_permlane16_swap(u, u, false, false)[0]; });
    const double b = moved(x, [](uint32_t u) { return (uint32_t)__builtin_amdgcn_permlane16_swap(u, u, false, false)[1]; });
    x = a + b;
    const double c = moved(x, [](uint32_t u) { return (uint32_t)__builtin_amdgcn_permlane32_swap(u, u, false, false)[0]; });
    const double d = moved(x, [](uint32_t u) { return (uint32_t)__builtin_amdgcn_permlane32_swap(u, u, false, false)[1]; });
    return c + d;
}

__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Over LANES (16, 32 or 64) lanes that lie together, the same in each.
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t x)
{
    x = larger(x, dpp<kXor1>(x));
    x = larger(x, dpp<kXor2>(x));
    x = larger(x, dpp<kHalfMirror>(x));
    x = larger(x, dpp<kMirror>(x));
    if constexpr (LANES >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        x = larger(r[0], r[1]);
    }
    if constexpr (LANES == 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        x = larger(r[0], r[1]);
    }
    return x;
}

constexpr uint32_t kNotFinite = 0x7f800000u;       // bits of |x| from there on

// The larger of `most` and what of x enters its block's largest: the bits of |x|, which are in the order of
// the values, or nothing where x is not finite.
__device__ __forceinline__ uint32_t with_size(uint32_t most, float x)
{
    const uint32_t a = bits(x) & 0x7fffffffu;
    return a < kNotFinite ? larger(most, a) : most;
}

// E of a block whose largest finite value has the bits u: 2^(e - 8), or the next where the
// mantissa passes 1.75 (448 = 1.75 * 2^8).
__device__ __forceinline__ uint32_t scale_of(uint32_t u)
{
    const int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < (int)kLeastScale ? kLeastScale : (uint32_t)e;
}

// 2^(E - 127) for every byte E.
__device__ __forceinline__ float scale_value(uint32_t E)
{
    if (E == 255) return __builtin_nanf("");
    return from_bits(E == 0 ? 0x00400000u : E << 23);
}

// Two codes in the half HI of `to`, rounded to nearest even from x 2^(127 - E).  (The conversions take the
// scale, and make NaN of what is not finite; nothing here is above 448 of it.)
typedef short short2_t __attribute__((ext_vector_type(2)));
template <bool HI>
__device__ __forceinline__ short2_t two_codes(short2_t to, float x0, float x1, float scale)
{
    return __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(to, x0, x1, scale, HI);
}
template <bool HI>
__device__ __forceinline__ short2_t two_codes(short2_t to, vec_t<_Float16, 2> x, float scale)
{
    return __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(to, x, scale, HI);
}
template <bool HI>
__device__ __forceinline__ short2_t two_codes(short2_t to, vec_t<__bf16, 2> x, float scale)
{
    return __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(to, x, scale, HI);
}

// The largest E is a block's whose largest is above 1.75 2^127: what is rounded to 2^128 there (code 0x78) is
// held as the number below it.
constexpr uint32_t kTopScale = 247;
__device__ __forceinline__ uint32_t below_top(uint32_t codes)
{
#pragma unroll
    for (int k = 0; k < 32; k += 8)
        if ((codes >> k & 0x7f) == 0x78) codes -= 1u << k;
    return codes;
}

// Four codes of x with E.
__device__ __forceinline__ uint32_t codes_of(float x0, float x1, float x2, float x3, uint32_t E)
{
    const float scale = from_bits(E << 23);
    short2_t r = {0, 0};
    r = two_codes<false>(r, x0, x1, scale);
    r = two_codes<true>(r, x2, x3, scale);
    const uint32_t c = __builtin_bit_cast(uint32_t, r);
    return E == kTopScale ? below_top(c) : c;
}

}  // namespace zo
