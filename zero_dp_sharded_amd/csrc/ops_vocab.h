// Shared by the operators over a vocabulary (ops_loss.hip, ops_logprobs.hip): the order of
// tiles, the factor that the logits' gradients are held with, and copies of operands that
// cannot be loaded as they lie.
#pragma once

#include "ops_common.h"
#include "ops_gemm.h"

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

}  // namespace
}  // namespace zo
