// Shared by the training operators' kernels (ops_*.hip): storage types, vectors
// of 16 bytes at any address, and sums over a wave in a fixed order.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace zo {

constexpr int kWave = 64;
constexpr int kCUs = 256;    // compute units of an MI355X: launch shapes are cut for it

template <typename T> struct Vec;    // W elements of T in 16 bytes
template <> struct Vec<_Float16> { static constexpr int W = 8; };
template <> struct Vec<__bf16> { static constexpr int W = 8; };
template <> struct Vec<float> { static constexpr int W = 4; };

template <typename T, int W> using vec_t = T __attribute__((ext_vector_type(W)));

// The same vector at an address aligned to one element only: the card loads and
// stores 16 bytes at any element's address, so rows of odd widths need no path
// of their own.
template <typename T, int W>
using any_vec = T __attribute__((ext_vector_type(W), aligned(sizeof(T))));

// NT: past the caches, for what is touched once and is larger than they are (a copy
// of 2 GiB reaches 6.6 TB/s so, and 5.0 without).
template <typename T, int W, bool NT = false>
__device__ __forceinline__ vec_t<T, W> load_vec(const T* p)
{
    const auto* v = reinterpret_cast<const any_vec<T, W>*>(p);
    if constexpr (NT) return __builtin_nontemporal_load(v);
    else return *v;
}

template <typename T, int W, bool NT = false>
__device__ __forceinline__ void store_vec(T* p, vec_t<T, W> x)
{
    auto* v = reinterpret_cast<any_vec<T, W>*>(p);
    if constexpr (NT) __builtin_nontemporal_store((any_vec<T, W>)x, v);
    else *v = x;
}

// Sum over the 64 lanes, the same in every lane (xor butterfly).
__device__ __forceinline__ float wave_sum(float x)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off, kWave);
    return x;
}

__device__ __forceinline__ double wave_sum(double x)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off, kWave);
    return x;
}

// Work-items of one launch: HIP counts a grid's in 32 bits, and larger work goes in
// consecutive launches.  (Defined smaller in a build of the tests.)
#ifndef ZO_MAX_LAUNCH_ITEMS
#define ZO_MAX_LAUNCH_ITEMS (int64_t(1) << 31)
#endif
constexpr int64_t kMaxLaunchItems = ZO_MAX_LAUNCH_ITEMS;

// `groups` workgroups of `lanes` lanes: launch(first, count) for each launch.
template <typename F>
void in_launches(int64_t groups, int lanes, F launch)
{
    const int64_t most = kMaxLaunchItems / lanes;
    for (int64_t first = 0; first < groups; first += most)
        launch(first, groups - first < most ? groups - first : most);
}

__host__ __device__ inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
__host__ __device__ inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

}  // namespace zo
