// One tile of C[i][j] = sum_k P(i,k) Q(j,k) with 2-byte operands and fp32 sums, for
// the three products of the vocabulary loss.
//
// A workgroup of 8 waves takes 256 x 256 results, 64 deep at a time: both
// operands' 256 x 64 pieces (32 KiB each) go from memory straight to LDS, double
// buffered (128 of the CU's 160 KiB), and each wave keeps 128 x 64 results in
// registers as 8 x 4 products of 16 x 16 x 32.  A step of 64 is 2048 cycles of
// the matrix cores for the CU's two waves per SIMD, against about 1536 cycles of
// LDS reads and 64 KiB of loads, which have the whole step to arrive.
//
// An operand lies in memory either with k contiguous (kInner: row i has its k
// side by side) or with k as its rows (kOuter).  Both are loaded as 16-byte
// chunks and kept in LDS as they lie; kOuter fragments are turned by the
// transposing LDS read, so no transposed copy of anything is made.  Rows and k
// past the ends come in as zeros by the buffer descriptor's range check.
//
// LDS banks: the chunk that a lane fetches is chosen so that chunk c of a row is
// kept at place c ^ key(row); the keys make the rows that one read touches lie in
// different banks (kInner: the 8 rows that read together; kOuter: the 4 or 8
// rows of k).
#pragma once

#include "ops_common.h"

namespace zo {

enum Layout { kInner = 0, kOuter = 1 };

constexpr int kTile = 256;      // results of a workgroup each way
constexpr int kDeep = 64;       // k of one step
constexpr int kGemmThreads = 512;
constexpr int kWaveI = 128, kWaveJ = 64;
constexpr int kOperandBytes = kTile * kDeep * 2;
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kLgkmDone = 0xc07f;                // s_waitcnt lgkmcnt(0) alone
constexpr uint32_t kOutOfRange = 0x7ffffff0u;    // a byte offset past every descriptor's end

typedef float f4 __attribute__((ext_vector_type(4)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef short s8 __attribute__((ext_vector_type(8)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

#define ZO_LDS __attribute__((address_space(3)))

template <typename T> struct Mfma;
template <> struct Mfma<__bf16> {
    static __device__ __forceinline__ f4 run(s8 a, s8 b, f4 c)
    {
        typedef __bf16 v __attribute__((ext_vector_type(8)));
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v, a),
                                                       __builtin_bit_cast(v, b), c, 0, 0, 0);
    }
};
template <> struct Mfma<_Float16> {
    static __device__ __forceinline__ f4 run(s8 a, s8 b, f4 c)
    {
        typedef _Float16 v __attribute__((ext_vector_type(8)));
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v, a),
                                                      __builtin_bit_cast(v, b), c, 0, 0, 0);
    }
};

// Where an operand lies: `rows` i (or j) by `depth` k, 2-byte elements.  kInner:
// element (i, k) at i * ld + k, `depth` a multiple of 8.  kOuter: at k * ld + i,
// `rows` a multiple of 8.  Base 16-byte aligned, ld a multiple of 8,
// ld <= 2^21 (an offset inside a tile stays below 2^30 bytes).
struct Operand {
    const void* base;
    int64_t ld;
    int64_t rows;
    int64_t depth;
};

// Loads of one operand: the wave's 4 of the 32 instructions of 1 KiB that fill a
// stage.  PERMUTED marks the operand whose 16-row products interleave (below).
template <Layout L, bool PERMUTED>
struct Loader {
    const char* base;        // of this tile at the current k
    int64_t left;            // bytes from base to the operand's end
    int64_t step;            // bytes from one step to the next
    uint32_t voff[4];
    int chunk_k[4];          // kInner: first k of the lane's chunk within the step
    int64_t k_left;          // kInner: k left from the current step on

    // the swizzle of a row's 8 chunks (kInner)
    static __device__ __forceinline__ int key_inner(int row)
    {
        return PERMUTED ? (row & 3) | ((row >> 4) & 1) << 2 : row & 7;
    }
    // the swizzle of a k row's 32 chunks (kOuter)
    static __device__ __forceinline__ int key_outer(int k)
    {
        return 2 * ((k & 3) | ((k >> 3) & 1) << 2);
    }

    __device__ __forceinline__ void init(const Operand& o, int64_t row0, int64_t k0, int wave, int lane)
    {
        if constexpr (L == kInner) {
            base = static_cast<const char*>(o.base) + (row0 * o.ld + k0) * 2;
            int64_t rows = o.rows - row0;
            rows = rows < kTile ? rows : kTile;
            left = ((rows - 1) * o.ld + o.depth - k0) * 2;
            step = kDeep * 2;
            k_left = o.depth - k0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = wave * 32 + q * 8 + (lane >> 3);
                const int chunk = (lane & 7) ^ key_inner(row);
                chunk_k[q] = chunk * 8;
                voff[q] = (uint32_t)((row * o.ld + chunk * 8) * 2);
            }
        } else {
            base = static_cast<const char*>(o.base) + (k0 * o.ld + row0) * 2;
            left = ((o.depth - k0 - 1) * o.ld + o.rows - row0) * 2;
            step = kDeep * o.ld * 2;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int k = wave * 8 + q * 2 + (lane >> 5);
                const int chunk = (lane & 31) ^ key_outer(k);
                voff[q] = (uint32_t)((k * o.ld + chunk * 8) * 2);
            }
        }
    }

    // Start the loads of the current step into the operand's stage at LDS byte
    // address `lds`, and move on.  They are done when the wave's vmcnt says so.
    // Written as assembly because the builtin makes the compiler wait for every
    // such load before the next LDS read, also of the other stage; there is no
    // output register that could be reused too early.
    __device__ __forceinline__ void issue(uint32_t lds, int wave)
    {
        const int64_t reach = 0x40000000;    // no offset inside a tile is larger
        const uint32_t range = left <= 0 ? 0u : (uint32_t)(left < reach ? left : reach);
        const uint64_t b = (uint64_t)base;
        u4 rsrc;
        rsrc[0] = __builtin_amdgcn_readfirstlane((uint32_t)b);
        rsrc[1] = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32) & 0xffffu);
        rsrc[2] = __builtin_amdgcn_readfirstlane(range);
        rsrc[3] = 0x00020000u;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t v = voff[q];
            if constexpr (L == kInner)
                if (chunk_k[q] >= k_left) v = kOutOfRange;
            const uint32_t m = __builtin_amdgcn_readfirstlane(lds + (wave * 4 + q) * 1024);
            asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                         :
                         : "s"(m), "v"(v), "s"(rsrc));
        }
        base += step;
        left -= step;
        if constexpr (L == kInner) k_left -= kDeep;
    }
};

// Fragments for one product of 16 x 16 x 32: lane l has row l % 16 and the 8 k from
// (l / 16) * 8.  A wave's part begins at row `w0` of the tile; product t of it
// takes rows w0 + 16 t + r, or with PERMUTED (t < 4) rows w0 + (r / 4) * 16 + 4 t + r % 4:
// then the four products give each lane 16 results side by side.
template <Layout L, bool PERMUTED>
struct Reader {
    uint32_t addr;       // kInner: of (t = 0, kk = 0); kOuter: before ^ (t << 5)

    __device__ __forceinline__ void init(uint32_t operand, int w0, int lane)
    {
        const int r = lane & 15, g = lane >> 4;
        if constexpr (L == kInner) {
            const int row = w0 + (PERMUTED ? (r >> 2) * 16 + (r & 3) : r);
            addr = operand + row * 128 + ((g ^ Loader<L, PERMUTED>::key_inner(row)) << 4);
        } else {
            const int k = g * 8 + (r >> 2);
            const int chunk = (w0 >> 3) | ((r & 3) >> 1);
            addr = operand + k * 512 + ((chunk ^ Loader<L, PERMUTED>::key_outer(k)) << 4) + (r & 1) * 8;
        }
    }

    __device__ __forceinline__ s8 get(uint32_t stage, int t, int kk) const
    {
        if constexpr (L == kInner) {
            // product t is 16 (PERMUTED: 4) rows further on; the other half of the
            // step's k is chunk ^ 4
            const uint32_t a = ((addr ^ (kk << 6)) + stage) + t * (PERMUTED ? 512 : 2048);
            return *(ZO_LDS const s8*)(uintptr_t)a;
        } else {
            const uint32_t a = ((addr ^ (t << 5)) + stage) + kk * 16384;
            const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZO_LDS s4*)(uintptr_t)a);
            const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZO_LDS s4*)(uintptr_t)(a + 2048));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
};

// acc[ti][tj][e]: result i = wave's i0 + 16 ti + lane % 16, and j = wave's j0 +
// 16 tj + 4 (lane / 16) + e, or with the permuted kInner Q j0 + 16 (lane / 16) + 4 tj + e.
// `steps` of kDeep from k0 on.  smem: 2 * kStageBytes.
template <typename T, Layout LP, Layout LQ>
__device__ __forceinline__ void gemm_tile(const Operand& P, const Operand& Q, int64_t i0, int64_t j0,
                                          int64_t k0, int steps, uint32_t smem, f4 (&acc)[8][4])
{
    constexpr bool PERM = LQ == kInner;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Loader<LP, false> lp;
    Loader<LQ, PERM> lq;
    lp.init(P, i0, k0, wave, lane);
    lq.init(Q, j0, k0, wave, lane);
    Reader<LP, false> rp;
    Reader<LQ, PERM> rq;
    rp.init(smem, (wave >> 2) * kWaveI, lane);
    rq.init(smem + kOperandBytes, (wave & 3) * kWaveJ, lane);
#pragma unroll
    for (int ti = 0; ti < 8; ++ti)
#pragma unroll
        for (int tj = 0; tj < 4; ++tj) acc[ti][tj] = f4{0, 0, 0, 0};
    if (steps <= 0) return;
    // Fragments of half a step (32 of k) are read while the half before is
    // multiplied; the barrier of a step stands between its two halves, where the
    // other half's fragments are on hand to go on with.
    s8 a0[4], b0[8], a1[4], b1[8];
    lp.issue(smem, wave);
    lq.issue(smem + kOperandBytes, wave);
    asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
    if (steps > 1) {
        lp.issue(smem + kStageBytes, wave);
        lq.issue(smem + kStageBytes + kOperandBytes, wave);
    }
#pragma unroll
    for (int tj = 0; tj < 4; ++tj) a0[tj] = rq.get(0, tj, 0);
#pragma unroll
    for (int ti = 0; ti < 8; ++ti) b0[ti] = rp.get(0, ti, 0);
    for (int s = 0; s < steps; ++s) {
        const uint32_t stage = (s & 1) ? kStageBytes : 0, other = kStageBytes - stage;
#pragma unroll
        for (int tj = 0; tj < 4; ++tj) a1[tj] = rq.get(stage, tj, 1);
#pragma unroll
        for (int ti = 0; ti < 8; ++ti) b1[ti] = rp.get(stage, ti, 1);
#pragma unroll
        for (int ti = 0; ti < 8; ++ti)
#pragma unroll
            for (int tj = 0; tj < 4; ++tj) acc[ti][tj] = Mfma<T>::run(a0[tj], b0[ti], acc[ti][tj]);
        // the next step's loads have arrived, for every wave; and every wave has all
        // that it reads of this stage (the products above stay above: they are what
        // the reads hide behind)
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(kLgkmDone);    // (the builtin: the compiler counts on it)
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        if (s + 2 < steps) {
            lp.issue(smem + stage, wave);
            lq.issue(smem + stage + kOperandBytes, wave);
        }
        if (s + 1 < steps) {
#pragma unroll
            for (int tj = 0; tj < 4; ++tj) a0[tj] = rq.get(other, tj, 0);
#pragma unroll
            for (int ti = 0; ti < 8; ++ti) b0[ti] = rp.get(other, ti, 0);
        }
#pragma unroll
        for (int ti = 0; ti < 8; ++ti)
#pragma unroll
            for (int tj = 0; tj < 4; ++tj) acc[ti][tj] = Mfma<T>::run(a1[tj], b1[ti], acc[ti][tj]);
    }
}

}  // namespace zo
