// One tile of C[i][j] = sum_k P(i,k) Q(j,k) with 2-byte operands and fp32 sums, for
// the three products of the vocabulary loss.
//
// A workgroup of 8 waves (2 by 4) takes 32 NI x 64 NJ results, 64 deep at a time:
// both operands' pieces go from memory straight to LDS, double buffered, and each
// wave keeps 16 NI x 16 NJ results in registers, as products of 16 x 16 x 32.
//
// What bounds it, for NI x NJ = 8 x 4 (256 x 256), from parts timed apart on 8192 x
// 8192 x 8192: the products alone take 615 us (1790 TFLOP/s, at the power limit), the
// LDS reads 320, the loads 690 (12.5 TB/s out of the L2s), all together 826.  So the
// larger tile, 256 x 320, which loads a tenth less for each product, is taken where
// it wastes no more at the edges; NI = 2 serves few rows, with room for more
// workgroups in a CU.  Loads are started right behind the barrier, all of them (spread
// among the products they arrive later: 10% slower), and never less than 64 deep
// (pieces of 64 bytes a row: 10% slower, even with four steps under way).
//
// An operand lies in memory either with k contiguous (kInner: row i has its k
// side by side) or with k as its rows (kOuter).  Both are loaded as 16-byte
// chunks and kept in LDS as they lie; kOuter fragments are turned by the
// transposing LDS read, so no transposed copy of anything is made.  Rows and k
// past the ends come in as zeros by the buffer descriptor's range check.
//
// LDS banks: the chunk that a lane fetches is chosen so that chunk c of a row is
// kept at place c ^ key(row); the keys make the rows that one read touches lie in
// different banks.
#pragma once

#include "ops_common.h"

namespace zo {

enum Layout { kInner = 0, kOuter = 1 };

constexpr int kDeep = 64;       // k of one step
constexpr int kGemmThreads = 512;
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
// element (i, k) at i * ld + k; kOuter: at k * ld + i.  Base 4-byte aligned, ld even,
// ld <= 2^21 (an offset inside a tile stays below 2^31 - 16 bytes).
// Loads are of 8 elements: a kInner depth is a multiple of 8; what a kOuter tile reads
// beyond `rows` goes into results that are none.
struct Operand {
    const void* base;
    int64_t ld;
    int64_t rows;
    int64_t depth;
    int64_t pairs = 0;       // kOuter, one step: of so many entries, in pairs (see pair_row)
    bool twice = false;      // with pairs: they lie once, and both of a pair are the same row
};

// The piece of an operand that a tile reads, as it moves along k.
struct Piece {
    const char* base;        // at the current k
    int64_t left;            // bytes from base to the operand's end
    int64_t step;            // bytes from one step to the next

    __device__ __forceinline__ u4 descriptor() const
    {
        const int64_t reach = 0x7fffff00;    // no offset inside a tile is larger
        const uint32_t range = left <= 0 ? 0u : (uint32_t)(left < reach ? left : reach);
        const uint64_t b = (uint64_t)base;
        u4 rsrc;
        rsrc[0] = __builtin_amdgcn_readfirstlane((uint32_t)b);
        rsrc[1] = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32) & 0xffffu);
        rsrc[2] = __builtin_amdgcn_readfirstlane(range);
        rsrc[3] = 0x00020000u;
        return rsrc;
    }
    __device__ __forceinline__ void advance()
    {
        base += step;
        left -= step;
    }
};

// The range check goes by words of 4 bytes: the one that an odd count of elements
// ends in is loaded.
__device__ __forceinline__ int64_t whole_words(int64_t bytes) { return (bytes + 3) & ~(int64_t)3; }

// One load of 1 KiB into LDS at byte address `lds`: the lane's 16 bytes at offset v.
// It is done when the wave's vmcnt says so.  Written as assembly because the
// builtin makes the compiler wait for every such load before the next LDS read, also of
// the other stage; there is no output register that could be reused too early.
__device__ __forceinline__ void load_to_lds(uint32_t v, const u4& rsrc, uint32_t lds)
{
    const uint32_t m = __builtin_amdgcn_readfirstlane(lds);
    asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(m), "v"(v), "s"(rsrc));
}

// kInner operand of 64 C rows: rows of 64 k (128 bytes) in LDS, 8 chunks each; a wave
// loads C times 8 rows.  C is 1 (64 rows), 4 or 5.
//
// Fragments: lane l has row l % 16 and the 8 k from (l / 16) * 8.  Product t of a wave
// takes rows w0 + 16 t + r; with RUNS products 0 to 3 take rows w0 + 16 (r / 4) + 4 t + r % 4
// of the first 256 (then the four give each lane 16 results side by side), and with C = 5
// product 4 takes 16 of the last 64.
template <int C, bool RUNS>
struct Inner {
    static constexpr int kBytes = C * 64 * kDeep * 2;
    Piece piece;
    int64_t k_left;
    uint32_t voff, voff_last, apart;
    int chunk_k, chunk_k_last;
    uint32_t addr, addr_last;

    // Rows that one read takes together: r, r + 1, ... r + 7; with runs {0..3, 16..19} + 4 t.
    static __device__ __forceinline__ int key(int row, bool runs)
    {
        return runs ? (row & 3) | ((row >> 4) & 1) << 2 : row & 7;
    }
    // The tile from row0 and k0 on.
    __device__ __forceinline__ void begin(const Operand& o, int64_t row0, int64_t k0)
    {
        piece.base = static_cast<const char*>(o.base) + (row0 * o.ld + k0) * 2;
        int64_t rows = o.rows - row0;
        rows = rows < C * 64 ? rows : C * 64;
        piece.left = whole_words(((rows - 1) * o.ld + o.depth - k0) * 2);
        piece.step = kDeep * 2;
        k_left = o.depth - k0;
    }
    // What a lane loads of any tile.
    __device__ __forceinline__ void lanes(const Operand& o, int wave, int lane)
    {
        // load q of wave w: rows 64 q + 8 w to + 7, with the key of row 8 w + ...
        const int row = wave * 8 + (lane >> 3);
        const int chunk = (lane & 7) ^ key(row, RUNS);
        chunk_k = chunk * 8;
        voff = (uint32_t)((row * o.ld + chunk * 8) * 2);
        if constexpr (C == 5 && RUNS) {
            const int last = (lane & 7) ^ key(row, false);
            chunk_k_last = last * 8;
            voff_last = (uint32_t)(((256 + row) * o.ld + last * 8) * 2);
        }
        apart = (uint32_t)(64 * o.ld * 2);
    }
    __device__ __forceinline__ void issue(uint32_t lds, int wave)
    {
        const u4 rsrc = piece.descriptor();
        uint32_t first = voff;
        asm volatile("" : "+v"(first));      // (added to here, not kept C times in registers)
#pragma unroll
        for (int q = 0; q < C; ++q) {
            uint32_t v = chunk_k >= k_left ? kOutOfRange : first + q * apart;
            if constexpr (C == 5 && RUNS)
                if (q == 4) v = chunk_k_last >= k_left ? kOutOfRange : voff_last;
            load_to_lds(v, rsrc, lds + (q * 8 + wave) * 1024);
        }
        piece.advance();
        k_left -= kDeep;
    }
    // w: which of the waves along this side
    __device__ __forceinline__ void reader(uint32_t lds, int w, int products, int lane)
    {
        const int r = lane & 15, g = lane >> 4;
        const int row = RUNS ? w * 64 + (r >> 2) * 16 + (r & 3) : w * 16 * products + r;
        addr = lds + row * 128 + ((g ^ key(row, RUNS)) << 4);
        if constexpr (C == 5 && RUNS) {
            const int last = 256 + w * 16 + r;
            addr_last = lds + last * 128 + ((g ^ key(last, false)) << 4);
        }
    }
    __device__ __forceinline__ s8 get(uint32_t stage, int t, int kk) const
    {
        // (the other half of the step's k is chunk ^ 4)
        uint32_t a = ((addr ^ (kk << 6)) + stage) + t * (RUNS ? 512 : 2048);
        if constexpr (C == 5 && RUNS)
            if (t == 4) a = (addr_last ^ (kk << 6)) + stage;
        return *(ZO_LDS const s8*)(uintptr_t)a;
    }
};

// Entries in pairs: rows 32 b to + 15 are the first halves of entries 16 b to + 15, rows
// 32 b + 16 to + 31 the second halves, so that products of 16 rows have both in one lane.
__host__ __device__ __forceinline__ int64_t pair_row(int64_t entry) { return (entry >> 4) * 32 + (entry & 15); }
__host__ __device__ __forceinline__ int64_t pair_rows(int64_t entries) { return (entries + 15) / 16 * 32; }
__device__ __forceinline__ int pair_entry(int row) { return (row >> 5) * 16 + (row & 15); }

// Byte offset of row k of a step.  Rows that are no entry's are zeros.
__device__ __forceinline__ uint32_t offset_of_k(const Operand& o, int k, int column)
{
    if (o.pairs > 0) {
        if (pair_entry(k) >= o.pairs) return kOutOfRange;
        if (o.twice) k = pair_entry(k);
    }
    return (uint32_t)((k * o.ld + column) * 2);
}


// 64 columns of a kOuter operand: 64 rows of k with 128 bytes each.
struct Outer64 {
    static constexpr int kBytes = 64 * kDeep * 2;
    uint32_t voff, addr;

    // 16 lanes read 4 rows of k, 32 lanes 8, 32 bytes of each: all in different banks
    static __device__ __forceinline__ int key(int k) { return 2 * ((k & 3) ^ ((k >> 3) & 1)); }
    __device__ __forceinline__ void init(const Operand& o, int col0, int wave, int lane)
    {
        const int k = wave * 8 + (lane >> 3);
        const int chunk = (lane & 7) ^ key(k);
        voff = offset_of_k(o, k, col0 + chunk * 8);
    }
    __device__ __forceinline__ void issue(const u4& rsrc, uint32_t lds, int wave)
    {
        load_to_lds(voff, rsrc, lds + wave * 1024);
    }
    __device__ __forceinline__ void reader(uint32_t lds, int w0, int lane)
    {
        const int r = lane & 15, g = lane >> 4, k = g * 8 + (r >> 2);
        const int chunk = (w0 >> 3) | ((r & 3) >> 1);
        addr = lds + k * 128 + ((chunk ^ key(k)) << 4) + (r & 1) * 8;
    }
    __device__ __forceinline__ s8 get(uint32_t stage, int t, int kk) const
    {
        const uint32_t a = ((addr ^ (t << 5)) + stage) + kk * 4096;
        const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZO_LDS s4*)(uintptr_t)a);
        const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZO_LDS s4*)(uintptr_t)(a + 512));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

// 256 columns: 64 rows of k with 512 bytes each.  With RUNS the four products of a wave
// take columns w0 + 16 (r / 4) + 4 t + r % 4, so that a lane's results lie side by
// side, at the price of bank conflicts: where storing is what takes the time.
template <bool RUNS>
struct Outer256 {
    static constexpr int kBytes = 256 * kDeep * 2;
    uint32_t voff[2], apart[RUNS ? 2 : 1], addr;     // (RUNS: there may be pairs)

    static __device__ __forceinline__ int key(int k) { return 2 * ((k & 3) | ((k >> 3) & 1) << 2); }
    __device__ __forceinline__ void init(const Operand& o, int wave, int lane)
    {
        // load q of wave w: rows 8 w + 2 q and + 1 of k; q and q + 2 have the same key
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int k = wave * 8 + q * 2 + (lane >> 5);
            const int chunk = (lane & 31) ^ key(k);
            if constexpr (RUNS) {
                voff[q] = offset_of_k(o, k, chunk * 8);
                apart[q] = offset_of_k(o, k + 4, chunk * 8) - voff[q];
            } else {
                voff[q] = (uint32_t)((k * o.ld + chunk * 8) * 2);
            }
        }
        if constexpr (!RUNS) apart[0] = (uint32_t)(4 * o.ld * 2);
    }
    __device__ __forceinline__ void issue(const u4& rsrc, uint32_t lds, int wave)
    {
        uint32_t first[2] = {voff[0], voff[1]};
        asm volatile("" : "+v"(first[0]), "+v"(first[1]));
#pragma unroll
        for (int q = 0; q < 4; ++q)
            load_to_lds(first[q & 1] + (q >> 1) * apart[RUNS ? q & 1 : 0], rsrc, lds + (wave * 4 + q) * 1024);
    }
    __device__ __forceinline__ void reader(uint32_t lds, int w0, int lane)
    {
        const int r = lane & 15, g = lane >> 4, k = g * 8 + (r >> 2);
        const int chunk = (w0 >> 3) | ((r & 3) >> 1);
        const int piece = RUNS ? (w0 >> 3) | (r & 3) * 2 : chunk;
        addr = lds + k * 512 + ((piece ^ key(k)) << 4) + (RUNS ? 0 : (r & 1) * 8);
    }
    __device__ __forceinline__ s8 get(uint32_t stage, int t, int kk) const
    {
        // (keys are even: bit 4 of the address is the chunk's own low bit)
        const uint32_t turn = RUNS ? (t >> 1) << 4 | (t & 1) << 3 : t << 5;
        const uint32_t a = ((addr ^ turn) + stage) + kk * 16384;
        const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZO_LDS s4*)(uintptr_t)a);
        const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZO_LDS s4*)(uintptr_t)(a + 2048));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

// kOuter operand of 64 C columns: 64, 256, or 256 and 64 beside them (C = 5).
// Product t of a wave with W products: columns 16 (w W + t); with C = 5 products 0 to 3
// lie in the 256 and product 4 in the 64, at 256 + 16 w.
template <int C, bool RUNS>
struct Outer {
    static_assert(C == 1 || C == 4 || (C == 5 && !RUNS), "");
    static constexpr int kWide = C == 1 ? 0 : Outer256<RUNS>::kBytes;
    static constexpr int kBytes = C * 64 * kDeep * 2;
    Piece piece;
    Outer256<RUNS> wide;
    Outer64 narrow;

    __device__ __forceinline__ void begin(const Operand& o, int64_t col0, int64_t k0)
    {
        piece.base = static_cast<const char*>(o.base) + (k0 * o.ld + col0) * 2;
        piece.left = whole_words(((o.depth - k0 - 1) * o.ld + o.rows - col0) * 2);
        piece.step = kDeep * o.ld * 2;
    }
    __device__ __forceinline__ void lanes(const Operand& o, int wave, int lane)
    {
        if constexpr (C >= 4) wide.init(o, wave, lane);
        if constexpr (C != 4) narrow.init(o, C == 5 ? 256 : 0, wave, lane);
    }
    __device__ __forceinline__ void issue(uint32_t lds, int wave)
    {
        const u4 rsrc = piece.descriptor();
        if constexpr (C >= 4) wide.issue(rsrc, lds, wave);
        if constexpr (C != 4) narrow.issue(rsrc, lds + kWide, wave);
        piece.advance();
    }
    __device__ __forceinline__ void reader(uint32_t lds, int w, int products, int lane)
    {
        if constexpr (C >= 4) wide.reader(lds, C == 5 ? w * 64 : w * 16 * products, lane);
        if constexpr (C != 4) narrow.reader(lds + kWide, C == 5 ? w * 16 : w * 16 * products, lane);
    }
    __device__ __forceinline__ s8 get(uint32_t stage, int t, int kk) const
    {
        if constexpr (C == 1) return narrow.get(stage, t, kk);
        else if constexpr (C == 5) return t == 4 ? narrow.get(stage, 0, kk) : wide.get(stage, t, kk);
        else return wide.get(stage, t, kk);
    }
};

template <Layout L, int C, bool RUNS> struct Side;
template <int C, bool RUNS> struct Side<kInner, C, RUNS> { using type = Inner<C, RUNS>; };
template <int C, bool RUNS> struct Side<kOuter, C, RUNS> { using type = Outer<C, RUNS>; };

// acc[ti][tj][e]: i by row_of(), j by column_of() below, within the tile.  One tile:
// begin(), then run(); a workgroup that goes on to another tile begins it from run()'s
// `free`, which is called when both stages have been read, so that its loads are under
// way during the last products and whatever is done with the results.
template <typename T, Layout LP, Layout LQ, int NI, int NJ>
struct Gemm {
    static constexpr int kTileI = 32 * NI, kTileJ = 64 * NJ;
    using PSide = typename Side<LP, NI / 2, false>::type;
    // a lane's results of products 0 to 3 lie side by side
    static constexpr bool kRuns = LQ == kInner || NI == 2;
    using QSide = typename Side<LQ, NJ, kRuns>::type;
    static constexpr int kStageBytes = PSide::kBytes + QSide::kBytes;
    static constexpr int kLds = 2 * kStageBytes;
    // Both halves' fragments beside the results, where 256 registers hold them.  (8 x 4:
    // 3% faster with P kInner; with both kOuter 1% slower.)
    static constexpr bool kAhead = LP == kInner && NI * NJ * 4 + 8 * (NI + NJ) <= 224;

    // First j of results acc[.][tj][0..3] of a lane, within the tile.
    static __device__ __forceinline__ int column_of(int tj, int wave, int lane)
    {
        const int w = wave & 3, g = lane >> 4;
        if (tj == 4) return 256 + w * 16 + g * 4;
        return kRuns ? w * 64 + g * 16 + tj * 4 : w * 64 + tj * 16 + g * 4;
    }
    static __device__ __forceinline__ int row_of(int ti, int wave, int lane)
    {
        return (wave >> 2) * 16 * NI + ti * 16 + (lane & 15);
    }

    struct Half {
        s8 a[NJ], b[NI];
    };
    static __device__ __forceinline__ void read(Half& f, const PSide& p, const QSide& q, uint32_t stage, int kk)
    {
#pragma unroll
        for (int tj = 0; tj < NJ; ++tj) f.a[tj] = q.get(stage, tj, kk);
#pragma unroll
        for (int ti = 0; ti < NI; ++ti) f.b[ti] = p.get(stage, ti, kk);
    }
    static __device__ __forceinline__ void multiply(const Half& f, f4 (&acc)[NI][NJ])
    {
#pragma unroll
        for (int ti = 0; ti < NI; ++ti)
#pragma unroll
            for (int tj = 0; tj < NJ; ++tj) acc[ti][tj] = Mfma<T>::run(f.a[tj], f.b[ti], acc[ti][tj]);
    }
    // The next step's loads have arrived, for every wave; and every wave has all that it
    // reads of this stage.  (What stands above stays above.)
    static __device__ __forceinline__ void turn()
    {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(kLgkmDone);    // (the builtin: the compiler counts on it)
        asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    }

    PSide p;
    QSide q;
    int wave;
    uint32_t smem;

    // lds: address of kLds bytes (kStageBytes where every tile has one step), a multiple
    // of 1024.
    __device__ __forceinline__ Gemm(const Operand& P, const Operand& Q, uint32_t lds) : smem(lds)
    {
        const int lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        p.lanes(P, wave, lane);
        q.lanes(Q, wave, lane);
        p.reader(smem, wave >> 2, NI, lane);
        q.reader(smem + PSide::kBytes, wave & 3, NJ, lane);
    }
    __device__ __forceinline__ void issue(uint32_t stage)
    {
        p.issue(smem + stage, wave);
        q.issue(smem + stage + PSide::kBytes, wave);
    }
    // Start on the tile at (i0, j0), `steps` of kDeep from k0 on.
    __device__ __forceinline__ void begin(const Operand& P, const Operand& Q, int64_t i0, int64_t j0, int64_t k0,
                                          int steps)
    {
        p.begin(P, i0, k0);
        q.begin(Q, j0, k0);
        if (steps > 0) issue(0);
        if (steps > 1) issue(kStageBytes);
    }
    template <typename F>
    __device__ __forceinline__ void run(int steps, f4 (&acc)[NI][NJ], F free)
    {
#pragma unroll
        for (int ti = 0; ti < NI; ++ti)
#pragma unroll
            for (int tj = 0; tj < NJ; ++tj) acc[ti][tj] = f4{0, 0, 0, 0};
        if (steps <= 0) return free();
        Half even;
        turn();
        if constexpr (kAhead) {
            // Fragments of half a step are read while the half before is multiplied; the
            // step's barrier stands between its halves, where the other half's
            // fragments are on hand to go on with.
            Half odd;
            read(even, p, q, 0, 0);
            for (int s = 0; s < steps; ++s) {
                const uint32_t stage = (s & 1) ? kStageBytes : 0, other = kStageBytes - stage;
                read(odd, p, q, stage, 1);
                multiply(even, acc);
                turn();
                if (s + 2 < steps) issue(stage);
                if (s + 1 < steps) read(even, p, q, other, 0);
                else free();
                multiply(odd, acc);
            }
        } else {
            for (int s = 0; s < steps; ++s) {
                const uint32_t stage = (s & 1) ? kStageBytes : 0;
                read(even, p, q, stage, 0);
                multiply(even, acc);
                read(even, p, q, stage, 1);
                turn();
                if (s + 2 < steps) issue(stage);
                if (s + 1 == steps) free();
                multiply(even, acc);
            }
        }
    }
};

}  // namespace zo
