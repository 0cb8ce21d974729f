// Matrix product of 8-bit operands with a power of two for every 128 elements of the depth
// (ops_scaled.h): C[i][j] = sum_k A[i][k] B[j][k], both with k along their rows.
//
// The matrix instruction takes 16 x 16 x 128 codes and a scale byte of each operand's row for
// them, so a block is one instruction: the scales cost no arithmetic, and sums stay in its fp32
// accumulators from the first block to the last.  (With scales that are no powers of two,
// every instruction's 4 results a lane would be multiplied and added by the vector unit: as
// many cycles again.)
//
// Large: a workgroup of 4 waves (2 by 2) takes 32 NI x 256 results, 128 deep at a time, both
// operands' pieces straight to LDS, double buffered.  A wave has 16 NI x 128 results, and
// with NI = 8 a SIMD's registers to itself: what is read from LDS is two thirds of what 8 waves
// would read.  (Which of a row's chunks stands at which k of an instruction does not
// matter, as long as both operands agree.)  With a wave alone on its SIMD nothing hides what it waits for:
// loads go between the products one by one, and the next tile's are under way before this one's
// results are written.  8192 x 8192 x 8192 to bf16 390 us, 2820 TFLOP/s (the library's fp8 product without
// scales 2640 here); 8192 x 20480 x 5120 650 call after call (the library 693), 684 to 810 among a profiler's passes:
// bound by the power that the card may take.  With scales by rows on B's side too, 8 bytes of them a step for one, 3 to
// 7% more: 8192 x 8192 x 8192 415, 20480 x 5120 x 8192 712 to 737 for 680.
// Few tiles, or tiles that end badly in rounds of the card: lower ones, or parts of the depth (product_plan).
// fp32 results: exact_kernel.
//
// Few rows: B is what costs.  A wave takes 16 of its rows straight to registers, the waves of a
// workgroup share the depth and add their sums in LDS: one launch, no workspace.  A row x 6400 x 1600 5.5 us, of
// which 1.6 are B's bytes: the launch, one trip to memory and the sums are the rest.

#include <type_traits>

#include "ops_common.h"
#include "ops_gemm.h"
#include "ops_internal.h"
#include "ops_scaled.h"

namespace zo {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));

constexpr int kBlock = kScaleBlock;

// s_waitcnt: all LDS reads done, and of the loads and stores to memory all but the last `left` (they end
// in the order of their issue).
constexpr int wait_for(int left) { return 0x0070 | (left & 15) | (left >> 4) << 14; }

constexpr int kThreads = 256;

// Workgroups go round the dies; each die gets a run of tiles that lie together.
constexpr uint32_t kDies = 8;

// The n-th tile in that order: 8 tiles of i by all of j, column by column, so that a die's L2 serves
// the tiles that share an operand.
__device__ __forceinline__ void tile_at(uint32_t n, uint32_t ti, uint32_t tj, uint32_t& i, uint32_t& j)
{
    constexpr uint32_t kGroup = 8;
    const uint32_t per = kGroup * tj, g = n / per, first = g * kGroup;
    const uint32_t high = ti - first < kGroup ? ti - first : kGroup;
    i = __builtin_amdgcn_readfirstlane(first + (n - g * per) % high);
    j = __builtin_amdgcn_readfirstlane((n - g * per) / high);
}

// The tile of workgroup `id` of as many as there are tiles.
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t tiles, uint32_t ti, uint32_t tj, uint32_t& i, uint32_t& j)
{
    const uint32_t die = id % kDies, q = tiles / kDies, r = tiles % kDies;
    tile_at(die * q + (die < r ? die : r) + id / kDies, ti, tj, i, j);
}

// ------------------------------------------------------------------ tiles

struct TileArgs {
    const uint8_t* a;
    const uint8_t* b;
    const uint8_t* a_exps;
    const uint8_t* b_exps;
    int64_t a_ld, b_ld, a_exps_ld, b_exps_ld;
    int64_t depth;
    int blocks;                // of the depth
    void* out;
    const void* bias;
    float* part;               // splits: fp32 parts [split][rows][cols], else NULL
    int64_t rows, cols, out_ld;
    uint32_t ti, tj;
    int splits;                // each at least one block
};

// A kernel's only argument, read again from where it lies: kept in registers from tile to tile its fields
// would not leave enough.
typedef const __attribute__((address_space(4))) TileArgs* ArgsAt;
__device__ __forceinline__ ArgsAt args_at()
{
    ArgsAt t = (ArgsAt)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(t));
    return t;
}

__device__ __forceinline__ int least_of(int64_t left, int most) { return left < most ? (int)left : most; }

// One load of 256 bytes into LDS at byte address `lds`: the lane's 4 bytes at offset v.  As
// load_to_lds.
__device__ __forceinline__ void load_words_to_lds(uint32_t v, const u4& rsrc, uint32_t lds)
{
    const uint32_t m = __builtin_amdgcn_readfirstlane(lds);
    asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"(m), "v"(v), "s"(rsrc));
}

// The scales of up to 256 rows and 2 steps in LDS: the two words of 4 bytes that a row's two may
// lie in, as they are aligned in memory, [2][256].  Whole words are read: those that the first
// and the last byte lie in have others before and behind them.
struct Scales {
    static constexpr int kBytes = 2 * 256 * 4;
    Piece piece;
    uint32_t from;             // a lane's row: its next byte, from the words' beginning on
    int skew;                  // of the rows that a lane needs: the first byte's place in its word

    // The steps from -back on (0 or 1).
    // (row strides up to 2^22: every offset is below 2^30)
    __device__ __forceinline__ void begin(const uint8_t* x, int ld, int rows, int blocks, int back, int wave, int row)
    {
        const int over = (int)(reinterpret_cast<uintptr_t>(x) & 3);
        piece.base = reinterpret_cast<const char*>(x) - over;
        piece.left = (over + (rows - 1) * ld + blocks + 3) & ~3;
        const int mine = wave * 64 + (threadIdx.x & 63);
        from = mine < rows ? (uint32_t)(over + mine * ld - back) : kOutOfRange;
        skew = over + row * ld - back;
    }
    // The next 2 steps', to LDS at `lds`.
    __device__ __forceinline__ void issue(uint32_t lds, int wave)
    {
        const u4 rsrc = piece.descriptor();
        const uint32_t at = from & ~3u;
        load_words_to_lds(at, rsrc, lds + wave * 256);
        load_words_to_lds(at + 4, rsrc, lds + 1024 + wave * 256);
        from += 2;
    }
    // Where the scale of step s is (counted from -back on), of row `row`.
    __device__ __forceinline__ uint32_t at(uint32_t lds, int row, int s) const
    {
        const int byte = ((skew + (s & ~1)) & 3) + (s & 1);
        return lds + row * 4 + (byte >> 2) * 1024 + (byte & 3);
    }
};

// One operand's rows of a tile: 32 Q rows of 128 codes in LDS, chunk c of 16 codes of a row at
// place c ^ key(row), so that the rows that one read touches lie in different banks.  A
// wave loads 8 rows at a time.
//
// Fragments: lane l has row l % 16 of a product, chunks g and g + 4 with g = l / 16.  Product t
// takes rows 16 t + r; with RUNS products 4 u to 4 u + 3 take rows 64 u + 16 (r / 4) + 4 (t % 4) + r % 4,
// and the four give each lane 16 results side by side.
template <int Q, bool RUNS>
struct Rows {
    static constexpr int kBytes = Q * 32 * kBlock;
    Piece piece;
    int left;                  // codes of a row from here on
    uint32_t voff, apart, addr;
    int chunk;                 // a lane's, in 16 codes

    static __device__ __forceinline__ int key(int row) { return RUNS ? (row & 3) | ((row >> 4) & 1) << 2 : row & 7; }
    // (row strides up to 2^22: every offset inside a tile is below 2^30)
    __device__ __forceinline__ void lanes(int ld, int wave, int lane)
    {
        const int row = wave * 8 + (lane >> 3);            // (32 rows on the key is the same)
        chunk = ((lane & 7) ^ key(row)) * 16;
        voff = (uint32_t)(row * ld + chunk);
        apart = (uint32_t)(32 * ld);
    }
    // x: the tile's first row at its first code; `rows` of them, `depth` codes.  No rows: zeros.
    __device__ __forceinline__ void begin(const uint8_t* x, int ld, int rows, int depth)
    {
        piece.base = reinterpret_cast<const char*>(x);
        piece.left = rows > 0 ? ((rows - 1) * ld + depth + 3) & ~3 : 0;
        piece.step = kBlock;
        left = rows > 0 ? depth : 0;
    }
    // A stage's loads, Q of them, to LDS at `lds` (the wave's place there).
    struct Loads {
        u4 rsrc;
        uint32_t first, by, lds;
        __device__ __forceinline__ void issue(int q) const { load_to_lds(first + q * by, rsrc, lds + q * 4096); }
    };
    __device__ __forceinline__ Loads next(uint32_t lds, int wave)
    {
        Loads l;
        l.rsrc = piece.descriptor();
        l.first = chunk >= left ? kOutOfRange : voff;
        l.by = chunk >= left ? 0 : apart;
        l.lds = lds + wave * 1024;
        asm volatile("" : "+v"(l.first));    // (added to there, not kept Q times in registers)
        piece.advance();
        left -= kBlock;
        return l;
    }
    // first: the wave's first row
    __device__ __forceinline__ void reader(uint32_t lds, int first, int lane)
    {
        const int r = lane & 15, g = lane >> 4;
        const int row = first + (RUNS ? (r >> 2) * 16 + (r & 3) : r);
        addr = lds + row * 128 + ((g ^ key(row)) << 4);
    }
    __device__ __forceinline__ v8i get(uint32_t stage, int t) const
    {
        const uint32_t on = RUNS ? (t >> 2) * 8192 + (t & 3) * 512 : t * 2048;
        const u4 lo = *(ZO_LDS const u4*)(uintptr_t)(addr + stage + on);
        const u4 hi = *(ZO_LDS const u4*)(uintptr_t)((addr ^ 64) + stage + on);
        return __builtin_bit_cast(v8i, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

template <int NI, bool SQUARE>
struct Tile {
    static constexpr int NJ = 8;
    static constexpr int kTileI = 32 * NI, kTileJ = 32 * NJ;
    static constexpr int H = NI / 2, HJ = NJ / 2;  // products of half a step
    using PSide = Rows<NI, false>;
    using QSide = Rows<NJ, true>;
    static constexpr int kStageBytes = PSide::kBytes + QSide::kBytes;
    static constexpr int kScaleBytes = 2 * Scales::kBytes;         // of both operands
    static constexpr int kOutRow = 256 + 16;       // bytes of a row of results on their way out
    static constexpr int kOutBytes = 16 * kOutRow; // a wave's
    static constexpr int kLds = 2 * (kStageBytes + kScaleBytes) + 4 * kOutBytes;
    // scales of B that a lane needs: a wave's 128 rows are one square's, this step's and the next
    static constexpr int NQ = SQUARE ? 2 : NJ;

    PSide p;
    QSide q;
    Scales pe, qe;
    int wave;
    uint32_t smem, scales;                         // LDS: the stages, the scales
    int pair_left;                                 // of the two stages to come those that there are
    uint32_t stage0;                               // the first of them
    uint32_t ps[NI], qs[NQ];                       // scales, each half read when the last step's has been used
    v8i a[NJ], b[NI];

    __device__ __forceinline__ Tile(ArgsAt t, uint32_t lds) : smem(lds), scales(lds + 2 * kStageBytes)
    {
        const int lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        p.lanes((int)t->a_ld, wave, lane);
        q.lanes((int)t->b_ld, wave, lane);
        p.reader(smem, (wave >> 1) * 16 * NI, lane);
        q.reader(smem + PSide::kBytes, (wave & 1) * 128, lane);
    }
    // For every wave: what it has to have read of LDS it has, and its loads but the last LEFT have arrived.
    template <int LEFT>
    static __device__ __forceinline__ void turn()
    {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(wait_for(LEFT));      // (the builtin: the compiler counts on it)
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    }
    static constexpr int kStageLoads = NI + NJ;          // a wave's, of a stage
    static constexpr int kStores = 4 * NI;               // a wave's, of a whole tile, at least
    // Scales of 2 steps, of an even or an odd pair.
    __device__ __forceinline__ void issue_scales(int pair)
    {
        const uint32_t to = scales + (pair & 1) * kScaleBytes;
        pe.issue(to, wave);
        qe.issue(to + Scales::kBytes, wave);
    }
    static __device__ __forceinline__ uint32_t byte_at(uint32_t at) { return *(ZO_LDS const uint8_t*)(uintptr_t)at; }
    __device__ __forceinline__ int row_i() const { return (wave >> 1) * 16 * NI + (threadIdx.x & 15); }
    __device__ __forceinline__ int row_j() const
    {
        const int r = threadIdx.x & 15;
        return SQUARE ? (wave & 1) : (wave & 1) * 128 + (r >> 2) * 16 + (r & 3);
    }
    // Of step s (at parity F) those of half I of A's rows, and of half J of B's.
    template <int I>
    __device__ __forceinline__ void read_ps(int s)
    {
        const uint32_t at = pe.at(scales + ((s >> 1) & 1) * kScaleBytes, row_i(), s);
#pragma unroll
        for (int k = I * H; k < (I + 1) * H; ++k) ps[k] = byte_at(at + k * 64);
    }
    template <int F, int J>
    __device__ __forceinline__ void read_qs(int s)
    {
        if (SQUARE && J == 1) return;
        const uint32_t at = qe.at(scales + ((s >> 1) & 1) * kScaleBytes + Scales::kBytes, row_j(), s);
        if constexpr (SQUARE) {
            qs[F] = byte_at(at);
        } else {
#pragma unroll
            for (int k = J * HJ; k < (J + 1) * HJ; ++k) qs[k] = byte_at(at + (k >> 2) * 256 + (k & 3) * 16);
        }
    }
    // Steps go in pairs, the first of a pair through the first stage; of an odd count the first is the
    // second of its pair.
    //
    // On to the tile at (i0, j0), `steps` blocks from b0 on: its scales are loaded, of its codes the first
    // two stages by begin_loads.  The second of a single step is zeros.
    __device__ __forceinline__ void begin(ArgsAt t, int64_t i0, int64_t j0, int b0, int steps)
    {
        const int depth = (int)t->depth - b0 * kBlock, blocks = t->blocks - b0, back = steps & 1;
        const int i = least_of(t->rows - i0, kTileI), j = least_of(t->cols - j0, kTileJ);
        p.begin(t->a + i0 * t->a_ld + b0 * kBlock, (int)t->a_ld, i, depth);
        q.begin(t->b + j0 * t->b_ld + b0 * kBlock, (int)t->b_ld, j, depth);
        pe.begin(t->a_exps + i0 * t->a_exps_ld + b0, (int)t->a_exps_ld, i, blocks, back, wave, row_i());
        const uint8_t* x = t->b_exps + (SQUARE ? j0 >> 7 : j0) * t->b_exps_ld + b0;
        qe.begin(x, (int)t->b_exps_ld, SQUARE ? (j > 128 ? 2 : 1) : j, blocks, back, wave, row_j());
        issue_scales(0);
        issue_scales(1);
        pair_left = steps > 1 ? 2 : 1;
        stage0 = back ? kStageBytes : 0;
    }
    // No tile: the loads of the next two stages bring zeros.
    __device__ __forceinline__ void begin_none()
    {
        p.left = q.left = 0;
        pair_left = 0;
        stage0 = 0;
    }
    __device__ __forceinline__ typename PSide::Loads begin_p(int n)
    {
        if (n >= pair_left) p.left = 0;
        return p.next(smem + (n ? kStageBytes - stage0 : stage0), wave);
    }
    __device__ __forceinline__ typename QSide::Loads begin_q(int n)
    {
        if (n >= pair_left) q.left = 0;
        return q.next(smem + (n ? kStageBytes - stage0 : stage0) + PSide::kBytes, wave);
    }
    // The n-th of the two stages.
    __device__ __forceinline__ void begin_loads(int n)
    {
        const auto lp = begin_p(n);
        const auto lq = begin_q(n);
#pragma unroll
        for (int k = 0; k < NI; ++k) lp.issue(k);
#pragma unroll
        for (int k = 0; k < NJ; ++k) lq.issue(k);
    }
    // Of the second stage, the last step's: the codes behind the depth's end, in the chunk that it ends
    // in, are other rows'.  Zeros instead.  (Both sides: 0 times NaN is none.)
    __device__ __forceinline__ void cut()
    {
        const int depth = (int)args_at()->depth;
        const int chunk = ((depth - 1) & (kBlock - 1)) >> 4, tail = depth & 15;
#pragma nounroll
        for (int row = threadIdx.x; row < kTileI + kTileJ; row += kThreads) {
            const bool second = row >= kTileI;
            const int r = second ? row - kTileI : row;
            const int key = second ? QSide::key(r) : PSide::key(r);
            ZO_LDS u4* to = (ZO_LDS u4*)(uintptr_t)(smem + kStageBytes + (second ? PSide::kBytes : 0) + r * 128 + ((chunk ^ key) << 4));
            u4 v = *to;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int keep = tail - 4 * k;             // bytes of this word
                v[k] = keep >= 4 ? v[k] : keep <= 0 ? 0 : v[k] & ((1u << (8 * keep)) - 1);
            }
            *to = v;
        }
        __syncthreads();
    }
    // A quarter of a step: rows half J of B by half I of A, and between its products `read` of 0 to 3.
    // The instruction is written out because its sums have to stay where they are: the
    // builtin's result may go to other registers, and with 256 of 512 of them sums the compiler
    // moves 100 a step.  (What it reads has been written by an s_nop 1 before at least; what it
    // writes is read by the next step's products, and by `settled`.)
    template <int F, int J, int I, typename R, typename L>
    __device__ __forceinline__ void multiply(f4 (&acc)[NI][NJ], R read, L load)
    {
#pragma unroll
        for (int j = 0; j < HJ; ++j) {
            read(j);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                asm volatile("s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0]"
                             : "+a"(acc[I * H + i][J * HJ + j])
                             : "v"(a[J * HJ + j]), "v"(b[I * H + i]), "v"(qs[SQUARE ? F : J * HJ + j]), "v"(ps[I * H + i]));
                load(j * H + i);
            }
        }
    }
    // Of n loads those that follow the k-th of a quarter's products.
    template <typename Loads>
    static __device__ __forceinline__ void spread(const Loads& l, int n, int k)
    {
#pragma unroll
        for (int q = n * k / (H * HJ); q < n * (k + 1) / (H * HJ); ++q) l.issue(q);
    }
    // The sums can be read: an instruction of 16 passes writes its last 18 wait states on.
    static __device__ __forceinline__ void settled(f4 (&acc)[NI][NJ])
    {
        asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) asm volatile("" : "+a"(acc[i][j]));
    }
    template <int J>
    __device__ __forceinline__ void read_a(uint32_t stage, int k)
    {
        a[J * HJ + k] = q.get(stage, J * HJ + k);
    }
    template <int I>
    __device__ __forceinline__ void read_b(uint32_t stage, int k)
    {
        if (k < H) b[I * H + k] = p.get(stage, I * H + k);
    }
    // What the first step, at parity F, begins with.
    template <int F>
    __device__ __forceinline__ void first(int s)
    {
        constexpr uint32_t stage = F ? kStageBytes : 0;
#pragma unroll
        for (int k = 0; k < HJ; ++k) read_a<0>(stage, k);
#pragma unroll
        for (int k = 0; k < H; ++k) read_b<F>(stage, k);
        read_ps<F>(s);
        read_qs<F, 0>(s);
    }
    // A step, in quarters.  Each is multiplied while what the next one lacks is read: first what the
    // step has, then its other half of A's rows, then of B's; behind the second barrier the next step's
    // first halves, each into registers that the quarter before has freed.  So the halves of A's
    // rows change places from step to step (F, the stage too).
    //
    // MORE: there are two steps more.  A's piece of the one after next is loaded during the second
    // quarter, when all have read this stage's, B's during the third.  The loads go between the products: a
    // wave that has its SIMD to itself waits for 8 loads in a row to be taken (512 cycles) while
    // nothing is multiplied.
    template <int F, bool MORE, typename B>
    __device__ __forceinline__ void half_step(int s, f4 (&acc)[NI][NJ], B behind)
    {
        constexpr uint32_t stage = F ? kStageBytes : 0;
        read_ps<1 - F>(s);
        multiply<F, 0, F>(acc, [&](int k) { read_b<1 - F>(stage, k); }, [](int) {});
        if constexpr (MORE) {
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(kLgkmDone);
            asm volatile("s_barrier" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            const auto loads = p.next(smem + stage, wave);
            read_qs<F, 1>(s);
            multiply<F, 0, 1 - F>(acc, [&](int k) { read_a<1>(stage, k); }, [&](int k) { spread(loads, NI, k); });
            turn<NI>();
        } else {
            read_qs<F, 1>(s);
            multiply<F, 0, 1 - F>(acc, [&](int k) { read_a<1>(stage, k); }, [](int) {});
            turn<0>();
        }
        behind();
    }
    template <int F, bool MORE>
    __device__ __forceinline__ void other_half(int s, f4 (&acc)[NI][NJ])
    {
        constexpr uint32_t stage = F ? kStageBytes : 0, other = kStageBytes - stage;
        read_qs<1 - F, 0>(s + 1);
        if constexpr (MORE) {
            const auto loads = q.next(smem + stage + PSide::kBytes, wave);
            multiply<F, 1, 1 - F>(acc, [&](int k) { read_a<0>(other, k); }, [&](int k) { spread(loads, NJ, k); });
        } else {
            multiply<F, 1, 1 - F>(acc, [&](int k) { read_a<0>(other, k); }, [](int) {});
        }
        read_ps<1 - F>(s + 1);
        multiply<F, 1, F>(acc, [&](int k) { read_b<1 - F>(other, k); }, [](int) {});
    }
    // acc[ti][tj][e]: i = row_of(ti), j = column_of(tj) + e, within the tile, begun with what the sums begin with.
    // `ends` says whether the last step is cut, `stored` that a whole tile's results have been stored since
    // begin_loads().  `next` begins the next tile (or none) when this one's stages have been read.
    // (No branch within the steps that repeat: with one the compiler keeps fewer sums in place.)
    template <typename N>
    __device__ __forceinline__ void run(int steps, bool ends, bool stored, f4 (&acc)[NI][NJ], N next)
    {
        // (the first stage; the second, and the stores, may still be under way)
        if (stored) turn<kStageLoads + kStores>();
        else turn<kStageLoads>();
        const int back = steps & 1, pairs = (steps + 1) / 2;
        int pair = back;
        if (back) {
            if (ends && steps == 1) cut();
            first<1>(1);
            if (steps > 1) {
                half_step<1, true>(1, acc, [&] { issue_scales(0); });
                other_half<1, true>(1, acc);
            }
        } else {
            first<0>(0);
        }
        for (; pair + 1 < pairs; ++pair) {
            half_step<0, true>(2 * pair, acc, [] {});
            other_half<0, true>(2 * pair, acc);
            half_step<1, true>(2 * pair + 1, acc, [&] { issue_scales(pair); });      // (of the pair two on)
            other_half<1, true>(2 * pair + 1, acc);
        }
        if (steps > 1) {
            half_step<0, false>(2 * pair, acc, [&] {
                if (ends) cut();
            });
            other_half<0, false>(2 * pair, acc);
        }
        half_step<1, false>(steps > 1 ? 2 * pair + 1 : 1, acc, next);
        // the last two quarters, and the next tile's first two stages
        {
            const auto lp = begin_p(0);
            const auto lq = begin_q(0);
            multiply<1, 1, 0>(acc, [](int) {}, [&](int k) {
                spread(lp, NI, k);
                spread(lq, NJ, k);
            });
        }
        {
            const auto lp = begin_p(1);
            const auto lq = begin_q(1);
            multiply<1, 1, 1>(acc, [](int) {}, [&](int k) {
                spread(lp, NI, k);
                spread(lq, NJ, k);
            });
        }
        settled(acc);
    }
    static __device__ __forceinline__ int column_of(int tj, int wave, int lane) { return (wave & 1) * 128 + (tj >> 2) * 64 + (lane >> 4) * 16 + (tj & 3) * 4; }
    static __device__ __forceinline__ int row_of(int ti, int wave, int lane) { return (wave >> 1) * 16 * NI + ti * 16 + (lane & 15); }
};

// A wave's results, 16 rows at a time through LDS at `room`, to be written in runs of 256 bytes: to the element
// `to` of the wave's first row and column, `rows` and `cols` of which there are from there on (WHOLE: all).
template <bool WHOLE, typename O, int NI, bool SQUARE>
__device__ __forceinline__ void put_tile(O* to, int64_t ld, int rows, int cols, uint32_t room, f4 (&acc)[NI][8])
{
    using G = Tile<NI, SQUARE>;
    constexpr int W = 16 / sizeof(O), RUNS = 4 / sizeof(O);        // runs of 64 columns in 256 bytes
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));      // (addresses are made here, and not kept in registers over the products)
    const uint32_t in = room + (lane & 15) * G::kOutRow + (lane >> 4) * 16 * sizeof(O);
    const uint32_t out = room + (lane >> 4) * G::kOutRow + (lane & 15) * 16;
    to += (lane >> 4) * ld + (lane & 15) * W;
    cols -= (lane & 15) * W;
    rows -= lane >> 4;
#pragma unroll
    for (int ti = 0; ti < NI; ++ti)
#pragma unroll
        for (int part = 0; part < 2 / RUNS; ++part) {
            // (what follows is not done ahead, for all rows at once)
#pragma unroll
            for (int k = 0; k < 4 * RUNS; ++k) asm volatile("" : "+a"(acc[ti][part * RUNS * 4 + k]));
#pragma unroll
            for (int run = 0; run < RUNS; ++run)
#pragma unroll
                for (int q = 0; q < 16 / W; ++q) {
                    vec_t<O, W> y;
#pragma unroll
                    for (int e = 0; e < W; ++e) y[e] = static_cast<O>(acc[ti][(part * RUNS + run) * 4 + ((q * W + e) >> 2)][e & 3]);
                    *(ZO_LDS u4*)(uintptr_t)(in + run * 128 + q * 16) = __builtin_bit_cast(u4, y);
                }
            asm volatile("" ::: "memory");         // (LDS takes a wave's accesses in their order)
            if constexpr (WHOLE) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    store_vec<O, W>(to + (ti * 16 + k * 4) * ld + part * 64,
                                    __builtin_bit_cast(vec_t<O, W>, *(ZO_LDS const u4*)(uintptr_t)(out + k * 4 * G::kOutRow)));
            } else {
                const int left = cols - part * 64;
#pragma nounroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t at = out + k * 4 * G::kOutRow;
                    O* p = to + (ti * 16 + k * 4) * ld + part * 64;
                    if (ti * 16 + k * 4 >= rows) continue;
                    if (left >= W) {
                        store_vec<O, W>(p, __builtin_bit_cast(vec_t<O, W>, *(ZO_LDS const u4*)(uintptr_t)at));
                    } else {
#pragma nounroll
                        for (int e = 0; e < left; ++e) p[e] = *(ZO_LDS const O*)(uintptr_t)(at + e * sizeof(O));
                    }
                }
            }
            asm volatile("" ::: "memory");
        }
}

template <typename O, int NI, bool SQUARE>
__device__ __forceinline__ void put_tile(O* to, int64_t ld, int rows, int cols, uint32_t room, f4 (&acc)[NI][8])
{
    if (rows == 16 * NI && cols == 128) put_tile<true, O, NI, SQUARE>(to, ld, rows, cols, room, acc);
    else put_tile<false, O, NI, SQUARE>(to, ld, rows, cols, room, acc);
}

__device__ __forceinline__ uint32_t lds_address(char* smem) { return (uint32_t)(uintptr_t)(ZO_LDS char*)smem; }

// A die's workgroups walk its tiles (each tile once for every split of the depth), and load the
// next while they store a tile's results.
template <typename T, int NI, bool SQUARE>
__global__ __launch_bounds__(kThreads, 1) void tile_kernel(TileArgs)
{
    using G = Tile<NI, SQUARE>;
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    const uint32_t lds = lds_address(smem);
    uint32_t at, mine, stride, n0;             // of the die's tiles: the next, all, to the one after; the first
    {
        const ArgsAt t = args_at();
        const uint32_t all = t->ti * t->tj * t->splits;
        const uint32_t die = blockIdx.x % kDies, q = all / kDies, r = all % kDies;
        mine = q + (die < r ? 1 : 0);
        n0 = die * q + (die < r ? die : r);
        stride = (gridDim.x + kDies - 1 - die) / kDies;        // workgroups of the die
        at = blockIdx.x / kDies;
    }
    if (at >= mine) return;
    G g(args_at(), lds);
    uint32_t bi = 0, bj = 0;
    int split = 0, steps = 0;
    bool ends = false, stored = false;
    auto place = [&] {
        const ArgsAt t = args_at();
        // (a die's share of all splits' tiles, one split after the other)
        uint32_t n = n0 + at;
        split = 0;
        if (t->splits > 1) {
            const uint32_t tiles = t->ti * t->tj;
            split = __builtin_amdgcn_readfirstlane(n / tiles);
            n -= (uint32_t)split * tiles;
        }
        tile_at(n, t->ti, t->tj, bi, bj);
        const int b0 = (int)((int64_t)t->blocks * split / t->splits);
        steps = (int)((int64_t)t->blocks * (split + 1) / t->splits) - b0;
        ends = b0 + steps == t->blocks && (t->depth & 15) != 0;
        g.begin(t, (int64_t)bi * G::kTileI, (int64_t)bj * G::kTileJ, b0, steps);
    };
    place();
    g.begin_loads(0);
    g.begin_loads(1);
    const int lane = threadIdx.x & 63;
    for (;;) {
        // this tile; place() goes on to the next
        const int64_t i = (int64_t)bi * G::kTileI, j = (int64_t)bj * G::kTileJ;
        const int now = steps, part = split;
        f4 acc[NI][8];
        {
            float first[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) first[k] = 0.0f;
            const ArgsAt t = args_at();
            if (t->bias != nullptr && t->part == nullptr) {
                const T* bias = static_cast<const T*>(t->bias) + j + G::column_of(0, g.wave, lane);
                const int left = least_of(t->cols - j, G::kTileJ) - G::column_of(0, g.wave, lane);
#pragma unroll
                for (int k = 0; k < 32; ++k) first[k] = (k >> 4) * 64 + (k & 15) < left ? (float)bias[(k >> 4) * 64 + (k & 15)] : 0.0f;
            }
#pragma unroll
            for (int ti = 0; ti < NI; ++ti)
#pragma unroll
                for (int tj = 0; tj < 8; ++tj)
                    acc[ti][tj] = f4{first[(tj >> 2) * 16 + (tj & 3) * 4], first[(tj >> 2) * 16 + (tj & 3) * 4 + 1],
                                     first[(tj >> 2) * 16 + (tj & 3) * 4 + 2], first[(tj >> 2) * 16 + (tj & 3) * 4 + 3]};
        }
        at += stride;
        g.run(now, ends, stored, acc, [&] {
            if (at < mine) place();
            else g.begin_none();
        });
        {
            const ArgsAt t = args_at();
            const int64_t i1 = i + (g.wave >> 1) * 16 * NI, j1 = j + (g.wave & 1) * 128;
            const int rows = least_of(t->rows - i1, 16 * NI), cols = least_of(t->cols - j1, 128);
            const uint32_t room = lds + 2 * (G::kStageBytes + G::kScaleBytes) + g.wave * G::kOutBytes;
            if (t->part != nullptr) put_tile<float, NI, SQUARE>(t->part + (part * t->rows + i1) * t->cols + j1, t->cols, rows, cols, room, acc);
            else put_tile<T, NI, SQUARE>(static_cast<T*>(t->out) + i1 * t->out_ld + j1, t->out_ld, rows, cols, room, acc);
            stored = rows == 16 * NI && cols == 128;
        }
        if (at >= mine) break;
    }
    // (zeros on their way to LDS)
    __builtin_amdgcn_s_waitcnt(wait_for(0));
}

// The parts of a split product, added in the order of the splits: W results a lane.
template <typename T, int W>
__global__ __launch_bounds__(256) void join_parts_kernel(const float* part, int splits, int64_t rows, int64_t cols, const T* bias, T* out,
                                                         int64_t out_ld, int64_t first)
{
    const int64_t all = rows * cols, at = ((first + blockIdx.x) * 256 + threadIdx.x) * W;
    if (at >= all) return;
    const int64_t i = at / cols, j = at - i * cols;
    float s[W];
#pragma unroll
    for (int e = 0; e < W; ++e) s[e] = bias != nullptr ? (float)bias[j + e] : 0.0f;
#pragma unroll 8
    for (int k = 0; k < splits; ++k) {
        const vec_t<float, W> x = *reinterpret_cast<const vec_t<float, W>*>(part + k * all + at);
#pragma unroll
        for (int e = 0; e < W; ++e) s[e] += x[e];
    }
    vec_t<T, W> y;
#pragma unroll
    for (int e = 0; e < W; ++e) y[e] = static_cast<T>(s[e]);
    store_vec<T, W>(out + i * out_ld + j, y);
}

// Codes whose rows cannot be loaded as they lie, to rows of ld (a multiple of 16) with zeros
// behind the depth: of one array or, from workgroup `first` on, of another.
struct Recode {
    const uint8_t* x;
    uint8_t* out;
    int64_t stride, rows;
};

__global__ __launch_bounds__(256) void recode_kernel(Recode a, Recode b, int64_t base, int64_t first, int64_t depth, int64_t ld)
{
    const int64_t group = base + blockIdx.x;
    const bool second = group >= first;
    const Recode r = second ? b : a;
    const int64_t at = ((group - (second ? first : 0)) * 256 + threadIdx.x) * 16;
    if (at >= r.rows * ld) return;
    const int64_t i = at / ld, c = at - i * ld;
    const uint8_t* x = r.x + i * r.stride + c;
    uint32_t v[4] = {0, 0, 0, 0};
    if (c + 16 <= depth) {
        __builtin_memcpy(v, x, 16);
    } else {
#pragma unroll
        for (int k = 0; k < 16; ++k)
            if (c + k < depth) v[k / 4] |= (uint32_t)x[k] << (8 * (k % 4));
    }
    *reinterpret_cast<uint4*>(r.out + at) = make_uint4(v[0], v[1], v[2], v[3]);
}

// ------------------------------------------------------------------ fp32 results
//
// The 8-bit instructions align 8 products at a time to the largest of them and keep 13 bits
// below it (measured: 1.3e-5 of a result's size in the mean, 2^-15.5 at most of the absolute sum).
// Of a 2-byte result that is a hundredth or a tenth of its rounding, of one in fp32 a hundred
// times its own; so those are summed by bf16 instructions, whose products are exact.  The operands'
// values, which bf16 holds, are written out first: 3 bytes a code in 5 TB/s, against the
// products' 2 operations for each of 256 results it meets.  4801 x 1601 x 4099: 21 us for the values,
// 106 for the product under a profiler (call after call 117 in all); its 182 tiles of 192 rows are one round of
// the 256 CUs, of which 74 have none.

struct ExactArgs {
    Operand a, b;
    float* out;                // fp32 results; of a split [split][rows][cols]
    const float* bias;
    int64_t rows, cols, out_ld, split_ld;
    uint32_t ti, tj;
    int64_t steps;             // of the whole depth
    int splits;
};

template <int NI, int NJ>
__global__ __launch_bounds__(kGemmThreads, 2) void exact_kernel(ExactArgs t, int64_t first)
{
    using G = Gemm<__bf16, kInner, kInner, NI, NJ>;
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    const uint32_t tiles = t.ti * t.tj, id = (uint32_t)first + blockIdx.x;
    const int64_t split = __builtin_amdgcn_readfirstlane(id / tiles);
    uint32_t bi, bj;
    tile_of(id % tiles, tiles, t.ti, t.tj, bi, bj);
    const int64_t s0 = t.steps * split / t.splits, s1 = t.steps * (split + 1) / t.splits;
    f4 acc[NI][NJ];
    G g(t.a, t.b, lds_address(smem));
    g.begin(t.a, t.b, (int64_t)bi * G::kTileI, (int64_t)bj * G::kTileJ, s0 * kDeep, (int)(s1 - s0));
    g.run((int)(s1 - s0), acc, [] {});
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int ti = 0; ti < NI; ++ti) {
        const int64_t i = (int64_t)bi * G::kTileI + G::row_of(ti, wave, lane);
        if (i >= t.rows) continue;
        float* to = t.out + split * t.split_ld + i * t.out_ld;
#pragma unroll
        for (int tj = 0; tj < NJ; ++tj) {
            const int64_t j = (int64_t)bj * G::kTileJ + G::column_of(tj, wave, lane);
            f4 y = acc[ti][tj];
            if (t.bias != nullptr) {
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] += j + e < t.cols ? t.bias[j + e] : 0.0f;
            }
            if (j + 4 <= t.cols) {
                store_vec<float, 4>(to + j, y);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (j + e < t.cols) to[j + e] = y[e];
            }
        }
    }
}

// ------------------------------------------------------------------ few rows

struct FewArgs {
    const uint8_t* a;
    const uint8_t* b;
    const uint8_t* a_exps;
    const uint8_t* b_exps;
    int64_t a_ld, b_ld, a_exps_ld, b_exps_ld;
    int64_t rows, cols, depth, out_ld;
    const void* bias;
    void* out;
    int waves;                 // of a workgroup
    int square;
};

// A lane's 32 codes of block s of a row; zeros behind the depth.
__device__ __forceinline__ v8i codes_at(const uint8_t* row, int64_t k, int64_t depth)
{
    v8i v;
    if (k + 32 <= depth) {
        __builtin_memcpy(&v, row + k, 32);
        return v;
    }
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        uint32_t x = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (k + 4 * w + e < depth) x |= (uint32_t)row[k + 4 * w + e] << (8 * e);
        v[w] = (int)x;
    }
    return v;
}

// The codes' products with their scales, added to c: in 8 bits, or exactly, as bf16 (a quarter of the
// depth at a time).
template <bool EXACT>
__device__ __forceinline__ f4 product_of(const v8i& a, const v8i& b, f4 c, uint32_t scale_a, uint32_t scale_b)
{
    if constexpr (!EXACT) {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, (int)scale_a, 0, (int)scale_b);
    } else {
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
        const float sa = scale_value(scale_a), sb = scale_value(scale_b);
        auto part = [](const v8i& x, int q, float s) {
            const b2 v[4] = {
                __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * q], s, false), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * q], s, true),
                __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * q + 1], s, false), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * q + 1], s, true)};
            s8 y;
            __builtin_memcpy(&y, v, 16);
            return y;
        };
#pragma unroll
        for (int q = 0; q < 4; ++q) c = Mfma<__bf16>::run(part(a, q, sa), part(b, q, sb), c);
        return c;
    }
}

// 16 rows of B and 16 MT of A.  Wave w takes blocks w, w + waves, ...
template <typename T, int MT>
__global__ __launch_bounds__(1024) void few_kernel(FewArgs f, int64_t first)
{
    constexpr bool EXACT = std::is_same<T, float>::value;
    __shared__ float sums[16][MT][16][17];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t n0 = (first + blockIdx.x) * 16;
    const int64_t n = n0 + r < f.cols ? n0 + r : f.cols - 1;
    const uint8_t* b = f.b + n * f.b_ld;
    const uint8_t* be = f.b_exps + (f.square ? n / kBlock : n) * f.b_exps_ld;
    const uint8_t* a[MT];
    const uint8_t* ae[MT];
    f4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int64_t m = t * 16 + r < f.rows ? t * 16 + r : f.rows - 1;
        a[t] = f.a + m * f.a_ld;
        ae[t] = f.a_exps + m * f.a_exps_ld;
        acc[t] = f4{0, 0, 0, 0};
    }
    const int whole = (int)(f.depth / kBlock), blocks = (int)ceil_div(f.depth, kBlock);
    // U blocks at a time, all of their loads under way before the first product
    auto blocks_from = [&](int s, auto count) {
        constexpr int U = decltype(count)::value;
        v8i x[U], y[U][MT];
        uint32_t sx[U], sy[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t at = s + u * f.waves;
            __builtin_memcpy(&x[u], b + at * kBlock + g * 32, 32);
            sx[u] = be[at];
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                __builtin_memcpy(&y[u][t], a[t] + at * kBlock + g * 32, 32);
                sy[u][t] = ae[t][at];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int t = 0; t < MT; ++t) acc[t] = product_of<EXACT>(x[u], y[u][t], acc[t], sx[u], sy[u][t]);
    };
    constexpr int U = MT == 1 ? 4 : 2;
    int s = wave;
    for (; s + (U - 1) * f.waves < whole; s += U * f.waves) blocks_from(s, std::integral_constant<int, U>{});
    for (; s < whole; s += f.waves) blocks_from(s, std::integral_constant<int, 1>{});
    if (blocks > whole && wave == whole % f.waves) {
        const int64_t k = (int64_t)whole * kBlock + g * 32;
        const v8i x = codes_at(b, k, f.depth);
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[t] = product_of<EXACT>(x, codes_at(a[t], k, f.depth), acc[t], be[whole], ae[t][whole]);
    }
    // a lane: column (of A's rows) r, results 4 g to 4 g + 3 of B's rows
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sums[wave][t][r][4 * g + e] = acc[t][e];
    __syncthreads();
    for (int k = threadIdx.x; k < MT * 256; k += f.waves * 64) {
        const int64_t m = k >> 4, j = n0 + (k & 15);
        if (m >= f.rows || j >= f.cols) continue;
        float s = 0.0f;
        for (int w = 0; w < f.waves; ++w) s += sums[w][m >> 4][m & 15][k & 15];
        if (f.bias != nullptr) s += (float)static_cast<const T*>(f.bias)[j];
        static_cast<T*>(f.out)[m * f.out_ld + j] = static_cast<T>(s);
    }
}

// ------------------------------------------------------------------ launches

// Rows up to which B may go straight to registers.
constexpr int64_t kFewRows = 32;

template <typename K>
hipError_t allow(K kernel, int lds)
{
    return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
}

// LDS of a CU.
constexpr int kCuLds = 160 << 10;

template <typename T, int NI, bool SQUARE>
hipError_t tiles(TileArgs t, hipStream_t s)
{
    using G = Tile<NI, SQUARE>;
    static_assert(product_tiles_in_cu(false, NI) == kCuLds / G::kLds, "a launch and its plan count the same workgroups to a CU");
    static const hipError_t allowed = allow(tile_kernel<T, NI, SQUARE>, G::kLds);
    if (allowed != hipSuccess) return allowed;
    t.ti = (uint32_t)ceil_div(t.rows, G::kTileI);
    t.tj = (uint32_t)ceil_div(t.cols, G::kTileJ);
    const int64_t all = (int64_t)t.ti * t.tj * t.splits, stand = kCUs * product_tiles_in_cu(false, NI);
    tile_kernel<T, NI, SQUARE><<<dim3((unsigned)(all < stand ? all : stand)), kThreads, G::kLds, s>>>(t);
    return hipSuccess;
}

template <typename T, int NI>
hipError_t tiles(const TileArgs& t, bool square, hipStream_t s)
{
    return square ? tiles<T, NI, true>(t, s) : tiles<T, NI, false>(t, s);
}

// What the tiles' loads need of an address and a row stride.
bool loads_as_it_is(const void* p, int64_t stride)
{
    return (reinterpret_cast<uintptr_t>(p) & 3) == 0 && stride % 4 == 0 && stride <= (1 << 22);
}

template <int NI, int NJ>
hipError_t exact(ExactArgs t, hipStream_t s)
{
    using G = Gemm<__bf16, kInner, kInner, NI, NJ>;
    static_assert(product_tiles_in_cu(true, NI) == kCuLds / G::kLds, "the plan counts the workgroups that a CU holds");
    static const hipError_t allowed = allow(exact_kernel<NI, NJ>, G::kLds);
    if (allowed != hipSuccess) return allowed;
    t.ti = (uint32_t)ceil_div(t.rows, G::kTileI);
    t.tj = (uint32_t)ceil_div(t.cols, G::kTileJ);
    in_launches((int64_t)t.ti * t.tj * t.splits, kGemmThreads, [&](int64_t first, int64_t count) {
        exact_kernel<NI, NJ><<<dim3((unsigned)count), kGemmThreads, G::kLds, s>>>(t, first);
    });
    return hipSuccess;
}

// fp32 results: the operands' values in bf16, and their product.
hipError_t exact(const ScaledProduct& a, const ProductPlan& p, float* part, hipStream_t s)
{
    void* wide_a = a.space + p.off_a;
    void* wide_b = a.space + p.off_b;
    hipError_t e = scaled_unpack(ScaledUnpack{a.a, a.a_exps, wide_a, p.m, p.k, a.a_stride, a.a_exps_stride, p.k_ld, p.k_ld, 0, false}, 2, s);
    if (e == hipSuccess) e = scaled_unpack(ScaledUnpack{a.b, a.b_exps, wide_b, p.n, p.k, a.b_stride, a.b_exps_stride, p.k_ld, p.k_ld, 0, a.square}, 2, s);
    if (e != hipSuccess) return e;
    ExactArgs t{};
    t.a = Operand{wide_a, p.k_ld, p.m, p.k_ld};
    t.b = Operand{wide_b, p.k_ld, p.n, p.k_ld};
    t.rows = p.m;
    t.cols = p.n;
    t.steps = ceil_div(p.k_ld, kDeep);
    t.splits = p.splits;
    t.out = p.splits > 1 ? part : static_cast<float*>(a.out);
    t.out_ld = p.splits > 1 ? p.n : a.out_stride;
    t.split_ld = p.m * p.n;
    t.bias = p.splits > 1 ? nullptr : static_cast<const float*>(a.bias);
    return p.ni == 8 ? exact<8, 4>(t, s) : p.ni == 6 ? exact<6, 4>(t, s) : exact<2, 4>(t, s);
}

template <typename T>
hipError_t product(const ScaledProduct& a, const ProductPlan& p, hipStream_t s)
{
    if (p.m == 0 || p.n == 0) return hipSuccess;
    float* part = reinterpret_cast<float*>(a.space + p.off_part);
    auto join = [&](int splits) {
        const T* bias = static_cast<const T*>(a.bias);
        T* out = static_cast<T*>(a.out);
        const int wide = p.n % 4 == 0 ? 4 : 1;
        in_launches(ceil_div(p.m * p.n, 256 * wide), 256, [&](int64_t first, int64_t count) {
            if (wide == 4) join_parts_kernel<T, 4><<<dim3((unsigned)count), 256, 0, s>>>(part, splits, p.m, p.n, bias, out, a.out_stride, first);
            else join_parts_kernel<T, 1><<<dim3((unsigned)count), 256, 0, s>>>(part, splits, p.m, p.n, bias, out, a.out_stride, first);
        });
    };
    if (p.k == 0) {                            // a sum of nothing
        join(0);
        return hipGetLastError();
    }
    // (of few rows also what the tiles would have to copy first: bytes at any address are loaded here)
    const bool as_it_is = loads_as_it_is(a.a, a.a_stride) && loads_as_it_is(a.b, a.b_stride);
    if (p.ni == 0 || (p.m <= kFewRows && !as_it_is)) {
        // waves of a workgroup, which share the depth: as many as find work, up to 16
        int waves = 1;
        while (waves < 16 && waves * 2 <= ceil_div(p.k, kBlock)) waves *= 2;
        const FewArgs f{a.a, a.b, a.a_exps, a.b_exps, a.a_stride, a.b_stride, a.a_exps_stride, a.b_exps_stride, p.m, p.n, p.k, a.out_stride,
                        a.bias, a.out, waves, a.square};
        in_launches(ceil_div(p.n, 16), waves * 64, [&](int64_t first, int64_t count) {
            if (p.m <= 16) few_kernel<T, 1><<<dim3((unsigned)count), waves * 64, 0, s>>>(f, first);
            else few_kernel<T, 2><<<dim3((unsigned)count), waves * 64, 0, s>>>(f, first);
        });
        return hipGetLastError();
    }
    if constexpr (std::is_same<T, float>::value) {
        const hipError_t e = exact(a, p, part, s);
        if (e == hipSuccess && p.splits > 1) join(p.splits);
        return e != hipSuccess ? e : hipGetLastError();
    } else {
    const uint8_t* ac = a.a;
    const uint8_t* bc = a.b;
    int64_t a_ld = a.a_stride, b_ld = a.b_stride;
    Recode copies[2];
    int many = 0;
    if (!loads_as_it_is(ac, a_ld)) {
        uint8_t* to = reinterpret_cast<uint8_t*>(a.space + p.off_a);
        copies[many++] = Recode{ac, to, a_ld, p.m};
        ac = to;
        a_ld = p.k_ld;
    }
    if (!loads_as_it_is(bc, b_ld)) {
        uint8_t* to = reinterpret_cast<uint8_t*>(a.space + p.off_b);
        copies[many++] = Recode{bc, to, b_ld, p.n};
        bc = to;
        b_ld = p.k_ld;
    }
    if (many > 0) {
        const int64_t first = ceil_div(copies[0].rows * p.k_ld, 4096);
        const int64_t all = first + (many > 1 ? ceil_div(copies[1].rows * p.k_ld, 4096) : 0);
        in_launches(all, 256, [&](int64_t base, int64_t count) {
            recode_kernel<<<dim3((unsigned)count), 256, 0, s>>>(copies[0], copies[many - 1], base, first, p.k, p.k_ld);
        });
    }
    TileArgs t{};
    t.a = ac;
    t.b = bc;
    t.a_ld = a_ld;
    t.b_ld = b_ld;
    t.depth = p.k;
    t.a_exps = a.a_exps;
    t.b_exps = a.b_exps;
    t.a_exps_ld = a.a_exps_stride;
    t.b_exps_ld = a.b_exps_stride;
    t.blocks = (int)ceil_div(p.k, kBlock);
    t.out = a.out;
    t.bias = a.bias;
    t.part = p.splits > 1 ? part : nullptr;
    t.rows = p.m;
    t.cols = p.n;
    t.out_ld = a.out_stride;
    t.splits = p.splits;
    hipError_t e = p.ni == 8 ? tiles<T, 8>(t, a.square, s) : p.ni == 4 ? tiles<T, 4>(t, a.square, s) : tiles<T, 2>(t, a.square, s);
    if (e != hipSuccess) return e;
    if (p.splits > 1) join(p.splits);
    return hipGetLastError();
    }
}

}  // namespace

ProductPlan product_plan(int64_t m, int64_t n, int64_t k, int type)
{
    ProductPlan p{};
    p.m = m;
    p.n = n;
    p.k = k;
    p.k_ld = round_up(k, 16);
    const int64_t blocks = ceil_div(k, kBlock);
    // The tile and the parts of the depth by what they should take, in us: a step of 256 x 256 x 128 1.2,
    // of 128 rows 0.71, of 64 0.66, a round's beginning and end 9, 4 and 3 (measured: 8192 x 1600 x 1600 30.2, 32.9 and
    // 49.5; 1024 x 6400 x 1600 26.1, 18.4 and 28.2; 512 x 6400 x 1600 24.7, 16.5 and 13.5); in bf16 2.8, of 192 rows
    // 2.2, of 64, two to a CU, 1.5 (4801 x 1601 x 4099: 256 rows 146.7, 192, in one round too, 116.6, 64 159.7;
    // 4000 x 4000 x 4000: 142.2, 194.3, 177.3).  Parts go through memory at 6 TB/s, and through a launch of 3 (1600 x
    // 1600 x 8192: 128 rows in two parts 39.4, in one 52.3; 6400 x 1600 x 8192: 256 rows in one 91.8, in two 119.9).
    p.exact = type == 3;
    double best = 0.0;
    p.splits = 1;
    for (int ni = 8; ni >= 2; ni -= 2) {
        if (ni == (p.exact ? 4 : 6)) continue;
        const int64_t tiles = ceil_div(m, 32 * ni) * ceil_div(n, 256), stand = kCUs * product_tiles_in_cu(p.exact, ni);
        const double step = p.exact ? (ni == 8 ? 2.8 : ni == 6 ? 2.2 : 1.5) : ni == 8 ? 1.2 : ni == 4 ? 0.71 : 0.66;
        const double ends = p.exact ? 4.0 : ni == 8 ? 9.0 : ni == 4 ? 4.0 : 3.0;
        const int64_t most = blocks / 2 > 1 ? blocks / 2 : 1;
        for (int64_t c = 1; c <= most && (c == 1 || tiles * c <= 4 * kCUs); ++c) {
            const double t = ceil_div(tiles * c, stand) * (ceil_div(blocks, c) * step + ends) + (c > 1 ? 2.0 * c * m * n * 4 / 6e6 + 3.0 : 0.0);
            if (best == 0.0 || t < best) {
                best = t;
                p.ni = ni;
                p.splits = (int)c;
            }
        }
    }
    // (the operands' values in bf16 first: 3 bytes a code at 5 TB/s, two launches)
    if (p.exact) best += (double)(m + n) * k * 3 / 5e6 + 6.0;
    // Few rows without tiles, where that should take less: what a wave reads of A grows with the rows (a row x 6400 x
    // 1600 10.6 us, 32 rows 10.6, in tiles 13.6; a row x 20480 x 5120 21.9, 32 rows 45, in tiles 25.6).
    if (m <= kFewRows && 8.5 + (double)n * k * 1e-6 * (0.145 + 0.0105 * m) < best + 5.0) {
        p.ni = 0;
        p.bytes = 256;
        return p;
    }
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t off = at;
        at += round_up(bytes, 256);
        return off;
    };
    p.off_part = take(p.splits > 1 ? p.splits * m * n * 4 : 0);
    p.off_a = take(m * p.k_ld * (p.exact ? 2 : 1));
    p.off_b = take(n * p.k_ld * (p.exact ? 2 : 1));
    p.bytes = at > 256 ? at : 256;
    return p;
}

hipError_t scaled_product(const ScaledProduct& a, const ProductPlan& p, int type, hipStream_t s)
{
    return type == 1 ? product<_Float16>(a, p, s) : type == 2 ? product<__bf16>(a, p, s) : product<float>(a, p, s);
}

}  // namespace zo
