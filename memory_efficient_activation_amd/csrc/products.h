// products.h -- the matrix products of the feed-forward operators on gfx950:
// tiles, the loop over them, the kernel for few tokens, operands in padded rows,
// and the choice of tiles.  gated_ffn.hip and linear.hip give them their
// epilogues and launch them.
//
// Every product is written as out[m][n] = sum_k Q(m, k) P(n, k).  The matrix
// cores (v_mfma_f32_16x16x32_bf16, v_mfma_f32_16x16x4_f32) take P as the operand
// whose rows index the four consecutive results a lane holds, so a lane's
// results are consecutive along n.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

#include "act_math.h"
#include "block_common.h"

namespace meblock {

using meswish::Coef;

// Products, by the operands' layout (k or the other dimension contiguous) and
// what they share.
enum Mode {
    kUp = 0,     // k contiguous in both; P two weights, 32 rows of each in turn
    kDx = 1,     // P n contiguous, Q k contiguous; two sums after each other
    kDw = 2,     // both the other way; two products with one P
    kLin = 3,    // as kUp with one weight
    kLinDx = 4,  // as kDx with one sum
    kLinDw = 5   // as kDw with one product
};

template <int MODE>
struct Form {
    static constexpr bool kPK = MODE == kUp || MODE == kLin;      // P's k contiguous
    static constexpr bool kQK = MODE != kDw && MODE != kLinDw;    // Q's k contiguous
    static constexpr bool kTwo = MODE == kUp;                     // P two weights
    static constexpr int kSums = MODE == kDx ? 2 : 1;
    static constexpr int kPlanes = MODE == kDw ? 2 : 1;           // products
};

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
#define MEBLOCK_LDS __attribute__((address_space(3)))

// One operand: two matrices of the same shape (Wg and Wu, dg and du, or x
// twice), `rows` of them along the dimension that is not summed.
template <typename T>
struct Operand {
    const T* base[2];
    int64_t ld[2];
    int rows;
};

// A product: what the loop over tiles and the sums of parts take.
template <typename T>
struct Product {
    Operand<T> p, q;
    int k;        // length of the sum (of each half, kDx)
    int q_cols;   // kDw, kLinDw: columns of q that may be read (padded)
    int tiles_m, tiles_n;
    T* out[2];
    int64_t ldo[2];
    int out_cols; // columns of out that are written
    // A sum that is split: `splits` binary32 parts, each [planes * q.rows]
    // [part_ld] (kUp: columns as P's rows, 32 of Wg and 32 of Wu in turn).
    float* part;
    int splits, part_ld;
};

// ---------------------------------------------------------------------------
// The activation and the product, on binary32 g and u.  P (precise): binary32
// calls; bfloat16 calls take the activations' shorter paths (2^-14 of f and f',
// against 2^-9 and more of the result's rounding).
// ---------------------------------------------------------------------------
template <class Op, bool P>
__device__ __forceinline__ float act_value(float x, const Coef& k)
{
    float key = 0.0f;
    float y = Op::template fwd<P>(x, k, key);
    if (Op::kHasRare && Op::template is_rare<false, P>(x, k))
        y = Op::fwd_rare(x, k);
    return y;
}

// dy f'(x).
template <class Op, bool P>
__device__ __forceinline__ float act_slope(float x, float dy, const Coef& k)
{
    float key = 0.0f;
    float d = Op::template bwd<P>(x, dy, k, key);
    if (Op::kHasRare && Op::template is_rare<true, P>(x, k))
        d = Op::bwd_rare(x, dy, k);
    return d;
}

// ---------------------------------------------------------------------------
// Matrix-core steps of 16 x 16 results.  A step is 64 bytes of k: 32 (bf16)
// or 16 (binary32) values; lane l holds row l % 16 and, of k, values
// 8 (l / 16) + j (bf16, one instruction) or 4 (l / 16) + j (binary32,
// instruction j): 16 consecutive bytes.
// ---------------------------------------------------------------------------
template <typename T> struct Step;

template <> struct Step<bf16_t> {
    typedef bf16x8 Frag;
    __device__ static f32x4 mma(Frag p, Frag q, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(p, q, c, 0, 0, 0);
    }
};

template <> struct Step<float> {
    typedef f32x4 Frag;
    __device__ static f32x4 mma(Frag p, Frag q, f32x4 c)
    {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(p[j], q[j], c, 0, 0, 0);
        return c;
    }
};

// Four consecutive k of column `lane % 16` out of 4 rows (k) x 16 columns:
// lane l of each 16 names the address of row l / 4, columns 4 (l % 4) ...
__device__ __forceinline__ i16x4 lds_transpose(const char* p)
{
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((MEBLOCK_LDS i16x4*)p);
}

// The row that lane l's row l % 16 of the 16 rows from `row0` (a multiple of
// 16) is: itself, or (PAIR, P with k contiguous) interleaved by fours with the
// other 16 of its 32.
template <bool PAIR>
__device__ __forceinline__ int frag_row(int row0)
{
    const int l = threadIdx.x % 64;
    return PAIR ? row0 / 32 * 32 + row0 / 16 % 2 * 4 + l % 16 / 4 * 8 + l % 4 : row0 + l % 16;
}

typedef short i16x8 __attribute__((ext_vector_type(8)));
__device__ __forceinline__ bf16x8 join(i16x4 lo, i16x4 hi)
{
    const i16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, v);
}

// ---------------------------------------------------------------------------
// Epilogues, from the accumulators: lane l holds, of each 16 x 16 results,
// row l % 16 (of m) and the four columns 4 (l / 16) ...  Where P has k
// contiguous (kUp, kLin) the fragments are read so that the first and second 16
// of 32 columns give a lane columns 8 (l / 16) ... and 8 (l / 16) + 4 ...: eight
// consecutive ones.  (kUp: a wave's columns are 32 hidden units of g and the same
// 32 of u in turn.)
// ---------------------------------------------------------------------------
// The lane, as a value the compiler computes where it is used: what follows
// from it does not occupy registers through the products.
__device__ __forceinline__ int late_lane()
{
    int l = threadIdx.x % 64;
    asm volatile("" : "+v"(l));
    return l;
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));

__device__ __forceinline__ void store4(bf16_t* p, f32x4 f)
{
    const u32x2 v = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])};
    *reinterpret_cast<u32x2_any*>(p) = v;
}
__device__ __forceinline__ void store4(float* p, f32x4 f)
{
    store16(p, Elem<float>::pack(reinterpret_cast<const float*>(&f)));
}

template <typename T>
__device__ __forceinline__ void store_some(T* p, f32x4 f, int n)  // the first n of four
{
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < n)
            p[j] = Elem<T>::put(f[j]);
}

// Results as they are: dx, dWg, dWu, or the parts of a split sum.
template <bool PAIR, typename U, int MT, int NT>
__device__ __forceinline__ void store_results(U* out, int64_t ld, int64_t rows, int cols, int64_t m0,
                                              int n0, const f32x4 (&acc)[MT][NT])
{
    const int l = late_lane();
    const int64_t m = m0 + l % 16;
    out += m * ld;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        if (m + 16 * i < rows)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int n = n0 + (PAIR ? 32 * (j / 2) + 8 * (l / 16) + 4 * (j % 2)
                                         : 16 * j + 4 * (l / 16));
                const int left = cols - n;
                if (left >= 4)
                    store4(out + n, acc[i][j]);
                else if (left > 0)
                    store_some(out + n, acc[i][j], left);
            }
        out += 16 * ld;
    }
}

// Eight consecutive values, as loaded.
template <typename T>
struct Eight {
    static constexpr int V = sizeof(T) / 2;
    u32x4 v[V];
    __device__ void load(const T* p)
    {
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = load16(p + i * Elem<T>::kPerVec);
    }
    __device__ void values(float* f) const
    {
#pragma unroll
        for (int i = 0; i < V; ++i)
            Elem<T>::unpack(v[i], f + i * Elem<T>::kPerVec);
    }
    __device__ static void store(T* p, const float* f)
    {
#pragma unroll
        for (int i = 0; i < V; ++i)
            store16(p + i * Elem<T>::kPerVec, Elem<T>::pack(f + i * Elem<T>::kPerVec));
    }
};

template <typename T>
__device__ __forceinline__ void store_some8(T* p, const float* f, int n)  // the first n of eight
{
    if (n >= 8) {
        Eight<T>::store(p, f);
    } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < n)
                p[j] = Elem<T>::put(f[j]);
    }
}

// What a wave needs of a matrix [rows][cols] beside its results (dh, dy, a
// residual): eight columns of row m + 16 i for each of MT rows and B groups of
// 32 columns; all in flight together.
template <typename T, int MT, int B>
struct Beside {
    Eight<T> v[MT * B];
    __device__ __forceinline__ void load(const T* base, int64_t ld, int rows, int cols, int64_t m0,
                                         int n0)
    {
        const int l = late_lane();
        const int64_t row = m0 + l % 16;
        const int n = n0 + 8 * (l / 16);
        const T* p = base + row * ld;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int b = 0; b < B; ++b)
                if (row + 16 * i < rows && n + 32 * b + 8 <= cols)
                    v[i * B + b].load(p + 16 * i * ld + n + 32 * b);
        // A row's last, partial vector, apart (the code of the wide loads
        // stays free of it).
        if (cols % 8 && n0 + 32 * B > cols)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const int c = n + 32 * b;
                    if (row + 16 * i < rows && c < cols && c + 8 > cols)
#pragma unroll
                        for (int k = 0; k < Eight<T>::V; ++k)
                            v[i * B + b].v[k] = load_chunk(
                                p + 16 * i * ld, c + k * Elem<T>::kPerVec, cols);
                    __builtin_amdgcn_sched_barrier(0);
                }
    }
};

// Tiles in an order that keeps the blocks of one XCD (every eighth block) on
// neighbouring tiles, whose operands they then share in that XCD's L2:
// columns of 8 tiles along m, then along n.  (bf16 16384 x 4096 x 16384: 80 %
// of the L2's requests hit, and HBM delivers 1.0 to 1.5 TB/s to the products.)
__device__ __forceinline__ void tile_of_block(int id, int tiles_m, int tiles_n, int& tm, int& tn)
{
    const int total = tiles_m * tiles_n;
    const int per = total / 8, rest = total % 8;
    const int xcd = id % 8, at = id / 8;
    id = xcd * per + (xcd < rest ? xcd : rest) + at;
    constexpr int kGroup = 8;
    const int width = kGroup * tiles_n;
    const int first = id / width * kGroup;
    const int rows = tiles_m - first < kGroup ? tiles_m - first : kGroup;
    tm = first + id % width % rows;
    tn = id % width / rows;
}

// Steps [first, total) of a sum of `total` steps: block row y's share.
__device__ __forceinline__ void part_of_sum(int splits, int part, int& first, int& total)
{
    const int whole = total;
    first = (int)((int64_t)whole * part / splits);
    total = (int)((int64_t)whole * (part + 1) / splits);
}

// A block's place among those of its product: the first of its tiles, how far it
// steps to the next one, its part of the sums.  In a launch of one product they are
// read where they are used, which holds no registers; of several, given.
struct OwnPlace {
    __device__ static int block() { return blockIdx.x; }
    __device__ static int blocks() { return gridDim.x; }
    __device__ static int part() { return blockIdx.y; }
};

struct GivenPlace {
    int block_, blocks_, part_;
    __device__ int block() const { return block_; }
    __device__ int blocks() const { return blocks_; }
    __device__ int part() const { return part_; }
};

// The LDS that tiles are loaded to: the same memory for every product of a kernel.
template <int BYTES>
__device__ __forceinline__ char* tile_memory()
{
    __shared__ __attribute__((aligned(1024))) char lds[BYTES];
    return lds;
}

// ---------------------------------------------------------------------------
// Products of matrices whose rows start on 16-byte boundaries.  WM x WN waves
// of (16 MT) x (16 NT) results each; k in steps of 128 bytes.  Operands go
// from memory to LDS directly (buffer loads with the LDS bit, 16 bytes a
// lane), two tiles of each operand in LDS: while one is multiplied the next
// one arrives.
//
// What bounds it, and why this shape (bf16, 16384 x 4096 -> 16384: forward
// 1400 TFLOP/s, recomputation 1250, dx 1320, dWg and dWu 1270; binary32 8192 x
// 2048 -> 4096: 147 of the 157 its matrix instructions have).  The matrix
// cores are busy 71 % of the cycles and the card lowers its clock (1.75 GHz)
// under the load: on zeros, which cost little power, the forward reaches 1580.
// Without the loads the loop alone would be at 2270, so the rest is the wait
// for them.  Measured against it: 16 x 16 matrix instructions instead of 32 x
// 32, forward 1304 to 1352; products, reads and loads in the order written
// instead of the compiler's, 1228 to 1304; eight waves of 128 x 64 against
// four of 128 x 128, 1272 and 1162; 64 bytes of k a step with four or five
// tiles in LDS, 1210 (twice the barriers, half lines fetched twice); loads
// spread over the next step, 1305 against 1346; lines of later steps touched
// into the L2 beforehand, 1490 to 1650 on zeros but 1217 to 1185 on numbers.
//
// The recomputation's 256 x 256 kernels have no register left (256 of 256): the
// binary32 one spills 60 (52 bytes of scratch), the bf16 one 2, all outside the
// products' loop, around the epilogue.
//
// A load writes 1 KiB of LDS in lane order, so the layouts that avoid bank
// conflicts are made by choosing which 16 bytes each lane fetches:
//   k contiguous: rows of 128 bytes; 16-byte slot s of row r holds chunk
//     s ^ (r / 2 % 8).  Sixteen lanes read one chunk of 16 consecutive rows,
//     which then covers all 64 banks once.  (P of kUp: of rows 8 a + b, a and
//     b < 4; s ^ (r / 2 % 2 + 2 (r / 8 % 4)) does the same for them.)
//   n contiguous: a k row holds the tile's columns.  bf16: 32-byte unit c of
//     row k holds unit c ^ (k % 4 + 4 (k / 8 % 2)); 32 lanes of a transposing
//     read take one unit of rows k .. k + 3 and k + 8 .. k + 11, again all
//     banks.  binary32: 64-byte unit c holds unit c ^ (k / 4 % 4).
// Chunks past the end of the sum lie outside the buffer descriptor's range
// (or are pointed there), which reads as zero.  Rows and columns past an
// edge repeat the last one: their results are not stored.
// ---------------------------------------------------------------------------
typedef int i32x4 __attribute__((ext_vector_type(4)));
constexpr uint32_t kBufferBytes = 0xc0000000u;  // no tile reaches this far
constexpr uint32_t kOutside = 0xf0000000u;

__device__ __forceinline__ void load_lds16(uint32_t lds, uint32_t offset, i32x4 rsrc)
{
    // The wait for it is explicit (wait_loads) and ends before a barrier.
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(offset), "s"(rsrc)
                 : "memory", "m0");
}

// The scalar registers of a descriptor may come from vector instructions, which
// a buffer load may read five issue slots later at the earliest; the compiler
// does not see into the assembly above.  (In the loop a row of products lies
// between.)
__device__ __forceinline__ void settle_descriptors()
{
    asm volatile("s_nop 4" : : : "memory");
}

// The block's barrier, over which no access to LDS moves.
__device__ __forceinline__ void meet()
{
    __builtin_amdgcn_s_barrier();
    asm volatile("" : : : "memory");
}

template <int N>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

__device__ __forceinline__ i32x4 buffer(const void* p, uint32_t bytes)
{
    const uint64_t a = (uint64_t)p;
    i32x4 r = {(int)(uint32_t)a, (int)(uint32_t)((a >> 32) & 0xffff), (int)bytes, 0x00020000};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = __builtin_amdgcn_readfirstlane(r[i]);
    return r;
}

constexpr int KB = 128;  // bytes of k a step

// A tile of ROWS values of m or n and one step of k, filled by WAVES waves.
template <typename T, bool KC, bool PAIR, int ROWS, int WAVES>
struct FastTile {
    static constexpr int E = Elem<T>::kPerVec;
    static constexpr int kK = KB / sizeof(T);
    static constexpr int kBytes = ROWS * KB;
    static constexpr int kRowBytes = KC ? KB : ROWS * (int)sizeof(T);
    static constexpr int kLoads = kBytes / 1024 / WAVES;  // of a wave
    static_assert(kLoads * WAVES * 1024 == kBytes, "whole loads");

    __device__ static int swizzle(int r)  // of 16-byte slots
    {
        if (KC)
            return PAIR ? r / 2 % 2 + r / 8 % 4 * 2 : r / 2 % 8;
        return sizeof(T) == 2 ? (r % 4 + r / 8 % 2 * 4) * 2 : r / 4 % 4 * 4;
    }
    // This lane's part of load i: the tile row it falls in and the chunk of it.
    __device__ static int row(int lane, int wave, int i)
    {
        return ((wave * kLoads + i) * 1024 + lane * 16) / kRowBytes;
    }
    __device__ static int chunk(int lane, int wave, int i)
    {
        static_assert(kRowBytes <= 1024, "a load covers whole rows");
        return lane * 16 % kRowBytes / 16 ^ swizzle(row(lane, wave, i));
    }
    __device__ static typename Step<T>::Frag frag(const char* lds, int step, int row0)
    {
        const int l = threadIdx.x % 64;
        if constexpr (KC) {
            const int r = frag_row<PAIR>(row0);
            return *reinterpret_cast<const typename Step<T>::Frag*>(
                lds + r * KB + ((step * 4 + l / 16) ^ swizzle(r % 32)) * 16);
        } else if constexpr (sizeof(T) == 2) {
            const int k = 8 * (l / 16) + l % 16 / 4;
            const char* p = lds + (step * 32 + k) * kRowBytes +
                            ((row0 / 8 + l % 4 / 2) ^ swizzle(k)) * 16 + l % 2 * 8;
            return join(lds_transpose(p), lds_transpose(p + 4 * kRowBytes));
        } else {
            const int k = 4 * (l / 16);
            const char* p = lds + (step * 16 + k) * kRowBytes +
                            ((row0 / 4 + l % 16 / 4) ^ swizzle(k)) * 16 + l % 4 * 4;
            f32x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = *reinterpret_cast<const float*>(p + j * kRowBytes);
            return v;
        }
    }
};

// The product of args a (a Product).  finish(m0, n0, plane, acc) ends a wave's
// tile: its results from row m0 and column n0 (of P's rows, kUp) on.
template <typename T, int MODE, int WM, int WN, int MT, int NT, bool PARTS, class Args, class Finish,
          class Place = OwnPlace>
__device__ __forceinline__ void product_tiles(const Args& a, const Finish& finish,
                                              const Place at = Place())
{
    using F = Form<MODE>;
    constexpr bool PK = F::kPK, QK = F::kQK;
    constexpr int BM = WM * MT * 16, BN = WN * NT * 16, WAVES = WM * WN;
    using PT = FastTile<T, PK, PK, BN, WAVES>;
    using QT = FastTile<T, QK, false, BM, WAVES>;
    constexpr int kK = PT::kK, E = Elem<T>::kPerVec, STEPS = KB / 64;
    constexpr int kStage = PT::kBytes + QT::kBytes;
    char* lds = tile_memory<2 * kStage>();
    const uint32_t lds0 = (uint32_t)(uintptr_t)(MEBLOCK_LDS char*)lds;

    const int tiles = a.tiles_m * a.tiles_n * F::kPlanes;
    const int steps = (a.k + kK - 1) / kK;
    // An empty sum is one step of zeros.
    int first = 0, total = steps == 0 ? 1 : F::kSums * steps;
    const int whole = total;
    if constexpr (PARTS)
        part_of_sum(a.splits, at.part(), first, total);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wm = wave / WN * (MT * 16), wn = wave % WN * (NT * 16);

    // The tile whose operands are being loaded: it runs ahead of the one that
    // is multiplied.
    int64_t m0;
    int n0, plane, tm, tn;
    // Offsets of this lane's 16 bytes in each load, from the tile's first
    // element; (kTwo) the second weight's from its own first row.
    uint32_t offp[PT::kLoads], offq[QT::kLoads];
    auto place_tile = [&](int tile) {
        const int lane = late_lane();
        plane = 0;
        if constexpr (F::kPlanes == 2) {
            tile_of_block(tile, 2 * a.tiles_m, a.tiles_n, tm, tn);
            plane = tm >= a.tiles_m;
            tm -= plane * a.tiles_m;
        } else {
            tile_of_block(tile, a.tiles_m, a.tiles_n, tm, tn);
        }
        m0 = (int64_t)tm * BM;
        n0 = tn * (F::kTwo ? BN / 2 : BN);
#pragma unroll
        for (int i = 0; i < PT::kLoads; ++i) {
            const int r = PT::row(lane, wave, i), c = PT::chunk(lane, wave, i) * E;
            if constexpr (PK) {
                // (kTwo) Rows of the tile: 32 of each weight in turn.
                int n = F::kTwo ? r / 64 * 32 + r % 32 : r;
                n = n0 + n < a.p.rows ? n : a.p.rows - 1 - n0;
                offp[i] = (uint32_t)((int64_t)n * a.p.ld[F::kTwo ? r / 32 % 2 : 0] + c) *
                          (uint32_t)sizeof(T);
            } else {
                const int n = n0 + c < a.p.rows ? c : a.p.rows - E - n0;
                offp[i] = (uint32_t)((int64_t)r * a.p.ld[0] + n) * (uint32_t)sizeof(T);
            }
        }
#pragma unroll
        for (int i = 0; i < QT::kLoads; ++i) {
            const int r = QT::row(lane, wave, i), c = QT::chunk(lane, wave, i) * E;
            if constexpr (QK) {
                const int m = m0 + r < a.q.rows ? r : (int)(a.q.rows - 1 - m0);
                offq[i] = (uint32_t)((int64_t)m * a.q.ld[0] + c) * (uint32_t)sizeof(T);
            } else {
                const int m = m0 + c < a.q_cols ? c : (int)(a.q_cols - E - m0);
                offq[i] = (uint32_t)((int64_t)r * a.q.ld[0] + m) * (uint32_t)sizeof(T);
            }
        }
    };

    // Where the next step's loads start, in scalar registers: address, bytes
    // left of the sum from there (what lies past them reads as zero).
    const char *curp, *curq;
    int64_t incp, incq, leftp, leftq;
    // (kTwo) A wave loads 32 rows of P, all of one weight.
    static_assert(!F::kTwo || PT::kLoads * 1024 == 32 * KB, "waves in turn");
    auto start = [&](int seg) {
        if constexpr (PK) {
            const bool up = F::kTwo && wave % 2;
            const T* w = up ? a.p.base[1] : a.p.base[0];
            const int64_t ld = up ? a.p.ld[1] : a.p.ld[0];
            curp = reinterpret_cast<const char*>(w + (int64_t)n0 * ld);
            incp = kK * (int64_t)sizeof(T);
            leftp = kBufferBytes;
        } else {
            const int64_t ld = a.p.ld[0];
            curp = reinterpret_cast<const char*>((seg ? a.p.base[1] : a.p.base[0]) + n0);
            incp = kK * ld * (int64_t)sizeof(T);
            leftp = ((int64_t)(a.k - 1) * ld + a.p.rows - n0) * (int64_t)sizeof(T);
        }
        if constexpr (QK) {
            curq = reinterpret_cast<const char*>((seg ? a.q.base[1] : a.q.base[0]) +
                                                 m0 * a.q.ld[0]);
            incq = kK * (int64_t)sizeof(T);
            leftq = kBufferBytes;
        } else {
            const int64_t ld = a.q.ld[0];
            curq = reinterpret_cast<const char*>((plane ? a.q.base[1] : a.q.base[0]) + m0);
            incq = kK * ld * (int64_t)sizeof(T);
            leftq = ((int64_t)(a.k - 1) * ld + a.q_cols - m0) * (int64_t)sizeof(T);
        }
    };
    i32x4 rp, rq;
    int ahead = first, tile_ahead = at.block();  // the step whose loads come next
    auto next_step = [&]() {
        if (ahead == total) {
            ahead = first;
            tile_ahead += at.blocks();
        }
        // Past the last tile nothing is read (zeros are written).
        const bool any = tile_ahead < tiles;
        const bool some = any && a.k > 0;
        if (ahead == first && any) {
            place_tile(tile_ahead);
            start(F::kSums == 2 && first >= steps && steps > 0);
            if constexpr (PARTS) {
                const int64_t skip = F::kSums == 2 && first >= steps ? first - steps : first;
                curp += skip * incp;
                curq += skip * incq;
                if constexpr (!PK)
                    leftp -= skip * incp;
                if constexpr (!QK)
                    leftq -= skip * incq;
            }
        } else if (F::kSums == 2 && ahead == steps && any) {
            start(1);
        }
        auto bytes = [&](int64_t left) {
            return some ? (uint32_t)(left < (int64_t)kBufferBytes ? left : (int64_t)kBufferBytes) : 0u;
        };
        rp = buffer(curp, bytes(leftp));
        rq = buffer(curq, bytes(leftq));
        curp += incp;
        curq += incq;
        if constexpr (!PK)
            leftp -= incp;
        if constexpr (!QK)
            leftq -= incq;
        if constexpr (PK || MODE == kLinDx) {
            // A last step that is cut short: chunks past the end are pointed
            // outside; the next tile has offsets of its own.  (kDx: zeros follow
            // in Q's rows.)
            if (ahead == whole - 1 && a.k % kK) {
                const int k0 = ahead * kK, lane = late_lane();
#pragma unroll
                for (int i = 0; PK && i < PT::kLoads; ++i)
                    offp[i] = k0 + PT::chunk(lane, wave, i) * E < a.k ? offp[i] : kOutside;
#pragma unroll
                for (int i = 0; i < QT::kLoads; ++i)
                    offq[i] = k0 + QT::chunk(lane, wave, i) * E < a.k ? offq[i] : kOutside;
            }
        }
        ++ahead;
    };
    const uint32_t ldsp = lds0 + wave * (PT::kLoads * 1024);
    const uint32_t ldsq = lds0 + PT::kBytes + wave * (QT::kLoads * 1024);
    constexpr int kLoads = PT::kLoads + QT::kLoads;
    auto issue = [&](uint32_t place, int i) {
        if (i < PT::kLoads)
            load_lds16(ldsp + place + i * 1024, offp[i], rp);
        else
            load_lds16(ldsq + place + (i - PT::kLoads) * 1024, offq[i - PT::kLoads], rq);
    };

    f32x4 acc[MT][NT];

    // Fragments: P's twice, one set multiplied while the next is read; Q's
    // once, each read again as soon as its products have been issued.
    typename Step<T>::Frag fp[2][NT], fq[MT];
    auto read_p = [&](int set, uint32_t place, int t, int j) {
        fp[set][j] = PT::frag(lds + place, t, wn + 16 * j);
    };
    auto read_q = [&](uint32_t place, int t, int i) {
        fq[i] = QT::frag(lds + place + PT::kBytes, t, wm + 16 * i);
    };
    static_assert(STEPS % 2 == 0, "P's sets alternate across steps");

    auto first_part = [&](uint32_t place) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
            read_p(0, place, 0, j);
#pragma unroll
        for (int i = 0; i < MT; ++i)
            read_q(place, 0, i);
    };
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        next_step();
        settle_descriptors();
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            issue(s * kStage, i);
    }
    wait_loads<kLoads>();
    meet();
    // Step s: its first fragments are in registers.  Its last reads are issued
    // before its last part; a row of products into that part (BG), the barrier
    // behind which step s + 1 is in LDS and the place of step s is free for
    // step s + 2.  Reads and loads are spread between the products; the
    // order is kept as written.
    constexpr int BG = 1;
    uint32_t place = 0;
#pragma unroll 1
    for (int tile = at.block(); tile < tiles; tile += at.blocks()) {
        int om, on, op = 0;  // this tile's place in the output
        if constexpr (F::kPlanes == 2) {
            tile_of_block(tile, 2 * a.tiles_m, a.tiles_n, om, on);
            op = om >= a.tiles_m;
            om -= op * a.tiles_m;
        } else {
            tile_of_block(tile, a.tiles_m, a.tiles_n, om, on);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                acc[i][j] = f32x4{};
        first_part(place);
        int s = first;
#pragma unroll 1
        do {
            const uint32_t next = place ^ kStage;
#pragma unroll
            for (int t = 0; t < STEPS; ++t) {
                const bool last = t == STEPS - 1;
                if (last)
                    next_step();
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        acc[i][j] = Step<T>::mma(fp[t & 1][j], fq[i], acc[i][j]);
                    if (last && i == BG) {
                        __builtin_amdgcn_sched_barrier(0);
                        wait_loads<0>();
                        asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
                        meet();
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    // The next part's fragments: Q's row i behind its products
                    // (and those the barrier held back), P's early.
                    const uint32_t from = last ? next : place;
                    const int part = last ? 0 : t + 1, lead = last ? BG : 0;
                    if (i >= lead) {
                        if (i == lead)
#pragma unroll
                            for (int k = 0; k < lead; ++k)
                                read_q(from, part, k);
                        read_q(from, part, i);
                        constexpr int kP = (NT + MT - BG - 1) / (MT - BG);  // P's fragments a row
#pragma unroll
                        for (int j = (i - lead) * kP; j < (i - lead + 1) * kP && j < NT; ++j)
                            read_p(~t & 1, from, part, j);
                    }
                    if (last && i >= BG) {
                        constexpr int kRows = MT - BG;
#pragma unroll
                        for (int k = (i - BG) * kLoads / kRows; k < (i - BG + 1) * kLoads / kRows;
                             ++k)
                            issue(place, k);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            place = next;
        } while (++s < total);
        // The next tile's first steps arrive meanwhile.
        finish((int64_t)om * BM + wm, on * BN + wn, op, acc);
    }
    wait_loads<0>();  // no load writes LDS after the block has ended
}

// ---------------------------------------------------------------------------
// Few tokens: the weights are read once, and their bytes bound the time.  A
// block takes 16 PT units and all (at most 16 QT) tokens; its NW waves
// take a share of the sum each, load the weights' fragments from memory
// straight into registers (16 bytes a lane at element alignment, U steps in
// flight) with x's fragments beside them (from the caches), and add their
// parts through LDS in the order of the wave.  bf16 4096 -> 16384 (268 MB of
// weights): 1 token 49 us, 24 tokens 56 (5.5 and 4.8 TB/s) where the weights come
// from memory; 43 and 51 called again on the same weights, of which the 256 MB
// Infinity Cache then holds most.
// ---------------------------------------------------------------------------
// H weights; finish(m, n, results of the weights) ends an element.
template <typename T, int H, int PT, int QT, int NW, int U, class Args, class Finish>
__device__ __forceinline__ void few_tokens(const Args& a, const Finish& finish)
{
    typedef typename Step<T>::Frag Frag;
    constexpr int E = Elem<T>::kPerVec, kK = 64 / sizeof(T), kTiles = H * PT * QT;
    __shared__ float part[NW][kTiles][256];
    const int l = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int n0 = blockIdx.x * (16 * PT);
    const int k0 = l / 16 * E;
    const T* w[H][PT];
    const T* x[QT];
#pragma unroll
    for (int j = 0; j < PT; ++j) {
        const int n = n0 + 16 * j + l % 16;
        const int64_t r = n < a.p.rows ? n : a.p.rows - 1;
#pragma unroll
        for (int h = 0; h < H; ++h)
            w[h][j] = a.p.base[h] + r * a.p.ld[h];
    }
#pragma unroll
    for (int i = 0; i < QT; ++i) {
        const int m = 16 * i + l % 16;
        x[i] = a.q.base[0] + (m < a.q.rows ? m : a.q.rows - 1) * a.q.ld[0];
    }
    f32x4 acc[H][PT][QT];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int j = 0; j < PT; ++j)
#pragma unroll
            for (int i = 0; i < QT; ++i)
                acc[h][j][i] = f32x4{};
    // N steps from k, loads first; the last step of the sum may be cut short.
    auto steps = [&](int64_t k, auto count, auto whole) {
        constexpr int N = decltype(count)::value;
        u32x4 fw[N][H][PT], fx[N][QT];
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int64_t kk = k + u * kK + k0;
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int j = 0; j < PT; ++j)
                    fw[u][h][j] = decltype(whole)::value ? load16(w[h][j] + kk)
                                                         : load_chunk(w[h][j], (int)kk, a.k);
#pragma unroll
            for (int i = 0; i < QT; ++i)
                fx[u][i] = decltype(whole)::value ? load16(x[i] + kk)
                                                  : load_chunk(x[i], (int)kk, a.k);
        }
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int j = 0; j < PT; ++j)
#pragma unroll
                    for (int i = 0; i < QT; ++i)
                        acc[h][j][i] = Step<T>::mma(__builtin_bit_cast(Frag, fw[u][h][j]),
                                                    __builtin_bit_cast(Frag, fx[u][i]),
                                                    acc[h][j][i]);
    };
    const int whole = a.k / kK, all = (a.k + kK - 1) / kK;
    int s = (int)((int64_t)all * wave / NW);
    const int end = (int)((int64_t)all * (wave + 1) / NW);
    const int full = end < whole ? end : whole;
    using std::integral_constant;
    for (; s + U <= full; s += U)
        steps((int64_t)s * kK, integral_constant<int, U>(), integral_constant<bool, true>());
    for (; s < full; ++s)
        steps((int64_t)s * kK, integral_constant<int, 1>(), integral_constant<bool, true>());
    if (s < end)
        steps((int64_t)s * kK, integral_constant<int, 1>(), integral_constant<bool, false>());
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int j = 0; j < PT; ++j)
#pragma unroll
            for (int i = 0; i < QT; ++i)
                *reinterpret_cast<f32x4*>(&part[wave][(h * PT + j) * QT + i][l * 4]) = acc[h][j][i];
    __syncthreads();
    for (int t = threadIdx.x; t < 256 * PT * QT; t += NW * 64) {
        const int n = t % (16 * PT), m = t / (16 * PT);
        const int tile = n / 16 * QT + m / 16, at = (n % 16 / 4 * 16 + m % 16) * 4 + n % 4;
        float r[H] = {};
#pragma unroll
        for (int v = 0; v < NW; ++v)
#pragma unroll
            for (int h = 0; h < H; ++h)
                r[h] += part[v][h * PT * QT + tile][at];
        if (m < a.q.rows)
            finish(m, n0 + n, r);
    }
}

// ---------------------------------------------------------------------------
// Up to three matrices in rows that start on 128-byte boundaries, zeros behind them:
// for the products above where the caller's rows do not start on 16-byte
// ones.  Measured against products that took rows at any alignment through
// registers (128 x 128 tiles): bf16 4096 x 2047 -> 8191 forward 789 us to 296,
// backward 2536 to 798; at 200 x 257 -> 131 the copy's launch costs 2 us of 16
// forward and the backward still gains, 47 to 31.
// ---------------------------------------------------------------------------
template <typename T>
struct PackArgs {
    const T* from[3];
    int64_t ld[3], rows[3];
    T* to;
    int cols, ld_to;
    int row_bits;  // 2^row_bits threads a row
};

template <typename T>
__device__ __forceinline__ void pack_rows(const PackArgs<T>& a)
{
    constexpr int E = Elem<T>::kPerVec;
    const int64_t rows = a.rows[0] + a.rows[1] + a.rows[2];
    const int per_block = 256 >> a.row_bits;
    for (int64_t row = (int64_t)blockIdx.x * per_block + (threadIdx.x >> a.row_bits); row < rows;
         row += (int64_t)gridDim.x * per_block) {
        int64_t r = row, ld = a.ld[0];
        const T* from = a.from[0];
        if (r >= a.rows[0]) {
            r -= a.rows[0];
            const bool third = r >= a.rows[1];
            r -= third ? a.rows[1] : 0;
            from = third ? a.from[2] : a.from[1];
            ld = third ? a.ld[2] : a.ld[1];
        }
        from += r * ld;
        T* to = a.to + row * a.ld_to;
        for (int c = (threadIdx.x & ((1 << a.row_bits) - 1)) * E; c < a.ld_to; c += E << a.row_bits)
            store16(to + c, load_chunk(from, c, a.cols));
    }
}

// ---------------------------------------------------------------------------
// The parts of a split sum, added in order: four columns a thread.
// ---------------------------------------------------------------------------
template <typename T, int MODE>
__device__ __forceinline__ void sum_parts(const Product<T>& a, int block)
{
    constexpr int kPlanes = Form<MODE>::kPlanes;
    const int64_t per_row = a.part_ld / 4, rows = (int64_t)a.q.rows * kPlanes;
    const int64_t at = (int64_t)block * 256 + threadIdx.x;
    if (at >= rows * per_row)
        return;
    const int64_t row = at / per_row;
    const int n = (int)(at % per_row) * 4;
    const float* p = a.part + row * a.part_ld + n;
    f32x4 v = f32x4{};
#pragma unroll 4  // four loads in flight
    for (int s = 0; s < a.splits; ++s)
        v += *reinterpret_cast<const f32x4*>(p + s * rows * a.part_ld);
    const int plane = row >= a.q.rows;
    T* out = (plane ? a.out[1] : a.out[0]) +
             (row - (plane ? a.q.rows : 0)) * (plane ? a.ldo[1] : a.ldo[0]) + n;
    const int left = a.out_cols - n;
    if (left >= 4)
        store4(out, v);
    else
        store_some(out, v, left);
}

// ---------------------------------------------------------------------------
// Host.
// ---------------------------------------------------------------------------

inline size_t padded(size_t hidden) { return (hidden + 63) / 64 * 64; }

constexpr int kCus = 256;

// How a product is computed: 256 x 256 tiles or 128 x 128, and in how many
// parts its sum is split.
struct Plan {
    bool big;
    int splits;
};

// The least of the estimated times.  A block's step of 128 bytes of k takes
// what its instructions take (a bf16 128 x 128 step 0.4 us of a CU, binary32
// 1.75 us; a 256 x 256 step 1.2 and 6.8 us), and no less than the 0.7 us its
// loads take, which two blocks of a CU share; parts are written and read
// again at some 4 TB/s, by one more launch (3 us).
//
// Measured both ways, bf16, tokens x dim x hidden:
//   256 x 256 against 128 x 128, unsplit: forward 16384 x 4096 x 16384 3118 us
//   against 3981, 64 x 4096 x 16384 86 against 58, 777 x 1000 x 2736 26
//   against 19; dWg and dWu 777 x 1000 x 2736 26 against 18.
//   dx, 128 x 128: 64 x 4096 x 16384 308 us whole, 104 in 4 parts, 64 in 16;
//   777 x 1000 x 2736 52, 25 in 4, 29 in 8; 16384 x 4096 x 16384 4017, 4456
//   in 2.  dx, 256 x 256 in parts against 128 x 128 in parts: 1024 x 4096 x
//   16384 246 against 297, 512 x 4096 x 16384 147 against 166.
// Binary32, 256 x 256 against 128 x 128, unsplit: 8192 x 2048 x 4096 forward
// 1853 us against 1904, dx 1857 against 1905; 2048 x 1024 x 4096 dWg and dWu
// 476 against 250; dx there 512 whole, 272 in 2 parts.
inline Plan make_plan(int64_t rows, int64_t cols, int64_t k, int planes, int sums, size_t es)
{
    const int64_t steps = (k + 128 / (int64_t)es - 1) / (128 / (int64_t)es) * sums;
    Plan best{false, 1};
    double least = 1e30;
    for (int big = 0; big < 2; ++big) {
        const int64_t side = big ? 256 : 128;
        const int64_t tiles = (rows + side - 1) / side * ((cols + side - 1) / side) * planes;
        const double work = big ? es == 2 ? 1.2 : 6.8 : es == 2 ? 0.4 : 1.75;
        for (int s = 1; s <= 32 && (s == 1 || s * 2 <= steps); s *= 2) {
            const int64_t blocks = (tiles * s + kCus - 1) / kCus;  // of a CU
            double step = work * (double)blocks, loads = 0.7 * (double)((blocks + 1) / 2);
            step = step > loads ? step : loads;
            double t = step * (double)((steps + s - 1) / s);
            if (s > 1)
                t += 3.0 + (double)(tiles * s) * (double)(side * side * 8) / 4e6;
            if (t < least) {
                least = t;
                best = Plan{big != 0, s};
            }
        }
    }
    return best;
}

// Columns of a part: P's rows (kUp) or the result's, in whole vectors.
inline int64_t part_ld(int mode, int64_t cols)
{
    return mode == kUp ? (cols + 63) / 64 * 128 : (cols + 3) / 4 * 4;
}

inline size_t part_bytes(int mode, int64_t rows, int64_t cols, int64_t k, size_t es)
{
    const int planes = mode == kDw ? 2 : 1;
    const Plan p = make_plan(rows, mode == kUp ? 2 * cols : cols, k, planes, mode == kDx ? 2 : 1, es);
    return p.splits > 1 ? (size_t)p.splits * planes * rows * part_ld(mode, cols) * sizeof(float) : 0;
}

// Blocks that are on the GPU together, by their LDS (160 KiB a CU); a
// multiple of the 8 XCDs.
inline int resident_blocks(int lds_bytes) { return kCus * ((160 << 10) / lds_bytes); }

// Launches a kernel of product_tiles over the tiles of bm x bn results (bn: of
// P's columns' results); sets the tiles.  resident > 0: at most so many blocks,
// each looping over tiles.
template <class Args>
inline int launch_tiles(Args& a, const void* fn, int bm, int bn, int planes, int block, int resident,
                        hipStream_t stream)
{
    a.tiles_m = (a.q.rows + bm - 1) / bm;
    a.tiles_n = (a.out_cols + bn - 1) / bn;
    // The kernel counts tiles in 31 bits; a launch has fewer than 2^32 threads.
    const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n * planes;
    if (tiles == 0)
        return MESWISH_OK;
    const int64_t grid = resident && tiles > resident ? resident : tiles;
    if (tiles > ((int64_t)1 << 30) || grid * block >= (int64_t)1 << 32)
        return MESWISH_EINVAL;
    void* args[] = {&a};
    return launch(fn, dim3((unsigned)grid, a.splits), block, args, stream);
}

inline int launch_over(const void* fn, int64_t n, void** args, hipStream_t stream)
{
    const int64_t grid = (n + 255) / 256;
    if (grid >= ((int64_t)1 << 24))
        return MESWISH_EINVAL;
    return launch(fn, dim3((unsigned)grid), 256, args, stream);
}

template <typename T>
inline Operand<T> operand(const void* a, int64_t lda, const void* b, int64_t ldb, size_t rows)
{
    return Operand<T>{{static_cast<const T*>(a), static_cast<const T*>(b)}, {lda, ldb}, (int)rows};
}

inline size_t packed_ld(size_t dim, size_t es) { return (dim * es + 127) / 128 * 128 / es; }

inline size_t lines(size_t bytes) { return (bytes + 127) / 128 * 128; }

}  // namespace meblock
