// gated_ffn.hip -- the gated feed-forward unit of libmeswish for gfx950,
// forward and backward.  Formulas and contracts: include/gated_ffn.h.
//
// Every product is written as out[m][n] = sum_k Q(m, k) P(n, k):
//
//   kUp  g and u:   P = Wg, Wu (k contiguous), Q = x (k contiguous), k = dim.
//        A block's columns hold the same hidden units of both projections,
//        32 of Wg then 32 of Wu, so one wave ends with g and u of the same
//        elements in its registers and applies the activation there: h, or
//        dg and du, are all that is written.
//   kDx  dx:        P = Wg, Wu (n contiguous), Q = dg, du (k contiguous):
//        one sum over hidden units of both, 2 hidden long.
//   kDw  dWg, dWu:  P = x (n contiguous), Q = dg, du (m contiguous),
//        k = tokens.
//
// dg and du are written in the tensors' type, also where that is bfloat16: they
// are the next products' operands, which the matrix cores take in that type
// (errors of the bf16 gradients against binary64 0.0023 to 0.0024 of their norm,
// 0.0017 from the results' own rounding alone).
//
// The matrix cores (v_mfma_f32_16x16x32_bf16, v_mfma_f32_16x16x4_f32) take
// P as the operand whose rows index the four consecutive results a lane
// holds, so a lane's results are consecutive along n.

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "act_math.h"
#include "block_common.h"
#include "gated_ffn.h"

namespace meblock {

using meswish::Coef;

enum Mode { kUp = 0, kDx = 1, kDw = 2 };

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

template <typename T>
struct GemmArgs {
    Operand<T> p, q;
    int k;        // length of the sum (of each half, kDx)
    int q_cols;   // kDw: columns of q that may be read (padded)
    int tiles_m, tiles_n;
    T* out[2];    // h, or dg and du; dx; dWg and dWu
    int64_t ldo[2];
    int out_cols; // columns of out that are written (kUp: padded, zeros past p.rows)
    const T* dh;  // kUp, backward
    int64_t lddh;
    T* h;         // kUp, backward: the forward's result, or NULL
    int64_t ldh;
    // A sum that is split: `splits` binary32 parts, each [planes * q.rows]
    // [part_ld] (kUp: columns as P's rows, 32 of Wg and 32 of Wu in turn).
    float* part;
    int splits, part_ld;
    int act;
    Coef coef;
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
// 16) is: itself, or (PAIR, P of kUp) interleaved by fours with the other 16
// of its 32.
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
// row l % 16 (of m) and the four columns 4 (l / 16) ...  kUp: a wave's
// columns are 32 hidden units of g and the same 32 of u in turn, and the
// fragments are read so that the first and second 16 of them give a lane
// units 8 (l / 16) ... and 8 (l / 16) + 4 ...: eight consecutive ones.
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

// What a wave needs of dh: eight units of row m + 16 i for each of its MT rows
// and NT / 4 groups of 32 columns; all in flight together.
template <typename T, int MT, int NT>
struct Upstream {
    Eight<T> v[MT * NT / 4];
    __device__ __forceinline__ void load(const GemmArgs<T>& a, int64_t m0, int n0)
    {
        const int l = late_lane();
        const int64_t row = m0 + l % 16;
        const int n = n0 + 8 * (l / 16);
        const T* p = a.dh + row * a.lddh;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int b = 0; b < NT / 4; ++b)
                if (row + 16 * i < a.q.rows && n + 32 * b + 8 <= a.p.rows)
                    v[i * (NT / 4) + b].load(p + 16 * i * a.lddh + n + 32 * b);
        // A row's last, partial vector, apart (the code of the wide loads
        // stays free of it).
        if (a.p.rows % 8 && n0 + 8 * NT > a.p.rows)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int b = 0; b < NT / 4; ++b) {
                    const int c = n + 32 * b;
                    if (row + 16 * i < a.q.rows && c < a.p.rows && c + 8 > a.p.rows)
#pragma unroll
                        for (int k = 0; k < Eight<T>::V; ++k)
                            v[i * (NT / 4) + b].v[k] = load_chunk(
                                p + 16 * i * a.lddh, c + k * Elem<T>::kPerVec, a.p.rows);
                    __builtin_amdgcn_sched_barrier(0);
                }
    }
};

// The unit on vectors of eight, without the activations' rare branches.  True
// in a lane that met one: the wave is then done again by gate_slow, to the
// same places.
template <class Op, typename T, bool BWD, int MT, int NT>
__device__ __forceinline__ bool gate_fast(const GemmArgs<T>& a, int64_t m0, int n0,
                                          const f32x4 (&acc)[MT][NT])
{
    constexpr bool P = sizeof(T) == 4;
    const int l = late_lane();
    int64_t row = m0 + l % 16;
    const int n = n0 + 8 * (l / 16);
    T* out0 = a.out[0] + row * a.ldo[0];
    T* out1 = BWD ? a.out[1] + row * a.ldo[1] : nullptr;
    T* outh = BWD && a.h ? a.h + row * a.ldh : nullptr;
    // Loaded here and not once before the choice of activation: what that
    // would let the compiler compute early (all of dh unpacked) does not fit
    // the registers.
    Upstream<T, MT, NT> d;
    if constexpr (BWD)
        d.load(a, m0, n0);
    float key = 0.0f;
#pragma unroll
    for (int t = 0; t < MT * NT / 4; ++t) {
        const int i = t / (NT / 4), b = t % (NT / 4) * 4;
        const int c = n + 8 * b;
        float o[8], du[8], h[8], up[8];
        if constexpr (BWD)
            d.v[t].values(up);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float g = acc[i][b + e / 4][e % 4], u = acc[i][b + 2 + e / 4][e % 4];
            const float f = Op::template fwd<P>(g, a.coef, key);
            if constexpr (BWD) {
                o[e] = Op::template bwd<P>(g, up[e] * u, a.coef, key);
                du[e] = up[e] * f;
                h[e] = f * u;
            } else {
                o[e] = f * u;
            }
        }
        const int left = a.p.rows - c;
        if (row < a.q.rows && c < a.out_cols) {
            if constexpr (BWD) {
                // The workspace's rows are padded: zeros past the last unit.
                if (left < 8)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        o[e] = e < left ? o[e] : 0.0f;
                        du[e] = e < left ? du[e] : 0.0f;
                    }
                Eight<T>::store(out0 + c, o);
                Eight<T>::store(out1 + c, du);
                if (a.h)
                    store_some8(outh + c, h, left);
            } else {
                store_some8(out0 + c, o, left);
            }
        }
        if (t % (NT / 4) == NT / 4 - 1) {
            row += 16;
            out0 += 16 * a.ldo[0];
            if constexpr (BWD) {
                out1 += 16 * a.ldo[1];
                if (a.h)
                    outh += 16 * a.ldh;
            }
        }
        __builtin_amdgcn_sched_barrier(0);  // few results at a time
    }
    return key > Op::template rare_thr<P>();
}

// One element of the unit's result, written where it belongs: exactly (with
// the rare branches).  c is below a.out_cols.
template <class Op, typename T, bool BWD>
__device__ __forceinline__ void gate_one(const GemmArgs<T>& a, int64_t m, int c, float g, float u)
{
    constexpr bool P = sizeof(T) == 4;
    if (c >= a.p.rows) {
        if constexpr (BWD) {
            // The workspace's rows are padded: zeros past the last unit.
            a.out[0][m * a.ldo[0] + c] = Elem<T>::put(0.0f);
            a.out[1][m * a.ldo[1] + c] = Elem<T>::put(0.0f);
        }
        return;
    }
    const float f = act_value<Op, P>(g, a.coef);
    if constexpr (BWD) {
        const float d = Elem<T>::get(a.dh[m * a.lddh + c]);
        a.out[0][m * a.ldo[0] + c] = Elem<T>::put(act_slope<Op, P>(g, d * u, a.coef));
        a.out[1][m * a.ldo[1] + c] = Elem<T>::put(d * f);
        if (a.h)
            a.h[m * a.ldh + c] = Elem<T>::put(f * u);
    } else {
        a.out[0][m * a.ldo[0] + c] = Elem<T>::put(f * u);
    }
}

// The same for the activation of the call.
template <typename T, bool BWD>
struct Gate {
    const GemmArgs<T>& a;
    __device__ __forceinline__ void operator()(int64_t m, int c, float g, float u) const
    {
        using namespace meswish;
        if (c >= a.out_cols)
            return;
        switch (a.act) {
        case kRelu:
            return gate_one<ActOp<kRelu>, T, BWD>(a, m, c, g, u);
        case kLeakyRelu:
            return gate_one<ActOp<kLeakyRelu>, T, BWD>(a, m, c, g, u);
        case kSigmoid:
            return gate_one<ActOp<kSigmoid>, T, BWD>(a, m, c, g, u);
        case kTanh:
            return gate_one<ActOp<kTanh>, T, BWD>(a, m, c, g, u);
        case kGeluErf:
            return gate_one<ActOp<kGeluErf>, T, BWD>(a, m, c, g, u);
        case kGeluTanh:
            return gate_one<ActOp<kGeluTanh>, T, BWD>(a, m, c, g, u);
        default:
            return gate_one<ActOp<kSwish>, T, BWD>(a, m, c, g, u);
        }
    }
};

// The whole wave again, four results of a lane at a time and element by element:
// for the activations' rare arguments (GELU below -6, tanh-GELU past |g| = 4.5 in
// binary32 and 10 in bf16; Swish and sigmoid past 86).  What it costs: with g ~ N(0, 1) next to nothing; with
// g ~ N(0, 3^2) nearly every wave comes here (bf16 16384 x 4096 -> 16384, GELU:
// forward 3.18 to 3.97 ms, recomputation 3.66 to 6.66; tanh-GELU 3.17 to 3.98, 3.49
// to 6.82; binary32 8192 x 2048 -> 4096 tanh-GELU 1.91 to 2.01 and 2.03 to 2.44).
// Swish takes no more there than at N(0, 1).
template <class Op, typename T, bool BWD, int MT, int NT>
__device__ __forceinline__ void gate_slow(const GemmArgs<T>& a, int64_t m0, int n0,
                                          const f32x4 (&acc)[MT][NT])
{
    const int l = late_lane();
#pragma unroll 1
    for (int t = 0; t < MT * NT / 2; ++t) {
        const int i = t / (NT / 2), j = t % (NT / 2);  // j: 32 units, then four of eight
        f32x4 g = f32x4{}, u = f32x4{};
#pragma unroll
        for (int k = 0; k < MT * NT / 2; ++k)  // a uniform choice of registers
            if (k == t) {
                g = acc[k / (NT / 2)][k % (NT / 2) / 2 * 4 + k % 2];
                u = acc[k / (NT / 2)][k % (NT / 2) / 2 * 4 + 2 + k % 2];
            }
        const int64_t m = m0 + l % 16 + 16 * i;
        const int n = n0 + 8 * (l / 16) + 32 * (j / 2) + 4 * (j % 2);
        if (m >= a.q.rows)
            continue;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < a.out_cols)
                gate_one<Op, T, BWD>(a, m, n + e, g[e], u[e]);
    }
}

template <class Op, typename T, bool BWD, int MT, int NT>
__device__ __forceinline__ void gate(const GemmArgs<T>& a, int64_t m0, int n0,
                                     const f32x4 (&acc)[MT][NT])
{
    if (__any(gate_fast<Op, T, BWD>(a, m0, n0, acc)))
        gate_slow<Op, T, BWD>(a, m0, n0, acc);
}

// n0: the wave's first column of P's rows (kUp) or of the result.
template <typename T, int MODE, bool BWD, bool PARTS, int MT, int NT>
__device__ __forceinline__ void epilogue(const GemmArgs<T>& a, int64_t m0, int n0, int plane,
                                         const f32x4 (&acc)[MT][NT])
{
    if constexpr (PARTS) {
        const int64_t part = (int64_t)blockIdx.y * (MODE == kDw ? 2 : 1) + plane;
        store_results<MODE == kUp>(a.part + part * a.q.rows * a.part_ld, a.part_ld, a.q.rows,
                                   a.part_ld, m0, n0, acc);
    } else if constexpr (MODE != kUp) {
        store_results<false>(plane ? a.out[1] : a.out[0], plane ? a.ldo[1] : a.ldo[0], a.q.rows,
                             a.out_cols, m0, n0, acc);
    } else {
        n0 /= 2;
        using namespace meswish;
        switch (a.act) {
        case kRelu:
            gate<ActOp<kRelu>, T, BWD>(a, m0, n0, acc);
            break;
        case kLeakyRelu:
            gate<ActOp<kLeakyRelu>, T, BWD>(a, m0, n0, acc);
            break;
        case kSigmoid:
            gate<ActOp<kSigmoid>, T, BWD>(a, m0, n0, acc);
            break;
        case kTanh:
            gate<ActOp<kTanh>, T, BWD>(a, m0, n0, acc);
            break;
        case kGeluErf:
            gate<ActOp<kGeluErf>, T, BWD>(a, m0, n0, acc);
            break;
        case kGeluTanh:
            gate<ActOp<kGeluTanh>, T, BWD>(a, m0, n0, acc);
            break;
        default:
            gate<ActOp<kSwish>, T, BWD>(a, m0, n0, acc);
            break;
        }
    }
}

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
__device__ __forceinline__ void part_of_sum(int splits, int& first, int& total)
{
    const int whole = total, y = blockIdx.y;
    first = (int)((int64_t)whole * y / splits);
    total = (int)((int64_t)whole * (y + 1) / splits);
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

template <typename T, int MODE, bool BWD, int WM, int WN, int MT, int NT, bool PARTS>
__global__ __launch_bounds__(WM * WN * 64, 2) void gemm_fast_kernel(const GemmArgs<T> a)
{
    constexpr bool PK = MODE == kUp, QK = MODE != kDw;
    constexpr int BM = WM * MT * 16, BN = WN * NT * 16, WAVES = WM * WN;
    using PT = FastTile<T, PK, PK, BN, WAVES>;
    using QT = FastTile<T, QK, false, BM, WAVES>;
    constexpr int kK = PT::kK, E = Elem<T>::kPerVec, STEPS = KB / 64;
    constexpr int kStage = PT::kBytes + QT::kBytes;
    __shared__ __attribute__((aligned(1024))) char lds[2 * kStage];
    const uint32_t lds0 = (uint32_t)(uintptr_t)(MEBLOCK_LDS char*)lds;

    const int tiles = a.tiles_m * a.tiles_n * (MODE == kDw ? 2 : 1);
    const int steps = (a.k + kK - 1) / kK;
    // An empty sum is one step of zeros.
    int first = 0, total = steps == 0 ? 1 : MODE == kDx ? 2 * steps : steps;
    const int whole = total;
    if constexpr (PARTS)
        part_of_sum(a.splits, first, total);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wm = wave / WN * (MT * 16), wn = wave % WN * (NT * 16);

    // The tile whose operands are being loaded: it runs ahead of the one that
    // is multiplied.
    int64_t m0;
    int n0, plane, tm, tn;
    // Offsets of this lane's 16 bytes in each load, from the tile's first
    // element; (kUp) Wu's from Wu's own first row.
    uint32_t offp[PT::kLoads], offq[QT::kLoads];
    auto place_tile = [&](int tile) {
        const int lane = late_lane();
        plane = 0;
        if constexpr (MODE == kDw) {
            tile_of_block(tile, 2 * a.tiles_m, a.tiles_n, tm, tn);
            plane = tm >= a.tiles_m;
            tm -= plane * a.tiles_m;
        } else {
            tile_of_block(tile, a.tiles_m, a.tiles_n, tm, tn);
        }
        m0 = (int64_t)tm * BM;
        n0 = tn * (MODE == kUp ? BN / 2 : BN);
#pragma unroll
        for (int i = 0; i < PT::kLoads; ++i) {
            const int r = PT::row(lane, wave, i), c = PT::chunk(lane, wave, i) * E;
            if constexpr (MODE == kUp) {
                // Rows of the tile: 32 of Wg, 32 of Wu, in turn.
                int n = r / 64 * 32 + r % 32;
                n = n0 + n < a.p.rows ? n : a.p.rows - 1 - n0;
                offp[i] = (uint32_t)((int64_t)n * a.p.ld[r / 32 % 2] + c) * (uint32_t)sizeof(T);
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
    // (kUp) A wave loads 32 rows of P, all of one weight.
    static_assert(MODE != kUp || PT::kLoads * 1024 == 32 * KB, "waves in turn");
    auto start = [&](int seg) {
        if constexpr (MODE == kUp) {
            const bool up = wave % 2;
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
    int ahead = first, tile_ahead = blockIdx.x;  // the step whose loads come next
    auto next_step = [&]() {
        if (ahead == total) {
            ahead = first;
            tile_ahead += gridDim.x;
        }
        // Past the last tile nothing is read (zeros are written).
        const bool any = tile_ahead < tiles;
        const bool some = any && a.k > 0;
        if (ahead == first && any) {
            place_tile(tile_ahead);
            start(MODE == kDx && first >= steps && steps > 0);
            if constexpr (PARTS) {
                const int64_t skip = MODE == kDx && first >= steps ? first - steps : first;
                curp += skip * incp;
                curq += skip * incq;
                if constexpr (!PK)
                    leftp -= skip * incp;
                if constexpr (!QK)
                    leftq -= skip * incq;
            }
        } else if (MODE == kDx && ahead == steps && any) {
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
        if constexpr (MODE == kUp) {
            // A last step that is cut short: chunks past the end are pointed
            // outside; the next tile has offsets of its own.
            if (ahead == whole - 1 && a.k % kK) {
                const int k0 = ahead * kK, lane = late_lane();
#pragma unroll
                for (int i = 0; i < PT::kLoads; ++i)
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
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        int om, on, op = 0;  // this tile's place in the output
        if constexpr (MODE == kDw) {
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
                        constexpr int kP = MT > NT ? 1 : 2;  // P's fragments a row
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
        epilogue<T, MODE, BWD, PARTS>(a, (int64_t)om * BM + wm, on * BN + wn, op, acc);
    }
    wait_loads<0>();  // no load writes LDS after the block has ended
}

// ---------------------------------------------------------------------------
// Few tokens: the weights are read once, and their bytes bound the time.  A
// block takes 16 PT hidden units and all (at most 16 QT) tokens; its NW waves
// take a share of the sum each, load the weights' fragments from memory
// straight into registers (16 bytes a lane at element alignment, U steps in
// flight) with x's fragments beside them (from the caches), and add their
// parts through LDS in the order of the wave.  bf16 4096 -> 16384 (268 MB of
// weights): 1 token 49 us, 24 tokens 56 (5.5 and 4.8 TB/s) where the weights come
// from memory; 43 and 51 called again on the same weights, of which the 256 MB
// Infinity Cache then holds most.
// ---------------------------------------------------------------------------
template <typename T, bool BWD, int PT, int QT, int NW>
__global__ __launch_bounds__(NW * 64) void few_tokens_kernel(const GemmArgs<T> a)
{
    typedef typename Step<T>::Frag Frag;
    constexpr int E = Elem<T>::kPerVec, kK = 64 / sizeof(T), kTiles = 2 * PT * QT;
    constexpr int U = PT * QT > 4 ? 2 : 4;
    __shared__ float part[NW][kTiles][256];
    const int l = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int n0 = blockIdx.x * (16 * PT);
    const int k0 = l / 16 * E;
    const T* w[2][PT];
    const T* x[QT];
#pragma unroll
    for (int j = 0; j < PT; ++j) {
        const int n = n0 + 16 * j + l % 16;
        const int64_t r = n < a.p.rows ? n : a.p.rows - 1;
        w[0][j] = a.p.base[0] + r * a.p.ld[0];
        w[1][j] = a.p.base[1] + r * a.p.ld[1];
    }
#pragma unroll
    for (int i = 0; i < QT; ++i) {
        const int m = 16 * i + l % 16;
        x[i] = a.q.base[0] + (m < a.q.rows ? m : a.q.rows - 1) * a.q.ld[0];
    }
    f32x4 acc[2][PT][QT];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < PT; ++j)
#pragma unroll
            for (int i = 0; i < QT; ++i)
                acc[h][j][i] = f32x4{};
    // N steps from k, loads first; the last step of the sum may be cut short.
    auto steps = [&](int64_t k, auto count, auto whole) {
        constexpr int N = decltype(count)::value;
        u32x4 fw[N][2][PT], fx[N][QT];
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int64_t kk = k + u * kK + k0;
#pragma unroll
            for (int h = 0; h < 2; ++h)
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
            for (int h = 0; h < 2; ++h)
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
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < PT; ++j)
#pragma unroll
            for (int i = 0; i < QT; ++i)
                *reinterpret_cast<f32x4*>(&part[wave][(h * PT + j) * QT + i][l * 4]) = acc[h][j][i];
    __syncthreads();
    const Gate<T, BWD> gate{a};
    for (int t = threadIdx.x; t < 256 * PT * QT; t += NW * 64) {
        const int n = t % (16 * PT), m = t / (16 * PT);
        const int tile = n / 16 * QT + m / 16, at = (n % 16 / 4 * 16 + m % 16) * 4 + n % 4;
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int v = 0; v < NW; ++v) {
            g += part[v][tile][at];
            u += part[v][PT * QT + tile][at];
        }
        if (m < a.q.rows)
            gate(m, n0 + n, g, u);
    }
}

// ---------------------------------------------------------------------------
// x, Wg and Wu in rows that start on 128-byte boundaries, zeros behind them:
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
__global__ __launch_bounds__(256) void pack_kernel(const PackArgs<T> a)
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
// The parts of a split sum, added in order.
// ---------------------------------------------------------------------------

// dx, dWg, dWu: four columns a thread.
template <typename T, int MODE>
__global__ __launch_bounds__(256) void sum_parts_kernel(const GemmArgs<T> a)
{
    constexpr int kPlanes = MODE == kDw ? 2 : 1;
    const int64_t per_row = a.part_ld / 4, rows = (int64_t)a.q.rows * kPlanes;
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at >= rows * per_row)
        return;
    const int64_t row = at / per_row;
    const int n = (int)(at % per_row) * 4;
    const float* p = a.part + row * a.part_ld + n;
    f32x4 v = f32x4{};
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

// g and u, and the unit: one element a thread.
template <typename T, bool BWD>
__global__ __launch_bounds__(256) void gate_parts_kernel(const GemmArgs<T> a)
{
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t m = at / a.out_cols;
    if (m >= a.q.rows)
        return;
    const int c = (int)(at % a.out_cols);
    const float* p = a.part + m * a.part_ld + c / 32 * 64 + c % 32;
    float g = 0.0f, u = 0.0f;
    for (int s = 0; s < a.splits; ++s) {
        g += p[0];
        u += p[32];
        p += (int64_t)a.q.rows * a.part_ld;
    }
    Gate<T, BWD>{a}(m, c, g, u);
}

// ---------------------------------------------------------------------------
// Host.
// ---------------------------------------------------------------------------

// Coefficients of the activation, in binary64 and split (see Coef): the table of
// meswish.hip, whose counter summaries hold for its exact text (a test compares the
// two).
static Coef make_coef(int act, float p)
{
    const double log2e = 1.44269504088896340735992468100189214;
    const double sqrt_2_over_pi = 0.797884560802865355879892119868763737;
    double c = 0.0;
    switch (act) {
    case MESWISH_ACT_SWISH:
        c = -(double)p * log2e;
        break;
    case MESWISH_ACT_SIGMOID:
        c = -log2e;
        break;
    case MESWISH_ACT_TANH:
        c = -2.0 * log2e;
        break;
    case MESWISH_ACT_GELU_ERF:
        c = -0.5 * log2e;
        break;
    case MESWISH_ACT_GELU_TANH:
        c = -2.0 * sqrt_2_over_pi * log2e;
        break;
    default:
        break;
    }
    const double cubic = 0.044715;
    Coef k;
    k.p = p;
    k.c_hi = (float)c;
    k.c_lo = (float)(c - (double)k.c_hi);
    k.aux_hi = (float)cubic;
    k.aux_lo = (float)(cubic - (double)k.aux_hi);
    return k;
}

static bool act_ok(int act, float param)
{
    if (act < MESWISH_ACT_SWISH || act > MESWISH_ACT_GELU_TANH || !isfinite(param))
        return false;
    // Swish's exponent coefficient must be a finite binary32 value.
    return act != MESWISH_ACT_SWISH || isfinite(make_coef(act, param).c_hi);
}

constexpr size_t kMaxTokens = (size_t)1 << 30;

static bool sizes_ok(size_t tokens, size_t dim, size_t hidden)
{
    return tokens < kMaxTokens && dim <= GATED_FFN_MAX_LD && hidden <= GATED_FFN_MAX_LD;
}

static bool matrix_ok(const void* p, size_t rows, size_t cols, size_t ld, size_t es)
{
    if (ld < cols || ld > GATED_FFN_MAX_LD)
        return false;
    return rows == 0 || cols == 0 || (p && aligned(p, es));
}

static size_t padded(size_t hidden) { return (hidden + 63) / 64 * 64; }

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
static Plan make_plan(int64_t rows, int64_t cols, int64_t k, int planes, int sums, size_t es)
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
static int64_t part_ld(int mode, int64_t cols)
{
    return mode == kUp ? (cols + 63) / 64 * 128 : (cols + 3) / 4 * 4;
}

static size_t part_bytes(int mode, int64_t rows, int64_t cols, int64_t k, size_t es)
{
    const int planes = mode == kDw ? 2 : 1;
    const Plan p = make_plan(rows, mode == kUp ? 2 * cols : cols, k, planes, mode == kDx ? 2 : 1, es);
    return p.splits > 1 ? (size_t)p.splits * planes * rows * part_ld(mode, cols) * sizeof(float) : 0;
}

// Most tokens of the kernel that reads the weights once.  bf16 4096 -> 16384,
// called again on the same weights, against 128 x 128 tiles: 1 token 43 us and 53, 24 tokens 50 and 57, 48 tokens
// 58.4 and 58.0, 64 tokens 63.5 and 58.5.  Up to 16 tokens a block has 16 hidden
// units; for more it has 32, so that x's fragments serve twice (24 tokens: 50 us
// against 56 with 16).
constexpr int kFewTokens = 32;

// Blocks that are on the GPU together, by their LDS (160 KiB a CU); a
// multiple of the 8 XCDs.
static int resident_blocks(int lds_bytes) { return kCus * ((160 << 10) / lds_bytes); }

static int launch_over(const void* fn, int64_t n, void** args, hipStream_t stream)
{
    const int64_t grid = (n + 255) / 256;
    if (grid >= ((int64_t)1 << 24))
        return MESWISH_EINVAL;
    return launch(fn, dim3((unsigned)grid), 256, args, stream);
}

// resident > 0: at most so many blocks, each looping over tiles: the next
// tile's first steps then arrive under the epilogue, which in kUp's backward
// moves four times a product's result (bf16 16384 x 4096 x 16384: 1261 TFLOP/s
// against 1219 with a block a tile; forward 1399 either way).  The other
// products' epilogues are short, and a block a tile balances them better
// (dWg and dWu 1307 TFLOP/s against 1253).
template <typename T, int MODE, bool BWD>
static int gemm_launch(GemmArgs<T>& a, const void* fn, int bm, int bn, int block, int resident,
                       hipStream_t stream)
{
    const int cols = MODE == kUp ? bn / 2 : bn;
    a.tiles_m = (a.q.rows + bm - 1) / bm;
    a.tiles_n = (a.out_cols + cols - 1) / cols;
    // The kernel counts tiles in 31 bits; a launch has fewer than 2^32 threads.
    const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n * (MODE == kDw ? 2 : 1);
    if (tiles == 0)
        return MESWISH_OK;
    const int64_t grid = resident && tiles > resident ? resident : tiles;
    if (tiles > ((int64_t)1 << 30) || grid >= ((int64_t)1 << 23))
        return MESWISH_EINVAL;
    void* args[] = {&a};
    int rc = launch(fn, dim3((unsigned)grid, a.splits), block, args, stream);
    if (rc != MESWISH_OK || a.splits == 1)
        return rc;
    if constexpr (MODE == kUp)
        return launch_over(reinterpret_cast<const void*>(&gate_parts_kernel<T, BWD>),
                           (int64_t)a.q.rows * a.out_cols, args, stream);
    else
        return launch_over(reinterpret_cast<const void*>(&sum_parts_kernel<T, MODE>),
                           (int64_t)a.q.rows * (MODE == kDw ? 2 : 1) * (a.part_ld / 4), args,
                           stream);
}

template <typename T, int MODE, bool BWD, int WM, int WN, int MT, int NT, bool PARTS>
static int gemm_fast(GemmArgs<T>& a, hipStream_t stream)
{
    constexpr int kLds = 2 * (WM * MT + WN * NT) * 16 * 128;
    return gemm_launch<T, MODE, BWD>(
        a,
        reinterpret_cast<const void*>(
            &gemm_fast_kernel<T, MODE, BWD && !PARTS, WM, WN, MT, NT, PARTS>),
        WM * MT * 16, WN * NT * 16, WM * WN * 64,
        MODE == kUp && !PARTS ? resident_blocks(kLds) : 0, stream);
}

template <typename T, bool BWD, int PT, int QT>
static int few_tokens(GemmArgs<T>& a, hipStream_t stream)
{
    void* args[] = {&a};
    return launch(reinterpret_cast<const void*>(&few_tokens_kernel<T, BWD, PT, QT, 8>),
                  dim3((unsigned)((a.out_cols + 16 * PT - 1) / (16 * PT))), 512, args, stream);
}

// part: memory for the parts of a split sum; k: the length that the plan (and
// the size of that memory) goes by.
template <typename T, int MODE, bool BWD>
static int gemm_run(GemmArgs<T>& a, int64_t k, float* part, hipStream_t stream)
{
    a.splits = 1;
    if (a.q.rows == 0 || a.out_cols == 0)
        return MESWISH_OK;
    if constexpr (MODE == kUp) {
        if (a.q.rows <= kFewTokens)
            return a.q.rows <= 16 ? few_tokens<T, BWD, 1, 1>(a, stream)
                                  : few_tokens<T, BWD, 2, 2>(a, stream);
    }
    // kUp's result is as wide as the workspace's rows; the plan goes by the
    // hidden units.
    const int64_t cols = MODE == kUp ? a.p.rows : a.out_cols;
    const Plan p = make_plan(a.q.rows, MODE == kUp ? 2 * cols : cols, k, MODE == kDw ? 2 : 1,
                             MODE == kDx ? 2 : 1, sizeof(T));
    a.splits = p.splits;
    a.part = part;
    a.part_ld = (int)part_ld(MODE, cols);
    if (p.big)
        return p.splits > 1 ? gemm_fast<T, MODE, BWD, 2, 4, 8, 4, true>(a, stream)
                            : gemm_fast<T, MODE, BWD, 2, 4, 8, 4, false>(a, stream);
    return p.splits > 1 ? gemm_fast<T, MODE, BWD, 2, 2, 4, 4, true>(a, stream)
                        : gemm_fast<T, MODE, BWD, 2, 2, 4, 4, false>(a, stream);
}

template <typename T>
static Operand<T> operand(const void* a, int64_t lda, const void* b, int64_t ldb, size_t rows)
{
    return Operand<T>{{static_cast<const T*>(a), static_cast<const T*>(b)}, {lda, ldb}, (int)rows};
}

// Every row of x, wg and wu starts on a 16-byte boundary and is whole vectors
// long, and one row distance serves both weights.
static bool aligned_rows(const void* x, size_t ldx, const void* wg, size_t ldwg, const void* wu,
                         size_t ldwu, size_t dim, size_t es)
{
    return dim * es % 16 == 0 && aligned(x, 16) && aligned(wg, 16) && aligned(wu, 16) &&
           ldx * es % 16 == 0 && ldwg * es % 16 == 0 && ldwg == ldwu;
}

static size_t packed_ld(size_t dim, size_t es) { return (dim * es + 127) / 128 * 128 / es; }

// The workspace: dg and du (backward), the packed operands (where rows are not
// aligned), the parts of one split sum at a time.  Each is whole 128-byte lines
// long.
struct Space {
    size_t grads, packed, part;
    size_t bytes() const { return grads + packed + part; }
};

static size_t lines(size_t bytes) { return (bytes + 127) / 128 * 128; }

static Space space(size_t tokens, size_t dim, size_t hidden, size_t es, bool backward, bool aligned)
{
    const int64_t m = (int64_t)tokens, d = (int64_t)dim, f = (int64_t)hidden;
    const bool few = tokens <= (size_t)kFewTokens;
    Space s{};
    // The kernel for few tokens takes any rows.
    if (!aligned && (backward || !few))
        s.packed = (tokens + 2 * hidden) * packed_ld(dim, es) * es;
    s.part = few ? 0 : part_bytes(kUp, m, f, d, es);
    if (backward) {
        s.grads = lines(2 * tokens * padded(hidden) * es);
        const size_t dx = part_bytes(kDx, m, d, f, es), dw = part_bytes(kDw, f, d, m, es);
        s.part = s.part > dx ? s.part : dx;
        s.part = s.part > dw ? s.part : dw;
    }
    return s;
}

// x, wg and wu as the products take them: as they are, or packed.
template <typename T>
struct Inputs {
    const T *x, *wg, *wu;
    int64_t ldx, ldg, ldu;
    int dim;  // in whole vectors, zeros behind the caller's (packed)

    int pack(T* to, size_t tokens, size_t hidden, hipStream_t stream)
    {
        constexpr int E = Elem<T>::kPerVec;
        const int64_t ld = (int64_t)packed_ld((size_t)dim, sizeof(T));
        PackArgs<T> a{{x, wg, wu},
                      {ldx, ldg, ldu},
                      {(int64_t)tokens, (int64_t)hidden, (int64_t)hidden},
                      to,
                      dim,
                      (int)ld,
                      0};
        while (a.row_bits < 8 && (E << a.row_bits) < ld)
            ++a.row_bits;
        x = to;
        wg = x + tokens * ld;
        wu = wg + hidden * ld;
        ldx = ldg = ldu = ld;
        dim = (dim + E - 1) / E * E;
        const int64_t rows = (int64_t)(tokens + 2 * hidden);
        if (rows == 0 || ld == 0)
            return MESWISH_OK;
        const int64_t blocks = ((rows << a.row_bits) + 255) / 256;
        void* args[] = {&a};
        return launch(reinterpret_cast<const void*>(&pack_kernel<T>),
                      dim3((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20)), 256, args, stream);
    }
};

// What a call was given, checked.
struct Call {
    int act;
    float param;
    const void *x, *wg, *wu, *dh;
    int64_t ldx, ldg, ldu, lddh;
    size_t tokens, dim, hidden;
    void *dx, *dwg, *dwu, *h;
    int64_t lddx, lddwg, lddwu, ldh;
    char* workspace;
    Space space;
    hipStream_t stream;
};

template <typename T, bool BWD>
static int run(const Call& c)
{
    Inputs<T> in{static_cast<const T*>(c.x),
                 static_cast<const T*>(c.wg),
                 static_cast<const T*>(c.wu),
                 c.ldx,
                 c.ldg,
                 c.ldu,
                 (int)c.dim};
    Inputs<T> as_given = in;
    float* part = reinterpret_cast<float*>(c.workspace + c.space.grads + c.space.packed);
    int rc = MESWISH_OK;
    if (c.space.packed)
        rc = in.pack(reinterpret_cast<T*>(c.workspace + c.space.grads), c.tokens, c.hidden, c.stream);
    if (rc != MESWISH_OK)
        return rc;
    const Inputs<T>& up = c.tokens <= (size_t)kFewTokens ? as_given : in;
    const int64_t fp = (int64_t)padded(c.hidden);
    T* dg = reinterpret_cast<T*>(c.workspace);
    T* du = dg + (int64_t)c.tokens * fp;
    GemmArgs<T> a{};
    a.p = operand<T>(up.wg, up.ldg, up.wu, up.ldu, c.hidden);
    a.q = operand<T>(up.x, up.ldx, up.x, up.ldx, c.tokens);
    a.k = up.dim;
    a.act = c.act;
    a.coef = make_coef(c.act, c.param);
    if constexpr (!BWD) {
        a.out[0] = static_cast<T*>(c.h);
        a.ldo[0] = c.ldh;
        a.out_cols = (int)c.hidden;
        return gemm_run<T, kUp, false>(a, (int64_t)c.dim, part, c.stream);
    }
    a.out[0] = dg;
    a.out[1] = du;
    a.ldo[0] = a.ldo[1] = fp;
    a.out_cols = (int)fp;
    a.dh = static_cast<const T*>(c.dh);
    a.lddh = c.lddh;
    a.h = static_cast<T*>(c.h);
    a.ldh = c.ldh;
    rc = gemm_run<T, kUp, true>(a, (int64_t)c.dim, part, c.stream);
    if (rc == MESWISH_OK && c.dx) {
        GemmArgs<T> b{};
        b.p = operand<T>(in.wg, in.ldg, in.wu, in.ldu, (size_t)in.dim);
        b.q = operand<T>(dg, fp, du, fp, c.tokens);
        b.k = (int)c.hidden;
        b.out[0] = static_cast<T*>(c.dx);
        b.ldo[0] = c.lddx;
        b.out_cols = (int)c.dim;
        rc = gemm_run<T, kDx, false>(b, (int64_t)c.hidden, part, c.stream);
    }
    if (rc == MESWISH_OK && c.dwg) {
        GemmArgs<T> b{};
        b.p = operand<T>(in.x, in.ldx, in.x, in.ldx, (size_t)in.dim);
        b.q = operand<T>(dg, fp, du, fp, c.hidden);
        b.k = (int)c.tokens;
        b.q_cols = (int)fp;
        b.out[0] = static_cast<T*>(c.dwg);
        b.out[1] = static_cast<T*>(c.dwu);
        b.ldo[0] = c.lddwg;
        b.ldo[1] = c.lddwu;
        b.out_cols = (int)c.dim;
        rc = gemm_run<T, kDw, false>(b, (int64_t)c.tokens, part, c.stream);
    }
    return rc;
}

template <bool BWD>
static int run_dtype(int dtype, const Call& c)
{
    return dtype == MESWISH_F32 ? run<float, BWD>(c) : run<bf16_t, BWD>(c);
}

// No output touches an input or another output.
static int apart(const Span* out, int nout, const Span* in, int nin)
{
    for (int o = 0; o < nout; ++o) {
        for (int i = 0; i < nin; ++i)
            if (overlaps(out[o], in[i]))
                return MESWISH_EALIAS;
        for (int i = 0; i < o; ++i)
            if (overlaps(out[o], out[i]))
                return MESWISH_EALIAS;
    }
    return MESWISH_OK;
}

}  // namespace meblock

using namespace meblock;

extern "C" size_t gated_ffn_workspace_bytes(size_t tokens, size_t dim, size_t hidden, int dtype,
                                            int backward, int aligned)
{
    if (!dtype_ok(dtype) || !sizes_ok(tokens, dim, hidden))
        return 0;
    const size_t es = elem_size(dtype);
    return space(tokens, dim, hidden, es, backward != 0, aligned && dim * es % 16 == 0).bytes();
}

extern "C" int gated_ffn_fwd(int act, float param, const void* x, size_t ldx, const void* wg,
                             size_t ldwg, const void* wu, size_t ldwu, size_t tokens, size_t dim,
                             size_t hidden, void* h, size_t ldh, void* workspace,
                             size_t workspace_bytes, int dtype, void* stream)
{
    if (!dtype_ok(dtype) || !act_ok(act, param) || !sizes_ok(tokens, dim, hidden))
        return MESWISH_EINVAL;
    const size_t es = elem_size(dtype);
    if (!matrix_ok(x, tokens, dim, ldx, es) || !matrix_ok(wg, hidden, dim, ldwg, es) ||
        !matrix_ok(wu, hidden, dim, ldwu, es) || !matrix_ok(h, tokens, hidden, ldh, es))
        return MESWISH_EINVAL;
    const Space sp = space(tokens, dim, hidden, es, false,
                           aligned_rows(x, ldx, wg, ldwg, wu, ldwu, dim, es));
    const size_t need = sp.bytes();
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
        return MESWISH_EINVAL;
    const Span in[] = {span(x, tokens, dim, ldx, es), span(wg, hidden, dim, ldwg, es),
                       span(wu, hidden, dim, ldwu, es)};
    const Span out[] = {span(h, tokens, hidden, ldh, es), span(workspace, need ? 1 : 0, need, need, 1)};
    int rc = apart(out, 2, in, 3);
    if (rc != MESWISH_OK || tokens == 0 || hidden == 0)
        return rc;
    Call c{};
    c.act = act, c.param = param;
    c.x = x, c.wg = wg, c.wu = wu, c.h = h;
    c.ldx = (int64_t)ldx, c.ldg = (int64_t)ldwg, c.ldu = (int64_t)ldwu, c.ldh = (int64_t)ldh;
    c.tokens = tokens, c.dim = dim, c.hidden = hidden;
    c.workspace = static_cast<char*>(workspace);
    c.space = sp;
    c.stream = static_cast<hipStream_t>(stream);
    return run_dtype<false>(dtype, c);
}

extern "C" int gated_ffn_bwd(int act, float param, const void* x, size_t ldx, const void* wg,
                             size_t ldwg, const void* wu, size_t ldwu, const void* dh, size_t lddh,
                             size_t tokens, size_t dim, size_t hidden, void* dx, size_t lddx,
                             void* dwg, size_t lddwg, void* dwu, size_t lddwu, void* h, size_t ldh,
                             void* workspace, size_t workspace_bytes, int dtype, void* stream)
{
    if (!dtype_ok(dtype) || !act_ok(act, param) || !sizes_ok(tokens, dim, hidden) ||
        (dwg == nullptr) != (dwu == nullptr))
        return MESWISH_EINVAL;
    const size_t es = elem_size(dtype);
    if (!matrix_ok(x, tokens, dim, ldx, es) || !matrix_ok(wg, hidden, dim, ldwg, es) ||
        !matrix_ok(wu, hidden, dim, ldwu, es) || !matrix_ok(dh, tokens, hidden, lddh, es) ||
        (dx && !matrix_ok(dx, tokens, dim, lddx, es)) ||
        (dwg && (!matrix_ok(dwg, hidden, dim, lddwg, es) || !matrix_ok(dwu, hidden, dim, lddwu, es))) ||
        (h && !matrix_ok(h, tokens, hidden, ldh, es)))
        return MESWISH_EINVAL;
    const Space sp = space(tokens, dim, hidden, es, true,
                           aligned_rows(x, ldx, wg, ldwg, wu, ldwu, dim, es));
    const size_t need = sp.bytes();
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
        return MESWISH_EINVAL;
    const Span in[] = {span(x, tokens, dim, ldx, es), span(wg, hidden, dim, ldwg, es),
                       span(wu, hidden, dim, ldwu, es), span(dh, tokens, hidden, lddh, es)};
    const Span out[] = {span(dx, dx ? tokens : 0, dim, lddx, es),
                        span(dwg, dwg ? hidden : 0, dim, lddwg, es),
                        span(dwu, dwu ? hidden : 0, dim, lddwu, es),
                        span(h, h ? tokens : 0, hidden, ldh, es),
                        span(workspace, need ? 1 : 0, need, need, 1)};
    int rc = apart(out, 5, in, 4);
    if (rc != MESWISH_OK)
        return rc;
    Call c{};
    c.act = act, c.param = param;
    c.x = x, c.wg = wg, c.wu = wu, c.dh = dh;
    c.ldx = (int64_t)ldx, c.ldg = (int64_t)ldwg, c.ldu = (int64_t)ldwu, c.lddh = (int64_t)lddh;
    c.tokens = tokens, c.dim = dim, c.hidden = hidden;
    c.dx = dx, c.dwg = dwg, c.dwu = dwu, c.h = h;
    c.lddx = (int64_t)lddx, c.lddwg = (int64_t)lddwg, c.lddwu = (int64_t)lddwu, c.ldh = (int64_t)ldh;
    c.workspace = static_cast<char*>(workspace);
    c.space = sp;
    c.stream = static_cast<hipStream_t>(stream);
    return run_dtype<true>(dtype, c);
}
