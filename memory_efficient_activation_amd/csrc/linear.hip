// linear.hip -- the matrix product with bias, activation and residual in its
// epilogue, for gfx950, forward and backward.  Formulas and contracts:
// include/linear.h.
//
// The products (products.h), out[m][n] = sum_k Q(m, k) P(n, k):
//
//   kLin    z:   P = W (k contiguous), Q = x (k contiguous), k = dim.  The
//        epilogue works on z in the accumulators: y, or dz, is all that is
//        written.
//   kLinDx  dx:  P = W (n contiguous), Q = dz (k contiguous), k = units.
//   kLinDw  dW:  P = x (n contiguous), Q = dz (m contiguous), k = tokens.
//
// dz is written in the tensors' type, also where that is bfloat16: it is the
// next products' operand, which the matrix cores take in that type (half a step,
// 2^-8 of an element at the most; dx and dW are off by 0.0023 of the norm where one
// rounding of the result alone gives 0.0017).  db sums it before that rounding.
// Without an activation dz is dy, read where it is.
//
// What bounds it, bf16: 16384 tokens the matrix cores at the clock the power limit
// leaves (16384 x 16384 -> 4096 with a residual 1.67 to 1.71 ms, 1.29 to 1.32 PFLOP/s,
// cores 70 % busy; 4096 -> 16384 with GELU 1.77 ms; backward 5.45 ms, 1.21 PFLOP/s of
// its three products: recomputation 2.07 ms, 52 % busy, as its epilogue reads dy,
// evaluates f' and writes dz; dx 1.65, dW 1.70); one token HBM (16384 -> 4096, 134 MB:
// 26.5 us); some hundred tokens the launches one after another, of which the backward
// has three to five.  Binary32: its matrix instructions, and counts of tiles just past
// the CUs' (1500 x 1000 -> 2730, 264 tiles of 128 on 256 CUs: in two parts, 528 blocks of
// half the sum and a second launch that reads 33 MB of parts, 115 us; whole, 135; 1536 x
// 1000 -> 2688, 252 tiles, 80).
//
// Two launches are joined where nothing orders them: dx with dW, and whatever is left
// to be added up at the end.

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "act_coef.h"
#include "linear.h"
#include "products.h"

namespace meblock {

namespace {

template <typename T>
struct LinArgs : Product<T> {  // out: y, or dz (columns padded, zeros past p.rows); dx; dW
    const T* bias;  // kLin: or NULL
    const T* r;     // kLin: the residual or NULL; backward: dy
    int64_t ldr;
    int act;
    Coef coef;
    // Backward, or NULL (no db): the waves' column sums of dz, a row of out_cols for
    // each 16 MT tokens (tiles that are no parts); dz in binary32, rows of out_cols.
    float *db, *wide;
};

struct IdentityOp {
    static constexpr bool kHasRare = false;
    template <bool P>
    __device__ static constexpr float rare_thr() { return 1.0f; }
    template <bool BWD, bool P>
    __device__ static bool is_rare(float, const Coef&) { return false; }
    template <bool P>
    __device__ static float fwd(float x, const Coef&, float&) { return x; }
    template <bool P>
    __device__ static float bwd(float, float dy, const Coef&, float&) { return dy; }
    __device__ static float fwd_rare(float x, const Coef&) { return x; }
    __device__ static float bwd_rare(float, float dy, const Coef&) { return dy; }
};

// Calls f with the call's activation.
template <class F>
__device__ __forceinline__ void with_act(int act, const F& f)
{
    using namespace meswish;
    switch (act) {
    case kSwish:
        return f(ActOp<kSwish>());
    case kRelu:
        return f(ActOp<kRelu>());
    case kLeakyRelu:
        return f(ActOp<kLeakyRelu>());
    case kSigmoid:
        return f(ActOp<kSigmoid>());
    case kTanh:
        return f(ActOp<kTanh>());
    case kGeluErf:
        return f(ActOp<kGeluErf>());
    case kGeluTanh:
        return f(ActOp<kGeluTanh>());
    default:
        return f(IdentityOp());
    }
}

// ---------------------------------------------------------------------------
// Epilogue of kLin.
// ---------------------------------------------------------------------------

// One element of y or dz, written where it belongs: exactly (with the rare
// branches).  c is below a.out_cols.  Its value before the rounding.
template <typename T, bool BWD>
__device__ __forceinline__ float lin_one(const LinArgs<T>& a, int64_t m, int c, float z)
{
    constexpr bool P = sizeof(T) == 4;
    T* out = a.out[0] + m * a.ldo[0] + c;
    if (c >= a.p.rows) {
        if constexpr (BWD)  // the workspace's rows are padded: zeros past the last unit
            *out = Elem<T>::put(0.0f);
        return 0.0f;
    }
    if (a.bias)
        z += Elem<T>::get(a.bias[c]);
    const float r = BWD || a.r ? Elem<T>::get(a.r[m * a.ldr + c]) : 0.0f;
    with_act(a.act, [&](auto op) {
        using Op = decltype(op);
        z = BWD ? act_slope<Op, P>(z, r, a.coef) : act_value<Op, P>(z, a.coef);
    });
    if (!BWD)
        z += r;
    *out = Elem<T>::put(z);
    return z;
}

// lin_one, and dz in binary32 where db's sums read it.
template <typename T, bool BWD>
__device__ __forceinline__ void lin_alone(const LinArgs<T>& a, int64_t m, int c, float z)
{
    z = lin_one<T, BWD>(a, m, c, z);
    if (BWD && a.wide)
        a.wide[m * a.out_cols + c] = z;
}

// Sum over the 16 lanes of a row, in every one of them.
__device__ __forceinline__ float sum16(float v)
{
#define LIN_ROR(N)                                                                          \
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(                             \
                                       0, __builtin_bit_cast(int, v), 0x120 + N, 0xf, 0xf, true))
    LIN_ROR(8);
    LIN_ROR(4);
    LIN_ROR(2);
    LIN_ROR(1);
#undef LIN_ROR
    return v;
}

// Eight values of the bias, zeros past its end and where there is none.
template <typename T>
__device__ __forceinline__ void load_bias(const T* bias, int c, int n, float* f)
{
    Eight<T> v;
#pragma unroll
    for (int k = 0; k < Eight<T>::V; ++k)
        v.v[k] = u32x4{0, 0, 0, 0};
    if (bias && c + 8 <= n)
        v.load(bias + c);
    v.values(f);
    if (bias && c + 8 > n)
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (c + e < n)
                f[e] = Elem<T>::get(bias[c + e]);
}

// f(0), f(1), ... f(N - 1), the numbers known to the compiler: a loop that it
// unrolls however long its body is (accumulators in a loop that it does not
// unroll go to scratch memory).
template <class F, int... I>
__device__ __forceinline__ void each(const F& f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>()), ...);
}

// z becomes f(z), or up f'(z), without the activations' rare branches.  True in a
// lane that met an argument of theirs (GELU below -6, Swish past 86, ...).
template <class Op, bool BWD, bool P>
__device__ __forceinline__ bool act8(float* z, const float* up, const Coef& k)
{
    float key = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        z[e] = BWD ? Op::template bwd<P>(z[e], up[e], k, key) : Op::template fwd<P>(z[e], k, key);
    return Op::kHasRare && key > Op::template rare_thr<P>();
}

// A wave's results, in vectors of eight.  The activation is chosen anew for every
// vector: eight copies of what loads and stores around it took more registers
// than there are.  The result has a bit for each vector, (i, b) at i NT / 2 + b, in
// which a lane met a rare argument: lin_rare does those again, to the same places
// (which is why y may not be the residual).  (bf16 16384 x 4096 -> 16384, GELU
// forward: z of standard deviation 1, where it is never needed, 1.68 ms; 1.4, where one
// vector in ten thousand is, 1.72 against 2.12 with whole waves done again; 1.8 1.99,
// 2.1 2.52, and from 2.5 on, where most vectors are, 2.8 to 3.0; the backward then 7.3 to
// 7.5 and not 5.4.  Tanh-GELU the same from a standard deviation of 3 and 4 on, Swish not
// up to 6.  Binary32 4096 x 2048 -> 4096, GELU forward 0.50 to 0.60 ms, backward 2.39 to
// 2.49.)
template <typename T, bool BWD, int MT, int NT>
__device__ __forceinline__ uint32_t lin_results(const LinArgs<T>& a, int64_t m0, int n0,
                                         const f32x4 (&acc)[MT][NT])
{
    constexpr bool P = sizeof(T) == 4;
    constexpr int MH = MT < 16 / (int)sizeof(T) ? MT : 16 / (int)sizeof(T);  // rows of dy or r in flight
    const int l = late_lane();
    uint32_t rare = 0;
    static_assert(MT * NT / 2 <= 32, "a bit a vector");
    each([&](auto group) {
        constexpr int b = decltype(group)::value;
        const int c = n0 + 32 * b + 8 * (l / 16), left = a.p.rows - c;
        int64_t row = m0 + l % 16;
        T* out = a.out[0] + row * a.ldo[0] + c;
        float bias[8];
        load_bias(a.bias, c, a.p.rows, bias);
        float sum[8] = {};
        each([&](auto part) {
            constexpr int i0 = decltype(part)::value * MH;
            Beside<T, MH, 1> d;
            if (BWD || a.r)
                d.load(a.r, a.ldr, a.q.rows, a.p.rows, m0 + 16 * i0, n0 + 32 * b);
#pragma unroll
            for (int t = 0; t < MH; ++t) {
                float o[8], up[8];
                if (BWD || a.r) {
                    d.v[t].values(up);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        up[e] = 0.0f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    o[e] = acc[i0 + t][2 * b + e / 4][e % 4] + bias[e];
                bool met = false;
                with_act(a.act, [&](auto op) { met = act8<decltype(op), BWD, P>(o, up, a.coef); });
                const bool again = __any(met);
                rare |= again ? 1u << ((i0 + t) * (NT / 2) + b) : 0u;
                if constexpr (!BWD)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        o[e] += up[e];
                if (row < a.q.rows && c < a.out_cols) {
                    if constexpr (BWD) {
                        // The workspace's rows are padded: zeros past the last unit.
                        if (left < 8)
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                o[e] = e < left ? o[e] : 0.0f;
                        Eight<T>::store(out, o);
                        if (!again)
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                sum[e] += o[e];
                    } else {
                        store_some8(out, o, left);
                    }
                }
                row += 16;
                out += 16 * a.ldo[0];
                __builtin_amdgcn_sched_barrier(0);  // few results at a time
            }
        }, std::make_integer_sequence<int, MT / MH>());
        if (BWD && a.db) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum[e] = sum16(sum[e]);
            if (l % 16 == 0 && c < a.out_cols)
                Eight<float>::store(a.db + m0 / (16 * MT) * a.out_cols + c, sum);
        }
    }, std::make_integer_sequence<int, NT / 2>());
    return rare;
}

// The vectors named by `rare` again, element by element.
template <typename T, bool BWD, int MT, int NT>
__device__ __forceinline__ void lin_rare(const LinArgs<T>& a, int64_t m0, int n0,
                                         const f32x4 (&acc)[MT][NT], uint32_t rare)
{
    const int l = late_lane();
#pragma unroll 1
    for (int t = 0; t < MT * NT; ++t) {
        if (!(rare >> (t / 2) & 1))
            continue;
        const int i = t / NT, j = t % NT;
        f32x4 z = f32x4{};
#pragma unroll
        for (int k = 0; k < MT * NT; ++k)  // a uniform choice of registers
            if (k == t)
                z = acc[k / NT][k % NT];
        const int64_t m = m0 + l % 16 + 16 * i;
        const int n = n0 + 32 * (j / 2) + 8 * (l / 16) + 4 * (j % 2);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            z[e] = m < a.q.rows && n + e < a.out_cols ? lin_one<T, BWD>(a, m, n + e, z[e]) : 0.0f;
        if (BWD && a.db) {
            // The row's own thread wrote the sum that these belong to.
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float v = sum16(z[e]);
                if (l % 16 == 0 && n + e < a.out_cols)
                    a.db[m0 / (16 * MT) * a.out_cols + n + e] += v;
            }
        }
    }
}

template <typename T, int MODE, bool BWD, bool PARTS, int MT, int NT>
__device__ __forceinline__ void lin_epilogue(const LinArgs<T>& a, int part, int64_t m0, int n0,
                                             const f32x4 (&acc)[MT][NT])
{
    if constexpr (PARTS) {
        store_results<MODE == kLin>(a.part + (int64_t)part * a.q.rows * a.part_ld, a.part_ld,
                                    a.q.rows, a.part_ld, m0, n0, acc);
    } else if constexpr (MODE != kLin) {
        store_results<false>(a.out[0], a.ldo[0], a.q.rows, a.out_cols, m0, n0, acc);
    } else {
        const uint32_t rare = lin_results<T, BWD>(a, m0, n0, acc);
        if (rare)
            lin_rare<T, BWD>(a, m0, n0, acc, rare);
    }
}

template <typename T, int MODE, bool BWD, int WM, int WN, int MT, int NT, bool PARTS, class Place>
__device__ __forceinline__ void lin_tiles_of(const LinArgs<T>& a, const Place at)
{
    product_tiles<T, MODE, WM, WN, MT, NT, PARTS>(
        a,
        [&](int64_t m0, int n0, int, const f32x4 (&acc)[MT][NT]) {
            lin_epilogue<T, MODE, BWD, PARTS>(a, at.part(), m0, n0, acc);
        },
        at);
}

template <typename T, int MODE, bool BWD, int WM, int WN, int MT, int NT, bool PARTS>
__global__ __launch_bounds__(WM * WN * 64, 2) void lin_tiles_kernel(const LinArgs<T> a)
{
    lin_tiles_of<T, MODE, BWD, WM, WN, MT, NT, PARTS>(a, OwnPlace());
}

// dx and dW by one launch, where both are made of 128 x 128 tiles: the blocks of
// dx, part after part, then those of dW.  (Backward, bf16, against a launch each:
// 100 x 1000 -> 1000, GELU 25.6 us and 28.2, 500 x 2000 -> 1000 20.1 and 30.0, 2000 x
// 2048 -> 2048, GELU 85 and 100, 6000 x 1000 -> 1000, GELU 87 and 91.)
template <typename T>
struct PairArgs {
    LinArgs<T> dx, dw;
    int dx_blocks;
};

template <typename T, bool DX_PARTS, bool DW_PARTS>
__global__ __launch_bounds__(256, 2) void lin_pair_kernel(const PairArgs<T> a)
{
    const int block = blockIdx.x;
    if (block < a.dx_blocks) {
        const int tiles = a.dx.tiles_m * a.dx.tiles_n;
        lin_tiles_of<T, kLinDx, false, 2, 2, 4, 4, DX_PARTS>(
            a.dx, GivenPlace{block % tiles, tiles, block / tiles});
    } else {
        const int tiles = a.dw.tiles_m * a.dw.tiles_n, b = block - a.dx_blocks;
        lin_tiles_of<T, kLinDw, false, 2, 2, 4, 4, DW_PARTS>(
            a.dw, GivenPlace{b % tiles, tiles, b / tiles});
    }
}

// 16 units a block, 16 waves with a share of the sum each.  (bf16 1 x 16384 -> 4096,
// waves and steps in flight: 16 and 2 27 us, 16 and 4 31, 8 and 4 34, 16 and 1 31, 8 and
// 2 33; 32 units a block 41.  5.0 TB/s; 1 x 4096 -> 16384 24 us, 5.6 TB/s.)
constexpr int kFewWaves = 16;

template <typename T, bool BWD, int QT>
__global__ __launch_bounds__(kFewWaves * 64) void lin_few_kernel(const LinArgs<T> a)
{
    few_tokens<T, 1, 1, QT, kFewWaves, 2>(a, [&](int m, int n, const float (&r)[1]) {
        if (n < a.out_cols)
            lin_alone<T, BWD>(a, m, n, r[0]);
    });
}

// The parts of a split sum: z, one element a thread.
template <typename T, bool BWD>
__global__ __launch_bounds__(256) void lin_parts_kernel(const LinArgs<T> a)
{
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t m = at / a.out_cols;
    if (m >= a.q.rows)
        return;
    const int c = (int)(at % a.out_cols);
    float z = 0.0f;
    if (c < a.p.rows) {
        const float* p = a.part + m * a.part_ld + c;
#pragma unroll 4  // four loads in flight
        for (int s = 0; s < a.splits; ++s) {
            z += *p;
            p += (int64_t)a.q.rows * a.part_ld;
        }
    }
    lin_alone<T, BWD>(a, m, c, z);
}

template <typename T>
__global__ __launch_bounds__(256) void lin_pack_kernel(const PackArgs<T> a)
{
    pack_rows(a);
}

// ---------------------------------------------------------------------------
// db: column sums of dz before its rounding, and what ends the backward.
//
// The epilogue of tiles leaves a row of sums for each wave's tokens; elsewhere (a
// split sum, few tokens, dy itself) dz's rows are read again, and where they are many
// first added up to shares: a block takes 64 vectors of columns and a share of the
// rows, one row a wave, and its waves' sums meet in LDS.  The last launch adds what
// there is to be added: the parts of dx and dW, and db's rows or shares, 64
// columns a block.
// ---------------------------------------------------------------------------
template <typename T>
struct ColArgs {
    const T* d;
    int64_t ld, rows;
    int cols;
    float* part;  // [shares][cols]
    int shares;
};

constexpr int kColUnroll = 8;  // rows of a thread in flight

// s += the rows from `row` on, `step` apart, of the vector of columns at e0.
template <typename T>
__device__ __forceinline__ void add_rows(const T* d, int64_t ld, int64_t row, int64_t end, int step,
                                         int e0, int cols, float* s)
{
    constexpr int E = Elem<T>::kPerVec, U = kColUnroll;
    for (; row + (U - 1) * step < end; row += U * step) {
        u32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            v[u] = load_chunk(d + (row + u * step) * ld, e0, cols);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[E];
            Elem<T>::unpack(v[u], f);
#pragma unroll
            for (int j = 0; j < E; ++j)
                s[j] += f[j];
        }
    }
    for (; row < end; row += step) {
        float f[E];
        Elem<T>::unpack(load_chunk(d + row * ld, e0, cols), f);
#pragma unroll
        for (int j = 0; j < E; ++j)
            s[j] += f[j];
    }
}

template <typename T>
__global__ __launch_bounds__(256) void lin_cols_kernel(const ColArgs<T> a)
{
    constexpr int E = Elem<T>::kPerVec;
    __shared__ float lds[4][64 * E];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int e0 = (blockIdx.x * 64 + lane) * E;
    const int64_t first = a.rows * blockIdx.y / a.shares, end = a.rows * (blockIdx.y + 1) / a.shares;
    float s[E] = {};
    if (e0 < a.cols)
        add_rows(a.d, a.ld, first + wave, end, 4, e0, a.cols, s);
#pragma unroll
    for (int j = 0; j < E; ++j)
        lds[wave][lane * E + j] = s[j];
    __syncthreads();
    for (int c = threadIdx.x; c < 64 * E; c += 256) {
        const int col = blockIdx.x * (64 * E) + c;
        if (col < a.cols)
            a.part[(int64_t)blockIdx.y * a.cols + col] =
                (lds[0][c] + lds[1][c]) + (lds[2][c] + lds[3][c]);
    }
}

template <typename T>
struct TailArgs {
    LinArgs<T> dx, dw;
    int dx_blocks, dw_blocks;  // 0: nothing to add
    const void* rows;          // of db's sums
    int64_t ld, count;
    int cols;
    T* db;
};

// R: the type of db's rows.
template <typename T, typename R>
__global__ __launch_bounds__(256) void lin_tail_kernel(const TailArgs<T> a)
{
    constexpr int E = Elem<R>::kPerVec, kLanes = 64 / E, kGroups = 256 / kLanes;
    __shared__ float lds[kGroups][64];
    int block = blockIdx.x;
    if (block < a.dx_blocks) {
        sum_parts<T, kLinDx>(a.dx, block);
        return;
    }
    block -= a.dx_blocks;
    if (block < a.dw_blocks) {
        sum_parts<T, kLinDw>(a.dw, block);
        return;
    }
    block -= a.dw_blocks;
    const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    const int e0 = block * 64 + lane * E;
    float s[E] = {};
    if (e0 < a.cols)
        add_rows(static_cast<const R*>(a.rows), a.ld, group, a.count, kGroups, e0, a.cols, s);
#pragma unroll
    for (int j = 0; j < E; ++j)
        lds[group][lane * E + j] = s[j];
    __syncthreads();
    const int col = block * 64 + threadIdx.x;
    if (threadIdx.x < 64 && col < a.cols) {
        float t = 0.0f;
        for (int g = 0; g < kGroups; ++g)
            t += lds[g][threadIdx.x];
        a.db[col] = Elem<T>::put(t);
    }
}

// ---------------------------------------------------------------------------
// Host.
// ---------------------------------------------------------------------------

constexpr size_t kMaxTokens = (size_t)1 << 30;

bool sizes_ok(size_t tokens, size_t dim, size_t units)
{
    return tokens < kMaxTokens && dim <= LINEAR_MAX_LD && units <= LINEAR_MAX_LD;
}

bool call_ok(int act, float param)
{
    return act == LINEAR_IDENTITY ? isfinite(param) : act_ok(act, param);
}

bool matrix_ok(const void* p, size_t rows, size_t cols, size_t ld, size_t es)
{
    if (ld < cols || ld > LINEAR_MAX_LD)
        return false;
    return rows == 0 || cols == 0 || (p && aligned(p, es));
}

bool rows_aligned(const void* p, size_t ld, size_t cols, size_t es)
{
    return aligned(p, 16) && ld * es % 16 == 0 && cols * es % 16 == 0;
}

// Whether z is computed by the kernel that reads the weight once, which takes any
// rows.  Each of its blocks reads all of x, from the caches; tiles read x less
// often, but split the sum and add its parts by a second kernel.  bf16, tokens x dim
// -> units, with x times blocks:
//   1 x 16384 -> 4096 (8 MB) 27 us against 35; 8 x 16384 -> 4096 (67 MB) 29 against
//   35; 32 x 4096 -> 4096 (67 MB) 14.0 against 15.6; 16 x 16384 -> 4096 (134 MB) 36
//   against 35.5; 24 x 4096 -> 16384 (201 MB) 44 against 31.5; 32 x 16384 -> 4096
//   (268 MB) 53 against 37.
// Rows that are not aligned would have to be copied for the tiles, the weight's too.
bool few_tokens_call(size_t tokens, size_t dim, size_t units, size_t es, bool aligned)
{
    return tokens <= 32 &&
           (!aligned || tokens * dim * es * ((units + 15) / 16) <= ((size_t)80 << 20));
}

// Shares of the rows in db's sums: about four blocks a CU, 32 rows a share at
// the least.
int col_shares(int64_t rows, int64_t cols, size_t es)
{
    const int64_t blocks = (cols * (int64_t)es + 1023) / 1024;
    int64_t s = (4 * kCus + blocks - 1) / (blocks ? blocks : 1);
    const int64_t most = (rows + 31) / 32;
    s = s < most ? s : most;
    return (int)(s < 1 ? 1 : s);
}

template <typename T, bool BWD, int QT>
int lin_few(LinArgs<T>& a, hipStream_t stream)
{
    void* args[] = {&a};
    return launch(reinterpret_cast<const void*>(&lin_few_kernel<T, BWD, QT>),
                  dim3((unsigned)((a.out_cols + 15) / 16)), kFewWaves * 64, args, stream);
}

template <typename T, int MODE, bool BWD, int WM, int WN, int MT, int NT, bool PARTS>
int lin_tiles(LinArgs<T>& a, hipStream_t stream)
{
    constexpr int kLds = 2 * (WM * MT + WN * NT) * 16 * 128;
    int rc = launch_tiles(
        a,
        reinterpret_cast<const void*>(
            &lin_tiles_kernel<T, MODE, BWD && !PARTS, WM, WN, MT, NT, PARTS>),
        WM * MT * 16, WN * NT * 16, 1, WM * WN * 64,
        MODE == kLin && !PARTS ? resident_blocks(kLds) : 0, stream);
    if (rc != MESWISH_OK || !PARTS)
        return rc;
    void* args[] = {&a};
    if constexpr (MODE == kLin)
        rc = launch_over(reinterpret_cast<const void*>(&lin_parts_kernel<T, BWD>),
                         (int64_t)a.q.rows * a.out_cols, args, stream);
    return rc;
}

// Products that share the GPU with dx or dW, for their plans: in binary32 the other
// of the two counts.  (Backward with both counted and each by itself, binary32: 1500 x
// 1000 -> 2730, GELU 278 us and 306, 300 x 1024 -> 1024 30 and 35; bf16: 300 x 1024 ->
// 1024, GELU 32.5 and 28.7, 6000 x 1000 -> 1000, GELU 97.5 and 85, 500 x 2000 -> 1000
// 19.9 and 20.1.)
int products_beside(size_t es, bool both) { return both && es == 4 ? 2 : 1; }

// How a product is computed, and where the parts of its sum go.
template <typename T>
Plan set_plan(LinArgs<T>& a, int mode, int64_t cols, int64_t k, float* part, int beside = 1)
{
    const Plan p = make_plan(a.q.rows, cols, k, beside, 1, sizeof(T));
    a.splits = p.splits;
    a.part = part;
    a.part_ld = (int)part_ld(mode, cols);
    return p;
}

template <typename T, bool DX_PARTS, bool DW_PARTS>
int lin_pair(PairArgs<T>& a, int64_t blocks, hipStream_t stream)
{
    void* args[] = {&a};
    return launch(reinterpret_cast<const void*>(&lin_pair_kernel<T, DX_PARTS, DW_PARTS>),
                  dim3((unsigned)blocks), 256, args, stream);
}

// few: by the kernel that reads the weight once.  (The parts of dx and dW are
// added by the backward's last launch.)
template <typename T, int MODE, bool BWD>
int lin_product(LinArgs<T>& a, bool few, const Plan& p, hipStream_t stream)
{
    if (a.q.rows == 0 || a.out_cols == 0)
        return MESWISH_OK;
    if constexpr (MODE == kLin) {
        if (few)
            return a.q.rows <= 16 ? lin_few<T, BWD, 1>(a, stream) : lin_few<T, BWD, 2>(a, stream);
    }
    if (p.big)
        return p.splits > 1 ? lin_tiles<T, MODE, BWD, 2, 4, 8, 4, true>(a, stream)
                            : lin_tiles<T, MODE, BWD, 2, 4, 8, 4, false>(a, stream);
    return p.splits > 1 ? lin_tiles<T, MODE, BWD, 2, 2, 4, 4, true>(a, stream)
                        : lin_tiles<T, MODE, BWD, 2, 2, 4, 4, false>(a, stream);
}

// dx and dW, either of which may be absent (no out[0]).
template <typename T>
int lin_grads(LinArgs<T>& dx, LinArgs<T>& dw, const Plan& px, const Plan& pw, hipStream_t stream)
{
    auto tiles = [](LinArgs<T>& a) {
        a.tiles_m = (a.q.rows + 127) / 128;
        a.tiles_n = (a.out_cols + 127) / 128;
        return (int64_t)a.tiles_m * a.tiles_n * a.splits;
    };
    if (dx.out[0] && dw.out[0] && !px.big && !pw.big) {
        const int64_t bx = tiles(dx), bw = tiles(dw);
        if (bx > 0 && bw > 0 && bx + bw < ((int64_t)1 << 23)) {
            PairArgs<T> a{dx, dw, (int)bx};
            if (dx.splits > 1)
                return dw.splits > 1 ? lin_pair<T, true, true>(a, bx + bw, stream)
                                     : lin_pair<T, true, false>(a, bx + bw, stream);
            return dw.splits > 1 ? lin_pair<T, false, true>(a, bx + bw, stream)
                                 : lin_pair<T, false, false>(a, bx + bw, stream);
        }
    }
    int rc = MESWISH_OK;
    if (dx.out[0])
        rc = lin_product<T, kLinDx, false>(dx, false, px, stream);
    if (rc == MESWISH_OK && dw.out[0])
        rc = lin_product<T, kLinDw, false>(dw, false, pw, stream);
    return rc;
}

// Rows of the column sums that a wave of tiles leaves, one for its tokens.
size_t wave_rows(size_t tokens, bool big)
{
    const size_t side = big ? 256 : 128;
    return 2 * ((tokens + side - 1) / side);
}

// Most rows that db's last launch adds without shares: a block adds 64 columns of
// them, 16 rows (bfloat16: 32) at a time.  (Backward, bf16, without shares against
// with them: 300 x 1024 -> 1024, GELU 28.8 us and 31.0, 500 x 2000 -> 1000 20.1 and
// 22.4, 1000 x 500 -> 1000 25.2 and 25.5, 2000 x 500 -> 500 59.6 and 29.0.)
constexpr size_t kTailRows = 512;

// The workspace: dz in padded rows (backward with an activation; in bfloat16 calls
// of few tokens or a split sum also in binary32, for db), the packed operands, the
// parts of z's sum or of dx's and dW's, db's sums of waves or its shares.  Each is whole
// 128-byte lines long.
struct Space {
    size_t dz, wide, xw, dy, part, db;
    size_t dw_part;  // where dW's parts are in `part`
    size_t bytes() const { return dz + wide + xw + dy + part + db; }
};

Space space(size_t tokens, size_t dim, size_t units, bool act, size_t es, bool backward, int align)
{
    const int64_t m = (int64_t)tokens, d = (int64_t)dim, f = (int64_t)units;
    const bool few = few_tokens_call(tokens, dim, units, es, align & LINEAR_ALIGNED_XW);
    Space s{};
    if (!(align & LINEAR_ALIGNED_XW) && (backward || !few))
        s.xw = (tokens + units) * packed_ld(dim, es) * es;
    if ((!backward || act) && !few)
        s.part = lines(part_bytes(kLin, m, f, d, es));
    if (backward) {
        const Plan plan = make_plan(m, f, d, 1, 1, es);
        const bool alone = act && (few || plan.splits > 1);
        if (act && !alone)
            s.db = wave_rows(tokens, plan.big) * padded(units) * sizeof(float);
        else
            s.db = (size_t)col_shares(m, f, alone ? sizeof(float) : es) * units * sizeof(float);
        s.db = lines(s.db);
        if (act)
            s.dz = lines(tokens * padded(units) * es);
        else if (!(align & LINEAR_ALIGNED_DY))
            s.dy = tokens * packed_ld(units, es) * es;
        if (alone && es < sizeof(float))
            s.wide = tokens * padded(units) * sizeof(float);
        // Whether one of them is wanted or both.
        auto most = [&](int mode, int64_t rows, int64_t k) {
            size_t parts = 1;
            for (const bool both : {false, true}) {
                const Plan p = make_plan(rows, d, k, products_beside(es, both), 1, es);
                parts = parts > (size_t)p.splits ? parts : (size_t)p.splits;
            }
            return parts > 1 ? lines(parts * rows * part_ld(mode, d) * sizeof(float)) : 0;
        };
        s.dw_part = most(kLinDx, m, f);
        const size_t grads = s.dw_part + most(kLinDw, f, m);
        s.part = s.part > grads ? s.part : grads;
    }
    return s;
}

// Rows of a matrix as the products take them.
template <typename T>
struct Rows {
    const T* p;
    int64_t ld;
    int cols;  // in whole vectors, zeros behind the caller's (packed)
};

// Packs up to two matrices of the same row length, after each other.
template <typename T>
int pack(Rows<T>& a, size_t arows, Rows<T>* b, size_t brows, T* to, hipStream_t stream)
{
    constexpr int E = Elem<T>::kPerVec;
    const int64_t ld = (int64_t)packed_ld((size_t)a.cols, sizeof(T));
    PackArgs<T> args{{a.p, b ? b->p : a.p, a.p},
                     {a.ld, b ? b->ld : a.ld, a.ld},
                     {(int64_t)arows, (int64_t)brows, 0},
                     to,
                     a.cols,
                     (int)ld,
                     0};
    while (args.row_bits < 8 && (E << args.row_bits) < ld)
        ++args.row_bits;
    const int cols = (a.cols + E - 1) / E * E;
    a = Rows<T>{to, ld, cols};
    if (b)
        *b = Rows<T>{to + (int64_t)arows * ld, ld, cols};
    const int64_t rows = (int64_t)(arows + brows);
    if (rows == 0 || ld == 0)
        return MESWISH_OK;
    const int64_t blocks = ((rows << args.row_bits) + 255) / 256;
    void* p[] = {&args};
    return launch(reinterpret_cast<const void*>(&lin_pack_kernel<T>),
                  dim3((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20)), 256, p, stream);
}

// The rows of db's sums: type R, ld elements apart.
template <typename R>
struct ColRows {
    const R* p;
    int64_t ld, count;
};

// Shares of the sums of d's columns.
template <typename R>
int add_up(const ColRows<R>& d, size_t cols, float* part, ColRows<float>& out, hipStream_t stream)
{
    const int shares = col_shares(d.count, (int64_t)cols, sizeof(R));
    out = ColRows<float>{part, (int64_t)cols, shares};
    ColArgs<R> a{d.p, d.ld, d.count, (int)cols, part, shares};
    void* args[] = {&a};
    constexpr int kCols = 64 * Elem<R>::kPerVec;
    return launch(reinterpret_cast<const void*>(&lin_cols_kernel<R>),
                  dim3((unsigned)((cols + kCols - 1) / kCols), (unsigned)shares), 256, args, stream);
}

// The backward's last launch, if there is anything left to add.
template <typename T, typename R>
int lin_tail(const LinArgs<T>& dx, const LinArgs<T>& dw, const ColRows<R>& rows, size_t cols, T* db,
             hipStream_t stream)
{
    auto blocks = [](const LinArgs<T>& a) {
        return a.out[0] && a.splits > 1 ? ((int64_t)a.q.rows * (a.part_ld / 4) + 255) / 256 : 0;
    };
    const int64_t bx = blocks(dx), bw = blocks(dw), bd = db ? (int64_t)(cols + 63) / 64 : 0;
    if (bx + bw + bd == 0)
        return MESWISH_OK;
    if (bx + bw + bd >= ((int64_t)1 << 24))
        return MESWISH_EINVAL;
    TailArgs<T> a{dx, dw, (int)bx, (int)bw, rows.p, rows.ld, rows.count, (int)cols, db};
    void* args[] = {&a};
    return launch(reinterpret_cast<const void*>(&lin_tail_kernel<T, R>),
                  dim3((unsigned)(bx + bw + bd)), 256, args, stream);
}

// What a call was given, checked.
struct Call {
    int act;
    float param;
    const void *x, *w, *bias, *r;  // r: the residual, or dy
    int64_t ldx, ldw, ldr;
    size_t tokens, dim, units;
    void *y, *dx, *dw, *dbias;
    int64_t ldy, lddx, lddw;
    bool few;  // tokens, for the kernel that reads the weight once
    char* workspace;
    Space space;
    hipStream_t stream;
};

template <typename T, bool BWD>
int run(const Call& c)
{
    Rows<T> x{static_cast<const T*>(c.x), c.ldx, (int)c.dim};
    Rows<T> w{static_cast<const T*>(c.w), c.ldw, (int)c.dim};
    const Rows<T> x_given = x, w_given = w;
    const bool few = c.few, act = c.act != LINEAR_IDENTITY;
    const int64_t dim = (int64_t)c.dim, units = (int64_t)c.units;
    char* at = c.workspace;
    T* dz = reinterpret_cast<T*>(at);
    float* wide = reinterpret_cast<float*>(at += c.space.dz);
    T* xw = reinterpret_cast<T*>(at += c.space.wide);
    T* dy = reinterpret_cast<T*>(at += c.space.xw);
    float* part = reinterpret_cast<float*>(at += c.space.dy);
    float* sums = reinterpret_cast<float*>(at += c.space.part);
    int rc = MESWISH_OK;
    // In the backward without an activation x serves dW alone and w dx.
    const bool need_x = !BWD || act || c.dw, need_w = !BWD || act || c.dx;
    if (c.space.xw)
        rc = pack(x, need_x ? c.tokens : 0, &w, need_w ? c.units : 0, xw, c.stream);
    Rows<T> d{static_cast<const T*>(c.r), c.ldr, (int)c.units};
    // db's rows: dy, dz in binary32 calls, or what the product leaves of dz in binary32.
    ColRows<T> rows{d.p, d.ld, (int64_t)c.tokens};
    ColRows<float> wide_rows{};
    bool of_waves = false;
    if (rc == MESWISH_OK && (!BWD || act)) {
        LinArgs<T> a{};
        const Rows<T>&p = few ? w_given : w, &q = few ? x_given : x;
        a.p = operand<T>(p.p, p.ld, p.p, p.ld, c.units);
        a.q = operand<T>(q.p, q.ld, q.p, q.ld, c.tokens);
        a.k = q.cols;
        a.bias = static_cast<const T*>(c.bias);
        a.r = d.p;
        a.ldr = d.ld;
        a.act = c.act;
        if (act)
            a.coef = unit_coef(c.act, c.param);
        const int64_t fp = (int64_t)padded(c.units);
        a.out[0] = BWD ? dz : static_cast<T*>(c.y);
        a.ldo[0] = BWD ? fp : c.ldy;
        a.out_cols = BWD ? (int)fp : (int)c.units;
        const Plan plan = set_plan(a, kLin, units, dim, part);
        if (BWD && c.dbias) {
            if (!few && plan.splits == 1) {
                a.db = sums;
                of_waves = true;
                wide_rows = ColRows<float>{sums, fp, (int64_t)wave_rows(c.tokens, plan.big)};
            } else if (c.space.wide) {
                a.wide = wide;
                wide_rows = ColRows<float>{wide, fp, (int64_t)c.tokens};
            }
        }
        rc = lin_product<T, kLin, BWD>(a, few, plan, c.stream);
        if (BWD) {
            d = Rows<T>{dz, fp, (int)fp};
            rows = ColRows<T>{dz, fp, (int64_t)c.tokens};
        }
    } else if (rc == MESWISH_OK && c.space.dy && (c.dx || c.dw)) {
        rc = pack<T>(d, c.tokens, nullptr, 0, dy, c.stream);
    }
    if constexpr (BWD) {
        LinArgs<T> dx{}, dw{};
        Plan px{}, pw{};
        if (c.dx) {
            dx.p = operand<T>(w.p, w.ld, w.p, w.ld, (size_t)w.cols);
            dx.q = operand<T>(d.p, d.ld, d.p, d.ld, c.tokens);
            dx.k = (int)c.units;
            dx.out[0] = static_cast<T*>(c.dx);
            dx.ldo[0] = c.lddx;
            dx.out_cols = (int)c.dim;
            px = set_plan(dx, kLinDx, dim, units, part, products_beside(sizeof(T), c.dw));
        }
        if (c.dw) {
            dw.p = operand<T>(x.p, x.ld, x.p, x.ld, (size_t)x.cols);
            dw.q = operand<T>(d.p, d.ld, d.p, d.ld, c.units);
            dw.k = (int)c.tokens;
            dw.q_cols = d.cols;
            dw.out[0] = static_cast<T*>(c.dw);
            dw.ldo[0] = c.lddw;
            dw.out_cols = (int)c.dim;
            pw = set_plan(dw, kLinDw, dim, (int64_t)c.tokens, part + c.space.dw_part / sizeof(float),
                          products_beside(sizeof(T), c.dx));
        }
        if (rc == MESWISH_OK)
            rc = lin_grads(dx, dw, px, pw, c.stream);
        T* db = units ? static_cast<T*>(c.dbias) : nullptr;
        if (rc == MESWISH_OK && db && !of_waves && c.tokens > kTailRows) {
            const ColRows<float> given = wide_rows;
            rc = given.p ? add_up(given, c.units, sums, wide_rows, c.stream)
                         : add_up(rows, c.units, sums, wide_rows, c.stream);
        }
        if (rc == MESWISH_OK)
            rc = wide_rows.p ? lin_tail(dx, dw, wide_rows, c.units, db, c.stream)
                             : lin_tail(dx, dw, rows, c.units, db, c.stream);
    }
    return rc;
}

template <bool BWD>
int run_dtype(int dtype, const Call& c)
{
    return dtype == MESWISH_F32 ? run<float, BWD>(c) : run<bf16_t, BWD>(c);
}

}  // namespace

}  // namespace meblock

using namespace meblock;

extern "C" size_t linear_workspace_bytes(size_t tokens, size_t dim, size_t units, int act, int dtype,
                                         int backward, int align)
{
    if (!dtype_ok(dtype) || !sizes_ok(tokens, dim, units) ||
        (act != LINEAR_IDENTITY && !act_ok(act, 1.0f)))
        return 0;
    const size_t es = elem_size(dtype);
    if (dim * es % 16)
        align &= ~LINEAR_ALIGNED_XW;
    if (units * es % 16)
        align &= ~LINEAR_ALIGNED_DY;
    const bool f = act != LINEAR_IDENTITY, bwd = backward != 0;
    const size_t need = space(tokens, dim, units, f, es, bwd, align).bytes();
    if (align & LINEAR_ALIGNED_XW || dim * es % 16)
        return need;
    // The call's rows may turn out aligned, and few tokens then take a split sum.
    const size_t other = space(tokens, dim, units, f, es, bwd, align | LINEAR_ALIGNED_XW).bytes();
    return need > other ? need : other;
}

extern "C" int linear_fwd(int act, float param, const void* x, size_t ldx, const void* w, size_t ldw,
                          const void* bias, const void* residual, size_t ldr, size_t tokens,
                          size_t dim, size_t units, void* y, size_t ldy, void* workspace,
                          size_t workspace_bytes, int dtype, void* stream)
{
    if (!dtype_ok(dtype) || !call_ok(act, param) || !sizes_ok(tokens, dim, units))
        return MESWISH_EINVAL;
    const size_t es = elem_size(dtype);
    if (!matrix_ok(x, tokens, dim, ldx, es) || !matrix_ok(w, units, dim, ldw, es) ||
        !aligned(bias, es) || (residual && !matrix_ok(residual, tokens, units, ldr, es)) ||
        !matrix_ok(y, tokens, units, ldy, es))
        return MESWISH_EINVAL;
    const int align = rows_aligned(x, ldx, dim, es) && rows_aligned(w, ldw, dim, es)
                          ? LINEAR_ALIGNED_XW : 0;
    const Space sp = space(tokens, dim, units, act != LINEAR_IDENTITY, es, false, align);
    const size_t need = sp.bytes();
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
        return MESWISH_EINVAL;
    const Span in[] = {span(x, tokens, dim, ldx, es), span(w, units, dim, ldw, es),
                       span(bias, bias ? 1 : 0, units, units, es),
                       span(residual, residual ? tokens : 0, units, ldr, es)};
    const Span out[] = {span(y, tokens, units, ldy, es), span(workspace, need ? 1 : 0, need, need, 1)};
    const int rc = apart(out, 2, in, 4);
    if (rc != MESWISH_OK || tokens == 0 || units == 0)
        return rc;
    Call c{};
    c.act = act, c.param = param;
    c.x = x, c.w = w, c.bias = bias, c.r = residual, c.y = y;
    c.ldx = (int64_t)ldx, c.ldw = (int64_t)ldw, c.ldr = (int64_t)ldr, c.ldy = (int64_t)ldy;
    c.tokens = tokens, c.dim = dim, c.units = units;
    c.workspace = static_cast<char*>(workspace);
    c.space = sp;
    c.few = few_tokens_call(tokens, dim, units, es, align & LINEAR_ALIGNED_XW);
    c.stream = static_cast<hipStream_t>(stream);
    return run_dtype<false>(dtype, c);
}

extern "C" int linear_bwd(int act, float param, const void* x, size_t ldx, const void* w, size_t ldw,
                          const void* bias, const void* dy, size_t lddy, size_t tokens, size_t dim,
                          size_t units, void* dx, size_t lddx, void* dw, size_t lddw, void* dbias,
                          void* workspace, size_t workspace_bytes, int dtype, void* stream)
{
    if (!dtype_ok(dtype) || !call_ok(act, param) || !sizes_ok(tokens, dim, units))
        return MESWISH_EINVAL;
    const size_t es = elem_size(dtype);
    const bool reads_x = act != LINEAR_IDENTITY || dw;
    if (((reads_x || x) && !matrix_ok(x, tokens, dim, ldx, es)) || !matrix_ok(w, units, dim, ldw, es) ||
        !aligned(bias, es) || !matrix_ok(dy, tokens, units, lddy, es) ||
        (dx && !matrix_ok(dx, tokens, dim, lddx, es)) ||
        (dw && !matrix_ok(dw, units, dim, lddw, es)) || !aligned(dbias, es))
        return MESWISH_EINVAL;
    const int align = ((!x || rows_aligned(x, ldx, dim, es)) && rows_aligned(w, ldw, dim, es)
                           ? LINEAR_ALIGNED_XW : 0) |
                      (rows_aligned(dy, lddy, units, es) ? LINEAR_ALIGNED_DY : 0);
    const Space sp = space(tokens, dim, units, act != LINEAR_IDENTITY, es, true, align);
    const size_t need = sp.bytes();
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
        return MESWISH_EINVAL;
    const Span in[] = {span(x, x ? tokens : 0, dim, ldx, es), span(w, units, dim, ldw, es),
                       span(bias, bias ? 1 : 0, units, units, es), span(dy, tokens, units, lddy, es)};
    const Span out[] = {span(dx, dx ? tokens : 0, dim, lddx, es), span(dw, dw ? units : 0, dim, lddw, es),
                        span(dbias, dbias ? 1 : 0, units, units, es),
                        span(workspace, need ? 1 : 0, need, need, 1)};
    const int rc = apart(out, 4, in, 4);
    if (rc != MESWISH_OK || (!dx && !dw && !dbias))
        return rc;
    Call c{};
    c.act = act, c.param = param;
    c.x = x, c.w = w, c.bias = bias, c.r = dy, c.dx = dx, c.dw = dw, c.dbias = dbias;
    c.ldx = (int64_t)ldx, c.ldw = (int64_t)ldw, c.ldr = (int64_t)lddy, c.lddx = (int64_t)lddx;
    c.lddw = (int64_t)lddw;
    c.tokens = tokens, c.dim = dim, c.units = units;
    c.workspace = static_cast<char*>(workspace);
    c.space = sp;
    c.few = few_tokens_call(tokens, dim, units, es, align & LINEAR_ALIGNED_XW);
    c.stream = static_cast<hipStream_t>(stream);
    return run_dtype<true>(dtype, c);
}
