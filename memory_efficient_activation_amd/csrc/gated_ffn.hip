// gated_ffn.hip -- the gated feed-forward unit of libmeswish for gfx950,
// forward and backward.  Formulas and contracts: include/gated_ffn.h.
//
// The products (products.h), out[m][n] = sum_k Q(m, k) P(n, k):
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


#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "act_coef.h"
#include "gated_ffn.h"
#include "products.h"

namespace meblock {

template <typename T>
struct GemmArgs : Product<T> {  // out: h, or dg and du (columns padded, zeros past p.rows); dx; dWg and dWu
    const T* dh;  // kUp, backward
    int64_t lddh;
    T* h;         // kUp, backward: the forward's result, or NULL
    int64_t ldh;
    int act;
    Coef coef;
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
    Beside<T, MT, NT / 4> d;
    if constexpr (BWD)
        d.load(a.dh, a.lddh, a.q.rows, a.p.rows, m0, n0);
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

template <typename T, int MODE, bool BWD, int WM, int WN, int MT, int NT, bool PARTS>
__global__ __launch_bounds__(WM * WN * 64, 2) void gemm_fast_kernel(const GemmArgs<T> a)
{
    product_tiles<T, MODE, WM, WN, MT, NT, PARTS>(
        a, [&](int64_t m0, int n0, int plane, const f32x4 (&acc)[MT][NT]) {
            epilogue<T, MODE, BWD, PARTS>(a, m0, n0, plane, acc);
        });
}

template <typename T, bool BWD, int PT, int QT, int NW>
__global__ __launch_bounds__(NW * 64) void few_tokens_kernel(const GemmArgs<T> a)
{
    const Gate<T, BWD> gate{a};
    few_tokens<T, 2, PT, QT, NW, 4>(a, [&](int m, int n, const float (&r)[2]) {
        gate(m, n, r[0], r[1]);
    });
}

template <typename T>
__global__ __launch_bounds__(256) void pack_kernel(const PackArgs<T> a)
{
    pack_rows(a);
}

// The parts of a split sum: dx, dWg, dWu.
template <typename T, int MODE>
__global__ __launch_bounds__(256) void sum_parts_kernel(const GemmArgs<T> a)
{
    sum_parts<T, MODE>(a, blockIdx.x);
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

Coef unit_coef(int act, float param) { return make_coef(act, param); }

bool act_ok(int act, float param)
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

// Most tokens of the kernel that reads the weights once.  bf16 4096 -> 16384,
// called again on the same weights, against 128 x 128 tiles: 1 token 43 us and 53, 24 tokens 50 and 57, 48 tokens
// 58.4 and 58.0, 64 tokens 63.5 and 58.5.  Up to 16 tokens a block has 16 hidden
// units; for more it has 32, so that x's fragments serve twice (24 tokens: 50 us
// against 56 with 16).
constexpr int kFewTokens = 32;

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
    int rc = launch_tiles(a, fn, bm, MODE == kUp ? bn / 2 : bn, Form<MODE>::kPlanes, block, resident,
                          stream);
    if (rc != MESWISH_OK || a.splits == 1 || a.tiles_m == 0 || a.tiles_n == 0)
        return rc;
    void* args[] = {&a};
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

// Every row of x, wg and wu starts on a 16-byte boundary and is whole vectors
// long, and one row distance serves both weights.
static bool aligned_rows(const void* x, size_t ldx, const void* wg, size_t ldwg, const void* wu,
                         size_t ldwu, size_t dim, size_t es)
{
    return dim * es % 16 == 0 && aligned(x, 16) && aligned(wg, 16) && aligned(wu, 16) &&
           ldx * es % 16 == 0 && ldwg * es % 16 == 0 && ldwg == ldwu;
}

// The workspace: dg and du (backward), the packed operands (where rows are not
// aligned), the parts of one split sum at a time.  Each is whole 128-byte lines
// long.
struct Space {
    size_t grads, packed, part;
    size_t bytes() const { return grads + packed + part; }
};

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
