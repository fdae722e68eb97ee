// residual_norm.hip -- the border between transformer blocks for gfx950: norms
// before and after it, gate, scales and the residual sum in one pass, forward
// and backward.  Formulas and contracts: include/residual_norm.h.
//
// Bound: HBM bandwidth (up to 20 flops an element forward, 35 backward).  Both
// directions read each row once and keep it in registers:
//   * A group of G threads owns a row, thread g the eight columns from 8 (V G) on
//     ...; V is 1 but for the widest rows.  G is 8 to 64 lanes of a wave, or 128 to
//     1024 threads whose sums meet in LDS.
//   * Variances are means of squared differences from the mean, from the
//     registers: no cancellation of E[x^2] - mean^2.
//   * Backward: a thread owns the same columns in every row its block takes, so
//     the five sums over rows stay in registers.  Each block writes one binary32
//     partial per column and sum; a second kernel adds them in a fixed order
//     (no atomics, deterministic).
//   * Where the sums over rows do not fit the registers beside the rows
//     (n > 8192), a kernel of its own takes them, from each row's two means.
//   * Rows past 16384 values are read again for each pass, one block per row.

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "block_common.h"
#include "residual_norm.h"

namespace meblock {

namespace {

constexpr int C = 8;  // columns of a thread and chunk

// ---------------------------------------------------------------------------
// Rows.
// ---------------------------------------------------------------------------

// Eight columns of a row, as loaded.  SMALL: rows may be shorter than a vector.
template <typename T, bool SMALL>
struct Chunk {
    static constexpr int E = Elem<T>::kPerVec, K = C / E;
    u32x4 v[K];
    // Without a branch (load_near); what lies past the row's end is some other
    // value of it.
    __device__ __forceinline__ void load(const T* row, int e0, int n)
    {
#pragma unroll
        for (int k = 0; k < K; ++k)
            v[k] = SMALL ? load_chunk(row, e0 + k * E, n) : load_near(row, e0 + k * E, n);
    }
    // The values, zeros past the row's end.
    __device__ __forceinline__ void values(float* f, int e0, int n) const
    {
#pragma unroll
        for (int k = 0; k < K; ++k)
            Elem<T>::unpack(SMALL ? v[k] : chunk_of<T>(v[k], e0 + k * E, n), f + k * E);
    }
};

template <typename T>
__device__ __forceinline__ void store_row(T* row, int e0, int n, const float* f)
{
    constexpr int E = Elem<T>::kPerVec;
#pragma unroll
    for (int k = 0; k < C / E; ++k)
        store_chunk(row, e0 + k * E, n, f + k * E);
}

// Eight parameters of n, `none` past the end and where there are none.
__device__ __forceinline__ void load_params(const void* p, int wide, int e0, int n, float none,
                                            float* f)
{
#pragma unroll
    for (int j = 0; j < C; ++j)
        f[j] = none;
    if (!p)
        return;
    if (e0 <= n - C) {
        if (wide) {
            const float* q = static_cast<const float*>(p) + e0;
            Elem<float>::unpack(load16(q), f);
            Elem<float>::unpack(load16(q + 4), f + 4);
        } else {
            Elem<bf16_t>::unpack(load16(static_cast<const bf16_t*>(p) + e0), f);
        }
    } else {
#pragma unroll
        for (int j = 0; j < C - 1; ++j)
            if (e0 + j < n)
                f[j] = wide ? static_cast<const float*>(p)[e0 + j]
                            : Elem<bf16_t>::get(static_cast<const bf16_t*>(p)[e0 + j]);
    }
}

__device__ __forceinline__ void put_param(void* p, int wide, int64_t at, float f)
{
    if (wide)
        static_cast<float*>(p)[at] = f;
    else
        static_cast<bf16_t*>(p)[at] = Elem<bf16_t>::put(f);
}

// Zeros past the row's end.
__device__ __forceinline__ void cut(float* f, int e0, int n)
{
    if (e0 > n - C)
#pragma unroll
        for (int j = 0; j < C; ++j)
            f[j] = e0 + j < n ? f[j] : 0.0f;
}

// Threads: G a row, T a block.
template <int G>
struct Block {
    static constexpr int kThreads = G > 512 ? G : 512;
    static constexpr int kGroups = kThreads / G;
    static constexpr int kWaves = G > 64 ? G / 64 : 1;
    static constexpr int kLds = G > 64 ? kThreads / 64 : 1;  // floats of one sum
};

// Sum of K values over each group of G threads, the result in every thread.
// Waves combine through `lds` (2 K Block::kLds floats); calls alternate between
// its halves (`turn`), so that one barrier a call is enough: a half is written
// again only after the barrier of the call between.
template <int G, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float* lds, int& turn)
{
#pragma unroll
    for (int m = 1; m < (G < 64 ? G : 64); m <<= 1)
#pragma unroll
        for (int k = 0; k < K; ++k)
            v[k] += __shfl_xor(v[k], m);
    if constexpr (G > 64) {
        constexpr int W = Block<G>::kWaves;
        lds += turn * (K * Block<G>::kLds);
        turn ^= 1;
        const int wave = threadIdx.x / 64;
        if (threadIdx.x % 64 == 0)
#pragma unroll
            for (int k = 0; k < K; ++k)
                lds[k * Block<G>::kLds + wave] = v[k];
        __syncthreads();
        const int first = wave / W * W;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w)
                s += lds[k * Block<G>::kLds + first + w];
            v[k] = s;
        }
    }
}

// ---------------------------------------------------------------------------
// Arguments.
// ---------------------------------------------------------------------------
struct RnArgs {
    int64_t rows;
    int n;
    float inv_n, skip, scale, eps;
    int center, wide;  // wide: binary32 parameters
    int64_t gates, gate_rows;  // gate_rows: rows that share a gate row
    const void *gate, *post_weight, *post_bias, *pre_weight, *pre_bias;
    const void *x, *z, *dy, *dout;  // backward: x is y
    int64_t ldx, ldz, lddy, lddout;
    void *y, *o;  // backward: dx, dz
    int64_t ldy, ldo;
    float *post_mean, *post_rstd, *pre_mean, *pre_rstd;  // written by the forward
    // Backward.  Work is cut into items: `shares` of each gate row's rows.
    int64_t shares;
    int by_group;     // an item is a group's, not a block's
    float* part;      // [blocks][4][n], or NULL
    float* gate_part; // [gates][shares][n], or NULL where dgate is written at once
    float* means;     // [rows][2], what the kernel for columns needs of rows
    void *dgate, *dparam[4];  // post weight, post bias, pre weight, pre bias
    int parts;
    int64_t vectors;  // of rn_sums_kernel
};

__device__ __forceinline__ const char* gate_of(const RnArgs& a, int64_t g)
{
    return static_cast<const char*>(a.gate) + g * a.n * (a.wide ? 4 : 2);
}

// ---------------------------------------------------------------------------
// Forward.
// ---------------------------------------------------------------------------

// Mean and 1 / sqrt(variance + eps) of a row; f becomes f - mean (zeros past its
// end).
template <int G, int V>
__device__ __forceinline__ void row_stats(const RnArgs& a, float (&f)[V][C], int g, float* lds,
                                          int& turn, float& mean, float& rstd)
{
    mean = 0.0f;
    if (a.center) {
        float s[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int j = 0; j < C; ++j)
                s[0] += f[v][j];
        row_sum<G>(s, lds, turn);
        mean = s[0] * a.inv_n;
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int j = 0; j < C; ++j)
                f[v][j] -= mean;
            cut(f[v], (v * G + g) * C, a.n);
        }
    }
    float q[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < C; ++j)
            q[0] = fmaf(f[v][j], f[v][j], q[0]);
    row_sum<G>(q, lds, turn);
    rstd = 1.0f / sqrtf(fmaf(q[0], a.inv_n, a.eps));
}

// TS, TB: the stream's type and the branches'.
template <typename TS, typename TB, bool POST, bool PRE, int G, int V>
__global__ __launch_bounds__(Block<G>::kThreads) void rn_fwd_kernel(const RnArgs a)
{
    constexpr int NG = Block<G>::kGroups;
    constexpr bool SMALL = G == 8;
    __shared__ float lds[2 * Block<G>::kLds];
    int turn = 0;
    const int g = threadIdx.x % G, grp = threadIdx.x / G, n = a.n;
    float qw[V][C], qb[V][C], gate[V][C], nw[V][C], nb[V][C];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e0 = (v * G + g) * C;
        load_params(a.gate, a.wide, e0, n, 1.0f, gate[v]);
        if constexpr (POST) {
            load_params(a.post_weight, a.wide, e0, n, 1.0f, qw[v]);
            load_params(a.post_bias, a.wide, e0, n, 0.0f, qb[v]);
        }
        if constexpr (PRE) {
            load_params(a.pre_weight, a.wide, e0, n, 1.0f, nw[v]);
            load_params(a.pre_bias, a.wide, e0, n, 0.0f, nb[v]);
        }
    }
    // Threads of one block agree on the trips and meet every barrier together.
    for (int64_t base = (int64_t)blockIdx.x * NG; base < a.rows; base += (int64_t)gridDim.x * NG) {
        const bool in = base + grp < a.rows;
        const int64_t row = in ? base + grp : a.rows - 1;
        Chunk<TB, SMALL> rz[V];
        Chunk<TS, SMALL> rx[V];
        const TB* z = static_cast<const TB*>(a.z) + row * a.ldz;
        const TS* x = static_cast<const TS*>(a.x) + row * a.ldx;
#pragma unroll
        for (int v = 0; v < V; ++v)
            rz[v].load(z, (v * G + g) * C, n);
#pragma unroll
        for (int v = 0; v < V; ++v)
            rx[v].load(x, (v * G + g) * C, n);
        if (a.gates > 1) {
            const char* p = gate_of(a, row / a.gate_rows);
#pragma unroll
            for (int v = 0; v < V; ++v)
                load_params(p, a.wide, (v * G + g) * C, n, 1.0f, gate[v]);
        }
        float f[V][C];
#pragma unroll
        for (int v = 0; v < V; ++v)
            rz[v].values(f[v], (v * G + g) * C, n);
        if constexpr (POST) {
            float mean, rstd;
            row_stats<G>(a, f, g, lds, turn, mean, rstd);
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int j = 0; j < C; ++j)
                    f[v][j] = fmaf(f[v][j] * rstd, qw[v][j], qb[v][j]);
            if (in && g == 0) {
                if (a.post_mean && a.center)
                    a.post_mean[row] = mean;
                if (a.post_rstd)
                    a.post_rstd[row] = rstd;
            }
        }
        TS* y = static_cast<TS*>(a.y) + row * a.ldy;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float fx[C];
            const int e0 = (v * G + g) * C;
            rx[v].values(fx, e0, n);
#pragma unroll
            for (int j = 0; j < C; ++j)
                f[v][j] = fmaf(a.scale, f[v][j] * gate[v][j], a.skip * fx[j]);
            if (in)
                store_row(y, e0, n, f[v]);
        }
        if constexpr (PRE) {
            // (Past the row's end f is 0: x, z and the post bias are.)
            float mean, rstd;
            row_stats<G>(a, f, g, lds, turn, mean, rstd);
            if (in && g == 0) {
                if (a.pre_mean && a.center)
                    a.pre_mean[row] = mean;
                if (a.pre_rstd)
                    a.pre_rstd[row] = rstd;
            }
            TB* o = static_cast<TB*>(a.o) + row * a.ldo;
#pragma unroll
            for (int v = 0; v < V; ++v) {
#pragma unroll
                for (int j = 0; j < C; ++j)
                    f[v][j] = fmaf(f[v][j] * rstd, nw[v][j], nb[v][j]);
                if (in)
                    store_row(o, (v * G + g) * C, n, f[v]);
            }
        }
    }
}

// Rows of any length: a pass over the row for each sum, one block of 1024
// threads.  y is computed anew in every pass (it may be rounded in memory).
template <typename TS, typename TB, bool POST, bool PRE>
__global__ __launch_bounds__(1024) void rn_fwd_long_kernel(const RnArgs a)
{
    constexpr int G = 1024;
    __shared__ float lds[2 * Block<G>::kLds];
    int turn = 0;
    const int n = a.n;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const TB* z = static_cast<const TB*>(a.z) + row * a.ldz;
        const TS* x = static_cast<const TS*>(a.x) + row * a.ldx;
        const char* gp = a.gate ? gate_of(a, row / a.gate_rows) : nullptr;
        // f(values from e0 on) over the row's chunks.
        auto over = [&](auto f) {
            for (int64_t e = (int64_t)threadIdx.x * C; e < n; e += 1024 * C)
                f((int)e);
        };
        auto of_z = [&](int e0, float* f) {
            Chunk<TB, true> c;
            c.load(z, e0, n);
            c.values(f, e0, n);
        };
        // Sum of the values, or of their squared differences from `mean`.
        auto sum = [&](auto of, float mean, bool square) {
            float s[1] = {0.0f};
            over([&](int e0) {
                float f[C];
                of(e0, f);
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    const float d = e0 + j < n ? f[j] - mean : 0.0f;
                    s[0] += square ? d * d : d;
                }
            });
            row_sum<G>(s, lds, turn);
            return s[0] * a.inv_n;
        };
        float zm = 0.0f, zr = 1.0f;
        if constexpr (POST) {
            if (a.center)
                zm = sum(of_z, 0.0f, false);
            zr = 1.0f / sqrtf(sum(of_z, zm, true) + a.eps);
            if (threadIdx.x == 0) {
                if (a.post_mean && a.center)
                    a.post_mean[row] = zm;
                if (a.post_rstd)
                    a.post_rstd[row] = zr;
            }
        }
        auto of_y = [&](int e0, float* f) {
            float fx[C], p[C];
            of_z(e0, f);
            if constexpr (POST) {
                load_params(a.post_weight, a.wide, e0, n, 1.0f, p);
                float b[C];
                load_params(a.post_bias, a.wide, e0, n, 0.0f, b);
#pragma unroll
                for (int j = 0; j < C; ++j)
                    f[j] = fmaf((f[j] - zm) * zr, p[j], b[j]);
            }
            load_params(gp, a.wide, e0, n, 1.0f, p);
            Chunk<TS, true> c;
            c.load(x, e0, n);
            c.values(fx, e0, n);
#pragma unroll
            for (int j = 0; j < C; ++j)
                f[j] = fmaf(a.scale, f[j] * p[j], a.skip * fx[j]);
        };
        float ym = 0.0f, yr = 1.0f;
        if constexpr (PRE) {
            if (a.center)
                ym = sum(of_y, 0.0f, false);
            yr = 1.0f / sqrtf(sum(of_y, ym, true) + a.eps);
            if (threadIdx.x == 0) {
                if (a.pre_mean && a.center)
                    a.pre_mean[row] = ym;
                if (a.pre_rstd)
                    a.pre_rstd[row] = yr;
            }
        }
        over([&](int e0) {
            float f[C], w[C], b[C];
            of_y(e0, f);
            store_row(static_cast<TS*>(a.y) + row * a.ldy, e0, n, f);
            if constexpr (PRE) {
                load_params(a.pre_weight, a.wide, e0, n, 1.0f, w);
                load_params(a.pre_bias, a.wide, e0, n, 0.0f, b);
#pragma unroll
                for (int j = 0; j < C; ++j)
                    f[j] = fmaf((f[j] - ym) * yr, w[j], b[j]);
                store_row(static_cast<TB*>(a.o) + row * a.ldo, e0, n, f);
            }
        });
    }
}

// ---------------------------------------------------------------------------
// Backward.
// ---------------------------------------------------------------------------

// (v - mean) rstd, zeros past the row's end (mean rstd may leave binary32, and 0
// times that is NaN).
__device__ __forceinline__ void normalize(float* f, float mean, float rstd, int e0, int n)
{
#pragma unroll
    for (int j = 0; j < C; ++j)
        f[j] = (f[j] - mean) * rstd;
    cut(f, e0, n);
}

// What rows of an item share.
struct Item {
    int64_t gate, first, end;
};

__device__ __forceinline__ Item item_of(const RnArgs& a, int64_t item)
{
    const int64_t g = item / a.shares, s = item % a.shares, r = g * a.gate_rows;
    return Item{g, r + a.gate_rows * s / a.shares, r + a.gate_rows * (s + 1) / a.shares};
}

// SUMS: with the sums over rows (n <= 8192).
template <typename TS, typename TB, bool POST, bool PRE, int G, int V, bool SUMS>
__global__ __launch_bounds__(Block<G>::kThreads) void rn_bwd_kernel(const RnArgs a)
{
    constexpr int NG = Block<G>::kGroups, T = Block<G>::kThreads;
    constexpr bool SMALL = G == 8;
    __shared__ float lds[4 * Block<G>::kLds];
    __shared__ float sums[SUMS && NG > 1 ? T * V * C : 1];
    int turn = 0;
    const int g = threadIdx.x % G, grp = threadIdx.x / G, n = a.n;
    float qw[V][C], qb[V][C], gate[V][C], nw[V][C];
    float ag[V][C], aqw[V][C], aqb[V][C], anw[V][C], anb[V][C];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e0 = (v * G + g) * C;
        if constexpr (POST) {
            load_params(a.post_weight, a.wide, e0, n, 1.0f, qw[v]);
            load_params(a.post_bias, a.wide, e0, n, 0.0f, qb[v]);
        }
        if constexpr (PRE)
            load_params(a.pre_weight, a.wide, e0, n, 1.0f, nw[v]);
#pragma unroll
        for (int j = 0; j < C; ++j)
            ag[v][j] = aqw[v][j] = aqb[v][j] = anw[v][j] = anb[v][j] = 0.0f;
    }
    const bool use_z = POST || a.dgate;
    const int64_t items = a.gates * a.shares;
    const int64_t unit = a.by_group ? (int64_t)blockIdx.x * NG + grp : blockIdx.x;
    const int64_t units = a.by_group ? (int64_t)gridDim.x * NG : gridDim.x;
    const int step = a.by_group ? 1 : NG, off = a.by_group ? 0 : grp;
    const int64_t trips = ((a.gate_rows + a.shares - 1) / a.shares + step - 1) / step;
    // Every thread of a block makes the same trips and meets every barrier; an
    // item or a row past the last counts as one whose results are not written.
    for (int64_t first = a.by_group ? (int64_t)blockIdx.x * NG : blockIdx.x; first < items;
         first += units) {
        const int64_t index = first + (unit - (a.by_group ? (int64_t)blockIdx.x * NG : blockIdx.x));
        const bool live = index < items;
        const Item it = item_of(a, live ? index : items - 1);
#pragma unroll
        for (int v = 0; v < V; ++v)
            load_params(a.gate ? gate_of(a, it.gate) : nullptr, a.wide, (v * G + g) * C, n, 1.0f,
                        gate[v]);
        for (int64_t t = 0; t < trips; ++t) {
            int64_t row = it.first + off + t * step;
            const bool in = live && row < it.end;
            row = in ? row : it.first;
            Chunk<TS, SMALL> ry[V], rdy[V];
            Chunk<TB, SMALL> rz[V], rdo[V];
            const TS* y = static_cast<const TS*>(a.x) + row * a.ldx;
            const TS* dy = static_cast<const TS*>(a.dy) + row * a.lddy;
            const TB* z = static_cast<const TB*>(a.z) + row * a.ldz;
            const TB* dout = static_cast<const TB*>(a.dout) + row * a.lddout;
            float ym = 0.0f, yr = 0.0f, zm = 0.0f, zr = 0.0f;
            if constexpr (PRE) {
                ym = a.center ? a.pre_mean[row] : 0.0f;
                yr = a.pre_rstd[row];
            }
            if constexpr (POST) {
                zm = a.center ? a.post_mean[row] : 0.0f;
                zr = a.post_rstd[row];
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e0 = (v * G + g) * C;
                if constexpr (PRE) {
                    ry[v].load(y, e0, n);
                    rdo[v].load(dout, e0, n);
                }
                if (a.dy)
                    rdy[v].load(dy, e0, n);
                if (use_z)
                    rz[v].load(z, e0, n);
            }
            float e[V][C];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (a.dy)
                    rdy[v].values(e[v], (v * G + g) * C, n);
                else
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        e[v][j] = 0.0f;
            }
            if constexpr (PRE) {
                float s[2] = {0.0f, 0.0f};
                float h[V][C], c[V][C];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int e0 = (v * G + g) * C;
                    ry[v].values(h[v], e0, n);
                    normalize(h[v], ym, yr, e0, n);
                    rdo[v].values(c[v], e0, n);
#pragma unroll
                    for (int j = 0; j < C; ++j) {
                        if (SUMS && in) {
                            anw[v][j] = fmaf(c[v][j], h[v][j], anw[v][j]);
                            anb[v][j] += c[v][j];
                        }
                        c[v][j] *= nw[v][j];
                        s[0] += c[v][j];
                        s[1] = fmaf(c[v][j], h[v][j], s[1]);
                    }
                }
                row_sum<G>(s, lds, turn);
                const float m1 = a.center ? s[0] * a.inv_n : 0.0f, m2 = s[1] * a.inv_n;
                if (!SUMS && in && g == 0 && a.means) {
                    a.means[2 * row] = m1;
                    a.means[2 * row + 1] = m2;
                }
#pragma unroll
                for (int v = 0; v < V; ++v) {
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        e[v][j] = fmaf(yr, (c[v][j] - m1) - h[v][j] * m2, e[v][j]);
                    cut(e[v], (v * G + g) * C, n);
                }
            }
            TS* dx = static_cast<TS*>(a.y) + row * a.ldy;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float f[C];
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    f[j] = a.skip * e[v][j];
                    e[v][j] *= a.scale;
                }
                if (in)
                    store_row(dx, (v * G + g) * C, n, f);
            }
            float h[V][C], s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e0 = (v * G + g) * C;
                if (use_z)
                    rz[v].values(h[v], e0, n);
                if constexpr (POST)
                    normalize(h[v], zm, zr, e0, n);
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    // e: t, then q, then (POST) q w_post.
                    if (SUMS && in && a.dgate)
                        ag[v][j] = fmaf(e[v][j],
                                        POST ? fmaf(h[v][j], qw[v][j], qb[v][j]) : h[v][j],
                                        ag[v][j]);
                    e[v][j] *= gate[v][j];
                    if constexpr (POST) {
                        if (SUMS && in) {
                            aqw[v][j] = fmaf(e[v][j], h[v][j], aqw[v][j]);
                            aqb[v][j] += e[v][j];
                        }
                        e[v][j] *= qw[v][j];
                        s[0] += e[v][j];
                        s[1] = fmaf(e[v][j], h[v][j], s[1]);
                    }
                }
            }
            if constexpr (POST) {
                row_sum<G>(s, lds, turn);
                const float m1 = a.center ? s[0] * a.inv_n : 0.0f, m2 = s[1] * a.inv_n;
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        e[v][j] = zr * ((e[v][j] - m1) - h[v][j] * m2);
            }
            TB* dz = static_cast<TB*>(a.o) + row * a.ldo;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (in)
                    store_row(dz, (v * G + g) * C, n, e[v]);
        }
        if (SUMS && a.dgate) {
            // The gate's gradient of this item.
            auto put = [&](int col, float f) {
                if (a.gate_part)
                    a.gate_part[index * n + col] = f;
                else
                    put_param(a.dgate, a.wide, it.gate * n + col, f);
            };
            if constexpr (NG > 1)
                if (!a.by_group) {
                    __syncthreads();  // of the item before
#pragma unroll
                    for (int v = 0; v < V; ++v)
#pragma unroll
                        for (int j = 0; j < C; ++j)
                            sums[grp * (G * V * C) + (v * G + g) * C + j] = ag[v][j];
                    __syncthreads();
                    for (int col = threadIdx.x; col < n; col += T) {
                        float f = 0.0f;
                        for (int k = 0; k < NG; ++k)
                            f += sums[k * (G * V * C) + col];
                        put(col, f);
                    }
                }
            if (NG == 1 || a.by_group) {
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        if (live && (v * G + g) * C + j < n)
                            put((v * G + g) * C + j, ag[v][j]);
            }
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int j = 0; j < C; ++j)
                    ag[v][j] = 0.0f;
        }
    }
    if (!SUMS || !a.part)
        return;
    float* part = a.part + (int64_t)blockIdx.x * 4 * n;
    auto flush = [&](int which, const float (&f)[V][C]) {
        if (!a.dparam[which])
            return;
        float* to = part + (int64_t)which * n;
        if constexpr (NG > 1) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int j = 0; j < C; ++j)
                    sums[grp * (G * V * C) + (v * G + g) * C + j] = f[v][j];
            __syncthreads();
            for (int col = threadIdx.x; col < n; col += T) {
                float s = 0.0f;
                for (int k = 0; k < NG; ++k)
                    s += sums[k * (G * V * C) + col];
                to[col] = s;
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int j = 0; j < C; ++j)
                    if ((v * G + g) * C + j < n)
                        to[(v * G + g) * C + j] = f[v][j];
        }
    };
    if constexpr (POST) {
        flush(0, aqw);
        flush(1, aqb);
    }
    if constexpr (PRE) {
        flush(2, anw);
        flush(3, anb);
    }
}

// Rows of any length: dx and dz, a pass over the row for each pair of sums and
// one to write, one block of 1024 threads.
template <typename TS, typename TB, bool POST, bool PRE>
__global__ __launch_bounds__(1024) void rn_bwd_long_kernel(const RnArgs a)
{
    constexpr int G = 1024;
    __shared__ float lds[4 * Block<G>::kLds];
    int turn = 0;
    const int n = a.n;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const char* gp = a.gate ? gate_of(a, row / a.gate_rows) : nullptr;
        float ym = 0.0f, yr = 0.0f, zm = 0.0f, zr = 0.0f;
        if constexpr (PRE) {
            ym = a.center ? a.pre_mean[row] : 0.0f;
            yr = a.pre_rstd[row];
        }
        if constexpr (POST) {
            zm = a.center ? a.post_mean[row] : 0.0f;
            zr = a.post_rstd[row];
        }
        auto over = [&](auto f) {
            for (int64_t e = (int64_t)threadIdx.x * C; e < n; e += 1024 * C)
                f((int)e);
        };
        auto means = [&](float (&s)[2]) {
            row_sum<G>(s, lds, turn);
            s[0] = a.center ? s[0] * a.inv_n : 0.0f;
            s[1] *= a.inv_n;
        };
        // do w_pre and yhat; q w_post and zhat.
        auto of_pre = [&](int e0, float* c, float* h) {
            Chunk<TS, true> y;
            Chunk<TB, true> d;
            y.load(static_cast<const TS*>(a.x) + row * a.ldx, e0, n);
            d.load(static_cast<const TB*>(a.dout) + row * a.lddout, e0, n);
            float w[C];
            load_params(a.pre_weight, a.wide, e0, n, 1.0f, w);
            y.values(h, e0, n);
            normalize(h, ym, yr, e0, n);
            d.values(c, e0, n);
#pragma unroll
            for (int j = 0; j < C; ++j)
                c[j] *= w[j];
        };
        float sy[2] = {0.0f, 0.0f}, sz[2] = {0.0f, 0.0f};
        auto of_e = [&](int e0, float* e) {
            Chunk<TS, true> d;
#pragma unroll
            for (int j = 0; j < C; ++j)
                e[j] = 0.0f;
            if (a.dy) {
                d.load(static_cast<const TS*>(a.dy) + row * a.lddy, e0, n);
                d.values(e, e0, n);
            }
            if constexpr (PRE) {
                float c[C], h[C];
                of_pre(e0, c, h);
#pragma unroll
                for (int j = 0; j < C; ++j)
                    e[j] = fmaf(yr, (c[j] - sy[0]) - h[j] * sy[1], e[j]);
            }
        };
        auto of_post = [&](int e0, float* e, float* h) {
            Chunk<TB, true> z;
            z.load(static_cast<const TB*>(a.z) + row * a.ldz, e0, n);
            float w[C];
            load_params(a.post_weight, a.wide, e0, n, 1.0f, w);
            z.values(h, e0, n);
            normalize(h, zm, zr, e0, n);
#pragma unroll
            for (int j = 0; j < C; ++j)
                e[j] *= w[j];
            cut(e, e0, n);
        };
        auto of_q = [&](int e0, float* e) {
            float w[C];
            load_params(gp, a.wide, e0, n, 1.0f, w);
#pragma unroll
            for (int j = 0; j < C; ++j)
                e[j] = a.scale * e[j] * w[j];
        };
        if constexpr (PRE) {
            float s[2] = {0.0f, 0.0f};
            over([&](int e0) {
                float c[C], h[C];
                of_pre(e0, c, h);
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    s[0] += c[j];
                    s[1] = fmaf(c[j], h[j], s[1]);
                }
            });
            means(s);
            sy[0] = s[0];
            sy[1] = s[1];
            if (threadIdx.x == 0 && a.means) {
                a.means[2 * row] = sy[0];
                a.means[2 * row + 1] = sy[1];
            }
        }
        if constexpr (POST) {
            over([&](int e0) {
                float e[C], h[C];
                of_e(e0, e);
                of_q(e0, e);
                of_post(e0, e, h);
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    sz[0] += e[j];
                    sz[1] = fmaf(e[j], h[j], sz[1]);
                }
            });
            means(sz);
        }
        over([&](int e0) {
            float e[C], f[C], h[C];
            of_e(e0, e);
#pragma unroll
            for (int j = 0; j < C; ++j)
                f[j] = a.skip * e[j];
            store_row(static_cast<TS*>(a.y) + row * a.ldy, e0, n, f);
            of_q(e0, e);
            if constexpr (POST) {
                of_post(e0, e, h);
#pragma unroll
                for (int j = 0; j < C; ++j)
                    e[j] = zr * ((e[j] - sz[0]) - h[j] * sz[1]);
            }
            store_row(static_cast<TB*>(a.o) + row * a.ldo, e0, n, e);
        });
    }
}

// Wide rows (n > 8192): the sums over rows, 256 threads of eight columns by an
// item's rows.
template <typename TS, typename TB, bool POST, bool PRE>
__global__ __launch_bounds__(256) void rn_cols_kernel(const RnArgs a)
{
    const int n = a.n;
    const int64_t first = ((int64_t)blockIdx.x * 256 + threadIdx.x) * C;
    if (first >= n)
        return;
    const int e0 = (int)first;
    float qw[C], qb[C], gate[C], nw[C];
    float ag[C], acc[4][C];
    load_params(a.post_weight, a.wide, e0, n, 1.0f, qw);
    load_params(a.post_bias, a.wide, e0, n, 0.0f, qb);
    load_params(a.pre_weight, a.wide, e0, n, 1.0f, nw);
#pragma unroll
    for (int j = 0; j < C; ++j)
        ag[j] = acc[0][j] = acc[1][j] = acc[2][j] = acc[3][j] = 0.0f;
    const int64_t items = a.gates * a.shares;
    const bool use_z = POST || a.dgate;
    for (int64_t index = blockIdx.y; index < items; index += gridDim.y) {
        const Item it = item_of(a, index);
        load_params(a.gate ? gate_of(a, it.gate) : nullptr, a.wide, e0, n, 1.0f, gate);
        for (int64_t row = it.first; row < it.end; ++row) {
            Chunk<TS, true> ry, rdy;
            Chunk<TB, true> rz, rdo;
            if constexpr (PRE) {
                ry.load(static_cast<const TS*>(a.x) + row * a.ldx, e0, n);
                rdo.load(static_cast<const TB*>(a.dout) + row * a.lddout, e0, n);
            }
            if (use_z) {
                if (a.dy)
                    rdy.load(static_cast<const TS*>(a.dy) + row * a.lddy, e0, n);
                rz.load(static_cast<const TB*>(a.z) + row * a.ldz, e0, n);
            }
            float e[C], h[C];
#pragma unroll
            for (int j = 0; j < C; ++j)
                e[j] = 0.0f;
            if (use_z && a.dy)
                rdy.values(e, e0, n);
            if constexpr (PRE) {
                float c[C];
                const float yr = a.pre_rstd[row], m1 = a.means[2 * row], m2 = a.means[2 * row + 1];
                ry.values(h, e0, n);
                normalize(h, a.center ? a.pre_mean[row] : 0.0f, yr, e0, n);
                rdo.values(c, e0, n);
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    acc[2][j] = fmaf(c[j], h[j], acc[2][j]);
                    acc[3][j] += c[j];
                    e[j] = fmaf(yr, (c[j] * nw[j] - m1) - h[j] * m2, e[j]);
                }
            }
            if (!use_z)
                continue;
            rz.values(h, e0, n);
            if constexpr (POST)
                normalize(h, a.center ? a.post_mean[row] : 0.0f, a.post_rstd[row], e0, n);
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const float t = a.scale * e[j];
                ag[j] = fmaf(t, POST ? fmaf(h[j], qw[j], qb[j]) : h[j], ag[j]);
                if constexpr (POST) {
                    acc[0][j] = fmaf(t * gate[j], h[j], acc[0][j]);
                    acc[1][j] = fmaf(t, gate[j], acc[1][j]);
                }
            }
        }
        if (a.dgate)
#pragma unroll
            for (int j = 0; j < C; ++j) {
                if (e0 + j < n) {
                    if (a.gate_part)
                        a.gate_part[index * n + e0 + j] = ag[j];
                    else
                        put_param(a.dgate, a.wide, it.gate * n + e0 + j, ag[j]);
                }
                ag[j] = 0.0f;
            }
    }
    if (!a.part)
        return;
    float* part = a.part + (int64_t)blockIdx.y * 4 * n + e0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (a.dparam[k])
#pragma unroll
            for (int j = 0; j < C; ++j)
                if (e0 + j < n)
                    part[(int64_t)k * n + j] = acc[k][j];
}

// The gradients of the parameters (vectors 0 to 3) and of the gate's rows (from
// 4 on) from their partial sums: 32 columns a block, 16 threads a column.
__global__ __launch_bounds__(512) void rn_sums_kernel(const RnArgs a)
{
    __shared__ float lds[16][33];
    const int c = threadIdx.x % 32, k = threadIdx.x / 32;
    for (int64_t which = blockIdx.y; which < a.vectors; which += gridDim.y) {
        const float* from;
        int64_t stride, count, to = 0;
        void* dst;
        if (which < 4) {
            from = a.part + which * a.n;
            stride = 4 * (int64_t)a.n;
            count = a.parts;
            dst = a.dparam[which];
        } else {
            from = a.gate_part + (which - 4) * a.shares * a.n;
            stride = a.n;
            count = a.shares;
            dst = a.dgate;
            to = (which - 4) * a.n;
        }
        if (!dst)
            continue;
        for (int64_t first = (int64_t)blockIdx.x * 32; first < a.n;
             first += (int64_t)gridDim.x * 32) {
            const int64_t col = first + c;
            float s = 0.0f;
            if (col < a.n)
                for (int64_t p = k; p < count; p += 16 * 8) {
                    float f[8];  // eight loads in flight
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        f[i] = p + 16 * i < count ? from[(p + 16 * i) * stride + col] : 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        s += f[i];
                }
            lds[k][c] = s;
            __syncthreads();
            if (k == 0 && col < a.n) {
                float t = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    t += lds[i][c];
                put_param(dst, a.wide, to + col, t);
            }
            __syncthreads();
        }
    }
}

// ---------------------------------------------------------------------------
// Host.
// ---------------------------------------------------------------------------

// Most blocks of the backward, each with its own partial sums: two of 512
// threads on a CU.
constexpr int kMaxParts = 512;
// Most blocks of the forward, each keeping its columns of the parameters.
constexpr int kFwdBlocks = 1024;
// Most blocks of the kernels of 1024 threads that loop over what is left: a
// launch has fewer than 2^32 threads.
constexpr int64_t kMaxGrid = 1 << 21;
constexpr int kSumsWidth = 8192;   // widest rows whose sums stay in registers
constexpr int kRowWidth = 16384;   // widest rows that do

template <typename TS, typename TB, bool POST, bool PRE, int G, int V>
int fwd_launch(RnArgs& a, hipStream_t stream)
{
    int64_t grid = (a.rows + Block<G>::kGroups - 1) / Block<G>::kGroups;
    if (grid > kFwdBlocks)
        grid = kFwdBlocks;
    void* args[] = {&a};
    return launch(reinterpret_cast<const void*>(&rn_fwd_kernel<TS, TB, POST, PRE, G, V>),
                  dim3((unsigned)grid), Block<G>::kThreads, args, stream);
}

// The smallest group whose chunks hold the row.
template <typename TS, typename TB, bool POST, bool PRE>
int fwd_run(RnArgs& a, hipStream_t stream)
{
    const int n = a.n;
    if (n <= 64)
        return fwd_launch<TS, TB, POST, PRE, 8, 1>(a, stream);
    if (n <= 256)
        return fwd_launch<TS, TB, POST, PRE, 32, 1>(a, stream);
    if (n <= 512)
        return fwd_launch<TS, TB, POST, PRE, 64, 1>(a, stream);
    if (n <= 1024)
        return fwd_launch<TS, TB, POST, PRE, 128, 1>(a, stream);
    if (n <= 2048)
        return fwd_launch<TS, TB, POST, PRE, 256, 1>(a, stream);
    if (n <= 4096)
        return fwd_launch<TS, TB, POST, PRE, 512, 1>(a, stream);
    if (n <= 8192)
        return fwd_launch<TS, TB, POST, PRE, 1024, 1>(a, stream);
    if (n <= kRowWidth)
        return fwd_launch<TS, TB, POST, PRE, 1024, 2>(a, stream);
    void* args[] = {&a};
    return launch(reinterpret_cast<const void*>(&rn_fwd_long_kernel<TS, TB, POST, PRE>),
                  dim3((unsigned)(a.rows < kMaxGrid ? a.rows : kMaxGrid)), 1024, args, stream);
}

int sums_launch(RnArgs& a, hipStream_t stream)
{
    const int64_t blocks = ((int64_t)a.n + 31) / 32;
    a.vectors = 4 + (a.dgate && a.gate_part ? a.gates : 0);
    const int64_t vectors = a.vectors < 32768 ? a.vectors : 32768;
    void* args[] = {&a};
    return launch(reinterpret_cast<const void*>(&rn_sums_kernel),
                  dim3((unsigned)(blocks < (1 << 14) ? blocks : 1 << 14), (unsigned)vectors), 512,
                  args, stream);
}

bool wants_params(const RnArgs& a)
{
    return a.dparam[0] || a.dparam[1] || a.dparam[2] || a.dparam[3];
}

// Cuts the rows into items for `blocks` blocks of `groups` rows at once (the
// most of either that the workspace is for): a share of a gate row's rows to a
// block; whole gate rows where there are more of them than blocks; and to a group
// where a block's groups would be idle for the few rows of a gate row.
void plan_items(RnArgs& a, int64_t groups, int64_t& blocks)
{
    a.by_group = groups > 1 && a.gates > 1 && a.gate_rows < 2 * groups;
    if (a.by_group) {
        a.shares = 1;
        blocks = (a.gates + groups - 1) / groups;
    } else {
        const int64_t most = (a.gate_rows + groups - 1) / groups;  // shares with work
        a.shares = kMaxParts / a.gates;
        a.shares = a.shares > most ? most : a.shares;
        a.shares = a.shares < 1 ? 1 : a.shares;
        blocks = a.gates * a.shares;
    }
    blocks = blocks < kMaxParts ? blocks : kMaxParts;
    if (a.shares == 1 && a.gates > 1)
        a.gate_part = nullptr;  // an item is a whole gate row: its sum is the gradient
    a.parts = (int)blocks;
}

template <typename TS, typename TB, bool POST, bool PRE, int G, int V, bool SUMS>
int bwd_launch(RnArgs& a, hipStream_t stream)
{
    int64_t blocks;
    RnArgs b = a;
    plan_items(b, Block<G>::kGroups, blocks);
    void* args[] = {&b};
    if (!SUMS) {  // a block a row; items are the other kernel's
        b.shares = b.gate_rows;
        b.by_group = 0;
        const int64_t rows = a.rows < kMaxGrid ? a.rows : kMaxGrid;
        blocks = rows;
    }
    int rc = launch(reinterpret_cast<const void*>(&rn_bwd_kernel<TS, TB, POST, PRE, G, V, SUMS>),
                    dim3((unsigned)blocks), Block<G>::kThreads, args, stream);
    if (rc != MESWISH_OK || !SUMS || !(wants_params(b) || (b.dgate && b.gate_part)))
        return rc;
    return sums_launch(b, stream);
}

template <typename TS, typename TB, bool POST, bool PRE>
int bwd_run(RnArgs& a, hipStream_t stream)
{
    const int n = a.n;
    if (n <= 64)
        return bwd_launch<TS, TB, POST, PRE, 8, 1, true>(a, stream);
    if (n <= 256)
        return bwd_launch<TS, TB, POST, PRE, 32, 1, true>(a, stream);
    if (n <= 512)
        return bwd_launch<TS, TB, POST, PRE, 64, 1, true>(a, stream);
    if (n <= 1024)
        return bwd_launch<TS, TB, POST, PRE, 128, 1, true>(a, stream);
    if (n <= 2048)
        return bwd_launch<TS, TB, POST, PRE, 256, 1, true>(a, stream);
    if (n <= 4096)
        return bwd_launch<TS, TB, POST, PRE, 512, 1, true>(a, stream);
    if (n <= kSumsWidth)
        return bwd_launch<TS, TB, POST, PRE, 1024, 1, true>(a, stream);
    int rc;
    if (n <= kRowWidth) {
        rc = bwd_launch<TS, TB, POST, PRE, 1024, 2, false>(a, stream);
    } else {
        void* args[] = {&a};
        rc = launch(reinterpret_cast<const void*>(&rn_bwd_long_kernel<TS, TB, POST, PRE>),
                    dim3((unsigned)(a.rows < kMaxGrid ? a.rows : kMaxGrid)), 1024, args, stream);
    }
    if (rc != MESWISH_OK || !(a.dgate || wants_params(a)))
        return rc;
    int64_t blocks;
    plan_items(a, 1, blocks);
    void* args[] = {&a};
    const int64_t cols = ((int64_t)n + 256 * C - 1) / (256 * C);
    rc = launch(reinterpret_cast<const void*>(&rn_cols_kernel<TS, TB, POST, PRE>),
                dim3((unsigned)cols, (unsigned)blocks), 256, args, stream);
    if (rc != MESWISH_OK || !(wants_params(a) || (a.dgate && a.gate_part)))
        return rc;
    return sums_launch(a, stream);
}

template <typename TS, typename TB, bool BWD>
int run_norms(RnArgs& a, bool post, bool pre, hipStream_t stream)
{
    if constexpr (BWD) {
        if (post && pre)
            return bwd_run<TS, TB, true, true>(a, stream);
        return post ? bwd_run<TS, TB, true, false>(a, stream)
                    : bwd_run<TS, TB, false, true>(a, stream);
    } else {
        if (post && pre)
            return fwd_run<TS, TB, true, true>(a, stream);
        return post ? fwd_run<TS, TB, true, false>(a, stream)
                    : fwd_run<TS, TB, false, true>(a, stream);
    }
}

template <bool BWD>
int run_types(RnArgs& a, const residual_norm_op& op, hipStream_t stream)
{
    if (op.stream_dtype == MESWISH_BF16)
        return run_norms<bf16_t, bf16_t, BWD>(a, op.post, op.pre, stream);
    return op.branch_dtype == MESWISH_BF16 ? run_norms<float, bf16_t, BWD>(a, op.post, op.pre, stream)
                                           : run_norms<float, float, BWD>(a, op.post, op.pre, stream);
}

bool matrix_ok(const void* p, size_t rows, size_t n, size_t ld, size_t es)
{
    if (!p || !aligned(p, es) || ld < n)
        return false;
    const size_t most = (size_t)1 << 59;
    return rows < most && (ld == 0 || rows == 0 || (rows - 1) < (most - n) / ld);
}

bool gates_ok(size_t rows, size_t n, size_t gates)
{
    const size_t most = (size_t)1 << 59;
    return gates >= 1 && rows % gates == 0 && (rows == 0 || gates <= rows) &&
           (n == 0 || gates < most / n);
}

bool op_ok(const residual_norm_op* op)
{
    return op && (op->post || op->pre) && dtype_ok(op->stream_dtype) && dtype_ok(op->branch_dtype) &&
           dtype_ok(op->param_dtype) &&
           !(op->stream_dtype == MESWISH_BF16 && op->branch_dtype == MESWISH_F32) &&
           isfinite(op->skip) && isfinite(op->scale) && isfinite(op->eps) && op->eps >= 0.0f &&
           op->n < ((size_t)1 << 31) && op->rows < ((size_t)1 << 59) &&
           gates_ok(op->rows, op->n, op->gates);
}

RnArgs common(const residual_norm_op& op)
{
    RnArgs a{};
    a.rows = (int64_t)op.rows;
    a.n = (int)op.n;
    a.inv_n = 1.0f / (float)op.n;
    a.skip = op.skip, a.scale = op.scale, a.eps = op.eps;
    a.center = op.center != 0;
    a.wide = op.param_dtype == MESWISH_F32;
    a.gate = op.gate;
    a.gates = op.gate ? (int64_t)op.gates : 1;
    a.gate_rows = a.rows / a.gates;
    a.post_weight = op.post ? op.post_weight : nullptr;
    a.post_bias = op.post ? op.post_bias : nullptr;
    a.pre_weight = op.pre ? op.pre_weight : nullptr;
    a.pre_bias = op.pre ? op.pre_bias : nullptr;
    return a;
}

// The spans of the parameters that a call reads.
int param_spans(const residual_norm_op& op, Span* s)
{
    const size_t ps = elem_size(op.param_dtype), n = op.n;
    int k = 0;
    s[k++] = span(op.gate, op.gate ? op.gates : 0, n, n, ps);
    for (const void* p : {op.post ? op.post_weight : nullptr, op.post ? op.post_bias : nullptr,
                          op.pre ? op.pre_weight : nullptr, op.pre ? op.pre_bias : nullptr})
        s[k++] = span(p, p ? 1 : 0, n, n, ps);
    return k;
}

bool params_aligned(const residual_norm_op& op)
{
    const size_t ps = elem_size(op.param_dtype);
    for (const void* p : {op.gate, op.post_weight, op.post_bias, op.pre_weight, op.pre_bias})
        if (!aligned(p, ps))
            return false;
    return true;
}

Span stats_span(const float* p, bool used, size_t rows)
{
    return span(p, used && p && rows ? 1 : 0, rows, rows, 4);
}

size_t line_up(size_t bytes) { return (bytes + 127) / 128 * 128; }

// The workspace: the blocks' partial sums, the gate's, two values a row.
struct RnSpace {
    size_t part, gate, means;
    size_t bytes() const { return part + gate + means; }
};

RnSpace rn_space(size_t rows, size_t n, size_t gates)
{
    const size_t parts = rows < (size_t)kMaxParts ? (rows ? rows : 1) : (size_t)kMaxParts;
    RnSpace s{};
    s.part = line_up(parts * 4 * n * sizeof(float));
    // Shares of a gate's rows are kept only if there are more than one, or one gate.
    s.gate = gates > 1 && gates > (size_t)kMaxParts / 2 ? 0 : line_up(parts * n * sizeof(float));
    s.means = n > (size_t)kSumsWidth ? line_up(2 * rows * sizeof(float)) : 0;
    return s;
}

}  // namespace

}  // namespace meblock

using namespace meblock;

extern "C" int residual_norm_fwd(const residual_norm_op* op, const void* x, size_t ldx, const void* z,
                                 size_t ldz, void* y, size_t ldy, void* o, size_t ldo,
                                 float* post_mean, float* post_rstd, float* pre_mean,
                                 float* pre_rstd, void* stream)
{
    if (!op_ok(op))
        return MESWISH_EINVAL;
    const size_t rows = op->rows, n = op->n;
    if (rows == 0 || n == 0)
        return MESWISH_OK;
    const size_t ss = elem_size(op->stream_dtype), bs = elem_size(op->branch_dtype);
    if (!matrix_ok(x, rows, n, ldx, ss) || !matrix_ok(z, rows, n, ldz, bs) ||
        !matrix_ok(y, rows, n, ldy, ss) || (op->pre && !matrix_ok(o, rows, n, ldo, bs)) ||
        !params_aligned(*op) || !aligned(post_mean, 4) || !aligned(post_rstd, 4) ||
        !aligned(pre_mean, 4) || !aligned(pre_rstd, 4))
        return MESWISH_EINVAL;
    Span in[7] = {span(x, rows, n, ldx, ss), span(z, rows, n, ldz, bs)};
    const int nin = 2 + param_spans(*op, in + 2);
    const bool center = op->center != 0;
    const Span out[] = {span(y, rows, n, ldy, ss), span(o, op->pre ? rows : 0, n, ldo, bs),
                        stats_span(post_mean, op->post && center, rows),
                        stats_span(post_rstd, op->post, rows),
                        stats_span(pre_mean, op->pre && center, rows),
                        stats_span(pre_rstd, op->pre, rows)};
    const int rc = apart(out, 6, in, nin);
    if (rc != MESWISH_OK)
        return rc;
    RnArgs a = common(*op);
    a.x = x, a.z = z, a.y = y, a.o = o;
    a.ldx = (int64_t)ldx, a.ldz = (int64_t)ldz, a.ldy = (int64_t)ldy, a.ldo = (int64_t)ldo;
    a.post_mean = post_mean, a.post_rstd = post_rstd;
    a.pre_mean = pre_mean, a.pre_rstd = pre_rstd;
    return run_types<false>(a, *op, static_cast<hipStream_t>(stream));
}

extern "C" size_t residual_norm_workspace_bytes(size_t rows, size_t n, size_t gates)
{
    if (n >= ((size_t)1 << 31) || rows >= ((size_t)1 << 59) || !gates_ok(rows, n, gates))
        return 0;
    return rn_space(rows, n ? n : 1, gates).bytes();
}

extern "C" int residual_norm_bwd(const residual_norm_op* op, const void* y, size_t ldy, const void* z,
                                 size_t ldz, const void* dy, size_t lddy, const void* dout,
                                 size_t lddout, const float* post_mean, const float* post_rstd,
                                 const float* pre_mean, const float* pre_rstd, void* dx, size_t lddx,
                                 void* dz, size_t lddz, void* dgate, void* dpost_weight,
                                 void* dpost_bias, void* dpre_weight, void* dpre_bias,
                                 void* workspace, size_t workspace_bytes, void* stream)
{
    if (!op_ok(op))
        return MESWISH_EINVAL;
    const size_t rows = op->rows, n = op->n;
    if (n == 0)
        return MESWISH_OK;
    const size_t ss = elem_size(op->stream_dtype), bs = elem_size(op->branch_dtype);
    const size_t ps = elem_size(op->param_dtype);
    const bool post = op->post != 0, pre = op->pre != 0, center = op->center != 0;
    if (!op->gate)
        dgate = nullptr;
    if (!post)
        dpost_weight = dpost_bias = nullptr;
    if (!pre)
        dpre_weight = dpre_bias = nullptr;
    const bool use_z = post || dgate;
    const size_t gates = op->gate ? op->gates : 1;
    const RnSpace sp = rn_space(rows, n, gates);
    if (!workspace || workspace_bytes < sp.bytes() || !aligned(workspace, 16) || !params_aligned(*op))
        return MESWISH_EINVAL;
    for (const void* p : {(const void*)dgate, (const void*)dpost_weight, (const void*)dpost_bias,
                          (const void*)dpre_weight, (const void*)dpre_bias})
        if (!aligned(p, ps))
            return MESWISH_EINVAL;
    if (rows > 0) {
        if ((pre && !matrix_ok(y, rows, n, ldy, ss)) || (use_z && !matrix_ok(z, rows, n, ldz, bs)) ||
            (dy && !matrix_ok(dy, rows, n, lddy, ss)) ||
            (pre && !matrix_ok(dout, rows, n, lddout, bs)) || !matrix_ok(dx, rows, n, lddx, ss) ||
            !matrix_ok(dz, rows, n, lddz, bs))
            return MESWISH_EINVAL;
        const struct { const float* p; bool used; } stats[] = {
            {post_mean, post && center}, {post_rstd, post}, {pre_mean, pre && center}, {pre_rstd, pre}};
        for (const auto& s : stats)
            if (s.used && (!s.p || !aligned(s.p, 4)))
                return MESWISH_EINVAL;
    }
    Span in[13] = {span(y, pre ? rows : 0, n, ldy, ss), span(z, use_z ? rows : 0, n, ldz, bs),
                   span(dy, dy ? rows : 0, n, lddy, ss), span(dout, pre ? rows : 0, n, lddout, bs),
                   stats_span(post_mean, post && center, rows), stats_span(post_rstd, post, rows),
                   stats_span(pre_mean, pre && center, rows), stats_span(pre_rstd, pre, rows)};
    const int nin = 8 + param_spans(*op, in + 8);
    Span out[8] = {span(dx, rows, n, lddx, ss), span(dz, rows, n, lddz, bs),
                   span(dgate, dgate ? gates : 0, n, n, ps)};
    int nout = 3;
    for (const void* p : {dpost_weight, dpost_bias, dpre_weight, dpre_bias})
        out[nout++] = span(p, p ? 1 : 0, n, n, ps);
    out[nout++] = span(workspace, 1, sp.bytes(), sp.bytes(), 1);
    const int rc = apart(out, nout, in, nin);
    if (rc != MESWISH_OK)
        return rc;
    RnArgs a = common(*op);
    a.x = y, a.z = z, a.dy = dy, a.dout = dout, a.y = dx, a.o = dz;
    a.ldx = (int64_t)ldy, a.ldz = (int64_t)ldz, a.lddy = (int64_t)lddy, a.lddout = (int64_t)lddout;
    a.ldy = (int64_t)lddx, a.ldo = (int64_t)lddz;
    a.post_mean = const_cast<float*>(post_mean), a.post_rstd = const_cast<float*>(post_rstd);
    a.pre_mean = const_cast<float*>(pre_mean), a.pre_rstd = const_cast<float*>(pre_rstd);
    a.dgate = dgate;
    a.dparam[0] = dpost_weight, a.dparam[1] = dpost_bias;
    a.dparam[2] = dpre_weight, a.dparam[3] = dpre_bias;
    char* at = static_cast<char*>(workspace);
    a.part = wants_params(a) ? reinterpret_cast<float*>(at) : nullptr;
    a.gate_part = sp.gate ? reinterpret_cast<float*>(at + sp.part) : nullptr;
    a.means = sp.means ? reinterpret_cast<float*>(at + sp.part + sp.gate) : nullptr;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (rows == 0) {  // sums over nothing: zeros
        if (!a.dgate && !wants_params(a))
            return MESWISH_OK;
        a.shares = 0;
        a.gate_part = reinterpret_cast<float*>(at);  // (of no shares: not read)
        return sums_launch(a, s);
    }
    return run_types<true>(a, *op, s);
}
