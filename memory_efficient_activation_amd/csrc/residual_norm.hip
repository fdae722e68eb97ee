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
//   * The last chunk of a row is moved back to end with it, so that loads and values
//     need no mask; a thread's next row is loaded under the work on this one.
// Measured, both norms, bf16 with binary32 parameters: 16384 x 4096 forward 100 us
// (5.4 TB/s), backward 175 us (4.6 TB/s, with the second launch, which adds the partial
// sums: 17 MB of the norms', with a gate 21); 1 x 4096 17 us, of which the host's call
// takes 12.  Rows of 65 to 128 values leave half or more of their 32 lanes without
// columns (200000 x 128 forward 57 us, 3.6 TB/s).

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "block_common.h"
#include "residual_norm.h"

namespace meblock {

namespace {

constexpr int C = 8;  // columns of a thread and chunk
constexpr int kColThreads = 256;  // of the sums over rows by themselves
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// Rows.
// ---------------------------------------------------------------------------

// An offset that the compiler adds where it is used: a row's address stays in
// scalar registers then, where else it would keep 64 bits a lane for every
// matrix through the loop over rows.
__device__ __forceinline__ uint32_t late_offset(int v)
{
    uint32_t u = (uint32_t)v;
    asm volatile("" : "+v"(u));
    return u;
}

// Eight columns of a row, as loaded.
template <typename T>
struct Chunk {
    static constexpr int E = Elem<T>::kPerVec, K = C / E;
    u32x4 v[K];
    __device__ __forceinline__ void load(const T* row, int col)
    {
        const char* p = reinterpret_cast<const char*>(row);
        const uint32_t at = late_offset(col * (int)sizeof(T));
#pragma unroll
        for (int k = 0; k < K; ++k)
            v[k] = load16(p + at + 16 * k);
    }
    // Zeros past the row's end (for rows of any length).
    __device__ __forceinline__ void load_cut(const T* row, int e0, int n)
    {
#pragma unroll
        for (int k = 0; k < K; ++k)
            v[k] = load_chunk(row, e0 + k * E, n);
    }
    // mask: 0 (zeros in the place of the values) or all ones.
    __device__ __forceinline__ void keep(uint32_t mask)
    {
#pragma unroll
        for (int k = 0; k < K; ++k)
            v[k] &= mask;
    }
    __device__ __forceinline__ void values(float* f) const
    {
#pragma unroll
        for (int k = 0; k < K; ++k)
            Elem<T>::unpack(v[k], f + k * E);
    }
};

template <typename T>
__device__ __forceinline__ void store8(T* row, int col, const float* f)
{
    constexpr int E = Elem<T>::kPerVec;
    char* p = reinterpret_cast<char*>(row);
    const uint32_t at = late_offset(col * (int)sizeof(T));
#pragma unroll
    for (int k = 0; k < C / E; ++k)
        store16(p + at + 16 * k, Elem<T>::pack(f + k * E));
}

template <typename T>
__device__ __forceinline__ void store_cut(T* row, int e0, int n, const float* f)
{
    constexpr int E = Elem<T>::kPerVec;
#pragma unroll
    for (int k = 0; k < C / E; ++k)
        store_chunk(row, e0 + k * E, n, f + k * E);
}

// The columns of a thread's chunk.  A chunk that would pass the row's end is moved
// back to end with it: it shares its first `shared` columns with the chunk before
// (or all eight), and both compute the same values there.  Sums over the row
// count them once.  So no load, store or value needs a mask.
struct Place {
    int col, shared;
    Place() = default;
    __device__ __forceinline__ Place(int e0, int n)
    {
        col = e0 <= n - C ? e0 : n - C;
        shared = e0 - col < C ? e0 - col : C;
    }
    __device__ __forceinline__ bool none() const { return shared == C; }
};

// Sum of f(j) over a chunk's columns, added to s.
template <class F>
__device__ __forceinline__ float chunk_sum(const Place& p, const F& f)
{
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < C; ++j)
        s = f(j, s);
    if (p.shared) {
        s = 0.0f;
#pragma unroll
        for (int j = 1; j < C; ++j)
            if (j >= p.shared)
                s = f(j, s);
    }
    return s;
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

// Eight parameters, whole.
__device__ __forceinline__ void put_params(void* p, int wide, int64_t at, const float* f)
{
    if (wide) {
        float* q = static_cast<float*>(p) + at;
        store16(q, Elem<float>::pack(f));
        store16(q + 4, Elem<float>::pack(f + 4));
    } else {
        store16(static_cast<bf16_t*>(p) + at, Elem<bf16_t>::pack(f));
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

// Which of the block's groups this thread is in, as a scalar where a group is whole
// waves: a row's address is one then, and its lanes need offsets alone.
template <int G>
__device__ __forceinline__ int group_of_thread()
{
    if constexpr (Block<G>::kGroups == 1)
        return 0;
    else if constexpr (G >= 64)
        return __builtin_amdgcn_readfirstlane(threadIdx.x / G);
    else
        return threadIdx.x / G;
}

// v plus its value in another lane: DPP within rows of 16 lanes, the lane swaps
// across them.  (Through LDS permutes an exchange held six address registers and
// waited for LDS six times.)
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v)
{
    const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true);
    return v + __builtin_bit_cast(float, o);
}

// Sum over each G lanes (8 to 64, at most a wave), the result in every lane.
template <int G>
__device__ __forceinline__ float lane_sum(float v)
{
    v = add_dpp<0xb1>(v);   // quad_perm 1 0 3 2
    v = add_dpp<0x4e>(v);   // quad_perm 2 3 0 1
    v = add_dpp<0x141>(v);  // row_half_mirror: the other four of eight
    if constexpr (G >= 16)
        v = add_dpp<0x140>(v);  // row_mirror: the other eight of 16
    if constexpr (G >= 32) {
        const uint32_t b = __builtin_bit_cast(uint32_t, v);
        const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
        const uint32_t lo = r[0], hi = r[1];
        v = __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
    }
    if constexpr (G >= 64) {
        const uint32_t b = __builtin_bit_cast(uint32_t, v);
        const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
        const uint32_t lo = r[0], hi = r[1];
        v = __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
    }
    return v;
}

// Sum of K values over each group of G threads, the result in every thread.
// Waves combine through `lds` (2 K Block::kLds floats); calls alternate between
// its halves (`turn`), so that one barrier a call is enough: a half is written
// again only after the barrier of the call between.
template <int G, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float* lds, int& turn)
{
#pragma unroll
    for (int k = 0; k < K; ++k)
        v[k] = lane_sum<(G < 64 ? G : 64)>(v[k]);
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
    const void *x, *z, *dy, *dout;  // backward: x is y; where there is no dy, it is y
    uint32_t dy_mask;               // under a mask of 0 (a load without a branch)
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

// Means and 1 / sqrt(variance + eps) of R rows; f becomes f - mean.
template <int G, int V, int R>
__device__ __forceinline__ void row_stats(const RnArgs& a, float (&f)[R][V][C], const Place (&at)[V],
                                          float* lds, int& turn, float (&mean)[R], float (&rstd)[R])
{
#pragma unroll
    for (int r = 0; r < R; ++r)
        mean[r] = 0.0f;
    if (a.center) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int v = 0; v < V; ++v)
                mean[r] += chunk_sum(at[v], [&](int j, float t) { return t + f[r][v][j]; });
        row_sum<G>(mean, lds, turn);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] *= a.inv_n;
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int j = 0; j < C; ++j)
                    f[r][v][j] -= mean[r];
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        rstd[r] = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
            rstd[r] += chunk_sum(at[v], [&](int j, float t) { return fmaf(f[r][v][j], f[r][v][j], t); });
    }
    row_sum<G>(rstd, lds, turn);
#pragma unroll
    for (int r = 0; r < R; ++r)
        rstd[r] = 1.0f / sqrtf(fmaf(rstd[r], a.inv_n, a.eps));
}

// TS, TB: the stream's type and the branches'.  R rows of a group at a time: their
// loads in flight together, their sums in one exchange.  (bf16, both norms, two rows
// and one: 16384 x 4096 99.7 us and 100.8, 200000 x 128 56.6 and 60.7.)
template <typename TS, typename TB, bool POST, bool PRE, int G, int V, int R>
__global__ __launch_bounds__(Block<G>::kThreads, 4) void rn_fwd_kernel(const RnArgs a)
{
    constexpr int NG = Block<G>::kGroups;
    __shared__ float lds[2 * R * Block<G>::kLds];
    int turn = 0;
    const int g = threadIdx.x % G, grp = group_of_thread<G>(), n = a.n;
    Place at[V];
    // scale w_post and scale b_post, with the gate where it is one for all rows.
    float qw[V][C], qb[V][C], nw[V][C], nb[V][C];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        at[v] = Place((v * G + g) * C, n);
        const int col = at[v].col;
        float gate[C];
        load_params(a.gates > 1 ? nullptr : a.gate, a.wide, col, n, 1.0f, gate);
        load_params(POST ? a.post_weight : nullptr, a.wide, col, n, 1.0f, qw[v]);
        load_params(POST ? a.post_bias : nullptr, a.wide, col, n, 0.0f, qb[v]);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            qw[v][j] *= a.scale * gate[j];
            qb[v][j] *= a.scale * gate[j];
        }
        if constexpr (PRE) {
            load_params(a.pre_weight, a.wide, col, n, 1.0f, nw[v]);
            load_params(a.pre_bias, a.wide, col, n, 0.0f, nb[v]);
        }
    }
    // z's rows are loaded while the rows before are worked on, x's at the start of
    // their own turn.
    Chunk<TB> rz[R][V];
    auto row_of = [&](int64_t base, int r) {
        const int64_t row = base + r * NG + grp;
        return row < a.rows ? row : a.rows - 1;
    };
    auto load_z = [&](int64_t base) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int v = 0; v < V; ++v)
                rz[r][v].load(static_cast<const TB*>(a.z) + row_of(base, r) * a.ldz, at[v].col);
    };
    // Threads of one block agree on the trips and meet every barrier together.
    const int64_t all = (int64_t)gridDim.x * (NG * R);
    int64_t base = (int64_t)blockIdx.x * (NG * R);
    load_z(base);
    for (; base < a.rows; base += all) {
        bool in[R];
        int64_t row[R];
        Chunk<TS> rx[R][V];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            row[r] = row_of(base, r);
            in[r] = base + r * NG + grp < a.rows;
#pragma unroll
            for (int v = 0; v < V; ++v)
                rx[r][v].load(static_cast<const TS*>(a.x) + row[r] * a.ldx, at[v].col);
        }
        __builtin_amdgcn_sched_barrier(0);
        float f[R][V][C], mean[R], rstd[R];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int v = 0; v < V; ++v)
                rz[r][v].values(f[r][v]);
        load_z(base + all);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (POST) {
            row_stats<G>(a, f, at, lds, turn, mean, rstd);
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        f[r][v][j] *= rstd[r];
                if (in[r] && g == 0) {
                    if (a.post_mean && a.center)
                        a.post_mean[row[r]] = mean[r];
                    if (a.post_rstd)
                        a.post_rstd[row[r]] = rstd[r];
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            TS* y = static_cast<TS*>(a.y) + row[r] * a.ldy;
            const char* p = a.gates > 1 ? gate_of(a, row[r] / a.gate_rows) : nullptr;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float fx[C];
                rx[r][v].values(fx);
#pragma unroll
                for (int j = 0; j < C; ++j)
                    f[r][v][j] = POST ? fmaf(f[r][v][j], qw[v][j], qb[v][j]) : f[r][v][j] * qw[v][j];
                if (a.gates > 1) {
                    float gate[C];
                    load_params(p, a.wide, at[v].col, n, 1.0f, gate);
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        f[r][v][j] *= gate[j];
                }
#pragma unroll
                for (int j = 0; j < C; ++j)
                    f[r][v][j] = fmaf(a.skip, fx[j], f[r][v][j]);
                if (in[r] && !at[v].none())
                    store8(y, at[v].col, f[r][v]);
            }
        }
        if constexpr (PRE) {
            row_stats<G>(a, f, at, lds, turn, mean, rstd);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (in[r] && g == 0) {
                    if (a.pre_mean && a.center)
                        a.pre_mean[row[r]] = mean[r];
                    if (a.pre_rstd)
                        a.pre_rstd[row[r]] = rstd[r];
                }
                TB* o = static_cast<TB*>(a.o) + row[r] * a.ldo;
#pragma unroll
                for (int v = 0; v < V; ++v) {
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        f[r][v][j] = fmaf(f[r][v][j] * rstd[r], nw[v][j], nb[v][j]);
                    if (in[r] && !at[v].none())
                        store8(o, at[v].col, f[r][v]);
                }
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
            Chunk<TB> c;
            c.load_cut(z, e0, n);
            c.values(f);
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
            Chunk<TS> c;
            c.load_cut(x, e0, n);
            c.values(fx);
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
            store_cut(static_cast<TS*>(a.y) + row * a.ldy, e0, n, f);
            if constexpr (PRE) {
                load_params(a.pre_weight, a.wide, e0, n, 1.0f, w);
                load_params(a.pre_bias, a.wide, e0, n, 0.0f, b);
#pragma unroll
                for (int j = 0; j < C; ++j)
                    f[j] = fmaf((f[j] - ym) * yr, w[j], b[j]);
                store_cut(static_cast<TB*>(a.o) + row * a.ldo, e0, n, f);
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

// Parameters in LDS, for a group's threads: in registers they would take those of
// a second block on the CU.
template <int G, int V>
struct Params {
    f32x4_t f[V][2][G];
    __device__ __forceinline__ void put(const void* p, int wide, int v, int g, int col, int n,
                                        float none)
    {
        float t[C];
        load_params(p, wide, col, n, none, t);
        f[v][0][g] = f32x4_t{t[0], t[1], t[2], t[3]};
        f[v][1][g] = f32x4_t{t[4], t[5], t[6], t[7]};
    }
    __device__ __forceinline__ void get(int v, int g, float* t) const
    {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                t[4 * k + j] = f[v][k][g][j];
    }
};

// The sums of a block's groups: to LDS, chunk by chunk, and a column's total, added
// in order of the group.
template <int G, int V>
__device__ __forceinline__ int own_slot(int v)
{
    return threadIdx.x / G * (G * V * C) + (v * G + (int)threadIdx.x % G) * C;
}

template <int G, int V>
__device__ __forceinline__ void to_lds(float* lds, const float (&f)[V][C])
{
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < C; ++j)
            lds[own_slot<G, V>(v) + j] = f[v][j];
}

template <int G, int V>
__device__ __forceinline__ float from_lds(const float* lds, int col, int n)
{
    // A last chunk that was moved back ends with the row.
    const int chunk = col / C, at = chunk * C <= n - C ? col : chunk * C + (col - (n - C));
    float t = 0.0f;
    for (int k = 0; k < Block<G>::kGroups; ++k)
        t += lds[k * (G * V * C) + at];
    return t;
}

// Keeps a branch one: the sums under it would be computed twice and selected, in as
// many registers again.
__device__ __forceinline__ void stay_branch() { asm volatile(""); }

// A row in two steps: the upper (PRE: y and do, e) and the lower (POST: z; dx and dz).
// What the first of them reads is loaded while the row before is in its second,
// the rest while the first is worked on.
//
// Three of the five sums over rows follow from two, as the gate is one for all
// rows of an item: with T0 = sum e and T1 = sum e zhat (or e z),
//     dw_post = scale gate T1,  db_post = scale gate T0,
//     dgate = scale (w_post T1 + b_post T0)  (scale T1 without post).
//
// SUMS: with the sums over rows (n <= 8192).  Z: z is read (POST, or for the
// gate's gradient).
template <typename TS, typename TB, bool POST, bool PRE, bool Z, int G, int V, bool SUMS>
__global__ __launch_bounds__(Block<G>::kThreads, 4) void rn_bwd_kernel(const RnArgs a)
{
    constexpr int NG = Block<G>::kGroups, T = Block<G>::kThreads;
    __shared__ float lds[4 * Block<G>::kLds];
    __shared__ Params<PRE ? G : 1, V> nw;
    // Groups' sums of one vector; of the post norm's parameters over the items.
    __shared__ float sums[SUMS && NG > 1 ? T * V * C : 1];
    __shared__ float post_sums[SUMS && POST && NG > 1 ? 2 : 1][SUMS && POST && NG > 1 ? T * V * C : 1];
    int turn = 0;
    const int g = threadIdx.x % G, grp = group_of_thread<G>(), n = a.n;
    Place at[V];
    float gw[V][C];  // scale gate w_post
    float t0[V][C], t1[V][C], anw[V][C], anb[V][C];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        at[v] = Place((v * G + g) * C, n);
        if constexpr (PRE)
            if (grp == 0)
                nw.put(a.pre_weight, a.wide, v, g, at[v].col, n, 1.0f);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            t0[v][j] = t1[v][j] = anw[v][j] = anb[v][j] = 0.0f;
            if constexpr (SUMS && POST && NG > 1)
                post_sums[0][own_slot<G, V>(v) + j] = post_sums[1][own_slot<G, V>(v) + j] = 0.0f;
        }
    }
    __syncthreads();
    float* part = a.part ? a.part + (int64_t)blockIdx.x * 4 * n : nullptr;
    const int64_t items = a.gates * a.shares;
    const int64_t own = a.by_group ? grp : 0, units = (int64_t)gridDim.x * (a.by_group ? NG : 1);
    const int step = a.by_group ? 1 : NG, off = a.by_group ? 0 : grp;
    const int64_t trips = ((a.gate_rows + a.shares - 1) / a.shares + step - 1) / step;
    bool begun = false;
    // Every thread of a block makes the same trips and meets every barrier; an
    // item or a row past the last counts as one whose results are not written.
    for (int64_t first = (int64_t)blockIdx.x * (a.by_group ? NG : 1); first < items; first += units) {
        const int64_t index = first + own;
        const bool live = index < items;
        const Item it = item_of(a, live ? index : items - 1);
        const char* gate = a.gate ? gate_of(a, it.gate) : nullptr;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            load_params(gate, a.wide, at[v].col, n, 1.0f, gw[v]);
            float w[C];
            load_params(POST ? a.post_weight : nullptr, a.wide, at[v].col, n, 1.0f, w);
#pragma unroll
            for (int j = 0; j < C; ++j)
                gw[v][j] *= a.scale * w[j];
        }
        Chunk<TS> ry[V], rdy[V];
        Chunk<TB> rz[V], rdo[V];
        float ym = 0.0f, yr = 0.0f, zm = 0.0f, zr = 0.0f;
        auto row_of = [&](int64_t t) {
            const int64_t row = it.first + off + t * step;
            return live && row < it.end ? row : it.first;
        };
        auto load_upper = [&](int64_t row) {
            const TS* y = static_cast<const TS*>(a.x) + row * a.ldx;
            const TB* dout = static_cast<const TB*>(a.dout) + row * a.lddout;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                ry[v].load(y, at[v].col);
                rdo[v].load(dout, at[v].col);
            }
            ym = a.pre_mean[row];
            yr = a.pre_rstd[row];
        };
        auto load_lower = [&](int64_t row) {
            const TS* dy = static_cast<const TS*>(a.dy) + row * a.lddy;
            const TB* z = static_cast<const TB*>(a.z) + row * a.ldz;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                rdy[v].load(dy, at[v].col);
                if constexpr (Z)
                    rz[v].load(z, at[v].col);
            }
            if constexpr (POST) {
                zm = a.post_mean[row];
                zr = a.post_rstd[row];
            }
        };
        if constexpr (PRE)
            load_upper(row_of(0));
        else
            load_lower(row_of(0));
        for (int64_t t = 0; t < trips; ++t) {
            const int64_t row = row_of(t), next = row_of(t + 1 < trips ? t + 1 : t);
            const bool in = live && it.first + off + t * step < it.end;
            float e[V][C];
            auto unpack_dy = [&]() {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    rdy[v].keep(a.dy_mask);
                    rdy[v].values(e[v]);
                }
            };
            if constexpr (PRE) {
                load_lower(row);
                __builtin_amdgcn_sched_barrier(0);
                float s[2] = {0.0f, 0.0f};
                float h[V][C], c[V][C];
                // (Without center the mean's place holds something else.)
                const float mean = a.center ? ym : 0.0f, rstd = yr;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    ry[v].values(h[v]);
                    rdo[v].values(c[v]);
                    float w[C];
                    nw.get(v, g, w);
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        h[v][j] = (h[v][j] - mean) * rstd;
                    if (SUMS && in) {
                        stay_branch();
#pragma unroll
                        for (int j = 0; j < C; ++j) {
                            anw[v][j] = fmaf(c[v][j], h[v][j], anw[v][j]);
                            anb[v][j] += c[v][j];
                        }
                    }
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        c[v][j] *= w[j];
                    s[0] += chunk_sum(at[v], [&](int j, float f) { return f + c[v][j]; });
                    s[1] += chunk_sum(at[v], [&](int j, float f) { return fmaf(c[v][j], h[v][j], f); });
                }
                row_sum<G>(s, lds, turn);
                const float m1 = a.center ? s[0] * a.inv_n : 0.0f, m2 = s[1] * a.inv_n;
                if (!SUMS && in && g == 0 && a.means) {
                    a.means[2 * row] = m1;
                    a.means[2 * row + 1] = m2;
                }
                __builtin_amdgcn_sched_barrier(0);
                unpack_dy();
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        e[v][j] = fmaf(rstd, (c[v][j] - m1) - h[v][j] * m2, e[v][j]);
                load_upper(next);
            } else {
                unpack_dy();
            }
            TS* dx = static_cast<TS*>(a.y) + row * a.ldy;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float f[C];
#pragma unroll
                for (int j = 0; j < C; ++j)
                    f[j] = a.skip * e[v][j];
                if (in && !at[v].none())
                    store8(dx, at[v].col, f);
            }
            __builtin_amdgcn_sched_barrier(0);
            float h[V][C], s[2] = {0.0f, 0.0f};
            const float mean = a.center ? zm : 0.0f, rstd = zr;
            if constexpr (Z)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    rz[v].values(h[v]);
            if constexpr (!PRE)
                load_lower(next);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if constexpr (POST)
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        h[v][j] = (h[v][j] - mean) * rstd;
                if (SUMS && Z && in) {
                    stay_branch();
#pragma unroll
                    for (int j = 0; j < C; ++j) {
                        t0[v][j] += e[v][j];
                        t1[v][j] = fmaf(e[v][j], h[v][j], t1[v][j]);
                    }
                }
#pragma unroll
                for (int j = 0; j < C; ++j)
                    e[v][j] *= gw[v][j];
                if constexpr (POST) {
                    s[0] += chunk_sum(at[v], [&](int j, float f) { return f + e[v][j]; });
                    s[1] += chunk_sum(at[v], [&](int j, float f) { return fmaf(e[v][j], h[v][j], f); });
                }
            }
            if constexpr (POST) {
                row_sum<G>(s, lds, turn);
                const float m1 = a.center ? s[0] * a.inv_n : 0.0f, m2 = s[1] * a.inv_n;
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        e[v][j] = rstd * ((e[v][j] - m1) - h[v][j] * m2);
            }
            TB* dz = static_cast<TB*>(a.o) + row * a.ldo;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (in && !at[v].none())
                    store8(dz, at[v].col, e[v]);
        }
        if constexpr (!(SUMS && Z))
            continue;
        // What the item's two sums give: the thread's own, so that no barrier is
        // needed before them.
        float f[V][C], b[C];
        if (a.dgate) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                load_params(POST ? a.post_weight : nullptr, a.wide, at[v].col, n, 1.0f, f[v]);
                load_params(POST ? a.post_bias : nullptr, a.wide, at[v].col, n, 0.0f, b);
#pragma unroll
                for (int j = 0; j < C; ++j)
                    f[v][j] = a.scale * (POST ? fmaf(f[v][j], t1[v][j], b[j] * t0[v][j]) : t1[v][j]);
            }
            void* to = a.gate_part ? static_cast<void*>(a.gate_part) : a.dgate;
            const int wide = a.gate_part ? 1 : a.wide;
            const int64_t at0 = (a.gate_part ? index : it.gate) * n;
            if (NG > 1 && !a.by_group) {
                __syncthreads();  // of the item before
                to_lds<G, V>(sums, f);
                __syncthreads();
                for (int col = threadIdx.x; col < n; col += T)
                    put_param(to, wide, at0 + col, from_lds<G, V>(sums, col, n));
            } else if (live) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (!at[v].none())
                        put_params(to, wide, at0 + at[v].col, f[v]);
            }
        }
        if (POST && part) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    load_params(gate, a.wide, at[v].col, n, 1.0f, f[v]);
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        f[v][j] = a.scale * f[v][j] * (k == 0 ? t1[v][j] : t0[v][j]);
                    if constexpr (NG > 1) {
#pragma unroll
                        for (int j = 0; j < C; ++j)
                            post_sums[k][own_slot<G, V>(v) + j] += f[v][j];
                    } else if (a.dparam[k] && !at[v].none()) {
                        // The thread's own columns of the block's partial sums.  Those
                        // that a chunk moved back shares are the chunk before's, which
                        // may be another wave's: each column is added to and written
                        // by one thread alone.
                        float* p = part + (int64_t)k * n;
                        if (begun) {
                            load_params(p, 1, at[v].col, n, 0.0f, b);
#pragma unroll
                            for (int j = 0; j < C; ++j)
                                f[v][j] += b[j];
                        }
                        if (at[v].shared == 0) {
                            store8(p, at[v].col, f[v]);
                        } else {
#pragma unroll
                            for (int j = 1; j < C; ++j)
                                if (j >= at[v].shared)
                                    p[at[v].col + j] = f[v][j];
                        }
                    }
                }
            }
            begun = true;
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int j = 0; j < C; ++j)
                t0[v][j] = t1[v][j] = 0.0f;
    }
    if (!SUMS || !part)
        return;
    if constexpr (PRE) {
#pragma unroll
        for (int k = 2; k < 4; ++k) {
            const float(&f)[V][C] = k == 2 ? anw : anb;
            if (!a.dparam[k])
                continue;
            float* to = part + (int64_t)k * n;
            if constexpr (NG > 1) {
                __syncthreads();
                to_lds<G, V>(sums, f);
                __syncthreads();
                for (int col = threadIdx.x; col < n; col += T)
                    to[col] = from_lds<G, V>(sums, col, n);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (!at[v].none())
                        store8(to, at[v].col, f[v]);
            }
        }
    }
    if constexpr (POST && NG > 1) {
        __syncthreads();
        for (int k = 0; k < 2; ++k)
            if (a.dparam[k])
                for (int col = threadIdx.x; col < n; col += T)
                    part[(int64_t)k * n + col] = from_lds<G, V>(post_sums[k], col, n);
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
            Chunk<TS> y;
            Chunk<TB> d;
            y.load_cut(static_cast<const TS*>(a.x) + row * a.ldx, e0, n);
            d.load_cut(static_cast<const TB*>(a.dout) + row * a.lddout, e0, n);
            float w[C];
            load_params(a.pre_weight, a.wide, e0, n, 1.0f, w);
            y.values(h);
            normalize(h, ym, yr, e0, n);
            d.values(c);
#pragma unroll
            for (int j = 0; j < C; ++j)
                c[j] *= w[j];
        };
        float sy[2] = {0.0f, 0.0f}, sz[2] = {0.0f, 0.0f};
        auto of_e = [&](int e0, float* e) {
            Chunk<TS> d;
#pragma unroll
            for (int j = 0; j < C; ++j)
                e[j] = 0.0f;
            if (a.dy_mask) {
                d.load_cut(static_cast<const TS*>(a.dy) + row * a.lddy, e0, n);
                d.values(e);
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
            Chunk<TB> z;
            z.load_cut(static_cast<const TB*>(a.z) + row * a.ldz, e0, n);
            float w[C];
            load_params(a.post_weight, a.wide, e0, n, 1.0f, w);
            z.values(h);
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
            store_cut(static_cast<TS*>(a.y) + row * a.ldy, e0, n, f);
            of_q(e0, e);
            if constexpr (POST) {
                of_post(e0, e, h);
#pragma unroll
                for (int j = 0; j < C; ++j)
                    e[j] = zr * ((e[j] - sz[0]) - h[j] * sz[1]);
            }
            store_cut(static_cast<TB*>(a.o) + row * a.ldo, e0, n, e);
        });
    }
}

// Rows whose sums do not fit the registers beside them (n > 8192, or shorter than
// a chunk: CUT): the sums over rows by themselves, a block 2048 columns of an item's
// rows, the next row's loads under this one's work.  As in rn_bwd_kernel T0 and T1
// give three of them.  Bound by HBM: it reads what the rows' kernel read once more
// (4096 x 16384, bf16: 537 MB).
template <typename TS, typename TB, bool POST, bool PRE, bool Z, bool CUT>
__global__ __launch_bounds__(kColThreads, 2) void rn_cols_kernel(const RnArgs a)
{
    const int n = a.n;
    const int64_t begin = (int64_t)blockIdx.x * (kColThreads * C), own = begin + threadIdx.x * C;
    if (own >= n)
        return;
    const Place at((int)own, CUT ? C : n);
    // A chunk moved back may begin before the block's columns.
    const int64_t base = begin > 0 ? begin - C : 0;
    const int off = CUT ? 0 : (int)(at.col - base);
    float nw[C], anw[C], anb[C], aqw[C], aqb[C];
    load_params(a.pre_weight, a.wide, at.col, n, 1.0f, nw);
#pragma unroll
    for (int j = 0; j < C; ++j)
        anw[j] = anb[j] = aqw[j] = aqb[j] = 0.0f;
    auto put = [&](void* to, int wide, int64_t index, const float* f) {
        if constexpr (CUT) {
            for (int j = 0; j < n; ++j)
                put_param(to, wide, index + j, f[j]);
        } else if (!at.none()) {
            put_params(to, wide, index + at.col, f);
        }
    };
    const int64_t items = a.gates * a.shares;
    for (int64_t index = blockIdx.y; index < items; index += gridDim.y) {
        const Item it = item_of(a, index);
        float t0[C], t1[C];
#pragma unroll
        for (int j = 0; j < C; ++j)
            t0[j] = t1[j] = 0.0f;
        Chunk<TS> ry, rdy;
        Chunk<TB> rz, rdo;
        float ym = 0.0f, yr = 0.0f, zm = 0.0f, zr = 0.0f, m1 = 0.0f, m2 = 0.0f;
        auto one = [&](auto& chunk, const auto* row) {
            if constexpr (CUT)
                chunk.load_cut(row, 0, n);
            else
                chunk.load(row + base, off);
        };
        auto load = [&](int64_t row) {
            if constexpr (PRE) {
                one(ry, static_cast<const TS*>(a.x) + row * a.ldx);
                one(rdo, static_cast<const TB*>(a.dout) + row * a.lddout);
                ym = a.pre_mean[row];
                yr = a.pre_rstd[row];
            }
            if constexpr (Z) {
                one(rdy, static_cast<const TS*>(a.dy) + row * a.lddy);
                one(rz, static_cast<const TB*>(a.z) + row * a.ldz);
                if constexpr (PRE) {
                    m1 = a.means[2 * row];
                    m2 = a.means[2 * row + 1];
                }
                if constexpr (POST) {
                    zm = a.post_mean[row];
                    zr = a.post_rstd[row];
                }
            }
        };
        if (it.first < it.end)
            load(it.first);
        for (int64_t row = it.first; row < it.end; ++row) {
            float e[C], h[C], c[C], z[C];
            if constexpr (Z) {
                rdy.keep(a.dy_mask);
                rdy.values(e);
                rz.values(z);
            }
            if constexpr (PRE) {
                ry.values(h);
                rdo.values(c);
            }
            // (Without center the means' places hold something else.)
            const float ymean = a.center ? ym : 0.0f, yrstd = yr, zmean = a.center ? zm : 0.0f,
                        zrstd = zr, mean1 = m1, mean2 = m2;
            load(row + 1 < it.end ? row + 1 : row);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (PRE)
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    h[j] = (h[j] - ymean) * yrstd;
                    anw[j] = fmaf(c[j], h[j], anw[j]);
                    anb[j] += c[j];
                    if constexpr (Z)
                        e[j] = fmaf(yrstd, (c[j] * nw[j] - mean1) - h[j] * mean2, e[j]);
                }
            if constexpr (Z)
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    if constexpr (POST)
                        z[j] = (z[j] - zmean) * zrstd;
                    t0[j] += e[j];
                    t1[j] = fmaf(e[j], z[j], t1[j]);
                }
        }
        if constexpr (Z) {
            float f[C], g[C];
            if (a.dgate) {
                load_params(POST ? a.post_weight : nullptr, a.wide, at.col, n, 1.0f, f);
                load_params(POST ? a.post_bias : nullptr, a.wide, at.col, n, 0.0f, g);
#pragma unroll
                for (int j = 0; j < C; ++j)
                    f[j] = a.scale * (POST ? fmaf(f[j], t1[j], g[j] * t0[j]) : t1[j]);
                put(a.gate_part ? static_cast<void*>(a.gate_part) : a.dgate,
                    a.gate_part ? 1 : a.wide, (a.gate_part ? index : it.gate) * n, f);
            }
            if constexpr (POST) {
                load_params(a.gate ? gate_of(a, it.gate) : nullptr, a.wide, at.col, n, 1.0f, g);
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    aqw[j] = fmaf(a.scale * g[j], t1[j], aqw[j]);
                    aqb[j] = fmaf(a.scale * g[j], t0[j], aqb[j]);
                }
            }
        }
    }
    if (!a.part)
        return;
    const float* acc[4] = {aqw, aqb, anw, anb};
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (a.dparam[k])
            put(a.part, 1, ((int64_t)blockIdx.y * 4 + k) * n, acc[k]);
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
// threads on a CU.  (1024, bf16: 16384 x 4096 205 us, 3000 x 2048 39.7 and not 28.4.)
constexpr int kMaxParts = 512;
// Most blocks of the forward, each keeping its columns of the parameters.  (512, 256
// and 1024, bf16: 16384 x 4096 99.7, 106.4 and 101.4 us; 16384 x 1024 25.5, 29.0, 26.4;
// 200000 x 128 56.6, 70.1, 54.7.)
constexpr int kFwdBlocks = 512;
// Most blocks of the kernels of 1024 threads that loop over what is left: a
// launch has fewer than 2^32 threads.
constexpr int64_t kMaxGrid = 1 << 21;
// Blocks of the sums over rows by themselves, for all columns: two on a CU.  More
// leave more partial sums to add (backward, both norms, bf16 / binary32: 4096 x 16384
// 264 / 525 us, of 1024 blocks 287 / 554, of 256 297 / 514; 1000 x 9001 64 / 93, 74 / 104
// and 65 / 90).
constexpr int kColBlocks = 512;
constexpr int kSumsWidth = 8192;   // widest rows whose sums stay in registers
constexpr int kRowWidth = 16384;   // widest rows that do

template <typename TS, typename TB, bool POST, bool PRE, int G, int V, int R>
int fwd_launch(RnArgs& a, hipStream_t stream)
{
    constexpr int NG = Block<G>::kGroups;
    int64_t grid = (a.rows + NG * R - 1) / (NG * R);
    if (grid > kFwdBlocks)
        grid = kFwdBlocks;
    void* args[] = {&a};
    return launch(reinterpret_cast<const void*>(&rn_fwd_kernel<TS, TB, POST, PRE, G, V, R>),
                  dim3((unsigned)grid), Block<G>::kThreads, args, stream);
}

template <typename TS, typename TB, bool POST, bool PRE>
int fwd_long(RnArgs& a, hipStream_t stream)
{
    void* args[] = {&a};
    return launch(reinterpret_cast<const void*>(&rn_fwd_long_kernel<TS, TB, POST, PRE>),
                  dim3((unsigned)(a.rows < kMaxGrid ? a.rows : kMaxGrid)), 1024, args, stream);
}

// The smallest group whose chunks hold the row (rows shorter than a chunk as
// long ones).
template <typename TS, typename TB, bool POST, bool PRE>
int fwd_run(RnArgs& a, hipStream_t stream)
{
    const int n = a.n;
    if (n < C)
        return fwd_long<TS, TB, POST, PRE>(a, stream);
    if (n <= 64)
        return fwd_launch<TS, TB, POST, PRE, 8, 1, 2>(a, stream);
    if (n <= 256)
        return fwd_launch<TS, TB, POST, PRE, 32, 1, 2>(a, stream);
    if (n <= 512)
        return fwd_launch<TS, TB, POST, PRE, 64, 1, 2>(a, stream);
    if (n <= 1024)
        return fwd_launch<TS, TB, POST, PRE, 128, 1, 2>(a, stream);
    if (n <= 2048)
        return fwd_launch<TS, TB, POST, PRE, 256, 1, 2>(a, stream);
    if (n <= 4096)
        return fwd_launch<TS, TB, POST, PRE, 512, 1, 2>(a, stream);
    if (n <= 8192)
        return fwd_launch<TS, TB, POST, PRE, 1024, 1, 2>(a, stream);
    if (n <= kRowWidth)
        return fwd_launch<TS, TB, POST, PRE, 1024, 2, 1>(a, stream);
    return fwd_long<TS, TB, POST, PRE>(a, stream);
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
void plan_items(RnArgs& a, int64_t groups, int64_t& blocks, int64_t parts = kMaxParts)
{
    a.by_group = groups > 1 && a.gates > 1 && a.gate_rows < 2 * groups;
    if (a.by_group) {
        a.shares = 1;
        blocks = (a.gates + groups - 1) / groups;
    } else {
        const int64_t most = (a.gate_rows + groups - 1) / groups;  // shares with work
        a.shares = parts / a.gates;
        a.shares = a.shares > most ? most : a.shares;
        a.shares = a.shares < 1 ? 1 : a.shares;
        blocks = a.gates * a.shares;
    }
    blocks = blocks < parts ? blocks : parts;
    if (a.shares == 1 && a.gates > 1)
        a.gate_part = nullptr;  // an item is a whole gate row: its sum is the gradient
    a.parts = (int)blocks;
}

template <typename TS, typename TB, bool POST, bool PRE, bool Z, int G, int V, bool SUMS>
int bwd_launch(RnArgs& a, hipStream_t stream)
{
    int64_t blocks;
    RnArgs b = a;
    // Where a block's one row is 32 KB or more of what is read (y and do, z, dy if it
    // is given), a block a CU has enough loads in flight and leaves half the partial
    // sums.  (512 and 256 blocks, both norms: 16384 x 4096 bf16 181 us and 175, 8192 x
    // 8192 197 and 176, 600 x 4096 binary32 38 and 26; 24 KB, 16384 x 4096 bf16 without
    // dy, 159 and 177, 10000 x 3000 bf16 93 and 108; four rows of 8 KB, 16384 x 1024 bf16,
    // 45 and 49.  At 36 KB, 10000 x 3000 beside a binary32 stream, the rule costs 3 %: 131
    // and 135.)
    const size_t read = a.n * ((PRE ? sizeof(TS) + sizeof(TB) : 0) + (a.dy_mask ? sizeof(TS) : 0) +
                               (Z ? sizeof(TB) : 0));
    const bool wide = Block<G>::kGroups == 1 && read >= 32768;
    plan_items(b, Block<G>::kGroups, blocks, wide ? kMaxParts / 2 : kMaxParts);
    void* args[] = {&b};
    int rc = launch(reinterpret_cast<const void*>(&rn_bwd_kernel<TS, TB, POST, PRE, Z, G, V, SUMS>),
                    dim3((unsigned)blocks), Block<G>::kThreads, args, stream);
    if (rc != MESWISH_OK || !SUMS || !(wants_params(b) || (b.dgate && b.gate_part)))
        return rc;
    return sums_launch(b, stream);
}

// The sums over rows by themselves.
template <typename TS, typename TB, bool POST, bool PRE, bool Z, bool CUT>
int cols_launch(RnArgs& a, hipStream_t stream)
{
    if (!a.dgate && !wants_params(a))
        return MESWISH_OK;
    const int64_t cols = ((int64_t)a.n + kColThreads * C - 1) / (kColThreads * C);
    int64_t blocks, parts = kColBlocks / cols;
    parts = parts < 1 ? 1 : parts < kMaxParts ? parts : kMaxParts;
    plan_items(a, 1, blocks, parts);
    void* args[] = {&a};
    const int rc = launch(reinterpret_cast<const void*>(&rn_cols_kernel<TS, TB, POST, PRE, Z, CUT>),
                          dim3((unsigned)cols, (unsigned)blocks), kColThreads, args, stream);
    if (rc != MESWISH_OK || !(wants_params(a) || (a.dgate && a.gate_part)))
        return rc;
    return sums_launch(a, stream);
}

template <typename TS, typename TB, bool POST, bool PRE, bool Z, bool CUT>
int bwd_long(RnArgs& a, hipStream_t stream)
{
    void* args[] = {&a};
    const int rc = launch(reinterpret_cast<const void*>(&rn_bwd_long_kernel<TS, TB, POST, PRE>),
                          dim3((unsigned)(a.rows < kMaxGrid ? a.rows : kMaxGrid)), 1024, args, stream);
    return rc == MESWISH_OK ? cols_launch<TS, TB, POST, PRE, Z, CUT>(a, stream) : rc;
}

template <typename TS, typename TB, bool POST, bool PRE, bool Z>
int bwd_run(RnArgs& a, hipStream_t stream)
{
    const int n = a.n;
    if (n < C)
        return bwd_long<TS, TB, POST, PRE, Z, true>(a, stream);
    if (n <= 64)
        return bwd_launch<TS, TB, POST, PRE, Z, 8, 1, true>(a, stream);
    if (n <= 256)
        return bwd_launch<TS, TB, POST, PRE, Z, 32, 1, true>(a, stream);
    if (n <= 512)
        return bwd_launch<TS, TB, POST, PRE, Z, 64, 1, true>(a, stream);
    if (n <= 1024)
        return bwd_launch<TS, TB, POST, PRE, Z, 128, 1, true>(a, stream);
    if (n <= 2048)
        return bwd_launch<TS, TB, POST, PRE, Z, 256, 1, true>(a, stream);
    if (n <= 4096)
        return bwd_launch<TS, TB, POST, PRE, Z, 512, 1, true>(a, stream);
    if (n <= kSumsWidth)
        return bwd_launch<TS, TB, POST, PRE, Z, 1024, 1, true>(a, stream);
    if (n > kRowWidth)
        return bwd_long<TS, TB, POST, PRE, Z, false>(a, stream);
    const int rc = bwd_launch<TS, TB, POST, PRE, Z, 1024, 2, false>(a, stream);
    return rc == MESWISH_OK ? cols_launch<TS, TB, POST, PRE, Z, false>(a, stream) : rc;
}

template <typename TS, typename TB, bool BWD>
int run_norms(RnArgs& a, bool post, bool pre, hipStream_t stream)
{
    if constexpr (BWD) {
        if (post)
            return pre ? bwd_run<TS, TB, true, true, true>(a, stream)
                       : bwd_run<TS, TB, true, false, true>(a, stream);
        return a.dgate ? bwd_run<TS, TB, false, true, true>(a, stream)
                       : bwd_run<TS, TB, false, true, false>(a, stream);
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
    s.means = n > (size_t)kSumsWidth || n < (size_t)C ? line_up(2 * rows * sizeof(float)) : 0;
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
            ((dy || !pre) && !matrix_ok(dy, rows, n, lddy, ss)) ||
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
    a.dy_mask = dy ? 0xffffffffu : 0;
    if (!dy)
        a.dy = y, a.lddy = a.ldx;
    if (!center)
        a.pre_mean = a.pre_rstd, a.post_mean = a.post_rstd;
    if (rows == 0) {  // sums over nothing: zeros
        if (!a.dgate && !wants_params(a))
            return MESWISH_OK;
        a.shares = 0;
        a.gate_part = reinterpret_cast<float*>(at);  // (of no shares: not read)
        return sums_launch(a, s);
    }
    return run_types<true>(a, *op, s);
}
