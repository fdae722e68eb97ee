// layer_norm.hip -- layer normalization of libmeswish for gfx950, forward
// and backward.  Formulas and contracts: include/layer_norm.h.
//
// Bound: HBM bandwidth (8 flops an element forward, 15 backward).  Measured on
// bf16 16384 x 4096: forward 44 us (6.1 TB/s of the rows read and written),
// backward 86 us (4.7 TB/s); the framework's plain copy moves 6.3 TB/s.  Both
// directions read each row once and keep it in registers, packed as loaded:
//   * A group of G threads owns a row, thread g holding the 16-byte vectors
//     g, G + g, ... (V of them).  G is 4 to 64 lanes of a wave, or a block of
//     128 to 1024 threads, so the sums of a row cost lane exchanges only, or
//     one exchange through LDS a batch of R rows.  (bf16 16384 x 4096 forward:
//     a block a row 44 us; a wave a row, V = 8, 66 us: its registers leave too
//     few waves.)  Rows are loaded without a branch, a row's last vector from
//     inside the row, and cut to length where they are used: with the branch
//     at the load the forward took 53 us.
//   * The variance is the mean of squared differences from the mean, from
//     the registers: no cancellation of E[x^2] - mean^2.
//   * Backward: a thread owns the same columns in every row its block takes,
//     so the sums for dweight and dbias stay in registers over the block's
//     rows.  Each block writes one binary32 partial per column; a second
//     kernel adds them in a fixed order (no atomics, deterministic).
//   * Rows longer than 1024 threads hold are read again for each pass (the
//     caches serve most of it), one block per row.

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "block_common.h"
#include "layer_norm.h"

namespace meblock {

// Most blocks of the backward, each with its own partial sums.  Chosen at width
// 4096 (bf16 16384 x 4096: 384 blocks 102 us, 512 92, 768 95, 1024 115: more of
// them write more parts), where a CU holds two blocks of 256 threads.  Wider rows
// have the same number: in bf16 the registers leave one block a CU there (up to
// 8192 values all 256 of them and 10 more as spill space; up to 16384 values 128 in
// blocks of 1024 threads, with 40 to 44 bytes of scratch), so that 512 blocks run
// in two rounds, and the partial sums are 34 and 67 MB.
constexpr int kMaxParts = 512;
// Most blocks of the forward, each keeping its columns of the parameters in
// registers: eight of 256 threads on a CU (bf16 16384 x 4096: 2048 blocks 47 us,
// 1536 55; one block a row, reading the parameters again, 64).
constexpr int kFwdBlocks = 2048;
// Most blocks of the kernels of 1024 threads, which loop over what is left: a
// launch has fewer than 2^32 threads.
constexpr int64_t kMaxGrid = 1 << 21;
static_assert(kMaxGrid * 1024 <= UINT32_MAX, "threads of a launch");

template <int G>
struct Group {
    static constexpr int kThreads = G > 64 ? G : 256;
    static constexpr int kGroups = kThreads / G;  // rows a block takes at once
    static constexpr int kWaves = G / 64;         // waves of a group, where it is whole waves
};

// Sum of K values over each group of G threads, the result in every thread.
// Waves combine through `lds` (2 K kWaves floats); calls alternate between
// its halves (`turn`), so that one barrier a call is enough: a half is written
// again only after the barrier of the call between.
template <int G, int K>
__device__ __forceinline__ void group_sum(float (&v)[K], float* lds, int& turn)
{
#pragma unroll
    for (int m = 1; m < (G < 64 ? G : 64); m <<= 1)
#pragma unroll
        for (int k = 0; k < K; ++k)
            v[k] += __shfl_xor(v[k], m);
    if constexpr (G > 64) {
        constexpr int W = Group<G>::kWaves;
        const int wave = threadIdx.x / 64;
        lds += turn * (K * W);
        turn ^= 1;
        if (threadIdx.x % 64 == 0)
#pragma unroll
            for (int k = 0; k < K; ++k)
                lds[k * W + wave] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w)
                s += lds[k * W + w];
            v[k] = s;
        }
    }
}

// Parameters e0 .. e0 + E - 1 of n, `none` past the end and where there are no
// parameters.
template <int E, typename P>
__device__ __forceinline__ void load_params(const P* p, int e0, int n, float none, float* f)
{
    constexpr int K = Elem<P>::kPerVec;
    if (p && e0 + E <= n && E >= K) {
#pragma unroll
        for (int j = 0; j < E; j += K)
            Elem<P>::unpack(load16(p + e0 + j), f + j);
    } else {
#pragma unroll
        for (int j = 0; j < E; ++j)
            f[j] = p && e0 + j < n ? Elem<P>::get(p[e0 + j]) : none;
    }
}

// Elements e0 ... of a row for a group of G, zeros past its end (REPEAT: other
// elements of the row) and zeros in rows past the last, in two steps (load_near).
// Rows shorter than a vector are of the smallest group alone, which loads the
// chunk at once.
template <int G, bool REPEAT = false, typename T>
__device__ __forceinline__ u32x4 load_row(const T* x, int64_t row, int64_t rows, int64_t ldx,
                                          int e0, int n)
{
    if constexpr (G != 4)
        return load_near(x + (row < rows ? row : rows - 1) * ldx, e0, n);
    else if constexpr (REPEAT)
        return load_repeat(x + row * ldx, e0, row < rows ? n : 0);
    else
        return load_chunk(x + row * ldx, e0, row < rows ? n : 0);
}

template <typename T, int G>
__device__ __forceinline__ u32x4 row_chunk(u32x4 v, int e0, int n)
{
    if constexpr (G == 4)
        return v;
    else
        return chunk_of<T>(v, e0, n);
}

// The chunks of x (REPEAT) and dy at e0; n: the row's length, 0 for a row past
// the last.
template <typename T, int G>
__device__ __forceinline__ void row_chunks(u32x4& x, u32x4& dy, int e0, int n)
{
    constexpr int E = Elem<T>::kPerVec;
    const int s = e0 - (n - E);
    if (G == 4 || s <= 0)
        return;
    dy = s < E ? shift_down<T>(dy, s) : u32x4{0, 0, 0, 0};
    if (s < E)
        x = rotate_down<T>(x, s);
    else if (n == 0)
        x = dy;
}

// ---------------------------------------------------------------------------
// Forward.
// ---------------------------------------------------------------------------
// The block keeps its columns of weight and bias in registers and loops over
// rows, R of a group at a time (their loads in flight together, their sums in
// one exchange).
template <typename T, typename P, int G, int V, int R>
__global__ __launch_bounds__(Group<G>::kThreads) void ln_fwd_kernel(
    const T* x, int64_t ldx, const P* __restrict__ w, const P* __restrict__ b, int64_t rows, int n,
    float eps, T* y, int64_t ldy, float* __restrict__ mean, float* __restrict__ rstd)
{
    constexpr int E = Elem<T>::kPerVec;
    constexpr int NG = Group<G>::kGroups;
    __shared__ float lds[G > 64 ? 2 * R * Group<G>::kWaves : 1];
    int turn = 0;
    const int g = threadIdx.x % G, grp = threadIdx.x / G;
    const float inv_n = 1.0f / (float)n;
    float wf[V][E], bf[V][E];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        load_params<E>(w, (v * G + g) * E, n, 1.0f, wf[v]);
        load_params<E>(b, (v * G + g) * E, n, 0.0f, bf[v]);
    }
    // Threads of one group agree on the rows; a group of whole blocks meets
    // every barrier together.
    for (int64_t base = (int64_t)blockIdx.x * (NG * R); base < rows;
         base += (int64_t)gridDim.x * (NG * R)) {
        u32x4 raw[R][V];
        float s[R], q[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = base + r * NG + grp;
#pragma unroll
            for (int v = 0; v < V; ++v)  // a row past the end counts as an empty one
                raw[r][v] = load_row<G>(x, row, rows, ldx, (v * G + g) * E, n);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int nr = base + r * NG + grp < rows ? n : 0;
            s[r] = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float f[E];
                raw[r][v] = row_chunk<T, G>(raw[r][v], (v * G + g) * E, nr);
                Elem<T>::unpack(raw[r][v], f);
#pragma unroll
                for (int j = 0; j < E; ++j)
                    s[r] += f[j];
            }
        }
        group_sum<G>(s, lds, turn);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s[r] *= inv_n;
            q[r] = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e0 = (v * G + g) * E;
                float f[E];
                Elem<T>::unpack(raw[r][v], f);
                if (e0 + E <= n) {
#pragma unroll
                    for (int j = 0; j < E; ++j)
                        q[r] = fmaf(f[j] - s[r], f[j] - s[r], q[r]);
                } else {
#pragma unroll
                    for (int j = 0; j < E; ++j)
                        q[r] += e0 + j < n ? (f[j] - s[r]) * (f[j] - s[r]) : 0.0f;
                }
            }
        }
        group_sum<G>(q, lds, turn);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = base + r * NG + grp;
            if (row >= rows)
                continue;
            const float rs = 1.0f / sqrtf(fmaf(q[r], inv_n, eps));
            if (g == 0) {
                if (mean)
                    mean[row] = s[r];
                if (rstd)
                    rstd[row] = rs;
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e0 = (v * G + g) * E;
                float f[E];
                Elem<T>::unpack(raw[r][v], f);
#pragma unroll
                for (int j = 0; j < E; ++j)
                    f[j] = fmaf((f[j] - s[r]) * rs, wf[v][j], bf[v][j]);
                store_chunk(y + row * ldy, e0, n, f);
            }
        }
    }
}

// Rows of any length: three passes over the row, one block of 1024 threads.
template <typename T, typename P>
__global__ __launch_bounds__(1024) void ln_fwd_long_kernel(
    const T* x, int64_t ldx, const P* __restrict__ w, const P* __restrict__ b, int64_t rows, int n,
    float eps, T* y, int64_t ldy, float* __restrict__ mean, float* __restrict__ rstd)
{
    constexpr int E = Elem<T>::kPerVec;
    __shared__ float lds[32];
    int turn = 0;
    const float inv_n = 1.0f / (float)n;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const T* xr = x + row * ldx;
        T* yr = y + row * ldy;
        float s[1] = {0.0f};
        for (int64_t e0 = (int64_t)threadIdx.x * E; e0 < n; e0 += 1024 * E) {
            float f[E];
            Elem<T>::unpack(load_chunk(xr, (int)e0, n), f);
#pragma unroll
            for (int j = 0; j < E; ++j)
                s[0] += f[j];
        }
        group_sum<1024>(s, lds, turn);
        const float mu = s[0] * inv_n;
        float q[1] = {0.0f};
        for (int64_t e0 = (int64_t)threadIdx.x * E; e0 < n; e0 += 1024 * E) {
            float f[E];
            Elem<T>::unpack(load_chunk(xr, (int)e0, n), f);
#pragma unroll
            for (int j = 0; j < E; ++j)
                q[0] += e0 + j < n ? (f[j] - mu) * (f[j] - mu) : 0.0f;
        }
        group_sum<1024>(q, lds, turn);
        const float r = 1.0f / sqrtf(fmaf(q[0], inv_n, eps));
        if (threadIdx.x == 0) {
            if (mean)
                mean[row] = mu;
            if (rstd)
                rstd[row] = r;
        }
        for (int64_t e0 = (int64_t)threadIdx.x * E; e0 < n; e0 += 1024 * E) {
            float f[E];
            Elem<T>::unpack(load_chunk(xr, (int)e0, n), f);
#pragma unroll
            for (int j = 0; j < E; ++j)
                f[j] = e0 + j < n ? fmaf((f[j] - mu) * r, w ? Elem<P>::get(w[e0 + j]) : 1.0f,
                                         b ? Elem<P>::get(b[e0 + j]) : 0.0f)
                                  : 0.0f;
            store_chunk(yr, (int)e0, n, f);
        }
    }
}

// ---------------------------------------------------------------------------
// Backward.
// ---------------------------------------------------------------------------

// A thread's columns of a block's partial sums.
template <int E, int G, int V>
__device__ __forceinline__ void store_part(float* pw, int n, int g, const float (&w)[V][E],
                                           const float (&b)[V][E])
{
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const int e = (v * G + g) * E + j;
            if (e < n) {
                pw[e] = w[v][j];
                pw[n + e] = b[v][j];
            }
        }
}

// R rows a group and batch: their sums share one exchange, and the next
// batch's loads are in flight while this one is worked on.  Past a row's end dy
// is zero and x repeats elements of the row: a zero there would make xhat
// -mean rstd, and 0 times that is NaN where it leaves binary32.
template <typename T, typename P, int G, int V, int R>
__global__ __launch_bounds__(Group<G>::kThreads) void ln_bwd_kernel(
    const T* x, int64_t ldx, const T* dy, int64_t lddy, const float* __restrict__ mean,
    const float* __restrict__ rstd, const P* __restrict__ w, int64_t rows, int n, T* dx,
    int64_t lddx, float* __restrict__ part)
{
    constexpr int E = Elem<T>::kPerVec;
    constexpr int NG = Group<G>::kGroups;
    __shared__ float lds[G > 64 ? 4 * R * Group<G>::kWaves : 1];
    int turn = 0;
    const int g = threadIdx.x % G, grp = threadIdx.x / G;
    const float inv_n = 1.0f / (float)n;
    float wf[V][E], aw[V][E], ab[V][E];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        load_params<E>(w, (v * G + g) * E, n, 1.0f, wf[v]);
#pragma unroll
        for (int j = 0; j < E; ++j)
            aw[v][j] = ab[v][j] = 0.0f;
    }
    u32x4 rx[R][V], rd[R][V];
    float mu[R], rs[R];
    auto load = [&](int64_t base) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = base + r * NG + grp;
            const bool in = row < rows;
            mu[r] = in ? mean[row] : 0.0f;
            rs[r] = in ? rstd[row] : 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                // A row past the end counts as an empty one (zeros).
                rx[r][v] = load_row<G, true>(x, row, rows, ldx, (v * G + g) * E, n);
                rd[r][v] = load_row<G>(dy, row, rows, lddy, (v * G + g) * E, n);
            }
        }
    };
    const int64_t step = (int64_t)gridDim.x * (NG * R);
    int64_t base = (int64_t)blockIdx.x * (NG * R);
    load(base);
    for (; base < rows; base += step) {
        float s[2 * R], m[R], t[R];
        u32x4 cx[R][V], cd[R][V];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = mu[r];
            t[r] = rs[r];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                cx[r][v] = rx[r][v];
                cd[r][v] = rd[r][v];
                // (A batch of one row is never past the end.)
                row_chunks<T, G>(cx[r][v], cd[r][v], (v * G + g) * E,
                                 NG * R == 1 || base + r * NG + grp < rows ? n : 0);
            }
        }
        if (base + step < rows)
            load(base + step);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float fx[E], fd[E];
                Elem<T>::unpack(cx[r][v], fx);
                Elem<T>::unpack(cd[r][v], fd);
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const float xh = (fx[j] - m[r]) * t[r];
                    const float gg = fd[j] * wf[v][j];
                    s1 += gg;
                    s2 = fmaf(gg, xh, s2);
                    aw[v][j] = fmaf(fd[j], xh, aw[v][j]);
                    ab[v][j] += fd[j];
                }
            }
            s[2 * r] = s1;
            s[2 * r + 1] = s2;
        }
        group_sum<G>(s, lds, turn);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = base + r * NG + grp;
            if (row >= rows)
                continue;
            const float m1 = s[2 * r] * inv_n, m2 = s[2 * r + 1] * inv_n;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float fx[E], fd[E];
                Elem<T>::unpack(cx[r][v], fx);
                Elem<T>::unpack(cd[r][v], fd);
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const float xh = (fx[j] - m[r]) * t[r];
                    fd[j] = t[r] * (fmaf(fd[j], wf[v][j], -m1) - xh * m2);
                }
                store_chunk(dx + row * lddx, (v * G + g) * E, n, fd);
            }
        }
    }
    if (!part)
        return;
    float* pw = part + (int64_t)blockIdx.x * 2 * n;
    if constexpr (NG > 1) {
        // The groups' columns, added in order of the group.
        constexpr int kSums = G * V * E;
        __shared__ float sums[2][NG * kSums];
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int at = grp * kSums + (v * G + g) * E + j;
                sums[0][at] = aw[v][j];
                sums[1][at] = ab[v][j];
            }
        __syncthreads();
        for (int e = threadIdx.x; e < 2 * n; e += Group<G>::kThreads) {
            const int which = e >= n, col = e - which * n;
            float t = 0.0f;
            for (int k = 0; k < NG; ++k)
                t += sums[which][k * kSums + col];
            pw[e] = t;
        }
    } else {
        store_part<E, G, V>(pw, n, g, aw, ab);
    }
}

// dweight and dbias from the blocks' partial sums: 32 columns a block at a
// time, 32 threads a column.
template <typename P>
__global__ __launch_bounds__(1024) void ln_params_kernel(const float* __restrict__ part, int parts,
                                                         int n, P* dweight, P* dbias)
{
    __shared__ float lds[32][33];
    const int c = threadIdx.x % 32, k = threadIdx.x / 32;
    const int64_t cols = 2 * (int64_t)n;  // dweight's, then dbias's
    for (int64_t first = (int64_t)blockIdx.x * 32; first < cols; first += (int64_t)gridDim.x * 32) {
        const int64_t col = first + c;
        float s = 0.0f;
        if (col < cols)
            for (int p = k; p < parts; p += 32 * 8) {
                float f[8];  // eight loads in flight
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    f[i] = p + 32 * i < parts ? part[(p + 32 * i) * cols + col] : 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s += f[i];
            }
        lds[k][c] = s;
        __syncthreads();
        // Thread (c', k') takes column k', part c': a half wave a column.
        float t = lds[c][k];
#pragma unroll
        for (int m = 16; m; m >>= 1)
            t += __shfl_xor(t, m);
        const int64_t out = first + k;
        if (c == 0 && out < cols) {
            P* dst = out < n ? dweight : dbias;
            if (dst)
                dst[out < n ? out : out - n] = Elem<P>::put(t);
        }
        __syncthreads();
    }
}

// Long rows: dx in two passes over the row.
template <typename T, typename P>
__global__ __launch_bounds__(1024) void ln_bwd_long_kernel(
    const T* x, int64_t ldx, const T* dy, int64_t lddy, const float* __restrict__ mean,
    const float* __restrict__ rstd, const P* __restrict__ w, int64_t rows, int n, T* dx,
    int64_t lddx)
{
    constexpr int E = Elem<T>::kPerVec;
    __shared__ float lds[64];
    int turn = 0;
    const float inv_n = 1.0f / (float)n;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const T* xr = x + row * ldx;
        const T* dr = dy + row * lddy;
        const float mu = mean[row], rs = rstd[row];
        float s[2] = {0.0f, 0.0f};
        for (int64_t e0 = (int64_t)threadIdx.x * E; e0 < n; e0 += 1024 * E) {
            float fx[E], fd[E];
            Elem<T>::unpack(load_chunk(xr, (int)e0, n), fx);
            Elem<T>::unpack(load_chunk(dr, (int)e0, n), fd);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                if (e0 + j >= n)
                    continue;
                const float gg = fd[j] * (w ? Elem<P>::get(w[e0 + j]) : 1.0f);
                s[0] += gg;
                s[1] = fmaf(gg, (fx[j] - mu) * rs, s[1]);
            }
        }
        group_sum<1024>(s, lds, turn);
        const float m1 = s[0] * inv_n, m2 = s[1] * inv_n;
        for (int64_t e0 = (int64_t)threadIdx.x * E; e0 < n; e0 += 1024 * E) {
            float fx[E], fd[E];
            Elem<T>::unpack(load_chunk(xr, (int)e0, n), fx);
            Elem<T>::unpack(load_chunk(dr, (int)e0, n), fd);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const float wj = w && e0 + j < n ? Elem<P>::get(w[e0 + j]) : 1.0f;
                fd[j] = rs * (fmaf(fd[j], wj, -m1) - (fx[j] - mu) * rs * m2);
            }
            store_chunk(dx + row * lddx, (int)e0, n, fd);
        }
    }
}

// Long rows: the blocks' partial column sums, 256 E columns by a share of
// the rows.
template <typename T>
__global__ __launch_bounds__(256) void ln_cols_kernel(const T* __restrict__ x, int64_t ldx,
                                                      const T* __restrict__ dy, int64_t lddy,
                                                      const float* __restrict__ mean,
                                                      const float* __restrict__ rstd, int64_t rows,
                                                      int n, float* __restrict__ part)
{
    constexpr int E = Elem<T>::kPerVec;
    const int64_t first = ((int64_t)blockIdx.x * 256 + threadIdx.x) * E;
    if (first >= n)
        return;
    const int e0 = (int)first;
    float aw[E], ab[E];
#pragma unroll
    for (int j = 0; j < E; ++j)
        aw[j] = ab[j] = 0.0f;
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        float fx[E], fd[E];
        Elem<T>::unpack(load_chunk(x + row * ldx, e0, n), fx);
        Elem<T>::unpack(load_chunk(dy + row * lddy, e0, n), fd);
        const float mu = mean[row], rs = rstd[row];
#pragma unroll
        for (int j = 0; j < E; ++j) {
            aw[j] = fmaf(fd[j], (fx[j] - mu) * rs, aw[j]);
            ab[j] += fd[j];
        }
    }
    float* pw = part + (int64_t)blockIdx.y * 2 * n + first;
#pragma unroll
    for (int j = 0; j < E; ++j)
        if (e0 + j < n) {
            pw[j] = aw[j];
            pw[(int64_t)n + j] = ab[j];
        }
}

// ---------------------------------------------------------------------------
// Host.
// ---------------------------------------------------------------------------

template <typename T, typename P>
struct LnArgs {
    const T *x, *dy;
    const P *w, *b;
    int64_t ldx, lddy, ldo, rows;
    int n;
    float eps;
    T* out;  // y or dx
    float *mean, *rstd, *part;
    P *dweight, *dbias;
    hipStream_t stream;
};

// 16-byte vectors a row.
template <typename T>
static int64_t chunks(int n)
{
    constexpr int E = Elem<T>::kPerVec;
    return ((int64_t)n + E - 1) / E;
}

template <typename T, typename P, int G, int V, int R>
static int fwd_launch(LnArgs<T, P>& a)
{
    constexpr int NG = Group<G>::kGroups;
    int64_t grid = (a.rows + NG * R - 1) / (NG * R);
    if (grid > kFwdBlocks)
        grid = kFwdBlocks;
    void* args[] = {&a.x, &a.ldx, &a.w, &a.b, &a.rows, &a.n, &a.eps, &a.out, &a.ldo, &a.mean,
                    &a.rstd};
    return launch(reinterpret_cast<const void*>(&ln_fwd_kernel<T, P, G, V, R>), dim3((unsigned)grid),
                  Group<G>::kThreads, args, a.stream);
}

// The smallest group whose vectors hold the row.  Which vectors and rows go with
// it was measured on bf16 tensors of 2^26 elements, group x vectors (us):
//   n = 64           8 x 1, 2 rows: 46             4 x 2, 2 rows: 49
//   n = 128 to 512   8 to 32 x 2, 2 rows: 43-45    16 to 64 x 1: 47-49; 1 row: 45-48
//   n = 1024         64 x 2, 2 rows: 43            32 x 4, 1 row: 44
//   n = 2048         128 x 2, 2 rows: 44           256 x 1, 2 rows: 52, 64 x 4, 1 row: 45
//   n = 4096         256 x 2, 2 rows: 44           512 x 1, 2 rows: 48
//   n = 8192         256 x 4, 1 row: 47            512 x 2, 1 row: 49
//   n = 16384        1024 x 2, 1 row: 65           512 x 4, 1 row: 65
// Binary32 is within 3 % of its best with the same choices (n = 8192: 1024 x 2
// 98, 512 x 4 95).
template <typename T, typename P>
static int fwd_run(LnArgs<T, P>& a)
{
    const int64_t c = chunks<T>(a.n);
    if (c <= 4)
        return fwd_launch<T, P, 4, 1, 2>(a);
    if (c <= 8)
        return fwd_launch<T, P, 8, 1, 2>(a);
    if (c <= 16)
        return fwd_launch<T, P, 8, 2, 2>(a);
    if (c <= 32)
        return fwd_launch<T, P, 16, 2, 2>(a);
    if (c <= 64)
        return fwd_launch<T, P, 32, 2, 2>(a);
    if (c <= 128)
        return fwd_launch<T, P, 64, 2, 2>(a);
    if (c <= 256)
        return fwd_launch<T, P, 128, 2, 2>(a);
    if (c <= 512)
        return fwd_launch<T, P, 256, 2, 2>(a);
    if (c <= 1024)
        return fwd_launch<T, P, 256, 4, 1>(a);
    if (c <= 2048)
        return fwd_launch<T, P, 1024, 2, 1>(a);
    int64_t grid = a.rows < kMaxGrid ? a.rows : kMaxGrid;
    void* args[] = {&a.x, &a.ldx, &a.w, &a.b, &a.rows, &a.n, &a.eps, &a.out, &a.ldo, &a.mean,
                    &a.rstd};
    return launch(reinterpret_cast<const void*>(&ln_fwd_long_kernel<T, P>), dim3((unsigned)grid),
                  1024, args, a.stream);
}

template <typename P>
static int params_launch(const float* part, int parts, int n, P* dweight, P* dbias,
                         hipStream_t stream)
{
    void* args[] = {&part, &parts, &n, &dweight, &dbias};
    const int64_t blocks = (2 * (int64_t)n + 31) / 32;
    return launch(reinterpret_cast<const void*>(&ln_params_kernel<P>),
                  dim3((unsigned)(blocks < kMaxGrid ? blocks : kMaxGrid)), 1024, args, stream);
}

template <typename T, typename P, int G, int V, int R>
static int bwd_launch(LnArgs<T, P>& a)
{
    constexpr int NG = Group<G>::kGroups;
    int64_t grid = (a.rows + NG * R - 1) / (NG * R);
    if (grid > kMaxParts)
        grid = kMaxParts;
    void* args[] = {&a.x, &a.ldx, &a.dy, &a.lddy, &a.mean, &a.rstd, &a.w, &a.rows, &a.n, &a.out,
                    &a.ldo, &a.part};
    int rc = launch(reinterpret_cast<const void*>(&ln_bwd_kernel<T, P, G, V, R>),
                    dim3((unsigned)grid), Group<G>::kThreads, args, a.stream);
    if (rc != MESWISH_OK || !a.part)
        return rc;
    return params_launch<P>(a.part, (int)grid, a.n, a.dweight, a.dbias, a.stream);
}

// As forward; here a thread also has the rows that follow in flight, and two
// vectors a thread gain nothing where one does (us):
//   n = 512          64 x 1, 2 rows: 75            32 x 2, 2 rows: 79
//   n = 1024         64 x 2, 1 row: 75             32 x 4, 1 row: 81
//   n = 2048         256 x 1, 2 rows: 79           128 x 2, 2 rows: 82
//   n = 4096         256 x 2, 2 rows: 86           512 x 1, 2 rows: 86
//   n = 8192         256 x 4, 1 row: 97            512 x 2, 2 rows: 101
//   n = 16384        1024 x 2, 1 row: 127          512 x 4, 1 row: 129
template <typename T, typename P>
static int bwd_run(LnArgs<T, P>& a)
{
    if (a.rows == 0)
        return a.part ? params_launch<P>(a.part, 0, a.n, a.dweight, a.dbias, a.stream) : MESWISH_OK;
    const int64_t c = chunks<T>(a.n);
    if (c <= 4)
        return bwd_launch<T, P, 4, 1, 2>(a);
    if (c <= 8)
        return bwd_launch<T, P, 8, 1, 2>(a);
    if (c <= 16)
        return bwd_launch<T, P, 16, 1, 2>(a);
    if (c <= 32)
        return bwd_launch<T, P, 32, 1, 2>(a);
    if (c <= 64)
        return bwd_launch<T, P, 64, 1, 2>(a);
    if (c <= 128)
        return bwd_launch<T, P, 64, 2, 1>(a);
    if (c <= 256)
        return bwd_launch<T, P, 256, 1, 2>(a);
    if (c <= 512)
        return bwd_launch<T, P, 256, 2, 2>(a);
    if (c <= 1024)
        return bwd_launch<T, P, 256, 4, 1>(a);
    if (c <= 2048)
        return bwd_launch<T, P, 1024, 2, 1>(a);
    if (a.part) {
        int64_t rowsplit = a.rows < kMaxParts ? a.rows : kMaxParts;
        void* args[] = {&a.x, &a.ldx, &a.dy, &a.lddy, &a.mean, &a.rstd, &a.rows, &a.n, &a.part};
        int rc = launch(reinterpret_cast<const void*>(&ln_cols_kernel<T>),
                        dim3((unsigned)((c + 255) / 256), (unsigned)rowsplit), 256, args, a.stream);
        if (rc == MESWISH_OK)
            rc = params_launch<P>(a.part, (int)rowsplit, a.n, a.dweight, a.dbias, a.stream);
        if (rc != MESWISH_OK)
            return rc;
    }
    int64_t grid = a.rows < kMaxGrid ? a.rows : kMaxGrid;
    void* args[] = {&a.x, &a.ldx, &a.dy, &a.lddy, &a.mean, &a.rstd, &a.w, &a.rows, &a.n, &a.out,
                    &a.ldo};
    return launch(reinterpret_cast<const void*>(&ln_bwd_long_kernel<T, P>), dim3((unsigned)grid),
                  1024, args, a.stream);
}

static bool matrix_ok(const void* p, size_t rows, size_t n, size_t ld, size_t es)
{
    if (!p || !aligned(p, es) || n >= ((size_t)1 << 31) || ld < n)
        return false;
    const size_t most = (size_t)1 << 59;
    return rows == 0 || (rows < most && n < most && (ld == 0 || (rows - 1) < (most - n) / ld));
}

}  // namespace meblock

using namespace meblock;

extern "C" size_t layer_norm_workspace_bytes(size_t rows, size_t n)
{
    if (n >= ((size_t)1 << 31))
        return 0;
    // At most one part a row.
    const size_t parts = rows < (size_t)kMaxParts ? (rows ? rows : 1) : (size_t)kMaxParts;
    return parts * 2 * (n ? n : 1) * sizeof(float);
}

extern "C" int layer_norm_fwd(const void* x, size_t ldx, const void* weight, const void* bias,
                              size_t rows, size_t n, float eps, void* y, size_t ldy, float* mean,
                              float* rstd, int dtype, int param_dtype, void* stream)
{
    if (!dtype_ok(dtype) || !dtype_ok(param_dtype) || !isfinite(eps) || eps < 0.0f)
        return MESWISH_EINVAL;
    if (rows == 0 || n == 0)
        return MESWISH_OK;
    const size_t es = elem_size(dtype), ps = elem_size(param_dtype);
    if (!matrix_ok(x, rows, n, ldx, es) || !matrix_ok(y, rows, n, ldy, es) ||
        !aligned(weight, ps) || !aligned(bias, ps) || !aligned(mean, 4) || !aligned(rstd, 4))
        return MESWISH_EINVAL;
    const Span sx = span(x, rows, n, ldx, es), sy = span(y, rows, n, ldy, es);
    const Span sw = span(weight, weight ? 1 : 0, n, n, ps), sb = span(bias, bias ? 1 : 0, n, n, ps);
    const Span sm = span(mean, mean ? 1 : 0, rows, rows, 4), sr = span(rstd, rstd ? 1 : 0, rows, rows, 4);
    if (!same_or_apart(sy, sx) || overlaps(sy, sw) || overlaps(sy, sb) || overlaps(sy, sm) ||
        overlaps(sy, sr) || overlaps(sm, sx) || overlaps(sr, sx) || overlaps(sm, sr) ||
        overlaps(sm, sw) || overlaps(sm, sb) || overlaps(sr, sw) || overlaps(sr, sb))
        return MESWISH_EALIAS;
    auto run = [&](auto t, auto p) {
        using T = decltype(t);
        using P = decltype(p);
        LnArgs<T, P> a{};
        a.x = static_cast<const T*>(x);
        a.w = static_cast<const P*>(weight);
        a.b = static_cast<const P*>(bias);
        a.ldx = (int64_t)ldx;
        a.ldo = (int64_t)ldy;
        a.rows = (int64_t)rows;
        a.n = (int)n;
        a.eps = eps;
        a.out = static_cast<T*>(y);
        a.mean = mean;
        a.rstd = rstd;
        a.stream = static_cast<hipStream_t>(stream);
        return fwd_run<T, P>(a);
    };
    if (dtype == MESWISH_F32)
        return param_dtype == MESWISH_F32 ? run(float(), float()) : run(float(), bf16_t());
    return param_dtype == MESWISH_F32 ? run(bf16_t(), float()) : run(bf16_t(), bf16_t());
}

extern "C" int layer_norm_bwd(const void* x, size_t ldx, const void* dy, size_t lddy,
                              const float* mean, const float* rstd, const void* weight, size_t rows,
                              size_t n, void* dx, size_t lddx, void* dweight, void* dbias,
                              void* workspace, size_t workspace_bytes, int dtype, int param_dtype,
                              void* stream)
{
    if (!dtype_ok(dtype) || !dtype_ok(param_dtype) || n >= ((size_t)1 << 31))
        return MESWISH_EINVAL;
    if (n == 0)
        return MESWISH_OK;
    const size_t es = elem_size(dtype), ps = elem_size(param_dtype);
    const bool sums = dweight || dbias;
    const size_t need = sums ? layer_norm_workspace_bytes(rows, n) : 0;
    if (sums && (!workspace || workspace_bytes < need || !aligned(workspace, 4)))
        return MESWISH_EINVAL;
    if (!aligned(dweight, ps) || !aligned(dbias, ps) || !aligned(weight, ps))
        return MESWISH_EINVAL;
    if (rows > 0 && (!matrix_ok(x, rows, n, ldx, es) || !matrix_ok(dy, rows, n, lddy, es) ||
                     !matrix_ok(dx, rows, n, lddx, es) || !mean || !rstd || !aligned(mean, 4) ||
                     !aligned(rstd, 4)))
        return MESWISH_EINVAL;
    // With no rows every pointer below but the sums' is empty.
    const Span in[] = {span(x, rows, n, ldx, es), span(dy, rows, n, lddy, es),
                       span(mean, rows ? 1 : 0, rows, rows, 4),
                       span(rstd, rows ? 1 : 0, rows, rows, 4),
                       span(weight, weight ? 1 : 0, n, n, ps)};
    const Span out[] = {span(dx, rows, n, lddx, es), span(dweight, dweight ? 1 : 0, n, n, ps),
                        span(dbias, dbias ? 1 : 0, n, n, ps), span(workspace, sums ? 1 : 0, need, need, 1)};
    for (int o = 0; o < 4; ++o) {
        for (int i = 0; i < 5; ++i)
            if (o == 0 && i < 2 ? !same_or_apart(out[o], in[i]) : overlaps(out[o], in[i]))
                return MESWISH_EALIAS;
        for (int i = 0; i < o; ++i)
            if (overlaps(out[o], out[i]))
                return MESWISH_EALIAS;
    }
    auto run = [&](auto t, auto p) {
        using T = decltype(t);
        using P = decltype(p);
        LnArgs<T, P> a{};
        a.x = static_cast<const T*>(x);
        a.dy = static_cast<const T*>(dy);
        a.w = static_cast<const P*>(weight);
        a.ldx = (int64_t)ldx;
        a.lddy = (int64_t)lddy;
        a.ldo = (int64_t)lddx;
        a.rows = (int64_t)rows;
        a.n = (int)n;
        a.out = static_cast<T*>(dx);
        a.mean = const_cast<float*>(mean);
        a.rstd = const_cast<float*>(rstd);
        a.part = sums ? static_cast<float*>(workspace) : nullptr;
        a.dweight = static_cast<P*>(dweight);
        a.dbias = static_cast<P*>(dbias);
        a.stream = static_cast<hipStream_t>(stream);
        return bwd_run<T, P>(a);
    };
    if (dtype == MESWISH_F32)
        return param_dtype == MESWISH_F32 ? run(float(), float()) : run(float(), bf16_t());
    return param_dtype == MESWISH_F32 ? run(bf16_t(), float()) : run(bf16_t(), bf16_t());
}
