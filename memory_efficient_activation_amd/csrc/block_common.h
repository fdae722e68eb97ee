// block_common.h -- what the layer-norm and gated feed-forward kernels
// share: element types, 16-byte accesses at element alignment, and host
// argument checks.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "meswish.h"

namespace meblock {

struct bf16_t {
    uint16_t bits;
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// The same 16 bytes at any element alignment: gfx950's global accesses take
// them (unaligned access mode), so odd row strides need no element path.
typedef u32x4 u32x4_any __attribute__((aligned(2)));

__device__ __forceinline__ u32x4 load16(const void* p) { return *static_cast<const u32x4_any*>(p); }
__device__ __forceinline__ void store16(void* p, u32x4 v) { *static_cast<u32x4_any*>(p) = v; }

typedef __bf16 hw_bf16x2 __attribute__((ext_vector_type(2)));

// Two binary32 values rounded to nearest even, as two bf16 (low half first).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    hw_bf16x2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

template <typename T> struct Elem;

template <> struct Elem<float> {
    static constexpr int kPerVec = 4;
    __device__ static float get(float v) { return v; }
    __device__ static float put(float v) { return v; }
    __device__ static void unpack(u32x4 v, float* f)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // A copy: the bit cast of a vector's element itself reads
            // element 0 whatever i is.
            const uint32_t bits = v[i];
            f[i] = __builtin_bit_cast(float, bits);
        }
    }
    __device__ static u32x4 pack(const float* f)
    {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = __builtin_bit_cast(uint32_t, f[i]);
        return v;
    }
};

template <> struct Elem<bf16_t> {
    static constexpr int kPerVec = 8;
    __device__ static float get(bf16_t v) { return __builtin_bit_cast(float, (uint32_t)v.bits << 16); }
    __device__ static bf16_t put(float v)
    {
        bf16_t r;
        r.bits = (uint16_t)(pack_bf16(v, 0.0f) & 0xffffu);
        return r;
    }
    __device__ static void unpack(u32x4 v, float* f)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __builtin_bit_cast(float, v[i] << 16);
            f[2 * i + 1] = __builtin_bit_cast(float, v[i] & 0xffff0000u);
        }
    }
    __device__ static u32x4 pack(const float* f)
    {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
        return v;
    }
};

// v without its first s elements (0 < s < kPerVec), zeros behind the rest.
template <typename T>
__device__ __forceinline__ u32x4 shift_down(u32x4 v, int s)
{
    constexpr int kPerWord = 4 / (int)sizeof(T);
    uint32_t a = v[0], b = v[1], c = v[2], d = v[3];
    if (s & 2 * kPerWord)
        a = c, b = d, c = d = 0;
    if (s & kPerWord)
        a = b, b = c, c = d, d = 0;
    if (kPerWord == 2 && s & 1) {
        a = a >> 16 | b << 16;
        b = b >> 16 | c << 16;
        c = c >> 16 | d << 16;
        d >>= 16;
    }
    return u32x4{a, b, c, d};
}

// v without its first s elements (0 < s < kPerVec), those behind the rest.
template <typename T>
__device__ __forceinline__ u32x4 rotate_down(u32x4 v, int s)
{
    constexpr int kPerWord = 4 / (int)sizeof(T);
    uint32_t a = v[0], b = v[1], c = v[2], d = v[3];
    if (s & 2 * kPerWord) {
        const uint32_t e = a, f = b;
        a = c, b = d, c = e, d = f;
    }
    if (s & kPerWord) {
        const uint32_t e = a;
        a = b, b = c, c = d, d = e;
    }
    if (kPerWord == 2 && s & 1) {
        const uint32_t e = a;
        a = a >> 16 | b << 16;
        b = b >> 16 | c << 16;
        c = c >> 16 | d << 16;
        d = d >> 16 | e << 16;
    }
    return u32x4{a, b, c, d};
}

// The last elements of a row, from e0 (e0 < n < e0 + kPerVec) on, zeros behind
// them: the row's last whole vector shifted down; a row shorter than a vector
// element by element.  Few registers: this is inlined wherever rows are read.
template <typename T>
__device__ __forceinline__ u32x4 load_tail(const T* row, int e0, int n)
{
    constexpr int E = Elem<T>::kPerVec, kPerWord = 4 / (int)sizeof(T);
    uint32_t a = 0, b = 0, c = 0, d = 0;
    if (n >= E) {
        return shift_down<T>(load16(row + n - E), e0 - (n - E));
    } else {
#pragma unroll 1
        for (int j = 0; j < n - e0; ++j) {
            uint32_t bits = 0;
            __builtin_memcpy(&bits, row + e0 + j, sizeof(T));
            bits <<= j % kPerWord * 16;
            const int w = j / kPerWord;
            a |= w == 0 ? bits : 0;
            b |= w == 1 ? bits : 0;
            c |= w == 2 ? bits : 0;
            d |= w == 3 ? bits : 0;
        }
    }
    return u32x4{a, b, c, d};
}

// Elements e0 .. e0 + kPerVec - 1 of a row of n, as one packed vector; those
// past the end are zero and are not read.  (Here and below whole vectors are
// told by e0 <= n - kPerVec: e0 + kPerVec passes 31 bits where n is nearly
// 2^31.)
template <typename T>
__device__ __forceinline__ u32x4 load_chunk(const T* row, int e0, int n)
{
    if (e0 <= n - Elem<T>::kPerVec)
        return load16(row + e0);
    return e0 < n ? load_tail(row, e0, n) : u32x4{0, 0, 0, 0};
}

// load_chunk in two steps, for rows of a vector or more: a load that takes no
// branch, so that several of them are in flight together, and what makes it
// the chunk, where it is used (n = 0 there: zeros).  For rows of registers, far
// from 2^31: with e0 <= n - kPerVec here the backward of 4096 x 16384 bf16 takes
// 129 us instead of 127.
template <typename T>
__device__ __forceinline__ u32x4 load_near(const T* row, int e0, int n)
{
    constexpr int E = Elem<T>::kPerVec;
    return load16(row + (e0 + E <= n ? e0 : n - E));
}

template <typename T>
__device__ __forceinline__ u32x4 chunk_of(u32x4 v, int e0, int n)
{
    const int s = e0 - (n - Elem<T>::kPerVec);
    if (s >= Elem<T>::kPerVec)
        return u32x4{0, 0, 0, 0};
    return s > 0 ? shift_down<T>(v, s) : v;
}

// load_chunk with other elements of the row, any of them, in the place of the
// zeros past its end (zeros where n = 0).
template <typename T>
__device__ __forceinline__ u32x4 load_repeat(const T* row, int e0, int n)
{
    constexpr int E = Elem<T>::kPerVec, kPerWord = 4 / (int)sizeof(T);
    if (e0 <= n - E)
        return load16(row + e0);
    if (n >= E) {
        const u32x4 v = load16(row + n - E);
        const int s = e0 - (n - E);
        return s < E ? rotate_down<T>(v, s) : v;
    }
    uint32_t a = 0, b = 0, c = 0, d = 0;
#pragma unroll 1
    for (int j = 0; n && j < E; ++j) {
        uint32_t bits = 0;
        __builtin_memcpy(&bits, row + (e0 + j < n ? e0 + j : 0), sizeof(T));
        bits <<= j % kPerWord * 16;
        const int w = j / kPerWord;
        a |= w == 0 ? bits : 0;
        b |= w == 1 ? bits : 0;
        c |= w == 2 ? bits : 0;
        d |= w == 3 ? bits : 0;
    }
    return u32x4{a, b, c, d};
}

template <typename T>
__device__ __forceinline__ void store_chunk(T* row, int e0, int n, const float* f)
{
    constexpr int E = Elem<T>::kPerVec;
    if (e0 <= n - E) {
        store16(row + e0, Elem<T>::pack(f));
        return;
    }
#pragma unroll
    for (int j = 0; j < E; ++j)
        if (e0 + j < n)
            row[e0 + j] = Elem<T>::put(f[j]);
}

// ---------------------------------------------------------------------------
// Host checks.
// ---------------------------------------------------------------------------

inline size_t elem_size(int dtype) { return dtype == MESWISH_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype == MESWISH_F32 || dtype == MESWISH_BF16; }
inline bool aligned(const void* p, size_t a) { return (uintptr_t)p % a == 0; }

// A matrix in memory: `rows` rows of `row_bytes` bytes, `ld_bytes` apart.
struct Span {
    uintptr_t p;
    size_t rows, row_bytes, ld_bytes;
    bool empty() const { return rows == 0 || row_bytes == 0; }
    uintptr_t end() const { return p + (rows - 1) * ld_bytes + row_bytes; }
};

inline Span span(const void* p, size_t rows, size_t cols, size_t ld, size_t es)
{
    return Span{(uintptr_t)p, rows, cols * es, ld * es};
}

// Two matrices share a byte.  Two column ranges of one matrix (the same row
// distance, rows that interleave without touching) do not.
inline bool overlaps(const Span& a, const Span& b)
{
    if (a.empty() || b.empty() || a.end() <= b.p || b.end() <= a.p)
        return false;
    if (a.ld_bytes == b.ld_bytes) {
        const size_t ld = a.ld_bytes;
        const size_t d = b.p >= a.p ? (b.p - a.p) % ld : (ld - (a.p - b.p) % ld) % ld;
        if (d >= a.row_bytes && d + b.row_bytes <= ld)
            return false;
    }
    return true;
}

// An output that coincides exactly with an input, or does not touch it.
inline bool same_or_apart(const Span& out, const Span& in)
{
    return (out.p == in.p && out.row_bytes == in.row_bytes &&
            (out.ld_bytes == in.ld_bytes || out.rows == 1)) ||
           !overlaps(out, in);
}

inline int launch(const void* fn, dim3 grid, int block, void** args, hipStream_t stream)
{
    return hipLaunchKernel(fn, grid, dim3(block), args, 0, stream) == hipSuccess ? MESWISH_OK
                                                                                 : MESWISH_EHIP;
}

}  // namespace meblock
