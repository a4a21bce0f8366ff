// Shared by the operators around the layer (strata_ops.h): host checks, and
// vector loads and stores of bf16 or fp32 rows as fp32 values.
#pragma once
#include "mfma.hpp"
#include "strata_ops.h"

namespace strata {

// Most tokens of a call: one 256-thread block each stays inside a grid's 2^32 threads.
constexpr int32_t MAX_ROWS = 1 << 23;
constexpr int32_t MAX_COLS = 1 << 24;   // longest row of dispatch and combine

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline bool bad_dtype(int32_t t) { return t != STRATA_X_BF16 && t != STRATA_X_F32; }
// Two buffers of a and b bytes that share memory (null or empty: none does).
inline bool overlap(const void *p, size_t a, const void *q, size_t b) {
    return p && q && a && b && (uintptr_t)p < (uintptr_t)q + b && (uintptr_t)q < (uintptr_t)p + a;
}
// A required row pointer: there and aligned.
inline bool bad_rows(const void *p) { return !p || !aligned16(p); }

// V consecutive values at p + i, aligned to V elements (up to 16 bytes at a
// time), as loaded.  Loads and conversions are apart so that a kernel can
// issue all its loads before it waits for the first.
template <typename E, int V> struct Raw;
template <int V> struct Raw<float, V> { float w[V]; };
template <int V> struct Raw<uint16_t, V> { uint32_t w[V >= 2 ? V / 2 : 1]; };

// Vector types of whole accesses, with the streaming hint (STREAM: what is
// read or written once and not soon again stays out of the caches' way).
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
template <bool STREAM, typename T> __device__ __forceinline__ T get(const T *p) {
    if constexpr (STREAM) return __builtin_nontemporal_load(p);
    return *p;
}
template <bool STREAM, typename T> __device__ __forceinline__ void put(T *p, T v) {
    if constexpr (STREAM) __builtin_nontemporal_store(v, p);
    else *p = v;
}

template <int V, bool STREAM = false>
__device__ __forceinline__ void load_raw(const uint16_t *p, int64_t i, Raw<uint16_t, V> &r) {
    if constexpr (V == 8) {
        const u32x4_t q = get<STREAM>((const u32x4_t *)(p + i));
#pragma unroll
        for (int j = 0; j < 4; ++j) r.w[j] = q[j];
    } else if constexpr (V == 4) {
        const u32x2_t q = get<STREAM>((const u32x2_t *)(p + i));
        r.w[0] = q[0];
        r.w[1] = q[1];
    } else if constexpr (V == 2) {
        r.w[0] = get<STREAM>((const uint32_t *)(p + i));
    } else {
        r.w[0] = p[i];
    }
}
template <int V, bool STREAM = false>
__device__ __forceinline__ void load_raw(const float *p, int64_t i, Raw<float, V> &r) {
    if constexpr (V >= 4) {
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            const f32x4_t q = get<STREAM>((const f32x4_t *)(p + i + j));
#pragma unroll
            for (int c = 0; c < 4; ++c) r.w[j + c] = q[c];
        }
    } else if constexpr (V == 2) {
        const f32x2_t q = get<STREAM>((const f32x2_t *)(p + i));
        r.w[0] = q[0];
        r.w[1] = q[1];
    } else {
        r.w[0] = p[i];
    }
}
template <typename E, int V> __device__ __forceinline__ void zero_raw(Raw<E, V> &r) {
#pragma unroll
    for (auto &w : r.w) w = 0;
}

// Value j of a loaded piece as fp32.
template <int V> __device__ __forceinline__ float value(const Raw<float, V> &r, int j) { return r.w[j]; }
template <int V> __device__ __forceinline__ float value(const Raw<uint16_t, V> &r, int j) {
    return __uint_as_float(V == 1 || !(j & 1) ? r.w[j / 2] << 16 : r.w[j / 2] & 0xFFFF0000u);
}

// Two values rounded to bf16 in one word (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{a, b}), bf16x2_t));
}

template <int V, bool STREAM = false>
__device__ __forceinline__ void store_values(uint16_t *p, int64_t i, const float (&v)[V]) {
    if constexpr (V == 8) {
        put<STREAM>((u32x4_t *)(p + i), u32x4_t{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                                                bf16_pair(v[6], v[7])});
    } else if constexpr (V == 4) {
        put<STREAM>((u32x2_t *)(p + i), u32x2_t{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])});
    } else if constexpr (V == 2) {
        put<STREAM>((uint32_t *)(p + i), bf16_pair(v[0], v[1]));
    } else {
        p[i] = f2bf(v[0]);
    }
}
template <int V, bool STREAM = false>
__device__ __forceinline__ void store_values(float *p, int64_t i, const float (&v)[V]) {
    if constexpr (V >= 4) {
#pragma unroll
        for (int j = 0; j < V; j += 4) put<STREAM>((f32x4_t *)(p + i + j), f32x4_t{v[j], v[j + 1], v[j + 2], v[j + 3]});
    } else if constexpr (V == 2) {
        put<STREAM>((f32x2_t *)(p + i), f32x2_t{v[0], v[1]});
    } else {
        p[i] = v[0];
    }
}

}  // namespace strata
