// Shared by the operators around the layer (strata_ops.h): host checks, and
// vector loads and stores of bf16 or fp32 rows as fp32 values.
#pragma once
#include "mfma.hpp"
#include "strata_ops.h"

namespace strata {

// Most tokens of a call: one 256-thread block each stays inside a grid's 2^32 threads.
constexpr int32_t MAX_ROWS = 1 << 23;

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline bool bad_dtype(int32_t t) { return t != STRATA_X_BF16 && t != STRATA_X_F32; }
// A required row pointer: there and aligned.
inline bool bad_rows(const void *p) { return !p || !aligned16(p); }

// V consecutive values at p + i (elements of E), aligned to V elements (up
// to 16 bytes at a time), as fp32.
template <int V> __device__ __forceinline__ void load_values(const uint16_t *p, int64_t i, float (&v)[V]) {
    if constexpr (V == 8) {
        const uint4 q = *(const uint4 *)(p + i);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    } else if constexpr (V == 4) {
        const uint2 q = *(const uint2 *)(p + i);
        v[0] = __uint_as_float(q.x << 16);
        v[1] = __uint_as_float(q.x & 0xFFFF0000u);
        v[2] = __uint_as_float(q.y << 16);
        v[3] = __uint_as_float(q.y & 0xFFFF0000u);
    } else if constexpr (V == 2) {
        const uint32_t q = *(const uint32_t *)(p + i);
        v[0] = __uint_as_float(q << 16);
        v[1] = __uint_as_float(q & 0xFFFF0000u);
    } else {
        v[0] = bf16_to_float(p[i]);
    }
}
template <int V> __device__ __forceinline__ void load_values(const float *p, int64_t i, float (&v)[V]) {
    if constexpr (V >= 4) {
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            const float4 q = *(const float4 *)(p + i + j);
            v[j] = q.x;
            v[j + 1] = q.y;
            v[j + 2] = q.z;
            v[j + 3] = q.w;
        }
    } else if constexpr (V == 2) {
        const float2 q = *(const float2 *)(p + i);
        v[0] = q.x;
        v[1] = q.y;
    } else {
        v[0] = p[i];
    }
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) { return (uint32_t)f2bf(a) | ((uint32_t)f2bf(b) << 16); }

template <int V> __device__ __forceinline__ void store_values(uint16_t *p, int64_t i, const float (&v)[V]) {
    if constexpr (V == 8) {
        *(uint4 *)(p + i) = make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                                       bf16_pair(v[6], v[7]));
    } else if constexpr (V == 4) {
        *(uint2 *)(p + i) = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
    } else if constexpr (V == 2) {
        *(uint32_t *)(p + i) = bf16_pair(v[0], v[1]);
    } else {
        p[i] = f2bf(v[0]);
    }
}
template <int V> __device__ __forceinline__ void store_values(float *p, int64_t i, const float (&v)[V]) {
    if constexpr (V >= 4) {
#pragma unroll
        for (int j = 0; j < V; j += 4) *(float4 *)(p + i + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    } else if constexpr (V == 2) {
        *(float2 *)(p + i) = make_float2(v[0], v[1]);
    } else {
        p[i] = v[0];
    }
}

}  // namespace strata
