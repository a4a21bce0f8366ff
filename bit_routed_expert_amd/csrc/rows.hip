// Token rows to their picks' slots and back (strata_moe_dispatch, _combine
// and their gradients).
//
// All four are bound by HBM: a pick's row is read or written once, a token's
// row once.  The work is token-major: a group of G threads takes one token,
// keeps a V-element piece of its row in registers and meets the k picked
// rows, so x and dout are read once however many picks a token has and
// every sum runs over r in order in one thread.  G is a power of two from 16
// to 256, V the widest vector up to 16 bytes that divides the row.
//
// Rows are read and written with the streaming hint: each once, and a prompt
// chunk's slots (168 MB) are most of what the caches hold.  4096 tokens of
// 2048 bf16, 10 picks of 512 experts, four sets of rows in turn: combine 40.0
// -> 34.4 us (5.9 TB/s), its gradient 74.0 -> 70.7 us (5.0 TB/s), dispatch
// 34.9 -> 34.5 us (5.4 TB/s); dispatch into the same slots over and over, which
// the last-level cache holds, 28.8 -> 34.7 us; with the experts' product right
// behind, within 1% either way.
#include "rows.hpp"

namespace strata {

constexpr int PB = 16;   // picked rows in flight per thread

// The positions (and weights) of up to PB picks r0.. of a token, -1 behind
// the k-th.  Groups of whole waves read them once, a pick to a lane, and pass
// them on as scalars; smaller groups read them lane by lane.
template <int G> struct Picks {
    int pos[PB];
    float w[PB];
    __device__ __forceinline__ void read(const int32_t *pt, const float *wt, int r0, int k, int rows) {
        if constexpr (G >= 64) {
            const int lane = threadIdx.x & 63;
            const int r = r0 + (lane & (PB - 1));
            const int p = r < k ? pt[r] : -1;
            const int v = wt ? __builtin_bit_cast(int, r < k ? wt[r] : 0.f) : __builtin_bit_cast(int, 1.f);
#pragma unroll
            for (int q = 0; q < PB; ++q) {
                const int c = __builtin_amdgcn_readlane(p, q);
                pos[q] = (uint32_t)c < (uint32_t)rows ? c : -1;
                w[q] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(v, q));
            }
        } else {
#pragma unroll
            for (int q = 0; q < PB; ++q) {
                pos[q] = -1;
                w[q] = 1.f;
                if (r0 + q < k) {
                    const int c = pt[r0 + q];
                    pos[q] = (uint32_t)c < (uint32_t)rows ? c : -1;
                    if (wt) w[q] = wt[r0 + q];
                }
            }
        }
    }
};

template <typename P, int G>
__global__ __launch_bounds__(256) void dispatch_kernel(const P *__restrict__ x, const int32_t *__restrict__ pos,
                                                       P *__restrict__ xs, int T, int k, int nc, int rows) {
    int t, lane;
    if (!row_group<G>(T, t, lane)) return;
    const int c0 = blockIdx.y * G + lane, step = gridDim.y * G;   // the blocks of a token share its row
    P v = c0 < nc ? x[(int64_t)t * nc + c0] : P{};
    for (int r0 = 0; r0 < k; r0 += PB) {
        Picks<G> pk;
        pk.read(pos + (int64_t)t * k, nullptr, r0, k, rows);
        for (int c = c0; c < nc; c += step) {
            if (c != c0 || r0) v = x[(int64_t)t * nc + c];
#pragma unroll
            for (int r = 0; r < PB; ++r)
                if (pk.pos[r] >= 0) put<true>(xs + (int64_t)pk.pos[r] * nc + c, v);
        }
    }
}

template <typename Y, typename O, int V, int G>
__global__ __launch_bounds__(256) void combine_rows_kernel(const Y *__restrict__ ys, const int32_t *__restrict__ pos,
                                                           const float *__restrict__ w, const O *base, O *out, int T,
                                                           int k, int d, int rows) {
    int t, lane;
    if (!row_group<G>(T, t, lane)) return;
    const int32_t *pt = pos + (int64_t)t * k;
    const float *wt = w ? w + (int64_t)t * k : nullptr;
    Picks<G> pk;
    pk.read(pt, wt, 0, k, rows);
    // the trip count is the group's, so that a second batch of picks is read by whole waves
    for (int i0 = blockIdx.y * (G * V); i0 < d; i0 += gridDim.y * (G * V)) {
        const int i = i0 + lane * V;
        const bool in = i < d;
        Raw<O, V> b;
        zero_raw(b);
        if (base && in) load_raw<V, true>(base, (int64_t)t * d + i, b);
        float s[V];
        for (int r0 = 0; r0 < k; r0 += PB) {
            if (k > PB) pk.read(pt, wt, r0, k, rows);
            Raw<Y, V> v[PB];
#pragma unroll
            for (int r = 0; r < PB; ++r)
                if (pk.pos[r] >= 0 && in) load_raw<V, true>(ys, (int64_t)pk.pos[r] * d + i, v[r]);
            if (r0 == 0) {
#pragma unroll
                for (int j = 0; j < V; ++j) s[j] = value<V>(b, j);
            }
#pragma unroll
            for (int r = 0; r < PB; ++r) {
                if (pk.pos[r] >= 0) {
#pragma unroll
                    for (int j = 0; j < V; ++j) s[j] = fmaf(pk.w[r], value<V>(v[r], j), s[j]);
                }
            }
        }
        if (in) store_values<V, true>(out, (int64_t)t * d + i, s);
    }
}

// Gradient of the combine: per token, each pick's row is read for its dot
// product with dout and written as w * dout in the same pass.
template <typename Y, typename O, int V, int G>
__global__ __launch_bounds__(256) void combine_back_kernel(const O *__restrict__ dout, const Y *ys,
                                                           const int32_t *__restrict__ pos,
                                                           const float *__restrict__ w, Y *dys, float *dw, float *dz,
                                                           int T, int k, int d, int rows) {
    constexpr int NG = 256 / G, NW = G / 64;   // tokens per block, waves per token
    __shared__ float part[NG][NW][32];
    int t, lane;
    const bool live = row_group<G>(T, t, lane);
    const int g = threadIdx.x / G, wv = (threadIdx.x % G) / 64;
    const bool dots = dw || dz;
    // lane r of the group's first wave ends with pick r: its weight and position, read while the rows are
    const int th = threadIdx.x % G;
    float wr = 0.f;
    int pr = -1;
    if (dz && live && th < k) {
        wr = w[(int64_t)t * k + th];
        pr = pos[(int64_t)t * k + th];
    }
    if (live) {
        const int32_t *pt = pos + (int64_t)t * k;
        const float *wt = w + (int64_t)t * k;
        for (int r0 = 0; r0 < k; r0 += PB) {
            Picks<G> pk;
            pk.read(pt, wt, r0, k, rows);
            float dot[PB];
#pragma unroll
            for (int r = 0; r < PB; ++r) dot[r] = 0.f;
            for (int i = lane * V; i < d; i += G * V) {
                Raw<O, V> oraw;
                load_raw<V, true>(dout, (int64_t)t * d + i, oraw);
                Raw<Y, V> v[PB];
#pragma unroll
                for (int r = 0; r < PB; ++r)
                    if (dots && pk.pos[r] >= 0) load_raw<V, true>(ys, (int64_t)pk.pos[r] * d + i, v[r]);
                float o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] = value<V>(oraw, j);
#pragma unroll
                for (int r = 0; r < PB; ++r) {
                    if (pk.pos[r] >= 0) {
                        if (dots) {
#pragma unroll
                            for (int j = 0; j < V; ++j) dot[r] = fmaf(o[j], value<V>(v[r], j), dot[r]);
                        }
                        if (dys) {
                            float q[V];
#pragma unroll
                            for (int j = 0; j < V; ++j) q[j] = pk.w[r] * o[j];
                            store_values<V, true>(dys, (int64_t)pk.pos[r] * d + i, q);
                        }
                    }
                }
            }
            if (dots) {
#pragma unroll
                for (int r = 0; r < PB; ++r) dot[r] = wave_sum_dpp(dot[r]);   // side by side; zeros behind the k-th
                if ((threadIdx.x & 63) == 63) {
#pragma unroll
                    for (int r = 0; r < PB; ++r) part[g][wv][r0 + r] = dot[r];
                }
            }
        }
    }
    if (!dots) return;
    __syncthreads();
    if (live && th < 32) {
        float s = 0.f;
        if (th < k) {
#pragma unroll
            for (int q = 0; q < NW; ++q) s += part[g][q][th];
            if (dw) dw[(int64_t)t * k + th] = s;
        }
        if (dz) {
            float q = (uint32_t)pr < (uint32_t)rows ? wr * s : 0.f;   // a skipped pick's weight enters no sum
            q += __shfl_xor(q, 16, 32);
            q += __shfl_xor(q, 8, 32);
            q += __shfl_xor(q, 4, 32);
            q += __shfl_xor(q, 2, 32);
            q += __shfl_xor(q, 1, 32);
            if (th < k) dz[(int64_t)t * k + th] = wr * (s - q);
        }
    }
}

namespace {

strata_status check_rows(const void *a, const void *b, const int32_t *pos, int32_t rows, int32_t T, int32_t k,
                         int32_t d) {
    if (T < 0 || rows < 0 || k < 1 || k > 32 || d < 1) return STRATA_EINVAL;
    if (T == 0) return STRATA_OK;
    if (!pos || bad_rows(b)) return STRATA_EINVAL;
    if (rows > 0 ? bad_rows(a) : (a && !aligned16(a))) return STRATA_EINVAL;
    if (T > MAX_ROWS || (int64_t)T * k > INT32_MAX || d > MAX_COLS) return STRATA_EUNSUPPORTED;
    return STRATA_OK;
}

template <typename P>
void launch_dispatch(const void *x, const int32_t *pos, void *xs, int T, int k, int nc, int rows, hipStream_t s) {
    const RowGroups q = row_groups(T, nc, 16);
#define DISPATCH(G)                                                                                                  \
    case G:                                                                                                          \
        STRATA_LAUNCH((dispatch_kernel<P, G>), row_grid(T, G, q.shares), dim3(256), 0, s, (const P *)x, pos, (P *)xs, T, k, nc, \
                      rows);                                                                                         \
        break;
    switch (q.threads) { DISPATCH(16) DISPATCH(32) DISPATCH(64) DISPATCH(128) DISPATCH(256) }
#undef DISPATCH
}

struct RowCall {
    const void *ys, *in;   // in: base (combine) or dout (its gradient)
    const int32_t *pos;
    const float *w;
    void *out;             // out, or dys
    float *dw, *dz;
    int T, k, d, rows;
    hipStream_t s;
};

struct Combine {
    template <typename Y, typename O, int V> static void run(const RowCall &c) {
        const RowGroups q = row_groups(c.T, c.d / V, 16);
#define COMBINE(G)                                                                                                 \
    case G:                                                                                                        \
        STRATA_LAUNCH((combine_rows_kernel<Y, O, V, G>), row_grid(c.T, G, q.shares), dim3(256), 0, c.s, (const Y *)c.ys, c.pos, \
                      c.w, (const O *)c.in, (O *)c.out, c.T, c.k, c.d, c.rows);                                    \
        break;
        switch (q.threads) { COMBINE(16) COMBINE(32) COMBINE(64) COMBINE(128) COMBINE(256) }
#undef COMBINE
    }
};

struct CombineBack {
    template <typename Y, typename O, int V> static void run(const RowCall &c) {
#define BACK(G)                                                                                                    \
    case G:                                                                                                        \
        STRATA_LAUNCH((combine_back_kernel<Y, O, V, G>), row_grid(c.T, G, 1), dim3(256), 0, c.s, (const O *)c.in,     \
                      (const Y *)c.ys, c.pos, c.w, (Y *)c.out, c.dw, c.dz, c.T, c.k, c.d, c.rows);                 \
        break;
        switch (row_groups(c.T, c.d / V, 64).threads) { BACK(64) BACK(128) BACK(256) }
#undef BACK
    }
};

// The widest pieces that divide the row: 8 values of bf16, 4 of fp32.
template <typename F, typename Y, typename O> void row_width(const RowCall &c) {
    if constexpr (sizeof(Y) == 2) {
        if (c.d % 8 == 0) return F::template run<Y, O, 8>(c);
    }
    if (c.d % 4 == 0) return F::template run<Y, O, 4>(c);
    if (c.d % 2 == 0) return F::template run<Y, O, 2>(c);
    return F::template run<Y, O, 1>(c);
}

template <typename F> strata_status row_types(const RowCall &c, int ydtype, int odtype) {
    const bool yb = ydtype == STRATA_X_BF16, ob = odtype == STRATA_X_BF16;
    if (yb && ob) row_width<F, uint16_t, uint16_t>(c);
    else if (yb) row_width<F, uint16_t, float>(c);
    else if (ob) row_width<F, float, uint16_t>(c);
    else row_width<F, float, float>(c);
    return hip_status(hipGetLastError());
}

}  // namespace

}  // namespace strata

using namespace strata;

extern "C" {

strata_status strata_moe_dispatch(const void *x, strata_xdtype xdtype, int32_t T, int32_t k, int32_t d,
                                  const int32_t *pos, void *xs, int32_t rows, void *stream) {
    if (bad_dtype(xdtype)) return STRATA_EINVAL;
    const strata_status st = check_rows(xs, x, pos, rows, T, k, d);
    if (st != STRATA_OK || T == 0 || rows == 0) return st;
    const hipStream_t s = (hipStream_t)stream;
    const int64_t bytes = (int64_t)d * (xdtype == STRATA_X_BF16 ? 2 : 4);
    if (bytes % 16 == 0) launch_dispatch<u32x4_t>(x, pos, xs, T, k, (int)(bytes / 16), rows, s);
    else if (bytes % 8 == 0) launch_dispatch<u32x2_t>(x, pos, xs, T, k, (int)(bytes / 8), rows, s);
    else if (bytes % 4 == 0) launch_dispatch<uint32_t>(x, pos, xs, T, k, (int)(bytes / 4), rows, s);
    else launch_dispatch<uint16_t>(x, pos, xs, T, k, (int)(bytes / 2), rows, s);
    return hip_status(hipGetLastError());
}

strata_status strata_moe_combine(const void *ys, strata_xdtype ydtype, int32_t rows, const int32_t *pos,
                                 const float *w, int32_t T, int32_t k, int32_t d, const void *base, void *out,
                                 strata_xdtype odtype, void *stream) {
    if (bad_dtype(ydtype) || bad_dtype(odtype)) return STRATA_EINVAL;
    const strata_status st = check_rows(ys, out, pos, rows, T, k, d);
    if (st != STRATA_OK || T == 0) return st;
    if (base && !aligned16(base)) return STRATA_EINVAL;
    return row_types<Combine>(RowCall{ys, base, pos, w, out, nullptr, nullptr, T, k, d, rows, (hipStream_t)stream},
                              ydtype, odtype);
}

strata_status strata_moe_dispatch_backward(const void *dxs, strata_xdtype xdtype, int32_t rows, const int32_t *pos,
                                           int32_t T, int32_t k, int32_t d, void *dx, void *stream) {
    return strata_moe_combine(dxs, xdtype, rows, pos, nullptr, T, k, d, nullptr, dx, xdtype, stream);
}

strata_status strata_moe_combine_backward(const void *dout, strata_xdtype odtype, const void *ys,
                                          strata_xdtype ydtype, int32_t rows, const int32_t *pos, const float *w,
                                          int32_t T, int32_t k, int32_t d, void *dys, float *dw, float *dz,
                                          void *stream) {
    if (bad_dtype(ydtype) || bad_dtype(odtype)) return STRATA_EINVAL;
    const strata_status st = check_rows(ys, dout, pos, rows, T, k, d);
    if (st != STRATA_OK || T == 0) return st;
    if (!w || (dys && !aligned16(dys))) return STRATA_EINVAL;
    if (!dys && !dw && !dz) return STRATA_OK;
    return row_types<CombineBack>(RowCall{ys, dout, pos, w, dys, dw, dz, T, k, d, rows, (hipStream_t)stream}, ydtype,
                                  odtype);
}

}  // extern "C"
