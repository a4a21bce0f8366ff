// Norms before and after a block with the branch's gate and residual scale
// (strata_block_norm), and their gradient.
//
//   n = y * rstd(y) * g_post;  r = a x + b G n;  u = r * rstd(r) * g_pre
//
// Bound by HBM: every row is read once and written once, so a row lives in
// the registers of G threads (VALS values each) from its first load to its
// last store, and the two norms are two sums over those registers (a wave
// sum by lane exchanges, then the waves' sums through LDS).  r and u are
// stored with the streaming hint: 4096 rows of 2048 bf16 20.0 -> 15.4 us (5.5
// TB/s), and a reader right behind loses as much as it gains; the gradient's
// stores are plain (76.5 us against 81.5 over 8191 rows, 4.8 TB/s).
//
// Gradient, with rr = rstd_r, ry = rstd_y, <,> over the row's d elements:
//   dR = dr + rr (g_pre du - r rr^2 <g_pre du, r> / d)
//   dx = a dR;  t = b dR G;  dgate = b dR n G' (summed over the row for a token gate)
//   dy = ry (t g_post - y ry <t g_post, y ry> / d)
//   dg_post = sum over rows t y ry;  dg_pre = sum over rows du r rr
// The gains' sums run over rows: each block keeps its own in registers over
// the rows it takes (block b: rows b, b + blocks, ...), writes them to the
// workspace, and a second launch adds the blocks in order, so the sums have
// one fixed order.
#pragma once
#include "ops.hpp"

namespace strata {

constexpr int BN_MAX_D = 8192;
constexpr int BN_BLOCKS = 512;    // most blocks of the gradient (rows of partial gain sums)

struct NormArgs {
    const void *x, *y, *gate, *dr, *du, *rin;
    const float *g_post, *g_pre, *rstd_y_in, *rstd_r_in;
    void *r, *u, *dx, *dy, *dgate;
    float *rstd_y, *rstd_r, *part_post, *part_pre, *dg_post, *dg_pre;
    int T, d, x_bf16, y_bf16, u_bf16;
    uint32_t flags;
    float a, b, eps;
    int blocks;
};

// A thread's VALS values of a row, as loaded: pieces of V at lane*V,
// (lane + G)*V, ...; a place past the row holds the row's first piece until
// get() makes it 0, so that no load waits behind a branch.  E: the row's
// type, or Any for one that the call names (the rarer widths).
struct Any {};
template <typename E, int V, int VALS, int G> struct Row {
    Raw<E, V> w[VALS / V];
    __device__ __forceinline__ void load(const void *p, int, int64_t row, int d, int lane) {
#pragma unroll
        for (int q = 0; q < VALS / V; ++q) {
            const int i = (q * G + lane) * V;
            load_raw<V>((const E *)p, row + (i < d ? i : 0), w[q]);
        }
    }
    __device__ __forceinline__ void get(int, int d, int lane, float (&v)[VALS]) const {
#pragma unroll
        for (int q = 0; q < VALS / V; ++q) {
            const bool in = (q * G + lane) * V < d;
#pragma unroll
            for (int j = 0; j < V; ++j) v[q * V + j] = in ? value<V>(w[q], j) : 0.f;
        }
    }
};
template <int V, int VALS, int G> struct Row<Any, V, VALS, G> {
    Row<float, V, VALS, G> f;
    Row<uint16_t, V, VALS, G> h;
    __device__ __forceinline__ void load(const void *p, int bf16, int64_t row, int d, int lane) {
        if (bf16) h.load(p, 1, row, d, lane);
        else f.load(p, 0, row, d, lane);
    }
    __device__ __forceinline__ void get(int bf16, int d, int lane, float (&v)[VALS]) const {
        if (bf16) h.get(1, d, lane, v);
        else f.get(0, d, lane, v);
    }
};

template <typename E, int V, int VALS, int G, bool STREAM = false>
__device__ __forceinline__ void row_store(void *p, int bf16, int64_t row, int d, int lane, const float (&v)[VALS]) {
    if constexpr (__is_same(E, Any)) {
        if (bf16) row_store<uint16_t, V, VALS, G, STREAM>(p, 1, row, d, lane, v);
        else row_store<float, V, VALS, G, STREAM>(p, 0, row, d, lane, v);
    } else {
#pragma unroll
        for (int q = 0; q < VALS / V; ++q) {
            const int i = (q * G + lane) * V;
            float e[V];
#pragma unroll
            for (int j = 0; j < V; ++j) e[j] = v[q * V + j];
            if (i < d) store_values<V, STREAM>((E *)p, row + i, e);
        }
    }
}

// Sum over the group's G threads, in every one of them.  red: one float per
// wave of the block; every thread of the block takes part.
template <int G> __device__ __forceinline__ float group_sum(float v, float *red) {
    v = wave_sum(v);
    if (G == 64) return v;
    __syncthreads();   // the sums read before are done with
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < G / 64; ++q) s += red[q];
    return s;
}

// The gate as it multiplies the branch (g) and the derivative of that (dg).
// Of the sigmoid, with e = exp(-v): g = 1 / (1 + e), and g' = g (1 - g) as e g^2,
// since for v > 0 the digits of 1 - g are lost to g's rounding (all from 17 on).
// Below -87, where g is next to the smallest number, e is held at 2^126 so that
// the product stays finite.
__device__ __forceinline__ void gate_value(float v, bool sigmoid, float &g, float &dg) {
    g = v;
    dg = 1.f;
    if (sigmoid) {
        const float e = __builtin_amdgcn_exp2f(-1.4426950408889634f * v);
        g = 1.f / (1.f + e);
        dg = fminf(e, 0x1p126f) * g * g;
    }
}

__device__ __forceinline__ float rstd_of(float sum, int d, float eps) { return 1.f / sqrtf(sum / (float)d + eps); }

template <typename X, typename Y, typename U, int V, int VALS, int G>
__global__ __launch_bounds__(256) void block_norm_kernel(NormArgs a) {
    __shared__ float red[4];
    const int lane = threadIdx.x % G;
    int t = (int)blockIdx.x * (256 / G) + (int)(threadIdx.x / G);
    t = __builtin_amdgcn_readfirstlane(t);
    const bool live = t < a.T;   // G = 256: every block's row; G = 64: no barriers below
    if (!live) return;
    const int d = a.d;
    const int64_t row = (int64_t)t * d;
    float x[VALS], y[VALS], gt[VALS], gp[VALS];
    float tg = 1.f;
    const bool post = a.flags & STRATA_POST_NORM, pre = a.flags & STRATA_PRE_NORM;
    const bool sig = a.flags & STRATA_GATE_SIGMOID, chan = a.flags & STRATA_GATE_CHANNEL;
    // every load first
    Row<X, V, VALS, G> xr;
    Row<Y, V, VALS, G> yr, gr;
    Row<float, V, VALS, G> pr, qr;
    if (a.y) yr.load(a.y, a.y_bf16, row, d, lane);
    xr.load(a.x, a.x_bf16, row, d, lane);
    if (chan) gr.load(a.gate, a.y_bf16, row, d, lane);
    if (a.flags & STRATA_GATE_TOKEN) tg = ((const float *)a.gate)[t];
    if (a.g_post) pr.load(a.g_post, 0, 0, d, lane);
    if (a.g_pre) qr.load(a.g_pre, 0, 0, d, lane);
    if (a.y) yr.get(a.y_bf16, d, lane, y);
    xr.get(a.x_bf16, d, lane, x);
    if (chan) gr.get(a.y_bf16, d, lane, gt);
    if (a.flags & STRATA_GATE_TOKEN) {
        float unused;
        gate_value(tg, sig, tg, unused);
    }
#pragma unroll
    for (int j = 0; j < VALS; ++j) x[j] *= a.a;
    if (a.y) {
        float ry = 1.f;
        if (post) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < VALS; ++j) ss = fmaf(y[j], y[j], ss);
            ry = rstd_of(group_sum<G>(ss, red), d, a.eps);
            if (a.rstd_y && lane == 0) a.rstd_y[t] = ry;
        }
        const float bt = a.b * tg;
        if (a.g_post) pr.get(0, d, lane, gp);
#pragma unroll
        for (int j = 0; j < VALS; ++j) {
            float n = y[j] * ry;
            if (a.g_post) n *= gp[j];
            float c = bt;
            if (chan) {
                float g, dg;
                gate_value(gt[j], sig, g, dg);
                c *= g;
            }
            x[j] = fmaf(c, n, x[j]);
        }
    }
    if (a.r) row_store<X, V, VALS, G, true>(a.r, a.x_bf16, row, d, lane, x);
    if (!pre) return;
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < VALS; ++j) {
        if (((j / V) * G + lane) * V < d) ss = fmaf(x[j], x[j], ss);
    }
    const float rr = rstd_of(group_sum<G>(ss, red), d, a.eps);
    if (a.rstd_r && lane == 0) a.rstd_r[t] = rr;
    if (a.g_pre) qr.get(0, d, lane, gp);
#pragma unroll
    for (int j = 0; j < VALS; ++j) {
        x[j] *= rr;
        if (a.g_pre) x[j] *= gp[j];
    }
    row_store<U, V, VALS, G, true>(a.u, a.u_bf16, row, d, lane, x);
}

// 256 / G rows at a time per block; the waves of a G = 64 block keep partial
// gain sums of their own and add them in LDS order at the end.
template <typename X, typename Y, typename U, int V, int VALS, int G>
__global__ __launch_bounds__(256) void block_norm_back_kernel(NormArgs a) {
    constexpr int NG = 256 / G;
    __shared__ float red[4];
    __shared__ float sums[NG > 1 ? NG : 1][NG > 1 ? VALS * G : 1];
    const int lane = threadIdx.x % G, grp = threadIdx.x / G;
    const int d = a.d;
    const bool post = a.flags & STRATA_POST_NORM, pre = a.flags & STRATA_PRE_NORM;
    const bool sig = a.flags & STRATA_GATE_SIGMOID, chan = a.flags & STRATA_GATE_CHANNEL,
               tok = a.flags & STRATA_GATE_TOKEN;
    float spost[VALS], spre[VALS], gpost[VALS], gpre[VALS];
#pragma unroll
    for (int j = 0; j < VALS; ++j) {
        spost[j] = spre[j] = 0.f;
        gpost[j] = gpre[j] = 1.f;
    }
    {
        Row<float, V, VALS, G> p, q;
        if (a.g_post) p.load(a.g_post, 0, 0, d, lane);
        if (a.g_pre) q.load(a.g_pre, 0, 0, d, lane);
        if (a.g_post) p.get(0, d, lane, gpost);
        if (a.g_pre) q.get(0, d, lane, gpre);
    }
    const bool branch = a.y && (a.dy || a.dgate || a.dg_post);
    const float inv_d = 1.f / (float)d;
    // The next row's loads are issued before the current row's sums (VALS = 8:
    // more values leave no registers for it).
    struct Loaded {
        Row<X, V, VALS, G> dr, r;
        Row<U, V, VALS, G> u;
        Row<Y, V, VALS, G> y, gate;
        float rr, ry, tg;
    };
    constexpr bool AHEAD = VALS == 8;
    const auto load = [&](int t, Loaded &q) {
        const int64_t row = (int64_t)t * d;
        if (pre) {
            q.u.load(a.du, a.u_bf16, row, d, lane);
            q.r.load(a.rin, a.x_bf16, row, d, lane);
            q.rr = a.rstd_r_in[t];
        }
        if (a.dr) q.dr.load(a.dr, a.x_bf16, row, d, lane);
        if (branch) {
            q.y.load(a.y, a.y_bf16, row, d, lane);
            if (chan) q.gate.load(a.gate, a.y_bf16, row, d, lane);
            if (post) q.ry = a.rstd_y_in[t];
            if (tok) q.tg = ((const float *)a.gate)[t];
        }
    };
    const int step = a.blocks * NG;
    int t = __builtin_amdgcn_readfirstlane((int)blockIdx.x * NG + grp);
    Loaded next;
    if (AHEAD && t < a.T) load(t, next);
    // one trip per row of the group; with G = 256 the whole block's, so its barriers meet
    for (; t < a.T; t += step) {
        const int64_t row = (int64_t)t * d;
        Loaded cur;
        if (AHEAD) {
            cur = next;
            if (t + step < a.T) load(t + step, next);
        } else {
            load(t, cur);
        }
        const float rr = pre ? cur.rr : 1.f, ry = post ? cur.ry : 1.f;
        float tg = 1.f, tdg = 1.f;
        float D[VALS];
        if (a.dr) {
            cur.dr.get(a.x_bf16, d, lane, D);
        } else {
#pragma unroll
            for (int j = 0; j < VALS; ++j) D[j] = 0.f;
        }
        if (pre) {
            float u[VALS], r[VALS];
            cur.u.get(a.u_bf16, d, lane, u);
            cur.r.get(a.x_bf16, d, lane, r);
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < VALS; ++j) {
                r[j] *= rr;                        // the normed row
                spre[j] = fmaf(u[j], r[j], spre[j]);
                u[j] *= gpre[j];
                s = fmaf(u[j], r[j], s);
            }
            s = group_sum<G>(s, red) * inv_d;
#pragma unroll
            for (int j = 0; j < VALS; ++j) D[j] = fmaf(rr, fmaf(-s, r[j], u[j]), D[j]);
        }
        if (a.dx) {
            float o[VALS];
#pragma unroll
            for (int j = 0; j < VALS; ++j) o[j] = a.a * D[j];
            row_store<X, V, VALS, G>(a.dx, a.x_bf16, row, d, lane, o);
        }
        if (!branch) continue;
        float y[VALS], gt[VALS];
        cur.y.get(a.y_bf16, d, lane, y);
        if (chan) cur.gate.get(a.y_bf16, d, lane, gt);
        if (tok) gate_value(cur.tg, sig, tg, tdg);
        const float bt = a.b * tg;
        float s = 0.f, sg = 0.f;
#pragma unroll
        for (int j = 0; j < VALS; ++j) {
            y[j] *= ry;                            // the normed row
            float c = bt;
            const float n = y[j] * gpost[j];
            if (tok) sg = fmaf(D[j], n, sg);
            if (chan) {
                float g, dg;
                gate_value(gt[j], sig, g, dg);
                c *= g;
                gt[j] = a.b * D[j] * n * dg;       // the gate's gradient
            }
            D[j] *= c;
            spost[j] = fmaf(D[j], y[j], spost[j]);
            D[j] *= gpost[j];
            s = fmaf(D[j], y[j], s);
        }
        if (chan && a.dgate) row_store<Y, V, VALS, G>(a.dgate, a.y_bf16, row, d, lane, gt);
        if (tok && a.dgate) {
            sg = group_sum<G>(sg, red);
            if (lane == 0) ((float *)a.dgate)[t] = a.b * sg * tdg;
        }
        if (a.dy) {
            if (post) {
                s = group_sum<G>(s, red) * inv_d;
#pragma unroll
                for (int j = 0; j < VALS; ++j) D[j] = ry * fmaf(-s, y[j], D[j]);
            }
            row_store<Y, V, VALS, G>(a.dy, a.y_bf16, row, d, lane, D);
        }
    }
#define GAIN_PART(ON, SUM, PART)                                                                   \
    if (ON) {                                                                                      \
        if (NG > 1) {                                                                              \
            __syncthreads();                                                                       \
            _Pragma("unroll") for (int j = 0; j < VALS; ++j) sums[grp][j * G + lane] = SUM[j];     \
            __syncthreads();                                                                       \
            if (grp == 0) {                                                                        \
                _Pragma("unroll") for (int j = 0; j < VALS; ++j) {                                 \
                    float q = sums[0][j * G + lane];                                               \
                    _Pragma("unroll") for (int g = 1; g < NG; ++g) q += sums[g][j * G + lane];     \
                    SUM[j] = q;                                                                    \
                }                                                                                  \
            }                                                                                      \
        }                                                                                          \
        if (grp == 0) row_store<float, V, VALS, G>(PART, 0, (int64_t)blockIdx.x * d, d, lane, SUM);       \
    }
    GAIN_PART(a.dg_post, spost, a.part_post)
    GAIN_PART(a.dg_pre, spre, a.part_pre)
#undef GAIN_PART
}

// Threads per row and values per thread: a wave alone up to 1024 columns (no
// barrier), a block above.
inline bool wave_rows(int d) { return d <= 1024; }

#define NORM_SIZES(KER, X, Y, U, V, GRID_WAVE, GRID_BLOCK)                                                            \
    do {                                                                                                              \
        if (a.d <= 512) STRATA_LAUNCH((KER<X, Y, U, V, 8, 64>), dim3(GRID_WAVE), dim3(256), 0, s, a);                 \
        else if (a.d <= 1024) STRATA_LAUNCH((KER<X, Y, U, V, 16, 64>), dim3(GRID_WAVE), dim3(256), 0, s, a);          \
        else if (a.d <= 2048) STRATA_LAUNCH((KER<X, Y, U, V, 8, 256>), dim3(GRID_BLOCK), dim3(256), 0, s, a);         \
        else if (a.d <= 4096) STRATA_LAUNCH((KER<X, Y, U, V, 16, 256>), dim3(GRID_BLOCK), dim3(256), 0, s, a);        \
        else STRATA_LAUNCH((KER<X, Y, U, V, 32, 256>), dim3(GRID_BLOCK), dim3(256), 0, s, a);                         \
    } while (0)

// Rows whose length is a multiple of 8, in pieces of 8 values (16 bytes of
// bf16, twice that of fp32): one instantiation per set of types.
template <typename X, typename Y, typename U> hipError_t block_norm_launch(const NormArgs &a, bool back, hipStream_t s) {
    if (back) NORM_SIZES(block_norm_back_kernel, X, Y, U, 8, (unsigned)a.blocks, (unsigned)a.blocks);
    else NORM_SIZES(block_norm_kernel, X, Y, U, 8, (unsigned)((a.T + 3) / 4), (unsigned)a.T);
    return hipGetLastError();
}

// The other lengths, in pieces of 2 or 1, with types that the call names.  The
// gradient holds so many registers that a SIMD has one wave, and above 4096
// columns some in memory.  4096 bf16 rows with both norms and a channel gate,
// forward and gradient, in us (and TB/s): 2048 columns 16 (5.1) and 29 (4.6),
// 2046 21 (4.1) and 54 (2.5), 2047 22 (3.8) and 63 (2.1), 8192 61 (5.5) and 165
// (3.3), 8190 73 (4.6) and 187 (2.9), 8191 176 (1.9) and 366 (1.5).
template <int V> hipError_t block_norm_launch_any(const NormArgs &a, bool back, hipStream_t s) {
    if (back) NORM_SIZES(block_norm_back_kernel, Any, Any, Any, V, (unsigned)a.blocks, (unsigned)a.blocks);
    else NORM_SIZES(block_norm_kernel, Any, Any, Any, V, (unsigned)((a.T + 3) / 4), (unsigned)a.T);
    return hipGetLastError();
}

}  // namespace strata
