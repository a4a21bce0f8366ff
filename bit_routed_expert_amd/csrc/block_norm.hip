// Norms before and after a block with the branch's gate and residual scale
// (strata_block_norm), and their gradient.
//
//   n = y * rstd(y) * g_post;  r = a x + b G n;  u = r * rstd(r) * g_pre
//
// Bound by HBM: every row is read once and written once, so a row lives in
// the registers of G threads (VALS values each) from its first load to its
// last store, and the two norms are two sums over those registers (a wave
// sum by lane exchanges, then the waves' sums through LDS).
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
#include <math.h>

#include "ops.hpp"

namespace strata {

constexpr int BN_MAX_D = 8192;
constexpr int BN_BLOCKS = 1024;    // most blocks of the gradient (rows of partial gain sums)

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

// A thread's VALS values of a row: pieces of V at lane*V, (lane + G)*V, ...;
// places past the row read as 0.
template <int V, int VALS, int G>
__device__ __forceinline__ void row_load(const void *p, int bf16, int64_t row, int d, int lane, float (&v)[VALS]) {
#define ROW_LOAD(T)                                                                 \
    _Pragma("unroll") for (int q = 0; q < VALS / V; ++q) {                          \
        const int i = (q * G + lane) * V;                                           \
        float e[V];                                                                 \
        _Pragma("unroll") for (int j = 0; j < V; ++j) e[j] = 0.f;                   \
        if (i < d) load_values<V>((const T *)p, row + i, e);                        \
        _Pragma("unroll") for (int j = 0; j < V; ++j) v[q * V + j] = e[j];          \
    }
    if (bf16) {
        ROW_LOAD(uint16_t)
    } else {
        ROW_LOAD(float)
    }
#undef ROW_LOAD
}

template <int V, int VALS, int G>
__device__ __forceinline__ void row_store(void *p, int bf16, int64_t row, int d, int lane, const float (&v)[VALS]) {
#define ROW_STORE(T)                                                                \
    _Pragma("unroll") for (int q = 0; q < VALS / V; ++q) {                          \
        const int i = (q * G + lane) * V;                                           \
        float e[V];                                                                 \
        _Pragma("unroll") for (int j = 0; j < V; ++j) e[j] = v[q * V + j];          \
        if (i < d) store_values<V>((T *)p, row + i, e);                             \
    }
    if (bf16) {
        ROW_STORE(uint16_t)
    } else {
        ROW_STORE(float)
    }
#undef ROW_STORE
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
__device__ __forceinline__ void gate_value(float v, bool sigmoid, float &g, float &dg) {
    g = v;
    dg = 1.f;
    if (sigmoid) {
        g = 1.f / (1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * v));
        dg = g * (1.f - g);
    }
}

__device__ __forceinline__ float rstd_of(float sum, int d, float eps) { return 1.f / sqrtf(sum / (float)d + eps); }

template <int V, int VALS, int G> __global__ __launch_bounds__(256) void block_norm_kernel(NormArgs a) {
    __shared__ float red[4];
    const int lane = threadIdx.x % G;
    int t = (int)blockIdx.x * (256 / G) + (int)(threadIdx.x / G);
    t = __builtin_amdgcn_readfirstlane(t);
    const bool live = t < a.T;   // G = 256: every block's row; G = 64: no barriers below
    if (!live) return;
    const int d = a.d;
    const int64_t row = (int64_t)t * d;
    float x[VALS], y[VALS], gt[VALS];
    float tg = 1.f;
    const bool post = a.flags & STRATA_POST_NORM, pre = a.flags & STRATA_PRE_NORM;
    const bool sig = a.flags & STRATA_GATE_SIGMOID, chan = a.flags & STRATA_GATE_CHANNEL;
    if (a.y) row_load<V, VALS, G>(a.y, a.y_bf16, row, d, lane, y);
    row_load<V, VALS, G>(a.x, a.x_bf16, row, d, lane, x);
    if (chan) row_load<V, VALS, G>(a.gate, a.y_bf16, row, d, lane, gt);
    if (a.flags & STRATA_GATE_TOKEN) {
        float unused;
        gate_value(((const float *)a.gate)[t], sig, tg, unused);
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
        float gp[VALS];
        if (a.g_post) row_load<V, VALS, G>(a.g_post, 0, 0, d, lane, gp);
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
    if (a.r) row_store<V, VALS, G>(a.r, a.x_bf16, row, d, lane, x);
    if (!pre) return;
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < VALS; ++j) {
        if (((j / V) * G + lane) * V < d) ss = fmaf(x[j], x[j], ss);
    }
    const float rr = rstd_of(group_sum<G>(ss, red), d, a.eps);
    if (a.rstd_r && lane == 0) a.rstd_r[t] = rr;
    float gp[VALS];
    if (a.g_pre) row_load<V, VALS, G>(a.g_pre, 0, 0, d, lane, gp);
#pragma unroll
    for (int j = 0; j < VALS; ++j) {
        x[j] *= rr;
        if (a.g_pre) x[j] *= gp[j];
    }
    row_store<V, VALS, G>(a.u, a.u_bf16, row, d, lane, x);
}

// 256 / G rows at a time per block; the waves of a G = 64 block keep partial
// gain sums of their own and add them in LDS order at the end.
template <int V, int VALS, int G> __global__ __launch_bounds__(256) void block_norm_back_kernel(NormArgs a) {
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
    if (a.g_post) row_load<V, VALS, G>(a.g_post, 0, 0, d, lane, gpost);
    if (a.g_pre) row_load<V, VALS, G>(a.g_pre, 0, 0, d, lane, gpre);
    const float inv_d = 1.f / (float)d;
    for (int t0 = (int)blockIdx.x * NG; t0 < a.T; t0 += a.blocks * NG) {
        const int t = __builtin_amdgcn_readfirstlane(t0 + grp);
        if (t >= a.T) break;   // only where G = 64: waves without barriers
        const int64_t row = (int64_t)t * d;
        float D[VALS];
        if (a.dr) {
            row_load<V, VALS, G>(a.dr, a.x_bf16, row, d, lane, D);
        } else {
#pragma unroll
            for (int j = 0; j < VALS; ++j) D[j] = 0.f;
        }
        if (pre) {
            float u[VALS], r[VALS];
            row_load<V, VALS, G>(a.du, a.u_bf16, row, d, lane, u);
            row_load<V, VALS, G>(a.rin, a.x_bf16, row, d, lane, r);
            const float rr = a.rstd_r_in[t];
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
            row_store<V, VALS, G>(a.dx, a.x_bf16, row, d, lane, o);
        }
        if (!a.y || !(a.dy || a.dgate || a.dg_post)) continue;
        float y[VALS], gt[VALS];
        row_load<V, VALS, G>(a.y, a.y_bf16, row, d, lane, y);
        const float ry = post ? a.rstd_y_in[t] : 1.f;
        float tg = 1.f, tdg = 1.f;
        if (tok) gate_value(((const float *)a.gate)[t], sig, tg, tdg);
        if (chan) row_load<V, VALS, G>(a.gate, a.y_bf16, row, d, lane, gt);
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
        if (chan && a.dgate) row_store<V, VALS, G>(a.dgate, a.y_bf16, row, d, lane, gt);
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
            row_store<V, VALS, G>(a.dy, a.y_bf16, row, d, lane, D);
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
        if (grp == 0) row_store<V, VALS, G>(PART, 0, (int64_t)blockIdx.x * d, d, lane, SUM);       \
    }
    GAIN_PART(a.dg_post, spost, a.part_post)
    GAIN_PART(a.dg_pre, spre, a.part_pre)
#undef GAIN_PART
}

// Gain gradients from the blocks' partial sums, added in block order: 32
// columns per block, 32 threads' worth of blocks side by side for each.
__global__ __launch_bounds__(1024) void block_norm_gains_kernel(NormArgs a) {
    __shared__ float s[32][33];
    const float *part = blockIdx.y ? a.part_pre : a.part_post;
    float *out = blockIdx.y ? a.dg_pre : a.dg_post;
    if (!out) return;
    const int c = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + c;
    float v = 0.f;
    if (i < a.d) {
#pragma unroll 4
        for (int b = q; b < a.blocks; b += 32) v += part[(int64_t)b * a.d + i];
    }
    s[q][c] = v;
    __syncthreads();
    if (threadIdx.x < 32 && blockIdx.x * 32 + threadIdx.x < a.d) {
        float t = 0.f;
#pragma unroll
        for (int b = 0; b < 32; ++b) t += s[b][threadIdx.x];
        out[blockIdx.x * 32 + threadIdx.x] = t;
    }
}

namespace {

strata_status check_norm(const strata_block_norm_args *p) {
    if (!p || p->T < 0 || p->d < 1) return STRATA_EINVAL;
    if (bad_dtype(p->x_dtype) || bad_dtype(p->y_dtype) || bad_dtype(p->u_dtype)) return STRATA_EINVAL;
    const uint32_t f = p->flags;
    if (f & ~31u) return STRATA_EINVAL;
    const bool tok = f & STRATA_GATE_TOKEN, chan = f & STRATA_GATE_CHANNEL;
    if ((tok && chan) || ((f & STRATA_GATE_SIGMOID) && !tok && !chan)) return STRATA_EINVAL;
    if (!(p->eps > 0.f) || !isfinite(p->eps) || !isfinite(p->resid_scale) || !isfinite(p->branch_scale))
        return STRATA_EINVAL;
    if (p->d > BN_MAX_D || p->T > MAX_ROWS) return STRATA_EUNSUPPORTED;
    return STRATA_OK;
}

// What the flags ask for and what is given have to agree.
strata_status check_norm_inputs(const strata_block_norm_args *p, const void *y, const void *gate, const float *g_post,
                                const float *g_pre) {
    const bool gated = p->flags & (STRATA_GATE_TOKEN | STRATA_GATE_CHANNEL);
    if (!y && (gated || (p->flags & STRATA_POST_NORM))) return STRATA_EINVAL;
    if (gated != (gate != nullptr)) return STRATA_EINVAL;
    if (g_post && !(p->flags & STRATA_POST_NORM)) return STRATA_EINVAL;
    if (g_pre && !(p->flags & STRATA_PRE_NORM)) return STRATA_EINVAL;
    return STRATA_OK;
}

NormArgs norm_args(const strata_block_norm_args *p) {
    NormArgs a{};
    a.T = p->T;
    a.d = p->d;
    a.x_bf16 = p->x_dtype == STRATA_X_BF16;
    a.y_bf16 = p->y_dtype == STRATA_X_BF16;
    a.u_bf16 = p->u_dtype == STRATA_X_BF16;
    a.flags = p->flags;
    a.a = p->resid_scale;
    a.b = p->branch_scale;
    a.eps = p->eps;
    return a;
}

// Threads per row and values per thread: a wave alone up to 1024 columns
// (no barrier), a block above.
bool wave_rows(int d) { return d <= 1024; }

int back_blocks(const strata_block_norm_args *p) {
    const int64_t rows = wave_rows(p->d) ? ((int64_t)p->T + 3) / 4 : p->T;
    return (int)(rows < BN_BLOCKS ? rows : BN_BLOCKS);
}

#define NORM_SIZES(KER, V, GRID_WAVE, GRID_BLOCK)                                                           \
    do {                                                                                                    \
        if (a.d <= 512) STRATA_LAUNCH((KER<V, 8, 64>), dim3(GRID_WAVE), dim3(256), 0, s, a);                \
        else if (a.d <= 1024) STRATA_LAUNCH((KER<V, 16, 64>), dim3(GRID_WAVE), dim3(256), 0, s, a);         \
        else if (a.d <= 2048) STRATA_LAUNCH((KER<V, 8, 256>), dim3(GRID_BLOCK), dim3(256), 0, s, a);        \
        else if (a.d <= 4096) STRATA_LAUNCH((KER<V, 16, 256>), dim3(GRID_BLOCK), dim3(256), 0, s, a);       \
        else STRATA_LAUNCH((KER<V, 32, 256>), dim3(GRID_BLOCK), dim3(256), 0, s, a);                        \
    } while (0)
// Pieces of 8 values where the row allows (16 bytes of bf16, twice that of fp32), else 2 or 1.
#define NORM_LAUNCH(KER, GRID_WAVE, GRID_BLOCK)                          \
    do {                                                                 \
        if (a.d % 8 == 0) NORM_SIZES(KER, 8, GRID_WAVE, GRID_BLOCK);     \
        else if (a.d % 2 == 0) NORM_SIZES(KER, 2, GRID_WAVE, GRID_BLOCK); \
        else NORM_SIZES(KER, 1, GRID_WAVE, GRID_BLOCK);                  \
    } while (0)

}  // namespace

}  // namespace strata

using namespace strata;

extern "C" {

strata_status strata_block_norm(const strata_block_norm_args *args, const void *x, const void *y, const void *gate,
                                const float *g_post, const float *g_pre, void *r, void *u, float *rstd_y,
                                float *rstd_r, void *stream) {
    strata_status st = check_norm(args);
    if (st != STRATA_OK || args->T == 0) return st;
    st = check_norm_inputs(args, y, gate, g_post, g_pre);
    if (st != STRATA_OK) return st;
    const bool pre = args->flags & STRATA_PRE_NORM, post = args->flags & STRATA_POST_NORM;
    if (bad_rows(x) || pre != (u != nullptr) || (!r && !u)) return STRATA_EINVAL;
    if ((rstd_y && !post) || (rstd_r && !pre)) return STRATA_EINVAL;
    if (!aligned16(y) || !aligned16(gate) || !aligned16(g_post) || !aligned16(g_pre) || !aligned16(r) || !aligned16(u))
        return STRATA_EINVAL;
    NormArgs a = norm_args(args);
    a.x = x;
    a.y = y;
    a.gate = gate;
    a.g_post = g_post;
    a.g_pre = g_pre;
    a.r = r;
    a.u = u;
    a.rstd_y = rstd_y;
    a.rstd_r = rstd_r;
    const hipStream_t s = (hipStream_t)stream;
    NORM_LAUNCH(block_norm_kernel, (unsigned)((a.T + 3) / 4), (unsigned)a.T);
    return hip_status(hipGetLastError());
}

size_t strata_block_norm_backward_workspace_bytes(const strata_block_norm_args *args) {
    if (check_norm(args) != STRATA_OK) return 0;
    const size_t n = (size_t)2 * back_blocks(args) * args->d * 4;
    return n ? n : 256;
}

strata_status strata_block_norm_backward(const strata_block_norm_args *args, const void *dr, const void *du,
                                         const void *r, const void *y, const void *gate, const float *g_post,
                                         const float *g_pre, const float *rstd_y, const float *rstd_r, void *dx,
                                         void *dy, void *dgate, float *dg_post, float *dg_pre, void *ws,
                                         size_t ws_bytes, void *stream) {
    strata_status st = check_norm(args);
    if (st != STRATA_OK) return st;
    const bool pre = args->flags & STRATA_PRE_NORM, post = args->flags & STRATA_POST_NORM;
    if ((dg_post && !post) || (dg_pre && !pre)) return STRATA_EINVAL;
    if (!aligned16(dg_post) || !aligned16(dg_pre)) return STRATA_EINVAL;
    const bool rows = args->T > 0, gains = dg_post || dg_pre;
    if (rows) {
        st = check_norm_inputs(args, y, gate, g_post, g_pre);
        if (st != STRATA_OK) return st;
        if (pre != (du != nullptr) || (!dr && !du) || (pre && (!r || !rstd_r))) return STRATA_EINVAL;
        if (y && post && !rstd_y) return STRATA_EINVAL;
        if ((dy && !y) || (dgate && !gate)) return STRATA_EINVAL;
        if (!aligned16(dr) || !aligned16(du) || !aligned16(r) || !aligned16(y) || !aligned16(gate) ||
            !aligned16(g_post) || !aligned16(g_pre) || !aligned16(dx) || !aligned16(dy) || !aligned16(dgate))
            return STRATA_EINVAL;
        if (gains && (!ws || !aligned16(ws))) return STRATA_EINVAL;
        if (gains && ws_bytes < strata_block_norm_backward_workspace_bytes(args)) return STRATA_EWORKSPACE;
    }
    NormArgs a = norm_args(args);
    a.dr = dr;
    a.du = du;
    a.rin = r;
    a.y = y;
    a.gate = gate;
    a.g_post = g_post;
    a.g_pre = g_pre;
    a.rstd_y_in = rstd_y;
    a.rstd_r_in = rstd_r;
    a.dx = dx;
    a.dy = dy;
    a.dgate = dgate;
    a.dg_post = dg_post;
    a.dg_pre = dg_pre;
    a.blocks = back_blocks(args);
    a.part_post = (float *)ws;
    a.part_pre = (float *)ws + (size_t)a.blocks * a.d;
    const hipStream_t s = (hipStream_t)stream;
    if (rows && (dx || dy || dgate || gains)) {
        NORM_LAUNCH(block_norm_back_kernel, (unsigned)a.blocks, (unsigned)a.blocks);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return hip_status(e);
    }
    if (gains) {   // no rows: no partial sums, zeros
        STRATA_LAUNCH(block_norm_gains_kernel, dim3((a.d + 31) / 32, 2), dim3(1024), 0, s, a);
        return hip_status(hipGetLastError());
    }
    return STRATA_OK;
}

}  // extern "C"
