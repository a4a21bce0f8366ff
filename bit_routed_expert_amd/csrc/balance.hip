// Balance losses of a router with the picks counted per expert, and the
// logits' gradient (strata_moe_balance, strata_moe_balance_backward).
//
// Both read the logits once: a wave takes a token, the row lies in its
// registers (up to 16 values a lane).  Forward, a lane adds its experts'
// probabilities over all tokens of the wave; the waves of a block are added
// in LDS, the blocks by a second launch, whose last block sums the losses
// over the experts.  No sum depends on the order in which blocks run.  A
// call of few tokens is one block of one launch.
#include "ops.hpp"

namespace strata {

constexpr int BAL_E = 1024;          // most experts
constexpr int BAL_WAVES = 8;         // of a block
constexpr int BAL_BLOCKS = 512;      // most blocks of the forward launch
constexpr int BAL_ONE = 64;          // tokens up to which one block does it all
constexpr int BAL_SLAB = 64;         // experts of a block of the second launch
constexpr int BAL_SLABS = BAL_E / BAL_SLAB;

struct BalanceArgs {
    const void *z;
    const int32_t *idx;
    const uint8_t *keep;
    int T, k, E, blocks;
    float *losses;
    int32_t *counts;
    float *prob, *lse;
    int32_t *tokens;
    // workspace of the two launches: per block the sums of p, the picks, of lse^2 and the tokens
    float *psum;
    int32_t *csum;
    float *zsum;
    int32_t *nsum;
    float *dots;        // per slab of experts the sum of counts * prob sums
    int32_t *ticket;
};

constexpr float LOG2E = 1.4426950408889634f, LOG2E_LOW = 1.925963033500912e-8f, LN2 = 0.6931471805599453f;

// e^x for x <= 0 to about 2^-23: the rounding of x log2(e) goes back in.
__device__ __forceinline__ float exp_of(float x) {
    const float y = x * LOG2E;
    const float r = fmaf(x, LOG2E, -y) + x * LOG2E_LOW;
    const float e = __builtin_amdgcn_exp2f(y);
    return y > -126.f ? fmaf(e, r * LN2, e) : e;   // far down e is 0, and r may be NaN at -inf
}

// C values of token t: value j of piece i is expert (64 i + lane) V + j; -inf behind the last one.
template <typename Z, int V, int C> struct LogitRow {
    Raw<Z, V> raw[C / V];
    __device__ __forceinline__ static int expert(int i) { return (64 * i + (int)(threadIdx.x & 63)) * V; }
    __device__ __forceinline__ void load(const Z *z, int64_t t, int E) {
#pragma unroll
        for (int i = 0; i < C / V; ++i)
            if (expert(i) < E) load_raw<V>(z, t * E + expert(i), raw[i]);
    }
    __device__ __forceinline__ void values(int E, float (&v)[C]) const {
#pragma unroll
        for (int i = 0; i < C / V; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) v[i * V + j] = expert(i) < E ? value<V>(raw[i], j) : -INFINITY;
    }
};

template <typename Z, int V, int C>
__global__ __launch_bounds__(64 * BAL_WAVES) void balance_rows_kernel(BalanceArgs a) {
    __shared__ float red[BAL_WAVES][64 * C];
    __shared__ int hist[BAL_E];
    __shared__ float zred[BAL_WAVES];
    __shared__ int nred[BAL_WAVES];
    const int th = threadIdx.x, lane = th & 63, w = __builtin_amdgcn_readfirstlane(th >> 6);
    for (int e = th; e < a.E; e += 64 * BAL_WAVES) hist[e] = 0;
    __syncthreads();
    const int first = blockIdx.x * BAL_WAVES + w, step = a.blocks * BAL_WAVES;
    const auto counted = [&](int t) { return t < a.T && (!a.keep || a.keep[t]); };
    float acc[C], zz = 0.f;
    int n = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.f;
    LogitRow<Z, V, C> row;
    int pick = -1;
    bool on = counted(first);
    const auto fetch = [&](int t) {
        row.load((const Z *)a.z, t, a.E);
        pick = lane < a.k ? a.idx[(int64_t)t * a.k + lane] : -1;
    };
    if (on) fetch(first);
    for (int64_t t = first; t < a.T; t += step) {
        float v[C];
        const int e = pick;
        const bool here = on;
        if (here) row.values(a.E, v);
        on = t + step < a.T && counted((int)(t + step));
        if (on) fetch((int)(t + step));
        if (!here) {
            if (lane == 0) a.lse[t] = 0.f;
            continue;
        }
        float m = v[0];
#pragma unroll
        for (int c = 1; c < C; ++c) m = fmaxf(m, v[c]);
        m = wave_max(m);
        if (m == -INFINITY) {   // nothing there, or NaN beside nothing
            bool nan = false;
#pragma unroll
            for (int c = 0; c < C; ++c) nan |= v[c] != v[c];
            if (!__any(nan)) {
                if (lane == 0) a.lse[t] = 0.f;
                continue;
            }
        }
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            v[c] = exp_of(v[c] - m);
            s += v[c];
        }
        s = wave_sum(s);
        const float lse = m + logf(s), r = 1.f / s;
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] = fmaf(v[c], r, acc[c]);
        zz = fmaf(lse, lse, zz);
        ++n;
        if (lane == 0) a.lse[t] = lse;
        if ((uint32_t)e < (uint32_t)a.E) atomicAdd(&hist[e], 1);
    }
#pragma unroll
    for (int i = 0; i < C / V; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) red[w][LogitRow<Z, V, C>::expert(i) + j] = acc[i * V + j];
    if (lane == 0) {
        zred[w] = zz;
        nred[w] = n;
    }
    __syncthreads();
    float z = 0.f;
    n = 0;
#pragma unroll
    for (int q = 0; q < BAL_WAVES; ++q) {
        z += zred[q];
        n += nred[q];
    }
    const bool one = a.blocks == 1;
    float dot = 0.f;
    for (int e = th; e < a.E; e += 64 * BAL_WAVES) {
        float p = 0.f;
#pragma unroll
        for (int q = 0; q < BAL_WAVES; ++q) p += red[q][e];
        const int c = hist[e];
        if (one) {
            p = n ? p / (float)n : 0.f;
            a.counts[e] = c;
            if (a.prob) a.prob[e] = p;
            dot = fmaf((float)c, p, dot);
        } else {
            a.psum[(int64_t)blockIdx.x * a.E + e] = p;
            a.csum[(int64_t)blockIdx.x * a.E + e] = c;
        }
    }
    if (one) {
        __syncthreads();   // zred has been read
        dot = wave_sum(dot);
        if (lane == 0) zred[w] = dot;
        __syncthreads();
        if (th == 0) {
            float d = 0.f;
#pragma unroll
            for (int q = 0; q < BAL_WAVES; ++q) d += zred[q];
            a.losses[0] = n ? d * (float)a.E / ((float)n * (float)a.k) : 0.f;
            a.losses[1] = n ? z / (float)n : 0.f;
            *a.tokens = n;
        }
    } else if (th == 0) {
        a.zsum[blockIdx.x] = z;
        a.nsum[blockIdx.x] = n;
        if (blockIdx.x == 0) *a.ticket = 0;
    }
}

// 64 experts to a block: 16 waves share the blocks' sums.  The block that takes
// the last ticket sums the losses, in the order of the slabs.
__global__ __launch_bounds__(1024) void balance_finish_kernel(BalanceArgs a) {
    __shared__ float pw[16][BAL_SLAB];
    __shared__ int cw[16][BAL_SLAB];
    __shared__ float zw[16];
    __shared__ int nw[16];
    const int th = threadIdx.x, lane = th & 63, w = __builtin_amdgcn_readfirstlane(th >> 6);
    const int e = blockIdx.x * BAL_SLAB + lane, ec = min(e, a.E - 1);
    float p = 0.f;
    int c = 0;
    const int per = (a.blocks + 15) / 16, b0 = w * per, b1 = min(b0 + per, a.blocks);
#pragma unroll 8
    for (int b = b0; b < b1; ++b) {
        p += a.psum[(int64_t)b * a.E + ec];
        c += a.csum[(int64_t)b * a.E + ec];
    }
    pw[w][lane] = p;
    cw[w][lane] = c;
    float z = th < a.blocks ? a.zsum[th] : 0.f;
    int n = th < a.blocks ? a.nsum[th] : 0;
    z = wave_sum(z);
    n = wave_sum(n);
    if (lane == 0) {
        zw[w] = z;
        nw[w] = n;
    }
    __syncthreads();
    if (w) return;
    z = 0.f;
    n = 0;
    p = 0.f;
    c = 0;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
        z += zw[q];
        n += nw[q];
        p += pw[q][lane];
        c += cw[q][lane];
    }
    p = n ? p / (float)n : 0.f;
    float dot = 0.f;
    if (e < a.E) {
        a.counts[e] = c;
        if (a.prob) a.prob[e] = p;
        dot = (float)c * p;
    }
    dot = wave_sum(dot);
    if (lane == 0) {
        __hip_atomic_store(&a.dots[blockIdx.x], dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const bool last =
            __hip_atomic_fetch_add(a.ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
        if (last) {
            float d = 0.f;
            for (int q = 0; q < (int)gridDim.x; ++q)
                d += __hip_atomic_load(&a.dots[q], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            a.losses[0] = n ? d * (float)a.E / ((float)n * (float)a.k) : 0.f;
            a.losses[1] = n ? z / (float)n : 0.f;
            *a.tokens = n;
        }
    }
}

struct BalanceBack {
    const void *z;
    const int32_t *idx;
    const uint8_t *keep;
    int T, k, E, blocks;
    const float *lse;
    const int32_t *counts, *tokens;
    const float *dlosses, *dpicks;
    void *dz;
};

// g is the same for every token and stays in registers.  The picks' gradients
// reach their experts through a row of LDS per wave: lane r holds pick r, the
// first of equal picks adds up all of them in order.
template <typename Z, int V, int C>
__global__ __launch_bounds__(256) void balance_back_kernel(BalanceBack a) {
    __shared__ __attribute__((aligned(16))) float add[4][64 * C];
    const int th = threadIdx.x, lane = th & 63, w = __builtin_amdgcn_readfirstlane(th >> 6);
    typedef LogitRow<Z, V, C> Row;
#pragma unroll
    for (int c = 0; c < C; ++c) add[w][c * 64 + lane] = 0.f;
    const float n = fmaxf((float)*a.tokens, 1.f);
    const float scale = a.dlosses[0] * (float)a.E / (n * n * (float)a.k), zscale = 2.f * a.dlosses[1] / n;
    float g[C];
#pragma unroll
    for (int i = 0; i < C / V; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) g[i * V + j] = Row::expert(i) < a.E ? scale * (float)a.counts[Row::expert(i) + j] : 0.f;
    const int step = a.blocks * 4;
    const auto counted = [&](int64_t t) { return t < a.T && (!a.keep || a.keep[t]); };
    Row row;
    float lse = 0.f, up = 0.f;
    int pick = -1;
    int64_t t = blockIdx.x * 4 + w;
    const auto fetch = [&](int64_t u) {
        row.load((const Z *)a.z, u, a.E);
        lse = a.lse[u];
        if (a.dpicks && lane < a.k) {
            pick = a.idx[u * a.k + lane];
            up = a.dpicks[u * a.k + lane];
        }
    };
    bool on = counted(t);
    if (on) fetch(t);
    for (; t < a.T; t += step) {
        float v[C];
        const float l = lse, mine = up;
        const int e = pick;
        bool here = on;
        if (here) row.values(a.E, v);
        on = counted(t + step);
        if (on) fetch(t + step);
        if (here && l == 0.f) {   // a row of -inf has lse 0 too
            bool any = false;
#pragma unroll
            for (int c = 0; c < C; ++c) any |= v[c] != -INFINITY;
            here = __any(any);
        }
        if (!here) {
#pragma unroll
            for (int c = 0; c < C; ++c) v[c] = 0.f;
        } else {
            float s = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                v[c] = exp_of(v[c] - l);
                s = fmaf(v[c], g[c], s);
            }
            s = wave_sum(s) - zscale * l;
#pragma unroll
            for (int c = 0; c < C; ++c) v[c] *= g[c] - s;
            if (a.dpicks) {
                const bool in = lane < a.k && (uint32_t)e < (uint32_t)a.E;
                float sum = 0.f;
                bool before = false;
                for (int r = 0; r < a.k; ++r) {
                    const int er = __builtin_amdgcn_readlane(e, r);
                    const float ur = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, mine), r));
                    sum += er == e ? ur : 0.f;
                    before |= er == e && r < lane;
                }
                const bool adds = in && !before;
                if (adds) add[w][e] = sum;
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int i = 0; i < C / V; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) v[i * V + j] += add[w][Row::expert(i) + j];
                __builtin_amdgcn_wave_barrier();
                if (adds) add[w][e] = 0.f;
                __builtin_amdgcn_wave_barrier();
            }
        }
#pragma unroll
        for (int i = 0; i < C / V; ++i) {
            float q[V];
#pragma unroll
            for (int j = 0; j < V; ++j) q[j] = v[i * V + j];
            if (Row::expert(i) < a.E) store_values<V>((Z *)a.dz, t * a.E + Row::expert(i), q);
        }
    }
}

namespace {

strata_status check_balance(int32_t T, int32_t k, int32_t E) {
    if (T < 0 || k < 1 || k > 32 || E < 1 || E > BAL_E) return STRATA_EINVAL;
    return T > MAX_ROWS ? STRATA_EUNSUPPORTED : STRATA_OK;
}

bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

// Blocks of the forward launch: a wave's tokens share the block's way through LDS and memory.
int balance_blocks(int T) {
    if (T <= BAL_ONE) return 1;
    const int b = (T + 2 * BAL_WAVES - 1) / (2 * BAL_WAVES);
    return b < BAL_BLOCKS ? b : BAL_BLOCKS;
}

size_t part_bytes(int64_t n) { return (size_t)((n * 4 + 255) / 256 * 256); }

// C values a lane hold the row, in pieces of V.
template <template <typename, int, int> class F, typename Z, int V, typename A> void by_length(const A &a, hipStream_t s) {
    if constexpr (V <= 4) {
        if (a.E <= 256) return F<Z, V, 4>::run(a, s);
    }
    if (a.E <= 512) return F<Z, V, 8>::run(a, s);
    F<Z, V, 16>::run(a, s);
}

// The widest pieces that divide the row.
template <template <typename, int, int> class F, typename Z, typename A> void by_width(const A &a, hipStream_t s) {
    if constexpr (sizeof(Z) == 2) {
        if (a.E % 8 == 0 && a.E > 256) return by_length<F, Z, 8>(a, s);
    }
    if (a.E % 4 == 0) return by_length<F, Z, 4>(a, s);
    if (a.E % 2 == 0) return by_length<F, Z, 2>(a, s);
    by_length<F, Z, 1>(a, s);
}

template <typename Z, int V, int C> struct Rows {
    static void run(const BalanceArgs &a, hipStream_t s) {
        STRATA_LAUNCH((balance_rows_kernel<Z, V, C>), dim3(a.blocks), dim3(64 * BAL_WAVES), 0, s, a);
    }
};
template <typename Z, int V, int C> struct Back {
    static void run(const BalanceBack &a, hipStream_t s) {
        STRATA_LAUNCH((balance_back_kernel<Z, V, C>), dim3(a.blocks), dim3(256), 0, s, a);
    }
};

}  // namespace

}  // namespace strata

using namespace strata;

extern "C" {

size_t strata_moe_balance_workspace_bytes(int32_t T, int32_t k, int32_t n_experts) {
    if (check_balance(T, k, n_experts) != STRATA_OK) return 0;
    const int b = balance_blocks(T);
    return b == 1 ? 256 : 2 * part_bytes((int64_t)b * n_experts) + 2 * part_bytes(b) + part_bytes(BAL_SLABS) + 256;
}

strata_status strata_moe_balance(const void *z, strata_xdtype zdtype, const int32_t *idx, const uint8_t *keep, int32_t T,
                                 int32_t k, int32_t n_experts, float *losses, int32_t *counts, float *prob, float *lse,
                                 int32_t *tokens, void *ws, size_t ws_bytes, void *stream) {
    if (bad_dtype(zdtype)) return STRATA_EINVAL;
    const strata_status st = check_balance(T, k, n_experts);
    if (st != STRATA_OK) return st;
    if (!losses || !counts || !tokens || !aligned4(losses) || !aligned4(counts) || !aligned4(prob) || !aligned4(tokens))
        return STRATA_EINVAL;
    if (T > 0 && (bad_rows(z) || !idx || !aligned4(idx) || !lse || !aligned4(lse) || bad_rows(ws))) return STRATA_EINVAL;
    if (T > 0 && ws_bytes < strata_moe_balance_workspace_bytes(T, k, n_experts)) return STRATA_EWORKSPACE;
    BalanceArgs a{z, idx, keep, T, k, n_experts, balance_blocks(T), losses, counts, prob, lse, tokens};
    const hipStream_t s = (hipStream_t)stream;
    if (a.blocks > 1) {
        char *p = (char *)ws;
        const auto take = [&](int64_t n) {
            char *q = p;
            p += part_bytes(n);
            return q;
        };
        a.psum = (float *)take((int64_t)a.blocks * a.E);
        a.csum = (int32_t *)take((int64_t)a.blocks * a.E);
        a.zsum = (float *)take(a.blocks);
        a.nsum = (int32_t *)take(a.blocks);
        a.dots = (float *)take(BAL_SLABS);
        a.ticket = (int32_t *)take(1);
    }
    if (zdtype == STRATA_X_BF16) by_width<Rows, uint16_t>(a, s);
    else by_width<Rows, float>(a, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.blocks == 1) return hip_status(e);
    STRATA_LAUNCH(balance_finish_kernel, dim3((a.E + BAL_SLAB - 1) / BAL_SLAB), dim3(1024), 0, s, a);
    return hip_status(hipGetLastError());
}

strata_status strata_moe_balance_backward(const void *z, strata_xdtype zdtype, const int32_t *idx, const uint8_t *keep,
                                          int32_t T, int32_t k, int32_t n_experts, const float *lse,
                                          const int32_t *counts, const int32_t *tokens, const float *dlosses,
                                          const float *dpicks, void *dz, void *stream) {
    if (bad_dtype(zdtype)) return STRATA_EINVAL;
    const strata_status st = check_balance(T, k, n_experts);
    if (st != STRATA_OK || T == 0) return st;
    if (bad_rows(z) || bad_rows(dz) || !lse || !counts || !tokens || !dlosses || !aligned4(lse) || !aligned4(counts) ||
        !aligned4(tokens) || !aligned4(dlosses) || !aligned4(dpicks) || (dpicks && (!idx || !aligned4(idx))))
        return STRATA_EINVAL;
    const int64_t want = ((int64_t)T + 3) / 4;
    BalanceBack a{z, idx, keep, T, k, n_experts, (int)(want < 2048 ? want : 2048), lse, counts, tokens, dlosses, dpicks, dz};
    if (zdtype == STRATA_X_BF16) by_width<Back, uint16_t>(a, (hipStream_t)stream);
    else by_width<Back, float>(a, (hipStream_t)stream);
    return hip_status(hipGetLastError());
}

}  // extern "C"
