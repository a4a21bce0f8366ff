// Balance losses of a router with the picks counted per expert, and the
// logits' gradient (strata_moe_balance, strata_moe_balance_backward).
//
// Both read the logits once: 16 to 64 lanes take a token, its row lies in
// their registers, 16 values a lane (so that a wave meets up to four tokens
// and their reductions run side by side).  Forward, a lane adds its experts'
// probabilities over all tokens it meets; the lanes of a block are added in
// LDS, the blocks by a second launch, whose last block sums the losses over
// the experts.  No sum depends on the order in which blocks run.  A call of
// few tokens is one block of one launch.
//
// 32768 rows of 512 fp32: 15 us (4.5 TB/s) and 5 us the second launch; bound by the
// reads and by each row's chain of maximum, sum and probabilities.  The gradient
// of 16384 rows of 512 bf16 14.3 us (2.3 TB/s), half of it the picks, which a
// token's lanes add in the picks' order through LDS.  5 rows: 3.2 us.
#include "ops.hpp"

namespace strata {

constexpr int BAL_E = 1024;          // most experts
constexpr int BAL_WAVES = 8;         // of a block
constexpr int BAL_BLOCKS = 512;      // most blocks of the forward launch
constexpr int BAL_ONE = 64;          // tokens up to which one block does it all
constexpr int BAL_C = 16;            // values of a row a lane holds
constexpr int BAL_SLAB = 16;         // experts of a block of the second launch
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

constexpr float LOG2E = 1.4426950408889634f;

// e^x for x <= 0, off by U |x| and the instruction's 1 ulp.
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * LOG2E); }

// Sum and maximum over the P lanes of a token, in all of them.
template <int P> __device__ __forceinline__ float row_sum(float v) {
    if constexpr (P > 32) v += lane_xor<32>(v);
    if constexpr (P > 16) v += lane_xor<16>(v);
    v += lane_xor<8>(v);
    v += lane_xor<4>(v);
    v += lane_xor<2>(v);
    return v + lane_xor<1>(v);
}
template <int P> __device__ __forceinline__ float row_max(float v) {
    if constexpr (P > 32) v = fmaxf(v, lane_xor<32>(v));
    if constexpr (P > 16) v = fmaxf(v, lane_xor<16>(v));
    v = fmaxf(v, lane_xor<8>(v));
    v = fmaxf(v, lane_xor<4>(v));
    v = fmaxf(v, lane_xor<2>(v));
    return fmaxf(v, lane_xor<1>(v));
}
// Whether any of the P lanes of this lane's token says so.
template <int P> __device__ __forceinline__ bool row_any(bool v) {
    const uint64_t m = __ballot(v);
    return P == 64 ? m != 0 : (m >> (threadIdx.x & (64 - P)) & ((1ull << (P & 63)) - 1)) != 0;
}

// A token's logits over P lanes: value j of piece i is expert (P i + lane) V + j; -inf behind the last one.
template <typename Z, int V, int P> struct LogitRow {
    Raw<Z, V> raw[BAL_C / V];
    __device__ __forceinline__ static int expert(int i) { return (P * i + (int)(threadIdx.x % P)) * V; }
    __device__ __forceinline__ void load(const Z *z, int64_t t, int E) {
#pragma unroll
        for (int i = 0; i < BAL_C / V; ++i)
            if (expert(i) < E) load_raw<V, true>(z, t * E + expert(i), raw[i]);
    }
    __device__ __forceinline__ void values(int E, float (&v)[BAL_C]) const {
#pragma unroll
        for (int i = 0; i < BAL_C / V; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) v[i * V + j] = expert(i) < E ? value<V>(raw[i], j) : -INFINITY;
    }
};

// Lanes of the tokens that do not count go along with zeros, so that the reductions run in whole waves.
template <typename Z, int V, int P> __global__ __launch_bounds__(64 * BAL_WAVES) void balance_rows_kernel(BalanceArgs a) {
    constexpr int C = BAL_C, W = BAL_WAVES, ROWS = 64 / P;   // tokens of a wave at a time
    __shared__ float red[W][P * C];
    __shared__ int hist[BAL_E];
    __shared__ float zred[W];
    __shared__ int nred[W];
    const int th = threadIdx.x, lane = th & 63, w = __builtin_amdgcn_readfirstlane(th >> 6), place = lane % P;
    const int step = a.blocks * W * ROWS;
    const auto counted = [&](int64_t t) { return t < a.T && (!a.keep || a.keep[t]); };
    float acc[C], zz = 0.f;
    int n = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.f;
    LogitRow<Z, V, P> row;
    int pick = -1;
    int64_t t = (int64_t)(blockIdx.x * W + w) * ROWS + lane / P;
    const int64_t first = (int64_t)(blockIdx.x * W + w) * ROWS;   // the wave's first token decides its trips
    const auto fetch = [&](int64_t u) {
        row.load((const Z *)a.z, u, a.E);
        pick = place < a.k ? a.idx[u * a.k + place] : -1;
    };
    if (t < a.T) fetch(t);   // the first ones counted or not; then flags two trips ahead of their rows' use
    bool on = counted(t), soon = counted(t + step);
    for (int e = th; e < a.E; e += 64 * W) hist[e] = 0;
    __syncthreads();
    for (int64_t f = first; f < a.T; f += step, t += step) {
        float v[C];
        const int e = pick;
        bool here = on;
        row.values(a.E, v);
        on = soon;
        if (on) fetch(t + step);
        soon = counted(t + 2 * (int64_t)step);
        float m = v[0];
#pragma unroll
        for (int c = 1; c < C; ++c) m = fmaxf(m, v[c]);
        m = row_max<P>(m);
        if (m == -INFINITY) {   // nothing there, or NaN beside nothing
            bool nan = false;
#pragma unroll
            for (int c = 0; c < C; ++c) nan |= v[c] != v[c];
            here = row_any<P>(nan) && here;
        }
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            v[c] = exp_of(v[c] - m);
            s += v[c];
        }
        s = row_sum<P>(s);
        const float lse = m + logf(s), r = 1.f / s;
        if (here) {
#pragma unroll
            for (int c = 0; c < C; ++c) acc[c] = fmaf(v[c], r, acc[c]);
            if (place == 0) {
                zz = fmaf(lse, lse, zz);
                ++n;
            }
            if ((uint32_t)e < (uint32_t)a.E) atomicAdd(&hist[e], 1);
        }
        if (place == 0 && t < a.T) a.lse[t] = here ? lse : 0.f;
    }
    zz = wave_sum(zz);
    n = wave_sum(n);
#pragma unroll
    for (int c = 0; c < C; ++c) {   // the wave's tokens, side by side
        if constexpr (P <= 16) acc[c] += lane_xor<16>(acc[c]);
        if constexpr (P <= 32) acc[c] += lane_xor<32>(acc[c]);
    }
    if (lane < P) {
#pragma unroll
        for (int i = 0; i < C / V; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) red[w][LogitRow<Z, V, P>::expert(i) + j] = acc[i * V + j];
    }
    if (lane == 0) {
        zred[w] = zz;
        nred[w] = n;
    }
    __syncthreads();
    float z = 0.f;
    n = 0;
#pragma unroll
    for (int q = 0; q < W; ++q) {
        z += zred[q];
        n += nred[q];
    }
    const bool one = a.blocks == 1;
    float dot = 0.f;
    for (int e = th; e < a.E; e += 64 * W) {
        float p = 0.f;
#pragma unroll
        for (int q = 0; q < W; ++q) p += red[q][e];
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
            for (int q = 0; q < W; ++q) d += zred[q];
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

// 16 experts to a block: its 64 groups of 16 lanes share the blocks' sums.  The
// block that takes the last ticket sums the losses, in the order of the slabs.
__global__ __launch_bounds__(1024) void balance_finish_kernel(BalanceArgs a) {
    __shared__ float pw[16][BAL_SLAB];
    __shared__ int cw[16][BAL_SLAB];
    __shared__ float zw[16];
    __shared__ int nw[16];
    const int th = threadIdx.x, lane = th & 63, w = __builtin_amdgcn_readfirstlane(th >> 6);
    const int col = th % BAL_SLAB, e = blockIdx.x * BAL_SLAB + col, ec = min(e, a.E - 1);
    float p = 0.f;
    int c = 0;
#pragma unroll 8
    for (int b = th / BAL_SLAB; b < a.blocks; b += 1024 / BAL_SLAB) {
        p += a.psum[(int64_t)b * a.E + ec];
        c += a.csum[(int64_t)b * a.E + ec];
    }
    float z = th < a.blocks ? a.zsum[th] : 0.f;
    int n = th < a.blocks ? a.nsum[th] : 0;
    p += lane_xor<16>(p);
    p += lane_xor<32>(p);
    c += lane_xor<16>(c);
    c += lane_xor<32>(c);
    z = wave_sum(z);
    n = wave_sum(n);
    if (lane < BAL_SLAB) {
        pw[w][lane] = p;
        cw[w][lane] = c;
    }
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
        p += pw[q][col];
        c += cw[q][col];
    }
    p = n ? p / (float)n : 0.f;
    float dot = 0.f;
    if (e < a.E && lane < BAL_SLAB) {
        a.counts[e] = c;
        if (a.prob) a.prob[e] = p;
        dot = (float)c * p;
    }
    dot = wave_sum(dot);
    int last = 0;
    if (lane == 0) {
        __hip_atomic_store(&a.dots[blockIdx.x], dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        last = __hip_atomic_fetch_add(a.ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
    }
    if (!__builtin_amdgcn_readfirstlane(last)) return;
    dot = lane < (int)gridDim.x ? __hip_atomic_load(&a.dots[lane], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.f;
    static_assert(BAL_SLABS <= 64, "a lane for every slab");
    dot = wave_sum(dot);
    if (lane == 0) {
        a.losses[0] = n ? dot * (float)a.E / ((float)n * (float)a.k) : 0.f;
        a.losses[1] = n ? z / (float)n : 0.f;
        *a.tokens = n;
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
// reach their experts through a row of LDS per token: lane r of the token
// holds pick r (P is k at least), and the lanes add one after the other, so
// that equal picks add up in order.
template <typename Z, int V, int P> __global__ __launch_bounds__(256) void balance_back_kernel(BalanceBack a) {
    constexpr int C = BAL_C, ROWS = 64 / P;
    __shared__ __attribute__((aligned(16))) float add[4][64 * C];
    const int th = threadIdx.x, lane = th & 63, w = __builtin_amdgcn_readfirstlane(th >> 6), place = lane % P;
    typedef LogitRow<Z, V, P> Row;
    float *const mine = &add[w][(lane / P) * P * C];   // this token's row
#pragma unroll
    for (int c = 0; c < C; ++c) add[w][c * 64 + lane] = 0.f;
    // the first tokens' rows ahead of all that waits, counted or not; then flags two trips ahead of their rows' use
    const int step = a.blocks * 4 * ROWS;
    const int64_t f0 = (int64_t)(blockIdx.x * 4 + w) * ROWS;
    int64_t t = f0 + lane / P;
    Row row;
    float lse = 0.f, up = 0.f;
    int pick = -1;
    const auto kept = [&](int64_t u) { return u < a.T && (!a.keep || a.keep[u]); };
    const auto fetch = [&](int64_t u) {
        row.load((const Z *)a.z, u, a.E);
        lse = a.lse[u];
        if (a.dpicks && place < a.k) {
            pick = a.idx[u * a.k + place];
            up = a.dpicks[u * a.k + place];
        }
    };
    if (t < a.T) fetch(t);
    bool on = kept(t), soon = kept(t + step);
    const float n = fmaxf((float)*a.tokens, 1.f);
    const float scale = a.dlosses[0] * (float)a.E / (n * n * (float)a.k), zscale = 2.f * a.dlosses[1] / n;
    int count[C];   // all of them under way at once (a branch around each load made a wait of each: 16.0 against 14.3 us for 16384 tokens)
#pragma unroll
    for (int i = 0; i < C / V; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) count[i * V + j] = a.counts[min(Row::expert(i) + j, a.E - 1)];
    float g[C];
#pragma unroll
    for (int c = 0; c < C; ++c) g[c] = scale * (float)count[c];   // behind the last expert p is 0
    for (int64_t f = f0; f < a.T; f += step, t += step) {
        float v[C];
        const float l = lse, u = up;
        const int e = pick;
        bool here = on;
        row.values(a.E, v);
        on = soon;
        if (on) fetch(t + step);
        soon = kept(t + 2 * (int64_t)step);
        bool any = l != 0.f;   // a row of -inf has lse 0 too
#pragma unroll
        for (int c = 0; c < C; ++c) any |= v[c] != -INFINITY;
        here = row_any<P>(any) && here;
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            v[c] = exp_of(v[c] - l);
            s = fmaf(v[c], g[c], s);
        }
        s = row_sum<P>(s) - zscale * l;
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] = here ? v[c] * (g[c] - s) : 0.f;
        if (a.dpicks) {
            const bool adds = here && place < a.k && (uint32_t)e < (uint32_t)a.E;
            for (int r = 0; r < a.k; ++r)   // a wave's LDS operations run in its order
                if (adds && place == r) __hip_atomic_fetch_add(&mine[e], u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < C / V; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) v[i * V + j] += mine[Row::expert(i) + j];
            __builtin_amdgcn_wave_barrier();
            if (adds) mine[e] = 0.f;
            __builtin_amdgcn_wave_barrier();
        }
        if (t < a.T) {
#pragma unroll
            for (int i = 0; i < C / V; ++i) {
                float q[V];
#pragma unroll
                for (int j = 0; j < V; ++j) q[j] = v[i * V + j];
                if (Row::expert(i) < a.E) store_values<V, true>((Z *)a.dz, t * a.E + Row::expert(i), q);
            }
        }
    }
}

namespace {

strata_status check_balance(int32_t T, int32_t k, int32_t E) {
    if (T < 0 || k < 1 || k > 32 || E < 1 || E > BAL_E) return STRATA_EINVAL;
    return T > MAX_ROWS ? STRATA_EUNSUPPORTED : STRATA_OK;
}

bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

// Lanes of a token: 16 values each hold its row, and a lane each its picks.
int balance_lanes(int E, int k) { return E > 512 ? 64 : E > 256 || k > 16 ? 32 : 16; }

// Blocks of the forward launch: a few trips of its waves share the block's way through LDS and memory.
int balance_blocks(int T, int E, int k) {
    if (T <= BAL_ONE) return 1;
    const int rows = BAL_WAVES * (64 / balance_lanes(E, k)), b = (T + 2 * rows - 1) / (2 * rows);
    return b < BAL_BLOCKS ? b : BAL_BLOCKS;
}

size_t part_bytes(int64_t n) { return (size_t)((n * 4 + 255) / 256 * 256); }

template <template <typename, int, int> class F, typename Z, int V, typename A> void by_length(const A &a, hipStream_t s) {
    switch (balance_lanes(a.E, a.k)) {
        case 16: return F<Z, V, 16>::run(a, s);
        case 32: return F<Z, V, 32>::run(a, s);
        default: F<Z, V, 64>::run(a, s);
    }
}

// The widest pieces that divide the row.
template <template <typename, int, int> class F, typename Z, typename A> void by_width(const A &a, hipStream_t s) {
    if constexpr (sizeof(Z) == 2) {
        if (a.E % 8 == 0) return by_length<F, Z, 8>(a, s);
    }
    if (a.E % 4 == 0) return by_length<F, Z, 4>(a, s);
    if (a.E % 2 == 0) return by_length<F, Z, 2>(a, s);
    by_length<F, Z, 1>(a, s);
}

template <typename Z, int V, int P> struct Rows {
    static void run(const BalanceArgs &a, hipStream_t s) {
        STRATA_LAUNCH((balance_rows_kernel<Z, V, P>), dim3(a.blocks), dim3(64 * BAL_WAVES), 0, s, a);
    }
};
template <typename Z, int V, int P> struct Back {
    static void run(const BalanceBack &a, hipStream_t s) {
        STRATA_LAUNCH((balance_back_kernel<Z, V, P>), dim3(a.blocks), dim3(256), 0, s, a);
    }
};

}  // namespace

}  // namespace strata

using namespace strata;

extern "C" {

size_t strata_moe_balance_workspace_bytes(int32_t T, int32_t k, int32_t n_experts) {
    if (check_balance(T, k, n_experts) != STRATA_OK) return 0;
    const int b = balance_blocks(T, n_experts, k);
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
    BalanceArgs a{z, idx, keep, T, k, n_experts, balance_blocks(T, n_experts, k), losses, counts, prob, lse, tokens};
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
    const int64_t rows = 4 * (64 / balance_lanes(n_experts, k)), want = (T + rows - 1) / rows;
    BalanceBack a{z, idx, keep, T, k, n_experts, (int)(want < 1024 ? want : 1024), lse, counts, tokens, dlosses, dpicks, dz};
    if (zdtype == STRATA_X_BF16) by_width<Back, uint16_t>(a, (hipStream_t)stream);
    else by_width<Back, float>(a, (hipStream_t)stream);
    return hip_status(hipGetLastError());
}

}  // extern "C"
