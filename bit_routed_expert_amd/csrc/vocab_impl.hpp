// Kernels of the vocabulary loss (vocab.hip).
#pragma once
#include "tile_impl.hpp"

namespace strata {

struct VocabArgs {
    const uint16_t *h, *W;          // the call's rows, the output matrix
    const int32_t *targets;
    const float *lse_in, *dloss, *dlse;
    float *loss, *lse;
    void *dh, *dW;
    int T, V, d, dh_bf16, dw_bf16, add;
    // workspace: the rows with a target, packed
    int32_t *n;                     // how many
    float *unit;                    // gradient: dz is kept as a multiple of it
    int32_t *map, *tc;              // their tokens and targets
    uint16_t *hc;                   // their rows
    float *zt;                      // forward: the target's logit
    float2 *part;                   // forward: [column tile][ldp] maximum and sum of a tile's row
    float *lc, *gc, *dc;            // gradient: lse, dloss + dlse, dloss
    uint16_t *dz;                   // gradient: [T][ldv] dz of a piece, its first bf16; `next` values on its second, then its third
    int64_t next;
    float *acc;                     // gradient: [splits][T][d] sums of dh
    int rows_block, ldp, tiles;     // tokens of a packing block, row length of part, column tiles
    // a piece of the vocabulary: columns v0 .. v0 + pw - 1, ldv a multiple of 8 from pw on
    int v0, pw, ldv, first, splits, span;
};

constexpr float VOCAB_LOG2E = 1.4426950408889634f;
__device__ __forceinline__ float exp_diff(float x, float m) { return __builtin_amdgcn_exp2f((x - m) * VOCAB_LOG2E); }

// This lane's 4 consecutive values of subtile (i, j), group q: row m0 + 32 i + lane % 32, column n0 + 32 j + 8 q + 4 (lane / 32).
template <int MT, int NT2, typename F>
__device__ __forceinline__ void each_quad(int m0, int n0, f32x16_t (&acc)[MT][NT2], F f) {
    const int l = threadIdx.x & 31, h = (threadIdx.x >> 5) & 1;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        __builtin_amdgcn_sched_barrier(0);   // no more than a subtile row's loads ahead: registers
#pragma unroll
        for (int j = 0; j < NT2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                f32x4_t v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                f(m0 + 32 * i + l, n0 + 32 * j + 8 * q + 4 * h, i, v);
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[i][j][4 * q + c] = v[c];
            }
    }
}

// acc * by += what the tile's C holds (rows below M, columns below Nn, Nn a multiple of 4).
template <int MT, int NT2>
__device__ __forceinline__ void add_tile(const void *C, int c_bf16, int m0, int M, int n0, int Nn, f32x16_t (&acc)[MT][NT2], float by = 1.f) {
    const uint32_t esz = c_bf16 ? 2 : 4;
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<void *>(C), 0, __builtin_amdgcn_readfirstlane((int)((uint32_t)M * (uint32_t)Nn * esz)), 0x00020000);
    each_quad<MT, NT2>(m0, n0, acc, [&](int m, int n, int, f32x4_t &v) {
        const uint32_t at = n < Nn ? ((uint32_t)m * (uint32_t)Nn + n) * esz : 0xFFFFFFF0u;
        if (c_bf16) {
            const u32x2_t w = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0));
            v = v * by + f32x4_t{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xFFFF0000u),
                                 __uint_as_float(w[1] << 16), __uint_as_float(w[1] & 0xFFFF0000u)};
        } else {
            v = v * by + __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
        }
    });
}

// Block -> (row tile, column tile) with nr row tiles: each XCD has a range of
// columns, four column tiles at a time, so that the 32 tiles under way on it
// share 8 row tiles and 4 column tiles of operands in its L2.
__device__ __forceinline__ bool vocab_tile(int nr, int nc, int &rt, int &ct) {
    const int64_t total = (int64_t)nr * nc, per = (total + 7) >> 3;
    const int64_t q = blockIdx.x >> 3, bb = (int64_t)(blockIdx.x & 7) * per + q;
    if (q >= per || bb >= total) return false;
    const int g = (int)(bb / (4 * nr)), wide = min(4, nc - 4 * g), at = (int)(bb - (int64_t)4 * nr * g);
    ct = 4 * g + at % wide;
    rt = at / wide;
    return true;
}

// The tokens of a call of up to 32 that have a target, a bit each.
__device__ __forceinline__ uint32_t few_tokens(const VocabArgs &a) {
    const int lane = threadIdx.x & 63;
    return (uint32_t)__ballot(lane < a.T && (uint32_t)a.targets[lane < a.T ? lane : 0] < (uint32_t)a.V);
}

// Place of the r-th set bit.
__device__ __forceinline__ int bit_of(uint32_t m, int r) {
    for (int i = 0; i < r; ++i) m &= m - 1;
    return __ffs((int)m) - 1;
}

// Tiles of the logits z = hc W^T of a piece.  GRAD 0: the maximum and the sum
// of each row's tile, and the targets' logits; else dz in that many bf16.  FEW: a
// call of up to 32 tokens takes its rows from h itself, no launch packs them.
template <int BM, int BN, int WM, int WN, int ST, int GRAD, int FEW = 0>
__global__ __launch_bounds__(64 * WM *WN) void vocab_logits_kernel(VocabArgs a) {
    constexpr int NT = 64 * WM * WN, MT = BM / 32 / WM, NT2 = BN / 32 / WN, C = 64;
    typedef Operand<BM, 0, NT, C> OA;
    typedef Operand<BN, 0, NT, C> OB;
    GROUP_BUFFERS(ST, OA, OB)
    static_assert(!FEW || BM == 32, "one tile of rows");
    const uint32_t there = FEW ? few_tokens(a) : 0;
    const int n = FEW ? __popc(there) : *a.n, nc = (a.pw + BN - 1) / BN;
    int rt, ct;
    if (!vocab_tile((n + BM - 1) / BM, nc, rt, ct)) return;
    rt = __builtin_amdgcn_readfirstlane(rt);
    ct = __builtin_amdgcn_readfirstlane(ct);
    const int row0 = rt * BM, rows = min(n - row0, BM), c0 = ct * BN;
    OA A;
    OB B;
    if constexpr (FEW) {
        A.init(a.h, a.d, 0, a.T, a.d);
#pragma unroll
        for (int i = 0; i < OA::LOADS; ++i) {   // rows from their tokens; behind the last one out of range
            const int r = (i * NT + (int)threadIdx.x) / OA::CH;
            A.off[i] = r < n ? A.off[i] + (uint32_t)(bit_of(there, r) - r) * (uint32_t)a.d * 2u : 0x80000000u;
        }
    } else {
        A.init(a.hc + (int64_t)row0 * a.d, a.d, 0, rows, a.d);
    }
    B.init(a.W + (int64_t)a.v0 * a.d, a.d, c0, a.pw, a.d);
    int m0, n0;
    wave_place<WM, WN, MT, NT2>(m0, n0);
    f32x16_t acc[MT][NT2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT2; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    const int steps = (a.d + C - 1) / C, l = threadIdx.x & 31, h = (threadIdx.x >> 5) & 1;
    const bool active = m0 < rows && c0 + n0 < a.pw;
    if (active) contract<ST, true, BM, BN, C, MT, NT2, 0, 0>(A, B, a0, b0, a1, b1, a2, b2, a3, b3, steps, m0, n0, acc);
    else contract<ST, false, BM, BN, C, MT, NT2, 0, 0>(A, B, a0, b0, a1, b1, a2, b2, a3, b3, steps, m0, n0, acc);
    if constexpr (GRAD == 0) {
        float2 *stat = (float2 *)a0;   // [BM][WN], once all waves have read their last step
        static_assert(BM * WN * 8 <= OA::BYTES, "the statistics fit");
        __syncthreads();
        if (!active) {
            for (int r = threadIdx.x & 63; r < 32 * MT; r += 64) stat[(m0 + r) * WN + n0 / (32 * NT2)] = float2{-INFINITY, 0.f};
        } else {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int row = row0 + m0 + 32 * i + l;
                const int want = (row < n ? FEW ? a.targets[bit_of(there, row)] : a.tc[row] : -1) - a.v0 - c0 - n0 - 4 * h;   // the target's place among the columns
                if (__any((uint32_t)want < 32u * NT2)) {
                    float picked = 0.f;
                    bool mine = false;
#pragma unroll
                    for (int j = 0; j < NT2; ++j)
#pragma unroll
                        for (int v = 0; v < 16; ++v) {
                            const int at = 32 * j + 8 * (v / 4) + (v & 3);
                            picked = at == want ? acc[i][j][v] : picked;
                            mine |= at == want;
                        }
                    if (mine) a.zt[row] = picked;
                }
                if (c0 + n0 + 32 * NT2 > a.pw) {   // columns behind the last one
#pragma unroll
                    for (int j = 0; j < NT2; ++j)
#pragma unroll
                        for (int v = 0; v < 16; ++v)
                            if (c0 + n0 + 4 * h + 32 * j + 8 * (v / 4) + (v & 3) >= a.pw) acc[i][j][v] = -INFINITY;
                }
                float m = -INFINITY, s = 0.f;
#pragma unroll
                for (int j = 0; j < NT2; ++j)
#pragma unroll
                    for (int v = 0; v < 16; ++v) m = fmaxf(m, acc[i][j][v]);
                m = fmaxf(m, lane_xor<32>(m));
                // one fma a value; what the rounding of m log2(e) makes of all of them goes back at the end
                const float base = m == -INFINITY ? 0.f : m * VOCAB_LOG2E;
                const float off = m == -INFINITY ? 0.f : fmaf(m, VOCAB_LOG2E, -base);
#pragma unroll
                for (int j = 0; j < NT2; ++j)
#pragma unroll
                    for (int v = 0; v < 16; ++v) s += __builtin_amdgcn_exp2f(fmaf(acc[i][j][v], VOCAB_LOG2E, -base));
                s *= __builtin_amdgcn_exp2f(-off);
                s += lane_xor<32>(s);
                if (h == 0) stat[(m0 + 32 * i + l) * WN + n0 / (32 * NT2)] = float2{m, s};
            }
        }
        __syncthreads();
        for (int r = threadIdx.x; r < rows; r += NT) {
            float2 p[WN];
            float m = -INFINITY, s = 0.f;
#pragma unroll
            for (int q = 0; q < WN; ++q) {
                p[q] = stat[r * WN + q];
                m = fmaxf(m, p[q].x);
            }
            const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int q = 0; q < WN; ++q) s += p[q].y * exp_diff(p[q].x, base);
            a.part[(int64_t)ct * a.ldp + row0 + r] = float2{m, s};
        }
    } else {
        if (!active) return;
        const float unit = *a.unit;
        float lse[MT], up[MT], un[MT];
        int want[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int row = min(row0 + m0 + 32 * i + l, n - 1);
            lse[i] = a.lc[row];
            up[i] = a.gc[row] / unit;
            un[i] = a.dc[row] / unit;
            want[i] = a.tc[row] - a.v0;
        }
        const bool ragged = c0 + n0 + 32 * NT2 > a.pw;   // columns behind the last one
        uint16_t *dz = a.dz + (int64_t)row0 * a.ldv;
        each_quad<MT, NT2>(m0, c0 + n0, acc, [&](int, int col, int i, f32x4_t &v) {
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = exp_diff(v[c], lse[i]) * up[i];
            if (ragged) {
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = col + c < a.pw ? v[c] : 0.f;
            }
        });
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int place = want[i] - c0 - n0 - 4 * h;
            if (__any((uint32_t)place < 32u * NT2)) {
#pragma unroll
                for (int j = 0; j < NT2; ++j)
#pragma unroll
                    for (int v = 0; v < 16; ++v) acc[i][j][v] -= 32 * j + 8 * (v / 4) + (v & 3) == place ? un[i] : 0.f;
            }
        }
        store_tile<MT, NT2>(dz, 1, m0, rows, c0 + n0, a.ldv, acc);
#pragma unroll
        for (int p = 1; p < GRAD; ++p) {   // what the pieces before leave
            each_quad<MT, NT2>(m0, c0 + n0, acc, [&](int, int, int, f32x4_t &v) {
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] -= bf16_to_float(f2bf(v[c]));
            });
            store_tile<MT, NT2>(dz + p * a.next, 1, m0, rows, c0 + n0, a.ldv, acc);
        }
    }
}

// An operand whose contraction goes over it PIECES times, each time `next` values on.
template <typename O, int C, int PIECES> struct Again : O {
    int64_t next;
    int steps;
    __device__ __forceinline__ void again(int64_t on, int n) {
        next = on;
        steps = n;
    }
    __device__ __forceinline__ void load(int s, uint8_t *dst) const {
        if (PIECES == 1 || s < steps) return O::load(s, dst);
        const int p = PIECES > 2 && s >= 2 * steps ? 2 : 1;
        O o = *this;
        o.base += p * next;
        o.load(s - p * steps, dst);
    }
};

// dW of a piece: rows are its vocabulary, the contraction runs over the tokens.
template <int BM, int BN, int WM, int WN, int ST, int C, int PIECES>
__global__ __launch_bounds__(64 * WM *WN) void vocab_dw_kernel(VocabArgs a) {
    constexpr int NT = 64 * WM * WN, MT = BM / 32 / WM, NT2 = BN / 32 / WN;
    typedef Again<Operand<BM, 1, NT, C>, C, PIECES> OA;
    typedef Again<Operand<BN, 1, NT, C>, C, PIECES> OB;
    GROUP_BUFFERS(ST, OA, OB)
    const int n = *a.n, nk = (a.d + BN - 1) / BN, nr = (a.pw + BM - 1) / BM;
    const int64_t total = (int64_t)nk * nr, per = (total + 7) >> 3;
    const int64_t bb = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= per || bb >= total) return;
    const int r0 = __builtin_amdgcn_readfirstlane((int)(bb / nk)) * BM, k0 = __builtin_amdgcn_readfirstlane((int)(bb % nk)) * BN;
    int m0, n0;
    wave_place<WM, WN, MT, NT2>(m0, n0);
    f32x16_t acc[MT][NT2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT2; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    const int steps = (n + C - 1) / C;
    const bool active = r0 + m0 < a.pw && k0 + n0 < a.d;
    OA A;
    OB B;
    B.init(a.hc, a.d, k0, a.d, n);
    A.init(a.dz, a.ldv, r0, a.pw, n);
    A.again(a.next, steps);
    B.again(0, steps);
    if (active) contract<ST, true, BM, BN, C, MT, NT2, 1, 1>(A, B, a0, b0, a1, b1, a2, b2, a3, b3, PIECES * steps, m0, n0, acc);
    else contract<ST, false, BM, BN, C, MT, NT2, 1, 1>(A, B, a0, b0, a1, b1, a2, b2, a3, b3, PIECES * steps, m0, n0, acc);
    if (!active) return;
    const int M = min(a.pw - r0, BM);
    char *C0 = (char *)a.dW + ((int64_t)a.v0 + r0) * a.d * (a.dw_bf16 ? 2 : 4);
    const float unit = *a.unit;
    if (!a.add) return store_tile<MT, NT2>(C0, a.dw_bf16, m0, M, k0 + n0, a.d, acc, unit);
    add_tile<MT, NT2>(C0, a.dw_bf16, m0, M, k0 + n0, a.d, acc, unit);
    store_tile<MT, NT2>(C0, a.dw_bf16, m0, M, k0 + n0, a.d, acc);
}

// dh of a piece, its columns cut into `splits` spans with sums of their own.
template <int BM, int BN, int WM, int WN, int ST, int PIECES>
__global__ __launch_bounds__(64 * WM *WN) void vocab_dh_kernel(VocabArgs a) {
    constexpr int NT = 64 * WM * WN, MT = BM / 32 / WM, NT2 = BN / 32 / WN, C = 64;
    typedef Again<Operand<BM, 0, NT, C>, C, PIECES> OA;
    typedef Again<Operand<BN, 1, NT, C>, C, PIECES> OB;
    GROUP_BUFFERS(ST, OA, OB)
    const int n = *a.n, nk = (a.d + BN - 1) / BN, nr = (n + BM - 1) / BM;
    const int64_t total = (int64_t)nk * nr * a.splits, per = (total + 7) >> 3;
    const int64_t bb = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= per || bb >= total) return;
    const int sp = __builtin_amdgcn_readfirstlane((int)(bb / ((int64_t)nk * nr)));
    const int at = (int)(bb - (int64_t)sp * nk * nr);
    const int row0 = __builtin_amdgcn_readfirstlane(at / nk) * BM, k0 = __builtin_amdgcn_readfirstlane(at % nk) * BN;
    const int c0 = sp * a.span, rows = min(n - row0, BM);
    int m0, n0;
    wave_place<WM, WN, MT, NT2>(m0, n0);
    f32x16_t acc[MT][NT2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT2; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    const int cda = min(a.span, a.ldv - c0), steps = c0 < a.pw ? (cda + C - 1) / C : 0;   // a last piece may leave spans without columns
    const bool active = m0 < rows && k0 + n0 < a.d;
    OA A;
    OB B;
    A.init(a.dz + (int64_t)row0 * a.ldv + c0, a.ldv, 0, rows, cda);
    B.init(a.W + ((int64_t)a.v0 + c0) * a.d, a.d, k0, a.d, min(a.span, a.pw - c0));
    A.again(a.next, steps);
    B.again(0, steps);
    if (active) contract<ST, true, BM, BN, C, MT, NT2, 0, 1>(A, B, a0, b0, a1, b1, a2, b2, a3, b3, PIECES * steps, m0, n0, acc);
    else contract<ST, false, BM, BN, C, MT, NT2, 0, 1>(A, B, a0, b0, a1, b1, a2, b2, a3, b3, PIECES * steps, m0, n0, acc);
    if (!active) return;
    float *C0 = a.acc + ((int64_t)sp * a.T + row0) * a.d;
    if (!a.first) add_tile<MT, NT2>(C0, 0, m0, rows, k0 + n0, a.d, acc);
    store_tile<MT, NT2>(C0, 0, m0, rows, k0 + n0, a.d, acc);
}

}  // namespace strata
