// Orthogonalised updates of small matrices: all steps of a matrix in one block.
//
// The shorter side (up to 32 RT) lies along the rows of X.  X stays in the
// registers in fp32, in the layout of the products' sums, so a X is where the
// sum of B X starts from; its fp16 copy, A and B lie in LDS.  X is read both
// along (X X^T) and, by the transposing reads, across (B X): its 16-byte
// chunks are permuted by the row so that 8 rows' equal chunks and 4 rows'
// equal 64-byte pieces lie in different banks.  Where A has fewer subtiles than
// the block has waves, its contraction is dealt to them and their sums meet in
// LDS.
//
// The diagonals of A and B, near which most of their norms lie, stay in fp32:
// A = D + A', A^2 = D^2 + D A' + A' D + A' A', B X = (diagonal) X + B' X.  With
// them rounded to fp16, b A and a X + B X, which nearly cancel, left matrices of
// equal singular values up to 7e-3 off, all in one direction.  16 of 128 x 256
// take 37.1 us in place of 34.5 for it, the other forms no more.
//
// B' meets X's fp16 copy, and so does B's diagonal ahead of the last two steps:
// its fp16 value stays in B', and what that rounding leaves meets X.  What X's
// rounding leaves is a matrix of full rank: B of it lies within what X has, but
// the diagonal of B alone does not and would be multiplied by a at every step (a
// gradient of a quarter of the directions came out 6.5e-3 off for 31 x 257, 3.2e-3
// for 128 x 256; 2.0e-3 so).  The last two steps, behind which one step at most
// does that, take X in fp32, which gradients of all directions gain by (128 x 256
// 1.7e-3, else 1.9e-3).
//
// 5 steps, against 3 launches of tiles a step: 16 matrices of 128 x 256 37 and 87
// us, 18 of 22 x 556 33 and 66, 6 of 73 x 274 53 and 76, 7 of 18 x 1225 58 and
// 81.  Bound by LDS reads and the turns between its four phases a step.  The three
// longer shapes (1 x 7, 2 x 4 and 2 x 3 subtiles a wave) spill 92 to 316 bytes a lane.
#pragma once
#include "orth_impl.hpp"

namespace strata {

// Permutation of the chunks of row r: its low three bits differ over 8 rows, bits 2 and 3 over 4.
__device__ __forceinline__ int small_swz(int r) { return (r & 1) << 2 | (r & 2) | (r >> 2 & 1) | (r & 2) << 2; }

template <int COLS> struct SmallRows {   // LDS rows of COLS fp16 values, a multiple of 32
    static constexpr int MASK = COLS % 128 == 0 ? 15 : COLS % 64 == 0 ? 7 : 3;
    __device__ __forceinline__ static int at(int r, int chunk) { return r * COLS * 2 + 16 * (chunk ^ (small_swz(r) & MASK)); }
    // 8 values of row r from 16 kk + 8 (lane / 32) on
    __device__ __forceinline__ static f16x8_t along(const uint8_t *t, int r, int kk) {
        return __builtin_bit_cast(f16x8_t, *(const u32x4_t *)(t + at(r, 2 * kk + (int)((threadIdx.x & 63) >> 5))));
    }
    // columns n0.. of rows 16 kk..
    __device__ __forceinline__ static f16x8_t across(const uint8_t *t, int n0, int kk) {
        const int i = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
        const int c = 16 * kk + 8 * (g >> 1) + (i >> 2), chunk = (n0 >> 3) + 2 * (g & 1) + ((i >> 1) & 1);
        typedef __attribute__((address_space(3))) s16x4_t lds4;
        const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(t + at(c, chunk) + 8 * (i & 1)));
        const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(t + at(c + 4, chunk) + 8 * (i & 1)));
        return __builtin_bit_cast(f16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    // a subtile's 16 values of this lane, row r, columns n0 + 8 q + 4 (lane / 32) + 0..3
    __device__ __forceinline__ static void put(uint8_t *t, int r, int n0, const f32x16_t &v) {
        const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            *(u32x2_t *)(t + at(r, (n0 >> 3) + q) + 8 * h) =
                u32x2_t{half_pair(v[4 * q], v[4 * q + 1]), half_pair(v[4 * q + 2], v[4 * q + 3])};
    }
};

// RT (1, 2 or 4) rows of subtiles of 32 x 32 hold X, 8 waves of MT x NT of them, WM = RT / MT rows of waves.
template <typename G, int RT, int MT, int NT> __global__ __launch_bounds__(512) void orth_small_kernel(OrthArgs a, int steps) {
    constexpr int WM = RT / MT, WN = 8 / WM, CT = WN * NT;
    constexpr int PA = RT * RT / 8 > 0 ? RT * RT / 8 : 1;   // subtiles of A a wave
    constexpr int KS = RT * RT < 8 ? 8 / (RT * RT) : 1;     // waves that share a subtile's contraction
    typedef SmallRows<CT * 32> XR;
    typedef SmallRows<RT * 32> AR;
    // B lies over the waves' sums of A, or, with none, over A
    constexpr int A_BYTES = RT * RT * 2048, SUMS = KS > 1 ? (8 - RT * RT) * 4096 : 0;
    __shared__ __attribute__((aligned(128))) uint8_t Xs[RT * CT * 2048], As[A_BYTES], more[SUMS ? SUMS : 128];
    static_assert(sizeof(Xs) + sizeof(As) + sizeof(more) + 256 * RT + 128 <= 160 * 1024 && (!SUMS || A_BYTES <= SUMS), "fits the LDS");
    __shared__ double sums[8];
    __shared__ __attribute__((aligned(16))) float dA[32 * RT], dB[32 * RT];   // the diagonals
    uint8_t *const Bs = SUMS ? more : As;
    const int th = threadIdx.x, lane = th & 63, l = lane & 31, h = lane >> 5, w = __builtin_amdgcn_readfirstlane(th >> 6);
    const int m0 = (w / WN) * 32 * MT, n0 = (w % WN) * 32 * NT;
    const bool tall = a.N > a.K;
    const int L = tall ? a.N : a.K;   // the longer side
    const G *g = (const G *)a.G + (int64_t)blockIdx.x * a.N * a.K;
    const bool live = m0 < a.side && n0 < L;   // this wave has values of X
    f32x16_t X[MT][NT];
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int m = m0 + 32 * i + l, c = n0 + 32 * j + 8 * q + 4 * h;
                float v[4] = {0.f, 0.f, 0.f, 0.f};
                if (m < a.side && c < L) {
                    if (!tall && a.K % 4 == 0) {
                        Raw<G, 4> r;
                        load_raw<4>(g, (int64_t)m * a.K + c, r);
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[k] = value<4>(r, k);
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (c + k < L) {
                                Raw<G, 1> r;
                                load_raw<1>(g, tall ? (int64_t)(c + k) * a.K + m : (int64_t)m * a.K + c + k, r);
                                v[k] = value<1>(r, 0);
                            }
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    s = fma((double)v[k], (double)v[k], s);
                    X[i][j][4 * q + k] = v[k];
                }
            }
#pragma unroll
    for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o, 64);
    if (lane == 0) sums[w] = s;
    if (th < 32 * RT) dB[th] = 0.f;   // also of rows without a subtile of A
    __syncthreads();
    s = 0.0;
#pragma unroll
    for (int q = 0; q < 8; ++q) s += sums[q];
    const double r = 1.0 / (sqrt(s) + (double)a.eps) * (double)a.size;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) X[i][j][v] = (float)((double)X[i][j][v] * r);
    const float unsize = 1.f / (a.size * a.size);
    const int kl = (L + 31) / 32, ks = (a.side + 31) / 32;   // 32s of either contraction
    // subtiles of A: row ar, columns ac + p; the kp-th of KS shares of the contraction
    const int kp = RT == 4 ? 0 : RT == 2 ? w >> 2 : w;
    const int ar = RT == 4 ? w >> 1 : RT == 2 ? (w >> 1) & 1 : 0, ac = RT == 4 ? 2 * (w & 1) : RT == 2 ? w & 1 : 0;
    const int on = (l >> 2 & 1) == h ? 4 * (l >> 3) + (l & 3) : -1;   // which of the 16 values lies on a diagonal, if one does
    const auto take = [&](f32x16_t &m) {   // it, left as zero
        float d = 0.f;
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            d = v == on ? m[v] : d;
            m[v] = v == on ? 0.f : m[v];
        }
        return d;
    };
    const bool squares = 32 * ar < a.side && 32 * ac < a.side;
    for (int step = 0; step < steps; ++step) {
        if (step) __syncthreads();   // everyone has read the last X
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) XR::put(Xs, m0 + 32 * i + l, n0 + 32 * j, X[i][j]);
        __syncthreads();
        f32x16_t A[PA];
#pragma unroll
        for (int p = 0; p < PA; ++p)
#pragma unroll
            for (int v = 0; v < 16; ++v) A[p][v] = 0.f;
        if (squares) {
            for (int k0 = kp; k0 < kl; k0 += KS)
#pragma unroll
                for (int kk = 2 * k0, u = 0; u < 2; ++u, ++kk) {
                    const f16x8_t x = XR::along(Xs, 32 * ar + l, kk);
#pragma unroll
                    for (int p = 0; p < PA; ++p) A[p] = mfma(XR::along(Xs, 32 * (ac + p) + l, kk), x, A[p]);
                }
        }
        if constexpr (KS > 1) {   // the shares' sums, in order
            float *const q = (float *)more;   // [wave behind the first shares'][value][lane]
            constexpr int T = RT * RT;
            if (kp) {
#pragma unroll
                for (int v = 0; v < 16; ++v) q[((w - T) * 16 + v) * 64 + lane] = A[0][v];
            }
            __syncthreads();
            if (!kp) {
#pragma unroll
                for (int v = 0; v < 16; ++v)
#pragma unroll
                    for (int k = 1; k < KS; ++k) A[0][v] += q[(((k - 1) * T + w) * 16 + v) * 64 + lane];
            }
        }
        const bool first = KS == 1 || kp == 0;   // of the waves that hold the same subtile
#pragma unroll
        for (int p = 0; p < PA; ++p) {
#pragma unroll
            for (int v = 0; v < 16; ++v) A[p][v] *= unsize;
            if (first) {
                if (ar == ac + p) {
                    const float d = take(A[p]);
                    if (on >= 0) dA[32 * ar + l] = d;
                }
                AR::put(As, 32 * ar + l, 32 * (ac + p), A[p]);
            }
        }
        __syncthreads();
        if (squares && first) {
            f32x16_t S[PA];
#pragma unroll
            for (int p = 0; p < PA; ++p)
#pragma unroll
                for (int v = 0; v < 16; ++v) S[p][v] = 0.f;
            for (int k0 = 0; k0 < ks; ++k0)
#pragma unroll
                for (int kk = 2 * k0, u = 0; u < 2; ++u, ++kk) {
                    const f16x8_t x = AR::along(As, 32 * ar + l, kk);
#pragma unroll
                    for (int p = 0; p < PA; ++p) S[p] = mfma(AR::along(As, 32 * (ac + p) + l, kk), x, S[p]);
                }
            const float di = dA[32 * ar + l];
            const bool late = step + 2 >= steps;
#pragma unroll
            for (int p = 0; p < PA; ++p) {
                float copy = 0.f;   // of the diagonal, what stays in B'
                if (ar == ac + p) {
                    const float d = fmaf(a.c, fmaf(di, di, take(S[p])), a.b * di);
                    copy = late ? 0.f : (float)(_Float16)d;
                    if (on >= 0) dB[32 * ar + l] = d - copy;
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x4_t dj = *(const f32x4_t *)&dA[32 * (ac + p) + 8 * q + 4 * h];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int v = 4 * q + k;
                        A[p][v] = fmaf(a.c, fmaf(di + dj[k], A[p][v], S[p][v]), a.b * A[p][v]);
                    }
                }
                if (ar == ac + p) {
#pragma unroll
                    for (int v = 0; v < 16; ++v) A[p][v] = v == on ? copy : A[p][v];
                }
            }
        }
        if constexpr (!SUMS) __syncthreads();   // B over A
#pragma unroll
        for (int p = 0; p < PA; ++p)
            if (first) AR::put(Bs, 32 * ar + l, 32 * (ac + p), A[p]);
        __syncthreads();
        if (live) {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const float d = a.a + dB[m0 + 32 * i + l];
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int v = 0; v < 16; ++v) X[i][j][v] *= d;
            }
            for (int k0 = 0; k0 < ks; ++k0)
#pragma unroll
                for (int kk = 2 * k0, u = 0; u < 2; ++u, ++kk) {
                    f16x8_t b[MT];
#pragma unroll
                    for (int i = 0; i < MT; ++i) b[i] = AR::along(Bs, m0 + 32 * i + l, kk);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const f16x8_t x = XR::across(Xs, n0 + 32 * j, kk);
#pragma unroll
                        for (int i = 0; i < MT; ++i) X[i][j] = mfma(x, b[i], X[i][j]);
                    }
                }
        }
    }
    const float scale = a.scale / a.size;
    uint16_t *out = a.out + (int64_t)blockIdx.x * a.N * a.K;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int m = m0 + 32 * i + l, c = n0 + 32 * j + 8 * q + 4 * h;
                if (m >= a.side || c >= L) continue;
                float v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = X[i][j][4 * q + k] * scale;
                if (!tall && a.K % 4 == 0) {
                    store_values<4>(out, (int64_t)m * a.K + c, v);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (c + k < L) out[tall ? (int64_t)(c + k) * a.K + m : (int64_t)m * a.K + c + k] = f2bf(v[k]);
                }
            }
}

}  // namespace strata
