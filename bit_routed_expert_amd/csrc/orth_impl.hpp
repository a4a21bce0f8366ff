// Kernels of the orthogonalised updates (orth.hip).
#pragma once
#include "tile_impl.hpp"

namespace strata {

// n matrices of N x K; side = min(N, K), the order of A and B.  X is kept
// times `size` (a power of two near sqrt(max(N, K)), so that its values are
// about 1 in size at the end).  hi, its fp16 rounding, lies in rows of ldx
// values, A and B in rows of lds; what lies in a row behind its last column is
// zero.  lo, what the rounding left, is the step kernel's alone and lies in the
// order of its lanes: 4 values to a lane, the wave's lanes side by side.  It is
// kept times 2^11: hi's values of 2^-5 to 2^-7 leave 2^-17 and less, of which
// fp16, subnormal below 2^-14, would hold a few bits (2^-24 is its least step),
// and nothing of values below 2^-13.  What hi leaves is at most 16 (next to
// 65504), so 2^11 of it is in range.
struct OrthArgs {
    const void *G;
    uint16_t *out;              // bf16 [n][N][K]
    double *norms;              // [n][parts] sums of squares
    uint16_t *hi, *next, *lo;   // X = hi + lo, the next X's hi
    uint16_t *A, *B;
    float *dA, *dB;             // [n][lds] what the rounding of A's diagonal left, and what B's lacks for both
    int n, N, K, side, ldx, lds, parts;
    int lo_in, lo_out, last;   // of a step: X's lo counts, X' gets one, X' goes to out
    float size, a, b, c, b_over_c, scale, eps;
};

constexpr float ORTH_LO = 0x1p11f;

__device__ __forceinline__ float half_value(uint32_t w, int high) { return half_to_float((uint16_t)(high ? w >> 16 : w)); }
__device__ __forceinline__ uint32_t half_pair(float a, float b) {
    typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, f16x2_t{(_Float16)a, (_Float16)b});
}

// The same, as bits that every use shares: rounded twice in one place and, fused
// with the product ahead of it, once in another, hi and what is subtracted for
// lo would differ (by 2^-11 at a tie).
__device__ __forceinline__ uint32_t half_pair_kept(float a, float b) {
    uint32_t w = half_pair(a, b);
    asm volatile("" : "+v"(w));
    return w;
}

// What hi (the pair w) leaves of a and b, as lo holds it.
__device__ __forceinline__ uint32_t half_pair_left(float a, float b, uint32_t w) {
    return half_pair((a - half_value(w, 0)) * ORTH_LO, (b - half_value(w, 1)) * ORTH_LO);
}

// Buffer of M rows of ld 16-bit values.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t half_rows(const void *p, int M, int ld) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, __builtin_amdgcn_readfirstlane((int)((uint32_t)M * (uint32_t)ld * 2u)),
                                             0x00020000);
}

// 16 values of a subtile as fp16 pairs to rows of ld: 16-byte stores after the wave's halves have exchanged groups.
__device__ __forceinline__ void store_halves(__amdgpu_buffer_rsrc_t r, int m0, int n0, int ld, int i, int j, const uint32_t (&w)[8]) {
    const int lane = threadIdx.x & 63, m = m0 + 32 * i + (lane & 31);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const auto s0 = __builtin_amdgcn_permlane32_swap(w[4 * q], w[4 * q + 2], false, false);
        const auto s1 = __builtin_amdgcn_permlane32_swap(w[4 * q + 1], w[4 * q + 3], false, false);
        const int n = n0 + 32 * j + 16 * q + 8 * (lane >> 5);
        const uint32_t at = n < ld ? ((uint32_t)m * (uint32_t)ld + n) * 2u : 0xFFFFFFF0u;
        __builtin_amdgcn_raw_buffer_store_b128(u32x4_t{s0[0], s1[0], s0[1], s1[1]}, r, at, 0, 0);
    }
}

// Tile (i, j), j <= i, number t of the lower half of a square of tiles.
__device__ __forceinline__ void lower_tile(int t, int &i, int &j) {
    i = (int)((sqrtf(8.f * (float)t + 1.f) - 1.f) * 0.5f);
    while (i * (i + 1) / 2 > t) --i;
    while ((i + 1) * (i + 2) / 2 <= t) ++i;
    j = t - i * (i + 1) / 2;
}

// Blocks dealt to the 8 XCDs in ranges.
__device__ __forceinline__ bool range_tile(int64_t total, int64_t &t) {
    const int64_t per = (total + 7) >> 3, q = blockIdx.x >> 3;
    t = (int64_t)(blockIdx.x & 7) * per + q;
    return q < per && t < total;
}

// Of a value per row i (TALL: column `lane` of 64 at most) that of a lane's value 4 q + k of subtile (i, j).
template <int TALL, int MT> __device__ __forceinline__ float diagonal(const float (&d)[MT], int i, int j, int q, int k) {
    if constexpr (!TALL) {
        return d[i];
    } else {
        const int bits = __builtin_bit_cast(int, d[0]), c = 32 * j + 8 * q + k;
        const int x = __builtin_amdgcn_readlane(bits, c), y = __builtin_amdgcn_readlane(bits, c + 4);
        return __builtin_bit_cast(float, (threadIdx.x >> 5) & 1 ? y : x);
    }
}

// a X, or (a + d) X with a d for each row (TALL: column), added to a tile's sums
// while the rows (TALL: columns) of the tile pass through LDS as an operand: a
// wave's subtiles that lie in step s.
template <int BN, int MT, int NT2, int TALL> struct AddX {
    f32x16_t (&acc)[MT][NT2];
    float a;
    const float (&d)[MT];   // of row 32 i + lane % 32; TALL: of column `lane`, in d[0]
    int from, m0, n0;   // the wave's first row (TALL: column) in the matrix; its place in the tile
    __device__ __forceinline__ void operator()(int s, const uint8_t *ta, const uint8_t *tb) const {
        constexpr int L = 32 * (TALL ? NT2 : MT);
        if (64 * s + 64 <= from || 64 * s >= from + L) return;
        const int l = threadIdx.x & 31, h = (threadIdx.x >> 5) & 1;
#pragma unroll
        for (int u = 0; u < (TALL ? NT2 : MT); ++u) {
            const int at = from + 32 * u - 64 * s;   // the subtile in the step
            if (at < 0 || at >= 64) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float f[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) f[k] = a + diagonal<TALL>(d, u, u, q, k);
#pragma unroll
                for (int v = 0; v < (TALL ? MT : NT2); ++v) {
                    const int i = TALL ? v : u, j = TALL ? u : v;
                    u32x2_t w;
                    if (TALL) {
                        const int r = m0 + 32 * i + l;
                        w = *(const u32x2_t *)(ta + r * 128 + 16 * (((at >> 3) + q) ^ along_swz(r)) + 8 * h);
                    } else {
                        const int c = at + l, chunk = ((n0 + 32 * j) >> 3) + q;
                        w = *(const u32x2_t *)(tb + c * (BN * 2) + 16 * (chunk ^ across_swz<BN>(c)) + 8 * h);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        acc[i][j][4 * q + k] = fmaf(f[k], half_value(w[k / 2], k & 1), acc[i][j][4 * q + k]);
                }
            }
        }
    }
};

// SQUARE 0: A = X X^T (ACROSS 1: X^T X), else B = b A + c A A: symmetric, so
// only the tiles of the lower half are computed.  Those off the diagonal are
// stored a second time, transposed: a wave turns its part in LDS, where 16-byte
// stores would otherwise be 2-byte ones.  b A is met as an operand passes
// through LDS (b/c A is, ahead of the factor c).  The diagonals, near which most
// of the norms lie, are known in fp32: what their rounding to fp16 left of B's
// (of A's, times b + 2 c A) meets X with a, without which matrices of equal
// singular values came out up to 7e-3 off, all in one direction.
template <int BM, int WM, int WN, int ST, int C, int SQUARE, int ACROSS>
__global__ __launch_bounds__(64 * WM *WN) void orth_square_kernel(OrthArgs a) {
    constexpr int NT = 64 * WM * WN, MT = BM / 32 / WM, NT2 = BM / 32 / WN;
    typedef Operand<BM, ACROSS, NT, C> OA;
    typedef Operand<BM, ACROSS, NT, C> OB;
    GROUP_BUFFERS(ST, OA, OB)
    const int nt = (a.side + BM - 1) / BM, tri = nt * (nt + 1) / 2;
    int64_t t;
    if (!range_tile((int64_t)a.n * tri, t)) return;
    const int e = __builtin_amdgcn_readfirstlane((int)(t / tri));
    int ti, tj;
    lower_tile(__builtin_amdgcn_readfirstlane((int)(t - (int64_t)e * tri)), ti, tj);
    ti = __builtin_amdgcn_readfirstlane(ti);
    tj = __builtin_amdgcn_readfirstlane(tj);
    const int64_t squares = (int64_t)a.side * a.lds;
    const uint16_t *A0 = a.A + e * squares;
    const uint16_t *X = SQUARE ? A0 : a.hi + (int64_t)e * a.N * a.ldx;
    const int ld = SQUARE ? a.lds : a.ldx, cd = ACROSS ? a.N : ld;
    const int r0 = ti * BM, k0 = tj * BM, M = min(a.side - r0, BM);
    OA A;
    OB B;
    A.init(X, ld, r0, a.side, cd);
    B.init(X, ld, k0, a.side, cd);
    int m0, n0;
    wave_place<WM, WN, MT, NT2>(m0, n0);
    f32x16_t acc[MT][NT2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT2; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    const int steps = (cd + C - 1) / C;
    const bool active = m0 < M && k0 + n0 < a.lds;
    if (!active) {
        contract<ST, false, BM, BM, C, MT, NT2, ACROSS, ACROSS, f16x8_t>(A, B, a0, b0, a1, b1, a2, b2, a3, b3, steps, m0, n0, acc);
    } else if constexpr (SQUARE) {
        const float none[MT] = {};
        const AddX<BM, MT, NT2, 1> hook{acc, a.b_over_c, none, k0 + n0, m0, n0};
        contract<ST, true, BM, BM, C, MT, NT2, 0, 0, f16x8_t>(A, B, a0, b0, a1, b1, a2, b2, a3, b3, steps, m0, n0, acc, hook);
    } else {
        contract<ST, true, BM, BM, C, MT, NT2, ACROSS, ACROSS, f16x8_t>(A, B, a0, b0, a1, b1, a2, b2, a3, b3, steps, m0, n0, acc);
    }
    uint16_t *to = (SQUARE ? a.B : a.A) + e * squares;
    const float r = SQUARE ? a.c : 1.f / (a.size * a.size);
    const int lane = threadIdx.x & 63, l = lane & 31, h = lane >> 5, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint32_t w[MT][NT2][8];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT2; ++j)
#pragma unroll
            for (int q = 0; q < 8; ++q) w[i][j][q] = half_pair_kept(acc[i][j][2 * q] * r, acc[i][j][2 * q + 1] * r);
    if (ti == tj && active) {   // this wave's values of the diagonal, and what their rounding left
        const int on = (l >> 2 & 1) == h ? 4 * (l >> 3) + (l & 3) : -1;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT2; ++j) {
                const int row = r0 + m0 + 32 * i + l;
                if (m0 + 32 * i != n0 + 32 * j) continue;
                float v = 0.f, x = 0.f;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    v = k == on ? acc[i][j][k] * r : v;
                    x = k == on ? half_value(w[i][j][k / 2], k & 1) : x;
                }
                if (on < 0 || row >= a.lds) continue;
                const int64_t at = (int64_t)e * a.lds + row;
                if (!SQUARE) a.dA[at] = v - x;
                else if (row >= a.side) a.dB[at] = 0.f;
                else a.dB[at] = fmaf(fmaf(2.f * a.c, half_to_float(A0[(int64_t)row * a.lds + row]), a.b), a.dA[at], v - x);
            }
    }
    if (ti != tj) {
        // the wave's part [32 NT2 columns][32 MT rows], rows 16 bytes apart from a multiple of the banks
        constexpr int LD = 32 * MT + 8, PER = ST == 2 ? 2 : 1, PART = OA::BYTES / PER;
        static_assert(32 * NT2 * LD * 2 <= PART && WM * WN <= 2 * ST * PER, "a place for every wave");
        __syncthreads();   // every wave has read its last step
        const int u = wv / PER;
        uint8_t *const p = (u == 0 ? a0 : u == 1 ? b0 : u == 2 ? a1 : u == 3 ? b1 : u == 4 ? a2 : u == 5 ? b2 : u == 6 ? a3 : b3) + wv % PER * PART;
        if (active) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT2; ++j)
#pragma unroll
                    for (int v = 0; v < 16; ++v) {
                        const int n = 32 * j + 8 * (v / 4) + 4 * h + (v & 3);
                        const uint32_t x = w[i][j][v / 2];
                        *(uint16_t *)(p + (n * LD + 32 * i + l) * 2) = (uint16_t)(v & 1 ? x >> 16 : x);
                    }
            const auto cols = half_rows(to + (int64_t)k0 * a.lds, min(a.side - k0, BM), a.lds);
            constexpr int CH = 4 * MT;   // 16-byte pieces of a row
#pragma unroll
            for (int q = 0; q < 32 * NT2 * CH / 64; ++q) {
                const int n = (64 * q + lane) / CH, c = (64 * q + lane) % CH, m = r0 + m0 + 8 * c;
                const u32x4_t x = *(const u32x4_t *)(p + (n * LD + 8 * c) * 2);
                const uint32_t at = m < a.lds ? ((uint32_t)(n0 + n) * (uint32_t)a.lds + m) * 2u : 0xFFFFFFF0u;
                __builtin_amdgcn_raw_buffer_store_b128(x, cols, at, 0, 0);
            }
        }
    }
    if (!active) return;
    const auto rows = half_rows(to + (int64_t)r0 * a.lds, M, a.lds);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT2; ++j) store_halves(rows, m0, k0 + n0, a.lds, i, j, w[i][j]);
}

// X' = a X + B X (TALL: a X + X B, B symmetric), the last one to out.
template <int BM, int BN, int WM, int WN, int ST, int TALL>
__global__ __launch_bounds__(64 * WM *WN) void orth_step_kernel(OrthArgs a) {
    constexpr int NT = 64 * WM * WN, MT = BM / 32 / WM, NT2 = BN / 32 / WN, C = 64;
    typedef Operand<BM, 0, NT, C> OA;
    typedef Operand<BN, !TALL, NT, C> OB;
    GROUP_BUFFERS(ST, OA, OB)
    const int nr = (a.N + BM - 1) / BM, nk = (a.K + BN - 1) / BN;
    int64_t t;
    if (!range_tile((int64_t)a.n * nr * nk, t)) return;
    const int e = __builtin_amdgcn_readfirstlane((int)(t / (nr * nk))), at = (int)(t - (int64_t)e * nr * nk);
    const int r0 = __builtin_amdgcn_readfirstlane(at / nk) * BM, k0 = __builtin_amdgcn_readfirstlane(at % nk) * BN;
    const int M = min(a.N - r0, BM);
    const int64_t xs = (int64_t)a.N * a.ldx;
    const uint16_t *X = a.hi + e * xs, *S = a.B + (int64_t)e * a.side * a.lds;
    OA A;
    OB B;
    if (TALL) {
        A.init(X, a.ldx, r0, a.N, a.ldx);
        B.init(S, a.lds, k0, a.side, a.lds);
    } else {
        A.init(S, a.lds, r0, a.side, a.lds);
        B.init(X, a.ldx, k0, a.ldx, a.N);
    }
    int m0, n0;
    wave_place<WM, WN, MT, NT2>(m0, n0);
    f32x16_t acc[MT][NT2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT2; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    const int steps = (a.lds + C - 1) / C;
    const int lane = threadIdx.x & 63, l = lane & 31, h = lane >> 5;
    float d[MT];
    {
        static_assert(NT2 <= 2, "a lane for each column");
        const float *dB = a.dB + (int64_t)e * a.lds;
#pragma unroll
        for (int i = 0; i < MT; ++i) d[i] = TALL && i ? 0.f : dB[min(TALL ? k0 + n0 + lane : r0 + m0 + 32 * i + l, a.lds - 1)];
    }
    if (m0 >= M || k0 + n0 >= a.ldx) {
        contract<ST, false, BM, BN, C, MT, NT2, 0, !TALL, f16x8_t>(A, B, a0, b0, a1, b1, a2, b2, a3, b3, steps, m0, n0, acc);
        return;
    }
    const AddX<BN, MT, NT2, TALL> hook{acc, a.a, d, TALL ? k0 + n0 : r0 + m0, m0, n0};
    contract<ST, true, BM, BN, C, MT, NT2, 0, !TALL, f16x8_t>(A, B, a0, b0, a1, b1, a2, b2, a3, b3, steps, m0, n0, acc, hook);
    u32x2_t *const lo = (u32x2_t *)a.lo + (t * (WM * WN) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * (MT * NT2 * 4 * 64) + lane;
    if (a.lo_in) {
        const float by = a.a * (1.f / ORTH_LO);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < NT2; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const u32x2_t w = lo[((i * NT2 + j) * 4 + q) * 64];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        acc[i][j][4 * q + k] = fmaf(by, half_value(w[k / 2], k & 1), acc[i][j][4 * q + k]);
                }
        }
    }
    if (a.last) {
        const float r = a.scale / a.size;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT2; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][j][v] *= r;
        uint16_t *to = a.out + ((int64_t)e * a.N + r0) * a.K;
        if (a.K % 8 == 0) return store_tile<MT, NT2>(to, 1, m0, M, k0 + n0, a.K, acc);
#pragma unroll
        for (int i = 0; i < MT; ++i)   // rows that 16 bytes do not divide
#pragma unroll
            for (int j = 0; j < NT2; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    const int m = m0 + 32 * i + l, n = k0 + n0 + 32 * j + 8 * (v / 4) + 4 * h + (v & 3);
                    if (m < M && n < a.K) to[(int64_t)m * a.K + n] = f2bf(acc[i][j][v]);
                }
        return;
    }
    const auto next = half_rows(a.next + e * xs + (int64_t)r0 * a.ldx, M, a.ldx);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT2; ++j) {
            uint32_t w[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) w[q] = half_pair_kept(acc[i][j][2 * q], acc[i][j][2 * q + 1]);
            if (a.lo_out) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    u32x2_t x;
#pragma unroll
                    for (int p = 0; p < 2; ++p)
                        x[p] = half_pair_left(acc[i][j][4 * q + 2 * p], acc[i][j][4 * q + 2 * p + 1], w[2 * q + p]);
                    lo[((i * NT2 + j) * 4 + q) * 64] = x;
                }
            }
            store_halves(next, m0, k0 + n0, a.ldx, i, j, w);
        }
}

}  // namespace strata
