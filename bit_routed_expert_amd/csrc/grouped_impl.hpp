// Kernels of the experts' grouped products (grouped.hip) on the tile products
// of tile_impl.hpp.
#pragma once
#include "tile_impl.hpp"

namespace strata {

constexpr int GP_E = 1024;        // most experts
constexpr int GP_RANKED = 64;     // experts up to which the weights' gradient orders them by rows

struct GroupItem {
    int32_t expert, row0, n;
};

struct GroupArgs {
    const uint16_t *A, *B;      // product: x, W; dgrad: dy, W; wgrad: dy, x
    void *C;
    const int32_t *offsets;
    GroupItem *items;           // tiles of up to tile_rows rows of one expert
    int32_t *n_items;
    int rows, E, N, K, tile_rows, c_bf16;
};

// Block -> (tile, column tile): the column tiles of a row tile, and the row
// tiles of an expert, on one XCD (blocks go to the 8 XCDs in turn).
__device__ __forceinline__ bool group_tile(int nct, int n_items, int &item, int &ct) {
    const int64_t total = (int64_t)nct * n_items;
    const int64_t per = (total + 7) >> 3;
    const int64_t q = blockIdx.x >> 3, bb = (blockIdx.x & 7) * per + q;
    if (q >= per || bb >= total) return false;
    item = (int)(bb / nct);
    ct = (int)(bb - (int64_t)item * nct);
    return true;
}

// Row tile `item` of the call, found from the offsets by a block of NT
// threads (each takes 1024 / NT experts), and how many there are in all.
template <int NT> struct FindItem {
    static constexpr int PE = GP_E / NT;
    int n[PE], lo[PE], first, total;
    __device__ __forceinline__ void scan(const GroupArgs &a, int *wsum) {
        const int th = threadIdx.x, lane = th & 63, w = th >> 6;
        int c = 0;
#pragma unroll
        for (int q = 0; q < PE; ++q) {
            const int e = th * PE + q;
            lo[q] = e < a.E ? min(max(a.offsets[e], 0), a.rows) : 0;
            const int hi = e < a.E ? min(max(a.offsets[e + 1], 0), a.rows) : 0;
            n[q] = max(hi - lo[q], 0);
            c += (n[q] + a.tile_rows - 1) / a.tile_rows;
        }
        int s = c;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int q = __shfl_up(s, o, 64);
            if (lane >= o) s += q;
        }
        if (lane == 63) wsum[w] = s;
        __syncthreads();
        total = 0;
#pragma unroll
        for (int q = 0; q < NT / 64; ++q) {
            const int v = wsum[q];
            s += q < w ? v : 0;
            total += v;
        }
        first = s - c;
    }
    __device__ __forceinline__ GroupItem get(const GroupArgs &a, int item, GroupItem *shared) const {
        int f = first;
#pragma unroll
        for (int q = 0; q < PE; ++q) {
            const int tiles = (n[q] + a.tile_rows - 1) / a.tile_rows;
            if (item >= f && item < f + tiles) {
                const int r = (item - f) * a.tile_rows;
                *shared = GroupItem{(int)threadIdx.x * PE + q, lo[q] + r, min(a.tile_rows, n[q] - r)};
            }
            f += tiles;
        }
        __syncthreads();
        return *shared;
    }
};

// BM x BN tiles, WM x WN waves, ST buffers; C rows are an expert's rows
// (product, dgrad).  LIST: the row tiles were listed by an earlier launch.
template <int BM, int BN, int WM, int WN, int ST, int TB, int LIST>
__global__ __launch_bounds__(64 * WM *WN) void grouped_rows_kernel(GroupArgs a) {
    constexpr int NT = 64 * WM * WN, MT = BM / 32 / WM, NT2 = BN / 32 / WN, C = 64;
    typedef Operand<BM, 0, NT, C> OA;
    typedef Operand<BN, TB, NT, C> OB;
    GROUP_BUFFERS(ST, OA, OB)
    const int Cd = TB ? a.N : a.K, Nn = TB ? a.K : a.N;
    int item, ct;
    GroupItem it;
    if (LIST) {
        if (!group_tile((Nn + BN - 1) / BN, *a.n_items, item, ct)) return;
        it = a.items[item];
    } else {
        __shared__ int wsum[NT / 64];
        __shared__ GroupItem found;
        FindItem<NT> f;
        f.scan(a, wsum);
        if (!group_tile((Nn + BN - 1) / BN, f.total, item, ct)) return;
        it = f.get(a, item, &found);
        it.expert = __builtin_amdgcn_readfirstlane(it.expert);
        it.row0 = __builtin_amdgcn_readfirstlane(it.row0);
        it.n = __builtin_amdgcn_readfirstlane(it.n);
    }
    OA A;
    OB B;
    A.init(a.A + (int64_t)it.row0 * Cd, Cd, 0, it.n, Cd);
    B.init(a.B + (int64_t)it.expert * a.N * a.K, TB ? Nn : Cd, ct * BN, Nn, Cd);
    int m0, n0;
    wave_place<WM, WN, MT, NT2>(m0, n0);
    f32x16_t acc[MT][NT2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT2; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    const int steps = (Cd + C - 1) / C;
    if (m0 >= it.n || ct * BN + n0 >= Nn) {   // no rows or no columns for this wave: it only stages
        contract<ST, false, BM, BN, C, MT, NT2, 0, TB>(A, B, a0, b0, a1, b1, a2, b2, a3, b3, steps, m0, n0, acc);
        return;
    }
    contract<ST, true, BM, BN, C, MT, NT2, 0, TB>(A, B, a0, b0, a1, b1, a2, b2, a3, b3, steps, m0, n0, acc);
    store_tile<MT, NT2>((char *)a.C + (int64_t)it.row0 * Nn * (a.c_bf16 ? 2 : 4), a.c_bf16, m0, it.n, ct * BN + n0, Nn,
                        acc);
}

// The expert with the r-th most rows (of equals the lower index), E <= 64: lane e ranks expert e.
__device__ __forceinline__ int expert_by_rows(const GroupArgs &a, int r) {
    const int lane = threadIdx.x & 63;
    const int n = lane < a.E ? (int)((uint32_t)a.offsets[lane + 1] - (uint32_t)a.offsets[lane]) : 0;
    int rank = 0;
    for (int j = 0; j < a.E; ++j) {
        const int o = __builtin_amdgcn_readlane(n, j);
        rank += (o > n || (o == n && j < lane)) ? 1 : 0;
    }
    return __ffsll((unsigned long long)__ballot(lane < a.E && rank == r)) - 1;
}

// C is an expert's [N][K] weights' gradient.  Rows go unevenly to experts, so
// a tile's work does too: with up to 64 experts each one's tiles are cut into
// quarters (which share rows in an XCD's L2), and the quarters go to the XCDs
// by falling row count.  With more experts they even out, and an expert's
// tiles stay on one XCD.  16 unevenly picked experts over 32768 rows, 1536 x
// 2048 (the largest with 6769, 5626 or 6646 rows): 208, 200 and 199 us, in
// order with an expert on one XCD 311, 288 and 330; even experts, 2048 x
// 2048: 259 and 260 us.
template <int BM, int BN, int WM, int WN, int ST, int C>
__global__ __launch_bounds__(64 * WM *WN) void grouped_wgrad_kernel(GroupArgs a) {
    constexpr int NT = 64 * WM * WN, MT = BM / 32 / WM, NT2 = BN / 32 / WN;
    typedef Operand<BM, 1, NT, C> OA;
    typedef Operand<BN, 1, NT, C> OB;
    GROUP_BUFFERS(ST, OA, OB)
    const int nk = (a.K + BN - 1) / BN, per_e = nk * ((a.N + BM - 1) / BM);
    int e, tn, tk;
    if (a.E <= GP_RANKED) {
        // quarter g of the expert of rank r: unit j = 4 r + g, dealt to the XCDs there and back
        const int nn = (a.N + BM - 1) / BM, hn = (nn + 1) / 2, hk = (nk + 1) / 2;
        const int x = blockIdx.x & 7, q = blockIdx.x >> 3, round = q / (hn * hk), t = q % (hn * hk);
        const int j = round * 8 + ((round & 1) ? 7 - x : x), g = j & 3;
        tn = (g >> 1) * hn + t / hk;
        tk = (g & 1) * hk + t % hk;
        if ((j >> 2) >= a.E || tn >= nn || tk >= nk) return;
        e = expert_by_rows(a, j >> 2);
    } else {
        int t;
        if (!group_tile(per_e, a.E, e, t)) return;
        tn = t / nk;
        tk = t % nk;
    }
    e = __builtin_amdgcn_readfirstlane(e);
    const int lo = __builtin_amdgcn_readfirstlane(min(max(a.offsets[e], 0), a.rows));
    const int hi = __builtin_amdgcn_readfirstlane(min(max(a.offsets[e + 1], 0), a.rows));
    const int cd = max(hi - lo, 0), r0 = tn * BM, k0 = tk * BN;
    OA A;
    OB B;
    A.init(a.A + (int64_t)lo * a.N, a.N, r0, a.N, cd);
    B.init(a.B + (int64_t)lo * a.K, a.K, k0, a.K, cd);
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
    if (r0 + m0 >= a.N || k0 + n0 >= a.K) {
        contract<ST, false, BM, BN, C, MT, NT2, 1, 1>(A, B, a0, b0, a1, b1, a2, b2, a3, b3, steps, m0, n0, acc);
        return;
    }
    contract<ST, true, BM, BN, C, MT, NT2, 1, 1>(A, B, a0, b0, a1, b1, a2, b2, a3, b3, steps, m0, n0, acc);
    store_tile<MT, NT2>((char *)a.C + ((int64_t)e * a.N + r0) * a.K * (a.c_bf16 ? 2 : 4), a.c_bf16, m0,
                        min(a.N - r0, BM), k0 + n0, a.K, acc);
}

}  // namespace strata
