// The experts' products over rows sorted by expert, with dense bf16 weights
// (strata_moe_grouped_product and its two gradients).
//
//   product  y[s]  = W_e x[s]            contraction over K
//   dgrad    dx[s] = W_e^T dy[s]         contraction over N
//   wgrad    dW_e  = sum_s dy[s] x[s]^T  contraction over the expert's rows
//
// Each is C[m][n] = sum_c A[m][c] B[n][c] over one expert's rows; what
// differs is whether an operand's c runs along memory or across it.  The
// expert's row count is only known on the device, so a first launch cuts the
// experts' rows into tiles and lists them (product and dgrad; wgrad's tiles
// are those of the weights).
#include "ops.hpp"

namespace strata {

constexpr int GP_E = 1024;         // most experts
constexpr int GP_TM = 64, GP_TN = 64, GP_TC = 32, GP_PAD = 8;

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

// One block: the rows of every expert (cut to 0..rows and made to ascend by
// a running maximum, so tiles never overlap and their number is bounded),
// then the list of tiles.
__global__ __launch_bounds__(1024) void grouped_plan_kernel(GroupArgs a) {
    __shared__ int32_t first[GP_E + 1];   // first tile of each expert
    __shared__ int32_t seg0[GP_E], seg1[GP_E];
    __shared__ int32_t wave[16];
    const int th = threadIdx.x, lane = th & 63, w = th >> 6;
    auto cut = [&](int i) { return min(max(a.offsets[i], 0), a.rows); };
    const int lo = th < a.E ? cut(th) : 0;
    int m = th < a.E ? cut(th + 1) : 0;
    m = max(m, lo);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int q = __shfl_up(m, o, 64);
        if (lane >= o) m = max(m, q);
    }
    if (lane == 63) wave[w] = m;
    __syncthreads();
    for (int q = 0; q < w; ++q) m = max(m, wave[q]);
    seg1[th] = m;
    __syncthreads();
    const int s0 = th == 0 ? lo : max(lo, seg1[th - 1]);
    seg0[th] = s0;
    const int n = th < a.E ? max(seg1[th] - s0, 0) : 0;
    const int tiles = (n + a.tile_rows - 1) / a.tile_rows;
    int s = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int q = __shfl_up(s, o, 64);
        if (lane >= o) s += q;
    }
    __syncthreads();
    if (lane == 63) wave[w] = s;
    __syncthreads();
    int total = 0;
    for (int q = 0; q < 16; ++q) {
        if (q < w) s += wave[q];
        total += wave[q];
    }
    first[th] = s - tiles;
    if (th == 0) {
        first[GP_E] = total;
        *a.n_items = total;
    }
    __syncthreads();
    for (int i = th; i < total; i += 1024) {
        int e = 0;   // the last expert whose first tile is at or before i
#pragma unroll
        for (int b = 512; b >= 1; b >>= 1)
            if (e + b < GP_E && first[e + b] <= i) e += b;
        const int r0 = seg0[e] + (i - first[e]) * a.tile_rows;
        a.items[i] = GroupItem{e, r0, min(a.tile_rows, seg1[e] - r0)};
    }
}

// 8 consecutive elements of row r, column c of a matrix [R][Cn] (zeros
// outside it; Cn % 8 == 0).
__device__ __forceinline__ uint4 load8(const uint16_t *p, int r, int R, int c, int Cn) {
    return r < R && c < Cn ? *(const uint4 *)(p + (int64_t)r * Cn + c) : make_uint4(0, 0, 0, 0);
}

// LDS tile [64][32] of an operand whose contraction runs along memory
// (rows r0.., columns c0..) or across it (rows c0.., columns r0..).
template <int ACROSS>
__device__ __forceinline__ void stage(uint16_t (*t)[GP_TC + GP_PAD], const uint16_t *p, int R, int Cn, int r0, int c0) {
    const int th = threadIdx.x;
    if (!ACROSS) {
        const int r = th >> 2, c = (th & 3) * 8;
        *(uint4 *)&t[r][c] = load8(p, r0 + r, R, c0 + c, Cn);
    } else {
        const int c = th >> 3, r = (th & 7) * 8;
        const uint4 q = load8(p, c0 + c, R, r0 + r, Cn);
        const uint32_t v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) t[r + j][c] = (uint16_t)(v[j >> 1] >> (16 * (j & 1)));
    }
}

// C tile [64][64] of one expert: A [M][Cd] (or [Cd][M] across), B [Nn][Cd]
// (or [Cd][Nn] across).
template <int TA, int TB>
__device__ __forceinline__ void tile_product(const uint16_t *A, const uint16_t *B, int M, int Nn, int Cd, int m0,
                                             int n0, void *C, int64_t c_row0, int c_bf16) {
    __shared__ __attribute__((aligned(16))) uint16_t as[GP_TM][GP_TC + GP_PAD];
    __shared__ __attribute__((aligned(16))) uint16_t bs[GP_TN][GP_TC + GP_PAD];
    const int th = threadIdx.x, lane = th & 63, w = th >> 6;
    const int l = lane & 31, h = lane >> 5, wm = (w >> 1) * 32, wn = (w & 1) * 32;
    f32x16_t acc;
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[v] = 0.f;
    for (int c0 = 0; c0 < Cd; c0 += GP_TC) {
        __syncthreads();
        stage<TA>(as, A, TA ? Cd : M, TA ? M : Cd, m0, c0);
        stage<TB>(bs, B, TB ? Cd : Nn, TB ? Nn : Cd, n0, c0);
        __syncthreads();
#pragma unroll
        for (int q = 0; q < GP_TC; q += 16) {
            const bf16x8_t av = __builtin_bit_cast(bf16x8_t, *(const u32x4_t *)&as[wm + l][q + 8 * h]);
            const bf16x8_t bv = __builtin_bit_cast(bf16x8_t, *(const u32x4_t *)&bs[wn + l][q + 8 * h]);
            acc = mfma(av, bv, acc);
        }
    }
#pragma unroll
    for (int v = 0; v < 16; ++v) {
        const int m = m0 + wm + 8 * (v >> 2) + 4 * h + (v & 3), n = n0 + wn + l;
        if (m < M && n < Nn) {
            const int64_t at = (c_row0 + m) * Nn + n;
            if (c_bf16) ((uint16_t *)C)[at] = f2bf(acc[v]);
            else ((float *)C)[at] = acc[v];
        }
    }
}

// Blocks: column tiles of every listed row tile.
template <int TB> __global__ __launch_bounds__(256) void grouped_rows_kernel(GroupArgs a) {
    const int item = blockIdx.x;
    if (item >= *a.n_items) return;
    const GroupItem it = a.items[item];
    const int Cd = TB ? a.N : a.K, Nn = TB ? a.K : a.N;
    tile_product<0, TB>(a.A + (int64_t)it.row0 * Cd, a.B + (int64_t)it.expert * a.N * a.K, it.n, Nn, Cd, 0,
                        blockIdx.y * GP_TN, a.C, it.row0, a.c_bf16);
}

__global__ __launch_bounds__(256) void grouped_wgrad_kernel(GroupArgs a) {
    const int e = blockIdx.z;
    const int lo = min(max(a.offsets[e], 0), a.rows), hi = min(max(a.offsets[e + 1], 0), a.rows);
    tile_product<1, 1>(a.A + (int64_t)lo * a.N, a.B + (int64_t)lo * a.K, a.N, a.K, max(hi - lo, 0), blockIdx.y * GP_TM,
                       blockIdx.x * GP_TN, a.C, (int64_t)e * a.N, a.c_bf16);
}

namespace {

constexpr size_t GP_HEAD = 256;   // the tile count, then the list

int64_t max_tiles(int64_t rows, int E, int tile_rows) { return rows / tile_rows + (rows < E ? rows : E); }

strata_status check_grouped(int32_t rows, int32_t E, int32_t N, int32_t K) {
    if (rows < 0) return STRATA_EINVAL;
    if (E < 1 || E > GP_E || N < 8 || K < 8 || N > 65536 || K > 65536 || N % 8 || K % 8 || (int64_t)N * K > (1 << 29))
        return STRATA_EUNSUPPORTED;
    return STRATA_OK;
}

strata_status grouped_call(const void *A, const void *B, const int32_t *offsets, int32_t rows, int32_t E, int32_t N,
                           int32_t K, void *C, strata_xdtype dtype, void *ws, size_t ws_bytes, GroupArgs &a) {
    if (bad_dtype(dtype)) return STRATA_EINVAL;
    const strata_status st = check_grouped(rows, E, N, K);
    if (st != STRATA_OK) return st;
    if (bad_rows(A) || bad_rows(B) || bad_rows(C) || bad_rows(ws) || !offsets) return STRATA_EINVAL;
    if (ws_bytes < strata_moe_grouped_workspace_bytes(rows, E, N, K)) return STRATA_EWORKSPACE;
    a.A = (const uint16_t *)A;
    a.B = (const uint16_t *)B;
    a.C = C;
    a.offsets = offsets;
    a.n_items = (int32_t *)ws;
    a.items = (GroupItem *)((char *)ws + GP_HEAD);
    a.rows = rows;
    a.E = E;
    a.N = N;
    a.K = K;
    a.tile_rows = GP_TM;
    a.c_bf16 = dtype == STRATA_X_BF16;
    return STRATA_OK;
}

template <int TB> strata_status grouped_rows(const GroupArgs &a, hipStream_t s) {
    STRATA_LAUNCH(grouped_plan_kernel, dim3(1), dim3(1024), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return hip_status(e);
    const int Nn = TB ? a.K : a.N;
    STRATA_LAUNCH((grouped_rows_kernel<TB>), dim3((unsigned)max_tiles(a.rows, a.E, GP_TM), (Nn + GP_TN - 1) / GP_TN),
                  dim3(256), 0, s, a);
    return hip_status(hipGetLastError());
}

}  // namespace

}  // namespace strata

using namespace strata;

extern "C" {

size_t strata_moe_grouped_workspace_bytes(int32_t rows, int32_t n_experts, int32_t N, int32_t K) {
    if (check_grouped(rows, n_experts, N, K) != STRATA_OK) return 0;
    return GP_HEAD + (size_t)(max_tiles(rows, n_experts, GP_TM) + 1) * sizeof(GroupItem);
}

strata_status strata_moe_grouped_product(const void *x, const void *W, const int32_t *offsets, int32_t rows,
                                         int32_t n_experts, int32_t N, int32_t K, void *y, strata_xdtype ydtype,
                                         void *ws, size_t ws_bytes, void *stream) {
    GroupArgs a{};
    const strata_status st =
        rows == 0 ? check_grouped(rows, n_experts, N, K)
                  : grouped_call(x, W, offsets, rows, n_experts, N, K, y, ydtype, ws, ws_bytes, a);
    if (st != STRATA_OK || rows == 0) return st;
    return grouped_rows<0>(a, (hipStream_t)stream);
}

strata_status strata_moe_grouped_dgrad(const void *dy, const void *W, const int32_t *offsets, int32_t rows,
                                       int32_t n_experts, int32_t N, int32_t K, void *dx, strata_xdtype xdtype,
                                       void *ws, size_t ws_bytes, void *stream) {
    GroupArgs a{};
    const strata_status st =
        rows == 0 ? check_grouped(rows, n_experts, N, K)
                  : grouped_call(dy, W, offsets, rows, n_experts, N, K, dx, xdtype, ws, ws_bytes, a);
    if (st != STRATA_OK || rows == 0) return st;
    return grouped_rows<1>(a, (hipStream_t)stream);
}

strata_status strata_moe_grouped_wgrad(const void *dy, const void *x, const int32_t *offsets, int32_t rows,
                                       int32_t n_experts, int32_t N, int32_t K, void *dW, strata_xdtype wdtype,
                                       void *ws, size_t ws_bytes, void *stream) {
    GroupArgs a{};
    // without rows dy and x may be null: dW stands in for them and is not read
    const bool none = rows == 0;
    const strata_status st = grouped_call(none ? dW : dy, none ? dW : x, offsets, rows, n_experts, N, K, dW, wdtype,
                                          ws, ws_bytes, a);
    if (st != STRATA_OK) return st;
    STRATA_LAUNCH(grouped_wgrad_kernel, dim3((K + GP_TN - 1) / GP_TN, (N + GP_TM - 1) / GP_TM, n_experts), dim3(256),
                  0, (hipStream_t)stream, a);
    return hip_status(hipGetLastError());
}

}  // extern "C"
