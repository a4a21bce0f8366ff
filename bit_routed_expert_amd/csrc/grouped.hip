// The experts' products over rows sorted by expert, with dense bf16 weights
// (strata_moe_grouped_product and its two gradients).
//
//   product  y[s]  = W_e x[s]            contraction over K
//   dgrad    dx[s] = W_e^T dy[s]         contraction over N
//   wgrad    dW_e  = sum_s dy[s] x[s]^T  contraction over the expert's rows
//
// Each is C[m][n] = sum_c A[m][c] B[n][c] over one expert's rows; what
// differs is whether an operand's c runs along memory or across it.  The
// expert's row count is only known on the device: in product and dgrad a
// first launch cuts the experts' rows into tiles and lists them, or, in a
// small grid, each block finds its own; wgrad's tiles are those of the
// weights.
#include "grouped_impl.hpp"

namespace strata {

// One block: the rows of every expert (cut to 0..rows and made to ascend by
// a running maximum, so tiles never overlap and their number is bounded),
// then the list of tiles.
__global__ __launch_bounds__(1024) void grouped_plan_kernel(GroupArgs a) {
    __shared__ int32_t first[GP_E];   // first tile of each expert
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
    if (th == 0) *a.n_items = total;
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

// ------------------------------------------------------------- few rows
// The product where most experts have no row and the others one or two (a
// decode or verify step): bound by the picked experts' weights, each read
// once from HBM.  A unit is a group of up to R rows of one expert that starts
// at its segment's row 0, R, 2R, ...; a block takes GV_N of its output
// columns, 16 to a wave.  The rows lie in LDS; a wave streams its 16 weight
// rows in whole (64 lanes x 16 bytes) from memory, two of them in flight, and
// sums each over its lanes.  No launch lists the units: a block finds the
// expert of "its" row by counting the segment ends at or before it.
constexpr int GV_R = 4, GV_N = 64, GV_MAX_K = 8192;
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float dot8(const u32x4_t &w, const u32x4_t &x, float c) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        c = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, (uint32_t)w[j]),
                                            __builtin_bit_cast(bf16x2_t, (uint32_t)x[j]), c, false);
    return c;
}

template <int R>
__device__ __forceinline__ void few_rows(const GroupArgs &a, const uint16_t *W, int row0, int n0, const uint8_t *xs) {
    const int lane = threadIdx.x & 63;
    const int K = a.K, steps = (K + 511) >> 9;
    const int wn = n0 + (threadIdx.x >> 6) * 16;
    float out[R];
#pragma unroll
    for (int r = 0; r < R; ++r) out[r] = 0.f;
    const int cols = min(16, a.N - wn);
    for (int j = 0; j < cols; j += 2) {   // N % 8 == 0: whole pairs
        const uint16_t *w0 = W + (int64_t)(wn + j) * K, *w1 = w0 + K;
        float c0[R], c1[R];
#pragma unroll
        for (int r = 0; r < R; ++r) c0[r] = c1[r] = 0.f;
#pragma unroll 4
        for (int s = 0; s < steps; ++s) {
            const int k = 512 * s + 8 * lane;
            if (k < K) {
                const u32x4_t v0 = *(const u32x4_t *)(w0 + k), v1 = *(const u32x4_t *)(w1 + k);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const u32x4_t x = *(const u32x4_t *)(xs + (int64_t)(r * K + k) * 2);
                    c0[r] = dot8(v0, x, c0[r]);
                    c1[r] = dot8(v1, x, c1[r]);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float s0 = wave_sum_dpp(c0[r]), s1 = wave_sum_dpp(c1[r]);
            const float t0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, s0), 63));
            const float t1 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, s1), 63));
            out[r] = lane == j ? t0 : lane == j + 1 ? t1 : out[r];
        }
    }
    if (lane < cols) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t at = (int64_t)(row0 + r) * a.N + wn + lane;
            if (a.c_bf16) ((uint16_t *)a.C)[at] = f2bf(out[r]);
            else ((float *)a.C)[at] = out[r];
        }
    }
}

__global__ __launch_bounds__(256) void grouped_few_kernel(GroupArgs a, int slabs) {
    extern __shared__ __attribute__((aligned(16))) uint8_t xs[];
    __shared__ int found[4];
    const int row = blockIdx.x / slabs, n0 = (blockIdx.x - row * slabs) * GV_N;
    const int th = threadIdx.x;
    // expert of the row: segment ends at or before it
    int c = 0;
    for (int e0 = 0; e0 < a.E; e0 += 256) {
        const bool done = e0 + th < a.E && a.offsets[e0 + th + 1] <= row;
        c += __popcll(__ballot(done));
    }
    if ((th & 63) == 0) found[th >> 6] = c;
    __syncthreads();
    const int e = found[0] + found[1] + found[2] + found[3];
    if (e >= a.E) return;   // behind the last expert
    const int lo = max(a.offsets[e], 0), hi = min(a.offsets[e + 1], a.rows);
    if (row < lo || row >= hi || ((row - lo) & (GV_R - 1))) return;   // its group's first row has it
    const int n = min(hi - row, GV_R);
    const int K = a.K;
    for (int i = th; i < n * K / 8; i += 256)
        *(u32x4_t *)(xs + 16 * i) = *(const u32x4_t *)(a.A + (int64_t)row * K + 8 * i);
    __syncthreads();
    const uint16_t *W = a.B + (int64_t)e * a.N * K;
    switch (n) {
        case 1: few_rows<1>(a, W, row, n0, xs); break;
        case 2: few_rows<2>(a, W, row, n0, xs); break;
        case 3: few_rows<3>(a, W, row, n0, xs); break;
        default: few_rows<4>(a, W, row, n0, xs); break;
    }
}

namespace {

constexpr size_t GP_HEAD = 256;     // the tile count, then the list
constexpr int GP_MIN_ROWS = 32;     // smallest row tile

// Rows against experts up to which the product goes without the matrix cores.
// Of 512 experts, 1536 x 2048, picked evenly: 50 rows 50 us (6.0 TB/s of the
// picked weights), the tiles 54; 128 rows 127 and 130.  Only the device knows how
// the rows fall: 128 rows that all pick one expert are 32 units that each stream
// its matrix, 35 us where the tiles take 14; 64 rows 16 and 14.
bool few_rows_path(int64_t rows, int E, int K) { return rows * 4 <= E && K <= GV_MAX_K; }

int64_t max_tiles(int64_t rows, int E, int tile_rows) { return rows / tile_rows + (rows < E ? rows : E); }

strata_status check_grouped(int32_t rows, int32_t E, int32_t N, int32_t K) {
    if (rows < 0) return STRATA_EINVAL;
    if (E < 1 || E > GP_E || N < 8 || K < 8 || N > 65536 || K > 65536 || N % 8 || K % 8 || (int64_t)N * K > (1 << 29))
        return STRATA_EUNSUPPORTED;
    // grids of fewer than 2^32 threads
    if (rows > (1 << 22) || (int64_t)E * N * K > ((int64_t)1 << 37)) return STRATA_EUNSUPPORTED;
    return STRATA_OK;
}

// A call without rows: nothing to do, whatever the pointers are.
strata_status check_no_rows(int32_t E, int32_t N, int32_t K, strata_xdtype dtype) {
    return bad_dtype(dtype) ? STRATA_EINVAL : check_grouped(0, E, N, K);
}

strata_status grouped_call(const void *A, const void *B, const int32_t *offsets, int32_t rows, int32_t E, int32_t N,
                           int32_t K, void *C, int64_t c_values, strata_xdtype dtype, void *ws, size_t ws_bytes,
                           GroupArgs &a) {
    if (bad_dtype(dtype)) return STRATA_EINVAL;
    const strata_status st = check_grouped(rows, E, N, K);
    if (st != STRATA_OK) return st;
    if (bad_rows(A) || bad_rows(B) || bad_rows(C) || bad_rows(ws) || !offsets) return STRATA_EINVAL;
    const size_t need = strata_moe_grouped_workspace_bytes(rows, E, N, K);
    if (ws_bytes < need) return STRATA_EWORKSPACE;
    // Blocks take their rows from the list in the workspace while others already store.
    if (overlap(C, (size_t)c_values * (dtype == STRATA_X_BF16 ? 2 : 4), ws, need)) return STRATA_EINVAL;
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
    a.c_bf16 = dtype == STRATA_X_BF16;
    return STRATA_OK;
}

// Blocks of a grid up to which each finds its own row tile; above, a launch
// before lists them.  The list costs a small grid 2 to 3 us, the search every
// round of blocks about 1, and 32-row tiles their second block on a CU (28 bytes
// of LDS too many).  Found and listed, 32 rows: 384 blocks 8.5 and 10.1 us, 600
// 14.3 and 14.5, 900 20.5 and 18.6, 1640 29 and 22; 128 rows: 348 blocks 10.6 and
// 13.6, 696 21.7 and 23.6, 1024 40.5 and 41.4, 4992 648 and 650; 256 rows: 288
// blocks 35 and 37, 864 219 and 219.
constexpr int64_t GP_FIND_BLOCKS = 512;

template <int BM, int BN, int WM, int WN, int ST, int TB> strata_status launch_rows(GroupArgs &a, hipStream_t s) {
    const int Nn = TB ? a.K : a.N;
    a.tile_rows = BM;
    const int64_t blocks = (max_tiles(a.rows, a.E, BM) * ((Nn + BN - 1) / BN) + 7) / 8 * 8;
    if constexpr (BM != 64) {   // 64-row tiles are for small grids
        if (blocks > GP_FIND_BLOCKS) {
            STRATA_LAUNCH(grouped_plan_kernel, dim3(1), dim3(1024), 0, s, a);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return hip_status(e);
            STRATA_LAUNCH((grouped_rows_kernel<BM, BN, WM, WN, ST, TB, 1>), dim3((unsigned)blocks), dim3(64 * WM * WN), 0, s, a);
            return hip_status(hipGetLastError());
        }
    }
    STRATA_LAUNCH((grouped_rows_kernel<BM, BN, WM, WN, ST, TB, 0>), dim3((unsigned)blocks), dim3(64 * WM * WN), 0, s, a);
    return hip_status(hipGetLastError());
}

// Tile by the rows an expert has on average, and by how many tiles there are
// (1536 x 2048 unless said).  Up to 16 rows, 32-row tiles: the weights bound it
// and more, smaller blocks keep more of them in flight (E = 16, 16 rows each:
// 18 us against 19 us for 128-row tiles; E = 512, 2 rows: 521 against 537);
// the same where 64 x 128 tiles would be fewer than 128 (4 experts of 64 rows:
// 12 against 18 us; 8 of 64 rows, 512 x 512: 5.7 against 6.5 with 64 rows).
// 64 x 128 where those are no more than the CUs, uneven experts counted with
// half a tile each (7 experts, 4011 rows, 264 x 624: 7.8 us against 11 with
// 32 and 128 rows; 16 of 64 rows, 1024 x 1024: 9.6 against 10 and 12; where
// they are twice the CUs, 8 of 1024 rows, 512 x 512: 16 against 12 with 128).
// Then 128 x 256 with three buffers (E = 512, 64 rows: 620 us, 5.6 TB/s,
// against 734 with 32 rows and 676 with 256).  From 384 rows on, and with
// tiles enough for the 256 CUs, 256 x 256, whose operands are read half as
// often (E = 16, 4096 rows: 362 against 398 us, 512 rows: 56 against 65; with
// 256 rows 46 against 30 us).
template <int TB> strata_status grouped_rows(GroupArgs &a, hipStream_t s) {
    const int64_t rows = a.rows, E = a.E;
    const int Nn = TB ? a.K : a.N;
    const int64_t tiles64 = (rows / 64 + (E + 1) / 2) * ((Nn + 127) / 128);
    if (rows <= 16 * E || tiles64 < 128) return launch_rows<GP_MIN_ROWS, 128, 1, 4, 4, TB>(a, s);
    if (tiles64 <= 256) return launch_rows<64, 128, 2, 2, 4, TB>(a, s);
    if (rows < 384 * E || rows / 256 * ((Nn + 255) / 256) < 192) return launch_rows<128, 256, 2, 4, 3, TB>(a, s);
    return launch_rows<256, 256, 2, 4, 2, TB>(a, s);
}

int64_t weight_blocks(const GroupArgs &a, int t) {
    const int64_t nn = (a.N + t - 1) / t, nk = (a.K + t - 1) / t;
    if (a.E <= GP_RANKED) return ((int64_t)a.E * 4 + 7) / 8 * 8 * ((nn + 1) / 2) * ((nk + 1) / 2);
    return (a.E * nn * nk + 7) / 8 * 8;
}

// Tiles of the weights' gradient (1536 x 2048 bf16 unless said).  256 square
// where there are many (512 experts of 16, 80 and 256 rows: 0.68, 0.88 and 1.36
// ms against 0.73, 1.05 and 1.51 with 128 square) or some with long
// contractions (16 experts of 1024 rows, fp32: 115 against 129 us; of 256 rows:
// 64 against 53).  Else 128 square, three blocks to a CU (4 experts of 1024
// rows, 2048 x 768: 20 us, 64 square 27), and 64 square where even those are
// fewer than the CUs (4 experts of 4096 rows, 128 x 128: 17 against 28 us).
// Steps of 32 in three buffers but for the smallest, of 64 in four: 32768 rows of
// 16 uneven experts in 256 square 210 us, with steps of 64 in two buffers 225;
// 16 experts of 256 rows in 128 square 46 against 53 us.
strata_status grouped_weights(const GroupArgs &a, hipStream_t s) {
    const int64_t large = (int64_t)a.E * ((a.N + 255) / 256) * ((a.K + 255) / 256);
    const int64_t small = (int64_t)a.E * ((a.N + 127) / 128) * ((a.K + 127) / 128);
    if (large >= 1024 || (large >= 512 && a.rows >= 512 * (int64_t)a.E))
        STRATA_LAUNCH((grouped_wgrad_kernel<256, 256, 2, 4, 3, 32>), dim3((unsigned)weight_blocks(a, 256)), dim3(512), 0, s, a);
    else if (small >= 256)
        STRATA_LAUNCH((grouped_wgrad_kernel<128, 128, 2, 2, 3, 32>), dim3((unsigned)weight_blocks(a, 128)), dim3(256), 0, s, a);
    else
        STRATA_LAUNCH((grouped_wgrad_kernel<64, 64, 1, 2, 4, 64>), dim3((unsigned)weight_blocks(a, 64)), dim3(128), 0, s, a);
    return hip_status(hipGetLastError());
}

}  // namespace

}  // namespace strata

using namespace strata;

extern "C" {

size_t strata_moe_grouped_workspace_bytes(int32_t rows, int32_t n_experts, int32_t N, int32_t K) {
    if (check_grouped(rows, n_experts, N, K) != STRATA_OK) return 0;
    return GP_HEAD + (size_t)(max_tiles(rows, n_experts, GP_MIN_ROWS) + 1) * sizeof(GroupItem);
}

strata_status strata_moe_grouped_product(const void *x, const void *W, const int32_t *offsets, int32_t rows,
                                         int32_t n_experts, int32_t N, int32_t K, void *y, strata_xdtype ydtype,
                                         void *ws, size_t ws_bytes, void *stream) {
    GroupArgs a{};
    const strata_status st =
        rows == 0 ? check_no_rows(n_experts, N, K, ydtype)
                  : grouped_call(x, W, offsets, rows, n_experts, N, K, y, (int64_t)rows * N, ydtype, ws, ws_bytes, a);
    if (st != STRATA_OK || rows == 0) return st;
    if (few_rows_path(rows, n_experts, K)) {
        const int slabs = (N + GV_N - 1) / GV_N;
        STRATA_LAUNCH(grouped_few_kernel, dim3((unsigned)rows * slabs), dim3(256), (size_t)GV_R * K * 2,
                      (hipStream_t)stream, a, slabs);
        return hip_status(hipGetLastError());
    }
    return grouped_rows<0>(a, (hipStream_t)stream);
}

strata_status strata_moe_grouped_dgrad(const void *dy, const void *W, const int32_t *offsets, int32_t rows,
                                       int32_t n_experts, int32_t N, int32_t K, void *dx, strata_xdtype xdtype,
                                       void *ws, size_t ws_bytes, void *stream) {
    GroupArgs a{};
    const strata_status st =
        rows == 0 ? check_no_rows(n_experts, N, K, xdtype)
                  : grouped_call(dy, W, offsets, rows, n_experts, N, K, dx, (int64_t)rows * K, xdtype, ws, ws_bytes, a);
    if (st != STRATA_OK || rows == 0) return st;
    return grouped_rows<1>(a, (hipStream_t)stream);
}

strata_status strata_moe_grouped_wgrad(const void *dy, const void *x, const int32_t *offsets, int32_t rows,
                                       int32_t n_experts, int32_t N, int32_t K, void *dW, strata_xdtype wdtype,
                                       void *ws, size_t ws_bytes, void *stream) {
    GroupArgs a{};
    // without rows dy and x may be null: dW stands in for them and is not read
    const bool none = rows == 0;
    const strata_status st = grouped_call(none ? dW : dy, none ? dW : x, offsets, rows, n_experts, N, K, dW,
                                          (int64_t)n_experts * N * K, wdtype, ws, ws_bytes, a);
    if (st != STRATA_OK) return st;
    return grouped_weights(a, (hipStream_t)stream);
}

}  // extern "C"
