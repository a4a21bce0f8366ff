// Softmax cross entropy over a vocabulary (strata_vocab_loss and its
// gradient): tile products of the packed rows with the output matrix whose
// epilogues never store the logits.
//
// A first launch packs the rows that have a target, so the others cost no
// products and their contents reach nothing.  Forward: the tiles of
// z = h W^T leave the maximum and the sum of exponentials of each row's tile
// (8 bytes for 128 or 256 logits), a last launch joins them.  Gradient, a
// piece of the vocabulary at a time: dz = (dloss + dlse) exp(z - lse) less
// dloss at the target, from the same tiles, as bf16 into the workspace (a
// piece is sized so that it stays in the last-level cache), then
// dW = dz^T h of the piece and dh += dz W, its contraction cut into spans
// where the tiles of dh are fewer than the CUs.  Where an output is fp32, dz is
// kept in three bf16 pieces, which hold fp32's 24 bits, and its products run over
// all of them: two hold 16, which left 2^-18 of every value of dz, 1 to 2e-6 of
// the gradients, where fp32 sums leave 1 to 3e-7 (at 7 for 5 units of products:
// 2047 tokens of 50001 x 1000 1455 us for 1058).  dz is kept
// over a unit, the first dloss without its exponent: of a mean, where all are the
// same 1/n, the targets' entries, the largest of each row, are then a power of two
// less a small number, which bf16 holds, and not 1/n, whose rounding would be the
// same in every row (up to 2^-8 of both gradients).
//
// 4096 tokens of 128000 x 2048, all products bound by the matrix cores at the clock
// the card's power leaves: the loss 1726 us (1.24 PFLOP/s), a piece of the
// gradient, 16384 columns and a quarter of the tokens without target, 210 us the
// logits, 166 dW and 198 dh.  5 tokens: 92 us, 5.7 TB/s of the matrix.
#include <cmath>

#include "vocab_impl.hpp"

namespace strata {

constexpr int VOCAB_V = 1 << 20, VOCAB_T = 1 << 20, VOCAB_D = 16384;

// Tokens with a target to their packed places; per token without one, the
// outputs' zeros.  A block finds the place of its first row by counting the
// targets of all tokens before it.
template <int GRAD> __global__ __launch_bounds__(256) void vocab_pack_kernel(VocabArgs a) {
    __shared__ int cnt[4], slot[256];
    const int th = threadIdx.x, lane = th & 63, w = __builtin_amdgcn_readfirstlane(th >> 6);
    const int t0 = blockIdx.x * a.rows_block, t1 = min(t0 + a.rows_block, a.T);
    const auto has = [&](int t) { return (uint32_t)a.targets[t] < (uint32_t)a.V; };
    int before = 0;
#pragma unroll 4
    for (int t = th; t < t0; t += 256) before += has(t) ? 1 : 0;
    before = wave_sum(before);
    if (lane == 0) cnt[w] = before;
    __syncthreads();
    int base = cnt[0] + cnt[1] + cnt[2] + cnt[3];
    if (GRAD && blockIdx.x == 0) {   // the unit of dz: the first weight's that is not zero, without its exponent
        __shared__ int first[4];
        int f = a.T;
        for (int t0 = 0; f == a.T && t0 < a.T; t0 += 256) {
            const int t = t0 + th;
            const uint64_t m = __ballot(t < a.T && has(t) && a.dloss[t] != 0.f);
            if (lane == 0) first[w] = m ? t0 + 64 * w + __builtin_ctzll(m) : a.T;
            __syncthreads();
            f = min(min(first[0], first[1]), min(first[2], first[3]));
            __syncthreads();
        }
        if (th == 0) *a.unit = f < a.T ? __uint_as_float((__float_as_uint(a.dloss[f]) & 0x7fffffu) | 0x3f800000u) : 1.f;
    }
    const int nv = a.d / 8;
    for (int c = t0; c < t1; c += 256) {
        __syncthreads();
        const int t = c + th;
        const bool in = t < t1, kept = in && has(t);
        const uint64_t m = __ballot(kept);
        if (lane == 0) cnt[w] = __popcll(m);
        __syncthreads();
        int at = base + __popcll(m & ((1ull << lane) - 1));
        for (int q = 0; q < w; ++q) at += cnt[q];
        base += cnt[0] + cnt[1] + cnt[2] + cnt[3];
        slot[th] = kept ? at : -1;
        if (kept) {
            a.map[at] = t;
            a.tc[at] = a.targets[t];
            if (GRAD) {
                const float u = a.dloss[t];
                a.lc[at] = a.lse_in[t];
                a.gc[at] = u + (a.dlse ? a.dlse[t] : 0.f);
                a.dc[at] = u;
            }
        } else if (in && !GRAD) {
            a.loss[t] = 0.f;
            a.lse[t] = 0.f;
        }
        __syncthreads();
        for (int r = w; r < min(256, t1 - c); r += 4) {
            const int s = __builtin_amdgcn_readfirstlane(slot[r]);
            const int64_t t = c + r;
            if (s >= 0) {
                const u32x4_t *from = (const u32x4_t *)(a.h + t * a.d);
                u32x4_t *to = (u32x4_t *)(a.hc + (int64_t)s * a.d);
                for (int i = lane; i < nv; i += 64) to[i] = from[i];
            } else if (GRAD && a.dh) {
                u32x4_t *to = (u32x4_t *)((char *)a.dh + t * a.d * (a.dh_bf16 ? 2 : 4));
                for (int i = lane; i < (a.dh_bf16 ? nv : 2 * nv); i += 64) to[i] = u32x4_t{0, 0, 0, 0};
            }
        }
    }
    if (t1 == a.T && th == 0) *a.n = base;
}

// The running maximum and sum of exponentials, met by another.
__device__ __forceinline__ void meet(float &m, float &s, float2 p) {
    const float u = fmaxf(m, p.x), b = u == -INFINITY ? 0.f : u;
    s = s * exp_diff(m, b) + p.y * exp_diff(p.x, b);
    m = u;
}

// A row's tiles joined: R rows to a block, 1024 / R threads to a row.  FEW: a
// block for each of up to 32 tokens, of which it finds the row itself.
template <int R, int FEW> __global__ __launch_bounds__(1024) void vocab_join_kernel(VocabArgs a) {
    __shared__ float2 sh[16][R];
    const int th = threadIdx.x, lane = th & 63, w = th >> 6;
    const int r = th % R, sub = th / R;
    int row = blockIdx.x * R + r, n = 0;
    if constexpr (FEW) {
        const uint32_t there = few_tokens(a);
        if (!(there >> blockIdx.x & 1)) {
            if (th == 0) a.loss[blockIdx.x] = a.lse[blockIdx.x] = 0.f;
            return;
        }
        row = __popc(there & ((1u << blockIdx.x) - 1));
        n = 32;
    } else {
        n = *a.n;
        if ((int)blockIdx.x * R >= n) return;
    }
    float m = -INFINITY, s = 0.f;
    if (row < n) {
#pragma unroll 4
        for (int c = sub; c < a.tiles; c += 1024 / R) meet(m, s, a.part[(int64_t)c * a.ldp + row]);
    }
#pragma unroll
    for (int o = R; o < 64; o <<= 1) meet(m, s, float2{__shfl_xor(m, o, 64), __shfl_xor(s, o, 64)});
    if (lane < R) sh[w][lane] = float2{m, s};
    __syncthreads();
    if (th >= R || row >= n) return;
    for (int q = 1; q < 16; ++q) meet(m, s, sh[q][r]);
    const float lse = m + logf(s);
    const int t = FEW ? (int)blockIdx.x : a.map[row];
    a.lse[t] = lse;
    a.loss[t] = lse - a.zt[row];
}

// dh of the rows with a target: the spans' sums added and rounded.
__global__ __launch_bounds__(256) void vocab_dh_out_kernel(VocabArgs a) {
    const int n = *a.n, nq = a.d / 4;
    const int64_t all = (int64_t)n * nq;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int row = (int)(i / nq), c = (int)(i - (int64_t)row * nq) * 4;
        f32x4_t v = {0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < a.splits; ++s) v += *(const f32x4_t *)(a.acc + ((int64_t)s * a.T + row) * a.d + c);
        const float unit = *a.unit, q[4] = {v[0] * unit, v[1] * unit, v[2] * unit, v[3] * unit};
        const int64_t at = (int64_t)a.map[row] * a.d + c;
        if (a.dh_bf16) store_values<4>((uint16_t *)a.dh, at, q);
        else store_values<4>((float *)a.dh, at, q);
    }
}

// dW without tokens.
__global__ __launch_bounds__(256) void vocab_zero_kernel(u32x4_t *p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = u32x4_t{0, 0, 0, 0};
}

namespace {

strata_status check_vocab(int32_t T, int32_t V, int32_t d) {
    if (T < 0) return STRATA_EINVAL;
    if (V < 1 || V > VOCAB_V || d < 8 || d % 8 || d > VOCAB_D || T > VOCAB_T || (int64_t)T * d > ((int64_t)1 << 33))
        return STRATA_EUNSUPPORTED;
    if ((int64_t)T * V > ((int64_t)1 << 38)) return STRATA_EUNSUPPORTED;   // a grid of fewer than 2^32 threads
    return STRATA_OK;
}

int64_t up_to(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

// Tiles, and what a round of them over the CUs costs (a tile of 256 square 100).
// A launch takes the tile whose rounds cost least: most calls have a few rounds
// or a part of one, and their number matters more than a tile's own rate.  By the
// tokens of the call: how many have a target only the device knows.  Calls of up
// to 32 tokens, which the matrix bounds, take tiles of 32 rows.  64 x 128 and, of
// dW, 64 square against 256 square and 128 square: 2655 tokens, 1287 x 160, both
// gradients, 99 -> 56 us; 128 x 256 against 256 square: 2828 tokens, 6228 x 1032,
// the loss, 73 -> 68 us.
enum Tile { ROWS_32, ROWS_64, ROWS_128, ROWS_256 };
constexpr int TILE_ROWS[] = {32, 64, 128, 256}, TILE_COLS[] = {128, 128, 256, 256}, TILE_COST[] = {12, 20, 56, 100};
int64_t tiles_of(Tile k, int64_t rows, int64_t cols) {
    return (rows + TILE_ROWS[k] - 1) / TILE_ROWS[k] * ((cols + TILE_COLS[k] - 1) / TILE_COLS[k]);
}
Tile logits_tile(int64_t T, int64_t pw) {
    if (T <= 32) return ROWS_32;
    Tile best = ROWS_256;
    int64_t least = INT64_MAX;
    for (const Tile k : {ROWS_256, ROWS_128, ROWS_64}) {
        const int64_t c = (tiles_of(k, T, pw) + 255) / 256 * TILE_COST[k];
        if (c < least) best = k, least = c;
    }
    return best;
}

// Tile of dh and the spans that its contraction over a piece's columns is cut
// into, 512 columns or more each; a span's sums cost as much as 8 of its rounds.
struct DhTile {
    Tile tile;
    int splits;
};
DhTile dh_tile(int64_t T, int64_t d, int64_t piece) {
    DhTile best{ROWS_32, 1};
    int64_t least = INT64_MAX;
    const int64_t most = piece / 512 > 1 ? piece / 512 : 1;
    for (const Tile k : {ROWS_256, ROWS_128, ROWS_64, ROWS_32}) {
        if ((T <= 32) != (k == ROWS_32)) continue;
        const int64_t t = tiles_of(k, T, d);
        int64_t s = t ? 256 / t : 1;
        s = s < 1 ? 1 : s > most ? most : s;
        const int64_t c = (t * s + 255) / 256 * TILE_COST[k] * 64 / s + 8 * s;
        if (c < least) best = DhTile{k, (int)s}, least = c;
    }
    return best;
}

// Tiles of dW, squares: one of 256 to a CU, up to three of 128 or two of 64, which alone on a CU take less.
enum Square { SQUARE_64, SQUARE_128, SQUARE_256 };
Square dw_tile(int64_t pw, int64_t d) {
    const auto count = [&](int64_t n) { return (pw + n - 1) / n * ((d + n - 1) / n); };
    const int64_t t256 = count(256), t128 = count(128), t64 = count(64);
    const int64_t c256 = (t256 + 255) / 256 * 100;
    const int64_t c128 = t128 <= 256 ? 35 : t128 <= 512 ? 55 : (t128 + 767) / 768 * 75;
    const int64_t c64 = t64 <= 256 ? 14 : (t64 + 511) / 512 * 18;
    return c64 < c128 && c64 < c256 ? SQUARE_64 : c128 < c256 ? SQUARE_128 : SQUARE_256;
}

struct VocabPlan {
    int piece;
    Tile tile;    // of the loss
    DhTile dh;
    size_t map, tc, hc, zt, part, lc, gc, dc, dz, acc, bytes;
};

// Columns of a piece: a bf16 dz of 128 MiB (two of them lie in the last-level
// cache), no fewer than 2048 so that a piece's products fill the CUs.  Half of it
// for fp32 outputs, whose three are past the cache, takes 2047 tokens of 50001 x
// 1000 from 1451 to 1387 us and 4001 of 32000 x 2048 from 3207 to 3510.
int piece_columns(int32_t T, int32_t V) {
    int64_t c = ((int64_t)1 << 26) / T / 256 * 256;
    if (c < 2048) c = 2048;
    const int64_t all = up_to(V, 256);
    return (int)(c < all ? c : all);
}

VocabPlan vocab_plan(int32_t T, int32_t V, int32_t d, bool grad) {
    VocabPlan p{};
    size_t at = 256;   // the count of rows
    const auto take = [&](size_t n) {
        const size_t q = at;
        at += (n + 255) / 256 * 256;
        return q;
    };
    p.map = take((size_t)T * 4);
    p.tc = take((size_t)T * 4);
    p.hc = take((size_t)T * d * 2);
    if (!grad) {
        p.zt = take((size_t)T * 4);
        p.tile = logits_tile(T, V);
        p.part = take((size_t)((V + TILE_COLS[p.tile] - 1) / TILE_COLS[p.tile]) * up_to(T, 16) * 8);
    } else {
        p.lc = take((size_t)T * 4);
        p.gc = take((size_t)T * 4);
        p.dc = take((size_t)T * 4);
        p.piece = piece_columns(T > 0 ? T : 1, V);
        p.dh = dh_tile(T, d, p.piece);
        p.dz = take((size_t)T * p.piece * 2 * 3);
        p.acc = take((size_t)p.dh.splits * T * d * 4);
    }
    p.bytes = at;
    return p;
}

bool bad_vector(const void *p) { return !p || ((uintptr_t)p & 3u); }

void vocab_common(VocabArgs &a, const VocabPlan &p, char *w) {
    a.n = (int32_t *)w;
    a.unit = (float *)w + 1;
    a.map = (int32_t *)(w + p.map);
    a.tc = (int32_t *)(w + p.tc);
    a.hc = (uint16_t *)(w + p.hc);
    a.rows_block = (int)up_to((a.T + 511) / 512, 16);
}

// Grid of nr x nc tiles dealt to 8 XCDs.
dim3 tile_grid(int64_t nr, int64_t nc) { return dim3((unsigned)up_to(nr * nc, 8)); }

#define VOCAB_TRY                                                 \
    do {                                                          \
        const hipError_t e_ = hipGetLastError();                  \
        if (e_ != hipSuccess) return hip_status(e_);              \
    } while (0)

template <int GRAD> strata_status launch_logits(const VocabArgs &a, Tile k, hipStream_t s) {
    const dim3 g = tile_grid((a.T + TILE_ROWS[k] - 1) / TILE_ROWS[k], (a.pw + TILE_COLS[k] - 1) / TILE_COLS[k]);
    if constexpr (GRAD != 0) {   // a forward call of few rows has its own
        if (k == ROWS_32) {
            STRATA_LAUNCH((vocab_logits_kernel<32, 128, 1, 4, 4, GRAD>), g, dim3(256), 0, s, a);
            return hip_status(hipGetLastError());
        }
    }
    if (k == ROWS_64) STRATA_LAUNCH((vocab_logits_kernel<64, 128, 2, 2, 4, GRAD>), g, dim3(256), 0, s, a);
    else if (k == ROWS_128) STRATA_LAUNCH((vocab_logits_kernel<128, 256, 2, 4, 3, GRAD>), g, dim3(512), 0, s, a);
    else STRATA_LAUNCH((vocab_logits_kernel<256, 256, 2, 4, 2, GRAD>), g, dim3(512), 0, s, a);
    return hip_status(hipGetLastError());
}

template <int PIECES> strata_status launch_dh(const VocabArgs &a, Tile k, hipStream_t s) {
    const dim3 g = tile_grid((int64_t)((a.T + TILE_ROWS[k] - 1) / TILE_ROWS[k]) * a.splits, (a.d + TILE_COLS[k] - 1) / TILE_COLS[k]);
    if (k == ROWS_32) STRATA_LAUNCH((vocab_dh_kernel<32, 128, 1, 4, 4, PIECES>), g, dim3(256), 0, s, a);
    else if (k == ROWS_64) STRATA_LAUNCH((vocab_dh_kernel<64, 128, 2, 2, 4, PIECES>), g, dim3(256), 0, s, a);
    else if (k == ROWS_128) STRATA_LAUNCH((vocab_dh_kernel<128, 256, 2, 4, 3, PIECES>), g, dim3(512), 0, s, a);
    else STRATA_LAUNCH((vocab_dh_kernel<256, 256, 2, 4, 2, PIECES>), g, dim3(512), 0, s, a);
    return hip_status(hipGetLastError());
}

template <int PIECES> strata_status launch_dw(const VocabArgs &a, hipStream_t s) {
    const auto grid = [&](int64_t n) { return tile_grid((a.pw + n - 1) / n, (a.d + n - 1) / n); };
    switch (dw_tile(a.pw, a.d)) {
        case SQUARE_64: STRATA_LAUNCH((vocab_dw_kernel<64, 64, 1, 2, 4, 64, PIECES>), grid(64), dim3(128), 0, s, a); break;
        case SQUARE_128: STRATA_LAUNCH((vocab_dw_kernel<128, 128, 2, 2, 3, 32, PIECES>), grid(128), dim3(256), 0, s, a); break;
        default: STRATA_LAUNCH((vocab_dw_kernel<256, 256, 2, 4, 3, 32, PIECES>), grid(256), dim3(512), 0, s, a);
    }
    return hip_status(hipGetLastError());
}

}  // namespace

}  // namespace strata

using namespace strata;

extern "C" {

size_t strata_vocab_loss_workspace_bytes(int32_t T, int32_t V, int32_t d) {
    return check_vocab(T, V, d) == STRATA_OK ? vocab_plan(T, V, d, false).bytes : 0;
}

size_t strata_vocab_loss_backward_workspace_bytes(int32_t T, int32_t V, int32_t d) {
    return check_vocab(T, V, d) == STRATA_OK ? vocab_plan(T, V, d, true).bytes : 0;
}

strata_status strata_vocab_loss(const void *h, const void *W, const int32_t *targets, int32_t T, int32_t V, int32_t d,
                                float *loss, float *lse, void *ws, size_t ws_bytes, void *stream) {
    const strata_status st = check_vocab(T, V, d);
    if (st != STRATA_OK || T == 0) return st;
    if (bad_rows(h) || bad_rows(W) || bad_vector(targets) || bad_vector(loss) || bad_vector(lse) || bad_rows(ws))
        return STRATA_EINVAL;
    const VocabPlan p = vocab_plan(T, V, d, false);
    if (ws_bytes < p.bytes) return STRATA_EWORKSPACE;
    // The packed rows' places and the tokens they go back to are read from here.
    const size_t n = (size_t)T * 4;
    if (overlap(ws, p.bytes, targets, n) || overlap(ws, p.bytes, loss, n) || overlap(ws, p.bytes, lse, n) ||
        overlap(targets, n, loss, n) || overlap(targets, n, lse, n))
        return STRATA_EINVAL;
    const hipStream_t s = (hipStream_t)stream;
    char *const w = (char *)ws;
    VocabArgs a{};
    a.h = (const uint16_t *)h;
    a.W = (const uint16_t *)W;
    a.targets = targets;
    a.loss = loss;
    a.lse = lse;
    a.T = T;
    a.V = V;
    a.d = d;
    vocab_common(a, p, w);
    a.zt = (float *)(w + p.zt);
    a.part = (float2 *)(w + p.part);
    a.ldp = (int)up_to(T, 16);
    a.pw = V;
    a.tiles = (V + TILE_COLS[p.tile] - 1) / TILE_COLS[p.tile];
    if (p.tile == ROWS_32) {   // packing and joining apart cost 5 tokens of 128000 x 2048 another 6 of 103 us
        STRATA_LAUNCH((vocab_logits_kernel<32, 128, 1, 4, 4, 0, 1>), tile_grid(1, a.tiles), dim3(256), 0, s, a);
        VOCAB_TRY;
        STRATA_LAUNCH((vocab_join_kernel<1, 1>), dim3(T), dim3(1024), 0, s, a);
        return hip_status(hipGetLastError());
    }
    STRATA_LAUNCH(vocab_pack_kernel<0>, dim3((T + a.rows_block - 1) / a.rows_block), dim3(256), 0, s, a);
    VOCAB_TRY;
    const strata_status lt = launch_logits<0>(a, p.tile, s);
    if (lt != STRATA_OK) return lt;
    STRATA_LAUNCH((vocab_join_kernel<16, 0>), dim3((T + 15) / 16), dim3(1024), 0, s, a);
    return hip_status(hipGetLastError());
}

strata_status strata_vocab_loss_backward(const void *h, const void *W, const int32_t *targets, int32_t T, int32_t V,
                                         int32_t d, const float *lse, const float *dloss, const float *dlse, void *dh,
                                         strata_xdtype dhdtype, void *dW, strata_xdtype dwdtype, uint32_t flags, void *ws,
                                         size_t ws_bytes, void *stream) {
    if ((dh && bad_dtype(dhdtype)) || (dW && bad_dtype(dwdtype)) || (flags & ~STRATA_ACCUMULATE)) return STRATA_EINVAL;
    const strata_status st = check_vocab(T, V, d);
    if (st != STRATA_OK) return st;
    if ((dh && !aligned16(dh)) || (dW && !aligned16(dW))) return STRATA_EINVAL;
    const bool add = flags & STRATA_ACCUMULATE;
    const hipStream_t s = (hipStream_t)stream;
    const size_t dw_bytes = (size_t)V * d * (dwdtype == STRATA_X_BF16 ? 2 : 4);
    if (T == 0) {
        if (!dW || add) return STRATA_OK;
        const int64_t n = (int64_t)(dw_bytes / 16), blocks = (n + 255) / 256;
        STRATA_LAUNCH(vocab_zero_kernel, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, s, (u32x4_t *)dW, n);
        return hip_status(hipGetLastError());
    }
    if (bad_rows(h) || bad_rows(W) || bad_vector(targets) || bad_vector(lse) || bad_vector(dloss) || (dlse && bad_vector(dlse)) ||
        bad_rows(ws))
        return STRATA_EINVAL;
    const VocabPlan p = vocab_plan(T, V, d, true);
    if (ws_bytes < p.bytes) return STRATA_EWORKSPACE;
    const size_t n = (size_t)T * 4, dh_bytes = dh ? (size_t)T * d * (dhdtype == STRATA_X_BF16 ? 2 : 4) : 0;
    if (overlap(ws, p.bytes, targets, n) || overlap(ws, p.bytes, dh, dh_bytes) || overlap(ws, p.bytes, dW, dw_bytes) ||
        overlap(targets, n, dh, dh_bytes) || overlap(targets, n, dW, dw_bytes))
        return STRATA_EINVAL;
    if (!dh && !dW) return STRATA_OK;
    char *const w = (char *)ws;
    VocabArgs a{};
    a.h = (const uint16_t *)h;
    a.W = (const uint16_t *)W;
    a.targets = targets;
    a.lse_in = lse;
    a.dloss = dloss;
    a.dlse = dlse;
    a.dh = dh;
    a.dW = dW;
    a.T = T;
    a.V = V;
    a.d = d;
    a.dh_bf16 = dhdtype == STRATA_X_BF16;
    a.dw_bf16 = dwdtype == STRATA_X_BF16;
    a.add = add;
    vocab_common(a, p, w);
    a.lc = (float *)(w + p.lc);
    a.gc = (float *)(w + p.gc);
    a.dc = (float *)(w + p.dc);
    a.dz = (uint16_t *)(w + p.dz);
    a.next = (int64_t)T * p.piece;
    a.acc = (float *)(w + p.acc);
    a.splits = p.dh.splits;
    const bool h3 = dh && !a.dh_bf16, w3 = dW && !a.dw_bf16;   // outputs that take all of dz
    STRATA_LAUNCH(vocab_pack_kernel<1>, dim3((T + a.rows_block - 1) / a.rows_block), dim3(256), 0, s, a);
    VOCAB_TRY;
    for (int v0 = 0; v0 < V; v0 += p.piece) {
        a.v0 = v0;
        a.pw = V - v0 < p.piece ? V - v0 : p.piece;
        a.ldv = (int)up_to(a.pw, 8);
        a.first = v0 == 0;
        a.span = (int)up_to((a.pw + a.splits - 1) / a.splits, 64);
        const Tile k = logits_tile(T, a.pw);
        strata_status q = h3 || w3 ? launch_logits<3>(a, k, s) : launch_logits<1>(a, k, s);
        if (q == STRATA_OK && dW) q = w3 ? launch_dw<3>(a, s) : launch_dw<1>(a, s);
        if (q == STRATA_OK && dh) q = h3 ? launch_dh<3>(a, p.dh.tile, s) : launch_dh<1>(a, p.dh.tile, s);
        if (q != STRATA_OK) return q;
    }
    if (!dh) return STRATA_OK;
    const int64_t blocks = ((int64_t)T * (d / 4) + 255) / 256;
    STRATA_LAUNCH(vocab_dh_out_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, a);
    return hip_status(hipGetLastError());
}

}  // extern "C"
