// Matrices orthogonalised by Newton-Schulz products (strata_orthogonalise).
//
//   A = X X^T,  B = b A + c A^2,  X' = a X + B X        (from the right where N > K)
//
// Three launches of tile products a step, over all matrices at once; b A, c,
// a X and the last scale are epilogues.  A and B are symmetric: only the
// tiles of their lower halves are computed.  The operands are fp16: the values
// are in known ranges (|X| and |A| at most about 1, X kept times a power of
// two), and 11 bits, with the diagonals of A and B in fp32, leave the result
// 5e-4 to 1.2e-3 off, less than its own rounding to bf16 (1.7e-3), where bf16's 8
// would leave 3e-3 to 12e-3.  X itself is hi + lo, 22 bits: with hi alone the rounding
// of X, a matrix of full rank, would be multiplied by a at every step like the
// small directions of G itself (3.4^5 = 485 in five steps; a gradient of 80 rows
// in 1536 x 2048 would come out 2% off).  The last of several steps takes hi
// alone: one factor a.
//
// 16 of 1536 x 2048, a step: A 116 us, B 84 (0.66 and 0.69 PFLOP/s of the halves
// computed), X' 184 (0.84); bound by what the products wait for their loads.
#include <cmath>

#include "orth_small.hpp"

namespace strata {

constexpr int ORTH_SIDE = 16384, ORTH_N = 1024, ORTH_PARTS = 64;

template <int V, typename G> __device__ __forceinline__ void piece_values(const G *p, int64_t i, float (&v)[V]) {
    Raw<G, V> r;
    load_raw<V>(p, i, r);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = value<V>(r, j);
}

// Sum of squares of a part of a matrix, in 64 bits.  Pieces of V values do not cross rows.
template <typename G, int V> __global__ __launch_bounds__(256) void orth_norm_kernel(OrthArgs a) {
    __shared__ double sh[4];
    const int e = blockIdx.y, part = blockIdx.x;
    const int64_t pieces = (int64_t)a.N * a.K / V, per = (pieces + a.parts - 1) / a.parts;
    const int64_t p0 = part * per, p1 = min(p0 + per, pieces);
    const G *g = (const G *)a.G + (int64_t)e * a.N * a.K;
    double s = 0.0;
#pragma unroll 4
    for (int64_t p = p0 + threadIdx.x; p < p1; p += 256) {
        float v[V];
        piece_values<V, G>(g, p * V, v);
#pragma unroll
        for (int j = 0; j < V; ++j) s = fma((double)v[j], (double)v[j], s);
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o, 64);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) a.norms[e * a.parts + part] = sh[0] + sh[1] + sh[2] + sh[3];
}

// 1 / (|G| + eps) of matrix e.
__device__ __forceinline__ double one_over_norm(const OrthArgs &a, int e) {
    static_assert(ORTH_PARTS <= 64, "a lane for each");
    const int lane = threadIdx.x & 63;
    double s = lane < a.parts ? a.norms[e * a.parts + lane] : 0.0;
#pragma unroll
    for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o, 64);
    return 1.0 / (sqrt(s) + (double)a.eps);
}

// No steps: out = scale G / (|G| + eps).
template <typename G, int V> __global__ __launch_bounds__(256) void orth_scale_kernel(OrthArgs a) {
    const int e = blockIdx.y;
    const double r = one_over_norm(a, e) * (double)a.scale;
    const int64_t m0 = (int64_t)e * a.N * a.K, all = (int64_t)a.N * a.K / V;
    for (int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x; p < all; p += (int64_t)gridDim.x * 256) {
        float v[V];
        piece_values<V, G>((const G *)a.G + m0, p * V, v);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = (float)((double)v[j] * r);
        store_values<V>(a.out + m0, p * V, v);
    }
}

// The tiles of a step, and their subtiles in the order of lo: tile, wave, row of subtiles, column.
struct StepShape {
    int bm, bn, wm, wn;
};

// X_0 = G / (|G| + eps), times size, as hi and lo: a wave takes a subtile of the
// steps' tiles, zeros where it lies outside the matrix.  201 MB to 101 us, 4 TB/s
// (a first step that read G in place of lo, in its few waves' epilogue, took 280 us
// for 215 and this kernel 50: the same in all for 16 of 1536 x 2048, but 316 for
// 307 us of 1 of 2048 x 2048 and 98 for 95 of 6 of 173 x 874).
template <typename G, int V> __global__ __launch_bounds__(512) void orth_start_kernel(OrthArgs a, StepShape k, int64_t all) {
    const int64_t s = (int64_t)blockIdx.x * 8 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (s >= all) return;
    const int mt = k.bm / 32 / k.wm, nt = k.bn / 32 / k.wn, per = k.wm * k.wn * mt * nt;
    const int64_t t = s / per;
    const int sub = (int)(s - t * per), j = sub % nt, i = sub / nt % mt, w = sub / (nt * mt);
    const int nk = (a.K + k.bn - 1) / k.bn, nr = (a.N + k.bm - 1) / k.bm;
    const int e = (int)(t / (nr * nk)), at = (int)(t - (int64_t)e * nr * nk);
    int m0, n0;
    wave_place_of(w, k.wm, k.wn, mt, nt, m0, n0);
    const int lane = threadIdx.x & 63, l = lane & 31, h = lane >> 5;
    const int row0 = at / nk * k.bm, m = row0 + m0 + 32 * i + l, n = at % nk * k.bn + n0 + 32 * j;
    // size / (|G| + eps) as two fp32 factors: alone it is past fp32 for norms below size / 3.4e38 (0 * inf for a matrix
    // of zeros and a small eps) and has lost bits for norms above size * 8.5e37.  For r within 2^-64 .. 2^64 u is 1.
    const double r = one_over_norm(a, e) * (double)a.size;
    const float u = r > 0x1p64 ? 0x1p64f : r < 0x1p-64 ? 0x1p-64f : 1.f, f = (float)(r / (double)u);
    const G *g = (const G *)a.G + (int64_t)e * a.N * a.K;
    float x[16];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int c = 0; c < 4; c += V) {
            float v[V];
#pragma unroll
            for (int p = 0; p < V; ++p) v[p] = 0.f;
            const int col = n + 8 * q + 4 * h + c;
            if (m < a.N && col < a.K) piece_values<V, G>(g, (int64_t)m * a.K + col, v);
#pragma unroll
            for (int p = 0; p < V; ++p) x[4 * q + c + p] = v[p] * u * f;
        }
    u32x2_t *const lo = (u32x2_t *)a.lo + s * 256 + lane;
    uint32_t w2[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        u32x2_t y;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const uint32_t z = half_pair_kept(x[4 * q + 2 * p], x[4 * q + 2 * p + 1]);
            w2[2 * q + p] = z;
            y[p] = half_pair_left(x[4 * q + 2 * p], x[4 * q + 2 * p + 1], z);
        }
        lo[q * 64] = y;
    }
    store_halves(half_rows(a.hi + ((int64_t)e * a.N + row0) * a.ldx, min(a.N - row0, k.bm), a.ldx), m0 + 32 * i, n, a.ldx, 0, 0, w2);
}

namespace {

strata_status check_orth(int32_t n, int32_t N, int32_t K) {
    if (n < 0 || N < 1 || K < 1) return STRATA_EINVAL;
    if (N > ORTH_SIDE || K > ORTH_SIDE || n > ORTH_N || (int64_t)n * N * K > ((int64_t)1 << 33)) return STRATA_EUNSUPPORTED;
    return STRATA_OK;
}

struct OrthPlan {
    int side, ldx, lds;
    size_t hi, next, lo, A, B, dA, dB, bytes;
};

// Tiles of a step by how many of 128 square there are: below 144, 64 x 128 (a
// step of 2 of 512 x 2048, 128 tiles: 10.0 us against 13.2; of 1 of 1000 x 1000:
// 11.4 against 14.5); up to 256, 128 square with four buffers (1 of 2048 x 2048:
// 27.6 against 33.6); below 1024 with two, two blocks of 8 waves to a CU (whole
// passes of 8 of 2048 x 768, 768 tiles: 318 us, 256 square 323; 32 of 512 x 512:
// 251 and 274, on one card: others take up to a tenth more of all four); then 256
// square, which spills 52 to 56 bytes a lane (4 of 2048 x 2048: 940, 128 square
// 980; 16 of 1536 x 2048: 1892 and 2055, 128 x 256 1956).
enum StepTile { STEP_64, STEP_128, STEP_128_TWO, STEP_256 };
constexpr StepShape STEP_SHAPES[] = {{64, 128, 2, 2}, {128, 128, 2, 2}, {128, 128, 2, 4}, {256, 256, 2, 4}};
StepTile step_tile(int32_t n, int32_t N, int32_t K) {
    const int64_t tiles = (int64_t)n * ((N + 127) / 128) * ((K + 127) / 128);
    return tiles < 144 ? STEP_64 : tiles <= 256 ? STEP_128 : tiles < 1024 ? STEP_128_TWO : STEP_256;
}

OrthPlan orth_plan(int32_t n, int32_t N, int32_t K) {
    OrthPlan p{};
    p.side = N < K ? N : K;
    p.ldx = (K + 7) / 8 * 8;
    p.lds = (p.side + 7) / 8 * 8;
    size_t at = (size_t)(n > 0 ? n : 1) * ORTH_PARTS * 8;
    const auto take = [&](size_t values) {
        const size_t q = at;
        at += (values * 2 + 255) / 256 * 256;
        return q;
    };
    const size_t x = (size_t)n * N * p.ldx, s = (size_t)n * p.side * p.lds;
    const StepShape k = STEP_SHAPES[step_tile(n, N, K)];
    const size_t rows = (size_t)(N + k.bm - 1) / k.bm * k.bm, cols = (size_t)(K + k.bn - 1) / k.bn * k.bn;
    p.hi = take(x);
    p.next = take(x);
    p.lo = take(n * rows * cols);   // whole tiles
    p.A = take(s);
    p.B = take(s);
    p.dA = take((size_t)n * p.lds * 2);
    p.dB = take((size_t)n * p.lds * 2);
    p.bytes = at;
    return p;
}

template <typename G, int V> hipError_t orth_begin(const OrthArgs &a, int steps, hipStream_t s) {
    STRATA_LAUNCH((orth_norm_kernel<G, V>), dim3(a.parts, a.n), dim3(256), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (steps == 0) {
        const int64_t blocks = ((int64_t)a.N * a.K / V + 1023) / 1024, most = 8192 / a.n + 1;
        STRATA_LAUNCH((orth_scale_kernel<G, V>), dim3((unsigned)(blocks < most ? blocks : most), a.n), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    const StepShape k = STEP_SHAPES[step_tile(a.n, a.N, a.K)];
    const int64_t tiles = (int64_t)a.n * ((a.N + k.bm - 1) / k.bm) * ((a.K + k.bn - 1) / k.bn), all = tiles * (k.bm / 32) * (k.bn / 32);
    STRATA_LAUNCH((orth_start_kernel<G, V < 4 ? V : 4>), dim3((unsigned)((all + 7) / 8)), dim3(512), 0, s, a, k, all);
    return hipGetLastError();
}

template <typename G> hipError_t orth_begin_width(const OrthArgs &a, int steps, hipStream_t s) {
    if (a.K % 8 == 0) return orth_begin<G, 8>(a, steps, s);
    if (a.K % 4 == 0) return orth_begin<G, 4>(a, steps, s);
    if (a.K % 2 == 0) return orth_begin<G, 2>(a, steps, s);
    return orth_begin<G, 1>(a, steps, s);
}

// Whether a matrix fits a block: its registers hold X, its LDS the fp16 copy, A and B.  The shorter side, and the
// longer side that goes with it.
enum SmallShape { SMALL_NONE, SMALL_32, SMALL_64, SMALL_64_LONG, SMALL_128, SMALL_128_LONG };
SmallShape small_shape(int32_t N, int32_t K) {
    const int side = N < K ? N : K, longer = N < K ? K : N;
    if (side <= 32 && longer <= 1792 && longer > 256) return SMALL_32;
    if (side <= 64 && longer <= 512) return SMALL_64;
    if (side <= 64 && longer <= 1024) return SMALL_64_LONG;
    if (side <= 128 && longer <= 256) return SMALL_128;
    return side <= 128 && longer <= 384 ? SMALL_128_LONG : SMALL_NONE;
}

template <typename G> hipError_t orth_small(const OrthArgs &a, int steps, SmallShape k, hipStream_t s) {
    const dim3 g(a.n), b(512);
    switch (k) {
        case SMALL_32: STRATA_LAUNCH((orth_small_kernel<G, 1, 1, 7>), g, b, 0, s, a, steps); break;
        case SMALL_64: STRATA_LAUNCH((orth_small_kernel<G, 2, 2, 2>), g, b, 0, s, a, steps); break;
        case SMALL_64_LONG: STRATA_LAUNCH((orth_small_kernel<G, 2, 2, 4>), g, b, 0, s, a, steps); break;
        case SMALL_128: STRATA_LAUNCH((orth_small_kernel<G, 4, 2, 2>), g, b, 0, s, a, steps); break;
        default: STRATA_LAUNCH((orth_small_kernel<G, 4, 2, 3>), g, b, 0, s, a, steps);
    }
    return hipGetLastError();
}

dim3 range_grid(int64_t tiles) { return dim3((unsigned)((tiles + 7) / 8 * 8)); }

template <int BM, int WM, int WN, int ST, int SQUARE, int ACROSS> void square(const OrthArgs &a, hipStream_t s) {
    const int64_t nt = (a.side + BM - 1) / BM;
    STRATA_LAUNCH((orth_square_kernel<BM, WM, WN, ST, 64, SQUARE, ACROSS>), range_grid(a.n * (nt * (nt + 1) / 2)), dim3(64 * WM * WN),
                  0, s, a);
}

template <int BM, int BN, int WM, int WN, int ST, int TALL> void step(const OrthArgs &a, hipStream_t s) {
    const int64_t nr = (a.N + BM - 1) / BM, nk = (a.K + BN - 1) / BN;
    STRATA_LAUNCH((orth_step_kernel<BM, BN, WM, WN, ST, TALL>), range_grid(a.n * nr * nk), dim3(64 * WM * WN), 0, s, a);
}

// Tiles of the symmetric products by how many there are (8 waves to a tile of
// 128, two blocks of two buffers to a CU or one of four; 4 waves to one of 64),
// us of X X^T and of A^2.  64 square below 112 tiles of 128 (4 of 768 x 768, 84
// tiles: 8.0 and 8.7 against 9.8 and 11.1; 2 of 512 x 2048, 20: 9.8 and 5.5
// against 14.9 and 8.9; 1 of 2048 x 2048, 136: 23 and 24 against 18 and 20).  128
// square with four buffers up to 256 tiles (8 of 2048 x 768, 168: 18.7 and 11.9
// against 23.2 and 13.4 with two), with two above (32 of 512 x 512, 320: 14.3 and
// 16.3 against 15.6 and 18.4; 16 of 1536 x 2048, 1248: 112 and 87 against 110 and
// 91).  256 square, whose tiles are few and all of one length, leaves more CUs
// idle than its fewer LDS reads save (the latter 123 and 112).
template <int SQUARE, int ACROSS> hipError_t squares(const OrthArgs &a, hipStream_t s) {
    const int64_t nt = (a.side + 127) / 128, tiles = a.n * (nt * (nt + 1) / 2);
    if (tiles < 112) square<64, 2, 2, 4, SQUARE, ACROSS>(a, s);
    else if (tiles <= 256) square<128, 2, 4, 4, SQUARE, ACROSS>(a, s);
    else square<128, 2, 4, 2, SQUARE, ACROSS>(a, s);
    return hipGetLastError();
}

template <int TALL> hipError_t steps_of(const OrthArgs &a, hipStream_t s) {
    switch (step_tile(a.n, a.N, a.K)) {
        case STEP_64: step<64, 128, 2, 2, 4, TALL>(a, s); break;
        case STEP_128: step<128, 128, 2, 2, 4, TALL>(a, s); break;
        case STEP_128_TWO: step<128, 128, 2, 4, 2, TALL>(a, s); break;
        default: step<256, 256, 2, 4, 2, TALL>(a, s);
    }
    return hipGetLastError();
}

}  // namespace

}  // namespace strata

using namespace strata;

extern "C" {

size_t strata_orthogonalise_workspace_bytes(int32_t n, int32_t N, int32_t K) {
    return check_orth(n, N, K) == STRATA_OK ? orth_plan(n, N, K).bytes : 0;
}

strata_status strata_orthogonalise(const void *G, strata_xdtype gdtype, int32_t n, int32_t N, int32_t K, int32_t steps,
                                   const float *coefficients, float scale, float eps, void *out, void *ws, size_t ws_bytes,
                                   void *stream) {
    if (bad_dtype(gdtype) || steps < 0 || steps > 32 || !coefficients || !std::isfinite(scale) || !(eps > 0.f) || !std::isfinite(eps))
        return STRATA_EINVAL;
    for (int i = 0; i < 3; ++i)
        if (!std::isfinite(coefficients[i])) return STRATA_EINVAL;
    const strata_status st = check_orth(n, N, K);
    if (st != STRATA_OK || n == 0) return st;
    if (bad_rows(G) || bad_rows(out) || bad_rows(ws)) return STRATA_EINVAL;
    const OrthPlan p = orth_plan(n, N, K);
    if (ws_bytes < p.bytes) return STRATA_EWORKSPACE;
    // Blocks read G while others may already store: only a matrix's own place is safe.
    const size_t values = (size_t)n * N * K;
    if (!(G == out && gdtype == STRATA_X_BF16) && overlap(G, values * (gdtype == STRATA_X_BF16 ? 2 : 4), out, values * 2))
        return STRATA_EINVAL;
    const hipStream_t s = (hipStream_t)stream;
    char *const w = (char *)ws;
    OrthArgs a{};
    a.G = G;
    a.out = (uint16_t *)out;
    a.norms = (double *)w;
    a.hi = (uint16_t *)(w + p.hi);
    a.next = (uint16_t *)(w + p.next);
    a.lo = (uint16_t *)(w + p.lo);
    a.A = (uint16_t *)(w + p.A);
    a.B = (uint16_t *)(w + p.B);
    a.dA = (float *)(w + p.dA);
    a.dB = (float *)(w + p.dB);
    a.n = n;
    a.N = N;
    a.K = K;
    a.side = p.side;
    a.ldx = p.ldx;
    a.lds = p.lds;
    const int64_t parts = ((int64_t)N * K + 16383) / 16384;
    a.parts = (int)(parts < ORTH_PARTS ? parts : ORTH_PARTS);
    a.size = exp2f(roundf(0.5f * log2f((float)(N > K ? N : K))));
    a.a = coefficients[0];
    a.b = coefficients[1];
    a.c = coefficients[2];
    // B = c (b/c A + A^2): a c too small beside b to show is made one that divides
    if (fabsf(a.c) < fabsf(a.b) * 0x1p-60f) a.c = a.b * 0x1p-60f;
    a.b_over_c = a.c != 0.f ? a.b / a.c : 0.f;
    a.scale = scale;
    a.eps = eps;
    const SmallShape k = small_shape(N, K);
    if (k != SMALL_NONE)
        return hip_status(gdtype == STRATA_X_BF16 ? orth_small<uint16_t>(a, steps, k, s) : orth_small<float>(a, steps, k, s));
    const bool tall = N > K;
    hipError_t e = gdtype == STRATA_X_BF16 ? orth_begin_width<uint16_t>(a, steps, s) : orth_begin_width<float>(a, steps, s);
    for (int i = 0; i < steps && e == hipSuccess; ++i) {
        const int left = steps - 1 - i;   // steps behind this one
        a.last = left == 0;
        a.lo_in = left > 0 || steps == 1;
        a.lo_out = left > 1;
        e = tall ? squares<0, 1>(a, s) : squares<0, 0>(a, s);
        if (e == hipSuccess) e = squares<1, 0>(a, s);
        if (e == hipSuccess) e = tall ? steps_of<1>(a, s) : steps_of<0>(a, s);
        uint16_t *const hi = a.hi;
        a.hi = a.next;
        a.next = hi;
    }
    return hip_status(e);
}

}  // extern "C"
