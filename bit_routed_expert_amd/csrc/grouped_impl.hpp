// Tile products of the experts' grouped products on the gfx950 matrix cores.
//
// One block computes a tile C[BM][BN] = sum_c A[m][c] B[n][c] of one expert.
// The contraction is cut into steps of C = 64 or 32; a step's tiles of A and B
// come into LDS by direct global->LDS loads (16 bytes a lane, no registers)
// while earlier steps run on the matrix cores: 2 to 4 buffers in turn, one
// barrier a step, met while the matrix cores still have the step's last 16 of
// the contraction ahead of them.
//
// An operand whose contraction runs along memory (x and W in the product)
// lies in LDS as it does in memory, 64 values (128 bytes) to a row; a lane's
// 8 values of a 32x32x16 product are one 16-byte read, and the row's chunks
// are permuted by the row number so that 32 rows' reads meet no bank twice.
// An operand whose contraction runs across memory (W in dgrad, both in wgrad)
// lies as C rows of BM or BN values; the transposing LDS reads of gfx950
// (four 16-bit rows of 16 columns per 16 lanes) hand each lane 4 values down
// a column, two of them make its 8.  There the 64-byte pieces of a row are
// permuted by the low two bits of the row number, so the four rows of a read
// lie in different banks.
//
// What lies outside an operand reads as zero by the range check of its
// buffer resource: rows behind the expert's last one, and the contraction
// behind its end (pushed out of range by hand where memory goes on there).
#pragma once
#include "ops.hpp"

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

// Permutation of the 16-byte chunks of staged row c (R values, a power of two
// of at least 64), across: the 64-byte pieces by the low bits of c.
template <int R> __device__ __forceinline__ int across_swz(int c) { return ((c & 3) << 2) & (R / 8 - 1); }

// The same of row r of an operand that lies along: 8 chunks.
__device__ __forceinline__ int along_swz(int r) { return (r ^ (r >> 3)) & 7; }

// One operand: R rows of it in the tile (m or n), NT threads stage C of the contraction.
template <int R, int ACROSS, int NT, int C> struct Operand {
    static constexpr int BYTES = R * C * 2, CH = C / 8, LOADS = R * CH / NT;
    static_assert(LOADS * NT == R * CH, "whole chunks per thread");
    static_assert(ACROSS || C == 64, "along_swz is for rows of 128 bytes");
    const uint16_t *base;       // along: first row's first value; across: first contraction row
    int ld, count, cd;          // row length in memory, rows of the tile in range (along), contraction
    uint32_t off[LOADS];        // byte offset of this thread's chunks at step 0

    // p: the operand's first value; tile rows r0.. of `total`.
    __device__ __forceinline__ void init(const uint16_t *p, int ld_, int r0, int total, int cd_) {
        ld = ld_;
        cd = cd_;
        count = ACROSS ? 0 : min(total - r0, R);
        base = ACROSS ? p : p + (int64_t)r0 * ld;
        const int th = threadIdx.x;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int q = i * NT + th;
            if (ACROSS) {
                const int c = q / (R / 8), at = q % (R / 8);
                off[i] = (uint32_t)c * (uint32_t)ld * 2u + (uint32_t)(r0 + 8 * (at ^ across_swz<R>(c))) * 2u;
            } else {
                const int r = q / CH, at = q % CH;
                off[i] = (uint32_t)r * (uint32_t)ld * 2u + (uint32_t)(8 * (at ^ along_swz(r))) * 2u;
            }
        }
    }

    __device__ __forceinline__ void load(int s, uint8_t *dst) const {
        const int th = threadIdx.x, wv = __builtin_amdgcn_readfirstlane(th >> 6);
        const int left = max(cd - s * C, 0);   // contraction from this step on (0: a load behind the end, all zeros)
        const uint16_t *p = ACROSS ? base + (int64_t)s * C * ld : base + (int64_t)s * C;
        const uint32_t bytes = ACROSS ? (uint32_t)min(left, C) * (uint32_t)ld * 2u
                                      : left ? ((uint32_t)(count - 1) * (uint32_t)ld + (uint32_t)left) * 2u : 0u;
        // the size in a scalar register whatever unit computed it: a resource in vector registers makes
        // every load a loop over the lanes
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint16_t *>(p), 0, __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            uint32_t o = off[i];
            if (!ACROSS && left < C) {   // a last short step: chunks behind the end
                const int q = i * NT + th;
                if (8 * ((q % CH) ^ along_swz(q / CH)) >= left) o = 0x80000000u;
            }
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                r, (__attribute__((address_space(3))) void *)(dst + (i * NT + wv * 64) * 16), 16, o, 0, 0, 0);
        }
    }
};

// The 8 values a lane feeds to one 32x32x16 product: tile rows r0 + lane%32,
// contraction 16 kk + 8 (lane/32) .. +8 of the staged step.
typedef short s16x4_t __attribute__((ext_vector_type(4)));
template <int R, int ACROSS, int C>
__device__ __forceinline__ bf16x8_t read_frag(const uint8_t *t, int r0, int kk) {
    const int lane = threadIdx.x & 63;
    if constexpr (!ACROSS) {
        const int r = r0 + (lane & 31), c = 2 * kk + (lane >> 5);
        return __builtin_bit_cast(bf16x8_t, *(const u32x4_t *)(t + (r * C * 2 + 16 * (c ^ along_swz(r)))));
    } else {
        const int i = lane & 15, g = lane >> 4;
        const int c = 16 * kk + 8 * (g >> 1) + (i >> 2);   // second read: c + 4, the same low bits
        const int chunk = (r0 >> 3) + 2 * (g & 1) + ((i >> 1) & 1);
        const int p = c * (R * 2) + 16 * (chunk ^ across_swz<R>(c)) + 8 * (i & 1);
        typedef __attribute__((address_space(3))) s16x4_t lds4;
        const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(t + p));
        const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(t + (p + 4 * R * 2)));
        return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
}

// All loads but the newest N done, this wave's LDS reads done, then the block's barrier.
template <int N> __device__ __forceinline__ void wait_and_meet() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | 0x70 | ((N >> 4) << 14));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// What a wave feeds to 16 of the contraction on its MT x NT2 subtiles of
// 32x32, twice: the next 16 are read while the current 16 are multiplied.
template <int MT, int NT2> struct Frags {
    bf16x8_t a[2][MT], b[2][NT2];
};
template <int BM, int BN, int C, int MT, int NT2, int TA, int TB>
__device__ __forceinline__ void read_frags(const uint8_t *ta, const uint8_t *tb, int m0,
                                           int n0, int kk, int set, Frags<MT, NT2> &f) {
#pragma unroll
    for (int j = 0; j < NT2; ++j) f.b[set][j] = read_frag<BN, TB, C>(tb, n0 + 32 * j, kk);
#pragma unroll
    for (int i = 0; i < MT; ++i) f.a[set][i] = read_frag<BM, TA, C>(ta, m0 + 32 * i, kk);
}

// Step s, whose first 16 are in set 0 of f already; leaves the next step's
// there.  Ahead of the step's last products every wave has read all of the
// step's buffers and the next step's loads are done: the barrier stands there,
// so its wait and the next step's first LDS reads hide behind products, and
// A's buffer is loaded again right behind it (step s + ST), B's at the start of
// the step after it.  Against a barrier at the start of a step (1536 x 2048):
// 32768 rows of 16 uneven experts, product 220 -> 212 us, dgrad 220 -> 215 us,
// wgrad 226 -> 208 us; 40960 rows of 512 experts, product 680 -> 666 us; 512
// experts of 16 rows, wgrad 740 -> 677 us.
// The scheduling barrier keeps the compiler from reading the whole step ahead,
// which costs more registers than the accumulators leave.  WAIT: a wave's loads
// that may still be under way at the barrier.  TAIL 1: no more steps to load
// but B's last; 2: none.  A wave that is not ACTIVE has no rows and only stages.
template <int ST, int BM, int BN, int C, int MT, int NT2, int TA, int TB, int WAIT, int TAIL, bool ACTIVE, typename OA,
          typename OB>
__device__ __forceinline__ void step_product(const OA &A, const OB &B, int s, int steps, uint8_t *ta, const uint8_t *tb,
                                             const uint8_t *na, const uint8_t *nb, uint8_t *wb, int m0, int n0,
                                             f32x16_t (&acc)[MT][NT2], Frags<MT, NT2> &f) {
    constexpr int KS = C / 16;
    const bool more = !TAIL || s + 1 < steps;
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
        __builtin_amdgcn_sched_barrier(0);
        if (ACTIVE && kk + 1 < KS) read_frags<BM, BN, C, MT, NT2, TA, TB>(ta, tb, m0, n0, kk + 1, (kk + 1) & 1, f);
        if (kk == 0 && TAIL < 2) B.load(s + ST - 1, wb);
        if (kk + 1 == KS && more) {
            wait_and_meet<WAIT>();
            if (ACTIVE) read_frags<BM, BN, C, MT, NT2, TA, TB>(na, nb, m0, n0, 0, 0, f);
            if (!TAIL) A.load(s + ST, ta);
        }
        if (ACTIVE) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT2; ++j) acc[i][j] = mfma(f.b[kk & 1][j], f.a[kk & 1][i], acc[i][j]);
        }
    }
}

// The contraction with ST buffers: step s is multiplied while the ST - 1
// behind it come in.  Loads behind the end fetch nothing and keep the count of
// loads in flight the same.  The compiler waits for a direct load ahead of an
// LDS read that it cannot tell from the load's target, which would undo the
// buffering: it can where both are the kernel's own distinct arrays, no
// pointer here is restrict (those scopes would hide the arrays'), reads are
// one addition away from their array, and the loop has one exit.
template <int ST, bool ACTIVE, int BM, int BN, int C, int MT, int NT2, int TA, int TB, typename OA, typename OB>
__device__ __forceinline__ void contract(const OA &A, const OB &B, uint8_t *a0, uint8_t *b0, uint8_t *a1, uint8_t *b1,
                                         uint8_t *a2, uint8_t *b2, uint8_t *a3, uint8_t *b3, int steps, int m0, int n0,
                                         f32x16_t (&acc)[MT][NT2]) {
    constexpr int L = OA::LOADS + OB::LOADS;   // a wave's loads per step
    constexpr int W = (ST - 2) * L;
    if (steps == 0) return;
    Frags<MT, NT2> f;
#define STEP(S, WAIT, TAIL, AR, BR, AN, BN_, BP) \
    step_product<ST, BM, BN, C, MT, NT2, TA, TB, WAIT, TAIL, ACTIVE>(A, B, S, steps, AR, BR, AN, BN_, BP, m0, n0, acc, f);
    A.load(0, a0);
    B.load(0, b0);
    if (steps == 1) {   // on its own: nothing to wait for but its loads
        wait_and_meet<0>();
        if (!ACTIVE) return;
#pragma unroll
        for (int kk = 0; kk < C / 16; ++kk) {
            read_frags<BM, BN, C, MT, NT2, TA, TB>(a0, b0, m0, n0, kk, 0, f);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT2; ++j) acc[i][j] = mfma(f.b[0][j], f.a[0][i], acc[i][j]);
        }
        return;
    }
    A.load(1, a1);
    if constexpr (ST > 2) {
        B.load(1, b1);
        A.load(2, a2);
    }
    if constexpr (ST > 3) {
        B.load(2, b2);
        A.load(3, a3);
    }
    wait_and_meet<W + OA::LOADS>();
    if (ACTIVE) read_frags<BM, BN, C, MT, NT2, TA, TB>(a0, b0, m0, n0, 0, 0, f);
    int s = 0;
    for (; s + ST < steps; s += ST) {
        if constexpr (ST == 2) {
            STEP(s, W, 0, a0, b0, a1, b1, b1)
            STEP(s + 1, W, 0, a1, b1, a0, b0, b0)
        } else if constexpr (ST == 3) {
            STEP(s, W, 0, a0, b0, a1, b1, b2)
            STEP(s + 1, W, 0, a1, b1, a2, b2, b0)
            STEP(s + 2, W, 0, a2, b2, a0, b0, b1)
        } else {
            STEP(s, W, 0, a0, b0, a1, b1, b3)
            STEP(s + 1, W, 0, a1, b1, a2, b2, b0)
            STEP(s + 2, W, 0, a2, b2, a3, b3, b1)
            STEP(s + 3, W, 0, a3, b3, a0, b0, b2)
        }
    }
    // the last one to ST steps; B of the last is the only load not issued yet
    if constexpr (ST == 2) STEP(s, W, 1, a0, b0, a1, b1, b1)
    else if constexpr (ST == 3) STEP(s, W, 1, a0, b0, a1, b1, b2)
    else STEP(s, W, 1, a0, b0, a1, b1, b3)
    if (s + 1 < steps) {
        constexpr int W1 = ST > 3 ? (ST - 3) * L : 0;
        if constexpr (ST == 2) STEP(s + 1, 0, 2, a1, b1, a0, b0, b0)
        else STEP(s + 1, W1, 2, a1, b1, a2, b2, b0)
    }
    if (ST > 2 && s + 2 < steps) STEP(s + 2, 0, 2, a2, b2, ST > 3 ? a3 : a0, ST > 3 ? b3 : b0, b1)
    if (ST > 3 && s + 3 < steps) STEP(s + 3, 0, 2, a3, b3, a0, b0, b2)
#undef STEP
    __builtin_amdgcn_s_waitcnt(0x0F70);   // no load outlives the block
}

// The ST buffers of a block's two operands.
#define GROUP_BUFFERS(ST, OA, OB)                                                                             \
    __shared__ __attribute__((aligned(128))) uint8_t a0[OA::BYTES], a1[OA::BYTES], b0[OB::BYTES], b1[OB::BYTES]; \
    __shared__ __attribute__((aligned(128))) uint8_t a2[ST > 2 ? OA::BYTES : 16], b2[ST > 2 ? OB::BYTES : 16],   \
        a3[ST > 3 ? OA::BYTES : 16], b3[ST > 3 ? OB::BYTES : 16];

// The wave's subtiles to C (row length Nn): tile rows m0.. of `M`, columns
// n0.. < Nn, C at the tile's first row.  B's fragments are the products'
// first operand, so a lane holds one row, columns 8 (v/4) + 4 (lane/32) + v%4
// of each subtile: 16-byte stores of fp32 as they are, of bf16 after the two
// halves of the wave have exchanged every other group of four.  Rows and
// columns outside the tile fall outside the buffer resource.
template <int MT, int NT2>
__device__ __forceinline__ void store_tile(void *C, int c_bf16, int m0, int M, int n0, int Nn,
                                           const f32x16_t (&acc)[MT][NT2]) {
    const int lane = threadIdx.x & 63, l = lane & 31, h = lane >> 5;
    const uint32_t esz = c_bf16 ? 2 : 4;
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(C, 0, (int)((uint32_t)M * (uint32_t)Nn * esz), 0x00020000);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const uint32_t row = (uint32_t)(m0 + 32 * i + l) * (uint32_t)Nn;
#pragma unroll
        for (int j = 0; j < NT2; ++j) {
            const f32x16_t &v = acc[i][j];
            if (c_bf16) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    // groups 2q and 2q+1 (4 values = 2 words each): after the swap words of 8 columns in a row
                    const auto s0 = __builtin_amdgcn_permlane32_swap(bf16_pair(v[8 * q], v[8 * q + 1]),
                                                                     bf16_pair(v[8 * q + 4], v[8 * q + 5]), false, false);
                    const auto s1 = __builtin_amdgcn_permlane32_swap(bf16_pair(v[8 * q + 2], v[8 * q + 3]),
                                                                     bf16_pair(v[8 * q + 6], v[8 * q + 7]), false, false);
                    const int n = n0 + 32 * j + 16 * q + 8 * h;
                    const uint32_t at = n < Nn ? (row + n) * 2u : 0xFFFFFFF0u;
                    __builtin_amdgcn_raw_buffer_store_b128(u32x4_t{s0[0], s1[0], s0[1], s1[1]}, r, at, 0, 0);
                }
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int n = n0 + 32 * j + 8 * q + 4 * h;
                    const uint32_t at = n < Nn ? (row + n) * 4u : 0xFFFFFFF0u;
                    __builtin_amdgcn_raw_buffer_store_b128(
                        __builtin_bit_cast(u32x4_t, f32x4_t{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]}), r, at, 0, 0);
                }
            }
        }
    }
}

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

// This wave's first row and column in the tile.  Waves go to the 4 SIMDs in
// turn; with 2 x 4 of them the second row of waves is turned by two, so that a
// tile with rows for half of them, or columns for one or two of the four,
// still keeps as many SIMDs busy as it has waves.  32768 rows of 16 experts,
// 1288 x 1288, the last tiles 8 wide, with waves outside them idle: product 128
// -> 121 us, wgrad 152 -> 130 us.
template <int WM, int WN, int MT, int NT2> __device__ __forceinline__ void wave_place(int &m0, int &n0) {
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), m = wv / WN;
    m0 = m * 32 * MT;
    n0 = (WM == 2 && WN == 4 ? (wv % WN) ^ (2 * m) : wv % WN) * 32 * NT2;
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
