// Picks sorted by expert: a stable counting sort of the T*k expert ids.
//
// The slot of a pick is the number of kept picks of lower experts plus the
// number of earlier picks of its own: base[e] + rank.  A block takes the
// picks 1024 at a time, one per thread.  Inside a wave the lanes with the
// same id are found by one ballot per id bit (their rank is a popcount);
// across the block's 16 waves each wave leaves its count per id in LDS and
// every lane adds those of the waves before its own.  No sum depends on an
// order that could change: the LDS atomics only add whole numbers.
//
// What bounds it: launches and round trips, not bytes (12 bytes a pick).  Up
// to SORT_ONCE picks every block counts all of them by itself (from the L2,
// into LDS counters kept several times over so that lanes with equal ids meet
// less), those before its own chunk in the upper half of the same counters:
// one launch, no counts exchanged.  Above, a first launch counts each block's
// picks and the second adds up the counts of the blocks before it (327680 picks
// 17 us).  One launch against two, E = 512: 6000 picks 5.4 and 7.4 us, 20480
// picks 6.7 and 7.9, 40960 picks 8.0 and 8.2, 65530 picks 9.8 and 9.3; 40960
// picks of 16 experts 8.0 and 7.1: with many picks each block's count of all
// of them through LDS costs what the second launch does.  The border is where
// the 16-bit halves end, since two launches also cost the host a second one.
#include "ops.hpp"

namespace strata {

constexpr int SORT_TH = 1024, SORT_WAVES = SORT_TH / 64, SORT_E = 1024;
constexpr int SORT_BLOCKS = 256;   // most blocks (rows of counts the second launch adds up)
constexpr int SORT_ONCE = 65535;     // picks that one 16-bit half of a counter holds
constexpr int SORT_CELLS = 8192;     // LDS counters: E times as many copies as fit, up to 32

struct SortArgs {
    const int32_t *idx;
    int32_t *counts, *offsets, *perm, *pos;
    int32_t *bcnt;      // [blocks][E]
    int64_t n;
    int E, blocks, bits, aligned;
    int64_t chunk;      // picks per block, a multiple of SORT_TH
};

// Id of pick i, E for a dropped one or none.
__device__ __forceinline__ int sort_key(const SortArgs &a, int64_t i) {
    const int e = i < a.n ? a.idx[i] : -1;
    return (uint32_t)e < (uint32_t)a.E ? e : a.E;
}

// Exclusive prefix sum of one value per thread over the block (v of thread e
// for expert e), the total in *total.
__device__ __forceinline__ int block_exclusive(int v, int *wsum, int *total) {
    const int th = threadIdx.x, lane = th & 63, w = th >> 6;
    int s = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int q = __shfl_up(s, o, 64);
        if (lane >= o) s += q;
    }
    if (lane == 63) wsum[w] = s;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int q = 0; q < SORT_WAVES; ++q) {
        const int c = wsum[q];
        before += q < w ? c : 0;
        all += c;
    }
    *total = all;
    return before + s - v;
}

// Slots of up to 1024 picks, this thread's at i with id e (E: none or
// dropped), given base[e] = first slot of expert e's next pick; base
// advances.  whist is all zero on entry and on return.
__device__ __forceinline__ void sort_place(const SortArgs &a, int64_t i, int e, int *base, uint16_t (*whist)[SORT_E]) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    uint64_t same = ~0ull;
    for (int b = 0; b < a.bits; ++b) {
        const bool bit = (e >> b) & 1;
        const uint64_t m = __ballot(bit);
        same &= bit ? m : ~m;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    const bool kept = e < a.E, first = kept && rank == 0;
    const int mine = __popcll(same);
    if (first) whist[w][e] = (uint16_t)mine;
    __syncthreads();
    if (kept) {
        int s = base[e] + rank;
#pragma unroll
        for (int q = 0; q < SORT_WAVES - 1; ++q) s += q < w ? (int)whist[q][e] : 0;
        if (a.pos) a.pos[i] = s;
        if (a.perm) a.perm[s] = (int32_t)i;
    } else if (i < a.n && a.pos) {
        a.pos[i] = -1;
    }
    __syncthreads();
    if (first) {
        atomicAdd(&base[e], mine);
        whist[w][e] = 0;
    }
    __syncthreads();
}

__device__ __forceinline__ void clear_whist(uint16_t (*whist)[SORT_E]) {
    uint32_t *p = (uint32_t *)whist;
#pragma unroll
    for (int q = 0; q < SORT_WAVES * SORT_E / 2 / SORT_TH; ++q) p[q * SORT_TH + threadIdx.x] = 0;
}

// First slots from the counts of this thread's expert: `mine` picks in all,
// `before` of them in earlier chunks; returns the kept picks.
__device__ __forceinline__ int sort_bases(const SortArgs &a, int mine, int before, int *base, int *wsum) {
    const int th = threadIdx.x;
    int kept;
    const int ex = block_exclusive(mine, wsum, &kept);
    base[th] = ex + before;
    if (blockIdx.x == 0) {
        if (th < a.E) {
            if (a.counts) a.counts[th] = mine;
            if (a.offsets) a.offsets[th] = ex;
        }
        if (th == 0 && a.offsets) a.offsets[a.E] = kept;
    }
    __syncthreads();
    return kept;
}

// Chunks of 1024 picks (SORT_ONCE is less than SORT_BLOCKS of them).
__global__ __launch_bounds__(SORT_TH) void sort_once_kernel(SortArgs a, int copies) {
    __shared__ int base[SORT_E];
    __shared__ uint16_t whist[SORT_WAVES][SORT_E];
    __shared__ uint32_t cells[SORT_CELLS];
    __shared__ int wsum[SORT_WAVES];
    const int th = threadIdx.x, n = (int)a.n, i0 = (int)blockIdx.x * SORT_TH;
    const int own = sort_key(a, i0 + th);
    clear_whist(whist);
    for (int q = th; q < copies * a.E; q += SORT_TH) cells[q] = 0;
    __syncthreads();
    uint32_t *mine = cells + (th & (copies - 1)) * a.E;   // a copy's cells lie together: lanes read them without conflicts
    const auto count = [&](int e, int i) {
        if ((uint32_t)e < (uint32_t)a.E) atomicAdd(&mine[e], i < i0 ? 0x10001u : 1u);
    };
    int c = 0;
    if (a.blocks == 1) {
        count(own, th);
        c = n;
    }
    if (a.aligned) {
        // 4 picks a load, 4 loads in flight; a load's picks lie in one chunk
        for (; c + 16 * SORT_TH <= n; c += 16 * SORT_TH) {
            int4 v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = *(const int4 *)(a.idx + c + (q * SORT_TH + th) * 4);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = c + (q * SORT_TH + th) * 4;
                count(v[q].x, i);
                count(v[q].y, i);
                count(v[q].z, i);
                count(v[q].w, i);
            }
        }
    }
    for (; c < n; c += 8 * SORT_TH) {
        int v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = c + q * SORT_TH + th < n ? a.idx[c + q * SORT_TH + th] : -1;
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (c + q * SORT_TH < n) count(v[q], c + q * SORT_TH + th);
    }
    __syncthreads();
    uint32_t sum = 0;
    if (th < a.E) {
#pragma unroll 8
        for (int q = 0; q < copies; ++q) sum += cells[q * a.E + th];
    }
    const int kept = sort_bases(a, (int)(sum & 0xFFFFu), (int)(sum >> 16), base, wsum);
    sort_place(a, i0 + th, own, base, whist);
    if (a.perm && i0 + th < n && i0 + th >= kept) a.perm[i0 + th] = -1;
}

__global__ __launch_bounds__(SORT_TH) void sort_count_kernel(SortArgs a) {
    __shared__ int hist[SORT_E];
    const int th = threadIdx.x;
    hist[th] = 0;
    __syncthreads();
    const int64_t i0 = (int64_t)blockIdx.x * a.chunk, i1 = min(i0 + a.chunk, a.n);
    for (int64_t i = i0 + th; i < i1; i += SORT_TH) {
        const int e = sort_key(a, i);
        if (e < a.E) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    if (th < a.E) a.bcnt[(int64_t)blockIdx.x * a.E + th] = hist[th];
}

__global__ __launch_bounds__(SORT_TH) void sort_place_kernel(SortArgs a) {
    __shared__ int base[SORT_E];
    __shared__ uint16_t whist[SORT_WAVES][SORT_E];
    __shared__ int wsum[SORT_WAVES];
    const int th = threadIdx.x, blk = blockIdx.x;
    clear_whist(whist);
    int before = 0, mine = 0;
    if (th < a.E) {
#pragma unroll 8
        for (int b = 0; b < a.blocks; ++b) {
            const int c = a.bcnt[(int64_t)b * a.E + th];
            before += b < blk ? c : 0;
            mine += c;
        }
    }
    const int kept = sort_bases(a, mine, before, base, wsum);
    const int64_t i0 = (int64_t)blk * a.chunk, i1 = min(i0 + a.chunk, a.n);
    for (int64_t c = i0; c < i1; c += SORT_TH) sort_place(a, c + th, sort_key(a, c + th), base, whist);
    if (a.perm)
        for (int64_t s = i0 + th; s < i1; s += SORT_TH)
            if (s >= kept) a.perm[s] = -1;
}

namespace {

bool sort_args_ok(int32_t T, int32_t k, int32_t E) {
    return T >= 0 && k >= 1 && k <= 32 && E >= 1 && E <= SORT_E;
}

void sort_plan(SortArgs &a) {
    const int64_t per = (a.n + SORT_BLOCKS - 1) / SORT_BLOCKS;
    a.chunk = per > SORT_TH ? (per + SORT_TH - 1) / SORT_TH * SORT_TH : SORT_TH;
    a.blocks = a.n ? (int)((a.n + a.chunk - 1) / a.chunk) : 1;   // without picks one block writes the zeros
    a.bits = 1;
    while ((a.E >> a.bits) != 0) ++a.bits;   // ids 0..E (E: dropped)
}

}  // namespace

}  // namespace strata

using namespace strata;

extern "C" {

size_t strata_moe_sort_workspace_bytes(int32_t T, int32_t k, int32_t n_experts) {
    if (!sort_args_ok(T, k, n_experts) || (int64_t)T * k > INT32_MAX) return 0;
    SortArgs a{};
    a.n = (int64_t)T * k;
    a.E = n_experts;
    sort_plan(a);
    return a.n <= SORT_ONCE ? 256 : (size_t)a.blocks * n_experts * 4;
}

strata_status strata_moe_sort(const int32_t *idx, int32_t T, int32_t k, int32_t n_experts, int32_t *counts,
                              int32_t *offsets, int32_t *perm, int32_t *pos, void *ws, size_t ws_bytes,
                              void *stream) {
    if (!sort_args_ok(T, k, n_experts)) return STRATA_EINVAL;
    if ((int64_t)T * k > INT32_MAX) return STRATA_EUNSUPPORTED;
    if (T > 0 && (!idx || !ws || !aligned16(ws))) return STRATA_EINVAL;
    if (T > 0 && ws_bytes < strata_moe_sort_workspace_bytes(T, k, n_experts)) return STRATA_EWORKSPACE;
    // Blocks read the picks (and, in two launches, each other's counts) while others write: slots from counts that
    // changed in between could lie outside perm.
    const size_t n = (size_t)T * k * 4;
    const size_t used = (int64_t)T * k > SORT_ONCE ? strata_moe_sort_workspace_bytes(T, k, n_experts) : 0;
    const struct {
        const void *p;
        size_t bytes;
    } outs[] = {{counts, (size_t)n_experts * 4}, {offsets, (size_t)(n_experts + 1) * 4}, {perm, n}, {pos, n}};
    for (const auto &o : outs)
        if (overlap(o.p, o.bytes, idx, n) || overlap(o.p, o.bytes, ws, used)) return STRATA_EINVAL;
    if (overlap(ws, used, idx, n)) return STRATA_EINVAL;
    SortArgs a{};
    a.idx = idx;
    a.counts = counts;
    a.offsets = offsets;
    a.perm = perm;
    a.pos = pos;
    a.bcnt = (int32_t *)ws;
    a.aligned = aligned16(idx);
    a.n = (int64_t)T * k;
    a.E = n_experts;
    sort_plan(a);
    const hipStream_t s = (hipStream_t)stream;
    if (a.n <= SORT_ONCE) {
        int copies = a.blocks > 4 ? 32 : a.blocks;   // fewer picks, fewer meetings
        while (copies * a.E > SORT_CELLS || (copies & (copies - 1))) --copies;
        STRATA_LAUNCH(sort_once_kernel, dim3(a.blocks), dim3(SORT_TH), 0, s, a, copies);
        return hip_status(hipGetLastError());
    }
    STRATA_LAUNCH(sort_count_kernel, dim3(a.blocks), dim3(SORT_TH), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return hip_status(e);
    STRATA_LAUNCH(sort_place_kernel, dim3(a.blocks), dim3(SORT_TH), 0, s, a);
    return hip_status(hipGetLastError());
}

}  // extern "C"
