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
// What bounds it: launch and round trips, not bytes (12 bytes a pick).  Up
// to ONE_BLOCK picks one block does everything in one launch.  Above that a
// first launch counts each block's picks per expert and a second one adds up
// the counts of the blocks before it by itself, so no third launch scans.
#include "ops.hpp"

namespace strata {

constexpr int SORT_TH = 1024, SORT_WAVES = SORT_TH / 64, SORT_E = 1024;
constexpr int SORT_BLOCKS = 256;   // most blocks (rows of counts the second launch adds up)
constexpr int ONE_BLOCK = 4096;

struct SortArgs {
    const int32_t *idx;
    int32_t *counts, *offsets, *perm, *pos;
    int32_t *bcnt;      // [blocks][E]
    int64_t n;
    int E, blocks, bits;
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

// Slots of the picks [i0, i1) given base[e] = first slot of expert e's next
// pick; base advances.  whist is all zero on entry and on return.
__device__ void sort_place(const SortArgs &a, int64_t i0, int64_t i1, int *base, uint16_t (*whist)[SORT_E]) {
    const int th = threadIdx.x, lane = th & 63, w = th >> 6;
    for (int64_t c = i0; c < i1; c += SORT_TH) {
        const int64_t i = c + th;
        const int e = i < i1 ? sort_key(a, i) : a.E;
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
        } else if (i < i1 && a.pos) {
            a.pos[i] = -1;
        }
        __syncthreads();
        if (first) {
            atomicAdd(&base[e], mine);
            whist[w][e] = 0;
        }
        __syncthreads();
    }
}

__device__ __forceinline__ void clear_whist(uint16_t (*whist)[SORT_E]) {
    uint32_t *p = (uint32_t *)whist;
#pragma unroll
    for (int q = 0; q < SORT_WAVES * SORT_E / 2 / SORT_TH; ++q) p[q * SORT_TH + threadIdx.x] = 0;
}

__global__ __launch_bounds__(SORT_TH) void sort_one_kernel(SortArgs a) {
    __shared__ int base[SORT_E];
    __shared__ uint16_t whist[SORT_WAVES][SORT_E];
    __shared__ int wsum[SORT_WAVES];
    const int th = threadIdx.x;
    base[th] = 0;
    clear_whist(whist);
    __syncthreads();
    for (int64_t i = th; i < a.n; i += SORT_TH) {
        const int e = sort_key(a, i);
        if (e < a.E) atomicAdd(&base[e], 1);
    }
    __syncthreads();
    const int mine = base[th];
    int kept;
    const int ex = block_exclusive(mine, wsum, &kept);
    base[th] = ex;
    if (th < a.E) {
        if (a.counts) a.counts[th] = mine;
        if (a.offsets) a.offsets[th] = ex;
    }
    if (th == 0 && a.offsets) a.offsets[a.E] = kept;
    __syncthreads();
    sort_place(a, 0, a.n, base, whist);
    if (a.perm)
        for (int64_t s = kept + th; s < a.n; s += SORT_TH) a.perm[s] = -1;
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
    int kept;
    const int ex = block_exclusive(mine, wsum, &kept);
    base[th] = ex + before;
    if (blk == 0) {
        if (th < a.E) {
            if (a.counts) a.counts[th] = mine;
            if (a.offsets) a.offsets[th] = ex;
        }
        if (th == 0 && a.offsets) a.offsets[a.E] = kept;
    }
    __syncthreads();
    const int64_t i0 = (int64_t)blk * a.chunk, i1 = min(i0 + a.chunk, a.n);
    sort_place(a, i0, i1, base, whist);
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
    a.chunk = (per + SORT_TH - 1) / SORT_TH * SORT_TH;
    a.blocks = a.chunk ? (int)((a.n + a.chunk - 1) / a.chunk) : 0;
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
    return a.n <= ONE_BLOCK ? 256 : (size_t)a.blocks * n_experts * 4;
}

strata_status strata_moe_sort(const int32_t *idx, int32_t T, int32_t k, int32_t n_experts, int32_t *counts,
                              int32_t *offsets, int32_t *perm, int32_t *pos, void *ws, size_t ws_bytes,
                              void *stream) {
    if (!sort_args_ok(T, k, n_experts)) return STRATA_EINVAL;
    if ((int64_t)T * k > INT32_MAX) return STRATA_EUNSUPPORTED;
    if (T > 0 && (!idx || !ws || !aligned16(ws))) return STRATA_EINVAL;
    if (T > 0 && ws_bytes < strata_moe_sort_workspace_bytes(T, k, n_experts)) return STRATA_EWORKSPACE;
    SortArgs a{};
    a.idx = idx;
    a.counts = counts;
    a.offsets = offsets;
    a.perm = perm;
    a.pos = pos;
    a.bcnt = (int32_t *)ws;
    a.n = (int64_t)T * k;
    a.E = n_experts;
    sort_plan(a);
    const hipStream_t s = (hipStream_t)stream;
    if (a.n <= ONE_BLOCK) {
        STRATA_LAUNCH(sort_one_kernel, dim3(1), dim3(SORT_TH), 0, s, a);
        return hip_status(hipGetLastError());
    }
    STRATA_LAUNCH(sort_count_kernel, dim3(a.blocks), dim3(SORT_TH), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return hip_status(e);
    STRATA_LAUNCH(sort_place_kernel, dim3(a.blocks), dim3(SORT_TH), 0, s, a);
    return hip_status(hipGetLastError());
}

}  // extern "C"
