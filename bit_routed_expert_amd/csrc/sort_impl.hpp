// Kernels of the stable counting sort (sort.hip), over a key that the caller
// names: what is sorted are the indices 0..n-1, key(i) is the id of the i-th
// (outside 0..E-1: dropped) and key.value(i) what perm holds for it.
#pragma once
#include "ops.hpp"

namespace strata {

constexpr int SORT_TH = 1024, SORT_WAVES = SORT_TH / 64, SORT_E = 1024;
constexpr int SORT_BLOCKS = 256;   // most blocks (rows of counts the second launch adds up)
constexpr int SORT_ONCE = 65535;     // picks that one 16-bit half of a counter holds
constexpr int SORT_CELLS = 8192;     // LDS counters: E times as many copies as fit, up to 32

struct SortArgs {
    int32_t *counts, *offsets, *perm, *pos;
    int32_t *bcnt;      // [blocks][E]
    int64_t n;
    int E, blocks, bits;
    int64_t chunk;      // picks per block, a multiple of SORT_TH
};

// The picks of a call: their ids as they lie in memory.
struct PickKey {
    static constexpr bool WIDE = true;   // 4 ids a load, where idx is aligned to them
    const int32_t *idx;
    int aligned;
    __device__ __forceinline__ int operator()(int64_t i) const { return idx[i]; }
    __device__ __forceinline__ int32_t value(int64_t i) const { return (int32_t)i; }
};

// Id of pick i, E for a dropped one or none.
template <typename Key> __device__ __forceinline__ int sort_key(const SortArgs &a, const Key &key, int64_t i) {
    const int e = i < a.n ? key(i) : -1;
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
template <typename Key>
__device__ __forceinline__ void sort_place(const SortArgs &a, const Key &key, int64_t i, int e, int *base, uint16_t (*whist)[SORT_E]) {
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
        if (a.perm) a.perm[s] = key.value(i);
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

// Chunks of 1024 picks (SORT_ONCE is less than SORT_BLOCKS of them): the work of block blockIdx.x of a.blocks.
template <typename Key> __device__ __forceinline__ void sort_once(const SortArgs &a, const Key &key, int copies) {
    __shared__ int base[SORT_E];
    __shared__ uint16_t whist[SORT_WAVES][SORT_E];
    __shared__ uint32_t cells[SORT_CELLS];
    __shared__ int wsum[SORT_WAVES];
    const int th = threadIdx.x, n = (int)a.n, i0 = (int)blockIdx.x * SORT_TH;
    const int own = sort_key(a, key, i0 + th);
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
    if constexpr (Key::WIDE) {
        if (key.aligned) {
            // 4 picks a load, 4 loads in flight; a load's picks lie in one chunk
            for (; c + 16 * SORT_TH <= n; c += 16 * SORT_TH) {
                int4 v[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = *(const int4 *)(key.idx + c + (q * SORT_TH + th) * 4);
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
    }
    for (; c < n; c += 8 * SORT_TH) {
        int v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = c + q * SORT_TH + th < n ? key(c + q * SORT_TH + th) : -1;
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
    sort_place(a, key, i0 + th, own, base, whist);
    if (a.perm && i0 + th < n && i0 + th >= kept) a.perm[i0 + th] = -1;
}

template <typename Key> __global__ __launch_bounds__(SORT_TH) void sort_once_kernel(SortArgs a, Key key, int copies) {
    sort_once(a, key, copies);
}

template <typename Key> __global__ __launch_bounds__(SORT_TH) void sort_count_kernel(SortArgs a, Key key) {
    __shared__ int hist[SORT_E];
    const int th = threadIdx.x;
    hist[th] = 0;
    __syncthreads();
    const int64_t i0 = (int64_t)blockIdx.x * a.chunk, i1 = min(i0 + a.chunk, a.n);
    for (int64_t i = i0 + th; i < i1; i += SORT_TH) {
        const int e = sort_key(a, key, i);
        if (e < a.E) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    if (th < a.E) a.bcnt[(int64_t)blockIdx.x * a.E + th] = hist[th];
}

template <typename Key> __global__ __launch_bounds__(SORT_TH) void sort_place_kernel(SortArgs a, Key key) {
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
    for (int64_t c = i0; c < i1; c += SORT_TH) sort_place(a, key, c + th, sort_key(a, key, c + th), base, whist);
    if (a.perm)
        for (int64_t s = i0 + th; s < i1; s += SORT_TH)
            if (s >= kept) a.perm[s] = -1;
}

inline void sort_plan(SortArgs &a) {
    const int64_t per = (a.n + SORT_BLOCKS - 1) / SORT_BLOCKS;
    a.chunk = per > SORT_TH ? (per + SORT_TH - 1) / SORT_TH * SORT_TH : SORT_TH;
    a.blocks = a.n ? (int)((a.n + a.chunk - 1) / a.chunk) : 1;   // without picks one block writes the zeros
    a.bits = 1;
    while ((a.E >> a.bits) != 0) ++a.bits;   // ids 0..E (E: dropped)
}

// Bytes of counts that a sort of a.n picks keeps between its launches.
inline size_t sort_counts_bytes(const SortArgs &a) { return a.n <= SORT_ONCE ? 0 : (size_t)a.blocks * a.E * 4; }

// Copies of the LDS counters for a sort in one launch.
inline int sort_copies(const SortArgs &a) {
    int copies = a.blocks > 4 ? 32 : a.blocks;   // fewer picks, fewer meetings
    while (copies * a.E > SORT_CELLS || (copies & (copies - 1))) --copies;
    return copies;
}

// The sort of a planned call.
template <typename Key> hipError_t launch_sort(const SortArgs &a, const Key &key, hipStream_t s) {
    if (a.n <= SORT_ONCE) {
        STRATA_LAUNCH(sort_once_kernel<Key>, dim3(a.blocks), dim3(SORT_TH), 0, s, a, key, sort_copies(a));
        return hipGetLastError();
    }
    STRATA_LAUNCH(sort_count_kernel<Key>, dim3(a.blocks), dim3(SORT_TH), 0, s, a, key);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    STRATA_LAUNCH(sort_place_kernel<Key>, dim3(a.blocks), dim3(SORT_TH), 0, s, a, key);
    return hipGetLastError();
}

}  // namespace strata
