// Row operators: a group of G threads takes one token's row, G a power of two
// up to 256.
#pragma once
#include "ops.hpp"

namespace strata {

// Token of this thread's group and its place in the group.
template <int G> __device__ __forceinline__ bool row_group(int T, int &t, int &lane) {
    t = (int)blockIdx.x * (256 / G) + (int)(threadIdx.x / G);
    if (G >= 64) t = __builtin_amdgcn_readfirstlane(t);
    lane = threadIdx.x % G;
    return t < T;
}

// Threads per token for nc pieces, and how many blocks share a token's row.
// Many tokens fill the chip by themselves: the largest group that leaves at
// most a quarter more threads idle than the best.  Few tokens: a thread per
// piece as far as a block goes, and the rest of the row to other blocks
// (combine of 7 tokens of 1927 values in 121 trips of 16 threads: 72 us, else
// 2.5).
struct RowGroups {
    int threads, shares;
};
constexpr int ROW_BLOCKS = 1024;   // blocks that fill the chip
inline RowGroups row_groups(int T, int64_t nc, int least) {
    int g = least;
    if (T >= ROW_BLOCKS) {
        int64_t best = INT64_MAX;
        for (int q = least; q <= 256; q *= 2) {
            const int64_t c = (nc + q - 1) / q * q;
            if (c < best) best = c;
        }
        for (int q = least; q <= 256; q *= 2)
            if ((nc + q - 1) / q * q * 4 <= best * 5) g = q;
    } else {
        while (g < 256 && g < nc) g *= 2;
    }
    const int64_t blocks = ((int64_t)T * g + 255) / 256, trips = (nc + g - 1) / g;
    const int64_t want = (ROW_BLOCKS + blocks - 1) / blocks;
    return RowGroups{g, (int)(want < trips ? want : trips)};
}

inline dim3 row_grid(int T, int g, int shares) {
    return dim3((unsigned)(((int64_t)T + 256 / g - 1) / (256 / g)), (unsigned)shares);
}

}  // namespace strata
