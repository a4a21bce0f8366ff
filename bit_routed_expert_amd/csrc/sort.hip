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
#include "sort_impl.hpp"

namespace strata {
namespace {

bool sort_args_ok(int32_t T, int32_t k, int32_t E) {
    return T >= 0 && k >= 1 && k <= 32 && E >= 1 && E <= SORT_E;
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
    a.counts = counts;
    a.offsets = offsets;
    a.perm = perm;
    a.pos = pos;
    a.bcnt = (int32_t *)ws;
    a.n = (int64_t)T * k;
    a.E = n_experts;
    sort_plan(a);
    return hip_status(launch_sort(a, PickKey{idx, aligned16(idx)}, (hipStream_t)stream));
}

}  // extern "C"
