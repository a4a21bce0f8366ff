// C entry points of the norms around a block: validation, the choice of the
// instantiation in block_norm_{f,h}{f,h}{f,h}.hip (types of x, y, u) and the
// sum of the gains' gradients.
#include <math.h>

#include "block_norm_impl.hpp"

namespace strata {

extern template hipError_t block_norm_launch<float, float, float>(const NormArgs &, bool, hipStream_t);
extern template hipError_t block_norm_launch<uint16_t, float, float>(const NormArgs &, bool, hipStream_t);
extern template hipError_t block_norm_launch<float, uint16_t, float>(const NormArgs &, bool, hipStream_t);
extern template hipError_t block_norm_launch<uint16_t, uint16_t, float>(const NormArgs &, bool, hipStream_t);
extern template hipError_t block_norm_launch<float, float, uint16_t>(const NormArgs &, bool, hipStream_t);
extern template hipError_t block_norm_launch<uint16_t, float, uint16_t>(const NormArgs &, bool, hipStream_t);
extern template hipError_t block_norm_launch<float, uint16_t, uint16_t>(const NormArgs &, bool, hipStream_t);
extern template hipError_t block_norm_launch<uint16_t, uint16_t, uint16_t>(const NormArgs &, bool, hipStream_t);
extern template hipError_t block_norm_launch_any<2>(const NormArgs &, bool, hipStream_t);
extern template hipError_t block_norm_launch_any<1>(const NormArgs &, bool, hipStream_t);

// Gain gradients from the blocks' partial sums, added in block order: 32
// columns per block, 32 threads' worth of blocks side by side for each.
__global__ __launch_bounds__(1024) void block_norm_gains_kernel(NormArgs a) {
    __shared__ float s[32][33];
    const float *part = blockIdx.y ? a.part_pre : a.part_post;
    float *out = blockIdx.y ? a.dg_pre : a.dg_post;
    if (!out) return;
    const int c = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + c;
    float v = 0.f;
    if (i < a.d) {
#pragma unroll 4
        for (int b = q; b < a.blocks; b += 32) v += part[(int64_t)b * a.d + i];
    }
    s[q][c] = v;
    __syncthreads();
    if (threadIdx.x < 32 && blockIdx.x * 32 + threadIdx.x < a.d) {
        float t = 0.f;
#pragma unroll
        for (int b = 0; b < 32; ++b) t += s[b][threadIdx.x];
        out[blockIdx.x * 32 + threadIdx.x] = t;
    }
}

namespace {

strata_status check_norm(const strata_block_norm_args *p) {
    if (!p || p->T < 0 || p->d < 1) return STRATA_EINVAL;
    if (bad_dtype(p->x_dtype) || bad_dtype(p->y_dtype) || bad_dtype(p->u_dtype)) return STRATA_EINVAL;
    const uint32_t f = p->flags;
    if (f & ~31u) return STRATA_EINVAL;
    const bool tok = f & STRATA_GATE_TOKEN, chan = f & STRATA_GATE_CHANNEL;
    if ((tok && chan) || ((f & STRATA_GATE_SIGMOID) && !tok && !chan)) return STRATA_EINVAL;
    if (!(p->eps > 0.f) || !isfinite(p->eps) || !isfinite(p->resid_scale) || !isfinite(p->branch_scale))
        return STRATA_EINVAL;
    if (p->d > BN_MAX_D || p->T > MAX_ROWS) return STRATA_EUNSUPPORTED;
    return STRATA_OK;
}

// What the flags ask for and what is given have to agree.
strata_status check_norm_inputs(const strata_block_norm_args *p, const void *y, const void *gate, const float *g_post,
                                const float *g_pre) {
    const bool gated = p->flags & (STRATA_GATE_TOKEN | STRATA_GATE_CHANNEL);
    if (!y && (gated || (p->flags & STRATA_POST_NORM))) return STRATA_EINVAL;
    if (gated != (gate != nullptr)) return STRATA_EINVAL;
    if (g_post && !(p->flags & STRATA_POST_NORM)) return STRATA_EINVAL;
    if (g_pre && !(p->flags & STRATA_PRE_NORM)) return STRATA_EINVAL;
    return STRATA_OK;
}

NormArgs norm_args(const strata_block_norm_args *p) {
    NormArgs a{};
    a.T = p->T;
    a.d = p->d;
    a.x_bf16 = p->x_dtype == STRATA_X_BF16;
    a.y_bf16 = p->y_dtype == STRATA_X_BF16;
    a.u_bf16 = p->u_dtype == STRATA_X_BF16;
    a.flags = p->flags;
    a.a = p->resid_scale;
    a.b = p->branch_scale;
    a.eps = p->eps;
    return a;
}

// Blocks of the gradient.  With gains' gradients asked for, one block takes up
// to two trips of rows by itself and leaves the sums where they belong: the
// second launch and its wait cost more than the second trip (2048 columns, 1
// row: 5.6 -> 3.4 us, 2 rows: 5.7 -> 4.8, 4096 columns, 2 rows: 7.1 -> 6.7) but
// for the longest rows (8192 columns, 2 rows: 10.1 -> 11.4 us, so one trip).
int back_blocks(const strata_block_norm_args *p, bool gains) {
    const int group = wave_rows(p->d) ? 4 : 1;
    if (gains && p->T > 0 && p->T <= (p->d <= 4096 ? 2 : 1) * group) return 1;
    const int64_t rows = ((int64_t)p->T + group - 1) / group;
    return (int)(rows < BN_BLOCKS ? rows : BN_BLOCKS);
}

hipError_t launch_norm(const NormArgs &a, bool back, hipStream_t s) {
    if (a.d % 8 == 0) {
        switch (a.x_bf16 | a.y_bf16 << 1 | a.u_bf16 << 2) {
            case 0: return block_norm_launch<float, float, float>(a, back, s);
            case 1: return block_norm_launch<uint16_t, float, float>(a, back, s);
            case 2: return block_norm_launch<float, uint16_t, float>(a, back, s);
            case 3: return block_norm_launch<uint16_t, uint16_t, float>(a, back, s);
            case 4: return block_norm_launch<float, float, uint16_t>(a, back, s);
            case 5: return block_norm_launch<uint16_t, float, uint16_t>(a, back, s);
            case 6: return block_norm_launch<float, uint16_t, uint16_t>(a, back, s);
            default: return block_norm_launch<uint16_t, uint16_t, uint16_t>(a, back, s);
        }
    }
    return a.d % 2 == 0 ? block_norm_launch_any<2>(a, back, s) : block_norm_launch_any<1>(a, back, s);
}

}  // namespace

}  // namespace strata

using namespace strata;

extern "C" {

strata_status strata_block_norm(const strata_block_norm_args *args, const void *x, const void *y, const void *gate,
                                const float *g_post, const float *g_pre, void *r, void *u, float *rstd_y,
                                float *rstd_r, void *stream) {
    strata_status st = check_norm(args);
    if (st != STRATA_OK || args->T == 0) return st;
    st = check_norm_inputs(args, y, gate, g_post, g_pre);
    if (st != STRATA_OK) return st;
    const bool pre = args->flags & STRATA_PRE_NORM, post = args->flags & STRATA_POST_NORM;
    if (bad_rows(x) || pre != (u != nullptr) || (!r && !u)) return STRATA_EINVAL;
    if ((rstd_y && !post) || (rstd_r && !pre)) return STRATA_EINVAL;
    if (!aligned16(y) || !aligned16(gate) || !aligned16(g_post) || !aligned16(g_pre) || !aligned16(r) || !aligned16(u))
        return STRATA_EINVAL;
    NormArgs a = norm_args(args);
    a.x = x;
    a.y = y;
    a.gate = gate;
    a.g_post = g_post;
    a.g_pre = g_pre;
    a.r = r;
    a.u = u;
    a.rstd_y = rstd_y;
    a.rstd_r = rstd_r;
    const hipStream_t s = (hipStream_t)stream;
    return hip_status(launch_norm(a, false, s));
}

size_t strata_block_norm_backward_workspace_bytes(const strata_block_norm_args *args) {
    if (check_norm(args) != STRATA_OK) return 0;
    const size_t n = (size_t)2 * back_blocks(args, true) * args->d * 4;
    return n ? n : 256;
}

strata_status strata_block_norm_backward(const strata_block_norm_args *args, const void *dr, const void *du,
                                         const void *r, const void *y, const void *gate, const float *g_post,
                                         const float *g_pre, const float *rstd_y, const float *rstd_r, void *dx,
                                         void *dy, void *dgate, float *dg_post, float *dg_pre, void *ws,
                                         size_t ws_bytes, void *stream) {
    strata_status st = check_norm(args);
    if (st != STRATA_OK) return st;
    const bool pre = args->flags & STRATA_PRE_NORM, post = args->flags & STRATA_POST_NORM;
    if ((dg_post && !post) || (dg_pre && !pre)) return STRATA_EINVAL;
    if (!aligned16(dg_post) || !aligned16(dg_pre)) return STRATA_EINVAL;
    const bool rows = args->T > 0, gains = dg_post || dg_pre;
    if (rows) {
        st = check_norm_inputs(args, y, gate, g_post, g_pre);
        if (st != STRATA_OK) return st;
        if (pre != (du != nullptr) || (!dr && !du) || (pre && (!r || !rstd_r))) return STRATA_EINVAL;
        if (y && post && !rstd_y) return STRATA_EINVAL;
        if ((dy && !y) || (dgate && !gate)) return STRATA_EINVAL;
        if (!aligned16(dr) || !aligned16(du) || !aligned16(r) || !aligned16(y) || !aligned16(gate) ||
            !aligned16(g_post) || !aligned16(g_pre) || !aligned16(dx) || !aligned16(dy) || !aligned16(dgate))
            return STRATA_EINVAL;
        if (gains && (!ws || !aligned16(ws))) return STRATA_EINVAL;
        if (gains && ws_bytes < strata_block_norm_backward_workspace_bytes(args)) return STRATA_EWORKSPACE;
    }
    NormArgs a = norm_args(args);
    a.dr = dr;
    a.du = du;
    a.rin = r;
    a.y = y;
    a.gate = gate;
    a.g_post = g_post;
    a.g_pre = g_pre;
    a.rstd_y_in = rstd_y;
    a.rstd_r_in = rstd_r;
    a.dx = dx;
    a.dy = dy;
    a.dgate = dgate;
    a.dg_post = dg_post;
    a.dg_pre = dg_pre;
    a.blocks = back_blocks(args, gains);
    const bool alone = a.blocks == 1 && rows;
    a.part_post = alone ? dg_post : (float *)ws;
    a.part_pre = alone ? dg_pre : (float *)ws + (size_t)a.blocks * a.d;
    const hipStream_t s = (hipStream_t)stream;
    if (rows && (dx || dy || dgate || gains)) {
        const hipError_t e = launch_norm(a, true, s);
        if (e != hipSuccess) return hip_status(e);
    }
    if (gains && !alone) {   // no rows: no partial sums, zeros
        STRATA_LAUNCH(block_norm_gains_kernel, dim3((a.d + 31) / 32, 2), dim3(1024), 0, s, a);
        return hip_status(hipGetLastError());
    }
    return STRATA_OK;
}

}  // extern "C"
