// Rows of a table by token id, and the table's gradient (strata_embed,
// strata_embed_backward).
//
// Forward: a group of threads takes a token and copies its row, scaled and
// converted; bound by HBM (5 rows of 2048: 2.3 us).
//
// Gradient: the tokens are sorted by id (a stable counting sort over the low
// and then the high 10 bits of the ids), the sorted list is cut into chunks
// of EB_ROWS, and a group of threads walks a chunk: equal ids lie together,
// so a row's sum stays in registers and is stored once.  A run of equal ids
// that crosses chunks (frequent tokens) leaves one partial sum per chunk,
// and a second launch joins them where the run starts.  No atomics: the
// order of every sum follows from the ids.  16384 tokens into 128000 x 2048 bf16:
// 127 us, 99 of them the table's zeros (5.3 TB/s) beside the sort's two passes, 19.5
// the chunks and 7 the runs; bound by the 524 MB of zeros.
//
// Up to EB_FEW tokens take one launch: a block for each token finds the tokens
// of the same id and, where its own is the first, adds their rows; others write
// the zeros between.  us against the launches above, of ids that differ and of one
// id alone: 9 tokens of 531 x 640 3.4 and 3.3 against 11.5 and 11.4; 128 3.5 and 10.7
// against 14 and 11.5; 256 3.7 and 19.4 against 12.4 and 13.8; 256 of 5000 x 2048,
// zeros included, in bf16 5.4 and 32 against 20 and 18, in fp32 8.1 and 36 against 19
// and 19.  One id's rows are added by the blocks of one token: up to 128 of them that
// is no loss, 256 take up to twice as long here, which differing ids, the usual ones,
// gain 2.4 to 3.7 times over.
#include <cmath>
#include <type_traits>

#include "rows.hpp"
#include "sort_impl.hpp"

namespace strata {

constexpr int EB_ROWS = 16;          // sorted tokens of a chunk
constexpr int EB_BITS = 10;          // of a sort pass
constexpr int EB_DIGIT = 1 << EB_BITS;
constexpr int EB_VOCAB = (1 << 20) - 1;
constexpr int EB_TOKENS = 1 << 22;
constexpr int EB_FEW = 256;          // tokens of a call of one launch, at most a block's threads
constexpr int EB_FEW_ZEROS = 2048;   // most blocks of its zeros

template <typename W, typename O, int V, int G>
__global__ __launch_bounds__(256) void embed_kernel(const W *__restrict__ table, const int32_t *__restrict__ ids, O *out,
                                                    int T, int vocab, int d, float scale) {
    int t, lane;
    if (!row_group<G>(T, t, lane)) return;
    const int id = ids[t];
    const bool there = (uint32_t)id < (uint32_t)vocab;
    for (int i = (blockIdx.y * G + lane) * V; i < d; i += gridDim.y * G * V) {
        Raw<W, V> v;
        zero_raw(v);
        if (there) load_raw<V>(table, (int64_t)id * d + i, v);
        float s[V];
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = there ? value<V>(v, j) * scale : 0.f;
        store_values<V>(out, (int64_t)t * d + i, s);
    }
}

// One digit of the token ids, in the order that src (null: the tokens' own) gives.
struct TokenKey {
    static constexpr bool WIDE = false;
    const int32_t *ids, *src;
    int shift, vocab;
    __device__ __forceinline__ int32_t value(int64_t i) const { return src ? src[i] : (int32_t)i; }
    __device__ __forceinline__ int operator()(int64_t i) const {
        const int t = value(i);
        if (t < 0) return -1;   // behind the last token with a row
        const int id = ids[t];
        return (uint32_t)id < (uint32_t)vocab ? (id >> shift) & (EB_DIGIT - 1) : -1;
    }
};

struct EmbedBack {
    const void *dout;
    const int32_t *ids, *order;   // order: tokens sorted by id, -1 behind the last with a row
    void *dW;
    float *head, *tail;           // per chunk the sum of a run from the chunk before, of one into the chunk after
    int T, d, chunks, add;
    float scale;
};

// Table row `id` of the gradient, columns i.. of it, from its sum.
template <typename W, int V> __device__ __forceinline__ void embed_store(const EmbedBack &a, int id, int i, const float (&s)[V]) {
    W *row = (W *)a.dW + (int64_t)id * a.d;
    float q[V];
    if (a.add) {
        Raw<W, V> old;
        load_raw<V>(row, i, old);
#pragma unroll
        for (int j = 0; j < V; ++j) q[j] = fmaf(a.scale, s[j], value<V>(old, j));
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) q[j] = a.scale * s[j];
    }
    store_values<V>(row, i, q);
}

template <typename W, typename O, int V, int G> __global__ __launch_bounds__(256) void embed_chunks_kernel(EmbedBack a) {
    constexpr int NG = 256 / G;
    __shared__ int tok[NG][EB_ROWS], key[NG][EB_ROWS + 2];   // key: the one before, the chunk's, the one behind (-1: none)
    int c, lane;
    const bool live = row_group<G>(a.chunks, c, lane);
    const int g = threadIdx.x / G;
    const int p0 = c * EB_ROWS;
    for (int r = lane; r < EB_ROWS + 2; r += G) {
        const int p = p0 + r - 1;
        const int t = live && p >= 0 && p < a.T ? a.order[p] : -1;
        key[g][r] = t >= 0 ? a.ids[t] : -1;
        if (r >= 1 && r <= EB_ROWS) tok[g][r - 1] = t;
    }
    __syncthreads();
    if (!live || tok[g][0] < 0) return;
    const O *dout = (const O *)a.dout;
    const bool from = key[g][0] == key[g][1], into = key[g][EB_ROWS + 1] >= 0 && key[g][EB_ROWS + 1] == key[g][EB_ROWS];
    for (int i = (blockIdx.y * G + lane) * V; i < a.d; i += gridDim.y * G * V) {
        float s[V];
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = 0.f;
        bool first = true;   // the chunk's first run
#pragma unroll
        for (int r0 = 0; r0 < EB_ROWS; r0 += 8) {
            Raw<O, V> v[8];
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (tok[g][r0 + r] >= 0) load_raw<V, true>(dout, (int64_t)tok[g][r0 + r] * a.d + i, v[r]);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                if (tok[g][r0 + r] < 0) continue;
                const int id = key[g][r0 + r + 1];
#pragma unroll
                for (int j = 0; j < V; ++j) s[j] += value<V>(v[r], j);
                const bool end = r0 + r + 1 == EB_ROWS;
                if (!end && key[g][r0 + r + 2] == id) continue;   // the run goes on
                if (first && from) store_values<V>(a.head, (int64_t)c * a.d + i, s);
                else if (end && into) store_values<V>(a.tail, (int64_t)c * a.d + i, s);
                else embed_store<W, V>(a, id, i, s);
                first = false;
#pragma unroll
                for (int j = 0; j < V; ++j) s[j] = 0.f;
            }
        }
    }
}

// A run that crosses chunks, where it starts: a block adds its tail and the
// heads of the chunks that it reaches, four waves a quarter of them each.
template <typename W, int V> __global__ __launch_bounds__(256) void embed_join_kernel(EmbedBack a) {
    __shared__ float part[3][64 * V];
    const int c = blockIdx.x, p1 = (c + 1) * EB_ROWS;   // the chunk behind starts there
    const auto id_at = [&](int p) {
        const int t = p < a.T ? a.order[p] : -1;
        return t >= 0 ? a.ids[t] : -1;
    };
    const int id = id_at(p1 - 1);
    if (id < 0 || id_at(p1) != id) return;                                            // no run leaves the chunk
    const int p0 = c * EB_ROWS;
    if (p0 > 0 && id_at(p0) == id && id_at(p0 - 1) == id) return;                     // it started before
    const int lane = threadIdx.x & 63;
    int n = 0;   // chunks behind this one that begin with the run: 64 at a time
    for (uint64_t m = ~0ull; m == ~0ull; n += __popcll(m)) m = __ballot(id_at((c + 1 + n + lane) * EB_ROWS) == id);
    const int last = c + n, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int per = (n + 3) / 4, b0 = c + 1 + w * per, b1 = min(b0 + per, last + 1);
    for (int i0 = blockIdx.y * 64 * V; i0 < a.d; i0 += gridDim.y * 64 * V) {
        const int i = i0 + lane * V;
        const bool in = i < a.d;
        float s[V];
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = 0.f;
        if (in) {
            if (w == 0) {
                Raw<float, V> v;
                load_raw<V>(a.tail, (int64_t)c * a.d + i, v);
#pragma unroll
                for (int j = 0; j < V; ++j) s[j] = value<V>(v, j);
            }
#pragma unroll 4
            for (int b = b0; b < b1; ++b) {
                Raw<float, V> v;
                load_raw<V>(a.head, (int64_t)b * a.d + i, v);
#pragma unroll
                for (int j = 0; j < V; ++j) s[j] += value<V>(v, j);
            }
        }
        if (w) {
#pragma unroll
            for (int j = 0; j < V; ++j) part[w - 1][lane * V + j] = s[j];
        }
        __syncthreads();
        if (w == 0 && in) {
#pragma unroll
            for (int q = 0; q < 3; ++q)
#pragma unroll
                for (int j = 0; j < V; ++j) s[j] += part[q][lane * V + j];
            embed_store<W, V>(a, id, i, s);
        }
        __syncthreads();
    }
}

// A call of few tokens: T * shares blocks for the tokens, the others for the zeros of `per` rows each.
template <typename W, typename O, int V> __global__ __launch_bounds__(256) void embed_few_kernel(EmbedBack a, int vocab, int shares, int per) {
    __shared__ int tok[EB_FEW], cnt[4];
    __shared__ uint32_t taken[((EB_VOCAB + EB_FEW_ZEROS) / EB_FEW_ZEROS + 31) / 32];
    const int th = threadIdx.x, lane = th & 63, w = __builtin_amdgcn_readfirstlane(th >> 6);
    const int b = blockIdx.x, id = th < a.T ? a.ids[th] : -1;
    if (b < a.T * shares) {
        const int t = b / shares, mine = a.ids[t];
        if ((uint32_t)mine >= (uint32_t)vocab) return;
        const uint64_t m = __ballot(id == mine);
        if (lane == 0) cnt[w] = __popcll(m);
        __syncthreads();
        int at = __popcll(m & ((1ull << lane) - 1)), n = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q < w) at += cnt[q];
            n += cnt[q];
        }
        if (id == mine) tok[at] = th;
        __syncthreads();
        if (tok[0] != t) return;
        const O *dout = (const O *)a.dout;
        for (int i = ((b - t * shares) * 256 + th) * V; i < a.d; i += shares * 256 * V) {
            float s[V];
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] = 0.f;
            const auto rows = [&](int r0, auto many) {
                constexpr int R = decltype(many)::value;
                Raw<O, V> v[R];
#pragma unroll
                for (int r = 0; r < R; ++r)   // behind the last one that again, so that no load waits behind a branch
                    load_raw<V, true>(dout, (int64_t)tok[min(r0 + r, n - 1)] * a.d + i, v[r]);
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (r0 + r < n) {
#pragma unroll
                        for (int j = 0; j < V; ++j) s[j] += value<V>(v[r], j);
                    }
            };
            int r0 = 0;
            for (; r0 + 16 <= n; r0 += 16) rows(r0, std::integral_constant<int, 16>());
            for (; r0 < n; r0 += 4) rows(r0, std::integral_constant<int, 4>());
            embed_store<W, V>(a, mine, i, s);
        }
        return;
    }
    const int v0 = (b - a.T * shares) * per, rows = min(per, vocab - v0);
    for (int i = th; i < (rows + 31) / 32; i += 256) taken[i] = 0;
    __syncthreads();
    const uint32_t at = (uint32_t)id - (uint32_t)v0;   // ids below 0 come out past every row
    if (at < (uint32_t)rows) atomicOr(&taken[at >> 5], 1u << (at & 31));
    __syncthreads();
    const uint32_t nq = (uint32_t)(a.d / V);
    const float zero[V] = {};
    for (int r = 0; r < rows; ++r) {
        if (taken[r >> 5] >> (r & 31) & 1) continue;
        for (uint32_t q = th; q < nq; q += 256) store_values<V>((W *)a.dW, (int64_t)(v0 + r) * a.d + q * V, zero);
    }
}

// n 16-byte pieces of zeros, and the bytes behind them: the share of block b of
// nb, in one piece (524 MB beside the sort: 126 us the gradient, 133 where the
// blocks go through it side by side).
__device__ __forceinline__ void embed_zeros(u32x4_t *p, int64_t n, int rest, int b, int nb) {
    const int64_t per = (n + nb - 1) / nb, i0 = b * per, i1 = min(i0 + per, n);
    for (int64_t i = i0 + threadIdx.x; i < i1; i += SORT_TH) p[i] = u32x4_t{0, 0, 0, 0};
    if (b == 0 && (int)threadIdx.x < rest) ((uint8_t *)(p + n))[threadIdx.x] = 0;
}

__global__ __launch_bounds__(SORT_TH) void embed_zero_kernel(u32x4_t *p, int64_t n, int rest) {
    embed_zeros(p, n, rest, blockIdx.x, gridDim.x);
}

// A pass of the sort, and beside it, on the CUs that the sort leaves idle, zeros for a part of the table.
__global__ __launch_bounds__(SORT_TH) void embed_sort_kernel(SortArgs a, TokenKey key, int copies, u32x4_t *p, int64_t n, int rest) {
    if ((int)blockIdx.x < a.blocks) sort_once(a, key, copies);
    else embed_zeros(p, n, rest, blockIdx.x - a.blocks, gridDim.x - a.blocks);
}

namespace {

struct EmbedCall {
    const void *table;
    const int32_t *ids;
    void *out;
    int T, V, d;
    float scale;
    hipStream_t s;
};

struct Forward {
    template <typename W, typename O, int V> static void run(const EmbedCall &c) {
        const RowGroups q = row_groups(c.T, c.d / V, 16);
#define EMBED(G)                                                                                                        \
    case G:                                                                                                             \
        STRATA_LAUNCH((embed_kernel<W, O, V, G>), row_grid(c.T, G, q.shares), dim3(256), 0, c.s, (const W *)c.table, c.ids, \
                      (O *)c.out, c.T, c.V, c.d, c.scale);                                                              \
        break;
        switch (q.threads) { EMBED(16) EMBED(32) EMBED(64) EMBED(128) EMBED(256) }
#undef EMBED
    }
};

struct BackCall {
    EmbedBack a;
    int d;
    hipStream_t s;
};

struct FewCall {
    EmbedBack a;
    int V, d;
    hipStream_t s;
};

struct Chunks {
    template <typename W, typename O, int V> static void run(const BackCall &c) {
        const RowGroups q = row_groups(c.a.chunks, c.d / V, 16);
#define CHUNKS(G)                                                                                                   \
    case G:                                                                                                         \
        STRATA_LAUNCH((embed_chunks_kernel<W, O, V, G>), row_grid(c.a.chunks, G, q.shares), dim3(256), 0, c.s, c.a); \
        break;
        switch (q.threads) { CHUNKS(16) CHUNKS(32) CHUNKS(64) CHUNKS(128) CHUNKS(256) }
#undef CHUNKS
    }
};

struct Join {
    template <typename W, typename O, int V> static void run(const BackCall &c) {
        if (!std::is_same<O, float>::value) return;   // the partial sums have one type
        const int slabs = (c.d + 64 * V - 1) / (64 * V);
        STRATA_LAUNCH((embed_join_kernel<W, V>), dim3(c.a.chunks, slabs < 64 ? slabs : 64), dim3(256), 0, c.s, c.a);
    }
};

struct Few {
    template <typename W, typename O, int V> static void run(const FewCall &c) {
        const int64_t pieces = c.d / V;
        int shares = (int)((pieces + 255) / 256);   // of a row
        shares = shares < 16 ? shares : 16;
        const int zeros = c.a.add ? 0 : c.V < EB_FEW_ZEROS ? c.V : EB_FEW_ZEROS, per = zeros ? (c.V + zeros - 1) / zeros : 1;
        STRATA_LAUNCH((embed_few_kernel<W, O, V>), dim3(c.a.T * shares + (zeros ? (c.V + per - 1) / per : 0)), dim3(256), 0, c.s, c.a,
                      c.V, shares, per);
    }
};

// The widest pieces that divide the row: 8 values where a row is bf16, else 4.
template <typename F, typename W, typename O, typename C> void embed_width(const C &c) {
    if constexpr (sizeof(W) == 2 || sizeof(O) == 2) {
        if (c.d % 8 == 0) return F::template run<W, O, 8>(c);
    }
    if (c.d % 4 == 0) return F::template run<W, O, 4>(c);
    if (c.d % 2 == 0) return F::template run<W, O, 2>(c);
    return F::template run<W, O, 1>(c);
}

template <typename F, typename C> hipError_t embed_types(const C &c, int wdtype, int odtype) {
    const bool wb = wdtype == STRATA_X_BF16, ob = odtype == STRATA_X_BF16;
    if (wb && ob) embed_width<F, uint16_t, uint16_t>(c);
    else if (wb) embed_width<F, uint16_t, float>(c);
    else if (ob) embed_width<F, float, uint16_t>(c);
    else embed_width<F, float, float>(c);
    return hipGetLastError();
}

// Sort plan of one pass over T tokens with ids of E values.
SortArgs pass_plan(int T, int E) {
    SortArgs a{};
    a.n = T;
    a.E = E;
    sort_plan(a);
    return a;
}

// n pieces of zeros and the bytes behind them.
struct Zeros {
    u32x4_t *p;
    int64_t n;
    int rest;
};
unsigned zero_blocks(int64_t n) {
    const int64_t b = (n + SORT_TH - 1) / SORT_TH;
    return (unsigned)(b < 1 ? 1 : b < 2048 ? b : 2048);
}

hipError_t sort_beside(const SortArgs &a, const TokenKey &key, const Zeros &z, hipStream_t s) {
    const unsigned more = z.n || z.rest ? zero_blocks(z.n) : 0;
    STRATA_LAUNCH(embed_sort_kernel, dim3(a.blocks + more), dim3(SORT_TH), 0, s, a, key, sort_copies(a), z.p, z.n, z.rest);
    return hipGetLastError();
}

struct BackPlan {
    int chunks;
    size_t order, half, counts, head, tail, bytes;   // offsets of the workspace's parts
};

BackPlan back_plan(int32_t T, int32_t d) {
    BackPlan p{};
    const auto pad = [](size_t n) { return (n + 255) / 256 * 256; };
    p.chunks = (T + EB_ROWS - 1) / EB_ROWS;
    p.half = pad((size_t)T * 4);
    p.counts = p.half + pad((size_t)T * 4);
    p.head = p.counts + pad(sort_counts_bytes(pass_plan(T, EB_DIGIT)));
    p.tail = p.head + pad((size_t)p.chunks * d * 4);
    p.bytes = p.tail + pad((size_t)p.chunks * d * 4) + 256;
    return p;
}

strata_status check_embed(int32_t T, int32_t V, int32_t d, int32_t most_tokens, int32_t most_rows) {
    if (T < 0 || V < 1 || d < 1) return STRATA_EINVAL;
    return T > most_tokens || d > MAX_COLS || V > most_rows ? STRATA_EUNSUPPORTED : STRATA_OK;
}

bool bad_ids(const int32_t *p) { return !p || ((uintptr_t)p & 3u); }

}  // namespace

}  // namespace strata

using namespace strata;

extern "C" {

strata_status strata_embed(const void *W, strata_xdtype wdtype, int32_t V, int32_t d, const int32_t *ids, int32_t T,
                           float scale, void *out, strata_xdtype odtype, void *stream) {
    if (bad_dtype(wdtype) || bad_dtype(odtype) || !std::isfinite(scale)) return STRATA_EINVAL;
    const strata_status st = check_embed(T, V, d, MAX_ROWS, MAX_COLS);
    if (st != STRATA_OK || T == 0) return st;
    if (bad_rows(W) || bad_rows(out) || bad_ids(ids)) return STRATA_EINVAL;
    return hip_status(embed_types<Forward>(EmbedCall{W, ids, out, T, V, d, scale, (hipStream_t)stream}, wdtype, odtype));
}

size_t strata_embed_backward_workspace_bytes(int32_t T, int32_t V, int32_t d) {
    if (check_embed(T, V, d, EB_TOKENS, EB_VOCAB) != STRATA_OK) return 0;
    return back_plan(T, d).bytes;
}

strata_status strata_embed_backward(const void *dout, strata_xdtype odtype, const int32_t *ids, int32_t T, int32_t V,
                                    int32_t d, float scale, void *dW, strata_xdtype wdtype, uint32_t flags, void *ws,
                                    size_t ws_bytes, void *stream) {
    if (bad_dtype(wdtype) || bad_dtype(odtype) || !std::isfinite(scale) || (flags & ~STRATA_ACCUMULATE)) return STRATA_EINVAL;
    const strata_status st = check_embed(T, V, d, EB_TOKENS, EB_VOCAB);
    if (st != STRATA_OK) return st;
    if (bad_rows(dW) || (T > 0 && (bad_rows(dout) || bad_ids(ids) || bad_rows(ws)))) return STRATA_EINVAL;
    const BackPlan p = back_plan(T, d);
    if (T > 0 && ws_bytes < p.bytes) return STRATA_EWORKSPACE;
    const hipStream_t s = (hipStream_t)stream;
    const bool add = flags & STRATA_ACCUMULATE;
    const int64_t bytes = (int64_t)V * d * (wdtype == STRATA_X_BF16 ? 2 : 4);
    // The sort's slots and the runs come from the ids and the workspace: neither may change under it.
    if (T > 0 && (overlap(dW, bytes, ws, p.bytes) || overlap(dW, bytes, ids, (size_t)T * 4) ||
                  overlap(ws, p.bytes, ids, (size_t)T * 4)))
        return STRATA_EINVAL;
    if (T > 0 && T <= EB_FEW)
        return hip_status(embed_types<Few>(FewCall{EmbedBack{dout, ids, nullptr, dW, nullptr, nullptr, T, d, 0, add, scale}, V, d, s}, wdtype,
                                           odtype));
    // The zeros: beside the sort's passes where those are one launch each.
    const bool two = V > EB_DIGIT, beside = T > 0 && T <= SORT_ONCE;
    Zeros z{(u32x4_t *)dW, add ? 0 : bytes / 16, add ? 0 : (int)(bytes % 16)};
    if (!add && !beside) {
        STRATA_LAUNCH(embed_zero_kernel, dim3(zero_blocks(z.n)), dim3(SORT_TH), 0, s, z.p, z.n, z.rest);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return hip_status(e);
    }
    if (T == 0) return STRATA_OK;
    char *const w = (char *)ws;
    int32_t *order = (int32_t *)(w + p.order);
    SortArgs a = pass_plan(T, two ? EB_DIGIT : V);
    a.bcnt = (int32_t *)(w + p.counts);
    a.perm = two ? (int32_t *)(w + p.half) : order;
    const int64_t n0 = two ? z.n / 2 : z.n;   // pieces of the first pass
    hipError_t e = beside ? sort_beside(a, TokenKey{ids, nullptr, 0, V}, Zeros{z.p, n0, two ? 0 : z.rest}, s)
                          : launch_sort(a, TokenKey{ids, nullptr, 0, V}, s);
    if (e != hipSuccess) return hip_status(e);
    if (two) {
        const int32_t *half = a.perm;
        a = pass_plan(T, ((V - 1) >> EB_BITS) + 1);
        a.bcnt = (int32_t *)(w + p.counts);
        a.perm = order;
        e = beside ? sort_beside(a, TokenKey{ids, half, EB_BITS, V}, Zeros{z.p + n0, z.n - n0, z.rest}, s)
                   : launch_sort(a, TokenKey{ids, half, EB_BITS, V}, s);
        if (e != hipSuccess) return hip_status(e);
    }
    BackCall c{EmbedBack{dout, ids, order, dW, (float *)(w + p.head), (float *)(w + p.tail), T, d, p.chunks, add, scale}, d, s};
    e = embed_types<Chunks>(c, wdtype, odtype);
    if (e != hipSuccess) return hip_status(e);
    return hip_status(embed_types<Join>(c, wdtype, STRATA_X_F32));
}

}  // extern "C"
