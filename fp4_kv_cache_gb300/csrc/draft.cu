// draft.cu -- trees of drafted tokens over the paged cache (include/csa2_draft.h): their positions and
// masks, and the rows that stay moved together.
#include "common.cuh"
#include "draft.cuh"
#include "internal.h"

namespace csa2 {
namespace {

// ---------------------------------------------------------------- positions and masks
constexpr int kTreeThreads = 128, kMaxNodes = 32 * CSA2D_MAX_WORDS;

// A CTA takes a request, a thread a node: it goes up to the root through the parents in shared memory
// and writes the mask's words as it leaves them, highest first (parents are lower nodes).  What
// bounds it is latency: the offsets, the parents, one step a level (4.1 us for 32 chains of six, 6.2 for
// four trees of up to 64).
__global__ void __launch_bounds__(kTreeThreads) tree_plan_kernel(const csa2d_tree_args P, uint32_t *d_status)
{
    __shared__ int32_t s_parent[kMaxNodes];
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_allow_dependents();
    auto held = [&](int32_t c) { return min(max(c, 0), P.n_tokens); };
    bool down = false;
    for (int b = tid; b < P.batch; b += kTreeThreads) down |= held(P.cu[b + 1]) < held(P.cu[b]);
    down = __syncthreads_or(down);
    if (down && blockIdx.x == 0 && tid == 0) dev_flag(d_status, CSA2_DEV_BAD_INDEX);
    auto none = [&](int64_t t) {
        P.pos[t] = -1;
        for (int w = 0; w < P.words; ++w) P.seen[t * P.words + w] = 0u;
    };
    // tokens of no request: before the first one's and behind the last one's
    const bool some = P.batch > 0 && !down;
    const int32_t begin = some ? held(P.cu[0]) : P.n_tokens, end = some ? held(P.cu[P.batch]) : P.n_tokens;
    for (int64_t i = (int64_t)blockIdx.x * kTreeThreads + tid; i < begin + (int64_t)(P.n_tokens - end); i += (int64_t)gridDim.x * kTreeThreads)
        none(i < begin ? i : end + (i - begin));
    if (!some) return;
    for (int b = blockIdx.x; b < P.batch; b += gridDim.x) {
        const int64_t c0 = P.cu[b], n = P.cu[b + 1] - c0;
        if (n <= 0) continue;
        const int32_t rows = P.lens[b];
        if (c0 < 0 || c0 + n > P.n_tokens || n > 32 * P.words || rows < n) {
            if (tid == 0) dev_flag(d_status, CSA2_DEV_BAD_INDEX);
            for (int64_t t = held(P.cu[b]) + tid; t < held(P.cu[b + 1]); t += kTreeThreads) none(t);
            continue;
        }
        __syncthreads();                                   // the request before has been read
        for (int i = tid; i < n; i += kTreeThreads) {
            int32_t p = P.parent[c0 + i];
            if (p < -1 || p >= i) {
                dev_flag(d_status, CSA2_DEV_BAD_INDEX);
                p = -1;
            }
            s_parent[i] = p;
        }
        __syncthreads();
        for (int i = tid; i < n; i += kTreeThreads) {
            uint32_t *row = P.seen + (c0 + i) * P.words;
            for (int w = P.words - 1; w > i >> 5; --w) row[w] = 0u;
            int w = i >> 5, depth = -1;
            uint32_t bits = 0;
            for (int k = i; k >= 0; k = s_parent[k]) {
                if (k >> 5 != w) {
                    row[w] = bits;
                    bits = 0;
                    while (--w > k >> 5) row[w] = 0u;
                }
                bits |= 1u << (k & 31);
                ++depth;
            }
            row[w] = bits;
            while (--w >= 0) row[w] = 0u;
            P.pos[c0 + i] = (int32_t)(rows - n) + depth;
        }
    }
}

// ---------------------------------------------------------------- rows that stay
constexpr int kMoveThreads = 128, kMoveAhead = 8;

// A CTA takes a request in one cache, a thread a column of its rows: 16 bytes of codes or a byte of
// scales, which it moves row by row down the path.  The path rises, so a row is read before anything
// is written there (path[j] > i for j > i), and no thread touches another's column.  Eight rows are on
// their way at a time.  Latency bounds it: offsets, path, table, row, store (32 requests in four caches
// 6.1 us, 64 in twenty 8.2).
__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const csa2d_compact_args P, const __grid_constant__ CacheSet set, uint32_t *d_status)
{
    const PagedView &C = set.c[blockIdx.y];
    const int b = blockIdx.x, tid = threadIdx.x;
    pdl_wait();
    pdl_allow_dependents();
    const int32_t keep = P.keep[b];
    const int64_t c0 = P.cu[b], n = P.cu[b + 1] - c0, base = P.lens[b] - n;
    const int32_t *path = P.path + (int64_t)b * P.max_path;
    bool bad = keep < 0 || keep > P.max_path || n < 0 || base < 0;
    if (P.pos && n > 0) bad |= c0 < 0 || c0 + n > P.n_tokens || P.pos[c0] < 0;      // the plan left it out
    if (!bad)
        for (int i = tid; i < keep; i += kMoveThreads) bad |= path[i] <= (i ? path[i - 1] : -1) || path[i] >= n;
    bad = __syncthreads_or(bad);
    if (blockIdx.y == 0 && tid == 0) {
        if (bad && keep != 0) dev_flag(d_status, CSA2_DEV_BAD_INDEX);
        if (P.delta && bad && n > 0 && base >= 0) P.delta[b] = min(P.delta[b], (int32_t)-n);
    }
    if (bad || keep == 0) return;
    const int32_t *table = P.block_table + (int64_t)b * P.width;
    auto slot = [&](int64_t row) -> int32_t {              // -1: in no page
        const int64_t page = row >> C.shift;
        const int32_t id = page < P.width ? table[page] : -1;
        return id < 0 || id >= C.n_pages ? -1 : (int32_t)((id << C.shift) + (row & ((1 << C.shift) - 1)));
    };
    uint8_t *codes = const_cast<uint8_t *>(C.codes), *scales = const_cast<uint8_t *>(C.scales);
    const int pieces = C.code_row / 16, columns = pieces + C.scale_row;
    for (int col = tid; col < columns; col += kMoveThreads) {
        for (int i0 = 0; i0 < keep; i0 += kMoveAhead) {
            uint4 v[kMoveAhead];
            int32_t to[kMoveAhead];
#pragma unroll
            for (int k = 0; k < kMoveAhead; ++k) {
                const int i = i0 + k;
                to[k] = -1;
                v[k] = make_uint4(0u, 0u, 0u, 0u);
                if (i >= keep) continue;
                const int32_t at = path[i];
                if (at == i) continue;
                const int32_t from = slot(base + at);
                to[k] = slot(base + i);
                if (from < 0 || to[k] < 0) {
                    if (col == 0) dev_flag(d_status, CSA2_DEV_BAD_INDEX);
                    to[k] = -1;
                } else if (col < pieces) {
                    v[k] = *reinterpret_cast<const uint4 *>(codes + C.code_at(from) + 16 * col);
                } else {
                    v[k].x = scales[C.scale_at(from) + col - pieces];
                }
            }
#pragma unroll
            for (int k = 0; k < kMoveAhead; ++k) {
                if (to[k] < 0) continue;
                if (col < pieces) *reinterpret_cast<uint4 *>(codes + C.code_at(to[k]) + 16 * col) = v[k];
                else scales[C.scale_at(to[k]) + col - pieces] = (uint8_t)v[k].x;
            }
        }
    }
}

} // namespace

cudaError_t launch_tree_plan(const csa2d_tree_args &a, uint32_t *d_status, cudaStream_t s)
{
    // CTAs: one a request while they fit the GPU a few times over; without requests, for the tokens
    const int64_t most = 8 * (int64_t)device_sm_count(), fill = (a.n_tokens + (int64_t)kTreeThreads - 1) / kTreeThreads;
    const int64_t want = a.batch > 0 ? a.batch : fill;
    return launch_pdl(tree_plan_kernel, dim3((unsigned)(want < most ? want : most)), dim3(kTreeThreads), 0, s, 1, a, d_status);
}

cudaError_t launch_compact(const csa2d_compact_args &a, const CacheSet &set, int n, uint32_t *d_status, cudaStream_t s)
{
    return launch_pdl(compact_kernel, dim3((unsigned)a.batch, (unsigned)n), dim3(kMoveThreads), 0, s, 1, a, set, d_status);
}

} // namespace csa2
