// shares.cu -- pages that several requests hold (include/csa2_draft.h): forked requests, ended ones, and
// the contents of pages.  shares[id] counts a page's holders beyond the first, so that pages fresh from
// csa2p_page_plan need no count.
#include "common.cuh"
#include "draft.cuh"
#include "internal.h"

namespace csa2 {
namespace {

constexpr int32_t kRefused = -2;            // in dst: the request was not forked

// ---------------------------------------------------------------- fork
constexpr int kForkThreads = 1024;
static_assert(kForkThreads == 32 * 32, "a lane for each warp");

struct ForkOf {
    int32_t from, len;                      // -1: no fork
    uint32_t flags;
    bool page;                              // takes a page
    int32_t last;                           // the last page, not full
};

__device__ __forceinline__ ForkOf fork_of(const csa2d_share_args &P, int shift, int b)
{
    ForkOf f{-1, 0, 0u, false, -1};
    const int32_t a = P.source[b];
    if (a < 0) return f;
    if (a >= P.batch || a == b || P.lens[b] > 0 || P.source[a] >= 0) {
        f.flags = CSA2_DEV_BAD_INDEX;
        return f;
    }
    const int32_t len = max(P.lens[a], 0), full = len >> shift, part = len & ((1 << shift) - 1);
    if (full > P.width - (part > 0)) {
        f.flags = CSA2P_DEV_TABLE_FULL;
        return f;
    }
    f.from = a;
    f.len = len;
    if (part) {
        f.last = P.block_table[(int64_t)a * P.width + full];
        f.page = f.last >= 0 && f.last < P.n_pages;
        if (f.last >= P.n_pages) f.flags = CSA2_DEV_BAD_INDEX;
    }
    return f;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// One CTA: who is forked, which free page each takes, the new lengths; a thread has one of 1,024
// requests at a time.  What it writes -- lengths and last entries of forked requests -- nobody else
// reads here: a source is no forked request.  Latency bounds it: source, lengths, last page, scan, page
// (with the shared pages, and an end of the same requests: 10.3 us for eight forks of 512 pages).
__global__ void __launch_bounds__(kForkThreads) page_fork_kernel(const csa2d_share_args P, const int shift, uint32_t *d_status)
{
    __shared__ int32_t s_warp[kForkThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_allow_dependents();
    const int32_t n_free = min(max(P.n_free[0], 0), P.free_cap);
    uint32_t flags = 0;
    int32_t all = 0;                                       // pages taken by the requests before
    for (int b0 = 0; b0 < P.batch; b0 += kForkThreads) {
        const int b = b0 + tid;
        const bool is = b < P.batch;
        ForkOf f{-1, 0, 0u, false, -1};
        if (is) f = fork_of(P, shift, b);
        flags |= f.flags;
        const uint32_t take = __ballot_sync(0xffffffffu, f.page);
        if (lane == 0) s_warp[warp] = __popc(take);
        __syncthreads();
        // every warp sums up all warps' numbers
        const int32_t mine = s_warp[lane];
        const int32_t earlier = (int32_t)__reduce_add_sync(0xffffffffu, lane < warp ? (uint32_t)mine : 0u);
        const int32_t at = n_free - 1 - (all + earlier + __popc(take & ((1u << lane) - 1)));
        all += (int32_t)__reduce_add_sync(0xffffffffu, (uint32_t)mine);
        __syncthreads();                                   // read before the next requests' are written
        if (!is) continue;
        int32_t src = -1, dst = -1, rows = 0;
        if (P.source[b] >= 0) {
            if (f.from < 0 || (f.page && at < 0)) {
                dst = kRefused;
                if (f.from >= 0) flags |= CSA2P_DEV_NO_PAGES;
            } else {
                const int32_t part = f.len & ((1 << shift) - 1);
                if (f.page) {
                    src = f.last;
                    dst = P.free_pages[at];
                    rows = part;
                }
                if (part) P.block_table[(int64_t)b * P.width + (f.len >> shift)] = f.page ? dst : f.last;
                P.lens[b] = f.len;
            }
        }
        P.src[b] = src;
        P.dst[b] = dst;
        P.rows[b] = rows;
    }
    if (flags) dev_flag(d_status, flags);
    __syncthreads();                                       // n_free has been read (a call without requests has no other)
    if (tid == 0) P.n_free[0] = max(n_free - all, 0);
}

// Table rows are gone through by a kernel of its own, a warp for 32 entries of four requests, a lane for an
// entry of all four: where they hold the same page, as answers to one prompt do, its count is changed once
// for all of them.  A fork, its copies and end for 16 prompts with 32 answers each and up to 1,024 pages: 22.6
// us, and 29.5 when a lane had eight entries of one request; 24.6 by groups of 16, 26.6 of 32 (a lane's loads
// wait for all its requests); without neighbours that share 15.4 and 15.9 (1,000 requests of 200 entries).
// One cluster that did this and what comes before was slower however few the pieces (the same requests: 41).
constexpr int kEach = 4, kPagesThreads = 256;
__device__ __forceinline__ int32_t pieces(int32_t width) { return (width - 1) / 32 + 1; }

// What a warp of the grid has: requests b .. b + 3, entry `at` of this lane.
struct Piece {
    int32_t b, at;
};
__device__ __forceinline__ Piece piece_of(const csa2d_share_args &P)
{
    const int32_t n = pieces(P.width);
    const int64_t i = (int64_t)blockIdx.x * (kPagesThreads / 32) + threadIdx.x / 32;
    return {(int32_t)min(i / n * kEach, (int64_t)P.batch), (int32_t)(i % n) * 32 + (int32_t)(threadIdx.x & 31)};
}

// Adds `by` to the count of each of a lane's pages, once for neighbours that are the same.
__device__ __forceinline__ void count_pages(const csa2d_share_args &P, const int32_t (&id)[kEach], int32_t by, uint32_t *d_status)
{
    int32_t run = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        run += by;
        if (k + 1 < kEach && id[k + 1] == id[k]) continue;
        if (id[k] >= P.n_pages) dev_flag(d_status, CSA2_DEV_BAD_INDEX);
        else if (id[k] >= 0) atomicAdd(P.shares + id[k], run);
        run = 0;
    }
}

// The full pages of forked requests.
__global__ void __launch_bounds__(kPagesThreads) page_share_kernel(const csa2d_share_args P, const int shift, uint32_t *d_status)
{
    pdl_wait();
    pdl_allow_dependents();
    const Piece w = piece_of(P);
    const int32_t mine = w.b + (threadIdx.x & 31);             // a lane looks a request up for the warp
    int32_t source = -1, full = 0;
    if ((threadIdx.x & 31) < kEach && mine < P.batch) {
        source = P.source[mine];
        if (source >= 0 && P.dst[mine] != kRefused) full = P.lens[mine] >> shift;
    }
    int32_t id[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int32_t a = __shfl_sync(0xffffffffu, source, k), n = __shfl_sync(0xffffffffu, full, k);
        id[k] = w.at < n ? P.block_table[(int64_t)a * P.width + w.at] : -1;
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k)
        if (w.at < __shfl_sync(0xffffffffu, full, k)) P.block_table[(int64_t)(w.b + k) * P.width + w.at] = id[k];
    count_pages(P, id, 1, d_status);
}

// ---------------------------------------------------------------- free
// The pages of ended requests lose a holder each; one without any is marked by a count below 0.
__global__ void __launch_bounds__(kPagesThreads) page_drop_kernel(const csa2d_share_args P, const int shift, uint32_t *d_status)
{
    pdl_wait();
    pdl_allow_dependents();
    const Piece w = piece_of(P);
    const int32_t mine = w.b + (threadIdx.x & 31);
    int32_t held = 0;
    if ((threadIdx.x & 31) < kEach && mine < P.batch && P.ends[mine] != 0)
        held = (int32_t)min(((int64_t)max(P.lens[mine], 0) + (1 << shift) - 1) >> shift, (int64_t)P.width);
    int32_t id[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k)
        id[k] = w.at < __shfl_sync(0xffffffffu, held, k) ? P.block_table[(int64_t)(w.b + k) * P.width + w.at] : -1;
    count_pages(P, id, -1, d_status);
}

// One cluster: marked pages go on the free list in the order of their ids, so that it does not depend
// on the order in which the counts fell.  Each CTA has a run of ids; it counts, learns what the runs
// before have, and places.  (Eight million pages: 26 us with the kernel before.)
constexpr int kListThreads = 1024, kListCtas = 8, kListEach = 4;

__global__ void __launch_bounds__(kListThreads) page_list_kernel(const csa2d_share_args P, uint32_t *d_status)
{
    __shared__ int32_t s_warp[32], s_count[kListCtas];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
    cluster_arrive();                                      // waited for before a peer is written to
    pdl_wait();
    pdl_allow_dependents();
    const int32_t n_free = min(max(P.n_free[0], 0), P.free_cap);
    constexpr int kTile = kListThreads * kListEach;
    const int64_t run = (((int64_t)P.n_pages + kListCtas - 1) / kListCtas + kTile - 1) / kTile * kTile;
    const int64_t first = cta * run, end = min(first + run, (int64_t)P.n_pages);
    int32_t count = 0;
    for (int64_t i = first + tid; i < end; i += kListThreads) count += P.shares[i] < 0;
    count = (int32_t)__reduce_add_sync(0xffffffffu, (uint32_t)count);
    if (lane == 0) s_warp[warp] = count;
    cluster_wait();
    __syncthreads();
    if (warp == 0) {
        count = (int32_t)__reduce_add_sync(0xffffffffu, (uint32_t)s_warp[lane]);
        if (lane < kListCtas) {                            // this CTA's count, into every CTA's list
            uint32_t at = (uint32_t)__cvta_generic_to_shared(&s_count[cta]);
            asm volatile("mapa.shared::cluster.u32 %0, %0, %1;\n\tst.shared::cluster.b32 [%0], %2;" : "+r"(at) : "r"(lane), "r"(count) : "memory");
        }
    }
    cluster_arrive();
    cluster_wait();
    int64_t place = n_free, all = n_free;
    for (int c = 0; c < kListCtas; ++c) {
        if (c < cta) place += s_count[c];
        all += s_count[c];
    }
    // a tile of ids at a time, four consecutive ones a thread
    for (int64_t t0 = first; t0 < end && s_count[cta] > 0; t0 += kTile) {
        const int64_t i0 = t0 + kListEach * tid;
        uint32_t mark = 0;
#pragma unroll
        for (int k = 0; k < kListEach; ++k) mark |= (uint32_t)(i0 + k < end && P.shares[i0 + k] < 0) << k;
        const int32_t n = __popc(mark);
        int32_t before = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t u = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += u;
        }
        __syncthreads();                                   // the tile before has been placed
        if (lane == 31) s_warp[warp] = before;
        __syncthreads();
        int32_t in_tile = 0;
        before -= n;
        for (int w = 0; w < kListThreads / 32; ++w) {
            if (w < warp) before += s_warp[w];
            in_tile += s_warp[w];
        }
        int64_t at = place + before;
#pragma unroll
        for (int k = 0; k < kListEach; ++k)
            if (mark >> k & 1u) {
                P.shares[i0 + k] = 0;
                if (at < P.free_cap) P.free_pages[at] = (int32_t)(i0 + k);
                ++at;
            }
        place += in_tile;
    }
    if (cta == 0 && tid == 0) {
        P.n_free[0] = (int32_t)min(all, (int64_t)P.free_cap);
        if (all > P.free_cap) dev_flag(d_status, CSA2P_DEV_TABLE_FULL);
    }
    for (int b = cta * kListThreads + tid; b < P.batch; b += kListCtas * kListThreads)
        if (P.ends[b] != 0) P.lens[b] = 0;
}

// ---------------------------------------------------------------- contents
constexpr int kCopyThreads = 256, kCopyEach = 6;    // loads of 16 bytes a thread has under way

__device__ __forceinline__ void copy_bytes(uint8_t *to, const uint8_t *from, int64_t n, int64_t first, int64_t step)
{
    const uintptr_t low = (uintptr_t)to | (uintptr_t)from;
    int64_t done = 0;
    if ((low & 15) == 0) {
        done = n & ~(int64_t)15;
        for (int64_t i = first; i < n / 16; i += kCopyEach * step) {
            uint4 v[kCopyEach];
#pragma unroll
            for (int k = 0; k < kCopyEach; ++k)
                if (i + k * step < n / 16) v[k] = reinterpret_cast<const uint4 *>(from)[i + k * step];
#pragma unroll
            for (int k = 0; k < kCopyEach; ++k)
                if (i + k * step < n / 16) reinterpret_cast<uint4 *>(to)[i + k * step] = v[k];
        }
    } else if ((low & 3) == 0) {
        done = n & ~(int64_t)3;
        for (int64_t i = first; i < n / 4; i += step) reinterpret_cast<uint32_t *>(to)[i] = reinterpret_cast<const uint32_t *>(from)[i];
    }
    for (int64_t i = done + first; i < n; i += step) to[i] = from[i];
}

// A CTA (or several, for large pages) takes a pair of pages in one cache.  Latency bounds it: ids, rows,
// loads, stores (eight part pages in four caches 4.1 us, 512 in four 10.3).
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const __grid_constant__ CacheSet set, const int32_t *src, const int32_t *dst,
                                                                 const int32_t *rows, uint32_t *d_status)
{
    const PagedView &C = set.c[blockIdx.y];
    pdl_wait();
    pdl_allow_dependents();
    const int32_t from = src[blockIdx.x], to = dst[blockIdx.x];
    if (from < 0 || to < 0 || from == to) return;
    if (from >= C.n_pages || to >= C.n_pages) {
        if (threadIdx.x == 0 && blockIdx.z == 0) dev_flag(d_status, CSA2_DEV_BAD_INDEX);
        return;
    }
    const int32_t page = 1 << C.shift;
    const int64_t n = rows ? min(max(rows[blockIdx.x], 0), page) : page;
    const int64_t first = (int64_t)blockIdx.z * kCopyThreads + threadIdx.x, step = (int64_t)gridDim.z * kCopyThreads;
    uint8_t *codes = const_cast<uint8_t *>(C.codes), *scales = const_cast<uint8_t *>(C.scales);
    copy_bytes(codes + to * C.code_page, codes + from * C.code_page, n * C.code_row, first, step);
    if (C.scale_row) copy_bytes(scales + to * C.scale_page, scales + from * C.scale_page, n * C.scale_row, first, step);
}

// CTAs of a warp for each piece of all the table rows.
unsigned piece_ctas(const csa2d_share_args &a)
{
    const int64_t n = ((int64_t)a.batch + kEach - 1) / kEach * ((a.width - 1) / 32 + 1);
    return (unsigned)((n + kPagesThreads / 32 - 1) / (kPagesThreads / 32));
}

} // namespace

cudaError_t launch_page_fork(const csa2d_share_args &a, uint32_t *d_status, cudaStream_t s)
{
    const int shift = __builtin_ctz((unsigned)a.page);
    const cudaError_t e = launch_pdl(page_fork_kernel, dim3(1), dim3(kForkThreads), 0, s, 1, a, shift, d_status);
    if (e != cudaSuccess) return e;
    return launch_pdl(page_share_kernel, dim3(piece_ctas(a)), dim3(kPagesThreads), 0, s, 1, a, shift, d_status);
}

cudaError_t launch_page_free(const csa2d_share_args &a, uint32_t *d_status, cudaStream_t s)
{
    const int shift = __builtin_ctz((unsigned)a.page);
    const cudaError_t e = launch_pdl(page_drop_kernel, dim3(piece_ctas(a)), dim3(kPagesThreads), 0, s, 1, a, shift, d_status);
    if (e != cudaSuccess) return e;
    return launch_pdl(page_list_kernel, dim3(kListCtas), dim3(kListThreads), 0, s, kListCtas, a, d_status);
}

cudaError_t launch_page_copy(const CacheSet &set, int n, const int32_t *src, const int32_t *dst, const int32_t *rows,
                             int32_t count, uint32_t *d_status, cudaStream_t s)
{
    int64_t most = 1;                                      // bytes of a page's codes
    for (int i = 0; i < n; ++i) {
        const int64_t bytes = (int64_t)set.c[i].code_row << set.c[i].shift;
        most = bytes > most ? bytes : most;
    }
    const int64_t z = (most + kCopyThreads * kCopyEach * 16 - 1) / (kCopyThreads * kCopyEach * 16);
    return launch_pdl(page_copy_kernel, dim3((unsigned)count, (unsigned)n, (unsigned)(z < 64 ? z : 64)), dim3(kCopyThreads), 0, s, 1, set, src, dst, rows, d_status);
}

} // namespace csa2
