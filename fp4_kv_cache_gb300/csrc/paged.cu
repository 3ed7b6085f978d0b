// paged.cu -- page bookkeeping, rotary positions with several axes, and the paged cache's
// write and read (include/csa2_paged.h).  The cache is the one of DeepSeek-V4.1-Flash report
// §2.4.4 (rows quantised after RoPE, RoPE and other channels in one format) laid out in pages.
#include "common.cuh"
#include "internal.h"
#include "paged.cuh"
#include "paged_decode.cuh"

namespace csa2 {
namespace {

// ---------------------------------------------------------------- bookkeeping
constexpr int kPlanThreads = 512;
constexpr int kPlanMaxReq = CSA2P_MAX_BATCH / kPlanThreads;     // requests a thread

struct PlanParams {
    int32_t batch, shift, width, free_cap, n_rows;
    const int32_t *lens, *delta, *n_free;
    int32_t *lens_out, *table, *free_pages, *n_free_out, *cu, *slot, *row_req, *row_pos;
};

struct Req {
    int64_t old_len, new_len;
    int32_t had, has;       // pages before and after, both within the table
    bool full;
};

__device__ __forceinline__ Req plan_req(const PlanParams &P, int b)
{
    Req r;
    r.old_len = max(P.lens[b], 0);
    r.new_len = r.old_len + P.delta[b];
    r.new_len = r.new_len < 0 ? 0 : (r.new_len > 0x7fffffff ? 0x7fffffff : r.new_len);
    const int64_t up = (int64_t(1) << P.shift) - 1;
    const int64_t had = (r.old_len + up) >> P.shift, has = (r.new_len + up) >> P.shift;
    r.full = has > P.width;
    r.had = (int32_t)(had < P.width ? had : P.width);
    r.has = (int32_t)(has < P.width ? has : P.width);
    return r;
}

// Largest i with a[i] <= x in the non-decreasing a[0..n] (a[0] = 0 <= x): runs of equal entries
// (requests that contribute nothing) are passed over, so a[i+1] > x where i < n.
__device__ __forceinline__ int last_at_or_below(const int32_t *a, int n, int32_t x)
{
    int lo = 0, hi = n + 1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int32_t hold31(int64_t v) { return (int32_t)(v > 0x7fffffff ? 0x7fffffff : v); }

// Exclusive sums of K numbers a thread over the block.
template <int K>
__device__ __forceinline__ void block_before(const int64_t (&own)[K], int64_t (&before)[K], int64_t (*s_warp)[32])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        int64_t v = own[k];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) s_warp[k][warp] = v;
        before[k] = v - own[k];
    }
    __syncthreads();
    if (warp < K) {
        int64_t v = lane < kPlanThreads / 32 ? s_warp[warp][lane] : 0;
        const int64_t mine = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        s_warp[warp][lane] = v - mine;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) before[k] += s_warp[k][warp];
}

// What the requests before each (and, last, all of them) add and move: [batch + 1] in shared memory.
struct PlanSums {
    int32_t *cu, *take, *back;      // rows added, pages taken, pages given back
};

// Entries that request b (threads without one: has = had = 0) gives back and that name a page.
// Called by whole warps: a thread counts a few entries itself, all 32 those of a request with many.
__device__ __forceinline__ int32_t pages_named(const PlanParams &P, int b, const Req &r)
{
    constexpr int32_t kFew = 4;
    const int lane = threadIdx.x & 31;
    const int32_t n = max(r.had - r.has, 0);
    int32_t count = 0;
#pragma unroll
    for (int32_t i = 0; i < kFew; ++i)
        if (n <= kFew && i < n) count += P.table[(int64_t)b * P.width + r.has + i] >= 0;
    uint32_t many = __ballot_sync(0xffffffffu, n > kFew);
    while (many) {
        const int from = __ffs((int)many) - 1;
        many &= many - 1;
        const int32_t *t = P.table + (int64_t)__shfl_sync(0xffffffffu, b, from) * P.width + __shfl_sync(0xffffffffu, r.has, from);
        const int32_t m = __shfl_sync(0xffffffffu, n, from);
        int32_t c = 0;
#pragma unroll 8
        for (int32_t i = lane; i < m; i += 32) c += t[i] >= 0;
        c = (int32_t)__reduce_add_sync(0xffffffffu, (uint32_t)c);
        if (lane == from) count = c;
    }
    return count;
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_ctas()
{
    uint32_t n;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void set_peer(int32_t *p, uint32_t rank)      // the peer's copy of shared *p: 1
{
    uint32_t at = (uint32_t)__cvta_generic_to_shared(p);
    asm volatile("mapa.shared::cluster.u32 %0, %0, %1;\n\tst.shared::cluster.b32 [%0], %2;" : "+r"(at) : "r"(rank), "r"(1) : "memory");
}

// Scans the requests, `per` consecutive ones a thread; entries given back are taken for pages.  One
// CTA tells (cu, status).
__device__ __forceinline__ void plan_scan(const PlanParams &P, const PlanSums &S, int64_t (*s_warp)[32], bool tell, uint32_t *d_status)
{
    const int per = (P.batch + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min((int)threadIdx.x * per, P.batch), b1 = min(b0 + per, P.batch);
    int64_t own[3] = {0, 0, 0}, before[3];
    for (int b = b0; b < b1; ++b) {
        const Req r = plan_req(P, b);
        own[0] += r.new_len > r.old_len ? r.new_len - r.old_len : 0;
        own[1] += max(r.has - r.had, 0);
        own[2] += max(r.had - r.has, 0);
        if (r.full && tell) dev_flag(d_status, CSA2P_DEV_TABLE_FULL);
    }
    block_before<3>(own, before, s_warp);
    for (int b = b0; b <= b1; ++b) {
        if (b == b1 && b != P.batch) break;                    // the next thread's first entry
        S.cu[b] = hold31(before[0]);
        S.take[b] = hold31(before[1]);
        S.back[b] = hold31(before[2]);
        if (tell) P.cu[b] = S.cu[b];
        if (b == b1) break;
        const Req r = plan_req(P, b);
        before[0] += r.new_len > r.old_len ? r.new_len - r.old_len : 0;
        before[1] += max(r.has - r.had, 0);
        before[2] += max(r.had - r.has, 0);
    }
    __syncthreads();
}

// Whether one of this thread's share of the entries given back names no page.  The cluster's CTAs share
// the entries out, 512 a warp, so that sixteen loads of a thread follow one another.
__device__ __forceinline__ bool plan_look(const PlanParams &P, const PlanSums &S, uint32_t rank, uint32_t peers)
{
    constexpr int kEach = 16;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t all = S.back[P.batch];
    int32_t seen = 0;
    for (int64_t i0 = 32ll * kEach * (rank * (kPlanThreads / 32) + warp); i0 < all; i0 += (int64_t)kEach * kPlanThreads * peers) {
        const int32_t *p[kEach];
        int b = last_at_or_below(S.back, P.batch, (int32_t)min(i0 + lane, (int64_t)all - 1));
        int32_t at = S.back[b], end = S.back[b + 1];
        const int32_t *t = P.table + (int64_t)b * P.width + plan_req(P, b).has;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int32_t i = (int32_t)min(i0 + lane + 32 * k, (int64_t)all - 1);
            if (i >= end) {
                while (S.back[b + 1] <= i) ++b;                // i < back[batch]: ends in time
                at = S.back[b];
                end = S.back[b + 1];
                t = P.table + (int64_t)b * P.width + plan_req(P, b).has;
            }
            p[k] = t + (i - at);
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k) seen |= *p[k];
    }
    return seen < 0;
}

// Counts the pages given back anew: those that the entries name.
__device__ __noinline__ void plan_recount(const PlanParams &P, const PlanSums &S, int64_t (*s_warp)[32])
{
    const int per = (P.batch + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min((int)threadIdx.x * per, P.batch), b1 = min(b0 + per, P.batch);
    int64_t named[1] = {0}, first[1];
    for (int k = 0; k < per; ++k) {                            // whole warps: pages_named
        const int b = b0 + k;
        Req r = {};
        if (b < b1) r = plan_req(P, b);
        const int32_t n = pages_named(P, b, r);
        if (b < b1) S.back[b] = n;
        named[0] += n;
    }
    block_before<1>(named, first, s_warp);
    for (int b = b0; b <= b1; ++b) {
        if (b == b1 && b != P.batch) break;
        const int32_t n = b < b1 ? S.back[b] : 0;
        S.back[b] = hold31(first[0]);
        first[0] += n;
    }
    __syncthreads();
}

// One block: all old lengths are read before the first new one is written.
__device__ __forceinline__ void new_lengths(const PlanParams &P, int32_t n_out)
{
    int32_t len_new[kPlanMaxReq];
#pragma unroll
    for (int k = 0; k < kPlanMaxReq; ++k) {
        const int b = threadIdx.x + k * kPlanThreads;
        if (b < P.batch) len_new[k] = (int32_t)plan_req(P, b).new_len;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPlanMaxReq; ++k) {
        const int b = threadIdx.x + k * kPlanThreads;
        if (b < P.batch) P.lens_out[b] = len_new[k];
    }
    if (threadIdx.x == 0) P.n_free_out[0] = n_out;
}

// Every CTA scans all the requests for itself -- rows added, pages taken, pages given back -- so
// that the rows, the taken pages and the returned pages can be shared out with no exchange.  No
// CTA writes what another may still read: table entries read are never written (a request takes or
// gives back, not both), and the free list is read below n_free and written above it.  Only the new
// lengths and count may go where the old ones are: then (`later`) a second kernel writes them, and
// with one CTA a barrier is enough.  A shortage leaves -1 in a table, which is no page to give back:
// the entries given back are looked at, shared out over the CTAs of a cluster, and counted only where
// one names no page.  What bounds it is the chain of loads, scans and barriers, not its bytes: 512
// requests of one new row take 7.1 us, 193 with room for 65,536 new rows and 30,000 pages given back
// 13.9 us (9.9 without the look; 16.7 with each CTA looking at all of them).
__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PlanParams P, const int later, uint32_t *d_status)
{
    extern __shared__ int32_t sm[];
    int32_t *s_cu = sm, *s_take = s_cu + P.batch + 1, *s_back = s_take + P.batch + 1;
    __shared__ int64_t s_warp[3][32];
    __shared__ int32_t s_hole;
    const int tid = threadIdx.x, n_cta = gridDim.x, cta = blockIdx.x;
    const uint32_t peers = cluster_ctas();
    if (tid == 0) s_hole = 0;
    if (peers > 1) cluster_arrive();
    pdl_wait();
    pdl_allow_dependents();
    const int n_free = min(max(P.n_free[0], 0), P.free_cap);
    const PlanSums S{s_cu, s_take, s_back};
    plan_scan(P, S, s_warp, cta == 0, d_status);
    if (peers > 1) cluster_wait();                             // the peers' marks are clear
    bool hole = false;
    if (s_back[P.batch] > 0) {
        hole = __syncthreads_or(plan_look(P, S, cluster_rank(), peers));
        if (peers > 1) {
            if (hole && tid < peers) set_peer(&s_hole, tid);
            cluster_arrive();
            cluster_wait();
            hole = *(volatile int32_t *)&s_hole;
        }
        if (hole) plan_recount(P, S, s_warp);
    }
    const int n_new = s_cu[P.batch], n_take = s_take[P.batch], n_back = s_back[P.batch];
    const int64_t top = (int64_t)n_free + n_back;
    if (tid == 0 && cta == 0) {
        if (n_take > top) dev_flag(d_status, CSA2P_DEV_NO_PAGES);
        if (n_new > P.n_rows) dev_flag(d_status, CSA2P_DEV_ROWS);
        if (top - n_take > P.free_cap) dev_flag(d_status, CSA2P_DEV_TABLE_FULL);
    }
    auto returned = [&](int i) -> int32_t {                    // i-th page given back
        const int b = last_at_or_below(s_back, P.batch, i);
        const Req r = plan_req(P, b);
        const int32_t *t = P.table + (int64_t)b * P.width + r.has;
        int32_t k = i - s_back[b];
        const int32_t n = r.had - r.has;
        if (s_back[b + 1] - s_back[b] == n) return t[k];
        for (int32_t j = 0; j < n; j += 16) {                  // some entries are no pages: the k-th that is
            uint32_t named = 0;
#pragma unroll
            for (int32_t u = 0; u < 16; ++u) named |= (uint32_t)(t[min(j + u, n - 1)] >= 0 && j + u < n) << u;
            const int32_t c = __popc(named);
            if (k < c) {
                for (; k > 0; --k) named &= named - 1;
                return t[j + __ffs((int)named) - 1];
            }
            k -= c;
        }
        return -1;
    };
    auto taken = [&](int i) -> int32_t {                       // i-th page handed out
        const int64_t at = top - 1 - i;
        return at < 0 ? -1 : at >= n_free ? returned((int)(at - n_free)) : P.free_pages[at];
    };
    const int step = n_cta * kPlanThreads, first = cta * kPlanThreads + tid;
    // ---- new rows, four a thread
    for (int64_t r0 = 4ll * first; r0 < P.n_rows; r0 += 4ll * step) {
        int32_t vs[4] = {-1, -1, -1, -1}, vr[4] = {-1, -1, -1, -1}, vp[4] = {-1, -1, -1, -1};
        int b = r0 < n_new ? last_at_or_below(s_cu, P.batch, (int32_t)r0) : 0;
        int64_t page_at = -1;
        int32_t page = -1;
        int last_b = -1;
        Req q = {};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t r = r0 + k;
            if (r >= n_new) break;
            while (s_cu[b + 1] <= r) ++b;                      // r < cu[batch]: ends in time
            if (b != last_b) { q = plan_req(P, b); last_b = b; page_at = -1; }
            const int64_t pos = q.old_len + (r - s_cu[b]);
            const int64_t j = pos >> P.shift;
            if (j != page_at) {
                page_at = j;
                page = j >= P.width ? -1 : j >= q.had ? taken(s_take[b] + (int)(j - q.had)) : P.table[(int64_t)b * P.width + j];
            }
            const int64_t sl = ((int64_t)page << P.shift) + (pos & ((int64_t(1) << P.shift) - 1));
            vs[k] = page < 0 || sl > 0x7fffffff ? -1 : (int32_t)sl;
            vr[k] = b;
            vp[k] = (int32_t)pos;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (r0 + k < P.n_rows) {
                P.slot[r0 + k] = vs[k];
                if (P.row_req) P.row_req[r0 + k] = vr[k];
                if (P.row_pos) P.row_pos[r0 + k] = vp[k];
            }
    }
    // ---- pages taken, into the tables
    for (int64_t i = first; i < n_take; i += step) {
        const int b = last_at_or_below(s_take, P.batch, (int32_t)i);
        P.table[(int64_t)b * P.width + plan_req(P, b).had + (i - s_take[b])] = taken((int)i);
    }
    // ---- pages given back and not taken again, onto the free list
    const int64_t left = top - n_take < 0 ? 0 : top - n_take;
    const int64_t keep = left < P.free_cap ? left : P.free_cap;
    if (!hole) {
        for (int64_t i = first; i < n_back; i += step)
            if (n_free + i < keep) P.free_pages[n_free + i] = returned((int)i);
    } else {
        // a warp a request, past the entries that are no pages (page by page, as above, a request of
        // 16,384 pages with one such entry took 7.7 ms; now 0.4)
        const int lane = tid & 31;
        for (int b = (cta * kPlanThreads + tid) >> 5; b < P.batch; b += step >> 5) {
            const Req r = plan_req(P, b);
            int64_t at = (int64_t)n_free + s_back[b];
#pragma unroll 8
            for (int32_t j0 = r.has; j0 < r.had; j0 += 32) {
                const int32_t id = j0 + lane < r.had ? P.table[(int64_t)b * P.width + j0 + lane] : -1;
                const uint32_t named = __ballot_sync(0xffffffffu, id >= 0);
                const int64_t to = at + __popc(named & ((1u << lane) - 1));
                if (id >= 0 && to < keep) P.free_pages[to] = id;
                at += __popc(named);
            }
        }
    }
    if (cta > 0) return;
    const int32_t n_out = (int32_t)keep;
    if (!later) new_lengths(P, n_out);
    else if (tid == 0) P.cu[0] = n_out;                        // carried over to the second kernel
}

// The new lengths and count, when they overwrite the old ones and several CTAs read those.  One
// block.  The count comes in cu[0], which is 0 otherwise.
__global__ void __launch_bounds__(kPlanThreads) page_plan_later_kernel(const PlanParams P)
{
    pdl_wait();
    pdl_allow_dependents();
    const int32_t n_out = P.cu[0];
    new_lengths(P, n_out);
    if (threadIdx.x == 0) P.cu[0] = 0;
}

// ---------------------------------------------------------------- rotation
// Turns the pairs of eight channels col .. col+7 that lie at or past channel c0 (even), with
// one rounding per product and per sum, as csa2_rope_quant_fp4 does.  at[]: the row's positions.
struct Positions { int32_t at[3]; };
__device__ __forceinline__ Positions row_positions(const RopeView &R, int64_t row, int64_t rows)
{
    const int half = R.dim >> 1;
    Positions p;
    p.at[0] = R.pos[row];
    p.at[1] = R.end0 < half ? R.pos[rows + row] : -1;
    p.at[2] = R.end1 < half ? R.pos[2 * rows + row] : -1;
    return p;
}
__device__ __forceinline__ void rotate8(float (&v)[8], int col, int c0, const RopeView &R, const Positions &at, uint32_t *d_status)
{
    const int half = R.dim >> 1;
    float c[4], s[4];
    bool on[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {                 // all on their way before the first is used
        const int i = (col + 2 * k - c0) >> 1;
        int32_t p = i < R.end0 ? at.at[0] : i < R.end1 ? at.at[1] : at.at[2];
        if (col + 2 * k < c0) p = -1;
        if (p >= R.n_pos) {
            dev_flag(d_status, CSA2_DEV_BAD_INDEX);
            p = -1;
        }
        on[k] = p >= 0;
        c[k] = 1.0f;
        s[k] = 0.0f;
        if (on[k]) {
            const float *cs = R.cs + (int64_t)p * R.dim + i;
            c[k] = cs[0];
            s[k] = cs[half];
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float a = v[2 * k], b = v[2 * k + 1];
        if (on[k]) {
            v[2 * k] = __fsub_rn(__fmul_rn(a, c[k]), __fmul_rn(b, s[k]));
            v[2 * k + 1] = __fadd_rn(__fmul_rn(a, s[k]), __fmul_rn(b, c[k]));
        }
    }
}

// The same where four pairs share an axis and lie aligned (RopeView.quads): position, then cosines
// and sines 16 bytes at a time, so that a kernel can have them on their way with its rows.
struct Turn {
    int32_t p;          // position, or -1: nothing to turn
    float4 c, s;
};
__device__ __forceinline__ int32_t turn_position(const RopeView &R, int col, int c0, int64_t row, int64_t rows)
{
    const int i = (col - c0) >> 1;
    return R.pos[((i >= R.end0) + (i >= R.end1)) * rows + row];
}
__device__ __forceinline__ void turn_load(Turn &t, const RopeView &R, int col, int c0, uint32_t *d_status)
{
    if (t.p >= R.n_pos) {
        dev_flag(d_status, CSA2_DEV_BAD_INDEX);
        t.p = -1;
    }
    if (t.p < 0) return;
    const float *cs = R.cs + (int64_t)t.p * R.dim + ((col - c0) >> 1);
    t.c = *reinterpret_cast<const float4 *>(cs);
    t.s = *reinterpret_cast<const float4 *>(cs + (R.dim >> 1));
}
__device__ __forceinline__ void turn8(float (&v)[8], const Turn &t)
{
    if (t.p < 0) return;
    const float c[4] = {t.c.x, t.c.y, t.c.z, t.c.w}, s[4] = {t.s.x, t.s.y, t.s.z, t.s.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float a = v[2 * k], b = v[2 * k + 1];
        v[2 * k] = __fsub_rn(__fmul_rn(a, c[k]), __fmul_rn(b, s[k]));
        v[2 * k + 1] = __fadd_rn(__fmul_rn(a, s[k]), __fmul_rn(b, c[k]));
    }
}

__device__ __forceinline__ void unpack8(uint4 raw, float (&v)[8])
{
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A thread takes pieces of eight channels (16 bytes) of one row of q; blockIdx.x = row, the
// row's pieces are shared by gridDim.y blocks.  In place (`same`) only the pieces that hold
// turned channels are visited; x and out are then the same memory, which a thread reads before it writes
// it, so neither is __restrict__.  HBM bounds it: 604 MB of three-axis rows out of place take 104 us,
// 5.8 TB/s; 32 x 64 rows (4.7 MB, from L2) take 2 us.
__global__ void __launch_bounds__(256) paged_rope_kernel(const uint16_t *x, int64_t x_row, int64_t x_head,
                                                         uint16_t *out, int64_t out_row, int64_t out_head, int32_t heads,
                                                         int32_t d, int32_t first_piece, int64_t rows,
                                                         const __grid_constant__ RopeView R,
                                                         uint32_t *d_status)
{
    pdl_wait();
    pdl_allow_dependents();
    const int64_t row = blockIdx.x;
    const int per_head = d / 8 - first_piece, n = heads * per_head, c0 = d - R.dim;
    for (int i = blockIdx.y * 256 + threadIdx.x; i < n; i += 256 * gridDim.y) {
        const int h = i / per_head, col = 8 * (first_piece + i - h * per_head);
        uint4 raw = *reinterpret_cast<const uint4 *>(x + row * x_row + h * x_head + col);
        if (R.dim > 0 && col + 8 > c0) {
            float v[8];
            unpack8(raw, v);
            if (R.quads) {
                Turn t;
                t.p = turn_position(R, col, c0, row, rows);
                turn_load(t, R, col, c0, d_status);
                turn8(v, t);
            } else {
                rotate8(v, col, c0, R, row_positions(R, row, rows), d_status);
            }
            raw = pack8(v);
        }
        *reinterpret_cast<uint4 *>(out + row * out_row + h * out_head + col) = raw;
    }
}

// ---------------------------------------------------------------- write
// Inputs here are not `const __restrict__`: these kernels begin while the one before them may still be
// writing x and the slots (they wait for it first), so that the memory is not read-only for as long as
// they run, which the loads of such pointers take for granted.
__device__ __forceinline__ float max_nan(float a, float b)      // NaN if either is
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Blocks of (d / 16, rows) threads: thread (x, y) takes sixteen channels of a row (32 bytes of x),
// a scale block of 32 channels is two neighbours of one warp (d / 16 is even).  16,384 rows of 576,
// MXFP4 (19 MB in, 5 MB out): 5.8 us without rotation (8.2 with eight channels a thread: as many
// instructions for the address and the scale), 9.1 with one axis, 12.2 with three; 32 rows 1.6 to 2.9.
// At 131,072 rows a scheduler issues in 58%, 69% and 75% of the cycles while DRAM runs at 59%, 41% and
// 26%: with rotation the issue bounds it, because 4 of a row's 36 threads turn and their warps' others wait.
// ROPE 0: none; 1: RopeView.quads (the same 16,384 rows through 2: 12.2 us, where 1 takes 9.1); 2: any.
template <int FMT, int ROPE>
__global__ void __launch_bounds__(1024) paged_write_kernel(const PagedView C, const uint16_t *x, int64_t ldx,
                                                           int32_t rows, const int32_t *slot,
                                                           const __grid_constant__ RopeView R, uint32_t *d_status)
{
    pdl_wait();
    pdl_allow_dependents();
    const int part = threadIdx.x, col = 16 * part, c0 = C.d - R.dim;
    // whole blocks go round together: the threads of a warp stay with each other's shuffles
    for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < rows; r0 += (int64_t)gridDim.x * blockDim.y) {
        const int64_t r = r0 + threadIdx.y;
        const bool in = r < rows;
        const int32_t sl = in ? slot[r] : -1;
        uint4 raw[2] = {};
        Turn turn[2] = {{-1, {}, {}}, {-1, {}, {}}};
        Positions at = {};
        if (in) {
            raw[0] = reinterpret_cast<const uint4 *>(x + r * ldx + col)[0];
            raw[1] = reinterpret_cast<const uint4 *>(x + r * ldx + col)[1];
            if (ROPE == 2 && col + 16 > c0) at = row_positions(R, r, rows);
            if (ROPE == 1 && col + 16 > c0) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (col + 8 * h >= c0) turn[h].p = turn_position(R, col + 8 * h, c0, r, rows);
#pragma unroll
                for (int h = 0; h < 2; ++h) turn_load(turn[h], R, col + 8 * h, c0, sl >= 0 ? d_status : nullptr);
            }
        }
        const bool act = sl >= 0 && sl < C.n_slots;
        if (sl >= C.n_slots && part == 0) dev_flag(d_status, CSA2_DEV_BAD_INDEX);
        float e[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            unpack8(raw[h], e[h]);
            if (ROPE == 1) turn8(e[h], turn[h]);
            if (ROPE == 2 && act && col + 8 * h + 8 > c0) rotate8(e[h], col + 8 * h, c0, R, at, d_status);
        }
        uint8_t *codes = const_cast<uint8_t *>(C.codes) + C.code_at(act ? sl : 0) + part * code_bytes<FMT>(16);
        if (FMT == CSA2P_BF16) {
            if (act) {
                reinterpret_cast<uint4 *>(codes)[0] = pack8(e[0]);
                reinterpret_cast<uint4 *>(codes)[1] = pack8(e[1]);
            }
            continue;
        }
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = max_nan(amax, fabsf(e[i >> 3][i & 7]));
        if (FMT != CSA2P_NVFP4_E4M3_16) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        if (!act) continue;
        const bool head = FMT == CSA2P_NVFP4_E4M3_16 || (part & 1) == 0;
        if (!(amax < INFINITY)) {
            if (head) dev_flag(d_status, CSA2_DEV_NONFINITE);
            amax = 0.0f;
        }
        uint32_t sbyte;
        if (FMT == CSA2P_MXFP8) {
            const int X = mx8_block_exponent(amax);
            const float inv = pow2_neg(X);
            uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i >> 2] |= e4m3_cvt(e[i >> 3][i & 7] * inv) << (8 * (i & 3));
            *reinterpret_cast<uint4 *>(codes) = make_uint4(w[0], w[1], w[2], w[3]);
            sbyte = (uint32_t)(X + 127);
        } else {
            uint32_t w[2] = {0u, 0u};
            if (FMT == CSA2P_NVFP4_E4M3_16) {
                sbyte = e4m3_block_scale(amax);
                const float sc = e4m3_value(sbyte);
                if (sc > 0.0f) {
#pragma unroll
                    for (int i = 0; i < 16; i += 2)
                        w[i >> 3] |= e2m1x2_cvt(__fdiv_rn(e[i >> 3][i & 7], sc), __fdiv_rn(e[i >> 3][(i & 7) + 1], sc)) << (4 * (i & 7));
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) w[i >> 3] |= (__float_as_uint(e[i >> 3][i & 7]) >> 31) << (4 * (i & 7) + 3);
                }
            } else {
                const int X = mx_block_exponent(amax);
                const float inv = pow2_neg(X);
#pragma unroll
                for (int i = 0; i < 16; i += 2)
                    w[i >> 3] |= e2m1x2_cvt(e[i >> 3][i & 7] * inv, e[i >> 3][(i & 7) + 1] * inv) << (4 * (i & 7));
                sbyte = (uint32_t)(X + 127);
            }
            *reinterpret_cast<uint2 *>(codes) = make_uint2(w[0], w[1]);
        }
        if (head) const_cast<uint8_t *>(C.scales)[C.scale_at(sl) + (FMT == CSA2P_NVFP4_E4M3_16 ? part : part >> 1)] = (uint8_t)sbyte;
    }
}

// ---------------------------------------------------------------- read
// Sixteen channels with a scale that one product cannot apply, or not finite: code x scale in
// float32 (exact), rounded to bf16 once.
template <int FMT>
__device__ __noinline__ void read_slow(Raw<FMT, 2> r, uint16_t *to)
{
    const float sc = FMT == CSA2P_NVFP4_E4M3_16 ? e4m3_value(r.sb & 0xffu)
                     : r.sb == 255u ? __uint_as_float(0x7fc00000u) : e8m0_value(r.sb);
#pragma unroll 1
    for (int e = 0; e < 16; ++e) {
        float x;
        if (FMT == CSA2P_MXFP8) {
            x = e4m3_value((r.w[(e >> 2) % Raw<FMT, 2>::kWords] >> (8 * (e & 3))) & 0xffu);
        } else {
            const uint32_t c = (r.w[(e >> 3) % Raw<FMT, 2>::kWords] >> (4 * (e & 7))) & 15u;
            x = c & 8u ? -e2m1_mag(c & 7u) : e2m1_mag(c & 7u);
        }
        to[e] = __bfloat16_as_ushort(__float2bfloat16_rn(x * sc));
    }
}

// Sixteen channels of one row a thread.  Two rows a thread, both asked for before the first is
// decoded, were slower at every size and coded format (16,384 rows of 576, MXFP4: 7.9 us; 131,072 rows,
// MXFP8: 62 against 41 us) and 4% faster for large bf16 reads only.  16,384 rows (5 MB in, 19 MB out)
// take 6.1 us, 32 rows 1.7 us; 524,288 rows 147 us, 5.2 TB/s.
template <int FMT>
__global__ void __launch_bounds__(1024) paged_read_kernel(const PagedView C, const int32_t *slot, int32_t rows,
                                                          uint16_t *out, int64_t ldo, uint32_t f0, uint32_t f4,
                                                          uint32_t *d_status)
{
    pdl_wait();
    pdl_allow_dependents();
    const int part = threadIdx.x;
    for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < rows; r0 += (int64_t)gridDim.x * blockDim.y) {
        const int64_t r = r0 + threadIdx.y;
        const int32_t sl = r < rows ? slot[r] : -1;
        if (sl >= C.n_slots && part == 0) dev_flag(d_status, CSA2_DEV_BAD_INDEX);
        if (sl < 0 || sl >= C.n_slots) continue;
        Raw<FMT, 2> raw;
        load_raw(raw, C.codes + C.code_at(sl) + part * code_bytes<FMT>(16),
                 C.scales + C.scale_at(sl) + (FMT == CSA2P_NVFP4_E4M3_16 ? part : part >> 1));
        uint16_t *to = out + r * ldo + 16 * part;
        if (FMT != CSA2P_BF16 && special(raw)) {
            read_slow(raw, to);
            continue;
        }
        uint32_t v[8];
        if (FMT == CSA2P_BF16) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = raw.w[i % Raw<FMT, 2>::kWords];
        } else {
            uint32_t p[8];
            decode(raw, p, f0, f4);
#pragma unroll
            for (int h = 0; h < 8; h += 4) {              // channels 0 4, 1 5, 2 6, 3 7 into order
                v[h] = prmt(p[h], p[h + 1], 0x5410u);
                v[h + 1] = prmt(p[h + 2], p[h + 3], 0x5410u);
                v[h + 2] = prmt(p[h], p[h + 1], 0x7632u);
                v[h + 3] = prmt(p[h + 2], p[h + 3], 0x7632u);
            }
        }
        reinterpret_cast<uint4 *>(to)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4 *>(to)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

// Threads (d / 16, rows a block: a multiple of 16, so whole warps) and blocks of the write and read
// kernels.
dim3 row_block(int32_t d) { return dim3((unsigned)(d / 16), (unsigned)(16 * (d < 256 ? 256 / d : 1))); }
unsigned row_grid(int32_t d, int64_t rows)
{
    const int64_t by = row_block(d).y, g = (rows + by - 1) / by, most = (int64_t)device_sm_count() * 8;
    return (unsigned)(g > most ? most : g);
}

} // namespace

bool paged_view(const csa2p_cache &c, PagedView &v)
{
    if (c.d < 32 || c.d > 1024 || c.d % 32) return false;
    if (c.page < 1 || c.page > 65536 || (c.page & (c.page - 1))) return false;
    if (c.n_pages < 0 || c.n_pages >= (int64_t(1) << 31) / c.page) return false;
    v.d = c.d;
    v.fmt = c.fmt;
    switch (c.fmt) {
    case CSA2P_MXFP4: v.code_row = c.d / 2; v.scale_row = c.d / 32; break;
    case CSA2P_NVFP4_E4M3_16: v.code_row = c.d / 2; v.scale_row = c.d / 16; break;
    case CSA2P_MXFP8: v.code_row = c.d; v.scale_row = c.d / 32; break;
    case CSA2P_BF16: v.code_row = 2 * c.d; v.scale_row = 0; break;
    default: return false;
    }
    const int64_t dense_c = (int64_t)c.page * v.code_row, dense_s = (int64_t)c.page * v.scale_row;
    v.code_page = c.code_stride ? c.code_stride : dense_c;
    v.scale_page = c.scale_stride ? c.scale_stride : dense_s;
    if (v.code_page < dense_c || v.code_page % 16 || v.scale_page < dense_s) return false;
    if (c.n_pages > 0 && (!c.codes || ((uintptr_t)c.codes & 15))) return false;
    if (c.n_pages > 0 && v.scale_row && !c.scales) return false;
    if (c.fmt == CSA2P_NVFP4_E4M3_16 && (((uintptr_t)c.scales & 1) || v.scale_page % 2)) return false;
    v.codes = static_cast<const uint8_t *>(c.codes);
    v.scales = static_cast<const uint8_t *>(c.scales);
    v.n_pages = (int32_t)c.n_pages;
    v.n_slots = c.n_pages * c.page;
    v.shift = __builtin_ctz((unsigned)c.page);
    return true;
}

cudaError_t launch_page_plan(const csa2p_plan_args &a, uint32_t *d_status, cudaStream_t s)
{
    PlanParams P;
    P.batch = a.batch;
    P.shift = __builtin_ctz((unsigned)a.page);
    P.width = a.width;
    P.free_cap = a.free_cap;
    P.n_rows = a.n_rows;
    P.lens = a.lens;
    P.delta = a.delta;
    P.n_free = a.n_free;
    P.lens_out = a.lens_out;
    P.table = a.block_table;
    P.free_pages = a.free_pages;
    P.n_free_out = a.n_free_out;
    P.cu = a.cu;
    P.slot = a.slot;
    P.row_req = a.row_req;
    P.row_pos = a.row_pos;
    const size_t smem = 3 * sizeof(int32_t) * ((size_t)a.batch + 1);
    if (smem > 40 * 1024) {
        const cudaError_t e = allow_smem(reinterpret_cast<const void *>(page_plan_kernel), 3 * (int)sizeof(int32_t) * (CSA2P_MAX_BATCH + 1));
        if (e != cudaSuccess) return e;
    }
    // four rows a thread; few rows: one CTA, which needs no second kernel, else clusters of eight
    int64_t ctas = ((int64_t)a.n_rows + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
    if (ctas > device_sm_count()) ctas = device_sm_count();
    const int cluster = ctas > 1 ? 8 : 1;
    ctas = ctas > 1 ? (ctas + cluster - 1) / cluster * cluster : 1;
    const bool later = ctas > 1 && (a.lens_out == a.lens || a.n_free_out == a.n_free);
    const cudaError_t e = launch_pdl(page_plan_kernel, dim3((unsigned)ctas), dim3(kPlanThreads), smem, s, cluster, P, later ? 1 : 0, d_status);
    if (e != cudaSuccess || !later) return e;
    return launch_pdl(page_plan_later_kernel, dim3(1), dim3(kPlanThreads), 0, s, 1, P);
}

cudaError_t launch_paged_rope(const uint16_t *x, int64_t x_row, int64_t x_head, uint16_t *out, int64_t out_row,
                              int64_t out_head, int32_t rows, int32_t heads, int32_t d, const RopeView &rope,
                              uint32_t *d_status, cudaStream_t s)
{
    if (rows == 0 || heads == 0) return cudaSuccess;
    const int first = out == x ? (d - rope.dim) / 8 : 0;
    const int64_t pieces = (int64_t)heads * (d / 8 - first);
    if (pieces == 0) return cudaSuccess;
    const int64_t most = (pieces + 255) / 256, want = (int64_t)device_sm_count() * 8 / rows;
    const int64_t split = want < 1 ? 1 : want > most ? most : want;
    return launch_pdl(paged_rope_kernel, dim3((unsigned)rows, (unsigned)split), dim3(256), 0, s, 1, x, x_row, x_head, out,
                      out_row, out_head, heads, d, first, (int64_t)rows, rope, d_status);
}

cudaError_t launch_paged_write(const PagedView &v, const uint16_t *x, int64_t ldx, int32_t rows, const int32_t *slot,
                               const RopeView &rope, uint32_t *d_status, cudaStream_t s)
{
#define CSA2P_PICK(K, N) (v.fmt == CSA2P_MXFP4 ? K<CSA2P_MXFP4, N> : v.fmt == CSA2P_NVFP4_E4M3_16 ? K<CSA2P_NVFP4_E4M3_16, N> \
                          : v.fmt == CSA2P_MXFP8 ? K<CSA2P_MXFP8, N> : K<CSA2P_BF16, N>)
    auto k = rope.dim == 0 ? CSA2P_PICK(paged_write_kernel, 0) : rope.quads ? CSA2P_PICK(paged_write_kernel, 1) : CSA2P_PICK(paged_write_kernel, 2);
#undef CSA2P_PICK
    return launch_pdl(k, dim3(row_grid(v.d, rows)), row_block(v.d), 0, s, 1, v, x, ldx, rows, slot, rope, d_status);
}

cudaError_t launch_paged_read(const PagedView &v, const int32_t *slot, int32_t rows, uint16_t *out, int64_t ldo,
                              uint32_t *d_status, cudaStream_t s)
{
    auto k = v.fmt == CSA2P_MXFP4 ? paged_read_kernel<CSA2P_MXFP4> : v.fmt == CSA2P_NVFP4_E4M3_16 ? paged_read_kernel<CSA2P_NVFP4_E4M3_16>
             : v.fmt == CSA2P_MXFP8 ? paged_read_kernel<CSA2P_MXFP8> : paged_read_kernel<CSA2P_BF16>;
    return launch_pdl(k, dim3(row_grid(v.d, rows)), row_block(v.d), 0, s, 1, v, slot, rows, out, ldo, kCodeAt0, kCodeAt4, d_status);
}

} // namespace csa2
