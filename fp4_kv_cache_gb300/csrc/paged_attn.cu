// paged_attn.cu -- csa2p_attn on the tensor cores (sm_103a): attention of new tokens over a paged
// latent cache shared by all heads (K = the row, V = its leading d_v dims).
//
// A request's queries are rows (token, head) = token x H + head, taken 64 at a time by a CTA.  Per
// tile of 128 keys, with the keys as the MMA's M dimension,
//   S^T [128 keys x 64 rows]  = K Q^T         (bf16 products, float32 sums, in tensor memory)
//   O^T [512 dims x 64 rows] += V^T P^T       (P = 2^(S - m) in bf16)
// so that the decoded rows, staged once as nine chunks of 64 dims, are K's operand and, read the
// other way, V's.  Chunk pairs go round: while the second product works through the dims in four
// blocks, the staging warps refill the chunks that a block has left, and the first product of the
// next tile follows them chunk by chunk.
//
// Softmax: a thread holds one key and half of the rows, so its logits are its own registers, its
// weights are half of one 128-byte row of P^T, and the weights' sums stay apart per thread until
// the row tile ends.  The maximum that the weights refer to is only moved when a logit exceeds it
// by more than 16 (log2): then, and for a row tile's first keys, it is reduced over the threads
// and O^T is rescaled.  Between moves a weight is at most 2^16: nothing is lost, since weights,
// sums and products are floats.
//
// Decoded rows (paged_decode.cuh) have the eight channels of a 16-byte piece in the order
// 0 4 1 5 2 6 3 7; Q is stored the same way, and the output is put back in order when it is written.
//
// Work is the list of (row tile, key tile) pairs, in equal runs for the GPU's SMs.  A row tile
// cut by the ends of runs leaves parts (O, m, l) in the workspace, which a second kernel joins.
// Every CTA works the list out for itself: no plan has to be made.
//
// Keys past a row tile's bounds, in bad pages or of rows that are not finite are staged as zeros
// and marked, so that what they hold reaches no query that does not see them.
//
// What bounds it.  A tile's two products are 68 MMAs of 128 x 64 x 16, 48 cycles each (the operands'
// way out of shared memory: 4 + 2 KB at 128 bytes a cycle), 3,264 cycles.  A tile takes about 7,000,
// because the staged rows fill the shared memory once (147 KB beside 74 KB of queries) and so the
// parts take turns: the second product's first block, then staging (4,100 cycles for 147 KB by 11
// warps: decoding runs at 52% of the issue slots, and the instruction cache is its next limit), then
// what is left of the first product, then the softmax (1,200).  2 x 1,024 tokens of 64 heads over 15k
// rows of MXFP4 take 5.92 ms: 755 TFLOP/s.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "paged.cuh"
#include "paged_decode.cuh"
#include "tc_util.cuh"

#include <atomic>

namespace csa2 {
namespace {

constexpr int kThreads = 640;           // warps 0-7 softmax, 8 MMA, 9-19 staging
constexpr int kMmaWarp = 8, kStageWarp = 9, kStageWarps = 11, kStageThreads = 32 * kStageWarps;
constexpr int kRing = 3;                // tiles whose rows are looked up: this one and two ahead
constexpr int kRows = 64, kKeys = 128;
constexpr int kQUnit = 8192;            // 64 rows x 64 dims of bf16, 128-byte swizzle
constexpr int kChunk = 16384;           // 128 keys x 64 dims
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 16.0f;          // the maximum moves when a logit is more than this above it
constexpr float kUnset = 1e30f;         // -maximum of a row that has seen no key

// shared memory: Q 9 units | chunks 0..7 | chunk 8, or P^T once S has been computed | the rest
constexpr int kOffK = 9 * kQUnit, kOffP = kOffK + 8 * kChunk, kOffMisc = kOffP + kChunk;

constexpr uint32_t kNoRow = 0xffffffffu;
struct TileAt {                          // a key tile, for everyone
    int64_t row0;                        // its row tile: first row in q, rows, place in lo and hi
    int32_t rows, item;
    int32_t key0;
    uint32_t flags;                      // kFirst ..
    int32_t nt;                          // key tiles of the row tile, over all CTAs
};
constexpr uint32_t kFirst = 1, kLast = 2;     // of this CTA's key tiles of the row tile
constexpr uint32_t kEdge = 4;                 // some row does not see every key
constexpr uint32_t kTail = 8, kPart = 16;     // the row tile began in a CTA before; others have parts of it

struct PartDesc {        // per CTA: the row tile it starts and does not finish
    int32_t parts;       // 0: none
    int32_t rows;
    int64_t row0;
};

struct AttnParams {
    PagedView C;
    int32_t batch, n_tokens, H, d_v, width, window, ratio, chunks, n_pv;
    float log2_scale;
    uint32_t f0, f4;              // see decode
    const uint16_t *q;
    const int32_t *table, *lens, *cu, *pos0, *start;
    uint16_t *out;
    float *lse;
    uint32_t *d_status;
    float *part_o, *part_ml;      // [2 CTAs][64][d_v], [2 CTAs][64][2]
    PartDesc *desc;               // [CTAs]
};

// ------------------------------------------------------------------ PTX
// The descriptors' upper words do not change: a product's two operands are told by their lower
// ones (the address and the leading offset).
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t upper, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %5, 0;\n\t"
                 "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}"
                 ::"r"(d), "r"(a), "r"(b), "r"(upper), "r"(idesc), "r"(acc) : "memory");
}
// What other threads have stored, and this one has seen arrive, comes before its MMAs' reads.  The
// fence stands here and not behind the stores: a staging warp would wait there for its own, about
// 300 cycles each time.
__device__ __forceinline__ void staged_fence()
{
    tc::fence_proxy_async_smem();
    tc::tc_fence_after();
}
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
using tc::mbar_wait;
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, const int32_t *abort)
{
    return mbar_wait(bar, parity, abort);
}
// The same for a warp that stays together: true when every lane has seen the phase.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, const int32_t *abort)
{
#pragma unroll 1
    for (uint32_t i = 0; i < tc::kSpinLimit; ++i) {
        if (__all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity))) return true;
        if ((i & 255u) == 255u && *(const volatile int32_t *)abort) return false;
    }
    return false;
}
// n bytes on their way to the L2 cache; address and n are multiples of 16
__device__ __forceinline__ void prefetch_l2(const void *p, int n)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(n) : "memory");
}
// the warp's largest; NaN counts only where there is nothing else
__device__ __forceinline__ float warp_max(float x)
{
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
// 256 softmax threads: barrier that tells all of them whether one of them says yes
__device__ __forceinline__ bool softmax_any(bool v)
{
    uint32_t any;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                 "barrier.red.or.aligned.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(any) : "r"((uint32_t)v) : "memory");
    return any != 0;
}

__device__ __forceinline__ int sw128(int row, int piece)
{
    return (row >> 3) * 1024 + (row & 7) * 128 + ((piece ^ (row & 7)) << 4);
}
// M = 128, N = 64, bf16 in, float32 sums; which operands lie with M or N contiguous
__device__ __forceinline__ constexpr uint32_t instr(int a_mn, int b_mn)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(kRows >> 3) << 17) | ((uint32_t)(kKeys >> 4) << 24);
}
// Reduces 16 values per thread over a warp by halving; afterwards lane L holds value L / 2.
template <bool MAX>
__device__ __forceinline__ float warp_reduce16(float (&v)[16], int lane)
{
#pragma unroll
    for (int st = 0; st < 4; ++st) {
        const int o = 16 >> st, n = 16 >> st;
        const bool upper = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float send = upper ? v[i] : v[i + n / 2], keep = upper ? v[i + n / 2] : v[i];
            const float recv = __shfl_xor_sync(0xffffffffu, send, o);
            v[i] = MAX ? fmaxf(keep, recv) : keep + recv;
        }
    }
    const float recv = __shfl_xor_sync(0xffffffffu, v[0], 1);
    return MAX ? fmaxf(v[0], recv) : v[0] + recv;
}

// ------------------------------------------------------------------ the work list
struct Item {                 // a row tile
    int32_t b, j;             // request, row tile of it
    int32_t rows;             // rows of the tile (1..64)
    int32_t len;              // rows of the cache that the table can reach
    int64_t row0, p0;         // first row in q; position of the request's first token there
    int32_t lo, hi;           // keys that some row of the tile may see
    int32_t lo_all, hi_all;   // keys that every row of the tile sees
    int32_t nt;               // key tiles, from lo on (at least one, maybe of no key)
    bool more;                // the request has further row tiles
    bool beyond;              // rows past the table may be visible
};

__device__ __forceinline__ void request_tokens(const AttnParams &P, int b, int32_t &first, int32_t &tokens)
{
    const int32_t c0 = min(max(P.cu[b], 0), P.n_tokens), c1 = min(max(P.cu[b + 1], c0), P.n_tokens);
    first = c0;
    tokens = c1 - c0;
}
// Requests that share rows: cu steps down within q.
__device__ __forceinline__ bool steps_down(const AttnParams &P, int b)
{
    return min(max(P.cu[b + 1], 0), P.n_tokens) < min(max(P.cu[b], 0), P.n_tokens);
}
__device__ __forceinline__ int32_t row_tiles(const AttnParams &P, int b)
{
    int32_t f, n;
    request_tokens(P, b, f, n);
    return (int32_t)(((int64_t)n * P.H + kRows - 1) / kRows);
}
// Keys [lo, hi) of the query at position p; none where lo >= hi.  Neither decreases with p.
__device__ __forceinline__ void bounds(const AttnParams &P, int64_t p, int32_t len, int32_t start, int64_t &lo, int32_t &hi, int64_t &end)
{
    // (a position of 2^32 - 1 and up counts as that one; only offsets far below 0 lead there)
    const int64_t e = p < 0 ? 0 : P.ratio == 1 ? p + 1 : (uint32_t)min(p + 1, (int64_t)0xffffffff) / (uint32_t)P.ratio;
    end = e;
    hi = (int32_t)(e < len ? e : len);
    lo = start > 0 ? start : 0;
    if (P.window > 0 && e - P.window > lo) lo = e - P.window;
}
__device__ __noinline__ Item load_item(const AttnParams &P, int b, int j)
{
    Item it;
    it.b = b;
    it.j = j;
    int32_t first, tokens;
    request_tokens(P, b, first, tokens);
    const int64_t left = (int64_t)tokens * P.H - (int64_t)j * kRows;
    it.row0 = (int64_t)first * P.H + (int64_t)j * kRows;
    it.rows = (int32_t)(left < kRows ? left : kRows);
    it.more = left > kRows;
    const int32_t held = max(P.lens[b], 0);
    const int64_t reach = (int64_t)P.width << P.C.shift;
    it.len = (int32_t)(held < reach ? held : reach);
    // Tokens that lie outside q count: those that are left keep their positions.
    const int64_t c0 = P.cu[b];
    it.p0 = (P.pos0 ? (int64_t)P.pos0[b] : held - (P.cu[b + 1] - c0)) + (first - c0);
    const int32_t start = P.start ? P.start[b] : 0;
    const uint32_t r0 = (uint32_t)j * kRows;               // rows of a call are fewer than 2^31
    const uint32_t t0 = r0 / (uint32_t)P.H, t1 = (r0 + it.rows - 1) / (uint32_t)P.H;
    int64_t e0, e1, l0, l1;
    bounds(P, it.p0 + t0, it.len, start, l0, it.hi_all, e0);
    bounds(P, it.p0 + t1, it.len, start, l1, it.hi, e1);
    it.lo = (int32_t)min(l0, (int64_t)it.hi);              // rows before the first query's are not read,
    it.lo_all = (int32_t)min(l1, (int64_t)it.hi);          // even where it sees none itself
    it.beyond = held > it.len && e1 > it.len;
    // The first tile begins with the first key, so that a window of 128 is one tile and not two that
    // begin at multiples of 128 (8 x 256 tokens of 64 heads, MXFP8: 1.6 times as long with two).
    it.nt = it.hi > it.lo ? (it.hi - it.lo - 1) / kKeys + 1 : 1;
    return it;
}

// Walks a CTA's run of (row tile, key tile) units.
struct Walk {
    Item it;
    int32_t off, n;           // this CTA's key tiles of the item: off .. off + n - 1
    int64_t left;             // units of the run after them
    int32_t at;               // tile of the item

    __device__ __forceinline__ void take()
    {
        const int32_t rest = it.nt - off;
        n = left < rest ? (int32_t)left : rest;
        left -= n;
        at = 0;
    }
    __device__ __forceinline__ bool begin(const AttnParams &P, int32_t b, int32_t j, int32_t first, int64_t units)
    {
        left = units;
        if (units <= 0) return false;
        it = load_item(P, b, j);
        off = first;
        take();
        return true;
    }
    // The next key tile; false at the end of the run.
    __device__ __forceinline__ bool next(const AttnParams &P)
    {
        if (++at < n) return true;
        if (left <= 0) return false;
        int b = it.b, j = it.j + 1;
        if (!it.more) {
            j = 0;
            do ++b; while (b < P.batch - 1 && row_tiles(P, b) == 0);
        }
        it = load_item(P, b, j);
        off = 0;
        take();
        return true;
    }
    __device__ __forceinline__ bool first() const { return at == 0; }
    __device__ __forceinline__ bool last() const { return at == n - 1; }
    __device__ __forceinline__ int32_t key0() const { return it.lo + (off + at) * kKeys; }
};

struct Misc {
    uint64_t full_k[5];                 // chunk pairs and chunk 8 staged
    uint64_t s_done, pv_done[4], full_p, rows[kRing], drained;
    uint2 row[kRing][kKeys];            // where a key's row lies: codes / 16 bytes, scales; kNoRow: no key
    TileAt tile[kRing];
    alignas(16) float m[kRows], nm[kRows], fac[kRows];   // maximum (log2), its negative, factor of a move
    float red[4][kRows];
    alignas(16) int32_t lo[4][kRows], hi[4][kRows];      // keys that a row sees, by row tile
    int64_t scan[kThreads / 32];
    int64_t item_unit;                  // first unit of this CTA's first item
    Walk walk[4];                       // of the upper half's warps: two tiles ahead
    uint32_t nan[2][4];                 // keys with a value that is not finite
    int32_t b, j, off;
    uint32_t tmem;
    int32_t abort;
};
constexpr int kSmem = kOffMisc + (int)sizeof(Misc);
static_assert(kSmem <= 232448, "does not fit the shared memory of a CTA");

// Block-wide exclusive sum over the threads.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *buf, int64_t &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    __syncthreads();
    if (lane == 31) buf[warp] = s;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += buf[w];
        all += buf[w];
    }
    total = all;
    return before + s - v;
}

// ------------------------------------------------------------------ the kernel
// FULL: rows of 576 channels with 512 values, so that the chunk counts are constants (windows of 128
// over MXFP8 147 us, a ragged E4M3-scaled step 964, the chunk 5,917; in the general instance 165, 1,020
// and 6,052).
template <int FMT, bool FULL>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_kernel(const __grid_constant__ AttnParams P)
{
    extern __shared__ __align__(1024) uint8_t sm[];
    const int chunks = FULL ? 9 : P.chunks, n_pv = FULL ? 4 : P.n_pv;
    const int n_blocks = FULL ? 18 : P.C.d / 32, pairs = FULL ? 4 : min((chunks + 1) / 2, 4);
    const bool tail = FULL || chunks > 8;             // chunk 8 is there
    Misc &M = *reinterpret_cast<Misc *>(sm + kOffMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x, ctas = gridDim.x;

    if (tid == 0) {
        for (int g = 0; g < 5; ++g) tc::mbar_init(&M.full_k[g], 16);
        for (int j = 0; j < 4; ++j) tc::mbar_init(&M.pv_done[j], 1);
        tc::mbar_init(&M.s_done, 1);
        tc::mbar_init(&M.full_p, 8);
        tc::mbar_init(&M.drained, 1);
        for (int i = 0; i < kRing; ++i) tc::mbar_init(&M.rows[i], 4);
        tc::fence_mbar_init();
        M.abort = 0;
    }
    if (tid < 8) M.nan[tid >> 2][tid & 3] = 0;
    if (warp == kMmaWarp) {
        tc::tmem_alloc(&M.tmem, 512);
        tc::tmem_relinquish();
    }
    pdl_wait();
    pdl_allow_dependents();

    // ---- the work list: row tiles of each request, then their key tiles, summed by all threads
    int64_t total, share;
    {
        int32_t *tiles_before = reinterpret_cast<int32_t *>(sm + kOffK);
        const int per = (P.batch + kThreads - 1) / kThreads;
        const int b0 = min(tid * per, P.batch), b1 = min(b0 + per, P.batch);
        int64_t own = 0, items;
        constexpr int64_t kDown = int64_t(1) << 40;        // more than all the tiles of a call
        for (int b = b0; b < b1; ++b) own += row_tiles(P, b) + (steps_down(P, b) ? kDown : 0);
        int64_t at = block_scan(own, M.scan, items);
        if (items >= kDown) {                              // two CTAs would write the same rows: none is done
            items = 0;
            if (tid == 0 && cta == 0) dev_flag(P.d_status, CSA2_DEV_BAD_INDEX);
        }
        for (int b = b0; b < b1; ++b) {
            tiles_before[b] = (int32_t)at;
            at += row_tiles(P, b);
        }
        if (tid == 0) tiles_before[P.batch] = (int32_t)items;
        __syncthreads();
        const int64_t chunk = (items + kThreads - 1) / kThreads;
        const int64_t i0 = min((int64_t)tid * chunk, items), i1 = min(i0 + chunk, items);
        int rb = 0;
        if (i0 < i1) {                                     // the request of item i0
            int lo = 0, hi = P.batch;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (tiles_before[mid] <= i0) lo = mid;
                else hi = mid;
            }
            rb = lo;
        }
        own = 0;
        int b = rb;
#pragma unroll 1
        for (int64_t i = i0; i < i1; ++i) {
            while (tiles_before[b + 1] <= i) ++b;
            own += load_item(P, b, (int)(i - tiles_before[b])).nt;
        }
        int64_t u = block_scan(own, M.scan, total);
        share = (total + ctas - 1) / ctas;
        const int64_t mine = share * cta;
        if (mine < total && mine >= u && mine < u + own) {  // this thread's items hold the run's start
            b = rb;
#pragma unroll 1
            for (int64_t i = i0; i < i1; ++i) {
                while (tiles_before[b + 1] <= i) ++b;
                const int j = (int)(i - tiles_before[b]), nt = load_item(P, b, j).nt;
                if (mine < u + nt) {
                    M.b = b;
                    M.j = j;
                    M.off = (int32_t)(mine - u);
                    M.item_unit = u;
                    break;
                }
                u += nt;
            }
        }
    }
    const int64_t start = share * cta;
    const int64_t units = start < total ? (start + share < total ? share : total - start) : 0;
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = M.tmem;            // S^T: columns 0..63, O^T block j: 64 + 64 j ..
    if (tid == 0) P.desc[cta].parts = 0;

    if (warp >= kStageWarp) {
        // ============================================================ staging
        // Task (chunk pair, 8 keys): lane (key, q) decodes the q-th scale block of 32 channels of
        // the pair.  A key's four lanes read 64 bytes of its row; so that eight lanes of a store hold
        // eight different columns, the second chunk's blocks start with their upper half.  Warp w
        // takes tasks w, w + 11, .., three a round; the product before is waited for, and what is
        // staged is signalled, between the tasks where that lets the other side start (a signal a
        // round: 7.0 ms where this takes 6.4).  Chunk 8 makes 16 tasks of half the size, spread so
        // that each warp has about the same.  Of 4-bit rows a round's codes of the next tile are on
        // their way as soon as its registers are free; 8- and 16-bit rows are read as they are needed,
        // since a tile ahead they would not fit the registers (MXFP8, 9 x 257 tokens over 4k rows:
        // 1.48 ms, against 1.23).
        const int w = warp - kStageWarp, key8 = lane >> 2, q = lane & 3;
        const bool swap = q >= 2;
        const int j0 = w < 9 ? 6 + w : 3 * (w - 9), jn = w < 9 ? (w == 0 ? 2 : 1) : 3, jstep = w < 9 ? 9 : 1;
        const int lane_code = q * code_bytes<FMT>(32), lane_scale = FMT == CSA2P_NVFP4_E4M3_16 ? 2 * q : q;
        const int place = kOffK + (q >> 1) * kChunk + key8 * 128;
        int col[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) col[i] = ((4 * (q & 1) + (i ^ (swap ? 2 : 0))) ^ key8) << 4;
        bool ok = true;
        constexpr bool kDeep = FMT == CSA2P_MXFP4 || FMT == CSA2P_NVFP4_E4M3_16;   // registers for a tile ahead
        auto live = [&](int task) { return task < 64 && (FULL || (task >> 4) < pairs); };
        const uint8_t *codes = P.C.codes + lane_code, *scales = P.C.scales + lane_scale;
        auto load_task = [&](Raw<FMT, 4> &r, uint2 a, int task) {
            const int cp = task >> 4;
            if (a.x != kNoRow && live(task) && (FULL || 4 * cp + q < n_blocks))
                load_raw(r, codes + (uint64_t)a.x * 16 + cp * code_bytes<FMT>(128), scales + a.y + cp * (FMT == CSA2P_NVFP4_E4M3_16 ? 8 : 4));
            else
                zero_raw(r);
        };
        auto load_round = [&](Raw<FMT, 4> (&r)[3], int ring, int k0) {
            uint2 a[3];
#pragma unroll
            for (int k = 0; k < 3; ++k) a[k] = M.row[ring][8 * ((w + kStageWarps * (k0 + k)) & 15) + key8];
#pragma unroll
            for (int k = 0; k < 3; ++k) load_task(r[k], a[k], w + kStageWarps * (k0 + k));
        };
        Raw<FMT, 2> r8[3];                            // chunk 8
        auto load_tail = [&](int ring) {
            // lane q takes channels 512 + 16 q ..; codes and scales are offset by lane_code, lane_scale
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                if (i >= jn) break;
                const uint2 a = M.row[ring][8 * (j0 + i * jstep) + key8];
                if (a.x != kNoRow && (FULL || 16 + (q >> 1) < n_blocks))
                    load_raw(r8[i], codes + (uint64_t)a.x * 16 - lane_code / 2 + code_bytes<FMT>(512),
                             scales + a.y - lane_scale + (FMT == CSA2P_NVFP4_E4M3_16 ? 32 + q : 16 + (q >> 1)));
                else
                    zero_raw(r8[i]);
            }
        };
        const int c8 = ((2 * q) ^ key8) << 4;
        // A block of the product before has left chunks 2 j, 2 j + 1; blocks are done in order.
        auto left = [&](uint32_t n, int j) {
            if (n > 0) ok = wait_bar(&M.pv_done[min(j, n_pv - 1)], (n - 1) & 1, &M.abort) && ok;
        };
        // Special channels of key group kg, as stored; a key that is not finite is marked.
        auto rest = [&](const auto &r, uint8_t *u, int col0, uint32_t n, int kg) {
            if (mend(r, u, col0)) atomicOr(&M.nan[n & 1][kg >> 2], 1u << (8 * (kg & 3) + key8));
        };
        // tasks w + 11 k for k = k0 .. k0 + K - 1
        auto store_tasks = [&](Raw<FMT, 4> *r, auto count, uint32_t n, int k0) {
            constexpr int K = decltype(count)::value;
            bool odd[K], any = false;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int task = w + kStageWarps * (k0 + k);
                uint32_t v[16];
                swap_raw(r[k], swap);
                decode(r[k], v, P.f0, P.f4);
                odd[k] = special(r[k]) && live(task);
                any |= odd[k];
                uint8_t *u = sm + place + (task >> 4) * 2 * kChunk + (task & 15) * 1024;
                if (live(task))
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<uint4 *>(u + col[i]) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            }
            if (any) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int task = w + kStageWarps * (k0 + k);
                    if (odd[k]) rest(r[k], sm + place + (task >> 4) * 2 * kChunk + (task & 15) * 1024, col[0], n, task & 15);
                }
            }
            __syncwarp();
            if (lane < K && live(w + kStageWarps * (k0 + lane))) tc::mbar_arrive(&M.full_k[(w + kStageWarps * (k0 + lane)) >> 4]);
        };
        auto store_tail = [&](uint32_t n) {
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                if (i >= jn) break;
                const int kg = j0 + i * jstep;
                uint32_t v[8];
                decode(r8[i], v, P.f0, P.f4);
                uint8_t *u = sm + kOffP + kg * 1024 + key8 * 128;
                *reinterpret_cast<uint4 *>(u + c8) = make_uint4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<uint4 *>(u + (c8 ^ 16)) = make_uint4(v[4], v[5], v[6], v[7]);
            }
            bool any = false;
#pragma unroll
            for (int i = 0; i < 3; ++i) any |= i < jn && special(r8[i]);
            if (any) {
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const int kg = j0 + i * jstep;
                    if (i < jn && special(r8[i])) rest(r8[i], sm + kOffP + kg * 1024 + key8 * 128, c8, n, kg);
                }
            }
            __syncwarp();
            if (lane < jn) tc::mbar_arrive(&M.full_k[4]);
        };
        using One = std::integral_constant<int, 1>;
        using Two = std::integral_constant<int, 2>;
        auto first_round = [&](Raw<FMT, 4> (&r)[3], uint32_t n) {
            left(n, 0);
            store_tasks(r, One{}, n, 0);
            left(n, min((w + 2 * kStageWarps) >> 4, pairs - 1));
            store_tasks(r + 1, Two{}, n, 1);
        };
        auto second_round = [&](Raw<FMT, 4> (&r)[3], uint32_t n) {
            left(n, 3);
            store_tasks(r, Two{}, n, 3);
            store_tasks(r + 2, One{}, n, 5);
            if (tail) store_tail(n);
        };
        Raw<FMT, 4> ra[3], rb[3];
        if (units > 0) {
            ok = wait_bar(&M.rows[0], 0, &M.abort);
            if (ok && kDeep) {
                load_round(ra, 0, 0);
                load_round(rb, 0, 3);
            }
        }
        int ring = 0;                                 // n mod kRing, and the parity of the ring's round
        uint32_t round = 0;
#pragma unroll 1
        for (uint32_t n = 0; n < (uint32_t)units; ++n) {
            const bool more = n + 1 < (uint32_t)units;
            const int ring1 = ring == kRing - 1 ? 0 : ring + 1;
            const uint32_t round1 = ring1 == 0 ? round ^ 1 : round;
            if (!__all_sync(0xffffffffu, ok)) break;
            // ---- the queries of a new row tile, once the old ones' last product is done
            if (M.tile[ring].flags & kFirst) {
                if (n > 0) ok = wait_bar(&M.s_done, (n - 1) & 1, &M.abort);
                if (!__all_sync(0xffffffffu, ok)) break;
                const int pieces = FULL ? 72 : P.C.d / 8, all = chunks * 8, rows = M.tile[ring].rows;
                const uint16_t *src = P.q + M.tile[ring].row0 * P.C.d;
                int r = (tid - 32 * kStageWarp) / 72, p = (tid - 32 * kStageWarp) % 72;
#pragma unroll 4
                for (int e = tid - 32 * kStageWarp; e < 64 * 72; e += kStageThreads) {
                    if (FULL || p < all) {
                        uint4 v = make_uint4(0u, 0u, 0u, 0u);
                        if (r < rows && (FULL || p < pieces)) v = *reinterpret_cast<const uint4 *>(src + (FULL ? 8 * e : r * P.C.d + 8 * p));
                        *reinterpret_cast<uint4 *>(sm + (p >> 3) * kQUnit + sw128(r, p & 7)) =
                            make_uint4(prmt(v.x, v.z, 0x5410u), prmt(v.x, v.z, 0x7632u), prmt(v.y, v.w, 0x5410u), prmt(v.y, v.w, 0x7632u));
                    }
                    p += kStageThreads % 72;
                    r += kStageThreads / 72;
                    if (p >= 72) {
                        p -= 72;
                        ++r;
                    }
                }
            }
            if (more) ok = wait_bar(&M.rows[ring1], round1, &M.abort) && ok;
            if (kDeep) {
                if (tail) load_tail(ring);
                first_round(ra, n);
                if (more) load_round(ra, ring1, 0);
                second_round(rb, n);
                if (more) load_round(rb, ring1, 3);
            } else {
                load_round(ra, ring, 0);
                first_round(ra, n);
                load_round(ra, ring, 3);
                if (tail) load_tail(ring);
                second_round(ra, n);
            }
            ring = ring1;
            round = round1;
        }
        if (!ok) M.abort = 1;
    } else if (warp == kMmaWarp) {
        // ============================================================ MMA
        // The whole warp goes through the loops, so that what they compute is the same for all of it
        // and stays in uniform registers; one thread issues.  (With one thread in the loops each MMA
        // took over 100 cycles to issue beside five busy warps, 48 to run.)
        const uint32_t base = tc::smem_u32(sm);
        const uint64_t dk = tc::smem_desc(base + kOffK, 16, 1024, tc::kSwizzle128B);
        const uint64_t dv = tc::smem_desc(base + kOffK, kChunk, 1024, tc::kSwizzle128B);
        const uint32_t upper = (uint32_t)(dk >> 32);      // stride, version, swizzle: the same for all
        const uint32_t k_lo = (uint32_t)dk, v_lo = (uint32_t)dv, q_lo = (uint32_t)tc::smem_desc(base, 16, 1024, tc::kSwizzle128B);
        const uint32_t p_lo = (uint32_t)tc::smem_desc(base + kOffP, kChunk, 1024, tc::kSwizzle128B);
        const bool leader = elect_one();
        bool ok = true;
        int ring = 0;
#pragma unroll 1
        for (uint32_t n = 0; n < (uint32_t)units; ++n) {
            // a pair of chunks as soon as it is staged; nothing but the MMAs between two waits
#pragma unroll 1
            for (int g = 0; 2 * g < chunks; ++g) {
                ok = wait_warp(&M.full_k[g], n & 1, &M.abort);
                if (!ok) break;
                staged_fence();
                if (leader) {
                    for (int c = 2 * g; c < min(2 * g + 2, chunks); ++c) {
                        const uint32_t a = k_lo + c * (kChunk / 16), b = q_lo + c * (kQUnit / 16);
#pragma unroll
                        for (int k = 0; k < 4; ++k) mma(tmem, a + k * 2, b + k * 2, upper, instr(0, 0), c + k != 0);
                    }
                }
            }
            if (!ok) break;
            const uint32_t later = (M.tile[ring].flags & kFirst) == 0;   // read before the softmax may go on
            ring = ring == kRing - 1 ? 0 : ring + 1;
            if (leader) tc::tc_commit(&M.s_done);
            ok = wait_warp(&M.full_p, n & 1, &M.abort);
            if (!ok) break;
            staged_fence();
            if (leader) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j >= n_pv) break;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma(tmem + 64 + 64 * j, v_lo + j * (2 * kChunk / 16) + k * 128, p_lo + k * 128, upper, instr(1, 1), k ? 1 : later);
                    tc::tc_commit(&M.pv_done[j]);
                }
            }
            __syncwarp();
        }
        if (!ok) M.abort = 1;
        __syncwarp();
        if (leader) tc::tc_commit(&M.drained);        // nothing may still run when the CTA leaves
        __syncwarp();
    } else {
        // ============================================================ softmax and output
        // Thread (key, half): the key of its tensor memory lane, rows 32 half .. 32 half + 31.
        const int quad = warp & 3, half = warp >> 2, key_in = 32 * quad + lane, c_lo = 32 * half;
        const uint32_t lane_t = tmem + ((uint32_t)(quad * 32) << 16) + c_lo;
        // The walk lies in shared memory, a copy for each warp that goes it: its 22 words would not
        // fit beside the logits (windows of 128 rows over an MXFP8 cache: 350 -> 326 us).
        Walk &walk = M.walk[quad];
        bool failed = false;
        int ahead_ring = 0, ib = -1;
        // What a tile needs, for everyone: where its keys' rows lie, and at a row tile's start the
        // rows' bounds.
        auto look = [&]() {
            const int32_t key0 = walk.key0();
            const uint32_t k = (uint32_t)key0 + key_in;
            uint2 at = make_uint2(kNoRow, 0u);
            if (k < (uint32_t)walk.it.hi) {
                const int32_t id = P.table[(int64_t)walk.it.b * P.width + (k >> P.C.shift)];
                if (id >= 0 && id < P.C.n_pages) {
                    const uint32_t in = k & ((1u << P.C.shift) - 1);
                    at.x = (uint32_t)((id * P.C.code_page + (int64_t)in * P.C.code_row) >> 4);
                    at.y = (uint32_t)(id * P.C.scale_page + (int64_t)in * P.C.scale_row);
                } else {
                    dev_flag(P.d_status, CSA2_DEV_BAD_INDEX);
                }
            }
            M.row[ahead_ring][key_in] = at;
            if (walk.first()) {
                ++ib;
                if (key_in < kRows) {                 // rows past the last: as the last
                    int32_t hi;
                    int64_t lo, e;
                    const uint32_t f = (uint32_t)walk.it.j * kRows + min(key_in, walk.it.rows - 1);
                    bounds(P, walk.it.p0 + f / (uint32_t)P.H, walk.it.len, P.start ? P.start[walk.it.b] : 0, lo, hi, e);
                    M.lo[ib & 3][key_in] = (int32_t)min(lo, (int64_t)hi);
                    M.hi[ib & 3][key_in] = hi;
                    if (walk.it.beyond && min((int64_t)P.lens[walk.it.b], e) > max((int64_t)walk.it.len, lo))
                        dev_flag(P.d_status, CSA2_DEV_BAD_INDEX);
                }
                if (key_in == 0) {
                    prefetch_l2(P.q + walk.it.row0 * P.C.d, walk.it.rows * P.C.d * 2);
                }
            }
            if (key_in == 0) {
                TileAt t;
                t.row0 = walk.it.row0;
                t.rows = walk.it.rows;
                t.item = ib & 3;
                t.key0 = key0;
                t.nt = walk.it.nt;
                t.flags = (walk.first() ? kFirst : 0) | (walk.last() ? kLast : 0) |
                          (key0 < walk.it.lo_all || key0 > walk.it.hi_all - kKeys ? kEdge : 0) | (walk.off > 0 ? kTail : 0) |
                          (walk.off > 0 || walk.off + walk.n < walk.it.nt ? kPart : 0);
                M.tile[ahead_ring] = t;
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&M.rows[ahead_ring]);
            ahead_ring = ahead_ring == kRing - 1 ? 0 : ahead_ring + 1;
        };
        bool more = false;                            // the walk has a tile that is not looked up yet
        auto go_on = [&]() {                          // after look
            __syncwarp();
            bool on = false;
            if (lane == 0) on = walk.next(P);
            __syncwarp();
            more = __any_sync(0xffffffffu, on);
        };
        if (half == 1) {
            if (lane == 0) more = walk.begin(P, M.b, M.j, M.off, units);
            __syncwarp();
            more = __any_sync(0xffffffffu, more);
            if (more) {
                look();
                go_on();
            }
            if (more) {
                look();
                go_on();
            }
        }
        float l[32];                                  // sums of weights: this thread's key in each tile
        int64_t unit = M.item_unit;                   // first unit of the item
        int ring = 0;
        uint32_t round = 0;
#pragma unroll 1
        for (uint32_t n = 0; n < (uint32_t)units; ++n) {
            const uint32_t ph = n & 1;
            failed |= __any_sync(0xffffffffu, !wait_bar(&M.rows[ring], round, &M.abort));
            const TileAt &T = M.tile[ring];
            const uint32_t flags = T.flags;
            const bool first = flags & kFirst, have = M.row[ring][key_in].x != kNoRow;
            if (first) {
                if (half == 0 && key_in < kRows) {
                    M.m[key_in] = -INFINITY;
                    M.nm[key_in] = kUnset;
                }
#pragma unroll
                for (int c = 0; c < 32; ++c) l[c] = 0.0f;
            }
            if (half == 1 && more) {
                // a tile looked up two ahead takes the place of the one before this one, whose staging
                // and softmax are done
                look();
                go_on();
            }
            failed |= __any_sync(0xffffffffu, !wait_bar(&M.full_k[tail ? 4 : pairs - 1], ph, &M.abort));
            const bool nan = (M.nan[ph][quad] >> lane) & 1u;
            const bool masked = (flags & kEdge) || __any_sync(0xffffffffu, nan || !have);
            failed |= __any_sync(0xffffffffu, !wait_bar(&M.s_done, ph, &M.abort));
            tc::tc_fence_after();
            // ---- logits that a row does not see become -inf, those of a key that is not finite NaN
            if (masked) {
                const int32_t key = (int32_t)((uint32_t)T.key0 + key_in), item = T.item;
#pragma unroll 1
                for (int c0 = 0; c0 < 32; c0 += 16) {
                    uint32_t r[16];
                    tc::tc_ld_32x32b_x16(lane_t + c0, r);
                    tc::tc_wait_ld();
#pragma unroll
                    for (int c = 0; c < 16; c += 4) {
                        const int4 lo = *reinterpret_cast<const int4 *>(&M.lo[item][c_lo + c0 + c]);
                        const int4 hi = *reinterpret_cast<const int4 *>(&M.hi[item][c_lo + c0 + c]);
                        auto seen = [&](uint32_t x, int l, int h) { return !(have && key >= l && key < h) ? 0xff800000u : nan ? 0x7fc00000u : x; };
                        r[c] = seen(r[c], lo.x, hi.x);
                        r[c + 1] = seen(r[c + 1], lo.y, hi.y);
                        r[c + 2] = seen(r[c + 2], lo.z, hi.z);
                        r[c + 3] = seen(r[c + 3], lo.w, hi.w);
                    }
                    tc::tc_st_32x32b_x16(lane_t + c0, r);
                }
                tc::tc_wait_st();
            }
            bool moved = first;
#pragma unroll 1
            while (true) {
                if (moved) {
                    // ---- new maxima, reduced over the keys
                    if (softmax_any(failed)) { failed = true; break; }
                    {
                        uint32_t r[32];
                        tc::tc_ld_32x32b_x32(lane_t, r);
                        tc::tc_wait_ld();
                        float top = -INFINITY;
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            const float x = warp_max(__uint_as_float(r[c]) * P.log2_scale);
                            top = lane == c ? x : top;
                        }
                        M.red[quad][c_lo + lane] = top;
                    }
                    softmax_any(false);
                    if (tid < kRows) {
                        const float top = fmaxf(fmaxf(M.red[0][tid], M.red[1][tid]), fmaxf(M.red[2][tid], M.red[3][tid])), m = M.m[tid];
                        float f = 1.0f;
                        if (top > m + kLazy || (m == -INFINITY && top > -INFINITY)) {
                            f = ex2(m - top);         // 0 for the first maximum
                            M.m[tid] = top;
                            M.nm[tid] = -top;
                        }
                        M.fac[tid] = f;
                    }
                    softmax_any(false);
                    if (!first) {
#pragma unroll
                        for (int c = 0; c < 32; ++c) l[c] *= M.fac[c_lo + c];
                        failed |= __any_sync(0xffffffffu, !wait_bar(&M.pv_done[n_pv - 1], ph ^ 1, &M.abort));
                        tc::tc_fence_after();
#pragma unroll 1
                        for (int j = 0; j < n_pv && !failed; ++j)
#pragma unroll 1
                            for (int c0 = 0; c0 < 32; c0 += 16) {
                                uint32_t o[16];
                                tc::tc_ld_32x32b_x16(lane_t + 64 + 64 * j + c0, o);
                                tc::tc_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * M.fac[c_lo + c0 + i]);
                                tc::tc_st_32x32b_x16(lane_t + 64 + 64 * j + c0, o);
                            }
                        tc::tc_wait_st();
                    }
                }
                // ---- weights: their bf16 values go to P^T; their sums stay in the thread
                uint32_t r[32], p[16];
                tc::tc_ld_32x32b_x32(lane_t, r);
                tc::tc_wait_ld();
                float over = -INFINITY;
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                    const float x = fmaf(__uint_as_float(r[c]), P.log2_scale, M.nm[c_lo + c]);
                    const float y = fmaf(__uint_as_float(r[c + 1]), P.log2_scale, M.nm[c_lo + c + 1]);
                    over = fmaxf(over, fmaxf(x, y));
                    const float ex = ex2(x), ey = ex2(y);
                    r[c] = __float_as_uint(ex);
                    r[c + 1] = __float_as_uint(ey);
                    const __nv_bfloat162 b = __floats2bfloat162_rn(ex, ey);
                    p[c / 2] = *reinterpret_cast<const uint32_t *>(&b);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<uint4 *>(sm + kOffP + sw128(key_in, 4 * half + i)) = make_uint4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
                // a logit far above its row's maximum: once more, with the maximum moved
                if (softmax_any(failed || (!moved && over > kLazy))) {
                    if (moved) { failed = true; break; }
                    moved = true;
                    continue;
                }
                tc::tc_fence_before();
                if (tid < 4) M.nan[ph][tid] = 0;
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&M.full_p);
#pragma unroll
                for (int c = 0; c < 32; ++c) l[c] += __uint_as_float(r[c]);
                break;
            }
            if (failed) break;
            if (flags & kLast) {
                // ---- output, or a part of it: sums over the keys, then a lane has one dim of every row
                const int rows = T.rows;
                const int64_t row0 = T.row0;
                const bool part = flags & kPart;
                const int32_t nt = T.nt;
#pragma unroll
                for (int c0 = 0; c0 < 32; c0 += 16) {
                    float v[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) v[c] = l[c0 + c];
                    const float sum = warp_reduce16<false>(v, lane);
                    if ((lane & 1) == 0) M.red[quad][c_lo + c0 + (lane >> 1)] = sum;
                }
                failed |= __any_sync(0xffffffffu, !wait_bar(&M.pv_done[n_pv - 1], ph, &M.abort));
                if (softmax_any(failed)) { failed = true; break; }
                tc::tc_fence_after();
                const int64_t slot = (2 * (int64_t)cta + ((flags & kTail) ? 0 : 1)) * kRows;
                if (tid < kRows) {
                    const float s = (M.red[0][tid] + M.red[1][tid]) + (M.red[2][tid] + M.red[3][tid]), m = M.m[tid];
                    M.fac[tid] = s == 0.0f ? 0.0f : 1.0f / s;
                    if (part) {
                        P.part_ml[(slot + tid) * 2] = m;
                        P.part_ml[(slot + tid) * 2 + 1] = s;
                    } else if (tid < rows && P.lse) {
                        P.lse[row0 + tid] = s == 0.0f ? -INFINITY : (m + log2f(s)) * kLn2;
                    }
                    if (part && !(flags & kTail) && tid == 0) {
                        PartDesc d;
                        d.parts = (int32_t)((unit + nt - 1) / share - cta + 1);
                        d.rows = rows;
                        d.row0 = row0;
                        P.desc[cta] = d;
                    }
                }
                softmax_any(false);
                // A lane has one dim of 16 rows.  Parts are stored like that, in the dims' order; an output
                // is packed in pairs of rows and turned over between the eight lanes of a 16-byte piece.
                const int dim_in = (key_in & ~7) | ((key_in & 1) << 2) | ((key_in & 7) >> 1), t = lane & 7;
#pragma unroll 1
                for (int i = 0; i < 2 * n_pv; ++i) {
                    const int r0 = c_lo + 16 * (i & 1), dim0 = 128 * (i >> 1);
                    if (r0 >= rows) continue;
                    uint32_t o[16], v[8];
                    tc::tc_ld_32x32b_x16(lane_t + 64 + 64 * (i >> 1) + 16 * (i & 1), o);
                    tc::tc_wait_ld();
                    if (part) {
                        float *to = P.part_o + (slot + r0) * P.d_v + dim0 + dim_in;
                        if (dim0 + dim_in < P.d_v)
#pragma unroll
                            for (int c = 0; c < 16; ++c) to[(int64_t)c * P.d_v] = __uint_as_float(o[c]);
                        continue;
                    }
#pragma unroll
                    for (int c = 0; c < 16; c += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(&M.fac[r0 + c]);
                        const __nv_bfloat162 x = __floats2bfloat162_rn(__uint_as_float(o[c]) * f.x, __uint_as_float(o[c + 1]) * f.y);
                        const __nv_bfloat162 y = __floats2bfloat162_rn(__uint_as_float(o[c + 2]) * f.z, __uint_as_float(o[c + 3]) * f.w);
                        v[c / 2] = *reinterpret_cast<const uint32_t *>(&x);
                        v[c / 2 + 1] = *reinterpret_cast<const uint32_t *>(&y);
                    }
#pragma unroll
                    for (int st = 4; st; st >>= 1) {
                        const bool up = (lane & st) != 0;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            if (k & st) continue;
                            const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? v[k] : v[k | st], st);
                            if (up) v[k] = got;
                            else v[k | st] = got;
                        }
                    }
                    // v[k]: rows r0 + 2 t, r0 + 2 t + 1 of the dim that place k stands for
                    uint16_t *to = P.out + (row0 + r0 + 2 * t) * P.d_v + dim0 + (key_in & ~7);
                    if (dim0 + (key_in & ~7) < P.d_v) {
                        if (r0 + 2 * t < rows)
                            *reinterpret_cast<uint4 *>(to) =
                                make_uint4(prmt(v[0], v[2], 0x5410u), prmt(v[4], v[6], 0x5410u), prmt(v[1], v[3], 0x5410u), prmt(v[5], v[7], 0x5410u));
                        if (r0 + 2 * t + 1 < rows)
                            *reinterpret_cast<uint4 *>(to + P.d_v) =
                                make_uint4(prmt(v[0], v[2], 0x7632u), prmt(v[4], v[6], 0x7632u), prmt(v[1], v[3], 0x7632u), prmt(v[5], v[7], 0x7632u));
                    }
                }
                tc::tc_fence_before();
                unit += nt;
            }
            ring = ring == kRing - 1 ? 0 : ring + 1;
            round ^= ring == 0;
        }
        if (failed) M.abort = 1;
    }
    __syncthreads();
    if (tid == 0 && (!tc::mbar_wait_bounded(&M.drained, 0) || M.abort)) dev_flag(P.d_status, CSA2_DEV_TIMEOUT);
    tc::tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

// Joins the parts of cut row tiles: o = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.  A warp takes
// a row; blockIdx.x = the CTA that began the row tile, whose part is its second slot and whose
// further parts are the first slots of the CTAs after it.
__global__ void __launch_bounds__(256) paged_attn_join_kernel(const __grid_constant__ AttnParams P)
{
    pdl_wait();
    pdl_allow_dependents();
    const PartDesc d = P.desc[blockIdx.x];
    if (d.parts <= 0) return;
    const int lane = threadIdx.x & 31;
    for (int row = blockIdx.y * 8 + (threadIdx.x >> 5); row < d.rows; row += 8 * gridDim.y) {
        auto slot = [&](int i) -> int64_t { return i == 0 ? 2 * (int64_t)blockIdx.x + 1 : 2 * ((int64_t)blockIdx.x + i); };
        float top = -INFINITY;
        for (int i = lane; i < d.parts; i += 32) top = fmaxf(top, P.part_ml[(slot(i) * kRows + row) * 2]);
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float base = top == -INFINITY ? 0.0f : top;
        float l = 0.0f;
        for (int i = lane; i < d.parts; i += 32) {
            const float *ml = P.part_ml + (slot(i) * kRows + row) * 2;
            l += ex2(ml[0] - base) * ml[1];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int64_t grow = d.row0 + row;
        for (int c = 4 * lane; c < P.d_v; c += 128) {
            float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
            for (int i = 0; i < d.parts; ++i) {
                const int64_t at = slot(i) * kRows + row;
                const float f = ex2(P.part_ml[at * 2] - base);
                const float4 v = *reinterpret_cast<const float4 *>(P.part_o + at * P.d_v + c);
                a.x = fmaf(f, v.x, a.x);
                a.y = fmaf(f, v.y, a.y);
                a.z = fmaf(f, v.z, a.z);
                a.w = fmaf(f, v.w, a.w);
            }
            const __nv_bfloat162 x = __floats2bfloat162_rn(a.x * inv, a.y * inv), y = __floats2bfloat162_rn(a.z * inv, a.w * inv);
            *reinterpret_cast<uint2 *>(P.out + grow * P.d_v + c) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
        }
        if (lane == 0 && P.lse) P.lse[grow] = l == 0.0f ? -INFINITY : (top + log2f(l)) * kLn2;
    }
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

} // namespace

cudaError_t allow_smem(const void *kernel, int bytes)
{
    constexpr int kMaxDevices = 64, kKernels = 12;
    static std::atomic<const void *> done[kMaxDevices][kKernels];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < kMaxDevices;
    if (known)
        for (int i = 0; i < kKernels; ++i)
            if (done[dev][i].load(std::memory_order_acquire) == kernel) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess || !known) return e;
    for (int i = 0; i < kKernels; ++i) {
        const void *none = nullptr;
        if (done[dev][i].compare_exchange_strong(none, kernel, std::memory_order_acq_rel) || none == kernel) break;
    }
    return cudaSuccess;
}

namespace {

template <bool FULL>
auto attn_kernel(int fmt) -> void (*)(AttnParams)
{
    switch (fmt) {
    case CSA2P_MXFP4: return paged_attn_kernel<CSA2P_MXFP4, FULL>;
    case CSA2P_NVFP4_E4M3_16: return paged_attn_kernel<CSA2P_NVFP4_E4M3_16, FULL>;
    case CSA2P_MXFP8: return paged_attn_kernel<CSA2P_MXFP8, FULL>;
    default: return paged_attn_kernel<CSA2P_BF16, FULL>;
    }
}

} // namespace

size_t paged_attn_ws_bytes(const csa2p_attn_args &a)
{
    const size_t ctas = device_sm_count(), rows = 2 * ctas * kRows;
    return up256(rows * a.d_v * sizeof(float)) + up256(rows * 2 * sizeof(float)) + up256(ctas * sizeof(PartDesc));
}

cudaError_t launch_paged_attn(const csa2p_attn_args &a, const PagedView &v, uint16_t *out, float *lse, void *ws,
                              uint32_t *d_status, cudaStream_t s)
{
    const int ctas = device_sm_count();
    AttnParams P;
    P.C = v;
    P.batch = a.batch;
    P.n_tokens = a.n_tokens;
    P.H = a.n_heads;
    P.d_v = a.d_v;
    P.width = a.width;
    P.window = a.window;
    P.ratio = a.ratio_m;
    P.chunks = (v.d + 63) / 64;
    P.n_pv = (a.d_v + 127) / 128;
    P.log2_scale = a.sm_scale * 1.4426950408889634f;
    P.f0 = kCodeAt0;
    P.f4 = kCodeAt4;
    P.q = a.q;
    P.table = a.block_table;
    P.lens = a.lens;
    P.cu = a.cu;
    P.pos0 = a.pos0;
    P.start = a.kv_start;
    P.out = out;
    P.lse = lse;
    P.d_status = d_status;
    const size_t rows = 2 * (size_t)ctas * kRows;
    char *w = static_cast<char *>(ws);
    P.part_o = reinterpret_cast<float *>(w);
    w += up256(rows * a.d_v * sizeof(float));
    P.part_ml = reinterpret_cast<float *>(w);
    w += up256(rows * 2 * sizeof(float));
    P.desc = reinterpret_cast<PartDesc *>(w);
    void (*k)(AttnParams) = v.d == 576 && a.d_v == 512 ? attn_kernel<true>(v.fmt) : attn_kernel<false>(v.fmt);
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(k), kSmem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(k, dim3((unsigned)ctas), dim3(kThreads), (size_t)kSmem, s, 1, P);
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_attn_join_kernel, dim3((unsigned)ctas, kRows / 8), dim3(256), 0, s, 1, P);
}

} // namespace csa2
