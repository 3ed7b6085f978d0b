// paged_attn.cu -- csa2p_attn on the tensor cores (sm_103a): attention of new tokens over a paged
// latent cache shared by all heads (K = the row, V = its leading d_v dims).
//
// A request's queries are rows (token, head) = token x H + head, taken 128 at a time by a cluster
// of two CTAs (cta_group::2, M = 128): each CTA owns 64 rows.  Per tile of 128 keys
//   S [128 rows x 128 keys]  = Q K^T        (bf16 products, float32 sums, in tensor memory)
//   O [128 rows x 512 dims] += P V          (P = 2^(S - m) in bf16)
// Each CTA stages the 64 keys of its half: decoded once, they serve the whole pair as B operand
// of S.  The B operand of O wants all 128 keys but only half of the dims in each CTA; its own
// keys' rows are in place, the peer's keys' own-dims chunks are decoded over chunks that S no
// longer needs.  So shared memory takes 104 KB of staging a tile instead of 2 x 147 KB, and the
// MMA's operand reads halve too: staging and MMA both live off shared memory's 128 B a cycle.
//
// Decoding a 4-bit code: bits s e e m of a code placed as bf16's sign, two exponent and one
// mantissa bit are the code's value x 2^-126 (subnormals included), so one bf16 product with
// 2^126 x scale gives the exact value.  To save shifts the two values of a register are nibbles k
// and k + 4 of a word: the eight channels of a 16-byte piece stand as 0 4 1 5 2 6 3 7, in Q the
// same way, and the output's columns are put back in order when they are written.
//
// Work is the list of (row tile, key tile) pairs, in equal runs for the clusters that fit the
// GPU.  A row tile cut by the ends of runs leaves parts (O, m, l) in the workspace, which
// a second kernel joins.  Every CTA works the list out for itself: no plan has to be made.
//
// Keys past a row's bounds, in bad pages or of rows that are not finite are staged as zeros
// and marked, so that what they hold reaches no query that does not see them.
#include "common.cuh"
#include "internal.h"
#include "paged.cuh"
#include "tc_util.cuh"

#include <cuda_bf16.h>

#include <atomic>

namespace csa2 {
namespace {

constexpr int kThreads = 512;           // warps 0-3 softmax, 4 MMA, 8-15 staging
constexpr int kStageWarp = 8, kStageThreads = 256;
constexpr int kRows = 128, kKeys = 128; // of a pair
constexpr int kUnit = 8192;             // 64 rows x 64 dims of bf16, 128-byte swizzle
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.0f;           // O is rescaled when a maximum grows by more than 2^8

// shared memory: Q 9 units | K stage 0, 1: chunks 0..7 | chunk 8 | P 2 units | the rest
constexpr int kOffK = 9 * kUnit, kOffR = kOffK + 16 * kUnit, kOffP = kOffR + kUnit, kOffMisc = kOffP + 2 * kUnit;

struct Misc {
    uint64_t full_k[2][3], full_z[2], full_p;   // the leader's: staged, probabilities written
    uint64_t s_done[2], pv_done[2], info[2];    // each CTA's
    uint64_t drained;
    uint64_t valid[2][2], nan[2][2];            // [stage][half]: keys there, keys not finite
    float top[2][2][64], sum[2][64];            // exchange between the halves of a row
    int64_t scan[32];
    int64_t start_unit, total, item_unit;       // this cluster's first unit; its item's first unit
    int32_t b, j, off;
    uint32_t tmem;
    int32_t abort;
};
constexpr int kSmem = kOffMisc + (int)sizeof(Misc);
static_assert(kSmem <= 232448, "does not fit the shared memory of a CTA");

struct PartDesc {        // per cluster: the item it starts and does not finish
    int32_t parts;       // 0: none
    int32_t rows;
    int64_t row0;
};

struct AttnParams {
    PagedView C;
    int32_t batch, n_tokens, H, d_v, width, window, ratio, chunks, v_chunks, n_pv;
    float log2_scale;
    const uint16_t *q;
    const int32_t *table, *lens, *cu, *pos0, *start;
    uint16_t *out;
    float *lse;
    uint32_t *d_status;
    float *part_o, *part_ml;      // [2 clusters][128][d_v], [2 clusters][128][2]
    PartDesc *desc;               // [clusters]
};

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_peer(uint32_t local, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}
__device__ __forceinline__ void arrive_at(const uint64_t *bar, uint32_t rank)   // CTA `rank`'s barrier
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];"
                 ::"r"(map_peer(tc::smem_u32(bar), rank)) : "memory");
}
__device__ __forceinline__ void st_peer_u8(const void *local, uint32_t rank, uint32_t v)
{
    asm volatile("st.shared::cluster.u8 [%0], %1;" ::"r"(map_peer(tc::smem_u32(local), rank)), "r"(v) : "memory");
}
// Bounded wait that also sees what the peer CTA released.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, const int32_t *abort)
{
#pragma unroll 1
    for (uint32_t i = 0; i < tc::kSpinLimit; ++i) {
        uint32_t ok;
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(tc::smem_u32(bar)), "r"(parity) : "memory");
        if (ok) return true;
        if ((i & 255u) == 255u && *(const volatile int32_t *)abort) return false;
    }
    return false;
}
__device__ __forceinline__ void mma2(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void commit2(uint64_t *bar)         // arrives at both CTAs' barrier
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(tc::smem_u32(bar)), "h"((uint16_t)3) : "memory");
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel)
{
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}
// 128 softmax threads: barrier that tells all of them whether any has failed
__device__ __forceinline__ bool softmax_sync(bool failed)
{
    uint32_t any;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                 "barrier.red.or.aligned.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(any) : "r"((uint32_t)failed) : "memory");
    return any != 0;
}

__device__ __forceinline__ int sw128(int row, int piece)
{
    return (row >> 3) * 1024 + (row & 7) * 128 + ((piece ^ (row & 7)) << 4);
}
__device__ __forceinline__ constexpr uint32_t instr(int n, int b_mn)   // M = 128, bf16 in, float32 sums
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

// ------------------------------------------------------------------ decoding
__device__ __forceinline__ __nv_bfloat162 bf2(uint32_t half)
{
    const __nv_bfloat16 h = __ushort_as_bfloat16((unsigned short)half);
    return __halves2bfloat162(h, h);
}
__device__ __forceinline__ uint32_t mul2(uint32_t v, __nv_bfloat162 m)
{
    const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&v), m);
    return *reinterpret_cast<const uint32_t *>(&x);
}

// Sixteen channels of a row as they lie in the cache, and their scale byte.
template <int FMT>
struct Raw {
    static constexpr int kWords = FMT == CSA2P_BF16 ? 8 : FMT == CSA2P_MXFP8 ? 4 : 2;
    uint32_t w[kWords];
    uint32_t sb;
};

template <int FMT>
__device__ __forceinline__ void load_raw(Raw<FMT> &r, const uint8_t *codes, const uint8_t *scales, int part)
{
    // part: which 16 channels of the row
    if (FMT == CSA2P_BF16) {
        const uint4 a = reinterpret_cast<const uint4 *>(codes)[2 * part], b = reinterpret_cast<const uint4 *>(codes)[2 * part + 1];
        r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
        r.w[4 % Raw<FMT>::kWords] = b.x; r.w[5 % Raw<FMT>::kWords] = b.y; r.w[6 % Raw<FMT>::kWords] = b.z; r.w[7 % Raw<FMT>::kWords] = b.w;
        r.sb = 0;
    } else if (FMT == CSA2P_MXFP8) {
        const uint4 a = reinterpret_cast<const uint4 *>(codes)[part];
        r.w[0] = a.x; r.w[1] = a.y; r.w[2 % Raw<FMT>::kWords] = a.z; r.w[3 % Raw<FMT>::kWords] = a.w;
        r.sb = scales[part >> 1];
    } else {
        const uint2 a = reinterpret_cast<const uint2 *>(codes)[part];
        r.w[0] = a.x; r.w[1] = a.y;
        r.sb = FMT == CSA2P_NVFP4_E4M3_16 ? scales[part] : scales[part >> 1];
    }
}
template <int FMT>
__device__ __forceinline__ void zero_raw(Raw<FMT> &r)
{
#pragma unroll
    for (int i = 0; i < Raw<FMT>::kWords; ++i) r.w[i] = 0u;
    r.sb = FMT == CSA2P_NVFP4_E4M3_16 ? 0u : 127u;
}

// Two 16-byte pieces (channels 0-7 and 8-15 in the order 0 4 1 5 2 6 3 7) of bf16.  Returns whether
// a value or the scale is not finite; the pieces are then zero.  Scale bytes that would take a
// product out of range (no quantised row has them) count as not finite.
template <int FMT>
__device__ __forceinline__ bool decode(const Raw<FMT> &r, uint4 (&o)[2])
{
    uint32_t v[8];
    bool bad = false;
    if (FMT == CSA2P_BF16) {
        uint32_t e = 0;
#pragma unroll
        for (int i = 0; i < Raw<FMT>::kWords; ++i) e |= ((r.w[i] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
        bad = e != 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                v[4 * h + 2 * k] = prmt(r.w[(4 * h + k) % Raw<FMT>::kWords], r.w[(4 * h + k + 2) % Raw<FMT>::kWords], 0x5410u);
                v[4 * h + 2 * k + 1] = prmt(r.w[(4 * h + k) % Raw<FMT>::kWords], r.w[(4 * h + k + 2) % Raw<FMT>::kWords], 0x7632u);
            }
    } else if (FMT == CSA2P_MXFP8) {
        // code bits as bf16 bits: value x 2^-120; x 2^(120 + sb - 127), in two products for large scales
        uint32_t e = 0;
#pragma unroll
        for (int i = 0; i < Raw<FMT>::kWords; ++i) e |= ((r.w[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
        bad = e != 0 || r.sb >= 247u;
        const __nv_bfloat162 m = bf2((min(r.sb, 134u) + 120u) << 7);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t a = prmt(r.w[(2 * h) % Raw<FMT>::kWords], r.w[(2 * h + 1) % Raw<FMT>::kWords], 0x4400u + 0x1111u * k);
                v[4 * h + k] = mul2((a & 0x80008000u) | ((a >> 4) & 0x07f007f0u), m);
            }
        if (r.sb > 134u) {
            const __nv_bfloat162 m2 = bf2((min(r.sb, 246u) - 134u + 127u) << 7);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = mul2(v[i], m2);
        }
    } else {
        const bool nv = FMT == CSA2P_NVFP4_E4M3_16;
        // E8M0: x 2^(126 + sb - 127); E4M3: x 2^126, then the scale (both products exact)
        const __nv_bfloat162 m = nv ? bf2(253u << 7) : bf2((min(r.sb, 128u) + 126u) << 7);
        bad = nv ? (r.sb & 0x7fu) == 0x7fu : r.sb >= 253u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t w = r.w[h];
            v[4 * h] = mul2(((w << 12) & 0x80008000u) | ((w << 6) & 0x01c001c0u), m);
            v[4 * h + 1] = mul2(((w << 8) & 0x80008000u) | ((w << 2) & 0x01c001c0u), m);
            v[4 * h + 2] = mul2(((w << 4) & 0x80008000u) | ((w >> 2) & 0x01c001c0u), m);
            v[4 * h + 3] = mul2((w & 0x80008000u) | ((w >> 6) & 0x01c001c0u), m);
        }
        if (nv) {
            const uint32_t bits = ((r.sb & 0x80u) << 8) | ((r.sb & 0x7fu) << 4);       // the scale x 2^-120
            const uint32_t sc = mul2(bits | (bits << 16), bf2(247u << 7));
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = mul2(v[i], *reinterpret_cast<const __nv_bfloat162 *>(&sc));
        } else if (r.sb > 128u) {
            const __nv_bfloat162 m2 = bf2((min(r.sb, 252u) - 128u + 127u) << 7);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = mul2(v[i], m2);
        }
    }
    if (bad) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0u;
    }
    o[0] = make_uint4(v[0], v[1], v[2], v[3]);
    o[1] = make_uint4(v[4], v[5], v[6], v[7]);
    return bad;
}

// ------------------------------------------------------------------ the work list
struct Item {                 // a row tile
    int32_t b, j;             // request, row tile of it
    int32_t first, tokens;    // its tokens in q
    int32_t rows;             // rows of the tile (1..128)
    int32_t len;              // rows of the cache that the table can reach
    int64_t p0;               // position of token 0
    int32_t lo, hi;           // keys that some row of the tile may see
    int32_t k0, nt;           // key tiles k0 .. k0 + nt - 1 (at least one, maybe of no key)
    bool beyond;              // some visible row lies past the table

    __device__ __forceinline__ int64_t row0(int H) const { return (int64_t)first * H + (int64_t)j * kRows; }
};

__device__ __forceinline__ void request_tokens(const AttnParams &P, int b, int32_t &first, int32_t &tokens)
{
    const int32_t c0 = min(max(P.cu[b], 0), P.n_tokens), c1 = min(max(P.cu[b + 1], c0), P.n_tokens);
    first = c0;
    tokens = c1 - c0;
}
__device__ __forceinline__ int32_t row_tiles(const AttnParams &P, int b)
{
    int32_t f, n;
    request_tokens(P, b, f, n);
    return (int32_t)(((int64_t)n * P.H + kRows - 1) / kRows);
}
// Keys [lo, hi) of the query at position p.
__device__ __forceinline__ void bounds(const AttnParams &P, int64_t p, int32_t len, int32_t start, int32_t &lo, int32_t &hi, int64_t &end)
{
    const int64_t e = p < 0 ? 0 : P.ratio == 1 ? p + 1 : (uint32_t)(p + 1) / (uint32_t)P.ratio;   // p + 1 < 2^32
    end = e;
    hi = (int32_t)(e < len ? e : len);
    int64_t l = start > 0 ? start : 0;
    if (P.window > 0 && e - P.window > l) l = e - P.window;
    lo = (int32_t)(l < hi ? l : hi);
}
__device__ __forceinline__ void load_item(const AttnParams &P, int b, int j, Item &it)
{
    it.b = b;
    it.j = j;
    request_tokens(P, b, it.first, it.tokens);
    const int64_t total = (int64_t)it.tokens * P.H;
    it.rows = (int32_t)(total - (int64_t)j * kRows < kRows ? total - (int64_t)j * kRows : kRows);
    const int32_t held = max(P.lens[b], 0);
    const int64_t reach = (int64_t)P.width << P.C.shift;
    it.len = (int32_t)(held < reach ? held : reach);
    it.p0 = P.pos0 ? (int64_t)P.pos0[b] : (int64_t)held - it.tokens;
    const int32_t start = P.start ? P.start[b] : 0;
    const uint32_t r0 = (uint32_t)j * kRows;               // rows of a call are fewer than 2^31
    const uint32_t t0 = r0 / (uint32_t)P.H, t1 = (r0 + it.rows - 1) / (uint32_t)P.H;
    int32_t lo0, hi0, lo1, hi1;
    int64_t e0, e1;
    bounds(P, it.p0 + t0, it.len, start, lo0, hi0, e0);
    bounds(P, it.p0 + t1, it.len, start, lo1, hi1, e1);
    it.lo = lo0;
    it.hi = hi1;
    it.beyond = held > it.len && e1 > it.len;
    it.k0 = lo0 / kKeys;
    it.nt = hi1 > lo0 ? (hi1 + kKeys - 1) / kKeys - it.k0 : 1;
}

// Walks a cluster's run of (row tile, key tile) units.
struct Walk {
    Item it;
    int32_t off, n;           // this cluster's key tiles of the item: off .. off + n - 1
    int64_t left;             // units of the run after them
    int32_t at;               // tile of the item

    __device__ __forceinline__ void take()
    {
        const int32_t rest = it.nt - off;
        n = left < rest ? (int32_t)left : rest;
        left -= n;
        at = 0;
    }
    __device__ __forceinline__ bool begin(const AttnParams &P, const Misc &M, int64_t units)
    {
        left = units;
        if (units <= 0) return false;
        load_item(P, M.b, M.j, it);
        off = M.off;
        take();
        return true;
    }
    // The next key tile; false at the end of the run.
    __device__ __forceinline__ bool next(const AttnParams &P)
    {
        if (++at < n) return true;
        if (left <= 0) return false;
        int b = it.b, j = it.j + 1;
        if ((int64_t)j * kRows >= (int64_t)it.tokens * P.H) {
            j = 0;
            do ++b; while (b < P.batch - 1 && row_tiles(P, b) == 0);
        }
        load_item(P, b, j, it);
        off = 0;
        take();
        return true;
    }
    __device__ __forceinline__ bool first() const { return at == 0; }
    __device__ __forceinline__ bool last() const { return at == n - 1; }
    __device__ __forceinline__ int32_t key0() const { return (it.k0 + off + at) * kKeys; }
};

// Block-wide exclusive sum over the 512 threads.
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
template <int FMT>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_kernel(const __grid_constant__ AttnParams P)
{
    extern __shared__ __align__(1024) uint8_t sm[];
    Misc &M = *reinterpret_cast<Misc *>(sm + kOffMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            for (int g = 0; g < 3; ++g) tc::mbar_init(&M.full_k[s][g], 2 * kStageThreads / 32);
            tc::mbar_init(&M.full_z[s], 2 * kStageThreads / 32);
            tc::mbar_init(&M.info[s], 2 * kStageThreads / 32);
            tc::mbar_init(&M.s_done[s], 1);
            tc::mbar_init(&M.pv_done[s], 1);
        }
        tc::mbar_init(&M.full_p, 8);
        tc::mbar_init(&M.drained, 1);
        tc::fence_mbar_init();
        M.abort = 0;
        M.start_unit = -1;
    }
    if (warp == 4) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tc::smem_u32(&M.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
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
        for (int b = b0; b < b1; ++b) own += row_tiles(P, b);
        int64_t at = block_scan(own, M.scan, items);
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
        Item it;
        for (int64_t i = i0; i < i1; ++i) {
            while (tiles_before[b + 1] <= i) ++b;
            load_item(P, b, (int)(i - tiles_before[b]), it);
            own += it.nt;
        }
        int64_t u = block_scan(own, M.scan, total);
        share = (total + clusters - 1) / clusters;
        const int64_t mine = share * cluster;
        if (mine < total && mine >= u && mine < u + own) {  // this thread's items hold the run's start
            b = rb;
            for (int64_t i = i0; i < i1; ++i) {
                while (tiles_before[b + 1] <= i) ++b;
                load_item(P, b, (int)(i - tiles_before[b]), it);
                if (mine < u + it.nt) {
                    M.b = b;
                    M.j = it.j;
                    M.off = (int32_t)(mine - u);
                    M.item_unit = u;
                    break;
                }
                u += it.nt;
            }
        }
    }
    const int64_t start = share * cluster;
    const int64_t units = start < total ? (start + share < total ? share : total - start) : 0;
    tc::tc_fence_before();
    __syncthreads();
    cluster_sync();                          // barriers and tensor memory of both CTAs are there
    tc::tc_fence_after();
    const uint32_t tmem = M.tmem;            // O: columns 0..255 (two blocks), S: 256 + 64 (tile & 1)
    if (tid == 0 && rank == 0) P.desc[cluster].parts = 0;

    if (warp >= kStageWarp) {
        // ============================================================ staging
        const int t = tid - kStageWarp * 32, key = t >> 2, quarter = t & 3;
        Walk w;
        bool go = w.begin(P, M, units), ok = true;
        // slot of a key of the walk's tile (-1: none)
        auto slot_of = [&](const Walk &v, int half) -> int32_t {
            const int32_t k = v.key0() + 64 * half + key;
            if (k < v.it.lo || k >= v.it.hi) return -1;
            const int32_t id = P.table[(int64_t)v.it.b * P.width + (k >> P.C.shift)];
            if (id < 0 || id >= P.C.n_pages) {
                if (quarter == 0 && half == (int)rank) dev_flag(P.d_status, CSA2_DEV_BAD_INDEX);
                return -1;
            }
            return (int32_t)(((uint32_t)id << P.C.shift) + (k & ((1 << P.C.shift) - 1)));
        };
        constexpr int kBatch = FMT == CSA2P_BF16 ? 3 : FMT == CSA2P_MXFP8 ? 5 : 9;   // chunks held in registers
        const int n_groups = (P.chunks + 2) / 3;
        Raw<FMT> own[kBatch];
        auto load_own = [&](int32_t sl, int c0) {
            const uint8_t *codes = P.C.codes + P.C.code_at(sl < 0 ? 0 : sl), *scales = P.C.scales + P.C.scale_at(sl < 0 ? 0 : sl);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                zero_raw(own[i]);
                if (sl >= 0 && c0 + i < P.chunks && (c0 + i) * 64 + quarter * 16 < P.C.d)
                    load_raw(own[i], codes, scales, (c0 + i) * 4 + quarter);
            }
        };
        int32_t sl_own = -1, sl_oth = -1;
        if (go) {
            sl_own = slot_of(w, (int)rank);
            sl_oth = slot_of(w, 1 - (int)rank);
            load_own(sl_own, 0);
        }
        for (uint32_t n = 0; go && ok; ++n) {
            const uint32_t s = n & 1, ph = (n >> 1) & 1;
            uint8_t *kbase = sm + kOffK + s * 8 * kUnit;
            // ---- the queries of a new row tile, once the old ones' last product is done
            if (w.first()) {
                if (n > 0) ok = wait_bar(&M.s_done[s ^ 1], ((n - 1) >> 1) & 1, &M.abort);
                if (!__all_sync(0xffffffffu, ok)) break;
                if (t == 0 && rank == 0 && w.it.beyond) dev_flag(P.d_status, CSA2_DEV_BAD_INDEX);
                const int pieces = P.C.d / 8, all = P.chunks * 8;
                const int64_t r0 = w.it.row0(P.H) + 64 * rank;
                const int mine = min(max(w.it.rows - 64 * (int)rank, 0), 64);
#pragma unroll 6
                for (int e = t; e < 64 * 72; e += kStageThreads) {
                    const int r = e / 72, p = e - 72 * r;
                    if (p >= all) continue;
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (r < mine && p < pieces) v = *reinterpret_cast<const uint4 *>(P.q + (r0 + r) * P.C.d + 8 * p);
                    *reinterpret_cast<uint4 *>(sm + (p >> 3) * kUnit + sw128(r, p & 7)) =
                        make_uint4(prmt(v.x, v.z, 0x5410u), prmt(v.x, v.z, 0x7632u), prmt(v.y, v.w, 0x5410u), prmt(v.y, v.w, 0x7632u));
                }
            }
            // ---- the next tile's slots, looked up while this one is decoded
            Walk nx = w;
            const bool more = nx.next(P);
            int32_t nx_own = -1, nx_oth = -1;
            if (more) {
                nx_own = slot_of(nx, (int)rank);
                nx_oth = slot_of(nx, 1 - (int)rank);
            }
            // ---- own keys
            if (n >= 2) ok = wait_bar(&M.pv_done[s], ((n - 2) >> 1) & 1, &M.abort);
            if (!__all_sync(0xffffffffu, ok)) break;
            bool bad = false;
#pragma unroll
            for (int c = 0; c < 9; ++c) {
                if (c < P.chunks) {
                    if (kBatch < 9 && c > 0 && c % kBatch == 0) load_own(sl_own, c);
                    if (c == 8 && n > 0) ok = wait_bar(&M.s_done[s ^ 1], ((n - 1) >> 1) & 1, &M.abort) && ok;
                    uint4 o[2];
                    bad |= decode(own[c % kBatch], o);
                    uint8_t *u = c < 8 ? kbase + c * kUnit : sm + kOffR;
                    *reinterpret_cast<uint4 *>(u + sw128(key, 2 * quarter)) = o[0];
                    *reinterpret_cast<uint4 *>(u + sw128(key, 2 * quarter + 1)) = o[1];
                }
                if (c % 3 == 2 || c == P.chunks - 1) {
                    if (c < P.chunks || c / 3 < n_groups) {
                        if (c == min(3 * (c / 3) + 2, P.chunks - 1)) {
                            tc::fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) arrive_at(&M.full_k[s][c / 3], 0);
                        }
                    }
                }
            }
            // which keys are there and finite: both CTAs' softmax wants it
            {
                const uint32_t have = __ballot_sync(0xffffffffu, sl_own >= 0), nan = __ballot_sync(0xffffffffu, bad);
                if (lane < 2) {
                    uint32_t hv = 0, nv = 0;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        hv |= ((have >> (4 * k)) & 1u) << k;
                        nv |= (((nan >> (4 * k)) & 15u) ? 1u : 0u) << k;
                    }
                    const uint8_t *pv = reinterpret_cast<const uint8_t *>(&M.valid[s][rank]) + (warp - kStageWarp);
                    const uint8_t *pn = reinterpret_cast<const uint8_t *>(&M.nan[s][rank]) + (warp - kStageWarp);
                    st_peer_u8(pv, (uint32_t)lane, hv);
                    st_peer_u8(pn, (uint32_t)lane, nv);
                    arrive_at(&M.info[s], (uint32_t)lane);
                }
            }
            // ---- the peer's keys, this CTA's dims: over chunks that S has read
            const bool own_dims = (int)rank * 2 < P.v_chunks;
            Raw<FMT> oth[4];
            {
                const uint8_t *codes = P.C.codes + P.C.code_at(sl_oth < 0 ? 0 : sl_oth), *scales = P.C.scales + P.C.scale_at(sl_oth < 0 ? 0 : sl_oth);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = (i >> 1) * 4 + 2 * (int)rank + (i & 1);
                    zero_raw(oth[i]);
                    if (sl_oth >= 0 && c < P.v_chunks && c * 64 + quarter * 16 < P.C.d) load_raw(oth[i], codes, scales, c * 4 + quarter);
                }
            }
            if (more) load_own(nx_own, 0);
            ok = wait_bar(&M.s_done[s], ph, &M.abort) && ok;
            if (!__all_sync(0xffffffffu, ok)) break;
            if (own_dims) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = (i >> 1) * 4 + 2 * (int)rank + (i & 1);
                    if (c < P.v_chunks) {
                        uint4 o[2];
                        decode(oth[i], o);
                        uint8_t *u = kbase + (c ^ 2) * kUnit;
                        *reinterpret_cast<uint4 *>(u + sw128(key, 2 * quarter)) = o[0];
                        *reinterpret_cast<uint4 *>(u + sw128(key, 2 * quarter + 1)) = o[1];
                    }
                }
                tc::fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) arrive_at(&M.full_z[s], 0);
            w = nx;
            sl_own = nx_own;
            sl_oth = nx_oth;
            go = more;
        }
        if (!ok) M.abort = 1;
    } else if (warp == 4) {
        // ============================================================ MMA (the leader's one thread)
        if (rank == 0 && lane == 0) {
            const uint32_t base = tc::smem_u32(sm);
            const uint64_t dq = tc::smem_desc(base, 16, 1024, tc::kSwizzle128B);
            const uint64_t dp = tc::smem_desc(base + kOffP, 16, 1024, tc::kSwizzle128B);
            const uint64_t dr = tc::smem_desc(base + kOffR, 16, 1024, tc::kSwizzle128B);
            Walk w;
            bool go = w.begin(P, M, units), ok = true, pending = false, pending_first = false;
            auto pv = [&](uint32_t n, bool first) {
                const uint32_t s = n & 1;
                ok = wait_bar(&M.full_p, n & 1, &M.abort) && wait_bar(&M.full_z[s], (n >> 1) & 1, &M.abort);
                if (!ok) return;
                tc::tc_fence_after();
                const uint64_t dv = tc::smem_desc(base + kOffK + s * 8 * kUnit, kUnit, 1024, tc::kSwizzle128B);
#pragma unroll 1
                for (int j = 0; j < P.n_pv; ++j)
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma2(tmem + 128 * j, dp + (k >> 2) * (kUnit / 16) + (k & 3) * 2,
                             dv + (4 * j + 2 * (k >> 2)) * (kUnit / 16) + (k & 3) * 128, instr(256, 1), !(first && k == 0));
                commit2(&M.pv_done[s]);
            };
            uint32_t n = 0;
            for (; go; ++n) {
                const uint32_t s = n & 1;
                if (w.first() && pending) {
                    pv(n - 1, pending_first);
                    pending = false;
                    if (!ok) break;
                }
                const uint64_t dk = tc::smem_desc(base + kOffK + s * 8 * kUnit, 16, 1024, tc::kSwizzle128B);
#pragma unroll 1
                for (int g = 0; 3 * g < P.chunks; ++g) {
                    ok = wait_bar(&M.full_k[s][g], (n >> 1) & 1, &M.abort);
                    if (!ok) break;
                    tc::tc_fence_after();
#pragma unroll
                    for (int i = 0; i < 3; ++i) {
                        const int c = 3 * g + i;
                        if (c < P.chunks) {
                            const uint64_t b = c < 8 ? dk + c * (kUnit / 16) : dr;
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma2(tmem + 256 + 64 * s, dq + c * (kUnit / 16) + k * 2, b + k * 2, instr(128, 0), (c | k) != 0);
                        }
                    }
                }
                if (!ok) break;
                commit2(&M.s_done[s]);
                if (pending) {
                    pv(n - 1, pending_first);
                    if (!ok) break;
                }
                pending = true;
                pending_first = w.first();
                go = w.next(P);
            }
            if (ok && pending) pv(n - 1, pending_first);
            if (!ok) M.abort = 1;
            commit2(&M.drained);                   // nothing may still run when the CTAs leave
        }
        __syncwarp();
    } else if (warp < 4) {
        // ============================================================ softmax and output
        const int row = tid & 63, half = tid >> 6;
        const uint32_t lane_t = tmem + ((uint32_t)(warp * 32) << 16);
        Walk w;
        bool go = w.begin(P, M, units), failed = false;
        int32_t lo = 0, hi = 0;
        float m = -INFINITY, l = 0.0f;
        int64_t unit = M.item_unit;                // first unit of the item
        for (uint32_t n = 0; go; ++n) {
            const uint32_t s = n & 1, ph = (n >> 1) & 1;
            if (w.first()) {
                const uint32_t f = (uint32_t)w.it.j * kRows + 64 * rank + row;
                lo = hi = 0;
                if (64 * (int)rank + row < w.it.rows) {
                    int64_t e;
                    bounds(P, w.it.p0 + f / (uint32_t)P.H, w.it.len, P.start ? P.start[w.it.b] : 0, lo, hi, e);
                }
                m = -INFINITY;
                l = 0.0f;
            }
            const int32_t k0 = w.key0() + 64 * half;
            failed |= __any_sync(0xffffffffu, !wait_bar(&M.info[s], ph, &M.abort) || !wait_bar(&M.s_done[s], ph, &M.abort));
            uint32_t r[64];
            float top = -INFINITY;
            if (!failed) {
                tc::tc_fence_after();
                tc::tc_ld_32x32b_x32(lane_t + 256 + 64 * s, *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
                tc::tc_ld_32x32b_x32(lane_t + 256 + 64 * s + 32, *reinterpret_cast<uint32_t(*)[32]>(&r[32]));
                tc::tc_wait_ld();
                // keys of this half that the row sees, as bits
                const int32_t a = max(lo - k0, 0), z = min(hi - k0, 64);
                uint64_t see = z > a ? (~0ull >> (64 - (z - a))) << a : 0ull;
                see &= M.valid[s][half];
                const uint64_t nan = see & M.nan[s][half];
                if (see != ~0ull) {
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        if (!((see >> c) & 1ull)) r[c] = 0xff800000u;
                }
                if (nan) {
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        if ((nan >> c) & 1ull) r[c] = 0x7fc00000u;
                }
                float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 64; ++c) t4[c & 3] = fmaxf(t4[c & 3], __uint_as_float(r[c]));
                top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * P.log2_scale;
            }
            M.top[s][half][row] = top;
            if (softmax_sync(failed)) { failed = true; break; }
            top = fmaxf(top, M.top[s][half ^ 1][row]);
            float f = 1.0f;
            if (top > m + kLazy || (m == -INFINITY && top > -INFINITY)) {
                f = ex2(m - top);                  // 0 for the first maximum
                m = top;
                l *= f;
            }
            const float mm = m == -INFINITY ? 0.0f : m;
            float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            uint32_t p[32];
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
                const float x = ex2(fmaf(__uint_as_float(r[c]), P.log2_scale, -mm));
                const float y = ex2(fmaf(__uint_as_float(r[c + 1]), P.log2_scale, -mm));
                s4[c & 2] += x;
                s4[(c & 2) + 1] += y;
                const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
                p[c / 2] = *reinterpret_cast<const uint32_t *>(&b);
            }
            l += (s4[0] + s4[1]) + (s4[2] + s4[3]);
            // the previous product of this row tile has read P and written O
            if (!w.first()) {
                failed |= __any_sync(0xffffffffu, !wait_bar(&M.pv_done[s ^ 1], ((n - 1) >> 1) & 1, &M.abort));
                if (!failed && __any_sync(0xffffffffu, f != 1.0f)) {
                    tc::tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 128 * P.n_pv; c += 16) {
                        uint32_t o[16];
                        tc::tc_ld_32x32b_x16(lane_t + c, o);
                        tc::tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tc::tc_st_32x32b_x16(lane_t + c, o);
                    }
                    tc::tc_wait_st();
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                *reinterpret_cast<uint4 *>(sm + kOffP + half * kUnit + sw128(row, i)) =
                    make_uint4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
            tc::fence_proxy_async_smem();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_at(&M.full_p, 0);
            if (w.last()) {
                // ---- output, or a part of it
                failed |= __any_sync(0xffffffffu, !wait_bar(&M.pv_done[s], ph, &M.abort));
                M.sum[half][row] = l;
                if (softmax_sync(failed)) { failed = true; break; }
                tc::tc_fence_after();
                l += M.sum[half ^ 1][row];
                const bool part = w.off > 0 || w.off + w.n < w.it.nt;
                const int in_tile = 64 * (int)rank + row;
                const bool live = in_tile < w.it.rows;
                const int64_t grow = w.it.row0(P.H) + in_tile;
                const int slot = 2 * cluster + (w.off > 0 ? 0 : 1);
                if (part) {
                    if (half == 0) {
                        P.part_ml[((int64_t)slot * kRows + in_tile) * 2] = m;
                        P.part_ml[((int64_t)slot * kRows + in_tile) * 2 + 1] = l;
                    }
                    if (w.off == 0 && tid == 0 && rank == 0) {
                        PartDesc d;
                        d.parts = (int32_t)((unit + w.it.nt - 1) / share - cluster + 1);
                        d.rows = w.it.rows;
                        d.row0 = w.it.row0(P.H);
                        P.desc[cluster] = d;
                    }
                } else if (half == 0 && live && P.lse) {
                    P.lse[grow] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
                }
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
                for (int j = 0; j < P.n_pv; ++j)
#pragma unroll 1
                    for (int c = 0; c < 128; c += 16) {
                        const int d0 = 256 * j + 128 * half + c;
                        uint32_t o[16];
                        tc::tc_ld_32x32b_x16(lane_t + 128 * j + c, o);
                        tc::tc_wait_ld();
#pragma unroll
                        for (int g = 0; g < 16; g += 8) {
                            if (!live || d0 + g >= P.d_v) continue;
                            float v[8];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                v[k] = __uint_as_float(o[g + 2 * k]);
                                v[k + 4] = __uint_as_float(o[g + 2 * k + 1]);
                            }
                            if (part) {
                                float4 *dst = reinterpret_cast<float4 *>(P.part_o + ((int64_t)slot * kRows + in_tile) * P.d_v + d0 + g);
                                dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                                dst[1] = make_float4(v[4], v[5], v[6], v[7]);
                            } else {
                                uint32_t x[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k] * inv, v[2 * k + 1] * inv);
                                    x[k] = *reinterpret_cast<const uint32_t *>(&b);
                                }
                                *reinterpret_cast<uint4 *>(P.out + grow * P.d_v + d0 + g) = make_uint4(x[0], x[1], x[2], x[3]);
                            }
                        }
                    }
                tc::tc_fence_before();
            }
            const int32_t nt = w.it.nt, was = w.last();
            go = w.next(P);
            if (was) unit += nt;
        }
        if (failed) M.abort = 1;
    }
    __syncthreads();
    if (tid == 0) {
        tc::mbar_wait_bounded(&M.drained, 0);
        if (M.abort) dev_flag(P.d_status, CSA2_DEV_TIMEOUT);
    }
    tc::tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 4) {
        tc::tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// Joins the parts of cut row tiles: o = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.  A warp takes
// a row; blockIdx.x = the cluster that began the row tile, whose part is its second slot and whose
// further parts are the first slots of the clusters after it.
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

// Clusters of two CTAs of this kernel that are resident at once on the current device.
int attn_clusters()
{
    return device_sm_count() / 2 > 0 ? device_sm_count() / 2 : 1;
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

} // namespace

size_t paged_attn_ws_bytes(const csa2p_attn_args &a)
{
    const size_t slots = 2 * (size_t)attn_clusters() * kRows;
    return up256(slots * a.d_v * sizeof(float)) + up256(slots * 2 * sizeof(float)) + up256(attn_clusters() * sizeof(PartDesc));
}

cudaError_t launch_paged_attn(const csa2p_attn_args &a, const PagedView &v, uint16_t *out, float *lse, void *ws,
                              uint32_t *d_status, cudaStream_t s)
{
    const int clusters = attn_clusters();
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
    P.v_chunks = (a.d_v + 63) / 64;
    P.n_pv = (a.d_v + 255) / 256;
    P.log2_scale = a.sm_scale * 1.4426950408889634f;
    P.q = a.q;
    P.table = a.block_table;
    P.lens = a.lens;
    P.cu = a.cu;
    P.pos0 = a.pos0;
    P.start = a.kv_start;
    P.out = out;
    P.lse = lse;
    P.d_status = d_status;
    const size_t slots = 2 * (size_t)clusters * kRows;
    char *w = static_cast<char *>(ws);
    P.part_o = reinterpret_cast<float *>(w);
    w += up256(slots * a.d_v * sizeof(float));
    P.part_ml = reinterpret_cast<float *>(w);
    w += up256(slots * 2 * sizeof(float));
    P.desc = reinterpret_cast<PartDesc *>(w);
    auto k = v.fmt == CSA2P_MXFP4 ? paged_attn_kernel<CSA2P_MXFP4>
             : v.fmt == CSA2P_NVFP4_E4M3_16 ? paged_attn_kernel<CSA2P_NVFP4_E4M3_16>
             : v.fmt == CSA2P_MXFP8 ? paged_attn_kernel<CSA2P_MXFP8> : paged_attn_kernel<CSA2P_BF16>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(k, dim3((unsigned)(2 * clusters)), dim3(kThreads), (size_t)kSmem, s, 2, P);
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_attn_join_kernel, dim3((unsigned)clusters, kRows / 8), dim3(256), 0, s, 1, P);
}

} // namespace csa2
