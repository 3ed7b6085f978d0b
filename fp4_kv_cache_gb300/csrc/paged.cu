// paged.cu -- page bookkeeping, rotary positions with several axes, and the paged cache's
// write and read (include/csa2_paged.h).  The cache is the one of DeepSeek-V4.1-Flash report
// §2.4.4 (rows quantised after RoPE, RoPE and other channels in one format) laid out in pages.
#include "common.cuh"
#include "internal.h"
#include "paged.cuh"

#include <cuda_bf16.h>

namespace csa2 {
namespace {

// ---------------------------------------------------------------- bookkeeping
constexpr int kPlanThreads = 1024;
constexpr int kPlanCluster = 8;

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

// One launch: every CTA (one, or a cluster of eight when there are many rows) scans all the
// requests for itself -- rows added, pages taken, pages given back -- so that the rows, the
// taken pages and the returned pages can then be shared out with no further exchange.  What
// another CTA may still read (lens, n_free) is overwritten only after a cluster barrier; table
// entries read are never written here (a request takes or gives back, not both), and the free
// list is read below n_free and written above it.
__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PlanParams P, uint32_t *d_status)
{
    extern __shared__ int32_t sm[];
    int32_t *s_cu = sm, *s_take = s_cu + P.batch + 1, *s_back = s_take + P.batch + 1;
    __shared__ int64_t s_warp[3][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n_cta = gridDim.x, cta = blockIdx.x;
    pdl_wait();
    pdl_allow_dependents();
    // ---- scan of the requests, `per` consecutive ones a thread
    const int per = (P.batch + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(tid * per, P.batch), b1 = min(b0 + per, P.batch);
    int64_t own[3] = {0, 0, 0};
    for (int b = b0; b < b1; ++b) {
        const Req r = plan_req(P, b);
        own[0] += r.new_len > r.old_len ? r.new_len - r.old_len : 0;
        own[1] += max(r.has - r.had, 0);
        own[2] += max(r.had - r.has, 0);
        if (r.full && cta == 0) dev_flag(d_status, CSA2P_DEV_TABLE_FULL);
    }
    int64_t before[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
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
    if (warp < 3) {
        int64_t v = s_warp[warp][lane];
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
    for (int k = 0; k < 3; ++k) before[k] += s_warp[k][warp];
    for (int b = b0; b <= b1; ++b) {
        if (b == b1 && b != P.batch) break;                    // the next thread's first entry
        s_cu[b] = hold31(before[0]);
        s_take[b] = hold31(before[1]);
        s_back[b] = hold31(before[2]);
        if (cta == 0) P.cu[b] = s_cu[b];
        if (b == b1) break;
        const Req r = plan_req(P, b);
        before[0] += r.new_len > r.old_len ? r.new_len - r.old_len : 0;
        before[1] += max(r.has - r.had, 0);
        before[2] += max(r.had - r.has, 0);
    }
    __syncthreads();
    const int n_new = s_cu[P.batch], n_take = s_take[P.batch], n_back = s_back[P.batch];
    const int n_free = min(max(P.n_free[0], 0), P.free_cap);
    const int64_t top = (int64_t)n_free + n_back;
    if (tid == 0 && cta == 0) {
        if (n_take > top) dev_flag(d_status, CSA2P_DEV_NO_PAGES);
        if (n_new > P.n_rows) dev_flag(d_status, CSA2P_DEV_ROWS);
        if (top - n_take > P.free_cap) dev_flag(d_status, CSA2P_DEV_TABLE_FULL);
    }
    auto returned = [&](int i) -> int32_t {                    // i-th page given back
        const int b = last_at_or_below(s_back, P.batch, i);
        return P.table[(int64_t)b * P.width + plan_req(P, b).has + (i - s_back[b])];
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
    for (int64_t i = first; i < n_back; i += step)
        if (n_free + i < left && n_free + i < P.free_cap) P.free_pages[n_free + i] = returned((int)i);
    int32_t len_new[16];                                       // per <= CSA2P_MAX_BATCH / 1024
    if (cta == 0)
#pragma unroll
        for (int k = 0; k < 16; ++k)
            if (b0 + k < b1) len_new[k] = (int32_t)plan_req(P, b0 + k).new_len;
    if (n_cta > 1)
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    else
        __syncthreads();
    if (cta == 0) {
#pragma unroll
        for (int k = 0; k < 16; ++k)
            if (b0 + k < b1) P.lens_out[b0 + k] = len_new[k];
        if (tid == 0) P.n_free_out[0] = (int32_t)(left < P.free_cap ? left : P.free_cap);
    }
}

// ---------------------------------------------------------------- rotation
// Turns the pairs of eight channels col .. col+7 that lie at or past channel c0 (even), with
// one rounding per product and per sum, as csa2_rope_quant_fp4 does.
__device__ __forceinline__ void rotate8(float (&v)[8], int col, int c0, const RopeView &R, int64_t row, int64_t rows,
                                        uint32_t *d_status)
{
    const int half = R.dim >> 1;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const int i = (col + e - c0) >> 1;
        if (col + e < c0) continue;
        const int axis = (i >= R.end0) + (i >= R.end1);
        const int64_t p = R.pos[axis * rows + row];
        if (p < 0) continue;
        if (p >= R.n_pos) {
            dev_flag(d_status, CSA2_DEV_BAD_INDEX);
            continue;
        }
        const float c = R.cs[p * R.dim + i], s = R.cs[p * R.dim + half + i], a = v[e], b = v[e + 1];
        v[e] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
        v[e + 1] = __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c));
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
// turned channels are visited.
__global__ void __launch_bounds__(256) paged_rope_kernel(const uint16_t *__restrict__ x, int64_t x_row, int64_t x_head,
                                                         uint16_t *out, int64_t out_row, int64_t out_head, int32_t heads,
                                                         int32_t d, int32_t first_piece, int64_t rows, const RopeView R,
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
            rotate8(v, col, c0, R, row, rows, d_status);
            raw = pack8(v);
        }
        *reinterpret_cast<uint4 *>(out + row * out_row + h * out_head + col) = raw;
    }
}

// ---------------------------------------------------------------- write
// A lane takes eight channels of one row (16 bytes of x); the lanes of a scale block are
// neighbours (4 for 32 channels, 2 for 16; d is a multiple of 32, so none straddles a row).
template <int FMT>
__global__ void __launch_bounds__(256) paged_write_kernel(const PagedView C, const uint16_t *__restrict__ x, int64_t ldx,
                                                          int32_t rows, const int32_t *__restrict__ slot,
                                                          const RopeView R, uint32_t *d_status)
{
    pdl_wait();
    pdl_allow_dependents();
    const int lanes = C.d / 8, c0 = C.d - R.dim;
    const int64_t total = (int64_t)rows * lanes, total32 = (total + 31) & ~int64_t(31);
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total32; t += (int64_t)gridDim.x * 256) {
        const int64_t r = t < total ? t / lanes : 0;
        const int sub8 = t < total ? (int)(t - r * lanes) : 0, col = 8 * sub8;
        const int32_t sl = t < total ? slot[r] : -1;
        const bool act = sl >= 0 && sl < C.n_slots;
        if (sl >= C.n_slots) dev_flag(d_status, CSA2_DEV_BAD_INDEX);
        float v[8];
        if (act) {
            unpack8(*reinterpret_cast<const uint4 *>(x + r * ldx + col), v);
            if (R.dim > 0 && col + 8 > c0) rotate8(v, col, c0, R, r, rows, d_status);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        }
        uint8_t *codes = const_cast<uint8_t *>(C.codes) + C.code_at(act ? sl : 0);
        if (FMT == CSA2P_BF16) {
            if (act) *reinterpret_cast<uint4 *>(codes + 2 * col) = pack8(v);
            continue;
        }
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7fffffffu);
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        if (FMT != CSA2P_NVFP4_E4M3_16) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        if (!act) continue;
        const bool head = (sub8 & (FMT == CSA2P_NVFP4_E4M3_16 ? 1 : 3)) == 0, finite = amax < 0x7f800000u;
        if (!finite && head) dev_flag(d_status, CSA2_DEV_NONFINITE);
        const float amax_f = __uint_as_float(finite ? amax : 0u);
        uint32_t sbyte;
        if (FMT == CSA2P_MXFP8) {
            const int X = mx8_block_exponent(amax_f);
            const float inv = pow2_neg(X);
            uint32_t w[2] = {0u, 0u};
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i >> 2] |= e4m3_cvt(v[i] * inv) << (8 * (i & 3));
            *reinterpret_cast<uint2 *>(codes + col) = make_uint2(w[0], w[1]);
            sbyte = (uint32_t)(X + 127);
        } else {
            uint32_t word = 0;
            if (FMT == CSA2P_NVFP4_E4M3_16) {
                sbyte = e4m3_block_scale(amax_f);
                const float sc = e4m3_value(sbyte);
                if (sc > 0.0f) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2)
                        word |= e2m1x2_cvt(__fdiv_rn(v[i], sc), __fdiv_rn(v[i + 1], sc)) << (4 * i);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) word |= (__float_as_uint(v[i]) >> 31) << (4 * i + 3);
                }
            } else {
                const int X = mx_block_exponent(amax_f);
                const float inv = pow2_neg(X);
#pragma unroll
                for (int i = 0; i < 8; i += 2) word |= e2m1x2_cvt(v[i] * inv, v[i + 1] * inv) << (4 * i);
                sbyte = (uint32_t)(X + 127);
            }
            *reinterpret_cast<uint32_t *>(codes + col / 2) = word;
        }
        if (head)
            const_cast<uint8_t *>(C.scales)[C.scale_at(sl) + col / (FMT == CSA2P_NVFP4_E4M3_16 ? 16 : 32)] = (uint8_t)sbyte;
    }
}

// ---------------------------------------------------------------- read
template <int FMT>
__global__ void __launch_bounds__(256) paged_read_kernel(const PagedView C, const int32_t *__restrict__ slot, int32_t rows,
                                                         uint16_t *__restrict__ out, int64_t ldo, uint32_t *d_status)
{
    pdl_wait();
    pdl_allow_dependents();
    const int lanes = C.d / 8;
    const int64_t total = (int64_t)rows * lanes;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += (int64_t)gridDim.x * 256) {
        const int64_t r = t / lanes;
        const int col = 8 * (int)(t - r * lanes);
        const int32_t sl = slot[r];
        if (sl < 0) continue;
        if (sl >= C.n_slots) {
            dev_flag(d_status, CSA2_DEV_BAD_INDEX);
            continue;
        }
        const uint8_t *codes = C.codes + C.code_at(sl);
        uint4 o;
        if (FMT == CSA2P_BF16) {
            o = *reinterpret_cast<const uint4 *>(codes + 2 * col);
        } else {
            const uint32_t sb = C.scales[C.scale_at(sl) + col / (FMT == CSA2P_NVFP4_E4M3_16 ? 16 : 32)];
            // code x scale is exact in float32 and rounded to bf16 once
            const float sc = FMT == CSA2P_NVFP4_E4M3_16 ? e4m3_value(sb)
                             : sb == 255u ? __uint_as_float(0x7fc00000u) : e8m0_value(sb);
            float v[8];
            if (FMT == CSA2P_MXFP8) {
                const uint2 w = *reinterpret_cast<const uint2 *>(codes + col);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = e4m3_value(((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 0xffu) * sc;
            } else {
                const uint32_t w = *reinterpret_cast<const uint32_t *>(codes + col / 2);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t c = (w >> (4 * i)) & 15u;
                    v[i] = (c & 8u ? -e2m1_mag(c & 7u) : e2m1_mag(c & 7u)) * sc;
                }
            }
            o = pack8(v);
        }
        *reinterpret_cast<uint4 *>(out + r * ldo + col) = o;
    }
}

int blocks_for(int64_t threads, int per_sm)
{
    const int64_t g = (threads + 255) / 256, most = (int64_t)device_sm_count() * per_sm;
    return (int)(g < 1 ? 1 : g > most ? most : g);
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
        const cudaError_t e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    const int ctas = a.n_rows > 4 * kPlanThreads ? kPlanCluster : 1;
    return launch_pdl(page_plan_kernel, dim3(ctas), dim3(kPlanThreads), smem, s, (unsigned)ctas, P, d_status);
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
    const int g = blocks_for((int64_t)rows * (v.d / 8), 16);
    auto k = v.fmt == CSA2P_MXFP4 ? paged_write_kernel<CSA2P_MXFP4>
             : v.fmt == CSA2P_NVFP4_E4M3_16 ? paged_write_kernel<CSA2P_NVFP4_E4M3_16>
             : v.fmt == CSA2P_MXFP8 ? paged_write_kernel<CSA2P_MXFP8> : paged_write_kernel<CSA2P_BF16>;
    return launch_pdl(k, dim3(g), dim3(256), 0, s, 1, v, x, ldx, rows, slot, rope, d_status);
}

cudaError_t launch_paged_read(const PagedView &v, const int32_t *slot, int32_t rows, uint16_t *out, int64_t ldo,
                              uint32_t *d_status, cudaStream_t s)
{
    const int g = blocks_for((int64_t)rows * (v.d / 8), 16);
    auto k = v.fmt == CSA2P_MXFP4 ? paged_read_kernel<CSA2P_MXFP4>
             : v.fmt == CSA2P_NVFP4_E4M3_16 ? paged_read_kernel<CSA2P_NVFP4_E4M3_16>
             : v.fmt == CSA2P_MXFP8 ? paged_read_kernel<CSA2P_MXFP8> : paged_read_kernel<CSA2P_BF16>;
    return launch_pdl(k, dim3(g), dim3(256), 0, s, 1, v, slot, rows, out, ldo, d_status);
}

} // namespace csa2
