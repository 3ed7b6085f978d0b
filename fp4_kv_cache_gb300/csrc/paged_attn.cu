// paged_attn.cu -- csa2p_attn: attention of new tokens over a paged latent cache.
//
// One block per (query token, 16 heads): the token's visible rows are decoded 32 at a time into
// shared memory as float32 and every warp runs an online softmax for two heads.
#include "common.cuh"
#include "internal.h"
#include "paged.cuh"

#include <cuda_bf16.h>

namespace csa2 {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kTile = 32, kHeads = 16, kMaxD = 576;

struct PagedAttnParams {
    PagedView C;
    int32_t batch, n_tokens, H, d_v, width, window, ratio;
    float log2_scale;
    const uint16_t *q;
    const int32_t *table, *lens, *cu, *pos0, *start;
    uint16_t *out;
    float *lse;
    uint32_t *d_status;
};

__device__ __forceinline__ float paged_value(const PagedView &C, int32_t sl, int c)
{
    const uint8_t *row = C.codes + C.code_at(sl);
    if (C.fmt == CSA2P_BF16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(row)[c] << 16);
    const bool nv = C.fmt == CSA2P_NVFP4_E4M3_16;
    const uint32_t sb = C.scales[C.scale_at(sl) + c / (nv ? 16 : 32)];
    const float sc = nv ? e4m3_value(sb) : sb == 255u ? __uint_as_float(0x7fc00000u) : e8m0_value(sb);
    if (C.fmt == CSA2P_MXFP8) return e4m3_value(row[c]) * sc;
    const uint32_t code = (row[c >> 1] >> (4 * (c & 1))) & 15u;
    return (code & 8u ? -e2m1_mag(code & 7u) : e2m1_mag(code & 7u)) * sc;
}

__global__ void __launch_bounds__(256) paged_attn_simple_kernel(const PagedAttnParams P)
{
    extern __shared__ float smf[];
    const int d = P.C.d, ld = d + 1, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float *sk = smf, *sq = sk + kTile * ld;
    __shared__ int32_t s_slot[kTile], s_bad[kTile];
    pdl_wait();
    pdl_allow_dependents();
    const int t = blockIdx.x, h0 = blockIdx.y * kHeads;
    // the request that holds token t: the last b with cu[b] <= t
    int lo = 0, hi = P.batch + 1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (P.cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    const int b = lo;
    if (b >= P.batch || P.cu[b] > t) return;
    const int first = P.cu[b], n = P.cu[b + 1] - first;
    const int64_t len = max(P.lens[b], 0);
    const int64_t p = (P.pos0 ? (int64_t)P.pos0[b] : len - n) + (t - first);
    const int64_t e = p < 0 ? 0 : (p + 1) / P.ratio;
    const int64_t k_hi = e < len ? e : len;
    int64_t k_lo = P.start ? P.start[b] : 0;
    if (P.window && e - P.window > k_lo) k_lo = e - P.window;
    k_lo = k_lo < 0 ? 0 : k_lo;
    const int n_h = min(kHeads, P.H - h0);
    for (int i = tid; i < n_h * d; i += 256)
        sq[i] = __uint_as_float((uint32_t)P.q[((int64_t)t * P.H + h0) * d + i] << 16);
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, acc[2][kMaxD / 32];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < kMaxD / 32; ++i) acc[k][i] = 0.0f;
    for (int64_t j0 = k_lo; j0 < k_hi; j0 += kTile) {
        __syncthreads();
        if (tid < kTile) {
            const int64_t j = j0 + tid, pg = j >> P.C.shift;
            int32_t sl = -1;
            if (j < k_hi) {
                const int32_t id = pg < P.width ? P.table[(int64_t)b * P.width + pg] : -1;
                if (id >= 0 && id < P.C.n_pages) sl = (int32_t)(((int64_t)id << P.C.shift) + (j & ((1 << P.C.shift) - 1)));
                else dev_flag(P.d_status, CSA2_DEV_BAD_INDEX);
            }
            s_slot[tid] = sl;
            s_bad[tid] = 0;
        }
        __syncthreads();
        for (int i = tid; i < kTile * d; i += 256) {
            const int r = i / d, c = i - r * d;
            float v = s_slot[r] >= 0 ? paged_value(P.C, s_slot[r], c) : 0.0f;
            if (!isfinite(v)) {                    // the row's weight becomes NaN
                s_bad[r] = 1;
                v = 0.0f;
            }
            sk[r * ld + c] = v;
        }
        __syncthreads();
        const bool key = s_slot[lane] >= 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int h = 2 * warp + k;
            if (h >= n_h) break;
            float s = 0.0f;
            for (int c = 0; c < d; ++c) s = fmaf(sq[h * d + c], sk[lane * ld + c], s);
            s = !key ? -INFINITY : s_bad[lane] ? __uint_as_float(0x7fc00000u) : s * P.log2_scale;
            float top = s;
#pragma unroll
            for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float m_new = fmaxf(m[k], top);
            if (m_new == -INFINITY && __all_sync(0xffffffffu, s == -INFINITY)) continue;
            const float pr = key ? exp2f(s - m_new) : 0.0f, f = exp2f(m[k] - m_new);
            float sum = pr;
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            l[k] = l[k] * f + sum;
            m[k] = m_new;
#pragma unroll
            for (int i = 0; i < kMaxD / 32; ++i) acc[k][i] *= f;
            for (int j = 0; j < kTile; ++j) {
                const float pj = __shfl_sync(0xffffffffu, pr, j);
#pragma unroll
                for (int i = 0; i < kMaxD / 32; ++i)
                    if (lane + 32 * i < P.d_v) acc[k][i] = fmaf(pj, sk[j * ld + lane + 32 * i], acc[k][i]);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int h = 2 * warp + k;
        if (h >= n_h) break;
        const int64_t row = (int64_t)t * P.H + h0 + h;
        const float inv = m[k] == -INFINITY && l[k] == 0.0f ? 0.0f : 1.0f / l[k];
#pragma unroll
        for (int i = 0; i < kMaxD / 32; ++i)
            if (lane + 32 * i < P.d_v) {
                const __nv_bfloat16 v = __float2bfloat16_rn(acc[k][i] * inv);
                P.out[row * P.d_v + lane + 32 * i] = *reinterpret_cast<const uint16_t *>(&v);
            }
        if (lane == 0 && P.lse) P.lse[row] = m[k] == -INFINITY && l[k] == 0.0f ? -INFINITY : (m[k] + log2f(l[k])) * kLn2;
    }
}

} // namespace

size_t paged_attn_ws_bytes(const csa2p_attn_args &) { return 0; }

cudaError_t launch_paged_attn(const csa2p_attn_args &a, const PagedView &v, uint16_t *out, float *lse, void *,
                              uint32_t *d_status, cudaStream_t s)
{
    PagedAttnParams P;
    P.C = v;
    P.batch = a.batch;
    P.n_tokens = a.n_tokens;
    P.H = a.n_heads;
    P.d_v = a.d_v;
    P.width = a.width;
    P.window = a.window;
    P.ratio = a.ratio_m;
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
    const int smem = (kTile * (v.d + 1) + kHeads * v.d) * (int)sizeof(float);
    const cudaError_t e = cudaFuncSetAttribute(paged_attn_simple_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_attn_simple_kernel, dim3((unsigned)a.n_tokens, (unsigned)((a.n_heads + kHeads - 1) / kHeads)),
                      dim3(256), (size_t)smem, s, 1, P);
}

} // namespace csa2
