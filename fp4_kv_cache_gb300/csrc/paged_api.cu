// paged_api.cu -- extern "C" entry points of include/csa2_paged.h: host-side validation before
// any launch; the kernels live in paged.cu and paged_attn.cu.
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "paged.cuh"

using namespace csa2;

namespace {

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
// Addresses of 4-byte values, NULL among them.
template <typename... P>
inline bool words(const P *...p) { return (aligned(p, 4) && ...); }
inline csa2_status from_cuda(cudaError_t e) { return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA; }
inline cudaStream_t as_stream(csa2_stream s) { return reinterpret_cast<cudaStream_t>(s); }
inline bool pow2_page(int32_t p) { return p >= 1 && p <= 65536 && (p & (p - 1)) == 0; }

// false: not a valid rotation of `rows` rows of d channels
bool rope_view(const csa2p_rope_axes *r, int32_t d, int32_t rows, RopeView &v)
{
    v = {nullptr, nullptr, 0, 0, 0, 0, 0};
    if (!r || r->rope_dim == 0) return true;
    if (r->rope_dim < 0 || r->rope_dim % 2 || r->rope_dim > d) return false;
    if (r->n_axes < 1 || r->n_axes > 3) return false;
    int64_t sum = 0;
    for (int k = 0; k < r->n_axes; ++k) {
        if (r->section[k] < 0) return false;
        sum += r->section[k];
    }
    if (sum != r->rope_dim / 2) return false;
    if (rows == 0) return true;                            // nothing is read: an empty tensor has no address
    if (!r->pos || !r->cos_sin || r->n_pos < 1 || !aligned(r->pos, 4) || !aligned(r->cos_sin, 4)) return false;
    v.pos = r->pos;
    v.cs = r->cos_sin;
    v.n_pos = r->n_pos;
    v.dim = r->rope_dim;
    v.end0 = r->section[0];
    v.end1 = r->n_axes > 1 ? r->section[0] + r->section[1] : r->section[0];
    v.quads = (d - v.dim) % 8 == 0 && v.dim % 8 == 0 && v.end0 % 4 == 0 && v.end1 % 4 == 0 && aligned(r->cos_sin, 16);
    return true;
}

// Whether no two of the vectors of d elements at r * row + h * head share one (row, head >= d where
// there are several).  Rows within heads, heads within rows: seen at once; else head by head.
bool apart(int64_t row, int64_t head, int32_t rows, int32_t heads, int32_t d)
{
    if (rows < 2 || heads < 2) return true;
    const __int128 R = row, H = head;
    if (R >= H * (heads - 1) + d || H >= R * (rows - 1) + d) return true;
    for (int64_t h = 1; h < heads; ++h) {
        const __int128 at = H * h, r = at / R;
        if (r >= rows) break;                              // and further off with every head
        if ((r > 0 && at - r * R < d) || (r + 1 < rows && (r + 1) * R - at < d)) return false;
    }
    return true;
}

// 0: fine, else the status to return
csa2_status attn_check(const csa2p_attn_args *a, PagedView &v)
{
    if (!a || !paged_view(a->cache, v)) return CSA2_ERR_INVALID_ARG;
    if (a->batch < 0 || a->batch > CSA2P_MAX_BATCH || a->n_tokens < 0) return CSA2_ERR_INVALID_ARG;
    if (a->n_heads < 1 || a->n_heads > 128) return CSA2_ERR_INVALID_ARG;
    if (a->d_v < 8 || a->d_v % 8 || a->d_v > v.d) return CSA2_ERR_INVALID_ARG;
    if (v.d > 576 || a->d_v > 512) return CSA2_ERR_UNSUPPORTED;
    // the kernel tells rows by 32-bit offsets: codes in 16 bytes, scales in bytes
    if (v.code_page * v.n_pages >= (int64_t(1) << 36) || v.scale_page * v.n_pages >= (int64_t(1) << 32)) return CSA2_ERR_UNSUPPORTED;
    if (a->width < 0 || a->window < 0 || a->ratio_m < 1) return CSA2_ERR_INVALID_ARG;
    // the kernel takes logits to base 2: the scale times log2(e) has to be a float
    if (!(a->sm_scale > 0.0f) || a->sm_scale > 2.3e38f) return CSA2_ERR_INVALID_ARG;
    if (a->batch == 0 || a->n_tokens == 0) return CSA2_OK;
    if ((int64_t)a->n_tokens * a->n_heads > 0x7fffffff - 128) return CSA2_ERR_INVALID_ARG;
    if (!a->q || !aligned(a->q, 16) || !a->lens || !a->cu || (a->width > 0 && !a->block_table)) return CSA2_ERR_INVALID_ARG;
    if (!words(a->block_table, a->lens, a->cu, a->pos0, a->kv_start)) return CSA2_ERR_INVALID_ARG;
    if (!a->pos0 && a->ratio_m != 1) return CSA2_ERR_INVALID_ARG;
    return CSA2_OK;
}

} // namespace

extern "C" {

csa2_status csa2p_page_plan(const csa2p_plan_args *a, uint32_t *d_status, csa2_stream stream)
{
    if (!a || a->batch < 0 || a->batch > CSA2P_MAX_BATCH || !pow2_page(a->page) || a->width < 1) return CSA2_ERR_INVALID_ARG;
    if (a->free_cap < 0 || a->n_rows < 0) return CSA2_ERR_INVALID_ARG;
    if (!a->n_free || !a->n_free_out || !a->cu) return CSA2_ERR_INVALID_ARG;
    if (a->batch > 0 && (!a->lens || !a->delta || !a->lens_out || !a->block_table)) return CSA2_ERR_INVALID_ARG;
    if ((a->free_cap > 0 && !a->free_pages) || (a->n_rows > 0 && !a->slot)) return CSA2_ERR_INVALID_ARG;
    if (!words(a->lens, a->delta, a->lens_out, a->block_table, a->free_pages, a->n_free, a->n_free_out, a->cu, a->slot,
               a->row_req, a->row_pos, d_status)) return CSA2_ERR_INVALID_ARG;
    return from_cuda(launch_page_plan(*a, d_status, as_stream(stream)));
}

csa2_status csa2p_rope(const uint16_t *x, int64_t x_row, int64_t x_head, uint16_t *out, int64_t out_row,
                       int64_t out_head, int32_t rows, int32_t heads, int32_t d, const csa2p_rope_axes *rope,
                       uint32_t *d_status, csa2_stream stream)
{
    RopeView v;
    if (rows < 0 || heads < 0 || d < 8 || d % 8 || d > (1 << 20) || !rope_view(rope, d, rows, v)) return CSA2_ERR_INVALID_ARG;
    if (rows == 0 || heads == 0) return CSA2_OK;
    if ((int64_t)heads * d > 0x7fffffff) return CSA2_ERR_INVALID_ARG;
    if (!x || !out || !aligned(x, 16) || !aligned(out, 16) || !words(d_status)) return CSA2_ERR_INVALID_ARG;
    if (x_row % 8 || x_head % 8 || out_row % 8 || out_head % 8) return CSA2_ERR_INVALID_ARG;
    if (x_row < 0 || x_head < 0 || (heads > 1 && out_head < d) || (rows > 1 && out_row < d)) return CSA2_ERR_INVALID_ARG;
    if (!apart(out_row, out_head, rows, heads, d)) return CSA2_ERR_INVALID_ARG;
    if (out == x && (x_row != out_row || x_head != out_head)) return CSA2_ERR_INVALID_ARG;
    return from_cuda(launch_paged_rope(x, x_row, x_head, out, out_row, out_head, rows, heads, d, v, d_status, as_stream(stream)));
}

csa2_status csa2p_write(const csa2p_cache *cache, const uint16_t *x, int64_t ldx, int32_t rows, const int32_t *slot,
                        const csa2p_rope_axes *rope, uint32_t *d_status, csa2_stream stream)
{
    PagedView v;
    RopeView r;
    if (!cache || !paged_view(*cache, v) || rows < 0 || !rope_view(rope, v.d, rows, r)) return CSA2_ERR_INVALID_ARG;
    if (rows == 0) return CSA2_OK;
    if (!x || !slot || !words(slot, d_status) || !aligned(x, 16) || ldx % 8 || ldx < v.d) return CSA2_ERR_INVALID_ARG;
    return from_cuda(launch_paged_write(v, x, ldx, rows, slot, r, d_status, as_stream(stream)));
}

csa2_status csa2p_read(const csa2p_cache *cache, const int32_t *slot, int32_t rows, uint16_t *out, int64_t ldo,
                       uint32_t *d_status, csa2_stream stream)
{
    PagedView v;
    if (!cache || !paged_view(*cache, v) || rows < 0) return CSA2_ERR_INVALID_ARG;
    if (rows == 0) return CSA2_OK;
    if (!out || !slot || !words(slot, d_status) || !aligned(out, 16) || ldo % 8 || ldo < v.d) return CSA2_ERR_INVALID_ARG;
    return from_cuda(launch_paged_read(v, slot, rows, out, ldo, d_status, as_stream(stream)));
}

size_t csa2p_attn_workspace_size(const csa2p_attn_args *a)
{
    PagedView v;
    if (attn_check(a, v) != CSA2_OK || a->batch == 0 || a->n_tokens == 0) return 0;
    return paged_attn_ws_bytes(*a);
}

csa2_status csa2p_attn(const csa2p_attn_args *a, uint16_t *out, float *lse, void *ws, size_t ws_bytes,
                       uint32_t *d_status, csa2_stream stream)
{
    PagedView v;
    const csa2_status st = attn_check(a, v);
    if (st != CSA2_OK) return st;
    if (a->batch == 0 || a->n_tokens == 0) return CSA2_OK;
    if (!out || !aligned(out, 16) || !words(lse, d_status)) return CSA2_ERR_INVALID_ARG;
    const size_t need = paged_attn_ws_bytes(*a);
    if (ws_bytes < need) return CSA2_ERR_WORKSPACE;
    if (need && (!ws || !aligned(ws, 16))) return CSA2_ERR_INVALID_ARG;
    return from_cuda(launch_paged_attn(*a, v, out, lse, need ? ws : nullptr, d_status, as_stream(stream)));
}

} // extern "C"
