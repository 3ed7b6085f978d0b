// draft_api.cu -- extern "C" entry points of include/csa2_draft.h: host-side validation before any
// launch; the kernels live in draft.cu, shares.cu, verify.cu and paged_attn.cuh.
#include <cuda_runtime.h>
#include <stdint.h>

#include "draft.cuh"
#include "internal.h"

using namespace csa2;

namespace {

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
// Addresses of 4-byte values, NULL among them.
template <typename... P>
inline bool words(const P *...p) { return (aligned(p, 4) && ...); }
inline csa2_status from_cuda(cudaError_t e) { return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA; }
inline cudaStream_t as_stream(csa2_stream s) { return reinterpret_cast<cudaStream_t>(s); }
inline bool batch_ok(int32_t b) { return b >= 0 && b <= CSA2P_MAX_BATCH; }

// 0: fine, else the status to return
csa2_status attn_check(const csa2d_tree_attn_args *a, PagedView &v)
{
    if (!a || !paged_view(a->cache, v)) return CSA2_ERR_INVALID_ARG;
    if (!batch_ok(a->batch) || a->n_tokens < 0) return CSA2_ERR_INVALID_ARG;
    if (a->n_heads < 1 || a->n_heads > 128) return CSA2_ERR_INVALID_ARG;
    if (a->d_v < 8 || a->d_v % 8 || a->d_v > v.d) return CSA2_ERR_INVALID_ARG;
    if (v.d > 576 || a->d_v > 512) return CSA2_ERR_UNSUPPORTED;
    // the kernel tells rows by 32-bit offsets: codes in 16 bytes, scales in bytes
    if (v.code_page * v.n_pages >= (int64_t(1) << 36) || v.scale_page * v.n_pages >= (int64_t(1) << 32)) return CSA2_ERR_UNSUPPORTED;
    if (a->width < 0 || a->window < 0 || a->words < 1 || a->words > CSA2D_MAX_WORDS) return CSA2_ERR_INVALID_ARG;
    // the kernel takes logits to base 2: the scale times log2(e) has to be a float
    if (!(a->sm_scale > 0.0f) || a->sm_scale > 2.3e38f) return CSA2_ERR_INVALID_ARG;
    if (a->batch == 0 || a->n_tokens == 0) return CSA2_OK;
    if ((int64_t)a->n_tokens * a->n_heads > 0x7fffffff - 128) return CSA2_ERR_INVALID_ARG;
    if (!a->q || !aligned(a->q, 16) || !a->lens || !a->cu || !a->seen || (a->width > 0 && !a->block_table)) return CSA2_ERR_INVALID_ARG;
    if (!words(a->block_table, a->lens, a->cu, a->seen, a->pos, a->kv_start)) return CSA2_ERR_INVALID_ARG;
    if (a->window > 0 && !a->pos) return CSA2_ERR_INVALID_ARG;
    return CSA2_OK;
}

// false: too many caches, or one that is none; `one`: of one page size
bool cache_set(const csa2p_cache *caches, int32_t n, bool one, CacheSet &set)
{
    if (n < 0 || n > CSA2D_MAX_CACHES || (n > 0 && !caches)) return false;
    for (int i = 0; i < n; ++i)
        if (!paged_view(caches[i], set.c[i]) || (one && set.c[i].shift != set.c[0].shift)) return false;
    return true;
}

bool shares_ok(const csa2d_share_args *a, const int32_t *which)
{
    if (!batch_ok(a->batch) || a->page < 1 || a->page > 65536 || (a->page & (a->page - 1))) return false;
    if (a->width < 1 || a->n_pages < 0 || a->free_cap < 0 || !a->n_free) return false;
    if (a->batch > 0 && (!which || !a->lens || !a->block_table)) return false;
    if ((a->n_pages > 0 && !a->shares) || (a->free_cap > 0 && !a->free_pages)) return false;
    return words(which, a->lens, a->block_table, a->shares, a->free_pages, a->n_free);
}

} // namespace

extern "C" {

csa2_status csa2d_tree_plan(const csa2d_tree_args *a, uint32_t *d_status, csa2_stream stream)
{
    if (!a || !batch_ok(a->batch) || a->n_tokens < 0 || a->words < 1 || a->words > CSA2D_MAX_WORDS) return CSA2_ERR_INVALID_ARG;
    if (a->n_tokens == 0) return CSA2_OK;
    if (!a->pos || !a->seen) return CSA2_ERR_INVALID_ARG;
    if (a->batch > 0 && (!a->parent || !a->lens || !a->cu)) return CSA2_ERR_INVALID_ARG;
    if (!words(a->parent, a->lens, a->cu, a->pos, a->seen, d_status)) return CSA2_ERR_INVALID_ARG;
    return from_cuda(launch_tree_plan(*a, d_status, as_stream(stream)));
}

size_t csa2d_tree_attn_workspace_size(const csa2d_tree_attn_args *a)
{
    PagedView v;
    if (attn_check(a, v) != CSA2_OK || a->batch == 0 || a->n_tokens == 0) return 0;
    return tree_attn_ws_bytes(*a);
}

csa2_status csa2d_tree_attn(const csa2d_tree_attn_args *a, uint16_t *out, float *lse, void *ws, size_t ws_bytes,
                            uint32_t *d_status, csa2_stream stream)
{
    PagedView v;
    const csa2_status st = attn_check(a, v);
    if (st != CSA2_OK) return st;
    if (a->batch == 0 || a->n_tokens == 0) return CSA2_OK;
    if (!out || !aligned(out, 16) || !words(lse, d_status)) return CSA2_ERR_INVALID_ARG;
    const size_t need = tree_attn_ws_bytes(*a);
    if (ws_bytes < need) return CSA2_ERR_WORKSPACE;
    if (need && (!ws || !aligned(ws, 16))) return CSA2_ERR_INVALID_ARG;
    return from_cuda(launch_tree_attn(*a, v, out, lse, need ? ws : nullptr, d_status, as_stream(stream)));
}

csa2_status csa2d_tree_verify(const csa2d_verify_args *a, uint32_t *d_status, csa2_stream stream)
{
    if (!a || !batch_ok(a->batch) || a->n_tokens < 0 || a->vocab < 1 || a->vocab > CSA2D_MAX_VOCAB) return CSA2_ERR_INVALID_ARG;
    if (a->type < CSA2D_F32 || a->type > CSA2D_BF16 || a->max_path < 1) return CSA2_ERR_INVALID_ARG;
    if (a->n_tokens > 1 && (a->p_row < a->vocab || (a->q && a->q_row < a->vocab))) return CSA2_ERR_INVALID_ARG;
    if (a->batch == 0) return CSA2_OK;
    if (!a->cu || !a->r || !a->keep || !a->path || !a->next_token || !a->delta) return CSA2_ERR_INVALID_ARG;
    if (a->n_tokens > 0 && (!a->p || !a->token || !a->parent || !a->u)) return CSA2_ERR_INVALID_ARG;
    const size_t value = a->type == CSA2D_F32 ? 4 : 2;
    if (!aligned(a->p, value) || !aligned(a->q, value)) return CSA2_ERR_INVALID_ARG;
    if (!words(a->token, a->parent, a->cu, a->u, a->r, a->keep, a->path, a->next_token, a->delta, a->pos, d_status)) return CSA2_ERR_INVALID_ARG;
    return from_cuda(launch_tree_verify(*a, d_status, as_stream(stream)));
}

csa2_status csa2d_compact(const csa2d_compact_args *a, const csa2p_cache *caches, int32_t n, uint32_t *d_status,
                          csa2_stream stream)
{
    CacheSet set;
    if (!a || !batch_ok(a->batch) || a->width < 0 || a->max_path < 0 || !cache_set(caches, n, true, set)) return CSA2_ERR_INVALID_ARG;
    if (a->batch == 0 || n == 0) return CSA2_OK;
    if (!a->lens || !a->cu || !a->keep || (a->width > 0 && !a->block_table) || (a->max_path > 0 && !a->path)) return CSA2_ERR_INVALID_ARG;
    if (a->pos && a->n_tokens < 0) return CSA2_ERR_INVALID_ARG;
    if (!words(a->block_table, a->lens, a->cu, a->path, a->keep, a->pos, a->delta, d_status)) return CSA2_ERR_INVALID_ARG;
    return from_cuda(launch_compact(*a, set, n, d_status, as_stream(stream)));
}

csa2_status csa2d_page_fork(const csa2d_share_args *a, uint32_t *d_status, csa2_stream stream)
{
    if (!a || !shares_ok(a, a->source) || !words(a->src, a->dst, a->rows, d_status)) return CSA2_ERR_INVALID_ARG;
    if (a->batch == 0) return CSA2_OK;
    if (!a->src || !a->dst || !a->rows) return CSA2_ERR_INVALID_ARG;
    return from_cuda(launch_page_fork(*a, d_status, as_stream(stream)));
}

csa2_status csa2d_page_free(const csa2d_share_args *a, uint32_t *d_status, csa2_stream stream)
{
    if (!a || !shares_ok(a, a->ends) || !words(d_status)) return CSA2_ERR_INVALID_ARG;
    if (a->batch == 0) return CSA2_OK;
    return from_cuda(launch_page_free(*a, d_status, as_stream(stream)));
}

csa2_status csa2d_page_copy(const csa2p_cache *caches, int32_t n, const int32_t *src, const int32_t *dst,
                            const int32_t *rows, int32_t count, uint32_t *d_status, csa2_stream stream)
{
    CacheSet set;
    if (count < 0 || !cache_set(caches, n, false, set)) return CSA2_ERR_INVALID_ARG;
    if (count == 0 || n == 0) return CSA2_OK;
    if (!src || !dst || !words(src, dst, rows, d_status)) return CSA2_ERR_INVALID_ARG;
    return from_cuda(launch_page_copy(set, n, src, dst, rows, count, d_status, as_stream(stream)));
}

} // extern "C"
