// draft.cuh -- launchers of the calls for drafted tokens and shared pages (include/csa2_draft.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/csa2_draft.h"
#include "paged.cuh"

namespace csa2 {

// The caches of one call, as a kernel's argument.
struct CacheSet {
    PagedView c[CSA2D_MAX_CACHES];
};

cudaError_t launch_tree_plan(const csa2d_tree_args &a, uint32_t *d_status, cudaStream_t s);

size_t tree_attn_ws_bytes(const csa2d_tree_attn_args &a);
cudaError_t launch_tree_attn(const csa2d_tree_attn_args &a, const PagedView &v, uint16_t *out, float *lse, void *ws,
                             uint32_t *d_status, cudaStream_t s);

cudaError_t launch_tree_verify(const csa2d_verify_args &a, uint32_t *d_status, cudaStream_t s);

cudaError_t launch_compact(const csa2d_compact_args &a, const CacheSet &set, int n, uint32_t *d_status, cudaStream_t s);
cudaError_t launch_page_fork(const csa2d_share_args &a, uint32_t *d_status, cudaStream_t s);
cudaError_t launch_page_free(const csa2d_share_args &a, uint32_t *d_status, cudaStream_t s);
cudaError_t launch_page_copy(const CacheSet &set, int n, const int32_t *src, const int32_t *dst, const int32_t *rows,
                             int32_t count, uint32_t *d_status, cudaStream_t s);

} // namespace csa2
