// paged.cuh -- addresses and launchers of the paged-cache calls (include/csa2_paged.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/csa2_paged.h"

namespace csa2 {

// A csa2p_cache resolved for the kernels: strides filled in, pages as a shift.
struct PagedView {
    const uint8_t *codes, *scales;
    int64_t code_page, scale_page;     // bytes between pages
    int64_t n_slots;                   // n_pages * page
    int32_t n_pages, shift, d, fmt;
    int32_t code_row, scale_row;       // bytes a row

    __host__ __device__ int64_t code_at(int32_t slot) const
    {
        return (int64_t)(slot >> shift) * code_page + (int64_t)(slot & ((1 << shift) - 1)) * code_row;
    }
    __host__ __device__ int64_t scale_at(int32_t slot) const
    {
        return (int64_t)(slot >> shift) * scale_page + (int64_t)(slot & ((1 << shift) - 1)) * scale_row;
    }
};

struct RopeView {
    const int32_t *pos;
    const float *cs;
    int64_t n_pos;
    int32_t dim, end0, end1;           // rotated channels; pairs below end0 take axis 0, below end1 axis 1
    int32_t quads;                     // every four pairs of eight channels share an axis and lie aligned
};

bool paged_view(const csa2p_cache &c, PagedView &v);    // false: not a valid cache

// Shared memory beyond the default has to be asked for once per kernel and device.  The limit is the
// kernel's own, for every thread of the process: always the same number of bytes for a kernel.
cudaError_t allow_smem(const void *kernel, int bytes);

cudaError_t launch_page_plan(const csa2p_plan_args &a, uint32_t *d_status, cudaStream_t s);
cudaError_t launch_paged_rope(const uint16_t *x, int64_t x_row, int64_t x_head, uint16_t *out, int64_t out_row,
                              int64_t out_head, int32_t rows, int32_t heads, int32_t d, const RopeView &rope,
                              uint32_t *d_status, cudaStream_t s);
cudaError_t launch_paged_write(const PagedView &v, const uint16_t *x, int64_t ldx, int32_t rows, const int32_t *slot,
                               const RopeView &rope, uint32_t *d_status, cudaStream_t s);
cudaError_t launch_paged_read(const PagedView &v, const int32_t *slot, int32_t rows, uint16_t *out, int64_t ldo,
                              uint32_t *d_status, cudaStream_t s);

size_t paged_attn_ws_bytes(const csa2p_attn_args &a);
cudaError_t launch_paged_attn(const csa2p_attn_args &a, const PagedView &v, uint16_t *out, float *lse, void *ws,
                              uint32_t *d_status, cudaStream_t s);

} // namespace csa2
