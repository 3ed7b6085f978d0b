// paged_attn.cu -- csa2p_attn: launches the kernel of paged_attn.cuh for tokens in a row.
#include <atomic>

#include "paged_attn.cuh"

namespace csa2 {

cudaError_t allow_smem(const void *kernel, int bytes)
{
    constexpr int kMaxDevices = 64, kKernels = 32;
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

size_t paged_attn_ws_bytes(const csa2p_attn_args &a) { return attn_ws_bytes(a.d_v); }

cudaError_t launch_paged_attn(const csa2p_attn_args &a, const PagedView &v, uint16_t *out, float *lse, void *ws,
                              uint32_t *d_status, cudaStream_t s)
{
    AttnParams P = attn_params(a, v, out, lse, ws, d_status);
    P.ratio = a.ratio_m;
    P.pos0 = a.pos0;
    return launch_attn<false>(P, s);
}

} // namespace csa2
