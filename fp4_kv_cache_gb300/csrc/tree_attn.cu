// tree_attn.cu -- csa2d_tree_attn: launches the kernel of paged_attn.cuh for the nodes of trees.
#include "draft.cuh"
#include "paged_attn.cuh"

namespace csa2 {

size_t tree_attn_ws_bytes(const csa2d_tree_attn_args &a) { return attn_ws_bytes(a.d_v); }

cudaError_t launch_tree_attn(const csa2d_tree_attn_args &a, const PagedView &v, uint16_t *out, float *lse, void *ws,
                             uint32_t *d_status, cudaStream_t s)
{
    AttnParams P = attn_params(a, v, out, lse, ws, d_status);
    P.seen = a.seen;
    P.pos = a.pos;
    P.words = a.words;
    return launch_attn<true>(P, s);
}

} // namespace csa2
