// Tensor-core decode attention that also keeps the scores, 3-bit keys:
// instantiations of the kernel template in tq_attn_mma.cuh for packed 2/3/4-bit
// values, contiguous and paged caches.
#include "tq_attn_mma.cuh"

namespace tq {

int launch_attn_mma_scores_k3(const AttnArgs &a, MmaPlan &plan, int vb, int nt, bool paged, cudaStream_t st) {
#define TQ_CASE(V, N) \
    if (vb == V && nt == N) \
        return paged ? launch_cfg<3, V, false, N, true, true>(a, plan, st) \
                     : launch_cfg<3, V, false, N, false, true>(a, plan, st);
    TQ_CASE(2, 1) TQ_CASE(3, 1) TQ_CASE(4, 1) TQ_CASE(2, 2) TQ_CASE(3, 2) TQ_CASE(4, 2)
#undef TQ_CASE
    return TQ_ERR_UNSUPPORTED;
}

int wait_failed_attn_k3w(unsigned *v, bool clear) { return read_wait_failed(v, clear); }

}  // namespace tq
