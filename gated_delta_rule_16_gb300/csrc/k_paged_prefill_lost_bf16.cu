// k_paged_prefill_lost_bf16.cu -- softmax attention of new tokens over the paged cache: the self-test of the tensor-core kernel's waits, bf16 caches.
#include "paged_prefill_tc.cuh"

namespace gdn {
namespace prefill {

cudaError_t launch_lost_bf16(const PrefillArgs &a, bool tma, int grid, int box, const CUtensorMap (&maps)[2], cudaStream_t stream) {
    return tma ? launch_tc<GDN_BF16, true, true>(a, grid, box, maps, stream) : launch_tc<GDN_BF16, false, true>(a, grid, box, maps, stream);
}

}  // namespace prefill
}  // namespace gdn
