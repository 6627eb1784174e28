// k_paged_prefill_e4m3_tma.cu -- softmax attention of new tokens over the paged cache: the tensor-core kernel for 8-bit caches, keys and values by TMA.
#include "paged_prefill_tc.cuh"

namespace gdn {
namespace prefill {

cudaError_t launch_e4m3_tma(const PrefillArgs &a, int grid, int box, const CUtensorMap (&maps)[2], cudaStream_t stream) {
    return launch_tc<GDN_E4M3, true>(a, grid, box, maps, stream);
}

}  // namespace prefill
}  // namespace gdn
