// k_paged_prefill_e4m3.cu -- softmax attention of new tokens over the paged cache: the tensor-core kernel for 8-bit caches whose pages are too small for TMA boxes.
#include "paged_prefill_tc.cuh"

namespace gdn {
namespace prefill {

cudaError_t launch_e4m3(const PrefillArgs &a, int grid, int box, const CUtensorMap (&maps)[2], cudaStream_t stream) {
    return launch_tc<GDN_E4M3, false>(a, grid, box, maps, stream);
}

}  // namespace prefill
}  // namespace gdn
