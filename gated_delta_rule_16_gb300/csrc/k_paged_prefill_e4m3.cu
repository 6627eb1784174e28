// k_paged_prefill_e4m3.cu -- softmax attention of new tokens over the paged cache: the tensor-core kernel for 8-bit caches.
#include "paged_prefill_tc.cuh"

namespace gdn {
namespace prefill {

cudaError_t launch_e4m3(const PrefillArgs &a, int grid, cudaStream_t stream) {
    return launch_tc<GDN_E4M3>(a, grid, stream);
}

}  // namespace prefill
}  // namespace gdn
