// k_paged_prefill_bf16.cu -- softmax attention of new tokens over the paged cache: the tensor-core kernel for bf16 caches.
#include "paged_prefill_tc.cuh"

namespace gdn {
namespace prefill {

cudaError_t launch_bf16(const PrefillArgs &a, int grid, cudaStream_t stream) {
    return launch_tc<GDN_BF16>(a, grid, stream);
}

}  // namespace prefill
}  // namespace gdn
