// k_paged_prefill_bf16.cu -- softmax attention of new tokens over the paged cache: the tensor-core kernel for bf16 caches whose pages are too small for TMA boxes.
#include "paged_prefill_tc.cuh"

namespace gdn {
namespace prefill {

cudaError_t launch_bf16(const PrefillArgs &a, int grid, int box, const CUtensorMap (&maps)[2], cudaStream_t stream) {
    return launch_tc<GDN_BF16, false>(a, grid, box, maps, stream);
}

}  // namespace prefill
}  // namespace gdn
