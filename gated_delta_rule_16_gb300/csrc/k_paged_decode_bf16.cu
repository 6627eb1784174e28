// k_paged_decode_bf16.cu -- one-token attention over a paged cache of GDN_BF16 values (paged_decode.cuh).
#include "paged_decode.cuh"

namespace gdn {
namespace paged {

template <>
cudaError_t launch_kind<GDN_BF16>(const AttendArgs &a, int64_t most_tiles16, cudaStream_t stream, int *grid) {
    return dispatch<GDN_BF16>(a, most_tiles16, stream, grid);
}

}  // namespace paged
}  // namespace gdn
