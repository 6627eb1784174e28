// k_paged_decode_e4m3.cu -- one-token attention over a paged cache of GDN_E4M3 values (paged_decode.cuh).
#include "paged_decode.cuh"

namespace gdn {
namespace paged {

template <>
cudaError_t launch_kind<GDN_E4M3>(const AttendArgs &a, int64_t most_tiles16, cudaStream_t stream, int *grid) {
    return dispatch<GDN_E4M3>(a, most_tiles16, stream, grid);
}

}  // namespace paged
}  // namespace gdn
