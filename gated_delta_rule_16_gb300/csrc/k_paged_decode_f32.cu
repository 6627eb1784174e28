// k_paged_decode_f32.cu -- one-token attention over a paged cache of GDN_F32 values (paged_decode.cuh).
#include "paged_decode.cuh"

namespace gdn {
namespace paged {

template <>
cudaError_t launch_kind<GDN_F32>(const AttendArgs &a, int64_t most_tiles16, cudaStream_t stream, int *grid) {
    return dispatch<GDN_F32>(a, most_tiles16, stream, grid);
}

}  // namespace paged
}  // namespace gdn
