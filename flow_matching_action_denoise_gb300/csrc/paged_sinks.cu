// Attention over a paged cache with a window and first tokens that stay visible (fm_sink_attention): the kernels of
// paged_tile.cuh and paged_decode.cuh for keys in two stretches.

#include "paged_decode.cuh"
#include "paged_tile.cuh"

namespace fm {

template cudaError_t tile_launch<Keys::kSinks>(const AttnParams&, int, bool, const CUtensorMap&, const CUtensorMap&, dim3,
                                               size_t, const LaunchOpts&);
template cudaError_t tile_configure<Keys::kSinks>();
template cudaError_t decode_launch<Keys::kSinks>(const AttnParams&, int, bool, const CUtensorMap&, const CUtensorMap&,
                                                 const LaunchOpts&);
template cudaError_t decode_configure<Keys::kSinks>();

}  // namespace fm
