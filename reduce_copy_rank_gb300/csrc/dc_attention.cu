// Paged attention: the kernels whose results are the outputs.
#include "dc_attention.cuh"

namespace dc {

cudaError_t launch_attend(const AttendParams& p, int dtype, int dim, bool pdl, cudaStream_t s, int* grid) {
  return launch_as<false>(p, dtype, dim, pdl, s, grid);
}

DC_BOUNDS_READER(take_bounds_attention)

}  // namespace dc
