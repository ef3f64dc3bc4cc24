// Paged attention: the kernels that leave parts, for attention to shared prefixes.
// (Kernels of their own: a branch for it costs the others 44 bytes of spills and 3 %
// of 128 ragged sequences, 348 -> 359 us; files of their own: compiled side by side.)
#include "dc_attention.cuh"

namespace dc {

cudaError_t launch_attend_parts(const AttendParams& p, int dtype, int dim, bool pdl, cudaStream_t s, int* grid) {
  return launch_as<true>(p, dtype, dim, pdl, s, grid);
}

DC_BOUNDS_READER(take_bounds_attention_parts)

}  // namespace dc
