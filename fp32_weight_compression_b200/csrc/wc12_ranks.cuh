// wc12_ranks.cuh -- which values of a row of r ranks the lanes of the product of
// t and B read (k_split12_adapters.cu).  Plain arithmetic, so that its bounds
// are tested on the host.
#pragma once

#include <cstdint>

namespace wc12a {

// In the step of 16 ranks from j on, the lanes with t = lane % 4 take 4 ranks
// from j + 4 t on.  r is a multiple of 8: the last step of one that is no
// multiple of 16 has them for t = 0 and 1 only.
__host__ __device__ inline bool has_ranks(uint32_t j, uint32_t t, uint32_t r) { return j + 4 * t < r; }
// Where such a lane reads: lanes without ranks the row's first four (and drop
// them), never past the row, behind whose last there may be nothing.
__host__ __device__ inline uint32_t ranks_from(uint32_t j, uint32_t t, uint32_t r) {
  return has_ranks(j, t, r) ? j + 4 * t : 0;
}

}  // namespace wc12a
