// Products of bf16 rows with weights in 4-bit codes, a zero for every group.
#include "gemm_w4_instances.hpp"

namespace tbg {

hipError_t launch_w4_bf16_zeros(const W4Params& p, int group, const TileChoice& c, hipStream_t stream) {
  return launch_w4_group<0, true>(p, group, c, stream);
}

}  // namespace tbg
