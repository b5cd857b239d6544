// Products of bf16 rows with weights in 4-bit codes, every zero 8.
#include "gemm_w4_instances.hpp"

namespace tbg {

hipError_t launch_w4_bf16(const W4Params& p, int group, const TileChoice& c, hipStream_t stream) {
  return launch_w4_group<0, false>(p, group, c, stream);
}

}  // namespace tbg
