// Ragged products, 64×64 tiles.
#include "gemm_grouped_instances.hpp"

namespace tbg {
template hipError_t launch_grouped_tile<64, 3>(const GroupedParams&, int, int, int, unsigned, hipStream_t);
template hipError_t launch_wgrad_tile<64, 3>(const GroupedParams&, int, int, unsigned, hipStream_t);
}  // namespace tbg
