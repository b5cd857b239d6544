// Ragged products, 128×128 tiles.
#include "gemm_grouped_instances.hpp"

namespace tbg {
template hipError_t launch_grouped_tile<128, 2>(const GroupedParams&, int, int, int, unsigned, hipStream_t);
template hipError_t launch_wgrad_tile<128, 2>(const GroupedParams&, int, int, unsigned, hipStream_t);
}  // namespace tbg
