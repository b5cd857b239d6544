// Dispatch of the ragged products over the built tiles (gemm_grouped_256.hip, _128, _64).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"

namespace tbg {

template <int B, int S>
hipError_t launch_grouped_tile(const GroupedParams& p, int in, int b_layout, int out, unsigned grid,
                               hipStream_t stream);
template <int B, int S>
hipError_t launch_wgrad_tile(const GroupedParams& p, int in, int out, unsigned grid, hipStream_t stream);

hipError_t launch_grouped(GroupedParams p, const TileChoice& c, int in, int b_layout, int out, hipStream_t stream) {
  p.tiles_m = (int)c.tiles_m;
  p.tiles_n = (int)c.tiles_n;
  const unsigned grid = (unsigned)c.grid;
  if (c.bm == 256) return launch_grouped_tile<256, 2>(p, in, b_layout, out, grid, stream);
  if (c.bm == 128) return launch_grouped_tile<128, 2>(p, in, b_layout, out, grid, stream);
  if (c.bm == 64) return launch_grouped_tile<64, 3>(p, in, b_layout, out, grid, stream);
  return hipErrorInvalidValue;
}

hipError_t launch_wgrad(GroupedParams p, const TileChoice& c, int in, int out, hipStream_t stream) {
  p.tiles_m = (int)c.tiles_m;
  p.tiles_n = (int)c.tiles_n;
  p.per_xcd = (int)c.per_xcd;
  p.by_rows = c.by_rows ? 1 : 0;
  const unsigned grid = (unsigned)c.grid;
  if (c.bm == 256) return launch_wgrad_tile<256, 2>(p, in, out, grid, stream);
  if (c.bm == 128) return launch_wgrad_tile<128, 2>(p, in, out, grid, stream);
  if (c.bm == 64) return launch_wgrad_tile<64, 3>(p, in, out, grid, stream);
  return hipErrorInvalidValue;
}

}  // namespace tbg
