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

hipError_t launch_grouped(GroupedParams p, int bm, int bn, int in, int b_layout, int out, hipStream_t stream) {
  p.tiles_n = (p.N + bn - 1) / bn;
  p.tiles_m = (int)ragged_tiles_bound(p.rows, p.groups, bm);
  // the XCD order deals ids in eighths: round the grid up so that every eighth fits
  const int64_t grid = ((int64_t)p.tiles_m * p.tiles_n + 7) / 8 * 8;
  if (grid == 0) return hipSuccess;
  if (grid > kMaxGrid) return hipErrorInvalidConfiguration;
  if (bm == 256 && bn == 256) return launch_grouped_tile<256, 2>(p, in, b_layout, out, (unsigned)grid, stream);
  if (bm == 128 && bn == 128) return launch_grouped_tile<128, 2>(p, in, b_layout, out, (unsigned)grid, stream);
  if (bm == 64 && bn == 64) return launch_grouped_tile<64, 3>(p, in, b_layout, out, (unsigned)grid, stream);
  return hipErrorInvalidValue;
}

hipError_t launch_wgrad(GroupedParams p, int bm, int bn, int in, int out, hipStream_t stream) {
  p.tiles_m = (p.M + bm - 1) / bm;
  p.tiles_n = (p.N + bn - 1) / bn;
  const int64_t per_group = (int64_t)p.tiles_m * p.tiles_n;
  if (per_group == 0 || p.groups == 0) return hipSuccess;
  p.per_xcd = per_group > 8 ? (int)(per_group / 8) : 1;
  p.by_rows = p.groups > 1 && p.groups <= 64 && p.rows >= 256 * p.groups;
  const int64_t round = 8ll * p.per_xcd, grid = (per_group * p.groups + round - 1) / round * round;
  if (grid > kMaxGrid) return hipErrorInvalidConfiguration;
  if (bm == 256 && bn == 256) return launch_wgrad_tile<256, 2>(p, in, out, (unsigned)grid, stream);
  if (bm == 128 && bn == 128) return launch_wgrad_tile<128, 2>(p, in, out, (unsigned)grid, stream);
  if (bm == 64 && bn == 64) return launch_wgrad_tile<64, 3>(p, in, out, (unsigned)grid, stream);
  return hipErrorInvalidValue;
}

}  // namespace tbg
