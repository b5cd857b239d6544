// Dispatch of the products with weights in 4-bit codes over one activation type (gemm_w4.hpp); one
// translation unit instantiates each.
#pragma once
#include "gemm_w4.hpp"

namespace tbg {

template <int IN, bool ZEROS, int G>
static hipError_t launch_w4_tile(const W4Params& p, const TileChoice& c, hipStream_t s) {
  const dim3 g((unsigned)c.grid), t(256);
  if (c.few && c.bn == 16) hipLaunchKernelGGL((gemm_w4_kernel<IN, ZEROS, G, 1>), g, t, 0, s, p);
  else if (c.few && c.bn == 32) hipLaunchKernelGGL((gemm_w4_kernel<IN, ZEROS, G, 2>), g, t, 0, s, p);
  else if (c.few) hipLaunchKernelGGL((gemm_w4_kernel<IN, ZEROS, G, 4>), g, t, 0, s, p);
  else if (c.bm == 16) hipLaunchKernelGGL((gemm_w4_panel_kernel<IN, ZEROS, G, 1, 2, 5>), g, t, 0, s, p);
  else if (c.bm == 32) hipLaunchKernelGGL((gemm_w4_panel_kernel<IN, ZEROS, G, 2, 2, 4>), g, t, 0, s, p);
  else hipLaunchKernelGGL((gemm_w4_panel_kernel<IN, ZEROS, G, 4, 2, 2>), g, t, 0, s, p);
  return hipGetLastError();
}

template <int IN, bool ZEROS>
static hipError_t launch_w4_group(const W4Params& p, int group, const TileChoice& c, hipStream_t s) {
  if (group == 32) return launch_w4_tile<IN, ZEROS, 32>(p, c, s);
  if (group == 64) return launch_w4_tile<IN, ZEROS, 64>(p, c, s);
  return launch_w4_tile<IN, ZEROS, 128>(p, c, s);
}

}  // namespace tbg
