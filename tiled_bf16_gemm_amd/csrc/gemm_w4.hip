// Instances and dispatch of the products with weights in 4-bit codes (gemm_w4.hpp).
#include "gemm_w4.hpp"

namespace tbg {

template <int IN, int G>
static hipError_t launch_tile(const W4Params& p, const TileChoice& c, hipStream_t s) {
  const dim3 g((unsigned)c.grid), t(256);
  if (c.bm == 16 && c.bn == 16) hipLaunchKernelGGL((gemm_w4_kernel<IN, G, 1, 1, 4>), g, t, 0, s, p);
  else if (c.bm == 16) hipLaunchKernelGGL((gemm_w4_kernel<IN, G, 1, 4, 4>), g, t, 0, s, p);
  else if (c.bm == 32) hipLaunchKernelGGL((gemm_w4_kernel<IN, G, 2, 4, 4>), g, t, 0, s, p);
  else hipLaunchKernelGGL((gemm_w4_kernel<IN, G, 4, 2, 4>), g, t, 0, s, p);
  return hipGetLastError();
}

template <int IN>
static hipError_t launch_group(const W4Params& p, int group, const TileChoice& c, hipStream_t s) {
  if (group == 32) return launch_tile<IN, 32>(p, c, s);
  if (group == 64) return launch_tile<IN, 64>(p, c, s);
  return launch_tile<IN, 128>(p, c, s);
}

hipError_t launch_w4_gemm(W4Params p, int in, int group, const TileChoice& c, hipStream_t stream) {
  p.g.tiles_m = (int)c.tiles_m;
  p.g.tiles_n = (int)c.tiles_n;
  p.g.group_m = 8;
  return in == 1 ? launch_group<1>(p, group, c, stream) : launch_group<0>(p, group, c, stream);
}

}  // namespace tbg
