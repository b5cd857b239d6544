// Instances and dispatch of the 4-bit products (gemm_mx4.hpp).
#include "gemm_mx4.hpp"

namespace tbg {

template <int BM, int BN, int S>
static hipError_t launch_mx4_tile(const Mx4GemmParams& p, int out_bf16, unsigned grid, hipStream_t stream) {
  const dim3 g(grid), t(kThreads);
  if (p.g.scaled) {
    if (out_bf16) hipLaunchKernelGGL((gemm_mx4_kernel<BM, BN, S, 1, 1>), g, t, 0, stream, p);
    else hipLaunchKernelGGL((gemm_mx4_kernel<BM, BN, S, 0, 1>), g, t, 0, stream, p);
  } else {
    if (out_bf16) hipLaunchKernelGGL((gemm_mx4_kernel<BM, BN, S, 1, 0>), g, t, 0, stream, p);
    else hipLaunchKernelGGL((gemm_mx4_kernel<BM, BN, S, 0, 0>), g, t, 0, stream, p);
  }
  return hipGetLastError();
}

template <int B, int S>
static hipError_t launch_mx4_walk(const Mx4GemmParams& p, int out_bf16, unsigned grid, hipStream_t stream) {
  const dim3 g(grid), t(kThreads);
  if (p.g.scaled) {
    if (out_bf16) hipLaunchKernelGGL((gemm_mx4_walk_kernel<B, S, 1, 1>), g, t, 0, stream, p);
    else hipLaunchKernelGGL((gemm_mx4_walk_kernel<B, S, 0, 1>), g, t, 0, stream, p);
  } else {
    if (out_bf16) hipLaunchKernelGGL((gemm_mx4_walk_kernel<B, S, 1, 0>), g, t, 0, stream, p);
    else hipLaunchKernelGGL((gemm_mx4_walk_kernel<B, S, 0, 0>), g, t, 0, stream, p);
  }
  return hipGetLastError();
}

hipError_t launch_mx4_gemm(Mx4GemmParams p, const TileChoice& c, int out_bf16, hipStream_t stream) {
  p.g.tiles_m = (int)c.tiles_m;
  p.g.tiles_n = (int)c.tiles_n;
  const unsigned g = (unsigned)c.grid;
  if (c.walks) return launch_mx4_walk<256, 2>(p, out_bf16, g, stream);
  if (c.bm == 128 && c.stages == 2) return launch_mx4_tile<128, 128, 2>(p, out_bf16, g, stream);
  if (c.bm == 64 && c.stages == 2) return launch_mx4_tile<64, 64, 2>(p, out_bf16, g, stream);
  if (c.bm == 64 && c.stages == 4) return launch_mx4_tile<64, 64, 4>(p, out_bf16, g, stream);
  if (c.bm == 32 && c.stages == 2) return launch_mx4_tile<32, 64, 2>(p, out_bf16, g, stream);
  if (c.bm == 32 && c.stages == 4) return launch_mx4_tile<32, 64, 4>(p, out_bf16, g, stream);
  return hipErrorInvalidValue;
}

}  // namespace tbg
