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

hipError_t launch_mx4_gemm(Mx4GemmParams p, int bm, int bn, int stages, int out_bf16, int cus, hipStream_t stream) {
  p.g.tiles_m = (p.g.rows + bm - 1) / bm;
  p.g.tiles_n = (p.g.N + bn - 1) / bn;
  if (p.g.offsets) p.g.tiles_m = (int)ragged_tiles_bound(p.g.rows, p.g.groups, bm);
  int64_t grid = (int64_t)p.g.tiles_m * p.g.tiles_n;
  if (grid == 0) return hipSuccess;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  const bool walks = bm == 256 && bn == 256 && stages == 2;
  if (p.g.offsets || walks) grid = (grid + 7) / 8 * 8;
  if (walks) {
    const int64_t walkers = cus >= 8 ? cus / 8 * 8 : 8;
    return launch_mx4_walk<256, 2>(p, out_bf16, (unsigned)(grid < walkers ? grid : walkers), stream);
  }
  if (grid > kMaxGrid) return hipErrorInvalidConfiguration;
  const unsigned g = (unsigned)grid;
  if (bm == 128 && bn == 128 && stages == 2) return launch_mx4_tile<128, 128, 2>(p, out_bf16, g, stream);
  if (bm == 64 && bn == 64 && stages == 2) return launch_mx4_tile<64, 64, 2>(p, out_bf16, g, stream);
  if (bm == 64 && bn == 64 && stages == 4) return launch_mx4_tile<64, 64, 4>(p, out_bf16, g, stream);
  if (bm == 32 && bn == 64 && stages == 2) return launch_mx4_tile<32, 64, 2>(p, out_bf16, g, stream);
  if (bm == 32 && bn == 64 && stages == 4) return launch_mx4_tile<32, 64, 4>(p, out_bf16, g, stream);
  return hipErrorInvalidValue;
}

}  // namespace tbg
