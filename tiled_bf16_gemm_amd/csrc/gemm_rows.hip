// Instances and dispatch of the products with few rows (gemm_rows.hpp).
#include "gemm_rows.hpp"

namespace tbg {

template <int FMT, int HALF>
static hipError_t launch_rows(const Mx4GemmParams& p, int out, unsigned grid, hipStream_t stream) {
  const dim3 g(grid), t(64 * kRowsWaves);
  if (p.g.scaled) {
    if (out) hipLaunchKernelGGL((gemm_rows_kernel<FMT, HALF, 1>), g, t, 0, stream, p);
    else hipLaunchKernelGGL((gemm_rows_kernel<FMT, 0, 1>), g, t, 0, stream, p);
  } else {
    if (out) hipLaunchKernelGGL((gemm_rows_kernel<FMT, HALF, 0>), g, t, 0, stream, p);
    else hipLaunchKernelGGL((gemm_rows_kernel<FMT, 0, 0>), g, t, 0, stream, p);
  }
  return hipGetLastError();
}

hipError_t launch_few_rows(Mx4GemmParams p, const TileChoice& c, int fmt, int out, hipStream_t stream) {
  p.g.tiles_m = (int)c.tiles_m;
  p.g.tiles_n = (int)c.tiles_n;
  const unsigned grid = (unsigned)c.grid;
  if (fmt == kRowsBf16) return launch_rows<kRowsBf16, 1>(p, out, grid, stream);
  if (fmt == kRowsF16) return launch_rows<kRowsF16, 2>(p, out, grid, stream);
  return launch_rows<kRowsMx4, 1>(p, out, grid, stream);
}

}  // namespace tbg
