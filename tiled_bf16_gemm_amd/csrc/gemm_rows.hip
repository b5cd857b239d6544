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

hipError_t launch_few_rows(Mx4GemmParams p, int fmt, int out, hipStream_t stream) {
  p.g.tiles_n = (p.g.N + 15) / 16;
  p.g.tiles_m = p.g.offsets ? (int)ragged_tiles_bound(p.g.rows, p.g.groups, 16) : 1;
  int64_t grid = (int64_t)p.g.tiles_m * p.g.tiles_n;
  if (p.g.offsets) grid = (grid + 7) / 8 * 8;
  else if (p.g.rows > 16) return hipErrorInvalidValue;
  if (grid == 0 || p.g.rows == 0) return hipSuccess;
  if (grid > kMaxGrid) return hipErrorInvalidConfiguration;
  if (fmt == kRowsBf16) return launch_rows<kRowsBf16, 1>(p, out, (unsigned)grid, stream);
  if (fmt == kRowsF16) return launch_rows<kRowsF16, 2>(p, out, (unsigned)grid, stream);
  return launch_rows<kRowsMx4, 1>(p, out, (unsigned)grid, stream);
}

}  // namespace tbg
