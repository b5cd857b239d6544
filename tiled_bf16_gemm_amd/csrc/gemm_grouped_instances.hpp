// Launchers of one tile size of the ragged products: picks the instance by input type, layout,
// output type and scaling.
#pragma once
#include "gemm_grouped.hpp"

namespace tbg {

template <int B, int S>
hipError_t launch_grouped_tile(const GroupedParams& p, int in, int b_layout, int out, unsigned grid,
                               hipStream_t stream) {
  const dim3 g(grid), t(kThreads);
#define TBG_GROUPED(IN, BL, OUT)                                                                                 \
  do {                                                                                                           \
    if (p.scaled) hipLaunchKernelGGL((gemm_grouped_kernel<B, B, S, IN, BL, OUT, 1>), g, t, 0, stream, p);        \
    else hipLaunchKernelGGL((gemm_grouped_kernel<B, B, S, IN, BL, OUT, 0>), g, t, 0, stream, p);                 \
    return hipGetLastError();                                                                                    \
  } while (0)
  if (in == 0 && b_layout == 0 && out == 0) TBG_GROUPED(0, 0, 0);
  if (in == 0 && b_layout == 0 && out == 1) TBG_GROUPED(0, 0, 1);
  if (in == 0 && b_layout == 1 && out == 0) TBG_GROUPED(0, 1, 0);
  if (in == 0 && b_layout == 1 && out == 1) TBG_GROUPED(0, 1, 1);
  if (in == 1 && b_layout == 0 && out == 0) TBG_GROUPED(1, 0, 0);
  if (in == 1 && b_layout == 0 && out == 2) TBG_GROUPED(1, 0, 2);
  if (in == 1 && b_layout == 1 && out == 0) TBG_GROUPED(1, 1, 0);
  if (in == 1 && b_layout == 1 && out == 2) TBG_GROUPED(1, 1, 2);
#undef TBG_GROUPED
  return hipErrorInvalidValue;
}

template <int B, int S>
hipError_t launch_wgrad_tile(const GroupedParams& p, int in, int out, unsigned grid, hipStream_t stream) {
  const dim3 g(grid), t(kThreads);
#define TBG_WGRAD(IN, OUT)                                                                                       \
  do {                                                                                                           \
    if (p.scaled) hipLaunchKernelGGL((gemm_wgrad_kernel<B, B, S, IN, OUT, 1>), g, t, 0, stream, p);              \
    else hipLaunchKernelGGL((gemm_wgrad_kernel<B, B, S, IN, OUT, 0>), g, t, 0, stream, p);                       \
    return hipGetLastError();                                                                                    \
  } while (0)
  if (in == 0 && out == 0) TBG_WGRAD(0, 0);
  if (in == 0 && out == 1) TBG_WGRAD(0, 1);
  if (in == 1 && out == 0) TBG_WGRAD(1, 0);
  if (in == 1 && out == 2) TBG_WGRAD(1, 2);
#undef TBG_WGRAD
  return hipErrorInvalidValue;
}

}  // namespace tbg
