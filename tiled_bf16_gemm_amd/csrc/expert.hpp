// Host-side launchers of the kernels around the products of expert layers (expert_sort.hip,
// expert_rows.hip), called by the C ABI in api_experts.hip, and the plan of a sort.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert_plan.hpp"
#include "fast_div.hpp"

namespace tbg {

struct SortParams {
  const int32_t* experts;
  int32_t* offsets;
  int32_t* source;
  int32_t* place;
  int32_t* table;  // counts of every part by id (more than one part)
  int64_t part;    // slots a part
  int slots, groups, bits;
};
hipError_t launch_expert_sort(SortParams p, const SortPlan& plan, hipStream_t stream);

// Rows to and from the groups.  Pitches in bytes; a unit is 16 bytes of a row of Y (of X, of dY) or, in a
// row shorter than that, one element; the last unit of a row is moved back to end with the row.
struct RowsParams {
  const uint8_t* in;    // dispatch: X; combine, combine_grad: Y
  const uint8_t* dout;  // combine_grad
  uint8_t* out;         // dispatch: the groups' rows; combine: the tokens' rows; combine_grad: dY
  float* dweights;
  const int32_t* place;
  const float* weights;
  int64_t ld_in, ld_dout, ld_out, cols;
  uint32_t tokens, top_k, rows, per_row, units;
  FastDiv div;  // by per_row
};
// size: bytes of an element
hipError_t launch_expert_dispatch(RowsParams p, int size, hipStream_t stream);
// y, out, d: 0 fp32, 1 bf16, 2 fp16 (out and d are fp32 or y)
hipError_t launch_expert_combine(RowsParams p, int y, int out, hipStream_t stream);
hipError_t launch_expert_combine_grad(RowsParams p, int y, int d, hipStream_t stream);

}  // namespace tbg
