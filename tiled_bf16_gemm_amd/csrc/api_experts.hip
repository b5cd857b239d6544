// The C ABI around the products of expert layers (include/tbg.h): slots sorted by expert, rows to the
// groups and back, and their gradients.  Argument checks on the host; kernels are enqueued on the
// caller's stream.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include "api_util.hpp"
#include "expert.hpp"
#include "tbg.h"

using tbg::check_device;
using tbg::fail;

namespace {

constexpr int64_t kMaxSlots = 1ll << 30;
constexpr int64_t kMaxCols = 1ll << 30;
constexpr int64_t kMaxTopK = 1024;
constexpr int64_t kMaxPitch = 1ll << 40;
constexpr int64_t kGroupLimit = 4096;

typedef long long ll;

bool off(const void* p, int bytes) { return ((uintptr_t)p % bytes) != 0; }

int size_of(tbg_dtype t) {
  switch (t) {
    case TBG_U8: case TBG_F8_E4M3: case TBG_F8_E5M2: return 1;
    case TBG_U16: case TBG_F16: case TBG_BF16: return 2;
    case TBG_U32: case TBG_F32: return 4;
    default: return 0;
  }
}

bool is_value(tbg_dtype t) { return t == TBG_F32 || t == TBG_BF16 || t == TBG_F16; }
int code_of(tbg_dtype t) { return t == TBG_BF16 ? 1 : t == TBG_F16 ? 2 : 0; }

// The sizes that the calls by token share.
tbg_status check_shape(int64_t tokens, int64_t top_k, int64_t rows, int64_t cols) {
  if (tokens < 0 || top_k < 0 || rows < 0 || cols < 0)
    return fail(TBG_ERR_INVALID_VALUE, "negative size tokens=%lld top_k=%lld rows=%lld cols=%lld", (ll)tokens, (ll)top_k,
                (ll)rows, (ll)cols);
  if (top_k > kMaxTopK) return fail(TBG_ERR_UNSUPPORTED, "top_k=%lld: at most %lld", (ll)top_k, (ll)kMaxTopK);
  if (tokens > kMaxSlots || rows > kMaxSlots || cols > kMaxCols || tokens * (top_k > 0 ? top_k : 1) > kMaxSlots)
    return fail(TBG_ERR_UNSUPPORTED, "tokens*top_k, rows and cols are limited to 2^30 (%lld x %lld, %lld, %lld)", (ll)tokens,
                (ll)top_k, (ll)rows, (ll)cols);
  return TBG_OK;
}

// One matrix of `rows` rows of cols elements of `size` bytes.
tbg_status check_matrix(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, int size) {
  if (ld < cols) return fail(TBG_ERR_INVALID_VALUE, "%s: a pitch of %lld below its %lld columns", name, (ll)ld, (ll)cols);
  if (ld > kMaxPitch) return fail(TBG_ERR_UNSUPPORTED, "%s: pitches are limited to 2^40 elements", name);
  if (rows > 0 && cols > 0 && !p) return fail(TBG_ERR_INVALID_VALUE, "%s is NULL", name);
  if (off(p, size)) return fail(TBG_ERR_MISALIGNED, "%s must be aligned to its elements", name);
  return TBG_OK;
}

// An array of 4-byte values.
tbg_status check_array(const char* name, const void* p, int64_t n) {
  if (n > 0 && !p) return fail(TBG_ERR_INVALID_VALUE, "%s is NULL", name);
  if (off(p, 4)) return fail(TBG_ERR_MISALIGNED, "%s must be 4-byte aligned", name);
  return TBG_OK;
}

tbg_status launch_status(const char* what, hipError_t e) {
  if (e == hipSuccess) return TBG_OK;
  return fail(TBG_ERR_HIP, "%s launch: %s", what, hipGetErrorString(e));
}

}  // namespace

extern "C" {

size_t tbg_expert_sort_workspace_query(int64_t slots, int64_t groups) {
  if (slots < 0 || groups < 0 || slots > kMaxSlots || groups > kGroupLimit) return 0;
  return (size_t)tbg::plan_expert_sort(slots, groups).bytes;
}

tbg_status tbg_expert_sort(int64_t slots, int64_t groups, const int32_t* experts, int32_t* offsets, int32_t* source,
                           int32_t* place, void* workspace, size_t workspace_bytes, void* stream) {
  if (slots < 0 || groups < 0)
    return fail(TBG_ERR_INVALID_VALUE, "negative size slots=%lld groups=%lld", (ll)slots, (ll)groups);
  if (slots > kMaxSlots || groups > kGroupLimit)
    return fail(TBG_ERR_UNSUPPORTED, "slots are limited to 2^30, groups to %lld (%lld, %lld)", (ll)kGroupLimit, (ll)slots,
                (ll)groups);
  tbg_status st = check_array("experts", experts, slots);
  if (st == TBG_OK) st = check_array("offsets", offsets, 1);
  if (st == TBG_OK) st = check_array("source", source, slots);
  if (st == TBG_OK) st = check_array("place", place, slots);
  if (st != TBG_OK) return st;
  const tbg::SortPlan plan = tbg::plan_expert_sort(slots, groups);
  if (plan.bytes > 0) {
    if (!workspace || workspace_bytes < (size_t)plan.bytes)
      return fail(TBG_ERR_OUT_OF_RANGE, "workspace of %lld bytes needed (have %zu)", (ll)plan.bytes,
                  workspace ? workspace_bytes : (size_t)0);
    if (off(workspace, 256)) return fail(TBG_ERR_MISALIGNED, "workspace must be 256-byte aligned");
  }
  st = check_device();
  if (st != TBG_OK) return st;
  tbg::SortParams p;
  memset(&p, 0, sizeof(p));
  p.experts = experts;
  p.offsets = offsets;
  p.source = source;
  p.place = place;
  p.table = (int32_t*)workspace;
  p.slots = (int)slots;
  p.groups = (int)groups;
  return launch_status("expert sort", tbg::launch_expert_sort(p, plan, (hipStream_t)stream));
}

tbg_status tbg_expert_dispatch(int64_t tokens, int64_t top_k, int64_t rows, int64_t cols, tbg_dtype dtype,
                               const void* X, int64_t ldx, const int32_t* place, void* out, int64_t ld_out,
                               void* stream) {
  tbg_status st = check_shape(tokens, top_k, rows, cols);
  if (st != TBG_OK) return st;
  const int size = size_of(dtype);
  if (size == 0) return fail(TBG_ERR_INVALID_VALUE, "unknown element type %d", (int)dtype);
  st = check_matrix("X", X, tokens, cols, ldx, size);
  if (st == TBG_OK) st = check_matrix("out", out, rows, cols, ld_out, size);
  if (st == TBG_OK) st = check_array("place", place, tokens * top_k);
  if (st != TBG_OK || tokens == 0 || top_k == 0 || rows == 0 || cols == 0) return st;
  st = check_device();
  if (st != TBG_OK) return st;
  tbg::RowsParams p;
  memset(&p, 0, sizeof(p));
  p.in = (const uint8_t*)X;
  p.out = (uint8_t*)out;
  p.place = place;
  p.ld_in = ldx * size;
  p.ld_out = ld_out * size;
  p.cols = cols;
  p.tokens = (uint32_t)tokens;
  p.top_k = (uint32_t)top_k;
  p.rows = (uint32_t)rows;
  return launch_status("expert dispatch", tbg::launch_expert_dispatch(p, size, (hipStream_t)stream));
}

tbg_status tbg_expert_combine(int64_t tokens, int64_t top_k, int64_t rows, int64_t cols, const void* Y, int64_t ldy,
                              tbg_dtype y_dtype, const int32_t* place, const float* weights, void* out,
                              int64_t ld_out, tbg_dtype out_dtype, void* stream) {
  tbg_status st = check_shape(tokens, top_k, rows, cols);
  if (st != TBG_OK) return st;
  if (!is_value(y_dtype)) return fail(TBG_ERR_INVALID_VALUE, "Y must be TBG_F32, TBG_BF16 or TBG_F16 (got %d)", (int)y_dtype);
  if (out_dtype != TBG_F32 && out_dtype != y_dtype)
    return fail(TBG_ERR_INVALID_VALUE, "out must be TBG_F32 or Y's type (got %d)", (int)out_dtype);
  const int size = size_of(y_dtype), size_out = size_of(out_dtype);
  st = check_matrix("Y", Y, top_k > 0 && tokens > 0 ? rows : 0, cols, ldy, size);
  if (st == TBG_OK) st = check_matrix("out", out, tokens, cols, ld_out, size_out);
  if (st == TBG_OK) st = check_array("place", place, tokens * top_k);
  if (st == TBG_OK) st = check_array("weights", weights, 0);
  if (st != TBG_OK || tokens == 0 || cols == 0) return st;
  st = check_device();
  if (st != TBG_OK) return st;
  tbg::RowsParams p;
  memset(&p, 0, sizeof(p));
  p.in = (const uint8_t*)Y;
  p.out = (uint8_t*)out;
  p.place = place;
  p.weights = weights;
  p.ld_in = ldy * size;
  p.ld_out = ld_out * size_out;
  p.cols = cols;
  p.tokens = (uint32_t)tokens;
  p.top_k = (uint32_t)top_k;
  p.rows = (uint32_t)rows;
  return launch_status("expert combine",
                       tbg::launch_expert_combine(p, code_of(y_dtype), code_of(out_dtype), (hipStream_t)stream));
}

tbg_status tbg_expert_combine_grad(int64_t tokens, int64_t top_k, int64_t rows, int64_t cols, const void* dout,
                                   int64_t ldd, tbg_dtype dout_dtype, const void* Y, int64_t ldy, tbg_dtype y_dtype,
                                   const int32_t* place, const float* weights, void* dY, int64_t ld_dy,
                                   float* dweights, void* stream) {
  tbg_status st = check_shape(tokens, top_k, rows, cols);
  if (st != TBG_OK) return st;
  if (!is_value(y_dtype)) return fail(TBG_ERR_INVALID_VALUE, "Y must be TBG_F32, TBG_BF16 or TBG_F16 (got %d)", (int)y_dtype);
  if (dout_dtype != TBG_F32 && dout_dtype != y_dtype)
    return fail(TBG_ERR_INVALID_VALUE, "dout must be TBG_F32 or Y's type (got %d)", (int)dout_dtype);
  const int size = size_of(y_dtype), size_d = size_of(dout_dtype);
  const int64_t used = top_k > 0 && tokens > 0 ? rows : 0;
  st = check_matrix("dout", dout, used > 0 ? tokens : 0, cols, ldd, size_d);
  if (st == TBG_OK) st = check_matrix("Y", Y, used, cols, ldy, size);
  if (st == TBG_OK) st = check_matrix("dY", dY, used, cols, ld_dy, size);
  if (st == TBG_OK) st = check_array("place", place, tokens * top_k);
  if (st == TBG_OK) st = check_array("weights", weights, 0);
  if (st == TBG_OK) st = check_array("dweights", dweights, tokens * top_k);
  if (st != TBG_OK || tokens == 0 || top_k == 0) return st;
  st = check_device();
  if (st != TBG_OK) return st;
  tbg::RowsParams p;
  memset(&p, 0, sizeof(p));
  p.in = (const uint8_t*)Y;
  p.dout = (const uint8_t*)dout;
  p.out = (uint8_t*)dY;
  p.dweights = dweights;
  p.place = place;
  p.weights = weights;
  p.ld_in = ldy * size;
  p.ld_dout = ldd * size_d;
  p.ld_out = ld_dy * size;
  p.cols = rows > 0 ? cols : 0;
  p.tokens = (uint32_t)tokens;
  p.top_k = (uint32_t)top_k;
  p.rows = (uint32_t)rows;
  return launch_status("expert combine_grad", tbg::launch_expert_combine_grad(p, code_of(y_dtype), code_of(dout_dtype),
                                                                              (hipStream_t)stream));
}

}  // extern "C"
