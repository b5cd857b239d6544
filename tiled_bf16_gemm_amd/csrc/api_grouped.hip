// The C ABI of the ragged and the 4-bit products (include/tbg.h): argument checks, repacking and the
// choice of a tile.  Host code only; kernels are enqueued on the caller's stream.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include "api_util.hpp"
#include "launch.hpp"
#include "tbg.h"
#include "tile_choice.hpp"

using tbg::check_device;
using tbg::fail;
using tbg::round_up;

namespace {

constexpr int64_t kMaxLd = (1ll << 22) - 1;     // elements of a 16-bit operand
constexpr int64_t kMaxPitch4 = (1ll << 23) - 16;  // bytes of a row of codes or scales
constexpr int64_t kMaxSize = 1ll << 30;
constexpr int64_t kMaxLdc = 1ll << 40;
constexpr int64_t kGroupLimit = 4096;

typedef long long ll;

bool off16(const void* p) { return ((uintptr_t)p % 16) != 0; }

// The part of the arguments that every ragged call shares.
tbg_status check_groups(int64_t groups, int64_t M, const int32_t* offsets) {
  if (groups < 0 || M < 0) return fail(TBG_ERR_INVALID_VALUE, "negative size groups=%lld M=%lld", (ll)groups, (ll)M);
  if (groups > kGroupLimit)
    return fail(TBG_ERR_UNSUPPORTED, "groups=%lld: at most %lld", (ll)groups, (ll)kGroupLimit);
  if (groups > 0 && !offsets) return fail(TBG_ERR_INVALID_VALUE, "offsets is NULL");
  if (((uintptr_t)offsets) % 4 != 0) return fail(TBG_ERR_MISALIGNED, "offsets must be 4-byte aligned");
  return TBG_OK;
}

tbg_status check_sizes(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0)
    return fail(TBG_ERR_INVALID_VALUE, "negative size %lld, %lld or %lld", (ll)M, (ll)N, (ll)K);
  if (M > kMaxSize || N > kMaxSize || K > kMaxSize)
    return fail(TBG_ERR_UNSUPPORTED, "sizes are limited to 2^30 (%lld, %lld, %lld)", (ll)M, (ll)N, (ll)K);
  return TBG_OK;
}

tbg_status check_ld(const char* name, int64_t ld, int64_t least, int64_t most) {
  if (ld < (least > 0 ? least : 1))
    return fail(TBG_ERR_INVALID_VALUE, "%s=%lld below its minimum %lld", name, (ll)ld, (ll)(least > 0 ? least : 1));
  if (ld > most) return fail(TBG_ERR_UNSUPPORTED, "%s=%lld: at most %lld", name, (ll)ld, (ll)most);
  return TBG_OK;
}

tbg_status check_types(tbg_dtype ab, tbg_dtype c) {
  if (ab != TBG_BF16 && ab != TBG_F16)
    return fail(TBG_ERR_INVALID_VALUE, "operands must be TBG_BF16 or TBG_F16 (got %d)", (int)ab);
  if (c != TBG_F32 && c != ab)
    return fail(TBG_ERR_INVALID_VALUE, "C must be TBG_F32 or the operands' type (got %d)", (int)c);
  return TBG_OK;
}

int out_code(tbg_dtype c) { return c == TBG_BF16 ? 1 : c == TBG_F16 ? 2 : 0; }
int out_size(tbg_dtype c) { return c == TBG_F32 ? 4 : 2; }

// ---- repacks -------------------------------------------------------------------------------
// One operand whose rows must start on 16-byte boundaries: `groups` matrices of rows × cols
// 16-bit values, `stride` elements apart, at pitch ld.
struct Repack {
  bool needed;
  int64_t ld;     // elements, after the repack (or the caller's)
  int64_t stride;
  size_t bytes;
};

Repack plan_repack(const void* p, int64_t groups, int64_t stride, int64_t rows, int64_t cols, int64_t ld,
                   bool whole_chunks) {
  Repack r{false, ld, stride, 0};
  if (rows <= 0 || cols <= 0 || groups <= 0) return r;
  r.needed = ld % 8 != 0 || off16(p) || (whole_chunks && cols % 8 != 0) || (groups > 1 && stride % 8 != 0);
  if (r.needed) {
    r.ld = round_up(cols, 8);
    r.stride = rows * r.ld;
    r.bytes = (size_t)round_up(groups * r.stride * 2, 256);
  }
  return r;
}

// What a repack reads: as plan_repack.
struct Operand {
  const void* p;
  int64_t groups, stride, rows, cols, ld;
};

// The repacks of both operands, a's into `area` and b's behind it; a and b then point to the copies.
// Matrices at one pitch throughout go out in one launch (both operands of a small weight gradient:
// 15.9 to 13.5 µs a call with the host).
hipError_t run_repacks(Operand& a, const Repack& ra, Operand& b, const Repack& rb, uint8_t* area, hipStream_t s) {
  tbg::PackJob jobs[2];
  int n = 0;
  hipError_t e = hipSuccess;
  auto add = [&](Operand& o, const Repack& r, uint8_t* dst) {
    if (!r.needed) return;
    tbg::PackJob j{(const uint8_t*)o.p, o.ld * 2, o.rows, o.cols * 2, dst, r.ld * 2};
    if (o.groups == 1 || o.stride == o.rows * o.ld) {
      j.rows = o.groups * o.rows;
      jobs[n++] = j;
    } else if (e == hipSuccess) {
      e = tbg::launch_pack_groups(j, o.groups, o.stride * 2, s);
    }
    o.p = dst;
  };
  add(a, ra, area);
  add(b, rb, area + ra.bytes);
  return e == hipSuccess ? tbg::launch_pack_jobs(jobs, n, s) : e;
}

tbg_status check_workspace(size_t need, const void* workspace, size_t have) {
  if (need == 0) return TBG_OK;
  if (!workspace || have < need)
    return fail(TBG_ERR_OUT_OF_RANGE, "workspace of %zu bytes needed (have %zu)", need, workspace ? have : (size_t)0);
  if (((uintptr_t)workspace) % 256 != 0) return fail(TBG_ERR_MISALIGNED, "workspace must be 256-byte aligned");
  return TBG_OK;
}

tbg_status launch_status(const char* what, hipError_t e) {
  if (e == hipSuccess) return TBG_OK;
  return fail(TBG_ERR_HIP, "%s launch: %s", what, hipGetErrorString(e));
}

// More workgroups than one launch takes: refused before anything is enqueued.
tbg_status check_grid(const tbg::TileChoice& c) {
  if (c.fits()) return TBG_OK;
  return fail(TBG_ERR_UNSUPPORTED, "too many tiles for one launch (%lld x %lld of %dx%d)", (ll)c.tiles_m, (ll)c.tiles_n,
              c.bm, c.bn);
}

}  // namespace

extern "C" {

size_t tbg_gemm_grouped_workspace_query(int64_t groups, int64_t M, int64_t N, int64_t K, tbg_dtype ab_dtype,
                                        const void* A, int64_t lda, const void* B, int64_t ldb, int64_t stride_b,
                                        tbg_b_layout bl) {
  if (ab_dtype != TBG_BF16 && ab_dtype != TBG_F16) return 0;
  if (groups <= 0 || M <= 0 || N <= 0 || K <= 0 || lda <= 0 || ldb <= 0) return 0;
  if (groups > kGroupLimit || M > kMaxSize || N > kMaxSize || K > kMaxSize) return 0;
  const bool nk = bl == TBG_B_NK;
  return plan_repack(A, 1, 0, M, K, lda, true).bytes +
         plan_repack(B, groups, stride_b, nk ? N : K, nk ? K : N, ldb, nk).bytes;
}

tbg_status tbg_gemm_grouped(int64_t groups, int64_t M, int64_t N, int64_t K, const int32_t* offsets, float alpha,
                            const void* A, int64_t lda, const void* B, int64_t ldb, int64_t stride_b, tbg_b_layout bl,
                            tbg_dtype ab_dtype, float beta, void* C, int64_t ldc, tbg_dtype c_dtype, void* workspace,
                            size_t workspace_bytes, void* stream) {
  tbg_status st = check_groups(groups, M, offsets);
  if (st == TBG_OK) st = check_sizes(M, N, K);
  if (st == TBG_OK) st = check_types(ab_dtype, c_dtype);
  if (st != TBG_OK) return st;
  if ((int)bl != TBG_B_KN && (int)bl != TBG_B_NK) return fail(TBG_ERR_INVALID_VALUE, "unknown b_layout %d", (int)bl);
  const bool scaled = !(alpha == 1.f && beta == 0.f);
  if (alpha == 0.f) {  // nothing of A or B is used
    K = 0;
    A = B = nullptr;
    lda = ldb = 1;
    stride_b = 0;
    bl = TBG_B_NK;
  }
  const bool nk = bl == TBG_B_NK;
  const int64_t b_rows = nk ? N : K, b_cols = nk ? K : N;
  st = check_ld("lda", lda, K, kMaxLd);
  if (st == TBG_OK) st = check_ld("ldb", ldb, alpha == 0.f ? 1 : b_cols, kMaxLd);
  if (st == TBG_OK) st = check_ld("ldc", ldc, N, kMaxLdc);
  if (st != TBG_OK) return st;
  if (groups > 1 && K > 0 && N > 0 && stride_b < (b_rows - 1) * ldb + b_cols)
    return fail(TBG_ERR_INVALID_VALUE, "stride_b=%lld below one matrix", (ll)stride_b);
  if (groups == 0 || M == 0 || N == 0) return TBG_OK;
  if (!C) return fail(TBG_ERR_INVALID_VALUE, "C is NULL");
  if (K > 0 && (!A || !B)) return fail(TBG_ERR_INVALID_VALUE, "A or B is NULL");
  const Repack ra = plan_repack(A, 1, 0, M, K, lda, true);
  const Repack rb = plan_repack(B, groups, stride_b, b_rows, b_cols, ldb, nk);
  st = check_workspace(ra.bytes + rb.bytes, workspace, workspace_bytes);
  if (st != TBG_OK) return st;
  int cus = 0;
  st = check_device(&cus);
  if (st != TBG_OK) return st;
  const tbg::TileChoice choice = tbg::choose_grouped(groups, M, N, K, nk, cus);
  st = check_grid(choice);
  if (st != TBG_OK) return st;
  hipStream_t s = (hipStream_t)stream;
  uint8_t* const area = tbg::repack_area(workspace, workspace_bytes, ra.bytes + rb.bytes);
  Operand oa{A, 1, 0, M, K, lda}, ob{B, groups, stride_b, b_rows, b_cols, ldb};
  hipError_t e = run_repacks(oa, ra, ob, rb, area, s);
  if (e != hipSuccess) return fail(TBG_ERR_HIP, "operand repack: %s", hipGetErrorString(e));
  tbg::GroupedParams p;
  memset(&p, 0, sizeof(p));
  p.A = (const uint8_t*)oa.p;
  p.B = (const uint8_t*)ob.p;
  p.C = C;
  p.offsets = offsets;
  p.lda = ra.ld * 2;
  p.ldb = rb.ld * 2;
  p.stride_b = rb.stride * 2;
  p.ldc = ldc;
  p.groups = (int)groups;
  p.rows = (int)M;
  p.N = (int)N;
  p.K = (int)K;
  p.group_m = 8;
  p.vec_store = tbg::rows_dword_aligned(C, ldc, out_size(c_dtype));
  p.alpha = alpha;
  p.beta = beta;
  p.scaled = scaled ? 1 : 0;
  tbg::log_choice("grouped gemm groups=%lld M=%lld N=%lld K=%lld B=%s in=%s out=%s: %s %dx%d; repack A %s, B %s",
                  (ll)groups, (ll)M, (ll)N, (ll)K, nk ? "nk" : "kn", ab_dtype == TBG_F16 ? "f16" : "bf16",
                  c_dtype == TBG_F32 ? "f32" : "16-bit", choice.few ? "rows" : "ring", choice.bm, choice.bn,
                  ra.needed ? "yes" : "no", rb.needed ? "yes" : "no");
  if (choice.few) {
    tbg::Mx4GemmParams q;
    memset(&q, 0, sizeof(q));
    q.g = p;
    e = tbg::launch_few_rows(q, choice, ab_dtype == TBG_F16, out_code(c_dtype), s);
  } else {
    e = tbg::launch_grouped(p, choice, ab_dtype == TBG_F16, (int)bl, out_code(c_dtype), s);
  }
  return launch_status("grouped gemm", e);
}

size_t tbg_gemm_grouped_wgrad_workspace_query(int64_t groups, int64_t M, int64_t P, int64_t Q, tbg_dtype ab_dtype,
                                              const void* X, int64_t ldx, const void* Y, int64_t ldy) {
  if (ab_dtype != TBG_BF16 && ab_dtype != TBG_F16) return 0;
  if (groups <= 0 || M <= 0 || P <= 0 || Q <= 0 || ldx <= 0 || ldy <= 0) return 0;
  if (groups > kGroupLimit || M > kMaxSize || P > kMaxSize || Q > kMaxSize) return 0;
  return plan_repack(X, 1, 0, M, P, ldx, false).bytes + plan_repack(Y, 1, 0, M, Q, ldy, false).bytes;
}

tbg_status tbg_gemm_grouped_wgrad(int64_t groups, int64_t M, int64_t P, int64_t Q, const int32_t* offsets,
                                  float alpha, const void* X, int64_t ldx, const void* Y, int64_t ldy,
                                  tbg_dtype ab_dtype, float beta, void* C, int64_t ldc, int64_t stride_c,
                                  tbg_dtype c_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  tbg_status st = check_groups(groups, M, offsets);
  if (st == TBG_OK) st = check_sizes(M, P, Q);
  if (st == TBG_OK) st = check_types(ab_dtype, c_dtype);
  if (st != TBG_OK) return st;
  const bool scaled = !(alpha == 1.f && beta == 0.f);
  if (alpha == 0.f) {  // no rows: the empty sum for every group
    M = 0;
    X = Y = nullptr;
    ldx = P > 0 ? P : 1;
    ldy = Q > 0 ? Q : 1;
  }
  st = check_ld("ldx", ldx, P, alpha == 0.f ? kMaxSize : kMaxLd);
  if (st == TBG_OK) st = check_ld("ldy", ldy, Q, alpha == 0.f ? kMaxSize : kMaxLd);
  if (st == TBG_OK) st = check_ld("ldc", ldc, Q, kMaxLdc);
  if (st != TBG_OK) return st;
  if (groups > 1 && P > 0 && Q > 0 && stride_c < (P - 1) * ldc + Q)
    return fail(TBG_ERR_INVALID_VALUE, "stride_c=%lld below one matrix", (ll)stride_c);
  if (groups == 0 || P == 0 || Q == 0) return TBG_OK;
  if (!C) return fail(TBG_ERR_INVALID_VALUE, "C is NULL");
  if (M > 0 && (!X || !Y)) return fail(TBG_ERR_INVALID_VALUE, "X or Y is NULL");
  const Repack rx = plan_repack(X, 1, 0, M, P, ldx, false), ry = plan_repack(Y, 1, 0, M, Q, ldy, false);
  st = check_workspace(rx.bytes + ry.bytes, workspace, workspace_bytes);
  if (st != TBG_OK) return st;
  int cus = 0;
  st = check_device(&cus);
  if (st != TBG_OK) return st;
  const tbg::TileChoice choice = tbg::choose_wgrad(groups, M, P, Q, cus);
  st = check_grid(choice);
  if (st != TBG_OK) return st;
  hipStream_t s = (hipStream_t)stream;
  uint8_t* const area = tbg::repack_area(workspace, workspace_bytes, rx.bytes + ry.bytes);
  Operand ox{X, 1, 0, M, P, ldx}, oy{Y, 1, 0, M, Q, ldy};
  hipError_t e = run_repacks(ox, rx, oy, ry, area, s);
  if (e != hipSuccess) return fail(TBG_ERR_HIP, "operand repack: %s", hipGetErrorString(e));
  tbg::GroupedParams p;
  memset(&p, 0, sizeof(p));
  p.A = (const uint8_t*)ox.p;
  p.B = (const uint8_t*)oy.p;
  p.C = C;
  p.offsets = offsets;
  p.lda = rx.ld * 2;
  p.ldb = ry.ld * 2;
  p.ldc = ldc;
  p.stride_c = groups > 1 ? stride_c : 0;
  p.groups = (int)groups;
  p.rows = (int)M;
  p.M = (int)P;
  p.N = (int)Q;
  p.group_m = 4;
  p.vec_store = tbg::rows_dword_aligned(C, ldc, out_size(c_dtype)) &&
                (p.stride_c * out_size(c_dtype)) % 4 == 0;
  p.alpha = alpha;
  p.beta = beta;
  p.scaled = scaled ? 1 : 0;
  tbg::log_choice("grouped wgrad groups=%lld M=%lld P=%lld Q=%lld in=%s out=%s: ring %dx%d; repack X %s, Y %s",
                  (ll)groups, (ll)M, (ll)P, (ll)Q, ab_dtype == TBG_F16 ? "f16" : "bf16",
                  c_dtype == TBG_F32 ? "f32" : "16-bit", choice.bm, choice.bn, rx.needed ? "yes" : "no", ry.needed ? "yes" : "no");
  e = tbg::launch_wgrad(p, choice, ab_dtype == TBG_F16, out_code(c_dtype), s);
  return launch_status("grouped wgrad", e);
}

}  // extern "C"

namespace {

tbg_status check_mx4(const char* what, int64_t rows, int64_t K, const void* codes, int64_t ld_codes,
                     const void* scales, int64_t ld_scales) {
  if (ld_codes < K / 2 || ld_scales < K / 32 || ld_codes < 0 || ld_scales < 0)
    return fail(TBG_ERR_INVALID_VALUE, "%s: pitches of %lld and %lld bytes for rows of %lld and %lld", what,
                (ll)ld_codes, (ll)ld_scales, (ll)(K / 2), (ll)(K / 32));
  if (ld_codes > kMaxPitch4 || ld_scales > kMaxPitch4)
    return fail(TBG_ERR_UNSUPPORTED, "%s: pitches are limited to 2^23-16 bytes", what);
  if (rows > 0 && K > 0 && (!codes || !scales)) return fail(TBG_ERR_INVALID_VALUE, "%s: codes or scales is NULL", what);
  if (off16(codes) || off16(scales) || ld_codes % 16 != 0 || ld_scales % 16 != 0)
    return fail(TBG_ERR_MISALIGNED, "%s: codes, scales and their pitches must be multiples of 16 bytes", what);
  return TBG_OK;
}

tbg_status check_conversion(int64_t rows, int64_t cols, const void* X, int64_t ldx, tbg_dtype x_dtype,
                            const void* codes, int64_t ld_codes, const void* scales, int64_t ld_scales) {
  if (rows < 0 || cols < 0) return fail(TBG_ERR_INVALID_VALUE, "negative size rows=%lld cols=%lld", (ll)rows, (ll)cols);
  if (x_dtype != TBG_F32 && x_dtype != TBG_BF16 && x_dtype != TBG_F16)
    return fail(TBG_ERR_INVALID_VALUE, "X must be TBG_F32, TBG_BF16 or TBG_F16 (got %d)", (int)x_dtype);
  if (cols > kMaxSize || rows > (1ll << 40)) return fail(TBG_ERR_UNSUPPORTED, "cols are limited to 2^30, rows to 2^40");
  const tbg_status st = check_ld("ldx", ldx, cols, kMaxLdc);
  if (st != TBG_OK) return st;
  if (rows > 0 && cols > 0 && !X) return fail(TBG_ERR_INVALID_VALUE, "X is NULL");
  if (((uintptr_t)X) % (x_dtype == TBG_F32 ? 4 : 2) != 0)
    return fail(TBG_ERR_MISALIGNED, "X must be aligned to its elements");
  const int64_t K = round_up(cols, 32);
  if (ld_codes < K / 2 || ld_scales < K / 32)
    return fail(TBG_ERR_INVALID_VALUE, "pitches of %lld and %lld bytes for rows of %lld and %lld", (ll)ld_codes,
                (ll)ld_scales, (ll)(K / 2), (ll)(K / 32));
  if (rows > 0 && cols > 0 && (!codes || !scales)) return fail(TBG_ERR_INVALID_VALUE, "codes or scales is NULL");
  if (off16(codes) || off16(scales) || ld_codes % 16 != 0 || ld_scales % 16 != 0)
    return fail(TBG_ERR_MISALIGNED, "codes, scales and their pitches must be multiples of 16 bytes");
  return TBG_OK;
}

tbg::Mx4Params conversion_params(int64_t cols, void* X, int64_t ldx, tbg_dtype x_dtype, void* codes, int64_t ld_codes,
                                 void* scales, int64_t ld_scales) {
  tbg::Mx4Params p;
  memset(&p, 0, sizeof(p));
  p.x = X;
  p.codes = (uint8_t*)codes;
  p.scales = (uint8_t*)scales;
  p.ldx = ldx * (x_dtype == TBG_F32 ? 4 : 2);
  p.ld_codes = ld_codes;
  p.ld_scales = ld_scales;
  p.cols = cols;
  p.per_row = (uint32_t)((cols + 31) / 32 * 4);
  return p;
}

// Both 4-bit products: groups < 0 is the dense one.
tbg_status mx4_gemm_impl(int64_t groups, int64_t M, int64_t N, int64_t K, const int32_t* offsets, float alpha,
                         const void* A, int64_t lda, const void* As, int64_t ld_as, const void* B, int64_t ldb,
                         int64_t stride_b, const void* Bs, int64_t ld_bs, int64_t stride_bs, float beta, void* C,
                         int64_t ldc, tbg_dtype c_dtype, void* stream) {
  const bool ragged = groups >= 0;
  tbg_status st = check_sizes(M, N, K);
  if (st != TBG_OK) return st;
  if (c_dtype != TBG_F32 && c_dtype != TBG_BF16) return fail(TBG_ERR_INVALID_VALUE, "C must be TBG_F32 or TBG_BF16");
  if (K % 32 != 0) return fail(TBG_ERR_INVALID_VALUE, "K=%lld is not a multiple of 32", (ll)K);
  st = check_ld("ldc", ldc, N, kMaxLdc);
  if (st != TBG_OK) return st;
  const bool scaled = !(alpha == 1.f && beta == 0.f);
  if (alpha == 0.f) {  // nothing of A or B is used
    K = 0;
    A = As = B = Bs = nullptr;
    lda = ld_as = ldb = ld_bs = stride_b = stride_bs = 0;
  }
  st = check_mx4("A", M, N > 0 ? K : 0, A, lda, As, ld_as);
  if (st == TBG_OK) st = check_mx4("B", N, M > 0 ? K : 0, B, ldb, Bs, ld_bs);
  if (st != TBG_OK) return st;
  if (ragged && groups > 1 && K > 0 && N > 0) {
    if (stride_b < (N - 1) * ldb + K / 2 || stride_bs < (N - 1) * ld_bs + K / 32)
      return fail(TBG_ERR_INVALID_VALUE, "stride_b=%lld or stride_bs=%lld below one matrix", (ll)stride_b, (ll)stride_bs);
    if (stride_b % 16 != 0 || stride_bs % 16 != 0)
      return fail(TBG_ERR_MISALIGNED, "stride_b and stride_bs must be multiples of 16 bytes");
  }
  if (groups == 0 || M == 0 || N == 0) return TBG_OK;
  if (!C) return fail(TBG_ERR_INVALID_VALUE, "C is NULL");
  int cus = 0;
  st = check_device(&cus);
  if (st != TBG_OK) return st;
  const tbg::TileChoice choice = tbg::choose_mx4(ragged ? groups : 0, M, N, K, cus);
  st = check_grid(choice);
  if (st != TBG_OK) return st;
  tbg::Mx4GemmParams p;
  memset(&p, 0, sizeof(p));
  p.g.A = (const uint8_t*)A;
  p.g.B = (const uint8_t*)B;
  p.g.C = C;
  p.g.offsets = ragged ? offsets : nullptr;
  p.g.lda = lda;
  p.g.ldb = ldb;
  p.g.stride_b = stride_b;
  p.g.ldc = ldc;
  p.g.groups = ragged ? (int)groups : 1;
  p.g.rows = (int)M;
  p.g.N = (int)N;
  p.g.K = (int)K;
  p.g.group_m = ragged ? 8 : 4;
  p.g.vec_store = tbg::rows_dword_aligned(C, ldc, out_size(c_dtype));
  p.g.alpha = alpha;
  p.g.beta = beta;
  p.g.scaled = scaled ? 1 : 0;
  p.As = (const uint8_t*)As;
  p.Bs = (const uint8_t*)Bs;
  p.ld_as = ld_as;
  p.ld_bs = ld_bs;
  p.stride_bs = stride_bs;
  tbg::log_choice("mx4 gemm groups=%lld M=%lld N=%lld K=%lld out=%s: %s %dx%d, %d stages",
                  (ll)(ragged ? groups : 1), (ll)M, (ll)N, (ll)K, c_dtype == TBG_F32 ? "f32" : "bf16",
                  choice.few ? "rows" : "ring", choice.bm, choice.bn, choice.stages);
  const hipError_t e = choice.few ? tbg::launch_few_rows(p, choice, 2, out_code(c_dtype), (hipStream_t)stream)
                                  : tbg::launch_mx4_gemm(p, choice, c_dtype == TBG_BF16, (hipStream_t)stream);
  return launch_status("mx4 gemm", e);
}

}  // namespace

extern "C" {

tbg_status tbg_mx4_quantize(int64_t rows, int64_t cols, const void* X, int64_t ldx, tbg_dtype x_dtype, void* codes,
                            int64_t ld_codes, void* scales, int64_t ld_scales, void* stream) {
  tbg_status st = check_conversion(rows, cols, X, ldx, x_dtype, codes, ld_codes, scales, ld_scales);
  if (st != TBG_OK || rows == 0 || cols == 0) return st;
  st = check_device();
  if (st != TBG_OK) return st;
  const tbg::Mx4Params p =
      conversion_params(cols, const_cast<void*>(X), ldx, x_dtype, codes, ld_codes, scales, ld_scales);
  const hipError_t e = tbg::launch_mx4_quantize(p, rows, out_code(x_dtype), (hipStream_t)stream);
  if (e != hipSuccess) return fail(TBG_ERR_HIP, "mx4 quantize launch: %s", hipGetErrorString(e));
  return TBG_OK;
}

tbg_status tbg_mx4_dequantize(int64_t rows, int64_t cols, const void* codes, int64_t ld_codes, const void* scales,
                              int64_t ld_scales, void* X, int64_t ldx, tbg_dtype x_dtype, void* stream) {
  tbg_status st = check_conversion(rows, cols, X, ldx, x_dtype, codes, ld_codes, scales, ld_scales);
  if (st != TBG_OK || rows == 0 || cols == 0) return st;
  st = check_device();
  if (st != TBG_OK) return st;
  const tbg::Mx4Params p = conversion_params(cols, X, ldx, x_dtype, const_cast<void*>(codes), ld_codes,
                                             const_cast<void*>(scales), ld_scales);
  const hipError_t e = tbg::launch_mx4_dequantize(p, rows, out_code(x_dtype), (hipStream_t)stream);
  if (e != hipSuccess) return fail(TBG_ERR_HIP, "mx4 dequantize launch: %s", hipGetErrorString(e));
  return TBG_OK;
}

tbg_status tbg_mx4_gemm(int64_t M, int64_t N, int64_t K, float alpha, const void* A, int64_t lda, const void* A_scales,
                        int64_t ld_as, const void* B, int64_t ldb, const void* B_scales, int64_t ld_bs, float beta,
                        void* C, int64_t ldc, tbg_dtype c_dtype, void* stream) {
  return mx4_gemm_impl(-1, M, N, K, nullptr, alpha, A, lda, A_scales, ld_as, B, ldb, 0, B_scales, ld_bs, 0, beta, C,
                       ldc, c_dtype, stream);
}

tbg_status tbg_mx4_gemm_grouped(int64_t groups, int64_t M, int64_t N, int64_t K, const int32_t* offsets, float alpha,
                                const void* A, int64_t lda, const void* A_scales, int64_t ld_as, const void* B,
                                int64_t ldb, int64_t stride_b, const void* B_scales, int64_t ld_bs, int64_t stride_bs,
                                float beta, void* C, int64_t ldc, tbg_dtype c_dtype, void* stream) {
  const tbg_status st = check_groups(groups, M, offsets);
  if (st != TBG_OK) return st;
  return mx4_gemm_impl(groups, M, N, K, offsets, alpha, A, lda, A_scales, ld_as, B, ldb, stride_b, B_scales, ld_bs,
                       stride_bs, beta, C, ldc, c_dtype, stream);
}

}  // extern "C"
