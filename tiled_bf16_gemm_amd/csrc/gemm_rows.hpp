// Products with few rows and few columns: one or a few tokens against a B stored N×K that gives the
// ring too few tiles to fill the chip, in 16 bits or microscaled 4 bits, dense or ragged.
//
// Such a product is bound by the time from the first load to the last: the ring's workgroups walk
// all of K one tile after another (64 columns each: 64 workgroups for N = 4096).  Here a workgroup
// owns 16 columns and up to 16 rows, its four waves split K, and every lane loads the pieces of its
// fragments straight into registers, one chunk (256 bytes per row, 16 KiB a workgroup) ahead of the
// products.  The waves' sums meet in LDS at the end and are added in wave order: one launch, no
// workspace, the same bits every time.  Measured against the ring (GPU time): one row in 4 bits,
// N = 4096, K = 16384 9.4 against 15.5 µs, N = K = 2048 3.5 against 5.5, N = 8192, K = 8192 9.9
// against 10.5; two rows in bf16, N = K = 4096 9.2 against 17.3.  From 3/4 of the CUs in 64-column
// tiles on the ring's whole-row copies win (N = 14336, K = 8192 in 4 bits: 15.2 against 12.4), and
// so does more than one fragment of rows or columns a workgroup here (both read A or B again).
//
// Lane l holds row (column) l%16 of a fragment; its piece j of a chunk is the 16 bytes 4j + l/16, so
// a load instruction takes 64 contiguous bytes of each of 16 rows.  In 4 bits a piece is one block
// of 32, its scale byte l/16 of dword j of the chunk's 16 scale bytes: one 16-byte load a chunk,
// shifted into byte 0 of the register the product reads.  Rows and columns past the end repeat the
// last one and are not stored; pieces past K are not loaded and count as zeros.
#pragma once
#include "gemm_common.hpp"
#include "gemm_mx4.hpp"
#include "ragged.hpp"

namespace tbg {

constexpr int kRowsBf16 = 0, kRowsF16 = 1, kRowsMx4 = 2;
constexpr int kChunkBytes = 256;  // of a row, per wave and step
constexpr int kRowsWaves = 4;

// One wave's operands for a chunk of one fragment.
template <int FMT>
struct RowsPiece {
  u32x4_t v[4];
  u32x4_t s;  // 4-bit: the chunk's 16 scale bytes
};

template <int FMT>
__device__ __forceinline__ void load_piece(RowsPiece<FMT>& p, const uint8_t* row, const uint8_t* scales, int chunk) {
#pragma unroll
  for (int j = 0; j < 4; ++j) p.v[j] = *(const u32x4_t*)(row + (int64_t)chunk * kChunkBytes + j * 64);
  if (FMT == kRowsMx4) p.s = *(const u32x4_t*)(scales + (int64_t)chunk * 16);
}

// The last chunk of a row when it is not whole: `left` bytes remain in it, a multiple of 16 in 4 bits; in
// 16 bits a repack has filled the last 16 bytes with zeros.
template <int FMT>
__device__ __forceinline__ void load_piece_end(RowsPiece<FMT>& p, const uint8_t* row, const uint8_t* scales, int chunk,
                                               int left, int g) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    p.v[j] = u32x4_t{0, 0, 0, 0};
    if ((4 * j + g) * 16 < left) p.v[j] = *(const u32x4_t*)(row + (int64_t)chunk * kChunkBytes + j * 64);
  }
  if (FMT == kRowsMx4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int blocks = left / 16 - 4 * j;  // blocks of dword j that exist: the others' bytes become zero
      uint32_t w = 0;
      if (blocks > 0) w = *(const uint32_t*)(scales + (int64_t)chunk * 16 + 4 * j);
      if (blocks > 0 && blocks < 4) w &= (1u << (8 * blocks)) - 1u;
      p.s[j] = w;
    }
  }
}

template <int FMT>
__device__ __forceinline__ void rows_products(f32x4_t& acc, const RowsPiece<FMT>& a, const RowsPiece<FMT>& b, int shift) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (FMT == kRowsMx4)
      mfma_mx4<false, 0>(acc, __builtin_bit_cast(i32x4_t, b.v[j]), __builtin_bit_cast(i32x4_t, a.v[j]), b.s[j] >> shift,
                         a.s[j] >> shift);
    else
      mfma16<false, FMT>(acc, __builtin_bit_cast(bf16x8_t, b.v[j]), __builtin_bit_cast(bf16x8_t, a.v[j]));
  }
}

template <int FMT, int OUT, int SCALED>
__global__ void __launch_bounds__(64 * kRowsWaves) gemm_rows_kernel(Mx4GemmParams p) {
  constexpr int W = kRowsWaves;
  __shared__ f32x4_t part[W][64];
  const GroupedParams& g = p.g;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RaggedTile t;
  if (g.offsets) {
    if (!ragged_tile<16>(g, 1, blockIdx.x, t)) return;
  } else {  // at most 16 rows
    t.group = 0;
    t.row0 = 0;
    t.rows = g.rows;
    t.tn = blockIdx.x;
  }
  const int n0 = t.tn * 16, quarter = lane >> 4, shift = 8 * quarter;
  const int row_bytes = FMT == kRowsMx4 ? g.K / 2 : g.K * 2;
  const int64_t row = t.row0 + min(lane & 15, t.rows - 1), col = min(n0 + (lane & 15), g.N - 1);
  const uint8_t* a_row = g.A + row * g.lda + quarter * 16;
  const uint8_t* b_row = g.B + (int64_t)t.group * g.stride_b + col * g.ldb + quarter * 16;
  const uint8_t* a_s = FMT == kRowsMx4 ? p.As + row * p.ld_as : nullptr;
  const uint8_t* b_s = FMT == kRowsMx4 ? p.Bs + (int64_t)t.group * p.stride_bs + col * p.ld_bs : nullptr;
  const int whole = row_bytes / kChunkBytes, left = row_bytes - whole * kChunkBytes;
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  RowsPiece<FMT> a0, b0, a1, b1;
  auto load = [&](RowsPiece<FMT>& a, RowsPiece<FMT>& b, int c) __attribute__((always_inline)) {
    load_piece<FMT>(b, b_row, b_s, c);
    load_piece<FMT>(a, a_row, a_s, c);
  };
  int c = wave;
  if (c < whole) load(a0, b0, c);
  for (; c < whole; c += 2 * W) {
    if (c + W < whole) load(a1, b1, c + W);
    rows_products<FMT>(acc, a0, b0, shift);
    if (c + W >= whole) break;
    if (c + 2 * W < whole) load(a0, b0, c + 2 * W);
    rows_products<FMT>(acc, a1, b1, shift);
  }
  if (left > 0 && wave == whole % W) {
    load_piece_end<FMT>(b0, b_row, b_s, whole, left, quarter);
    load_piece_end<FMT>(a0, a_row, a_s, whole, left, quarter);
    rows_products<FMT>(acc, a0, b0, shift);
  }
  part[wave][lane] = acc;
  __syncthreads();
  // Lane l of a wave holds C[l%16][4(l/16) .. +3]; thread t adds up element t%4 of lane t/4.
  float x = 0.f;
#pragma unroll
  for (int w = 0; w < W; ++w) x += ((const float*)part[w])[threadIdx.x];
  const int l = threadIdx.x >> 2, r = l & 15, n = n0 + 4 * (l >> 4) + (threadIdx.x & 3);
  if (r >= t.rows || n >= g.N) return;
  const int64_t at = (int64_t)(t.row0 + r) * g.ldc + n;
  if constexpr (OUT != 0) {
    typename Half4<OUT>::elem* dst = (typename Half4<OUT>::elem*)g.C + at;
    if (SCALED) x = g.beta != 0.f ? g.alpha * x + g.beta * (float)*dst : g.alpha * x;
    *dst = (typename Half4<OUT>::elem)x;
  } else {
    float* dst = (float*)g.C + at;
    if (SCALED) x = g.beta != 0.f ? g.alpha * x + g.beta * *dst : g.alpha * x;
    *dst = x;
  }
}

}  // namespace tbg
