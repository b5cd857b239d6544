// Products with weights in whole 4-bit codes and a scale for every group of the sum's index:
//   C[m][n] = sum over groups g of s[g][n] · (sum over k in g of A[m][k] · (c[n][k] - z[g][n]))
// The inner sums run on the 16-bit matrix instruction: c - z is a whole number of at most eight bits,
// which bf16 and fp16 hold exactly, so nothing is rounded before the fp32 sums, and the scale
// multiplies a group's finished sum.  (Weights multiplied out to 16 bits would be rounded first.)
//
// What bounds it is W: few rows read every code once, and a code has half a byte.  At the rate of memory a
// lane has about 28 vector instructions for the eight codes of a dword, so decoding is what the kernel is
// built around:
//   fp16  (code | 0x6400) is 1024 + c, packed two to a register; a packed add (or, for the nibble four bits
//         up, a packed multiply-add by 1/16) makes it c - z.  9 instructions a dword.
//   bf16  has no packed add.  A byte 0..15 read as E4M3 is c·2^-9, exactly (subnormals are linear, and so is
//         the first binade), and the packed conversion from E4M3 with scale 2^9 makes it c: 7 instructions
//         a dword.  z is taken off after the group: sum a·(c - z) = sum a·c - z·(sum a), the sum of a being one
//         more product, against ones, for all the columns of the wave.  Where a is infinite or near the
//         end of its range that difference may not exist although the definition's sum does: a
//         workgroup that meets a result which is not finite computes its tile again from c - z itself
//         (28 instructions a dword).
//
// Lane l holds column l%16 of a fragment and 16 bytes, the 32 codes of quarter l/16 of a block of 128.  The
// product wants the four quarters of 32 codes side by side in a step, so that a step never crosses a group:
// four half-wave and row swaps turn the quarters' dwords over (a 4×4 transpose), and step j has k =
// 32j + 8(l/16) .. +7.  A's fragment is the 16 bytes at that k, its values in the order in which decoding
// leaves the codes.
//
// A workgroup owns 16·FM rows and 16·FN columns; its waves split K by blocks of 128 and their sums meet in
// LDS, added in wave order: one launch, no workspace, the same bits every time.  Rows and columns past the
// end repeat the last one and are not stored.
#pragma once
#include "gemm_common.hpp"
#include "ragged.hpp"

namespace tbg {

constexpr int kW4Block = 128;  // codes of a row that a wave takes at a time: 64 bytes

// 16 bytes at any 2-byte boundary (gfx9 takes unaligned multi-dword accesses).
struct __attribute__((packed, aligned(2))) W4Raw16 { uint32_t w[4]; };

__device__ __forceinline__ uint32_t low_halves(uint32_t x, uint32_t y) { return __builtin_amdgcn_perm(y, x, 0x05040100u); }
__device__ __forceinline__ uint32_t high_halves(uint32_t x, uint32_t y) { return __builtin_amdgcn_perm(y, x, 0x07060302u); }

// A's eight values in the order of decode: fp16 04 15 26 37, bf16 02 46 13 57.
template <int IN>
__device__ __forceinline__ bf16x8_t order_a(const u32x4_t& a) {
  u32x4_t r;
  if (IN == 1) r = u32x4_t{low_halves(a[0], a[2]), high_halves(a[0], a[2]), low_halves(a[1], a[3]), high_halves(a[1], a[3])};
  else r = u32x4_t{low_halves(a[0], a[1]), low_halves(a[2], a[3]), high_halves(a[0], a[1]), high_halves(a[2], a[3])};
  return __builtin_bit_cast(bf16x8_t, r);
}

typedef _Float16 f16x2v_t __attribute__((ext_vector_type(2)));

// The eight codes of a dword as values: fp16 c - z; bf16 c, or with EXACT c - z.
template <int IN, bool EXACT>
__device__ __forceinline__ bf16x8_t decode(uint32_t w, float z) {
  u32x4_t r;
  if constexpr (IN == 1) {
    const _Float16 one = (_Float16)(-1024.f - z), sixteen = (_Float16)(-64.f - z);
    const f16x2v_t off1 = {one, one}, off16 = {sixteen, sixteen}, part = {(_Float16)0.0625f, (_Float16)0.0625f};
    const uint32_t v = w >> 8;
    auto pair = [](uint32_t x, uint32_t mask) { return __builtin_bit_cast(f16x2v_t, (x & mask) | 0x64006400u); };
    r[0] = __builtin_bit_cast(uint32_t, pair(w, 0x000F000Fu) + off1);
    r[1] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(pair(w, 0x00F000F0u), part, off16));
    r[2] = __builtin_bit_cast(uint32_t, pair(v, 0x000F000Fu) + off1);
    r[3] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(pair(v, 0x00F000F0u), part, off16));
  } else if constexpr (EXACT) {
    auto value = [&](int i) { return __float_as_uint((float)((w >> (4 * i)) & 15u) - z); };  // whole: its low half is 0
    r[0] = high_halves(value(0), value(2));
    r[1] = high_halves(value(4), value(6));
    r[2] = high_halves(value(1), value(3));
    r[3] = high_halves(value(5), value(7));
  } else {
    const uint32_t even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.f, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.f, true));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.f, false));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.f, true));
  }
  return __builtin_bit_cast(bf16x8_t, r);
}

// Dword d of quarter q becomes dword q of quarter d.
__device__ __forceinline__ void turn_quarters(u32x4_t& b) {
  auto swap32 = [](uint32_t& x, uint32_t& y) {
    const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
    x = r[0];
    y = r[1];
  };
  auto swap16 = [](uint32_t& x, uint32_t& y) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
    x = r[0];
    y = r[1];
  };
  uint32_t r0 = b[0], r1 = b[1], r2 = b[2], r3 = b[3];
  swap32(r0, r2);
  swap32(r1, r3);
  swap16(r0, r1);
  swap16(r2, r3);
  b = u32x4_t{r0, r1, r2, r3};
}

// What a wave holds of a block of 128 codes: FM fragments of rows, FN of columns.
template <int G, int FM, int FN>
struct W4Block {
  static constexpr int Groups = kW4Block / G;
  u32x4_t a[FM][4];
  u32x4_t b[FN];
  uint16_t s[Groups][FN];
  uint8_t z[Groups][FN];
};

// Where a lane reads: its rows of A (at its quarter's 16 bytes), its columns' codes, scales and zeros.
template <int FM, int FN>
struct W4Lane {
  const uint8_t* a[FM];
  const uint8_t* b[FN];
  const uint16_t* s;
  const uint8_t* z;  // null: every zero is 8
  int64_t ld_s, ld_z;
  int col[FN];
};

// Block c; ALL: it is whole, else it has `steps` steps of 32 (what is past them is left unread).
template <bool ALL, int G, int FM, int FN>
__device__ __forceinline__ void load_block(W4Block<G, FM, FN>& k, const W4Lane<FM, FN>& l, int c, int steps, int quarter) {
#pragma unroll
  for (int n = 0; n < FN; ++n) {
    k.b[n] = u32x4_t{0, 0, 0, 0};
    if (ALL || quarter < steps) k.b[n] = *(const u32x4_t*)(l.b[n] + (int64_t)c * 64);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      if (ALL || j < steps) {
        const W4Raw16 r = *(const W4Raw16*)(l.a[m] + (int64_t)c * 256 + j * 64);
        k.a[m][j] = u32x4_t{r.w[0], r.w[1], r.w[2], r.w[3]};
      }
    }
#pragma unroll
  for (int g = 0; g < W4Block<G, FM, FN>::Groups; ++g) {
    if (!ALL && g * (G / 32) >= steps) break;
    const int64_t row = (int64_t)c * W4Block<G, FM, FN>::Groups + g;
#pragma unroll
    for (int n = 0; n < FN; ++n) {
      k.s[g][n] = l.s[row * l.ld_s + l.col[n]];
      k.z[g][n] = l.z ? l.z[row * l.ld_z + l.col[n]] : (uint8_t)8;
    }
  }
}

template <int IN>
__device__ __forceinline__ float scale_value(uint16_t s) {
  if (IN == 1) return (float)__builtin_bit_cast(_Float16, s);
  return __uint_as_float((uint32_t)s << 16);
}

template <bool ALL, int IN, bool EXACT, int G, int FM, int FN>
__device__ __forceinline__ void block_products(f32x4_t (&acc)[FM][FN], W4Block<G, FM, FN>& k, int steps) {
  constexpr bool Sums = IN == 0 && !EXACT;  // z is taken off after the group
  const u32x4_t ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
  for (int n = 0; n < FN; ++n) turn_quarters(k.b[n]);
#pragma unroll
  for (int g = 0; g < W4Block<G, FM, FN>::Groups; ++g) {
    if (!ALL && g * (G / 32) >= steps) break;
    f32x4_t sum[FM][FN], of_a[FM];
    float z[FN];
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      of_a[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int n = 0; n < FN; ++n) sum[m][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int n = 0; n < FN; ++n) z[n] = (float)k.z[g][n];
#pragma unroll
    for (int i = 0; i < G / 32; ++i) {
      const int j = g * (G / 32) + i;
      bf16x8_t a[FM];
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        a[m] = order_a<IN>(k.a[m][j]);
        if (Sums) mfma16<false, IN>(of_a[m], a[m], __builtin_bit_cast(bf16x8_t, ones));
      }
#pragma unroll
      for (int n = 0; n < FN; ++n) {
        const bf16x8_t b = decode<IN, EXACT>(k.b[n][j], z[n]);
#pragma unroll
        for (int m = 0; m < FM; ++m) mfma16<false, IN>(sum[m][n], a[m], b);
      }
    }
#pragma unroll
    for (int n = 0; n < FN; ++n) {
      const float s = scale_value<IN>(k.s[g][n]);
#pragma unroll
      for (int m = 0; m < FM; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = Sums ? fmaf(-z[n], of_a[m][i], sum[m][n][i]) : sum[m][n][i];
          acc[m][n][i] = fmaf(s, x, acc[m][n][i]);
        }
    }
  }
}

// The wave's share of the K loop: blocks wave, wave + W, ..., one ahead of the products.
template <int IN, bool EXACT, int G, int FM, int FN, int W>
__device__ __forceinline__ void w4_sums(f32x4_t (&acc)[FM][FN], const W4Lane<FM, FN>& l, int K, int wave, int quarter) {
  const int whole = K / kW4Block, left = K % kW4Block / 32;
#pragma unroll
  for (int m = 0; m < FM; ++m)
#pragma unroll
    for (int n = 0; n < FN; ++n) acc[m][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  W4Block<G, FM, FN> k0, k1;
  int c = wave;
  if (c < whole) load_block<true>(k0, l, c, 4, quarter);
  for (; c < whole; c += 2 * W) {
    if (c + W < whole) load_block<true>(k1, l, c + W, 4, quarter);
    block_products<true, IN, EXACT>(acc, k0, 4);
    if (c + W >= whole) break;
    if (c + 2 * W < whole) load_block<true>(k0, l, c + 2 * W, 4, quarter);
    block_products<true, IN, EXACT>(acc, k1, 4);
  }
  if (left > 0 && wave == whole % W) {
    load_block<false>(k0, l, whole, left, quarter);
    block_products<false, IN, EXACT>(acc, k0, left);
  }
}

template <int IN, int G, int FM, int FN, int W>
__global__ void __launch_bounds__(64 * W) gemm_w4_kernel(W4Params p) {
  __shared__ f32x4_t part[W][FM * FN][64];
  const GroupedParams& g = p.g;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), quarter = lane >> 4;
  RaggedTile t;
  if (g.offsets) {
    if (!ragged_tile<16 * FM>(g, g.group_m, blockIdx.x, t)) return;
  } else {
    int first, count, tm;
    xcd_share(g.tiles_m * g.tiles_n, blockIdx.x, first, count);
    if ((int)(blockIdx.x >> 3) >= count) return;
    band_tile(first + (blockIdx.x >> 3), g.tiles_m, g.tiles_n, g.group_m, tm, t.tn);
    t.group = 0;
    t.row0 = tm * 16 * FM;
    t.rows = g.rows - t.row0;
  }
  const int n0 = t.tn * 16 * FN;
  W4Lane<FM, FN> l;
  l.s = p.scales + (int64_t)t.group * p.stride_s;
  l.z = p.zeros ? p.zeros + (int64_t)t.group * p.stride_z : nullptr;
  l.ld_s = p.ld_s;
  l.ld_z = p.ld_z;
#pragma unroll
  for (int m = 0; m < FM; ++m) {
    int64_t row = t.row0 + min(16 * m + (lane & 15), t.rows - 1);
    if (p.source && g.K > 0) {
      const int slot = max(p.source[row], 0);
      row = min((int)fast_div((uint32_t)slot, p.top_k), p.a_rows - 1);
    }
    l.a[m] = g.A + row * g.lda + quarter * 16;
  }
#pragma unroll
  for (int n = 0; n < FN; ++n) {
    l.col[n] = min(n0 + 16 * n + (lane & 15), g.N - 1);
    l.b[n] = g.B + (int64_t)t.group * g.stride_b + (int64_t)l.col[n] * g.ldb + quarter * 16;
  }
  // Thread threadIdx.x + 64·W·i of the tile's elements, a row's columns side by side.
  constexpr int Each = 4 * FM * FN / W;
  float x[Each];
  auto compute = [&](auto exact) __attribute__((always_inline)) {
    f32x4_t acc[FM][FN];
    w4_sums<IN, decltype(exact)::value, G, FM, FN, W>(acc, l, g.K, wave, quarter);
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int n = 0; n < FN; ++n) part[wave][m * FN + n][lane] = acc[m][n];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < Each; ++i) {
      const int e = threadIdx.x + 64 * W * i, r = e / (16 * FN), n = e % (16 * FN);
      const int at = (((r >> 4) * FN + (n >> 4)) * 64 + ((r & 15) >> 2) * 16 + (n & 15)) * 4 + (r & 3);
      x[i] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) x[i] += ((const float*)part[w])[at];
    }
  };
  compute(std::false_type{});
  if constexpr (IN == 0) {
    bool finite = true;
#pragma unroll
    for (int i = 0; i < Each; ++i) finite = finite && fabsf(x[i]) <= 3.4028235e38f;
    if (__syncthreads_or(!finite)) compute(std::true_type{});
  }
#pragma unroll
  for (int i = 0; i < Each; ++i) {
    const int e = threadIdx.x + 64 * W * i, r = e / (16 * FN), n = n0 + e % (16 * FN);
    if (r >= t.rows || n >= g.N) continue;
    const int64_t at = (int64_t)(t.row0 + r) * g.ldc + n;
    typedef typename Half4<IN == 1 ? 2 : 1>::elem half;
    float v = x[i];
    if (g.scaled) {
      v *= g.alpha;
      if (g.beta != 0.f) v = fmaf(g.beta, p.out16 ? (float)((const half*)g.C)[at] : ((const float*)g.C)[at], v);
    }
    if (p.out16) ((half*)g.C)[at] = (half)v;
    else ((float*)g.C)[at] = v;
  }
}

}  // namespace tbg
