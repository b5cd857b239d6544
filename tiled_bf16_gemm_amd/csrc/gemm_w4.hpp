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
//         result that is not finite is computed again from c - z itself (28 instructions a dword), and
//         it alone is stored from there, so that what a row holds never shows in another row's bits.
//         The price of the seven instructions: what the two sums are off by goes with |a|·(c + z), not
//         with |a|·|c - z|.  K = 4096, squared positive activations, 95 % of the codes at their zero of 7, scale
//         1: off by up to 4.8e-4 where the values' root mean square is 96 (fp16 0.9e-4, an fp32 product 0.7e-4), and
//         by 3.2e-4 where every code is 7; activations around zero 3.8e-5 (fp16 4.3e-5).
//
// Lane l holds column l%16 of a fragment and 16 bytes, the 32 codes of quarter l/16 of a block of 128.  The
// product wants the four quarters of 32 codes side by side in a step, so that a step never crosses a group:
// four half-wave and row swaps turn the quarters' dwords over (a 4×4 transpose), and step j has k =
// 32j + 8(l/16) .. +7.  A's fragment is the 16 bytes at that k, its values in the order in which decoding
// leaves the codes.
//
// Two kernels, both one launch without a workspace, with the same bits every time: for few tiles the waves of
// a workgroup split K and their sums meet in LDS, added in wave order; for many they split N and share A's
// blocks in LDS.  Rows and columns past the end repeat the last one and are not stored.  choose_w4
// (tile_choice.hpp) has both sides' figures.
//
// Measured: 1 × 14336 × 4096 9.3 µs (30 MB, 3.3 TB/s: 8 blocks in a row a wave after the launch); 64 rows over 40 of
// 64 experts of 4096 × 2048 39.5 µs (173 MB, 4.4 TB/s); 2008 rows over 64 of 2048 × 4096 118-127 µs, where vector
// instructions issue in 77 % of the busy cycles and products in 37 %.  Taking z off with products against -z in the same
// sum (152 vector instructions a block for 164, 32 products for 24) was 3 to 8 % slower there.
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

// A zero as decode wants it: bf16 a float; fp16 -1024 - z in the upper half (z is below the last place of 1024, so its
// bits are those of -1024 and z's).
template <int IN>
__device__ __forceinline__ uint32_t zero_word(uint32_t z) {
  return IN == 1 ? z << 16 | 0xE4000000u : __float_as_uint((float)z);
}

// What decode's masks are held in: an instruction takes one constant from a scalar register, so (w & m) | o is a single
// one only where o is in a vector register.  (Left to the compiler they are two with a literal each.)
template <int IN>
struct W4Masks {
  uint32_t low = 0x000F000Fu, high = 0x00F000F0u, bits = 0x64006400u;
  __device__ __forceinline__ W4Masks() {
    if constexpr (IN == 1) {
      asm("" : "+s"(low));
      asm("" : "+s"(high));
      asm("" : "+v"(bits));
    }
  }
};

// The eight codes of a dword as values: fp16 c - z; bf16 c, or with EXACT c - z.  z: zero_word.
template <int IN, bool EXACT>
__device__ __forceinline__ bf16x8_t decode(uint32_t w, uint32_t z, const W4Masks<IN>& m) {
  u32x4_t r;
  if constexpr (IN == 1) {
    const _Float16 one = __builtin_bit_cast(f16x2v_t, z)[1], sixteen = one + (_Float16)960.f;  // -64 - z, exactly
    const f16x2v_t off1 = {one, one}, off16 = {sixteen, sixteen}, part = {(_Float16)0.0625f, (_Float16)0.0625f};
    const uint32_t v = w >> 8;
    auto pair = [&](uint32_t x, uint32_t mask) { return __builtin_bit_cast(f16x2v_t, (x & mask) | m.bits); };
    r[0] = __builtin_bit_cast(uint32_t, pair(w, m.low) + off1);
    r[1] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(pair(w, m.high), part, off16));
    r[2] = __builtin_bit_cast(uint32_t, pair(v, m.low) + off1);
    r[3] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(pair(v, m.high), part, off16));
  } else if constexpr (EXACT) {
    auto value = [&](int i) {  // whole: its low half is 0
      return __float_as_uint((float)((w >> (4 * i)) & 15u) - __uint_as_float(z));
    };
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

// Exchanges the upper half of x's lanes with the lower of y's; the odd rows of 16 lanes of x with the even ones of y.
__device__ __forceinline__ void swap_halves(uint32_t& x, uint32_t& y) {
  const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
  x = r[0];
  y = r[1];
}
__device__ __forceinline__ void swap_rows(uint32_t& x, uint32_t& y) {
  const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
  x = r[0];
  y = r[1];
}

// Dword d of quarter q becomes dword q of quarter d.
__device__ __forceinline__ void turn_quarters(u32x4_t& b) {
  uint32_t r0 = b[0], r1 = b[1], r2 = b[2], r3 = b[3];
  swap_halves(r0, r2);
  swap_halves(r1, r3);
  swap_rows(r0, r1);
  swap_rows(r2, r3);
  b = u32x4_t{r0, r1, r2, r3};
}

// What a wave holds of the weights of a block of 128 codes, FN fragments of columns: the codes of a lane's column and
// quarter, and scale and zero of the group that the quarter lies in.
template <int FN>
struct W4Weights {
  u32x4_t b[FN];
  uint16_t s[FN];
  uint8_t z[FN];
};

// Where a lane reads its columns' codes, scales and zeros: offsets from the tile's bases, which are the same for
// every lane.
template <int FN>
struct W4Columns {
  const uint8_t* b;  // the first column's codes
  const uint8_t* s;  // its scales
  const uint8_t* z;  // its zeros
  int64_t block_s, block_z;  // bytes from one block's scales (zeros) to the next one's
  uint32_t group_s, group_z;  // and from one group's
  uint32_t at_b[FN], col[FN];
};

// Columns n0, n0 + 1, ... of W_group, the lane's at n0 + 16·n + lane%16.
template <int G, int FN>
__device__ __forceinline__ W4Columns<FN> w4_columns(const W4Params& p, int group, int n0, int lane) {
  W4Columns<FN> l;
  l.b = p.g.B + (int64_t)group * p.g.stride_b + (int64_t)n0 * p.g.ldb;
  l.s = (const uint8_t*)(p.scales + (int64_t)group * p.stride_s + n0);
  l.z = p.zeros ? p.zeros + (int64_t)group * p.stride_z + n0 : nullptr;
  l.block_s = kW4Block / G * 2 * p.ld_s;
  l.block_z = kW4Block / G * p.ld_z;
  l.group_s = (uint32_t)(2 * p.ld_s);
  l.group_z = (uint32_t)p.ld_z;
#pragma unroll
  for (int n = 0; n < FN; ++n) {
    l.col[n] = (uint32_t)max(min(16 * n + (lane & 15), p.g.N - 1 - n0), 0);
    l.at_b[n] = l.col[n] * (uint32_t)p.g.ldb;
  }
  return l;
}

// Block c, of which `steps` steps of 32 exist (ALL: four).  What is past them repeats what exists; the products
// leave it out.  Nothing is computed with what is loaded here, which would wait for it.
template <bool ALL, bool ZEROS, int G, int FN>
__device__ __forceinline__ void load_weights(W4Weights<FN>& k, const W4Columns<FN>& l, int c, int steps, int quarter) {
  const uint8_t *b = l.b + (int64_t)c * 64, *s = l.s + c * l.block_s, *z = l.z + c * l.block_z;
  const bool in = ALL || quarter < steps;
  const uint32_t q = in ? quarter * 16 : 0, g = in ? quarter / (G / 32) : 0;
#pragma unroll
  for (int n = 0; n < FN; ++n) k.b[n] = *(const u32x4_t*)(b + (l.at_b[n] + q));
#pragma unroll
  for (int n = 0; n < FN; ++n) {
    k.s[n] = *(const uint16_t*)(s + (g * l.group_s + 2 * l.col[n]));
    if (ZEROS) k.z[n] = z[g * l.group_z + l.col[n]];
  }
}

// The activations of a block in registers, one fragment of 16 rows; row: the lane's row at its quarter's bytes.
struct W4Rows {
  u32x4_t a[4];
};

template <bool ALL>
__device__ __forceinline__ void load_rows(W4Rows& k, const uint8_t* row, int c, int steps) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (!ALL) k.a[j] = u32x4_t{0, 0, 0, 0};
    if (ALL || j < steps) {
      const W4Raw16 r = *(const W4Raw16*)(row + (int64_t)c * 256 + j * 64);
      k.a[j] = u32x4_t{r.w[0], r.w[1], r.w[2], r.w[3]};
    }
  }
}

// The row of A that row r of the groups reads.
__device__ __forceinline__ int64_t w4_row(const W4Params& p, int r) {
  if (!p.source || p.g.K == 0) return r;
  return min((int)fast_div((uint32_t)max(p.source[r], 0), p.top_k), p.a_rows - 1);
}

template <int IN>
__device__ __forceinline__ float scale_value(uint16_t s) {
  if (IN == 1) return (float)__builtin_bit_cast(_Float16, s);
  return __uint_as_float((uint32_t)s << 16);
}

// A group's scale and zero (zero_word) for a lane's column.
struct W4Scale {
  float s;
  uint32_t z;
};

// The groups' scales and zeros for every quarter, from the quarters that hold them: a scale and a zero are one dword,
// whose rows of 16 lanes are copied to the others with the swaps of turn_quarters.  (A load for every group and column
// would be 16 of 22 loads a block for groups of 32 with zeros and two fragments: 33 × 2049 × 8160 16.2 µs, so 13.0; with the masks of W4Masks 12.5.)
template <int IN, bool ZEROS, int G, int FN>
struct W4Scales {
  static constexpr int Groups = kW4Block / G;
  uint32_t v[Groups][FN];

  __device__ __forceinline__ W4Scales(const W4Weights<FN>& k) {
#pragma unroll
    for (int n = 0; n < FN; ++n) {
      uint32_t r[4];
      r[0] = k.s[n] | (ZEROS ? (uint32_t)k.z[n] << 16 : 0u) | (IN == 1 && ZEROS ? 0xE4000000u : 0u);
      if (G == 32) {  // rows 0 0 2 2 and 1 1 3 3
        r[1] = r[0];
        swap_rows(r[0], r[1]);
        r[3] = r[1];
        swap_halves(r[1], r[3]);
      }
      if (G <= 64) {
        r[2] = r[0];
        swap_halves(r[0], r[2]);
      }
#pragma unroll
      for (int g = 0; g < Groups; ++g) v[g][n] = r[G == 64 ? 2 * g : g];
    }
  }
  __device__ __forceinline__ W4Scale operator()(int g, int n) const {
    const uint32_t x = v[g][n];
    return W4Scale{scale_value<IN>((uint16_t)x), !ZEROS ? zero_word<IN>(8) : IN == 1 ? x : zero_word<IN>(x >> 16)};
  }
};

// The lane's group of a block from step `steps` on does not exist: its scale counts as zero (and A's values as zeros).
template <int G, int FN>
__device__ __forceinline__ void end_weights(W4Weights<FN>& k, int steps, int quarter) {
#pragma unroll
  for (int n = 0; n < FN; ++n)
    if (quarter / (G / 32) * (G / 32) >= steps) k.s[n] = 0;
}

// acc += the products of a block whose codes are b.  fragment(m, j) gives A's fragment m of step j, in decode's
// order, scale(g, n) the scale and zero of group g of the block.
template <int IN, bool EXACT, int G, int FM, int FN, class Fragment, class Scale>
__device__ __forceinline__ void block_products(f32x4_t (&acc)[FM][FN], u32x4_t (&b)[FN], Fragment fragment, Scale scale) {
  constexpr bool Sums = IN == 0 && !EXACT;  // z is taken off after the group
  const u32x4_t ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
  for (int n = 0; n < FN; ++n) turn_quarters(b[n]);
  f32x4_t sum[FM][FN], of_a[FM];
  W4Scale sz[FN];
  const W4Masks<IN> masks;
  bf16x8_t a[2][FM];
#pragma unroll
  for (int m = 0; m < FM; ++m) a[0][m] = fragment(m, 0);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    constexpr int Steps = G / 32;
    if (j % Steps == 0) {
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        of_a[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int n = 0; n < FN; ++n) sum[m][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int n = 0; n < FN; ++n) sz[n] = scale(j / Steps, n);
    }
    if (j < 3) {
#pragma unroll
      for (int m = 0; m < FM; ++m) a[(j + 1) & 1][m] = fragment(m, j + 1);
    }
    if (Sums) {
#pragma unroll
      for (int m = 0; m < FM; ++m) mfma16<false, IN>(of_a[m], a[j & 1][m], __builtin_bit_cast(bf16x8_t, ones));
    }
#pragma unroll
    for (int n = 0; n < FN; ++n) {
      const bf16x8_t v = decode<IN, EXACT>(b[n][j], sz[n].z, masks);
#pragma unroll
      for (int m = 0; m < FM; ++m) mfma16<false, IN>(sum[m][n], a[j & 1][m], v);
    }
    if (j % Steps == Steps - 1) {
#pragma unroll
      for (int n = 0; n < FN; ++n)
#pragma unroll
        for (int m = 0; m < FM; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = Sums ? fmaf(-__uint_as_float(sz[n].z), of_a[m][i], sum[m][n][i]) : sum[m][n][i];
            acc[m][n][i] = fmaf(sz[n].s, x, acc[m][n][i]);
          }
      // The sums are used up here: moved into a later block of the code they would stay in registers until there.
#pragma unroll
      for (int n = 0; n < FN; ++n)
#pragma unroll
        for (int m = 0; m < FM; ++m) asm volatile("" : "+v"(acc[m][n]));
    }
    // Steps stay in this order: decoded further ahead of their products they would take the registers of another
    // wave, which hides one's decoding under the other's products.
    __builtin_amdgcn_sched_barrier(0);
  }
}

template <int FM, int FN>
__device__ __forceinline__ void clear_sums(f32x4_t (&acc)[FM][FN]) {
#pragma unroll
  for (int m = 0; m < FM; ++m)
#pragma unroll
    for (int n = 0; n < FN; ++n) acc[m][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
}

__device__ __forceinline__ bool is_finite(float x) { return fabsf(x) <= 3.4028235e38f; }

// The tile of this workgroup; false when there is none (the grid is an upper bound).
template <int BM>
__device__ __forceinline__ bool w4_tile(const GroupedParams& g, RaggedTile& t) {
  if (g.offsets) return ragged_tile<BM>(g, g.group_m, blockIdx.x, t);
  int first, count, tm;
  xcd_share(g.tiles_m * g.tiles_n, blockIdx.x, first, count);
  if ((int)(blockIdx.x >> 3) >= count) return false;
  band_tile(first + (blockIdx.x >> 3), g.tiles_m, g.tiles_n, g.group_m, tm, t.tn);
  t.group = 0;
  t.row0 = tm * BM;
  t.rows = g.rows - t.row0;
  return true;
}

// C[row][n] from the sum x.
template <int IN>
__device__ __forceinline__ void w4_store(const W4Params& p, int64_t row, int n, float x) {
  const GroupedParams& g = p.g;
  typedef typename Half4<IN == 1 ? 2 : 1>::elem half;
  const int64_t at = row * g.ldc + n;
  if (g.scaled) {
    x *= g.alpha;
    if (g.beta != 0.f) x = fmaf(g.beta, p.out16 ? (float)((const half*)g.C)[at] : ((const float*)g.C)[at], x);
  }
  if (p.out16) ((half*)g.C)[at] = (half)x;
  else ((float*)g.C)[at] = x;
}

// Stores the fragment of 16 rows and 16 columns at r0, n0 of a tile with a result that is not finite; x: the lane's
// sums.  Those that are not finite are computed again from c - z itself, by the wave over the whole of K; the others stay
// as they are, as sums of another order would depend on the tile's other rows.  Rarely taken, so it is kept small.
template <int IN, bool ZEROS, int G>
__device__ __forceinline__ void w4_exact_fragment(const W4Params& p, const RaggedTile& t, int r0, int n0, const f32x4_t& x) {
  const int lane = threadIdx.x & 63, quarter = lane >> 4;
  const GroupedParams& g = p.g;
  const uint8_t* const row = g.A + w4_row(p, t.row0 + min(r0 + (lane & 15), t.rows - 1)) * g.lda + quarter * 16;
  const W4Columns<1> l = w4_columns<G, 1>(p, t.group, n0, lane);
  f32x4_t acc[1][1];
  clear_sums(acc);
  const bool good = is_finite(x[0]) && is_finite(x[1]) && is_finite(x[2]) && is_finite(x[3]);
  const int whole = g.K / kW4Block, left = g.K % kW4Block / 32;
  const int blocks = __ballot(!good) != 0 ? whole + (left > 0) : 0;
#pragma unroll 1
  for (int c = 0; c < blocks; ++c) {
    const int steps = c < whole ? 4 : left;
    W4Weights<1> k;
    W4Rows a;
    load_weights<false, ZEROS, G>(k, l, c, steps, quarter);
    load_rows<false>(a, row, c, steps);
    end_weights<G>(k, steps, quarter);
    block_products<IN, true, G>(acc, k.b, [&](int, int j) __attribute__((always_inline)) {
      return order_a<IN>(a.a[j]);
    }, W4Scales<IN, ZEROS, G, 1>(k));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + 4 * quarter + i, n = n0 + (lane & 15);
    if (r < t.rows && n < g.N) w4_store<IN>(p, t.row0 + r, n, is_finite(x[i]) ? x[i] : acc[0][0][i]);
  }
}

// ---- the waves split K ---------------------------------------------------------------------------

constexpr int kW4Waves = 4;  // eight: 1 × 14336 × 4096 11.6 µs for 10.1, 33 × 2049 × 8160 14.7 for 14.3, before a scale's load by quarter

// For few tiles: a workgroup owns 16 rows and 16·FN columns, and its waves split K; everything goes straight from
// memory to registers, a block ahead of the products.
template <int IN, bool ZEROS, int G, int FN>
__global__ void __launch_bounds__(64 * kW4Waves, 2) gemm_w4_kernel(W4Params p) {
  constexpr int W = kW4Waves;
  __shared__ f32x4_t part[W][FN][64];
  const GroupedParams& g = p.g;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), quarter = lane >> 4;
  RaggedTile t;
  if (!w4_tile<16>(g, t)) return;
  const int n0 = t.tn * 16 * FN;
  const W4Columns<FN> l = w4_columns<G, FN>(p, t.group, n0, lane);
  const uint8_t* const row = g.A + w4_row(p, t.row0 + min(lane & 15, t.rows - 1)) * g.lda + quarter * 16;
  // The wave's share of K: consecutive blocks (a cache line of codes holds two).
  const int whole = g.K / kW4Block, left = g.K % kW4Block / 32;
  const int first = (int)((uint32_t)whole * wave / W), end = (int)((uint32_t)whole * (wave + 1) / W);
  f32x4_t acc[1][FN];
  clear_sums(acc);
  W4Weights<FN> k0, k1;
  W4Rows x0, x1;
  auto load = [&](W4Weights<FN>& k, W4Rows& x, int c) __attribute__((always_inline)) {
    load_weights<true, ZEROS, G>(k, l, c, 4, quarter);
    load_rows<true>(x, row, c, 4);
  };
  auto products = [&](W4Weights<FN>& k, const W4Rows& x) __attribute__((always_inline)) {
    block_products<IN, false, G>(acc, k.b, [&](int, int j) __attribute__((always_inline)) {
      return order_a<IN>(x.a[j]);
    }, W4Scales<IN, ZEROS, G, FN>(k));
  };
  if (first < end) {
    // Every load of the loop is issued on every path (past the end the last block again): the waits before the
    // products can then count the loads behind them instead of draining all of them.
    load(k0, x0, first);
    int c = first;
    for (; c + 2 <= end; c += 2) {
      load(k1, x1, c + 1);
      products(k0, x0);
      load(k0, x0, min(c + 2, end - 1));
      products(k1, x1);
    }
    if (c < end) products(k0, x0);
  }
  if (left > 0 && wave == W - 1) {
    load_weights<false, ZEROS, G>(k0, l, whole, left, quarter);
    load_rows<false>(x0, row, whole, left);
    end_weights<G>(k0, left, quarter);
    products(k0, x0);
  }
#pragma unroll
  for (int n = 0; n < FN; ++n) part[wave][n][lane] = acc[0][n];
  __syncthreads();
  // Thread threadIdx.x takes elements threadIdx.x + 256·i of the tile, a row's columns side by side.
  float x[FN];
  bool finite = true;
#pragma unroll
  for (int i = 0; i < FN; ++i) {
    const int e = threadIdx.x + 64 * W * i, r = e / (16 * FN), n = e % (16 * FN);
    const int at = ((n >> 4) * 64 + (r >> 2) * 16 + (n & 15)) * 4 + (r & 3);
    x[i] = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) x[i] += ((const float*)part[w])[at];
    finite = finite && is_finite(x[i]);
  }
  if constexpr (IN == 0) {
    if (__syncthreads_or(!finite)) {
#pragma unroll 1
      for (int n = wave; n < FN; n += W) {
        f32x4_t y = {0.f, 0.f, 0.f, 0.f};  // x of the lane's elements of fragment n
        int at = lane;  // (a value of its own: part's address, kept in a register from the stores above, made
        asm volatile("" : "+v"(at));  // those wait for the loads past the end: 16 × 4096 × 4096 8.1 µs for 7.8)
#pragma unroll
        for (int w = 0; w < W; ++w) y += part[w][n][at];
        if (n0 + 16 * n < g.N) w4_exact_fragment<IN, ZEROS, G>(p, t, 0, n0 + 16 * n, y);
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < FN; ++i) {
    const int e = threadIdx.x + 64 * W * i, r = e / (16 * FN), n = n0 + e % (16 * FN);
    if (r < t.rows && n < g.N) w4_store<IN>(p, t.row0 + r, n, x[i]);
  }
}

// ---- the waves split N ---------------------------------------------------------------------------

// A block of A in LDS: rows of 128 values at a pitch of 272 bytes, which puts the 16 rows of a fragment read on
// 16 different groups of four banks.  Its values lie in decode's order.
constexpr int kW4Pitch = 272;

// For more rows: a workgroup owns 16·FM rows and 64·FN columns, a wave 16·FN of them over the whole of K.  A's
// blocks go through LDS (a block is read once for the workgroup, and put into decode's order once), and so do
// the scales and zeros, as fp32 pairs; two buffers in turn with one barrier a block.  The codes go straight to
// the registers of the wave that owns their columns, a block ahead.  PER: workgroups a CU, by the registers they leave
// each other; a ring of two blocks (D) and more waves hide more than a ring of four and three waves a SIMD: 256 × 14336 × 4096
// in 16 rows 81 -> 77 µs, 32 64 -> 59, 64 55 -> 54; with groups of 32 and zeros 98 -> 92, 84 -> 76, 72 -> 72.
template <int IN, bool ZEROS, int G, int FM, int FN, int PER>
__global__ void __launch_bounds__(256, PER) gemm_w4_panel_kernel(W4Params p) {
  constexpr int D = 2, Ahead = FM == 1 ? 2 : 1, Columns = 64 * FN, Groups = kW4Block / G, Pairs = Groups * Columns;
  constexpr int Each = (Pairs + 255) / 256;
  __shared__ __attribute__((aligned(16))) uint8_t panel[2][16 * FM * kW4Pitch];
  __shared__ W4Scale pair[2][Pairs];
  const GroupedParams& g = p.g;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), quarter = lane >> 4;
  RaggedTile t;
  if (!w4_tile<16 * FM>(g, t)) return;
  const int first = t.tn * Columns, n0 = first + wave * 16 * FN;
  const int blocks = (g.K + kW4Block - 1) / kW4Block, last = blocks - 1, left = g.K % kW4Block / 32;
  // Steps of 32 of block c.  What does not exist of the last block repeats what exists when it is loaded and is
  // cleared on its way into LDS (so that nothing waits for a load where it is issued).
  auto steps_of = [&](int c) __attribute__((always_inline)) { return c < last || left == 0 ? 4 : left; };

  // thread i copies 16 bytes of rows i/16, i/16 + 16, ... of A
  const int chunk = threadIdx.x & 15;
  const uint8_t* a[FM];
#pragma unroll
  for (int m = 0; m < FM; ++m)
    a[m] = g.A + w4_row(p, t.row0 + min(16 * m + (int)(threadIdx.x >> 4), t.rows - 1)) * g.lda;
  const int to = (threadIdx.x >> 4) * kW4Pitch + chunk * 16, from = (lane & 15) * kW4Pitch + quarter * 16;
  W4Raw16 next[Ahead][FM];
  auto load_a = [&](int c, int slot) __attribute__((always_inline)) {
    c = min(c, last);
    const uint32_t at = chunk < 4 * steps_of(c) ? chunk * 16 : 0;
#pragma unroll
    for (int m = 0; m < FM; ++m) next[slot][m] = *(const W4Raw16*)(a[m] + ((int64_t)c * 256 + at));
  };
  auto store_a = [&](int c, int slot) __attribute__((always_inline)) {
    if (left > 0 && c >= last && chunk >= 4 * left) {
#pragma unroll
      for (int m = 0; m < FM; ++m) next[slot][m] = W4Raw16{{0, 0, 0, 0}};
    }
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      const W4Raw16& r = next[slot][m];
      *(bf16x8_t*)(panel[c & 1] + 16 * m * kW4Pitch + to) = order_a<IN>(u32x4_t{r.w[0], r.w[1], r.w[2], r.w[3]});
    }
  };

  // and pairs i, i + 256, ... of the groups' scales and zeros
  const uint8_t* const s_base = (const uint8_t*)(p.scales + (int64_t)t.group * p.stride_s + first);
  const uint8_t* const z_base = ZEROS ? p.zeros + (int64_t)t.group * p.stride_z + first : nullptr;
  uint16_t s_next[2][Each];
  uint8_t z_next[2][Each];
  // lane offsets of a pair, and of the block's first group, which stands in for one that does not exist
  uint32_t at_s[Each], at_z[Each], col[Each];
#pragma unroll
  for (int e = 0; e < Each; ++e) {
    const uint32_t i = threadIdx.x + 256 * e, of = i / Columns % Groups;
    col[e] = min(i % Columns, (uint32_t)(g.N - 1 - first));
    at_s[e] = of * (uint32_t)(2 * p.ld_s) + 2 * col[e];
    at_z[e] = of * (uint32_t)p.ld_z + col[e];
  }
  auto load_s = [&](int c, int slot) __attribute__((always_inline)) {
    c = min(c, last);
    const int steps = steps_of(c);
    const uint8_t *s = s_base + (int64_t)c * (Groups * 2 * p.ld_s), *z = z_base + (int64_t)c * (Groups * p.ld_z);
#pragma unroll
    for (int e = 0; e < Each; ++e) {
      const bool in = (int)((threadIdx.x + 256 * e) / Columns) * (G / 32) < steps;
      s_next[slot][e] = *(const uint16_t*)(s + (in ? at_s[e] : 2 * col[e]));
      if (ZEROS) z_next[slot][e] = z[in ? at_z[e] : col[e]];
    }
  };
  auto store_s = [&](int c, int slot) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < Each; ++e) {
      const int i = threadIdx.x + 256 * e;
      float s = scale_value<IN>(s_next[slot][e]);
      if (left > 0 && c >= last && i / Columns * (G / 32) >= left) s = 0.f;
      if (Pairs % 256 == 0 || i < Pairs) pair[c & 1][i] = W4Scale{s, zero_word<IN>(ZEROS ? z_next[slot][e] : 8)};
    }
  };

  const W4Columns<FN> l = w4_columns<G, FN>(p, t.group, min(n0, g.N - 1), lane);
  u32x4_t b[D][FN];
  auto load_b = [&](int d, int c) __attribute__((always_inline)) {
    c = min(c, last);
    const uint8_t* base = l.b + (int64_t)c * 64;
    const uint32_t q = quarter < steps_of(c) ? quarter * 16 : 0;
#pragma unroll
    for (int n = 0; n < FN; ++n) b[d][n] = *(const u32x4_t*)(base + (l.at_b[n] + q));
  };

  f32x4_t acc[FM][FN];
  clear_sums(acc);
  auto step = [&](int c, int d) __attribute__((always_inline)) {
    load_a(c + Ahead, d % Ahead);
    load_s(c + 2, d & 1);
    load_b((d + D - 1) % D, c + D - 1);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // block c is in LDS
    const uint8_t* at = panel[c & 1] + from;
    const W4Scale* sz = pair[c & 1] + wave * 16 * FN + (lane & 15);
    block_products<IN, false, G>(acc, b[d], [&](int m, int j) __attribute__((always_inline)) {
      return *(const bf16x8_t*)(at + 16 * m * kW4Pitch + j * 64);
    }, [&](int g, int n) __attribute__((always_inline)) { return sz[g * Columns + 16 * n]; });
    // the last readers of the other buffers passed the barrier above
    store_a(c + 1, (d + 1) % Ahead);
    store_s(c + 1, (d + 1) & 1);
  };
  if (blocks > 0) {
    load_a(0, 0);
    load_s(0, 0);
    if (Ahead == 2) load_a(1, 1);
    load_s(1, 1);
#pragma unroll
    for (int d = 0; d < D - 1; ++d) load_b(d, d);
    store_a(0, 0);
    store_s(0, 0);
    int c = 0;
    for (; c + D <= blocks; c += D)
#pragma unroll
      for (int d = 0; d < D; ++d) step(c + d, d);
#pragma unroll
    for (int d = 0; d < D - 1; ++d)
      if (c + d < blocks) step(c + d, d);
  }
  if constexpr (IN == 0) {
    bool finite = true;
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int n = 0; n < FN; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) finite = finite && is_finite(acc[m][n][i]);
    if (__ballot(!finite) != 0) {  // the wave's own columns
#pragma unroll 1
      for (int f = 0; f < FM * FN; ++f) {
        f32x4_t x = acc[0][0];
#pragma unroll
        for (int j = 1; j < FM * FN; ++j)
          if (f == j) x = acc[j / FN][j % FN];
        if (n0 + f % FN * 16 < g.N) w4_exact_fragment<IN, ZEROS, G>(p, t, f / FN * 16, n0 + f % FN * 16, x);
      }
      return;
    }
  }
#pragma unroll
  for (int m = 0; m < FM; ++m)
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 16 * m + 4 * quarter + i, col = n0 + 16 * n + (lane & 15);
        if (r < t.rows && col < g.N) w4_store<IN>(p, t.row0 + r, col, acc[m][n][i]);
      }
}

}  // namespace tbg
