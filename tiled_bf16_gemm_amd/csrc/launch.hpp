// Host-side launchers of the kernels, called by the C ABI in api.hip.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fast_div.hpp"
#include "tbg_desc.hpp"
#include "tile_choice.hpp"

namespace tbg {

// Arguments of one GEMM launch (see gemm_kernel.hip).  The barrier ring, the producer ring and
// the fp8 ring read their operands through `da` and `db`, the descriptors of the operand boxes
// that the host encodes with tbg_encode_tiled ("2 · Le Tensor Memory Accelerator" §2.3: built
// once on the host, handed to the kernel): base address, row pitch in bytes and extents (A {K, M};
// B {K, N} stored N×K, {N, K} stored K×N).  A, B, lda and ldb stay for the convolution kernel.
struct GemmParams {
  const uint16_t* A;
  const uint16_t* B;
  void* C;
  int64_t lda, ldb, ldc;  // elements
  int M, N, K;
  int kchunks;     // 16-byte chunks along K present in memory (ceil(K/8)); data past K there is zero
  int tiles_m, tiles_n, group_m;
  int vec_store;   // C's base and row pitch are multiples of 4 bytes: whole 16-byte pieces may be stored
  float alpha, beta;
  int scaled;      // 0: C = A·B; 1: C = alpha·A·B + beta·C (C read only when beta != 0)
  // Clock-recording instances only (a measurement build outside the C ABI): per workgroup the
  // 100 MHz real-time and shader-clock counter deltas from its start to its end.  Null otherwise.
  uint64_t* clock;
  DescImpl da, db;  // operand box descriptors (zero when K = 0: every copy is masked)
};

// Arguments of one implicit-GEMM convolution launch (gemm_conv.hpp).  `g` carries what the
// GEMM epilogue needs: M = N*OH*OW output pixels, N = K output channels, C = Y, ldc = ldy,
// vec_store, alpha/beta/scaled, and the tile grid.  X and W have a channel pitch of c8 (a
// multiple of 8; channels c8 > c >= C hold zeros after packing).
struct ConvParams {
  GemmParams g;
  const uint16_t* X;   // NHWC, channel pitch c8
  const uint16_t* W;   // K × (R·S·c8): filter k, tap (r, s), channel c at k*ldw + (r*S + s)*c8 + c
  int64_t ldw;         // R * S * c8
  uint32_t x_bytes;    // bytes of X (below 2^31)
  int n, h, w, c8, r, s, oh, ow;
  int ph, pw, sh, sw, dh, dw;
  int cblocks;         // ceil(c8 / 64): 64-channel blocks per tap
};

// Arguments of the halo convolution (gemm_conv_halo.hpp): stride 1, channels a multiple of 32.
// A workgroup computes `tr` whole output rows of one image (tr·ow <= 448 pixels) for 128 output
// channels; the input window those rows need (hh × hw pixels, zero outside the image) is copied
// into LDS once per 32-channel block and every filter tap reads it there.
struct HaloParams {
  ConvParams c;        // c.g.tiles_m = images × tiles per image, c.g.tiles_n = ceil(k / 128)
  int tr, tpi;         // output rows per tile, tiles per image
  int hh, hw, ns;      // window rows, columns, pixels (hh·hw)
  int hat, hb;         // 1 KiB copy atoms per window image, its LDS bytes (hat·1024)
  int cb32, rs;        // 32-channel blocks, filter taps
  FastDiv div_hw, div_ow;
  int tap_off[9];      // LDS byte offset of tap v = r·S + s from tap 0 in a window image (v < rs, rs <= 9)
};

hipError_t launch_im2col_copy(const DescIm2col& d, const int32_t* host_coords, const int32_t* coords_dev, uint32_t n,
                              void* dst, hipStream_t stream);
// Convolution with workgroup tile bm × bn (256×256, 256×128, 128×128 or 64×64); fills the grid.
hipError_t launch_conv(ConvParams cp, int bm, int bn, int out_bf16, hipStream_t stream);
bool conv_tile_built(int bm, int bn);
// Fills the halo fields of `hp` from hp.c (shape fields set); false with `why` set when the shape
// does not fit the halo kernel.  hs_out: window atoms each wave copies per filter tap (1..4).
bool plan_conv_halo(HaloParams& hp, int* hs_out, const char** why);
hipError_t launch_conv_halo(const HaloParams& hp, int hs, int out_bf16, hipStream_t stream);

hipError_t launch_tiled_store(const DescImpl& d, const int32_t* host_coords, const int32_t* coords_dev, uint32_t n,
                              const void* src, hipStream_t stream);
hipError_t launch_tiled_copy(const DescImpl& d, const int32_t* host_coords, const int32_t* coords_dev, uint32_t n,
                             void* dst, hipStream_t stream);
// Operand-copy pipelines of the GEMM (values of tbg_pipeline).
enum GemmPipeline { kPipeRing = 1, kPipeProducer = 2 };

// One built kernel configuration; tiles_m / tiles_n of `p` must be set.
typedef hipError_t (*GemmLauncher)(const GemmParams& p, int b_layout, int out_bf16, hipStream_t stream);
// IN: input element type of the products, 0 bf16, 1 fp16.
template <int BM, int BN, int S, int IN>
hipError_t launch_ring(const GemmParams& p, int b_layout, int out_bf16, hipStream_t stream);
template <int BM, int BN, int S, int IN>
hipError_t launch_pc(const GemmParams& p, int b_layout, int out_bf16, hipStream_t stream);

// The launcher of (pipeline, tile bm × bn, stages) for input type `in`, or nullptr when that
// configuration is not built.
GemmLauncher find_gemm(int pipeline, int bm, int bn, int stages, int in = 0);
// Readable list of the built configurations of a pipeline (for error messages).
const char* gemm_configs_text(int pipeline, int in = 0);

// A kernel configuration for an M×N product on a device with num_cus compute units.  Zero
// arguments are open: pipeline 0 = either pipeline, bm = bn = 0 = any tile, stages 0 = each
// candidate's default.  Returns false when no built configuration matches what is fixed.
struct GemmChoice {
  int pipeline, bm, bn, stages;
};
bool choose_gemm(int64_t M, int64_t N, int num_cus, int pipeline, int bm, int bn, int stages, GemmChoice& out,
                 int in = 0);
// Launch a built configuration; fills tiles_m / tiles_n.  Returns hipErrorInvalidValue for a
// configuration find_gemm does not know.
hipError_t launch_gemm(GemmParams p, int pipeline, int bm, int bn, int stages, int b_layout, int out_bf16,
                       hipStream_t stream, int in = 0);
// One repack: `rows` rows of `row_bytes` bytes at pitch ld_src (bytes, any alignment) into
// pitch ld_dst (bytes, a multiple of 16), zero-filled past row_bytes.
struct PackJob {
  const uint8_t* src;
  int64_t ld_src, rows, row_bytes;
  uint8_t* dst;
  int64_t ld_dst;
};
// Runs n (1 or 2) repacks in one launch.
hipError_t launch_pack_jobs(const PackJob* jobs, int n, hipStream_t stream);
// `groups` repacks like `j`, their sources group_stride bytes apart, their results dense.
hipError_t launch_pack_groups(const PackJob& j, int64_t groups, int64_t group_stride, hipStream_t stream);
// Arguments of the ragged products (gemm_grouped.hpp).  Pitches of A and B in bytes, of C in
// elements; group e holds rows offsets[e] .. offsets[e+1]-1 (device memory) of `rows`.
//   rows product:     A rows × K, B_e at B + e·stride_b, C rows × N
//   weight gradient:  A rows × M, B rows × N, C_e M × N at C + e·stride_c (elements)
struct GroupedParams {
  const uint8_t* A;
  const uint8_t* B;
  void* C;
  const int32_t* offsets;
  int64_t lda, ldb, stride_b, ldc, stride_c;
  int groups, rows;
  int M, N, K;
  int tiles_m, tiles_n, group_m;  // rows product over offsets: tiles_m bounds all groups' tile rows
  int per_xcd;     // weight gradient: consecutive tiles of a group per XCD
  int by_rows;     // weight gradient: the groups run in the order of their rows (at most 64 groups)
  int vec_store;
  float alpha, beta;
  int scaled;
};
// in: 0 bf16, 1 fp16; out: 0 fp32, 1 bf16, 2 fp16 (a 16-bit output has the input's type).  Tiles
// 256×256, 128×128, 64×64; the launchers fill the tile counts from a choice that fits().
hipError_t launch_grouped(GroupedParams p, const TileChoice& c, int in, int b_layout, int out, hipStream_t stream);
hipError_t launch_wgrad(GroupedParams p, const TileChoice& c, int in, int out, hipStream_t stream);

// Arguments of the 4-bit conversions (mx4_quantize.hip): pitches in bytes; per_row = 4 units of 8
// values for every block of 32 (ceil(cols / 32) blocks); units and div are filled by the launcher.
struct Mx4Params {
  void* x;
  uint8_t* codes;
  uint8_t* scales;
  int64_t ldx, ld_codes, ld_scales, cols;
  uint32_t per_row, units;
  FastDiv div;
};
// dt: 0 fp32, 1 bf16, 2 fp16 (the type of x)
hipError_t launch_mx4_quantize(const Mx4Params& p, int64_t rows, int dt, hipStream_t stream);
hipError_t launch_mx4_dequantize(const Mx4Params& p, int64_t rows, int dt, hipStream_t stream);

// Arguments of the 4-bit products (gemm_mx4.hpp): g.A and g.B hold codes (pitches in bytes, K a
// multiple of 32), As and Bs the scale bytes; g.offsets null: one dense product of g.rows rows.
struct Mx4GemmParams {
  GroupedParams g;
  const uint8_t* As;
  const uint8_t* Bs;
  int64_t ld_as, ld_bs, stride_bs;
};
// Tiles 256×256 (a workgroup for each CU walks them) and 128×128 with 2 stages, 64×64 and 32×64 with
// 2 or 4.
hipError_t launch_mx4_gemm(Mx4GemmParams p, const TileChoice& c, int out_bf16, hipStream_t stream);
// Products with few rows (gemm_rows.hpp), B stored N×K, at most 16 rows when dense; fmt 0 bf16, 1
// fp16 (A, B and their pitches as GroupedParams), 2 microscaled 4-bit; out as launch_grouped.
hipError_t launch_few_rows(Mx4GemmParams p, const TileChoice& c, int fmt, int out, hipStream_t stream);

// Arguments of the products with weights in 4-bit codes (gemm_w4.hpp): g.A activations (rows at lda bytes),
// g.B codes (N rows at ldb bytes, a matrix of a group stride_b bytes after the last), g.offsets null: one dense
// product of g.rows rows.  Scales and zeros K/group × N at ld_s (ld_z) elements, matrices at stride_s (stride_z).
struct W4Params {
  GroupedParams g;
  const uint16_t* scales;
  const uint8_t* zeros;   // null in the launchers without zeros
  int64_t ld_s, stride_s, ld_z, stride_z;
  const int32_t* source;  // null, or row r reads row source[r] / top_k of A's a_rows
  FastDiv top_k;
  int a_rows;
  int out16;              // C has A's type, else fp32
};
// By A's type and whether zeros are given; group 32, 64 or 128; the tile counts come from `c`.
hipError_t launch_w4_bf16(const W4Params& p, int group, const TileChoice& c, hipStream_t stream);
hipError_t launch_w4_bf16_zeros(const W4Params& p, int group, const TileChoice& c, hipStream_t stream);
hipError_t launch_w4_f16(const W4Params& p, int group, const TileChoice& c, hipStream_t stream);
hipError_t launch_w4_f16_zeros(const W4Params& p, int group, const TileChoice& c, hipStream_t stream);

// fp8 GEMM (gemm_fp8.hpp): p in units of two fp8 values (lda, ldb, K, kchunks as for 16-bit data
// of half the width); fmt 0 E4M3, 1 E5M2; tiles 256×256, 128×128, 64×64.
hipError_t launch_fp8(GemmParams p, int bm, int bn, int fmt, int out_bf16, hipStream_t stream);
bool fp8_tile_built(int bm, int bn);

}  // namespace tbg
