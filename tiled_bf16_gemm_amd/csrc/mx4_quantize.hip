// Microscaled 4-bit data: quantisation of fp32, bf16 and fp16 rows and the way back.
//
// A block is 32 values along a row (the sum's index of a product).  With m = max |x| over the block,
//   e = clamp(floor(log2 m) - 2, -127, 127),   scale byte = e + 127 (E8M0),
//   code = E2M1(x / 2^e): 0, 0.5, 1, 1.5, 2, 3, 4 or 6 with a sign, rounded to nearest even and
//   clipped to 6 (m / 2^e lies in [4, 8));
// the OCP Microscaling Formats specification, version 1.0, sections 5.3.3 and 6.3.  floor(log2 m) is
// m's exponent field, so the byte is max(field, 2) - 2, subnormal and zero maxima included.  A
// block that holds a NaN or an infinity has field 255: its byte is 255 (NaN) and its codes 0.
//
// Both directions move bytes: 4 lanes share a block, a lane holds 8 consecutive values (one or two
// 16-byte loads, one dword of codes), so a wave's loads and stores are contiguous runs.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fast_div.hpp"
#include "launch.hpp"

namespace tbg {

namespace {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

// Eight values as they lie in memory; rows may start at any element, so the vector loads and
// stores carry the element's alignment only (gfx9 takes unaligned multi-dword accesses).
struct __attribute__((packed, aligned(2))) Raw16 { uint32_t w[4]; };
struct __attribute__((packed, aligned(4))) Raw32 { uint32_t w[8]; };

template <int DT>  // 0 fp32, 1 bf16, 2 fp16
struct Values {
  static constexpr int Bytes = DT == 0 ? 4 : 2;
  uint32_t w[DT == 0 ? 8 : 4];
};

// The lane's values from column c0 of a row of `cols`; those past the row are zero.
template <int DT>
__device__ __forceinline__ Values<DT> load8(const uint8_t* row, int64_t c0, int64_t cols) {
  Values<DT> v;
  const uint8_t* p = row + c0 * Values<DT>::Bytes;
  if (c0 + 8 <= cols) {
    if constexpr (DT == 0) {
      const Raw32 r = *(const Raw32*)p;
#pragma unroll
      for (int i = 0; i < 8; ++i) v.w[i] = r.w[i];
    } else {
      const Raw16 r = *(const Raw16*)p;
#pragma unroll
      for (int i = 0; i < 4; ++i) v.w[i] = r.w[i];
    }
    return v;
  }
  if constexpr (DT == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v.w[i] = c0 + i < cols ? ((const uint32_t*)p)[i] : 0u;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = c0 + 2 * i < cols ? ((const uint16_t*)p)[2 * i] : 0u;
      const uint32_t hi = c0 + 2 * i + 1 < cols ? ((const uint16_t*)p)[2 * i + 1] : 0u;
      v.w[i] = lo | hi << 16;
    }
  }
  return v;
}

// Bits of the largest magnitude among the lane's values, in fp32's format.  Magnitudes compare
// as unsigned integers in every one of the formats, infinities and NaN above all finite values.
template <int DT>
__device__ __forceinline__ uint32_t largest(const Values<DT>& v) {
  if constexpr (DT == 0) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, v.w[i] & 0x7FFFFFFFu);
    return m;
  } else {
    u16x2_t m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, v.w[i] & 0x7FFF7FFFu));
    const uint32_t h = max((uint32_t)m[0], (uint32_t)m[1]);
    if (DT == 1) return h << 16;
    return __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)h));
  }
}

// Eight codes, the first value in the lowest nibble (conversion: to nearest even, clipped).
template <int DT>
__device__ __forceinline__ uint32_t codes8(const Values<DT>& v, float scale) {
  uint32_t c = 0;
  if constexpr (DT == 0) {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(v.w[0]), __uint_as_float(v.w[1]), scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(v.w[2]), __uint_as_float(v.w[3]), scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(v.w[4]), __uint_as_float(v.w[5]), scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(v.w[6]), __uint_as_float(v.w[7]), scale, 3);
  } else if constexpr (DT == 1) {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, v.w[0]), scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, v.w[1]), scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, v.w[2]), scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, v.w[3]), scale, 3);
  } else {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, v.w[0]), scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, v.w[1]), scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, v.w[2]), scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, v.w[3]), scale, 3);
  }
  return c;
}

// 2^(byte - 127): byte 0 is the subnormal 2^-127, 255 is NaN.
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23);
}

// Maximum over the four lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xf, 0xf, true));  // lanes 1 0 3 2
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xf, 0xf, true));  // lanes 2 3 0 1
}

// A thread's unit is 8 values of a row; the units of a row are a multiple of 4 (whole blocks),
// so a quad always holds one block and the tests below are uniform over it.
template <int DT>
__global__ void __launch_bounds__(256) mx4_quantize_kernel(Mx4Params p) {
  const uint32_t t = blockIdx.x * 256u + threadIdx.x;
  if (t >= p.units) return;
  const uint32_t r = fast_div(t, p.div), u = t - r * p.per_row;
  const Values<DT> v = load8<DT>((const uint8_t*)p.x + (int64_t)r * p.ldx, (int64_t)u * 8, p.cols);
  const uint32_t field = quad_max(largest<DT>(v)) >> 23;
  const bool bad = field == 255;
  const uint32_t byte = bad ? 255u : max(field, 2u) - 2u;
  const uint32_t c = codes8<DT>(v, scale_of(byte));
  *(uint32_t*)(p.codes + (int64_t)r * p.ld_codes + u * 4) = bad ? 0u : c;
  if ((u & 3) == 0) p.scales[(int64_t)r * p.ld_scales + (u >> 2)] = (uint8_t)byte;
}

// The lane's eight values of codes `c` at a row's column c0 (those past the row are not written).
template <int DT>
__global__ void __launch_bounds__(256) mx4_dequantize_kernel(Mx4Params p) {
  const uint32_t t = blockIdx.x * 256u + threadIdx.x;
  if (t >= p.units) return;
  const uint32_t r = fast_div(t, p.div), u = t - r * p.per_row;
  const uint32_t c = *(const uint32_t*)(p.codes + (int64_t)r * p.ld_codes + u * 4);
  const uint32_t byte = p.scales[(int64_t)r * p.ld_scales + (u >> 2)];
  const float scale = scale_of(byte);
  uint8_t* dst = (uint8_t*)p.x + (int64_t)r * p.ldx + (int64_t)u * 8 * Values<DT>::Bytes;
  Values<DT> v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t pair = c >> (8 * i);
    if constexpr (DT == 0) {
      const f32x2_t f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(pair, scale, 0);
      v.w[2 * i] = byte == 255 ? 0x7FC00000u : __float_as_uint(f[0]);
      v.w[2 * i + 1] = byte == 255 ? 0x7FC00000u : __float_as_uint(f[1]);
    } else if constexpr (DT == 1) {
      v.w[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(pair, scale, 0));
      if (byte == 255) v.w[i] = 0x7FC07FC0u;
    } else {
      v.w[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(pair, scale, 0));
      if (byte == 255) v.w[i] = 0x7E007E00u;
    }
  }
  const int64_t left = p.cols - (int64_t)u * 8;
  if (left >= 8) {
    if constexpr (DT == 0) {
      Raw32 o;
#pragma unroll
      for (int i = 0; i < 8; ++i) o.w[i] = v.w[i];
      *(Raw32*)dst = o;
    } else {
      Raw16 o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o.w[i] = v.w[i];
      *(Raw16*)dst = o;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i >= left) break;
    if constexpr (DT == 0) ((uint32_t*)dst)[i] = v.w[i];
    else ((uint16_t*)dst)[i] = (uint16_t)(v.w[i >> 1] >> (16 * (i & 1)));
  }
}

// Rows that one launch takes: their units are numbered in 32 bits.
template <class Launch>
hipError_t by_rows(Mx4Params p, int64_t rows, Launch launch) {
  const int64_t most = ((1ll << 32) - 256) / p.per_row;
  p.div = make_fast_div(p.per_row);
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t n = rows - r < most ? rows - r : most;
    Mx4Params q = p;
    q.x = (uint8_t*)p.x + r * p.ldx;
    q.codes = p.codes + r * p.ld_codes;
    q.scales = p.scales + r * p.ld_scales;
    q.units = (uint32_t)(n * p.per_row);
    launch(q, (q.units + 255) / 256);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_mx4_quantize(const Mx4Params& p, int64_t rows, int dt, hipStream_t stream) {
  return by_rows(p, rows, [&](const Mx4Params& q, unsigned grid) {
    if (dt == 0) hipLaunchKernelGGL((mx4_quantize_kernel<0>), dim3(grid), dim3(256), 0, stream, q);
    else if (dt == 1) hipLaunchKernelGGL((mx4_quantize_kernel<1>), dim3(grid), dim3(256), 0, stream, q);
    else hipLaunchKernelGGL((mx4_quantize_kernel<2>), dim3(grid), dim3(256), 0, stream, q);
  });
}

hipError_t launch_mx4_dequantize(const Mx4Params& p, int64_t rows, int dt, hipStream_t stream) {
  return by_rows(p, rows, [&](const Mx4Params& q, unsigned grid) {
    if (dt == 0) hipLaunchKernelGGL((mx4_dequantize_kernel<0>), dim3(grid), dim3(256), 0, stream, q);
    else if (dt == 1) hipLaunchKernelGGL((mx4_dequantize_kernel<1>), dim3(grid), dim3(256), 0, stream, q);
    else hipLaunchKernelGGL((mx4_dequantize_kernel<2>), dim3(grid), dim3(256), 0, stream, q);
  });
}

}  // namespace tbg
