// Rows to the groups of their experts and back, and the gradients of the way back.
//
//   dispatch      out[place[t,j]] = X[t]
//   combine       out[t] = sum over j of w[t,j]·Y[place[t,j]]          (fp32, j ascending, rounded once)
//   combine_grad  dY[place[t,j]] = w[t,j]·dout[t],  dw[t,j] = sum over the columns of Y[place[t,j]]·dout[t]
//
// All three move bytes, and all go by token: a token's row is read once for its k rows of the groups
// (by row of the groups it would be read k times), and the rows of one token are its own, so no two
// workgroups write the same row and nothing is added across workgroups.  A lane takes 16 bytes of a
// row; the last unit of a row is moved back to end with the row, so that rows of any length take only
// whole 16-byte accesses (the bytes that two units share get the same values from both).  Rows shorter
// than that go element by element.
//
// Bound by memory: 8192 tokens of 8 KiB, dispatch to 2 rows each 38 µs (5.3 TB/s), combine of 8 rows each
// 103 µs (5.9), combine_grad of 2 rows each 52 µs (6.5, part of it from the cache).  Few tokens are a launch:
// combine of 8 tokens, 8 rows each, 3.7 µs.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert.hpp"
#include "ragged.hpp"

namespace tbg {

namespace {

// 16 bytes of a row, which may start at any byte (gfx9 takes unaligned multi-dword accesses).
typedef uint32_t Raw16 __attribute__((ext_vector_type(4), aligned(1)));

// Values of a type: 0 fp32, 1 bf16, 2 fp16.
template <int DT> struct Elem;
template <> struct Elem<0> { typedef float type; };
template <> struct Elem<1> { typedef __bf16 type; };
template <> struct Elem<2> { typedef _Float16 type; };

// V consecutive values at any element's boundary.
template <int DT, int V>
struct VecOf {
  typedef typename Elem<DT>::type type __attribute__((ext_vector_type(V), aligned(sizeof(typename Elem<DT>::type))));
};
template <int DT>
struct VecOf<DT, 1> {
  typedef typename Elem<DT>::type type;
};
template <int DT, int V>
using Vec = typename VecOf<DT, V>::type;

template <int DT, int V>
__device__ __forceinline__ float value_of(const Vec<DT, V>& x, int i) {
  if constexpr (V == 1) return (float)x;
  else return (float)x[i];
}
template <int DT, int V>
__device__ __forceinline__ void set_value(Vec<DT, V>& x, int i, float f) {
  if constexpr (V == 1) x = (typename Elem<DT>::type)f;
  else x[i] = (typename Elem<DT>::type)f;
}

// Rows of the groups that the last-level cache cannot hold are read and written past it (NT), which leaves
// it to the rest; those that fit may still be in it, or be read from it next.  That form exists where many rows
// meet: dispatch to three and more rows a token, combine of five and more, gradients of rows of more than 128 units;
// those choose by kCacheBytes, the others are cached at any size.  Both sides, µs cached / past the cache, bf16, by
// MiB of the groups' rows (gradients: of Y and dY), the same buffers call after call:
//                                      128        256        512        1024
//   dispatch, 8 KiB rows, 1 a token   35 / 35    91 / 69   184 / 180  368 / 376   cached
//                         2           26 / 27    72 / 49   142 / 106  290 / 287   cached
//                         3           23 / 27    69 / 53   140 / 105  275 / 274   by size
//                         8           22 / 31    49 / 57   121 / 112  250 / 225   by size
//   combine, 8 KiB rows,  1           36 / 45    95 / 84   191 / 192  378 / 374   cached
//                         2           27 / 32    71 / 57   142 / 110  282 / 270   cached
//                         4           25 / 29    60 / 54   124 / 104  252 / 209   cached
//                         8           25 / 30    53 / 55   116 /  99  239 / 200   by size
//   gradients, 2 a token, 256 B rows  45 / 61   128 / 121  239 / 225              cached
//                         2000 B      26 / 33    66 / 64   138 / 116  280 / 233   cached
//                         8 KiB       23 / 29    72 / 56   127 /  99  254 / 192   by size
// (The cached kernels lose up to a quarter from 256 MiB on; a form past the cache for two to four rows a token would
// gain that.)
// (O names the type, O::type, so that its alignment stays with it.)
template <int NT, class O>
__device__ __forceinline__ typename O::type load_from(const uint8_t* at) {
  typedef typename O::type T;
  if constexpr (NT != 0) return __builtin_nontemporal_load((const T*)at);
  else return *(const T*)at;
}
template <int NT, class O>
__device__ __forceinline__ void store_to(uint8_t* at, typename O::type v) {
  typedef typename O::type T;
  if constexpr (NT != 0) __builtin_nontemporal_store(v, (T*)at);
  else *(T*)at = v;
}

// The first column of a unit: the last unit of a row ends with the row.
template <int V>
__device__ __forceinline__ int64_t unit_column(uint32_t u, int64_t cols) {
  const int64_t c = (int64_t)u * V;
  return c + V <= cols ? c : cols - V;
}

// ---- dispatch ------------------------------------------------------------------------------------

template <int SHORT> struct Unit { typedef Raw16 type; };
template <> struct Unit<1> { typedef uint8_t type; };
template <> struct Unit<2> { typedef uint16_t type; };
template <> struct Unit<4> { typedef uint32_t type; };

// SHORT 0: units of 16 bytes; else rows below 16 bytes, one element of SHORT bytes a unit.  J: rows in flight.
template <int SHORT, int J, int NT>
__global__ void __launch_bounds__(256) dispatch_kernel(RowsParams p) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= p.units) return;
  const uint32_t t = fast_div(i, p.div), u = i - t * p.per_row;
  constexpr int Bytes = SHORT ? SHORT : 16;
  typedef typename Unit<SHORT>::type T;
  const int64_t at = unit_column<Bytes>(u, p.cols);  // cols and columns count bytes here
  const int32_t* place = p.place + (int64_t)t * p.top_k;
  const T v = *(const T*)(p.in + (int64_t)t * p.ld_in + at);
  uint8_t* out = p.out + at;
  for (uint32_t j0 = 0; j0 < p.top_k; j0 += J) {
    uint32_t row[J];
#pragma unroll
    for (int j = 0; j < J; ++j) row[j] = j0 + j < p.top_k ? (uint32_t)place[j0 + j] : ~0u;
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (row[j] < p.rows) store_to<NT, Unit<SHORT>>(out + (int64_t)row[j] * p.ld_out, v);
  }
}

// ---- combine -------------------------------------------------------------------------------------

// Y: type of the rows, O: type of the sum, V: values a unit, J: rows in flight.
template <int Y, int O, int V, int J, int NT>
__global__ void __launch_bounds__(256) combine_kernel(RowsParams p) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= p.units) return;
  const uint32_t t = fast_div(i, p.div), u = i - t * p.per_row;
  const int64_t c = unit_column<V>(u, p.cols);
  const int32_t* place = p.place + (int64_t)t * p.top_k;
  const float* weights = p.weights ? p.weights + (int64_t)t * p.top_k : nullptr;
  typedef Vec<Y, V> In;
  const uint8_t* in = p.in + c * (int64_t)sizeof(typename Elem<Y>::type);
  float sum[V];
#pragma unroll
  for (int v = 0; v < V; ++v) sum[v] = 0.f;
  for (uint32_t j0 = 0; j0 < p.top_k; j0 += J) {
    uint32_t row[J];
    float w[J];
    In y[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      row[j] = j0 + j < p.top_k ? (uint32_t)place[j0 + j] : ~0u;
      w[j] = weights && j0 + j < p.top_k ? weights[j0 + j] : 1.f;
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (row[j] < p.rows) y[j] = load_from<NT, VecOf<Y, V>>(in + (int64_t)row[j] * p.ld_in);
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (row[j] < p.rows) {
#pragma unroll
        for (int v = 0; v < V; ++v) sum[v] = fmaf(w[j], value_of<Y, V>(y[j], v), sum[v]);
      }
  }
  Vec<O, V> o;
#pragma unroll
  for (int v = 0; v < V; ++v) set_value<O, V>(o, v, sum[v]);
  *(Vec<O, V>*)(p.out + (int64_t)t * p.ld_out + c * (int64_t)sizeof(typename Elem<O>::type)) = o;
}

// ---- combine_grad --------------------------------------------------------------------------------

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// A workgroup of W waves a token; J of its rows at a time.  Y: type of the rows, D: of dout.
template <int Y, int D, int V, int J, int W, int NT>
__global__ void __launch_bounds__(64 * W) combine_grad_kernel(RowsParams p) {
  __shared__ float part[W][J];
  const uint32_t t = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t* place = p.place + (int64_t)t * p.top_k;
  typedef typename Elem<Y>::type elem;
  const uint8_t* dout = p.dout + (int64_t)t * p.ld_dout;
  for (uint32_t j0 = 0; j0 < p.top_k; j0 += J) {
    uint32_t row[J];
    float w[J], dot[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const bool in = j0 + j < p.top_k;
      row[j] = in ? (uint32_t)place[j0 + j] : ~0u;
      w[j] = in && p.weights ? p.weights[(int64_t)t * p.top_k + j0 + j] : 1.f;
      dot[j] = 0.f;
    }
    for (uint32_t u = threadIdx.x; u < p.per_row; u += 64 * W) {
      const int64_t c = unit_column<V>(u, p.cols);
      const int shared = (int)((int64_t)u * V - c);  // values that the unit before has counted
      const Vec<D, V> d = *(const Vec<D, V>*)(dout + c * (int64_t)sizeof(typename Elem<D>::type));
      Vec<Y, V> y[J];
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (row[j] < p.rows)
          y[j] = load_from<NT, VecOf<Y, V>>(p.in + (int64_t)row[j] * p.ld_in + c * (int64_t)sizeof(elem));
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (row[j] >= p.rows) continue;
        Vec<Y, V> g;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float x = value_of<D, V>(d, v);
          dot[j] = v >= shared ? fmaf(value_of<Y, V>(y[j], v), x, dot[j]) : dot[j];
          set_value<Y, V>(g, v, w[j] * x);
        }
        store_to<NT, VecOf<Y, V>>(p.out + (int64_t)row[j] * p.ld_out + c * (int64_t)sizeof(elem), g);
      }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const float s = wave_sum(dot[j]);
      if (W > 1 && lane == 0) part[wave][j] = s;
      if (W == 1 && lane == 0 && j0 + j < p.top_k) p.dweights[(int64_t)t * p.top_k + j0 + j] = s;
    }
    if (W > 1) {
      __syncthreads();
      if (threadIdx.x < J && j0 + threadIdx.x < p.top_k) {
        float s = 0.f;
        for (int k = 0; k < W; ++k) s += part[k][threadIdx.x];
        p.dweights[(int64_t)t * p.top_k + j0 + threadIdx.x] = s;
      }
      __syncthreads();
    }
  }
}

// Whether the groups' rows fill the last-level cache.
constexpr int64_t kCacheBytes = 256ll << 20;
bool past_cache(const RowsParams& p, int size) {
  const int64_t held = (int64_t)p.tokens * p.top_k;
  return (held < p.rows ? held : p.rows) * p.cols * size >= kCacheBytes;
}

// Tokens that one launch takes: their units are numbered in 32 bits.
template <class Launch>
hipError_t by_tokens(const RowsParams& p, Launch launch) {
  const int64_t most = ((1ll << 32) - 256) / p.per_row, all = p.tokens;
  for (int64_t t = 0; t < all; t += most) {
    const int64_t n = all - t < most ? all - t : most;
    RowsParams q = p;
    q.tokens = (uint32_t)n;
    q.units = (uint32_t)(n * p.per_row);
    q.place += t * p.top_k;
    if (q.weights) q.weights += t * p.top_k;
    launch(q, t, (unsigned)((q.units + 255ull) / 256));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int SHORT>
hipError_t dispatch_units(RowsParams p, hipStream_t s) {
  constexpr int Bytes = SHORT ? SHORT : 16;
  p.per_row = (uint32_t)((p.cols + Bytes - 1) / Bytes);
  p.div = make_fast_div(p.per_row);
  return by_tokens(p, [&](RowsParams q, int64_t t, unsigned grid) {
    q.in += t * p.ld_in;
    // (figures at load_from)
    if (p.top_k <= 2) hipLaunchKernelGGL((dispatch_kernel<SHORT, 2, 0>), dim3(grid), dim3(256), 0, s, q);
    else if (!past_cache(p, 1)) hipLaunchKernelGGL((dispatch_kernel<SHORT, 8, 0>), dim3(grid), dim3(256), 0, s, q);
    else hipLaunchKernelGGL((dispatch_kernel<SHORT, 8, 1>), dim3(grid), dim3(256), 0, s, q);
  });
}

template <int Y, int O, int V>
hipError_t combine_units(RowsParams p, hipStream_t s) {
  p.per_row = (uint32_t)((p.cols + V - 1) / V);
  p.div = make_fast_div(p.per_row);
  return by_tokens(p, [&](RowsParams q, int64_t t, unsigned grid) {
    q.out += t * p.ld_out;
    // (figures at load_from)
    const bool past = past_cache(p, (int)sizeof(typename Elem<Y>::type));
    if (p.top_k <= 2) hipLaunchKernelGGL((combine_kernel<Y, O, V, 2, 0>), dim3(grid), dim3(256), 0, s, q);
    else if (p.top_k <= 4) hipLaunchKernelGGL((combine_kernel<Y, O, V, 4, 0>), dim3(grid), dim3(256), 0, s, q);
    else if (!past) hipLaunchKernelGGL((combine_kernel<Y, O, V, 8, 0>), dim3(grid), dim3(256), 0, s, q);
    else hipLaunchKernelGGL((combine_kernel<Y, O, V, 8, 1>), dim3(grid), dim3(256), 0, s, q);
  });
}

template <int Y, int O>
hipError_t combine_types(const RowsParams& p, hipStream_t s) {
  constexpr int V = Y == 0 ? 4 : 8;
  return p.cols >= V ? combine_units<Y, O, V>(p, s) : combine_units<Y, O, 1>(p, s);
}

template <int Y, int D, int V, int J, int W, int NT>
hipError_t grad_launch(const RowsParams& p, hipStream_t s) {
  const int64_t most = (1 << 22) - 1;  // workgroups of 256 threads a launch, counted in 32 bits
  for (int64_t t = 0; t < p.tokens; t += most) {
    const int64_t n = p.tokens - t < most ? p.tokens - t : most;
    RowsParams q = p;
    q.dout += t * p.ld_dout;
    q.place += t * p.top_k;
    if (q.weights) q.weights += t * p.top_k;
    q.dweights += t * p.top_k;
    hipLaunchKernelGGL((combine_grad_kernel<Y, D, V, J, W, NT>), dim3((unsigned)n), dim3(64 * W), 0, s, q);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Waves a token: one for rows of up to 128 units (2047 tokens, 4 rows of 126 units each: 9.9 µs with one wave, 10.2
// with two, 11.3 with four), else four (8192 tokens, 2 rows of 512 units: 71, 68, 67).  Past the cache, where the
// rows are long, by those of Y and dY together (figures at load_from).
template <int Y, int D, int V, int J>
hipError_t grad_rows(const RowsParams& p, hipStream_t s) {
  if (p.per_row <= 128) return grad_launch<Y, D, V, J, 1, 0>(p, s);
  if (!past_cache(p, 2 * (int)sizeof(typename Elem<Y>::type))) return grad_launch<Y, D, V, J, 4, 0>(p, s);
  return grad_launch<Y, D, V, J, 4, 1>(p, s);
}

template <int Y, int D, int V>
hipError_t grad_units(RowsParams p, hipStream_t s) {
  p.per_row = (uint32_t)((p.cols + V - 1) / V);
  if (p.top_k <= 2) return grad_rows<Y, D, V, 2>(p, s);
  if (p.top_k <= 4) return grad_rows<Y, D, V, 4>(p, s);
  return grad_rows<Y, D, V, 8>(p, s);
}

template <int Y, int D>
hipError_t grad_types(const RowsParams& p, hipStream_t s) {
  constexpr int V = Y == 0 ? 4 : 8;
  return p.cols >= V ? grad_units<Y, D, V>(p, s) : grad_units<Y, D, 1>(p, s);
}

}  // namespace

hipError_t launch_expert_dispatch(RowsParams p, int size, hipStream_t stream) {
  p.cols *= size;
  if (p.cols >= 16) return dispatch_units<0>(p, stream);
  if (size == 4) return dispatch_units<4>(p, stream);
  return size == 2 ? dispatch_units<2>(p, stream) : dispatch_units<1>(p, stream);
}

hipError_t launch_expert_combine(RowsParams p, int y, int out, hipStream_t stream) {
  if (y == 0) return combine_types<0, 0>(p, stream);
  if (y == 1) return out ? combine_types<1, 1>(p, stream) : combine_types<1, 0>(p, stream);
  return out ? combine_types<2, 2>(p, stream) : combine_types<2, 0>(p, stream);
}

hipError_t launch_expert_combine_grad(RowsParams p, int y, int d, hipStream_t stream) {
  if (y == 0) return grad_types<0, 0>(p, stream);
  if (y == 1) return d ? grad_types<1, 1>(p, stream) : grad_types<1, 0>(p, stream);
  return d ? grad_types<2, 2>(p, stream) : grad_types<2, 0>(p, stream);
}

}  // namespace tbg
