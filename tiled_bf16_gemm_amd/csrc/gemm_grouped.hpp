// Ragged products of 16-bit operands: the rows of group e times B_e, and the weight gradient
// X_eᵀ·Y_e whose sum runs over the rows of group e.
//
// Both run the barrier ring (gemm_ring.hpp): the same workgroup tiles, LDS layouts, copy atoms,
// products and epilogue.  What is new is where a tile lies (ragged.hpp) and that either operand
// may be stored with the sum's index outermost: the gradient's X and Y both are, so its A
// fragments are read with the transposing LDS read as well.
//
// Bounds.  An operand with the sum's index innermost (kc) has its rows past the tile masked in
// the lane offsets and its 16-byte chunks past K by the chunk count; one with the sum's index
// outermost (ko) has its columns masked in the lane offsets and its rows past the end by the
// buffer range, which ends at the last row of the group (gradient) or of B_e: rows of the next
// group, whatever they hold, never enter a sum.
#pragma once
#include "gemm_common.hpp"
#include "gemm_ring.hpp"
#include "ragged.hpp"

namespace tbg {

// Storage of an operand relative to the sum's index.
constexpr int kSumOuter = 0, kSumInner = 1;

// One operand's box in a workgroup tile.  `origin` is the address of its first row (kSumInner)
// or first column (kSumOuter) at the sum's index 0; `lines` counts the rows (columns) that exist
// from there; `sum` is the number of the sum's terms.
struct TileBox {
  rsrc_t r0;
  uint32_t pitch, step;  // bytes per memory row; bytes per K tile
  int lines;
  int chunks;    // kSumInner: 16-byte chunks of the sum's index in a row
  int64_t rem0;  // kSumOuter: bytes from the origin to the end of the last row
};

template <int L>
__device__ __forceinline__ TileBox make_box(const uint8_t* origin, uint32_t pitch, int lines, int sum) {
  TileBox b;
  b.pitch = pitch;
  b.lines = lines;
  b.chunks = (sum + 7) >> 3;
  if (L == kSumInner) {
    b.r0 = make_rsrc(origin, 0x7FFFFFFFull);
    b.step = 128u;
    b.rem0 = 0;
  } else {
    b.r0 = make_rsrc(origin, 0);
    b.step = pitch * kBK;
    // to a whole dword: the range check works on dwords (the 16-byte chunk that straddles the
    // last column is loaded whole and feeds only outputs that are never written)
    const int64_t rem = sum > 0 ? ((int64_t)(sum - 1) * pitch + (int64_t)lines * 2 + 3) & ~(int64_t)3 : 0;
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)rem);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)rem >> 32));
    b.rem0 = (int64_t)(((uint64_t)hi << 32) | lo);
  }
  return b;
}

// Buffer descriptor of K tile kt; INTERIOR: the tile lies wholly inside the sum.
template <int L, bool INTERIOR>
__device__ __forceinline__ rsrc_t box_rsrc(const TileBox& b, int kt, bool live) {
  const uint64_t off = (uint64_t)kt * b.step;
  rsrc_t r = rsrc_advance(b.r0, off);
  if (L == kSumOuter) {
    if (INTERIOR) {
      r.z = 0x7FFFFFFF;
    } else {
      CopyPlan c;
      c.rem_b0 = b.rem0;
      r.z = kn_range(c, off, live);
    }
  }
  return r;
}

// The wave's copy atoms of one operand: AT of the box's atoms, lane offsets and chunk numbers.
template <int L, int AT>
__device__ __forceinline__ void box_lanes(LaneChunk (&lc)[AT], const TileBox& b, int wave, int lane) {
  const int box = (wave * AT) >> 3;  // kSumOuter: which 64 columns
#pragma unroll
  for (int i = 0; i < AT; ++i) {
    if (L == kSumInner) {
      const int row = 8 * (AT * wave + i);
      lc[i] = lane_chunk<kSwizzle128B2Row>(row, lane, b.pitch);
      mask_row(lc[i], row + (lane >> 3), b.lines);
    } else {
      lc[i] = lane_chunk<kSwizzleKnTr>(8 * ((wave * AT + i) & 7), lane, b.pitch);
      lc[i].offset += 128u * box;
      if (lc[i].chunk >= ((b.lines - 64 * box + 7) >> 3)) lc[i].offset = kOobOffset;
    }
  }
}

// Fragment read addresses of one operand for wave row/column w; F fragments of 16 lines.
template <int L, int F>
struct BoxFrag {
  static constexpr int Q = F < 4 ? F : 4;
  uint32_t lane, col[2];
  uint32_t tr[Q][2];
  int w;
};

template <int L, int F>
__device__ __forceinline__ BoxFrag<L, F> make_box_frag(int w, int lane) {
  BoxFrag<L, F> f;
  f.w = w;
  if (L == kSumInner) {
    const int row = w * 16 * F + (lane & 15), x = (row >> 1) & 7;
    f.lane = (uint32_t)row * 128u;
    f.col[0] = (uint32_t)((lane >> 4) ^ x) * 16u;
    f.col[1] = (uint32_t)((4 + (lane >> 4)) ^ x) * 16u;
  } else {
    // as make_frag_addr: lane 16g + 4e + q supplies 8 bytes at row 8g + 4h + e, columns 4q..4q+3
    const int tg = lane >> 4, te = (lane >> 2) & 3, tq = lane & 3;
#pragma unroll
    for (int q = 0; q < BoxFrag<L, F>::Q; ++q)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int f4 = F >= 4 ? q : 2 * w + q;
        const int r = 8 * tg + 4 * h + te, c = f4 * 2 + (tq >> 1);
        f.tr[q][h] = (uint32_t)r * 128u + (uint32_t)((c ^ row_xor<kSwizzleKnTr>(r)) * 16) + (uint32_t)((tq & 1) * 8);
      }
  }
  return f;
}

template <int L, int F>
__device__ __forceinline__ bf16x8_t read_box_frag(const BoxFrag<L, F>& f, const uint8_t* s, int kk, int i) {
  if (L == kSumInner) return *(const bf16x8_t*)(s + f.lane + i * 2048 + f.col[kk]);
  const int box = F >= 4 ? f.w * (F / 4) + (i >> 2) : 0, q = F >= 4 ? (i & 3) : i;
  const uint8_t* base = s + box * 8192 + kk * 4096;
  const bf16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
      (__attribute__((address_space(3))) bf16x4_t*)(base + f.tr[q][0]));
  const bf16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
      (__attribute__((address_space(3))) bf16x4_t*)(base + f.tr[q][1]));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// The ring over one workgroup tile: acc += A·B over `sum` terms.  The schedule is the barrier
// ring's (gemm_ring.hpp): k-step 0, the stage barrier, k-step 1 with the next tile's first
// fragments and the copies of tile kt+S; products in serpentine order.
template <class T, int S, int AL, int BL>
__device__ __forceinline__ void ring_product(f32x4_t (&acc)[T::FN][T::FM], uint8_t* smem, const TileBox& ba,
                                             const TileBox& bb, int sum, int wave, int lane) {
  constexpr int FM = T::FM, FN = T::FN, AT = T::AtomsA, BT = T::AtomsB, A = T::Atoms, P = T::Products, R = T::Reads;
  const int ktiles = sum > 0 ? (sum + kBK - 1) / kBK : 1;
  LaneChunk la[AT], lb[BT];
  box_lanes<AL, AT>(la, ba, wave, lane);
  box_lanes<BL, BT>(lb, bb, wave, lane);
  const BoxFrag<AL, FM> fa = make_box_frag<AL, FM>(wave >> 1, lane);
  const BoxFrag<BL, FN> fb = make_box_frag<BL, FN>(wave & 1, lane);
  const uint32_t smem_addr = lds_addr_of(smem);

  struct Copy {
    rsrc_t ra, rb;
    uint32_t lds_a, lds_b;
    int valid;
  };
  auto make_copy = [&](int kt, int stage, auto interior) __attribute__((always_inline)) {
    constexpr bool in = decltype(interior)::value;
    Copy c;
    c.ra = box_rsrc<AL, in>(ba, kt, kt < ktiles);
    c.rb = box_rsrc<BL, in>(bb, kt, kt < ktiles);
    c.valid = (AL == kSumInner ? ba.chunks : bb.chunks) - kt * (kBK / 8);
    c.lds_a = smem_addr + stage * T::StageBytes + AT * wave * 1024;
    c.lds_b = smem_addr + stage * T::StageBytes + T::ABytes + BT * wave * 1024;
    return c;
  };
  // a kSumInner chunk test as in copy_atom: the atoms of one parity share their chunk
  auto atom = [&](const Copy& c, int j, auto interior) __attribute__((always_inline)) {
    constexpr bool in = decltype(interior)::value;
    if (j < AT) {
      issue_atom_if(c.ra, c.lds_a, j * 1024, la[j].offset, in || AL == kSumOuter || la[j & 1].chunk < c.valid);
    } else {
      const int i = j - AT;
      issue_atom_if(c.rb, c.lds_b, i * 1024, lb[i].offset, in || BL == kSumOuter || lb[i & 1].chunk < c.valid);
    }
  };
  auto read = [&](Frags<T>& f, const uint8_t* s, int kk, int i) __attribute__((always_inline)) {
    if (i < FM) f.a[i] = read_box_frag<AL, FM>(fa, s, kk, i);
    else f.b[i - FM] = read_box_frag<BL, FN>(fb, s + T::ABytes, kk, i - FM);
  };
  auto step = [&](const Frags<T>& cur, Frags<T>& nxt, const uint8_t* s, int kk, const Copy& c, auto copies,
                  auto interior) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
#pragma unroll
      for (int r = (i * R + P - 1) / P; r < ((i + 1) * R + P - 1) / P; ++r) read(nxt, s, kk, r);
      if (decltype(copies)::value && i >= P / (2 * A)) {
        constexpr int H = P / (2 * A);
#pragma unroll
        for (int j = ((i - H) * A + P - 1) / P; j < ((i + 1 - H) * A + P - 1) / P; ++j) atom(c, j, interior);
      }
      const int fn = i / FM, fm = (fn & 1) ? FM - 1 - i % FM : i % FM;
      mfma16<T::AsmMfma, T::In>(acc[fn][fm], cur.b[fn], cur.a[fm]);
    }
  };

  Frags<T> f0, f1;
#pragma unroll
  for (int t = 0; t < S; ++t) {
    const Copy c = make_copy(t, t, std::false_type{});
#pragma unroll
    for (int j = 0; j < A; ++j) atom(c, j, std::false_type{});
  }
  stage_barrier<A*(S - 1)>();  // tile 0 landed; tiles 1..S-1 may be in flight
#pragma unroll
  for (int r = 0; r < R; ++r) read(f0, smem, 0, r);
  auto tile = [&](int kt, auto stage, auto interior) __attribute__((always_inline)) {
    constexpr int cur = decltype(stage)::value, nxt = cur + 1 == S ? 0 : cur + 1;
    step(f0, f1, smem + cur * T::StageBytes, 1, Copy{}, std::false_type{}, interior);
    stage_barrier<A*(S - 2)>();  // tile kt+1 landed, stage `cur` free
    step(f1, f0, smem + nxt * T::StageBytes, 0, make_copy(kt + S, cur, interior), std::true_type{}, interior);
  };
  int kt = 0;
  for (; kt + 2 * S < ktiles; kt += S)
    for_stages<S>([&](auto st) __attribute__((always_inline)) { tile(kt + decltype(st)::value, st, std::true_type{}); });
  for (; kt + S <= ktiles; kt += S)
    for_stages<S>([&](auto st) __attribute__((always_inline)) { tile(kt + decltype(st)::value, st, std::false_type{}); });
  for_stages<S - 1>([&](auto st) __attribute__((always_inline)) {
    if (kt + decltype(st)::value < ktiles) tile(kt + decltype(st)::value, st, std::false_type{});
  });
  drain_acc<T>(acc);
  stage_barrier<0>();
}

// What store_tile reads of its arguments.
__device__ __forceinline__ GemmParams store_params(void* C, int64_t ldc, int M, int N, int vec_store, float alpha,
                                                   float beta) {
  GemmParams q;
  q.C = C;
  q.ldc = ldc;
  q.M = M;
  q.N = N;
  q.vec_store = vec_store;
  q.alpha = alpha;
  q.beta = beta;
  return q;
}

// C[r] = alpha·A[r]·B_e + beta·C[r] for the rows r of group e.
template <int BM, int BN, int S, int IN, int BL, int OUT, int SCALED>
__global__ void __launch_bounds__(kThreads, (RingCfg<BM, BN, S>::MinBlocks)) gemm_grouped_kernel(GroupedParams p) {
  using T = TileCfg<BM, BN, IN>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[RingCfg<BM, BN, S>::LdsBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RaggedTile t;
  if (!ragged_tile<BM>(p, p.group_m, blockIdx.x, t)) return;
  const int n0 = t.tn * BN;
  const uint8_t* b = p.B + (int64_t)t.group * p.stride_b + (BL == kSumInner ? (int64_t)n0 * p.ldb : (int64_t)n0 * 2);
  const TileBox ba = make_box<kSumInner>(p.A + (int64_t)t.row0 * p.lda, (uint32_t)p.lda, t.rows, p.K);
  const TileBox bb = make_box<BL>(b, (uint32_t)p.ldb, p.N - n0, p.K);
  f32x4_t acc[T::FN][T::FM];
  zero_acc<T>(acc);
  ring_product<T, S, kSumInner, BL>(acc, smem, ba, bb, p.K, wave, lane);
  const GemmParams q = store_params(p.C, p.ldc, t.row0 + t.rows, p.N, p.vec_store, p.alpha, p.beta);
  store_tile<T, OUT, SCALED>(acc, smem + wave * (T::RingBytes / 4), q, t.row0 + (wave >> 1) * T::TM,
                             n0 + (wave & 1) * T::TN, lane);
}

// C_e = alpha·X[rows of e]ᵀ·Y[rows of e] + beta·C_e; A holds X, B holds Y, M and N their widths.
template <int BM, int BN, int S, int IN, int OUT, int SCALED>
__global__ void __launch_bounds__(kThreads, (RingCfg<BM, BN, S>::MinBlocks)) gemm_wgrad_kernel(GroupedParams p) {
  using T = TileCfg<BM, BN, IN>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[RingCfg<BM, BN, S>::LdsBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  GradTile t;
  if (!grad_tile(p, blockIdx.x, t)) return;
  const int g = t.group, begin = t.begin, sum = t.rows;
  const int m0 = t.tm * BM, n0 = t.tn * BN;
  const TileBox ba = make_box<kSumOuter>(p.A + (int64_t)begin * p.lda + (int64_t)m0 * 2, (uint32_t)p.lda, p.M - m0, sum);
  const TileBox bb = make_box<kSumOuter>(p.B + (int64_t)begin * p.ldb + (int64_t)n0 * 2, (uint32_t)p.ldb, p.N - n0, sum);
  f32x4_t acc[T::FN][T::FM];
  zero_acc<T>(acc);
  ring_product<T, S, kSumOuter, kSumOuter>(acc, smem, ba, bb, sum, wave, lane);
  uint8_t* C = (uint8_t*)p.C + (int64_t)g * p.stride_c * (OUT != 0 ? 2 : 4);
  const GemmParams q = store_params(C, p.ldc, p.M, p.N, p.vec_store, p.alpha, p.beta);
  store_tile<T, OUT, SCALED>(acc, smem + wave * (T::RingBytes / 4), q, m0 + (wave >> 1) * T::TM,
                             n0 + (wave & 1) * T::TN, lane);
}

}  // namespace tbg
