// Products of microscaled 4-bit operands (E2M1 codes, one E8M0 scale per 32 values along K) on
// gfx950's scaled 16×16×128 matrix instruction: C = A·Bᵀ, A M×K, B stored N×K, dense or with the
// rows in ragged groups and one B per group; fp32 accumulation.
//
// A K tile is 256 values, 128 bytes of codes per row: in bytes the ring, its copy atoms, LDS
// layout, fragment reads and epilogue are those of the 16-bit kernels (gemm_ring.hpp), and a
// k-step of 64 bytes is one 16×16×128 product per fragment pair.  Two things are new.
//  * Scales.  A K tile has 8 scale bytes per row.  They reach LDS as 16-byte chunks, 16 blocks,
//    of a row: one copy for two K tiles, 64 rows per atom (256×256: two atoms per wave and pair
//    of tiles, next to 32 atoms of codes).  The instruction takes a lane's scale from one byte of
//    a register, chosen by an immediate.
//  * Placement.  Lane l multiplies row l%16 and, in k-step kk, block 2(l/16)+kk of the tile (not
//    4kk + l/16): its two k-steps then need two neighbouring scale bytes, one 16-bit LDS read per
//    fragment and K tile.  The sum runs over the tile's blocks in another order, the same for A
//    and B.  The copies place block 2g+kk of a row where the 16-bit kernels have chunk 4kk+g, so
//    the fragment reads, free of bank conflicts, are unchanged.
// Bounds: rows past the tile and code chunks past K are masked copies (zero codes); scale rows past
// the tile too, and scale bytes past the last block, whatever the row's padding holds, are zeroed
// in registers in the tiles at the end of K (a NaN scale would turn zero codes into NaN).
#pragma once
#include "gemm_common.hpp"
#include "gemm_grouped.hpp"
#include "gemm_ring.hpp"
#include "ragged.hpp"

namespace tbg {

typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));
typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));

// One 16×16×128 product of 4-bit fragments; byte KK of sa and sb holds the lane's scales.  ASM as
// in mfma16 (drain_acc after the loop).
template <bool ASM, int KK>
__device__ __forceinline__ void mfma_mx4(f32x4_t& acc, const i32x4_t& a, const i32x4_t& b, uint32_t sa, uint32_t sb) {
  static_assert(KK == 0 || KK == 1, "one of the two blocks of a K tile");
  if (!ASM) {
    const i32x8_t x = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, y = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc, 4, 4, KK, (int)sa, KK, (int)sb);
  } else if (KK == 0) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                 : "+a"(acc) : "v"(a), "v"(b), "v"(sa), "v"(sb));
  } else {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                 : "+a"(acc) : "v"(a), "v"(b), "v"(sa), "v"(sb));
  }
}

template <int BM, int BN, int S>
struct Mx4Cfg {
  using T = TileCfg<BM, BN>;
  static_assert(S % 2 == 0, "a pair of K tiles shares its scale copies");
  static constexpr int RowsA = BM < 64 ? 64 : BM;           // an atom's 64 rows are all A's or all B's
  static constexpr int Rows = RowsA + BN;
  static constexpr int ScaleBytes = Rows * 16;             // scales of one pair of K tiles
  static constexpr int Buffers = S / 2 + 1 <= 2 ? 2 : 4;   // pairs held: the S/2 in flight and the one in use
  static constexpr int ScaleAtoms = Rows < 256 ? 1 : Rows / 256;  // per wave and pair
  // Fewer than 256 rows leave waves without scale rows; they copy zeros into a spare area, so
  // that every wave counts the same copies.
  static constexpr int SpareBytes = Rows < 256 ? 2048 : 0;
  static constexpr int ScaleArea = Buffers * ScaleBytes + SpareBytes;
  static constexpr int LdsBytes = S * T::StageBytes + ScaleArea;
  static constexpr int MinBlocks = 2 * LdsBytes <= 160 * 1024 ? 2 : 1;
  static_assert(LdsBytes <= 160 * 1024, "the ring must fit in LDS");
  static_assert((S - 1) * T::Atoms + S / 2 * ScaleAtoms <= 63, "copies in flight must fit the vmcnt counter");
};

// The operands of one workgroup tile: code and scale buffers from the tile's first row, rows that
// exist from there, blocks of 32 along K.
struct Mx4Box {
  rsrc_t ra, rb, ras, rbs;
  uint32_t pitch_a, pitch_b, pitch_as, pitch_bs;
  int rows_a, rows_b, blocks;
};

// Scale buffer of `rows` rows: it ends with the last row's last block (to a whole dword), so the
// 16-byte copy at a row's end reads nothing behind the operand.
__device__ __forceinline__ rsrc_t scale_rsrc(const uint8_t* first, int64_t pitch, int rows, int blocks) {
  return make_rsrc(first, rows > 0 ? (uint64_t)((int64_t)(rows - 1) * pitch + ((blocks + 3) & ~3)) : 0);
}

struct Mx4Frags {
  i32x4_t a[8], b[8];
};

// acc += A·Bᵀ over one workgroup tile.  Schedule of the barrier ring; the copies of an even K tile
// bring the scales of its pair along, and k-step 1 reads the next tile's scales next to its first
// fragments.  Copies in flight behind the awaited tile: T·(S-2) code atoms and, as S is even, the
// scales of (S-2)/2 pairs.
template <class C, int S>
__device__ __forceinline__ void mx4_ring(f32x4_t (&acc)[C::T::FN][C::T::FM], uint8_t* smem, const Mx4Box& box,
                                         int wave, int lane) {
  using T = typename C::T;
  constexpr int FM = T::FM, AT = T::AtomsA, BT = T::AtomsB, A = T::Atoms, P = T::Products, R = T::Reads;
  constexpr int SA = C::ScaleAtoms;
  const int ktiles = box.blocks > 0 ? (box.blocks + 7) / 8 : 1;
  const int g = lane >> 4;

  // Codes: atom slot p of a row holds block 2(p%4) + p/4.
  LaneChunk la[AT], lb[BT];
  auto code_lanes = [&](LaneChunk& lc, int row, uint32_t pitch, int lines) __attribute__((always_inline)) {
    const LaneChunk s = lane_chunk<kSwizzle128B2Row>(row, lane, 0);
    const int block = 2 * (s.chunk & 3) + (s.chunk >> 2);
    lc.chunk = block;
    lc.offset = (uint32_t)(row + (lane >> 3)) * pitch + (uint32_t)block * 16u;
    mask_row(lc, row + (lane >> 3), lines);
  };
#pragma unroll
  for (int i = 0; i < AT; ++i) code_lanes(la[i], 8 * (AT * wave + i), box.pitch_a, box.rows_a);
#pragma unroll
  for (int i = 0; i < BT; ++i) code_lanes(lb[i], 8 * (BT * wave + i), box.pitch_b, box.rows_b);
  // Scales: row `line` of the BM + BN scale rows (A's, then B's), 16 bytes each.
  uint32_t ls[SA];
  const int line0 = 64 * SA * wave;  // this wave's first scale row, uniform: all A's or all B's
  const bool scales_a = line0 < C::RowsA, scales_none = line0 >= C::Rows;
  const uint32_t pitch_s = scales_a ? box.pitch_as : box.pitch_bs;
#pragma unroll
  for (int i = 0; i < SA; ++i) {
    const int row = line0 - (scales_a ? 0 : C::RowsA) + 64 * i + lane;
    ls[i] = scales_none || row >= (scales_a ? min(box.rows_a, T::BM) : box.rows_b) ? kOobOffset : (uint32_t)row * pitch_s;
  }
  const rsrc_t rs0 = scales_a ? box.ras : box.rbs;

  const uint32_t smem_addr = lds_addr_of(smem);
  const uint32_t scale_addr = smem_addr + S * T::StageBytes;
  struct Copy {
    rsrc_t ra, rb, rs;
    uint32_t lds_a, lds_b, lds_s;
    int valid;
    bool live_s;
  };
  auto make_copy = [&](int kt, int stage) __attribute__((always_inline)) {
    Copy c;
    const uint64_t off = (uint64_t)kt * 128u;
    c.ra = rsrc_advance(box.ra, off);
    c.rb = rsrc_advance(box.rb, off);
    c.valid = box.blocks - kt * 8;
    c.lds_a = smem_addr + stage * T::StageBytes + AT * wave * 1024;
    c.lds_b = smem_addr + stage * T::StageBytes + T::ABytes + BT * wave * 1024;
    const int pair = kt >> 1;
    c.rs = rsrc_advance(rs0, (uint64_t)pair * 16u);
    c.rs.z = max(rs0.z - pair * 16, 0);
    c.live_s = pair * 16 < box.blocks;
    c.lds_s = scale_addr + (scales_none ? C::Buffers * C::ScaleBytes + (wave & 1) * 1024
                                        : (pair & (C::Buffers - 1)) * C::ScaleBytes + line0 * 16);
    return c;
  };
  auto atom = [&](const Copy& c, int j, auto interior) __attribute__((always_inline)) {
    constexpr bool in = decltype(interior)::value;
    if (j < AT) {
      issue_atom_if(c.ra, c.lds_a, j * 1024, la[j].offset, in || la[j & 1].chunk < c.valid);
    } else if (j < A) {
      const int i = j - AT;
      issue_atom_if(c.rb, c.lds_b, i * 1024, lb[i].offset, in || lb[i & 1].chunk < c.valid);
    } else {
      issue_atom_if(c.rs, c.lds_s, (j - A) * 1024, ls[j - A], in || c.live_s);
    }
  };

  const int wm = wave >> 1, wn = wave & 1;
  const FragAddr<T> fa = make_frag_addr<T>(wm, wn, lane);
  auto read = [&](Mx4Frags& f, const uint8_t* s, int kk, int i) __attribute__((always_inline)) {
    if (i < FM) f.a[i] = *(const i32x4_t*)(s + fa.a_lane + i * 2048 + fa.a_col[kk]);
    else f.b[i - FM] = *(const i32x4_t*)(s + T::ABytes + fa.b_lane + (i - FM) * 2048 + fa.b_col[kk]);
  };
  // Scale bytes of fragment i for K tile kt: blocks 2g and 2g+1 of the row.
  const uint8_t* const scales = smem + S * T::StageBytes;
  const int sa_lane = (wm * T::TM + (lane & 15)) * 16 + 2 * g, sb_lane = (C::RowsA + wn * T::TN + (lane & 15)) * 16 + 2 * g;
  auto read_scale = [&](uint32_t (&s)[R], int kt, int i) __attribute__((always_inline)) {
    const uint8_t* buf = scales + ((kt >> 1) & (C::Buffers - 1)) * C::ScaleBytes + (kt & 1) * 8;
    s[i] = *(const uint16_t*)(buf + (i < FM ? sa_lane + i * 256 : sb_lane + (i - FM) * 256));
  };
  // Zero the bytes of blocks past the end.  The empty statement keeps the masking next to the
  // reads: products written as assembly must not follow a vector instruction that writes their
  // operand directly.
  auto mask_scales = [&](uint32_t (&s)[R], int kt) __attribute__((always_inline)) {
    const int left = box.blocks - kt * 8 - 2 * g;
    const uint32_t keep = left >= 2 ? 0xFFFFu : left == 1 ? 0xFFu : 0u;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      s[i] &= keep;
      asm volatile("" : "+v"(s[i]));
    }
  };

  // KK: which k-step the products are; the fragments of the other are read meanwhile.
  auto step = [&](const Mx4Frags& cur, Mx4Frags& nxt, const uint32_t (&s)[R], uint32_t (&s_nxt)[R], const uint8_t* from,
                  auto kk, const Copy& c, auto scale_copy, int next_kt, auto interior) __attribute__((always_inline)) {
    constexpr int KK = decltype(kk)::value;
    constexpr int NA = KK == 1 ? A + (decltype(scale_copy)::value ? SA : 0) : 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
#pragma unroll
      for (int r = (i * R + P - 1) / P; r < ((i + 1) * R + P - 1) / P; ++r) {
        read(nxt, from, 1 - KK, r);
        if (KK == 1) read_scale(s_nxt, next_kt, r);
      }
      if (NA > 0) {
        constexpr int H = P / (2 * (NA > 0 ? NA : 1));
        if (i >= H) {
#pragma unroll
          for (int j = ((i - H) * NA + P - 1) / P; j < ((i + 1 - H) * NA + P - 1) / P; ++j) atom(c, j, interior);
        }
      }
      const int fn = i / FM, fm = (fn & 1) ? FM - 1 - i % FM : i % FM;
      mfma_mx4<T::AsmMfma, KK>(acc[fn][fm], cur.b[fn], cur.a[fm], s[FM + fn], s[fm]);
    }
    if (NA > 0) {
      constexpr int H = P / (2 * (NA > 0 ? NA : 1));
#pragma unroll
      for (int j = ((P - H) * NA + P - 1) / P; j < NA; ++j) atom(c, j, interior);
    }
    if (KK == 1 && !decltype(interior)::value) mask_scales(s_nxt, next_kt);
  };

  Mx4Frags f0, f1;
  uint32_t s0[R], s1[R];
#pragma unroll
  for (int t = 0; t < S; ++t) {
    const Copy c = make_copy(t, t);
    if (t % 2 == 0) {
#pragma unroll
      for (int j = A; j < A + SA; ++j) atom(c, j, std::false_type{});
    }
#pragma unroll
    for (int j = 0; j < A; ++j) atom(c, j, std::false_type{});
  }
  stage_barrier<A*(S - 1) + SA*(S / 2 - 1)>();  // tile 0 and its pair's scales landed
#pragma unroll
  for (int r = 0; r < R; ++r) {
    read(f0, smem, 0, r);
    read_scale(s0, 0, r);
  }
  mask_scales(s0, 0);
  typedef std::integral_constant<int, 0> K0;
  typedef std::integral_constant<int, 1> K1;
  auto tile = [&](int kt, auto stage, auto interior) __attribute__((always_inline)) {
    constexpr int cur = decltype(stage)::value, nxt = cur + 1 == S ? 0 : cur + 1;
    typedef std::integral_constant<bool, cur % 2 == 0> Even;
    uint32_t (&s)[R] = cur % 2 == 0 ? s0 : s1;
    uint32_t (&sn)[R] = cur % 2 == 0 ? s1 : s0;
    step(f0, f1, s, sn, smem + cur * T::StageBytes, K0{}, Copy{}, Even{}, kt + 1, interior);
    stage_barrier<A*(S - 2) + SA*(S / 2 - 1)>();  // tile kt+1 (and its scales) landed, stage `cur` free
    step(f1, f0, s, sn, smem + nxt * T::StageBytes, K1{}, make_copy(kt + S, cur), Even{}, kt + 1, interior);
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

// C = alpha·A·Bᵀ + beta·C, or with offsets the same for the rows of each group with its own B.
template <int BM, int BN, int S, int OUT, int SCALED>
__global__ void __launch_bounds__(kThreads, (Mx4Cfg<BM, BN, S>::MinBlocks)) gemm_mx4_kernel(Mx4GemmParams p) {
  using C = Mx4Cfg<BM, BN, S>;
  using T = typename C::T;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LdsBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RaggedTile t;
  if (p.g.offsets) {
    if (!ragged_tile<BM>(p.g.offsets, p.g.groups, p.g.rows, p.g.tiles_n, p.g.group_m, blockIdx.x, t)) return;
  } else {
    int tm;
    map_tile(blockIdx.x, gridDim.x, p.g.tiles_m, p.g.tiles_n, p.g.group_m, tm, t.tn);
    t.group = 0;
    t.row0 = tm * BM;
    t.rows = p.g.rows - t.row0;
  }
  const int n0 = t.tn * BN;
  Mx4Box b;
  b.blocks = p.g.K / 32;
  b.rows_a = t.rows;
  b.rows_b = p.g.N - n0;
  b.pitch_a = (uint32_t)p.g.lda;
  b.pitch_b = (uint32_t)p.g.ldb;
  b.pitch_as = (uint32_t)p.ld_as;
  b.pitch_bs = (uint32_t)p.ld_bs;
  b.ra = make_rsrc(p.g.A + (int64_t)t.row0 * p.g.lda, 0x7FFFFFFFull);
  b.rb = make_rsrc(p.g.B + (int64_t)t.group * p.g.stride_b + (int64_t)n0 * p.g.ldb, 0x7FFFFFFFull);
  b.ras = scale_rsrc(p.As + (int64_t)t.row0 * p.ld_as, p.ld_as, min(b.rows_a, BM), b.blocks);
  b.rbs = scale_rsrc(p.Bs + (int64_t)t.group * p.stride_bs + (int64_t)n0 * p.ld_bs, p.ld_bs, min(b.rows_b, BN), b.blocks);
  f32x4_t acc[T::FN][T::FM];
  zero_acc<T>(acc);
  mx4_ring<C, S>(acc, smem, b, wave, lane);
  const GemmParams q = store_params(p.g.C, p.g.ldc, t.row0 + t.rows, p.g.N, p.g.vec_store, p.g.alpha, p.g.beta);
  store_tile<T, OUT, SCALED>(acc, smem + wave * (T::RingBytes / 4), q, t.row0 + (wave >> 1) * T::TM,
                             n0 + (wave & 1) * T::TN, lane);
}

}  // namespace tbg
