// Products of microscaled 4-bit operands (E2M1 codes, one E8M0 scale per 32 values along K) on
// gfx950's scaled 16×16×128 matrix instruction: C = A·Bᵀ, A M×K, B stored N×K, dense or with the
// rows in ragged groups and one B per group; fp32 accumulation.
//
// A K tile is 256 values, 128 bytes of codes per row: in bytes the ring, its copy atoms, LDS
// layout, fragment reads and epilogue are those of the 16-bit kernels (gemm_ring.hpp), and a
// k-step of 64 bytes is one 16×16×128 product per fragment pair.  Two things are new.
//  * Scales.  A K tile has 8 scale bytes per row.  They reach LDS as the 32 bytes of four K tiles (a
//    quad), 32 rows per copy atom, two buffers of 32 bytes a row (256×256: 4 atoms per wave and
//    quad next to 64 atoms of codes; the ring and the buffers are the whole 160 KiB of LDS).  Copies
//    of 16 bytes per row, for two K tiles, took as many atoms but twice the cache lines (8192³
//    241 against 234 µs, 2048³ 11.4 against 11.0).  The two 16-byte halves of rows 8..15 of 16 are
//    exchanged in LDS, so that a fragment's 16 rows, 32 bytes apart, are read from distinct banks.  The
//    instruction takes a lane's scale from one byte of a register, chosen by an immediate.
//  * Placement.  Lane l multiplies row l%16 and, in k-step kk, block 2·pair(l/16)+kk of the tile
//    (not 4kk + l/16): its two k-steps then need two neighbouring scale bytes, one 16-bit LDS read
//    per fragment and K tile.  The sum runs over the tile's blocks in another order, the same for A
//    and B.  pair = 0, 3, 1, 2: the 16-byte read serves lanes 0-3, 12-15, 20-27 (and the like)
//    together, whose rows' 2-row swizzle keeps two columns apart in the banks only if their numbers
//    differ by an exclusive or of 1, 6 or 7; 2·pair of neighbouring lane groups differ by 6.  The
//    copies stay in the rows' own order.
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
  static_assert(S == 2 || S == 4, "stages divide the four K tiles of a quad");
  static constexpr int Rows = BM + BN;
  static constexpr int QuadBytes = Rows * 32;              // scales of four K tiles
  static constexpr int ScaleAtoms = (Rows / 32 + 3) / 4;   // per wave and quad (32×64: the last wave has none)
  static constexpr int RowsWave = 32 * ScaleAtoms;         // each wave's are all A's or all B's
  static constexpr int LdsBytes = S * T::StageBytes + 2 * QuadBytes;
  // Workgroups per CU, as many as LDS holds (it is given out in pieces of 1280 bytes).
  static constexpr int MinBlocks = 128 / ((LdsBytes + 1279) / 1280);
  static_assert(BM % RowsWave == 0, "whole waves of A's rows");
  static_assert(LdsBytes <= 160 * 1024, "the ring must fit in LDS");
  static_assert((S - 1) * T::Atoms + ScaleAtoms <= 63, "copies in flight must fit the vmcnt counter");
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

// The copies of one workgroup tile: the wave's lanes of every atom, and the atoms of a K tile.
template <class C, int S>
struct Mx4Copies {
  using T = typename C::T;
  static constexpr int AT = T::AtomsA, BT = T::AtomsB, A = T::Atoms, SA = C::ScaleAtoms;
  struct Copy {
    rsrc_t ra, rb, rs;
    uint32_t lds_a, lds_b, lds_s;
    int valid;
    bool live_s;
  };
  Mx4Box box;
  LaneChunk la[AT], lb[BT];
  uint32_t ls[SA];
  rsrc_t rs0;
  uint32_t ring, scales;  // LDS addresses: the ring; this wave's first scale row
  int wave;

  __device__ __forceinline__ void set(const Mx4Box& b, const uint8_t* smem, int wave_, int lane) {
    box = b;
    wave = wave_;
#pragma unroll
    for (int i = 0; i < AT; ++i) {
      la[i] = lane_chunk<kSwizzle128B2Row>(8 * (AT * wave + i), lane, box.pitch_a);
      mask_row(la[i], 8 * (AT * wave + i) + (lane >> 3), box.rows_a);
    }
#pragma unroll
    for (int i = 0; i < BT; ++i) {
      lb[i] = lane_chunk<kSwizzle128B2Row>(8 * (BT * wave + i), lane, box.pitch_b);
      mask_row(lb[i], 8 * (BT * wave + i) + (lane >> 3), box.rows_b);
    }
    // Scales: two lanes per row, the halves exchanged in rows 8..15 of 16.
    const int line0 = C::RowsWave * wave;  // this wave's first scale row: all A's or all B's
    const bool of_a = line0 < T::BM;
    const uint32_t pitch_s = of_a ? box.pitch_as : box.pitch_bs;
#pragma unroll
    for (int i = 0; i < SA; ++i) {
      const int row = line0 - (of_a ? 0 : T::BM) + 32 * i + (lane >> 1);
      const uint32_t half = (uint32_t)((lane & 1) ^ ((lane >> 4) & 1));
      ls[i] = row >= (of_a ? box.rows_a : box.rows_b) ? kOobOffset : (uint32_t)row * pitch_s + half * 16u;
    }
    rs0 = of_a ? box.ras : box.rbs;
    ring = lds_addr_of(smem);
    scales = ring + S * T::StageBytes + line0 * 32;
  }

  __device__ __forceinline__ Copy tile(int kt, int stage) const {
    Copy c;
    const uint64_t off = (uint64_t)kt * 128u;
    c.ra = rsrc_advance(box.ra, off);
    c.rb = rsrc_advance(box.rb, off);
    c.valid = box.blocks - kt * 8;
    c.lds_a = ring + stage * T::StageBytes + AT * wave * 1024;
    c.lds_b = ring + stage * T::StageBytes + T::ABytes + BT * wave * 1024;
    return c;
  }
  __device__ __forceinline__ void quad(Copy& c, int q) const {
    c.rs = rsrc_advance(rs0, (uint64_t)q * 32u);
    c.rs.z = max(rs0.z - q * 32, 0);
    c.live_s = q * 32 < box.blocks;
    c.lds_s = scales + (q & 1) * C::QuadBytes;
  }
  // atoms 0..A-1: codes; A + i: scale atom i
  template <bool INTERIOR>
  __device__ __forceinline__ void atom(const Copy& c, int j) const {
    if (j < AT) {
      issue_atom_if(c.ra, c.lds_a, j * 1024, la[j].offset, INTERIOR || la[j & 1].chunk < c.valid);
    } else if (j < A) {
      const int i = j - AT;
      issue_atom_if(c.rb, c.lds_b, i * 1024, lb[i].offset, INTERIOR || lb[i & 1].chunk < c.valid);
    } else if (C::RowsWave * 4 == C::Rows || C::RowsWave * wave < C::Rows) {
      issue_atom_if(c.rs, c.lds_s, (j - A) * 1024, ls[j - A], INTERIOR || c.live_s);
    }
  }
  // The first quad's scales (into the first buffer) and the K tiles FROM .. TO-1 of the first S.
  template <int FROM, int TO>
  __device__ __forceinline__ void start() const {
    if (FROM == 0) {
      Copy c = tile(0, 0);
      quad(c, 0);
#pragma unroll
      for (int j = A; j < A + SA; ++j) atom<false>(c, j);
    }
#pragma unroll
    for (int t = FROM; t < TO; ++t) {
      const Copy c = tile(t, t);
#pragma unroll
      for (int j = 0; j < A; ++j) atom<false>(c, j);
    }
  }
};

// acc += A·Bᵀ over one workgroup tile whose first copies are on their way (start()), and nothing
// newer but what WAIT counts: the first barrier lets WAIT of the wave's memory operations be in
// flight.  Schedule of the barrier ring, four K tiles (a quad) per iteration; the first two tiles of
// a quad bring the next quad's scales along, half each, and k-step 1 reads the next tile's scales
// next to its first fragments.  A barrier lets the code atoms of the S-2 tiles behind the awaited
// one be in flight; scale atoms among them (a wave's own number) only make it wait for a few more
// copies than it needs.
template <class C, int S, int WAIT>
__device__ __forceinline__ void mx4_ring(f32x4_t (&acc)[C::T::FN][C::T::FM], const uint8_t* smem,
                                         const Mx4Copies<C, S>& copies, int wave, int lane) {
  using T = typename C::T;
  using Copy = typename Mx4Copies<C, S>::Copy;
  constexpr int FM = T::FM, A = T::Atoms, P = T::Products, R = T::Reads;
  constexpr int SA = C::ScaleAtoms;
  const int blocks = copies.box.blocks;
  const int ktiles = blocks > 0 ? (blocks + 7) / 8 : 1;
  const int pair = (0x2130 >> (4 * (lane >> 4))) & 15;  // 0, 3, 1, 2 (lane groups 0..3)
  const int wm = wave >> 1, wn = wave & 1;
  // Fragment rows start at multiples of 16, so the swizzle is the lane's own.
  const uint32_t lane_row = (uint32_t)(lane & 15) * 128u, swz = (lane >> 1) & 7;
  const uint32_t col[2] = {lane_row + ((2 * pair) ^ swz) * 16u, lane_row + ((2 * pair + 1) ^ swz) * 16u};
  auto read = [&](Mx4Frags& f, const uint8_t* s, int kk, int i) __attribute__((always_inline)) {
    if (i < FM) f.a[i] = *(const i32x4_t*)(s + wm * T::TM * 128 + i * 2048 + col[kk]);
    else f.b[i - FM] = *(const i32x4_t*)(s + T::ABytes + wn * T::TN * 128 + (i - FM) * 2048 + col[kk]);
  };
  // Scale bytes of fragment i for K tile `quad`, QT (0..3): blocks 2·pair and 2·pair+1.
  const uint8_t* const scales = smem + S * T::StageBytes;
  const int lane_s = (lane & 15) * 32 + 2 * pair, swap = (lane >> 3) & 1;
  auto read_scale = [&](uint32_t (&s)[R], int quad, auto qt, int i) __attribute__((always_inline)) {
    constexpr int QT = decltype(qt)::value;
    const uint8_t* buf = scales + (quad & 1) * C::QuadBytes + lane_s + ((QT >> 1) ^ swap) * 16 + (QT & 1) * 8;
    s[i] = *(const uint16_t*)(buf + (i < FM ? wm * T::TM * 32 + i * 512 : (T::BM + wn * T::TN) * 32 + (i - FM) * 512));
  };
  // Zero the bytes of blocks past the end.  A product may read a register two wait states after a vector
  // instruction wrote it, which the compiler does not see to for products written as assembly: the
  // empty statements, the wait and those products are all volatile, so they stay in this order.
  auto mask_scales = [&](uint32_t (&s)[R], int kt) __attribute__((always_inline)) {
    const int left = blocks - kt * 8 - 2 * pair;
    const uint32_t keep = left >= 2 ? 0xFFFFu : left == 1 ? 0xFFu : 0u;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      s[i] &= keep;
      asm volatile("" : "+v"(s[i]));
    }
    if (T::AsmMfma) asm volatile("s_nop 1");
  };

  // One k-step: KK says which blocks the products take; the fragments of the other k-step are
  // read meanwhile, and with KK = 1 the scales of K tile `next` (QN of its quad), the code atoms
  // of `c` and its scale atoms S0 .. S0+NS-1 go out.
  auto step = [&](const Mx4Frags& cur, Mx4Frags& nxt, const uint32_t (&s)[R], uint32_t (&s_nxt)[R], const uint8_t* from,
                  auto kk, const Copy& c, auto s0, auto ns, int next, auto qn,
                  auto interior) __attribute__((always_inline)) {
    constexpr int KK = decltype(kk)::value, S0 = decltype(s0)::value;
    constexpr int NA = KK == 1 ? A + decltype(ns)::value : 0;
    constexpr int H = P / (2 * (NA > 0 ? NA : 1));
    auto go = [&](int j) __attribute__((always_inline)) {
      copies.template atom<decltype(interior)::value>(c, j < A ? j : j + S0);
    };
#pragma unroll
    for (int i = 0; i < P; ++i) {
#pragma unroll
      for (int r = (i * R + P - 1) / P; r < ((i + 1) * R + P - 1) / P; ++r) {
        read(nxt, from, 1 - KK, r);
        if (KK == 1) read_scale(s_nxt, next >> 2, qn, r);
      }
      if (NA > 0 && i >= H) {
#pragma unroll
        for (int j = ((i - H) * NA + P - 1) / P; j < ((i + 1 - H) * NA + P - 1) / P; ++j) go(j);
      }
      const int fn = i / FM, fm = (fn & 1) ? FM - 1 - i % FM : i % FM;
      mfma_mx4<T::AsmMfma, KK>(acc[fn][fm], cur.b[fn], cur.a[fm], s[FM + fn], s[fm]);
    }
    if (NA > 0) {
#pragma unroll
      for (int j = ((P - H) * NA + P - 1) / P; j < NA; ++j) go(j);
    }
    if (KK == 1 && !decltype(interior)::value) mask_scales(s_nxt, next);
  };

  Mx4Frags f0, f1;
  uint32_t s0[R], s1[R];
  stage_barrier<WAIT>();  // the first quad's scales and tile 0 landed
#pragma unroll
  for (int r = 0; r < R; ++r) {
    read(f0, smem, 0, r);
    read_scale(s0, 0, std::integral_constant<int, 0>{}, r);
  }
  mask_scales(s0, 0);
  typedef std::integral_constant<int, 0> K0;
  typedef std::integral_constant<int, 1> K1;
  // K tile kt, the q-th of its quad (kt - q is a multiple of 4), in stage q % S.
  auto tile = [&](int kt, auto q, auto interior) __attribute__((always_inline)) {
    constexpr int Q = decltype(q)::value, cur = Q % S, nxt = (Q + 1) % S;
    // the next quad's scale atoms: the first half (rounded up) with tile 0, the others with tile 1
    constexpr int First = (SA + 1) / 2, S0 = Q == 1 ? First : 0, NS = Q == 0 ? First : Q == 1 ? SA - First : 0;
    typedef std::integral_constant<int, S0> Begin;
    typedef std::integral_constant<int, NS> Count;
    typedef std::integral_constant<int, (Q + 1) % 4> Next;
    uint32_t (&s)[R] = Q % 2 == 0 ? s0 : s1;
    uint32_t (&sn)[R] = Q % 2 == 0 ? s1 : s0;
    step(f0, f1, s, sn, smem + cur * T::StageBytes, K0{}, Copy{}, Begin{}, Count{}, kt + 1, Next{}, interior);
    stage_barrier<A*(S - 2)>();  // tile kt+1 (and its scales) landed, stage `cur` free
    Copy c = copies.tile(kt + S, cur);
    if (NS > 0) copies.quad(c, (kt >> 2) + 1);
    step(f1, f0, s, sn, smem + nxt * T::StageBytes, K1{}, c, Begin{}, Count{}, kt + 1, Next{}, interior);
  };
  int kt = 0;
  for (; kt + 4 + S < ktiles; kt += 4)
    for_stages<4>([&](auto q) __attribute__((always_inline)) { tile(kt + decltype(q)::value, q, std::true_type{}); });
  for (; kt + 4 <= ktiles; kt += 4)
    for_stages<4>([&](auto q) __attribute__((always_inline)) { tile(kt + decltype(q)::value, q, std::false_type{}); });
  for_stages<3>([&](auto q) __attribute__((always_inline)) {
    if (kt + decltype(q)::value < ktiles) tile(kt + decltype(q)::value, q, std::false_type{});
  });
  drain_acc<T>(acc);
  stage_barrier<0>();
}

// The operands of tile t.
template <class T>
__device__ __forceinline__ Mx4Box mx4_box(const Mx4GemmParams& p, const RaggedTile& t) {
  const int n0 = t.tn * T::BN;
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
  b.ras = scale_rsrc(p.As + (int64_t)t.row0 * p.ld_as, p.ld_as, min(b.rows_a, T::BM), b.blocks);
  b.rbs = scale_rsrc(p.Bs + (int64_t)t.group * p.stride_bs + (int64_t)n0 * p.ld_bs, p.ld_bs, min(b.rows_b, T::BN),
                     b.blocks);
  return b;
}

template <class T, int OUT, int SCALED, int PARK>
__device__ __forceinline__ void mx4_store(const f32x4_t (&acc)[T::FN][T::FM], uint8_t* park, const Mx4GemmParams& p,
                                          const RaggedTile& t, int wave, int lane) {
  const GemmParams q = store_params(p.g.C, p.g.ldc, t.row0 + t.rows, p.g.N, p.g.vec_store, p.g.alpha, p.g.beta);
  store_tile<T, OUT, SCALED, PARK>(acc, park, q, t.row0 + (wave >> 1) * T::TM, t.tn * T::BN + (wave & 1) * T::TN, lane);
}

// C = alpha·A·Bᵀ + beta·C, or with offsets the same for the rows of each group with its own B: one
// tile per workgroup.
template <int BM, int BN, int S, int OUT, int SCALED>
__global__ void __launch_bounds__(kThreads, (Mx4Cfg<BM, BN, S>::MinBlocks)) gemm_mx4_kernel(Mx4GemmParams p) {
  using C = Mx4Cfg<BM, BN, S>;
  using T = typename C::T;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LdsBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RaggedTile t;
  if (p.g.offsets) {
    if (!ragged_tile<BM>(p.g, p.g.group_m, blockIdx.x, t)) return;
  } else {
    int tm;
    map_tile(blockIdx.x, gridDim.x, p.g.tiles_m, p.g.tiles_n, p.g.group_m, tm, t.tn);
    t.group = 0;
    t.row0 = tm * BM;
    t.rows = p.g.rows - t.row0;
  }
  Mx4Copies<C, S> copies;
  copies.set(mx4_box<T>(p, t), smem, wave, lane);
  copies.template start<0, S>();
  f32x4_t acc[T::FN][T::FM];
  zero_acc<T>(acc);
  mx4_ring<C, S, T::Atoms*(S - 1)>(acc, smem, copies, wave, lane);
  mx4_store<T, OUT, SCALED, T::RingBytes / 4>(acc, smem + wave * (T::RingBytes / 4), p, t, wave, lane);
}

// The same with a workgroup per CU that walks its XCD's tiles.  A 4-bit tile has a quarter of a
// 16-bit one's K tiles, so what lies between the K loops weighs four times as much (of the 21 µs of
// a tile with K = 2048: 1.0 to find it, 1.9 until its first K tile has landed, 4.4 to store it);
// here the first K tile of the next tile is on its way while a tile is stored, from a park in the
// second scale buffer (4 KiB a wave; the copies in flight go to the ring and the first).  Both first
// K tiles ahead of the stores were 2-3 % slower on operands that come from HBM.  One tile per workgroup
// and this, µs: 8192³ 222.3, 218.7; 4 groups of 2048 rows, N = 8192, K = 2048 101.4, 96.6, 32 of 256
// 133.2, 125.2; 32 groups of 500 rows, N = 4096 101.9, 93.1, and level with B from HBM (107.5).
template <int B, int S, int OUT, int SCALED>
__global__ void __launch_bounds__(kThreads, 1) gemm_mx4_walk_kernel(Mx4GemmParams p) {
  using C = Mx4Cfg<B, B, S>;
  using T = typename C::T;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LdsBytes];
  constexpr int Park = C::QuadBytes / 4;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RaggedPlan plan{};
  if (p.g.offsets) plan = ragged_plan<B>(p.g.offsets, p.g.groups, p.g.rows, p.g.tiles_n);
  else plan.tiles = p.g.tiles_m * p.g.tiles_n;
  int first, count;
  xcd_share(plan.tiles, blockIdx.x, first, count);
  auto find = [&](int i, RaggedTile& t) __attribute__((always_inline)) {
    if (p.g.offsets) {
      ragged_find<B>(plan, p.g.offsets, p.g.groups, p.g.rows, p.g.tiles_n, p.g.group_m, first + i, t);
    } else {
      int tm;
      band_tile(first + i, p.g.tiles_m, p.g.tiles_n, p.g.group_m, tm, t.tn);
      t.group = 0;
      t.row0 = tm * B;
      t.rows = p.g.rows - t.row0;
    }
  };
  int i = blockIdx.x >> 3;
  if (i >= count) return;
  RaggedTile t, next;
  Mx4Copies<C, S> copies;
  find(i, t);
  copies.set(mx4_box<T>(p, t), smem, wave, lane);
  copies.template start<0, 1>();
  for (;;) {
    copies.template start<1, S>();
    i += gridDim.x >> 3;
    const bool more = i < count;
    if (more) find(i, next);
    f32x4_t acc[T::FN][T::FM];
    zero_acc<T>(acc);
    mx4_ring<C, S, T::Atoms*(S - 1)>(acc, smem, copies, wave, lane);
    if (more) {
      copies.set(mx4_box<T>(p, next), smem, wave, lane);
      copies.template start<0, 1>();
    }
    keep_acc<T>(acc);
    mx4_store<T, OUT, SCALED, Park>(acc, smem + S * T::StageBytes + C::QuadBytes + wave * Park, p, t, wave, lane);
    if (!more) return;
    t = next;
  }
}

}  // namespace tbg
