// Which kernel and tile the ragged and the 4-bit products take, and how many workgroups that makes.
// Host arithmetic only: the C ABI chooses here before it enqueues anything, so a call with more
// workgroups than one launch takes is refused with its operands and workspace as they were.
#pragma once
#include <math.h>
#include <stdint.h>

namespace tbg {

// Workgroups one launch takes: it counts its threads (256 a workgroup) in 32 bits.
constexpr int64_t kMaxGrid = (1 << 24) - 1;

// Whether one launch of a chunk a thread, 256 to a workgroup, takes both repacks of a call (0 chunks:
// there is none) and numbers each one's chunks in 32 bits.
inline bool one_pack_launch(uint64_t chunks0, uint64_t chunks1) {
  const uint64_t most = (uint64_t)kMaxGrid * 256;
  return chunks0 <= most && chunks1 <= most && (chunks0 + 255) / 256 + (chunks1 + 255) / 256 <= (uint64_t)kMaxGrid;
}

// Upper bound of the tiles of height bm over any split of `rows` rows into `groups` groups.
inline int64_t ragged_tiles_bound(int64_t rows, int64_t groups, int64_t bm) {
  const int64_t g = groups < rows ? groups : rows;
  return (rows + g * (bm - 1)) / bm;
}

struct TileChoice {
  bool few;            // the kernel of few rows (16×16), else a ring
  bool walks;          // each workgroup takes one tile after another
  int bm, bn, stages;
  int64_t tiles_m, tiles_n;  // tiles_m bounds the tile rows of all groups (weight gradient: one group's)
  int64_t per_xcd;     // weight gradient: consecutive tiles of a group per XCD
  bool by_rows;        // weight gradient: the groups run in the order of their rows
  int64_t grid;        // workgroups
  // One launch takes them, and the tiles are numbered in 32 bits.
  bool fits() const { return grid <= kMaxGrid && (!walks || tiles_m <= (INT32_MAX - 8) / tiles_n); }
};

inline int64_t tile_count(int64_t n, int64_t b) { return (n + b - 1) / b; }
// The XCD order deals ids in eighths: the grid is rounded up so that every eighth fits.
inline int64_t whole_eighths(int64_t n) { return (n + 7) / 8 * 8; }

// ---- the choice of a tile -------------------------------------------------------------------
// A round of tiles, one on every slot the chip has for them, takes about `fixed` µs to start and to
// store and `per` µs for each K tile (128 bytes of a row); the smaller tiles share a CU, and a
// round that does not fill costs them only `part` of one, since the next tiles start as others end.
// The figures are fitted to every tile's time on thousands of shapes (MI355X, 4 to 64 groups of 70 to
// 2048 rows on average, N of 256 to 14336, K of 256 to 8192; the 4-bit ones also dense): the tile
// chosen takes 1.0 % (16-bit rows), 1.4 % (weight gradient) and 0.9 % (4 bits) longer than the
// best one on average.  Outside that range (one to three groups, 8 to 69 rows a group, widths off 64;
// 249 shapes, either layout of B) it takes up to 1.7 % longer on average, 23 % at worst, but the times
// are no prediction there (31 groups of 258 rows, K×N at a pitch of 4000 bytes, K = 1001: 71 µs for 50).
struct TileTime {
  int b, per_cu;
  double fixed, per, part;
};
const TileTime kTilesRows[] = {{256, 1, 9.2, 0.98, 1.0}, {128, 2, 3.65, 0.97, 0.13}, {64, 3, 2.3, 0.61, 0.58}};
const TileTime kTilesGrad[] = {{256, 1, 14.2, 0.88, 1.0}, {128, 2, 4.1, 1.05, 0.1}, {64, 3, 4.6, 0.52, 0.45}};
const TileTime kTiles4[] = {{256, 1, 10.5, 0.98, 1.0}, {128, 2, 4.1, 1.05, 0.135}, {64, 2, 4.2, 0.42, 0.63}};

inline double tile_time(const TileTime& t, double tiles, double ktiles, int cus) {
  double rounds = tiles / ((double)t.per_cu * cus);
  if (rounds <= 1) rounds = 1;
  else if (t.part == 1.0) rounds = ceil(rounds);
  else rounds += t.part;
  return rounds * (t.fixed + t.per * ktiles);
}

// The tile for `groups` groups that share `rows` rows.  How the rows split is not known here:
// groups of the average size are assumed, each ending half way into its last tile.  Up to 64 (128)
// rows a group the product is bound by the bytes of B, which a tile of 64 (128) rows reads as
// well with less of it masked (64 groups, N = K = 2048, 16 bits: 64 rows 130 µs with 64-row tiles,
// 153 with 128; 128 rows 159 µs with 128, 182 with 256).
inline int choose_rows_tile(const TileTime (&t)[3], double groups, double rows, int64_t N, double ktiles, int cus) {
  const double average = rows / groups;
  int best = 64;
  double best_time = 0;
  for (const TileTime& c : t) {
    if ((c.b > 64 && average <= 64) || (c.b > 128 && average <= 128)) continue;
    const double per = groups > 1 ? average / c.b + 0.5 : ceil(average / c.b);
    const double tiles = groups * (per > 1 ? per : 1) * (double)tile_count(N, c.b);
    const double time = tile_time(c, tiles, ktiles, cus);
    if (best_time == 0 || time < best_time) {
      best = c.b;
      best_time = time;
    }
  }
  return best;
}

// Tiles of 64 columns that groups of up to 64 rows make.
inline double narrow_tiles(double groups, int64_t N) { return groups * (double)tile_count(N, 64); }

// Whether the kernel of few rows (gemm_rows.hpp, with both sides' figures) takes a product.
inline bool takes_few_rows(double groups, double rows, int64_t N, int cus) {
  return rows <= 16 * groups && narrow_tiles(groups, N) < 0.75 * cus;
}

// The workgroups of a product over `rows` rows: tiles of bm × bn, ragged or dense (groups == 0).
inline void set_row_tiles(TileChoice& c, int64_t groups, int64_t rows, int64_t N) {
  c.tiles_m = groups > 0 ? ragged_tiles_bound(rows, groups, c.bm) : tile_count(rows, c.bm);
  c.tiles_n = tile_count(N, c.bn);
  c.grid = c.tiles_m * c.tiles_n;
  if (groups > 0) c.grid = whole_eighths(c.grid);
}

// 16-bit rows times B_e (at least one of each); nk: B_e stored N×K.
inline TileChoice choose_grouped(int64_t groups, int64_t M, int64_t N, int64_t K, bool nk, int cus) {
  TileChoice c{};
  const double active = (double)(groups < M ? groups : M);
  c.few = nk && takes_few_rows(active, (double)M, N, cus);
  c.bm = c.bn = c.few ? 16 : choose_rows_tile(kTilesRows, active, (double)M, N, ceil((double)K / 64), cus);
  set_row_tiles(c, groups, M, N);
  return c;
}

// The weight gradient: every group has the same tiles, its rows are the sum's terms.
inline TileChoice choose_wgrad(int64_t groups, int64_t M, int64_t P, int64_t Q, int cus) {
  TileChoice c{};
  double best = 0;
  for (const TileTime& t : kTilesGrad) {
    const double tiles = (double)groups * (double)tile_count(P, t.b) * (double)tile_count(Q, t.b);
    const double time = tile_time(t, tiles, ceil((double)M / (double)groups / 64), cus);
    if (!c.bm || time < best) {
      c.bm = c.bn = t.b;
      best = time;
    }
  }
  c.tiles_m = tile_count(P, c.bm);
  c.tiles_n = tile_count(Q, c.bn);
  const int64_t per_group = c.tiles_m * c.tiles_n;
  c.per_xcd = per_group > 8 ? per_group / 8 : 1;
  const int64_t round = 8 * c.per_xcd;
  c.grid = tile_count(per_group * groups, round) * round;
  // The longest groups first (up to 64, a lane each): every workgroup ranks them itself, 0.3 µs for 4
  // groups, 0.8 for 16 and 2.7 for 64, and the last to start are the short ones.  By number and by rows,
  // µs: from 1024 rows a group 8 of 2048, 4096×2048 263.5, 250.2; 32 of 1024, 1024×1024 120.7, 106.8; 32
  // of 1024, 4096×4096 1130, 1181 (the worst); at 512 rows 16 groups, 256×256 12.1, 12.9; at 256 rows 64
  // groups, 1024×1024 76.4, 98.8.
  c.by_rows = groups > 1 && groups <= 64 && M >= 1024 * groups;
  return c;
}

// 4-bit rows, dense (groups == 0) or ragged.
inline TileChoice choose_mx4(int64_t groups, int64_t M, int64_t N, int64_t K, int cus) {
  TileChoice c{};
  const bool ragged = groups > 0;
  const double active = ragged ? (double)(groups < M ? groups : M) : 1.0;
  c.few = takes_few_rows(active, (double)M, N, cus) && (ragged || M <= 16);
  // Up to 32 rows a group: 32-row tiles, which copy half as many masked rows of A as 64-row ones (40
  // groups of one or two rows, N = 4096, K = 2048: 34.7 against 40.0 µs).
  c.stages = 2;
  if (c.few) {
    c.bm = c.bn = 16;
    c.stages = 1;
  } else if ((double)M <= 32 * active) {
    c.bm = 32;
    c.bn = 64;
  } else {
    c.bm = c.bn = choose_rows_tile(kTiles4, active, (double)M, N, ceil((double)K / 256), cus);
  }
  // The tiles of 64 columns have rings of two and of four stages.  Two take less LDS, so more workgroups
  // share a CU and hide each other's copies; up to 1.5 workgroups a CU there are no others, and over a
  // long K the depth pays whatever their number.  2 against 4 stages in µs, 20 rows, by workgroups a CU:
  //   K = 2048   1: 7.6, 6.7    1.5: 8.7, 8.8     2: 9.4, 9.6     4: 14.3, 15.6   10: 38.0, 41.6
  //   K = 4096   1: 11.6, 9.6   1.5: 12.4, 12.3   2: 13.9, 14.2   4: 29.9, 31.1   10: 69.9, 69.5
  //   K = 8192   1: 18.6, 14.3  1.5: 26.6, 22.8   2: 37.1, 33.2   4: 68.9, 61.1   10: 132, 122
  // (60 rows, and 16 groups of 10 or 50, alike; between K = 4096 and 8192 either may lead by a tenth)
  if (c.bn == 64) {
    const double tall = (double)M / active / c.bm, workgroups = narrow_tiles(active, N) * (tall > 1 ? tall : 1);
    if (workgroups <= 1.5 * cus || K >= 8192) c.stages = 4;
  }
  c.walks = c.bm == 256;
  set_row_tiles(c, groups, M, N);
  if (c.walks) {
    const int64_t walkers = cus >= 8 ? cus / 8 * 8 : 8, tiles = whole_eighths(c.grid);
    c.grid = tiles < walkers ? tiles : walkers;
  }
  return c;
}

// Rows times weights in 4-bit codes (gemm_w4.hpp), dense (groups == 0) or ragged.  The panel kernel (128 columns
// and 16, 32 or 64 rows a workgroup, A in LDS) needs a workgroup for every CU; below that the waves of a workgroup of
// 16 rows split K, over as many columns (64, 32, 16) as leave most of the CUs a workgroup.  One limit serves every
// group: at 32 × 14336 it leaves 21.0 for 19.4 µs in groups of 128, where the panel would take 28.6 for 23.0 in groups
// of 32 with zeros.  µs, K = 4096, group 128, bf16, by rows × columns; split K with 16, 32, 64 columns, then panels
// of 16, 32, 64 rows:
//     1 ×  4096    5.1   6.1   8.3   17.9  23.0  34.1        64 ×  4096   23.6  16.3  12.4   19.0  24.3  36.2
//     1 × 14336   12.5  10.6  10.0   18.7  23.8  35.0        64 ×  8192   44.0  28.5  21.2   19.5  24.4  36.1
//    16 × 14336   23.4  16.4  12.8   19.0  23.9  35.3        64 × 14336   75.9  47.8  37.6   26.1  24.6  36.0
//    32 × 14336   39.5  28.5  21.0   19.4  24.4  36.0       256 ×  4096   84.2  52.2  36.9   25.8  24.6  35.7
//   (group 32,    40.8  29.6  23.0   28.6  31.8  47.1       256 × 14336    281   172   118   79.2  59.6  54.9
//    with zeros)
// 64 groups, 64 rows (8 of 64 experts for 8 tokens), N = 4096, K = 2048: 64.6, 51.0, 47.9; 40.5, 49.2, 73.7;
// 2008 rows, N = 2048, K = 4096, group 64 with zeros: 383, 240, 176; 140, 127, 160.
inline TileChoice choose_w4(int64_t groups, int64_t M, int64_t N, int cus) {
  TileChoice c{};
  const double active = groups > 0 ? (double)(groups < M ? groups : M) : 1.0, rows = (double)M / active;
  auto tiles = [&](int bm, int bn) {  // ragged groups of the average size, each ending half way into its last tile
    const double per = groups > 1 ? rows / bm + 0.5 : ceil(rows / bm);
    return active * (per > 1 ? per : 1) * (double)tile_count(N, bn);
  };
  const double most = 0.75 * cus;
  c.few = tiles(16, 128) < cus;
  if (c.few) {
    c.bm = 16;
    c.bn = tiles(16, 64) >= most ? 64 : tiles(16, 32) >= most ? 32 : 16;
  } else {
    c.bm = rows > 32 && tiles(64, 128) >= most ? 64 : rows > 16 && tiles(32, 128) >= most ? 32 : 16;
    c.bn = 128;
  }
  set_row_tiles(c, groups, M, N);
  c.grid = whole_eighths(c.grid);
  return c;
}

}  // namespace tbg
