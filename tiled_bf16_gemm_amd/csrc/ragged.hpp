// Ragged groups on the device: which rows belong to a group, and which tile of which group a
// workgroup computes.
//
// Group e holds rows offsets[e] .. offsets[e+1]-1.  The offsets stay in device memory (a router
// writes them there, and a captured graph replays with new ones), so the host only knows the
// number of rows and of groups: it launches as many workgroups as the worst split needs
// (ragged_tiles_bound) and each workgroup finds its tile from the offsets, every wave for itself: a
// lane counts the tiles of its share of the groups, one prefix sum over the lanes places them, and
// the lane whose range holds the workgroup's number answers.  That is one dependent load and ≈30
// vector instructions before the K loop, against a launch of its own (and a table in a workspace)
// for a planning kernel.  Offsets are clamped to the rows that exist and to their running maximum, so
// no value in them takes an access outside the operands, no row has two groups, and there are never
// more tiles than the grid was made for.  The maximum over the lanes before costs a dozen dependent
// instructions and, past 64 groups, a second pass over a lane's offsets: only a wave that
// meets a descending pair takes it (a ballot in front).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"

namespace tbg {

// Rows of group g: begin .. end-1, inside least .. rows whatever the offsets hold (0 <= least <= rows).
__device__ __forceinline__ void group_rows(const int32_t* offsets, int g, int least, int rows, int& begin, int& end) {
  begin = min(max(offsets[g], least), rows);
  end = min(max(offsets[g + 1], begin), rows);
}

// Inclusive prefix sum over the 64 lanes (all active): four shifts inside rows of 16 lanes, then
// the last lane of a row broadcast into the rows after it.
__device__ __forceinline__ int wave_prefix_sum(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);  // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);  // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);  // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast:31 into rows 2 and 3
  return v;
}

// Maximum over the lanes before this one (lane 0: 0) of a value that is not negative; all lanes
// active.
__device__ __forceinline__ int wave_max_before(int v) {
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));  // as wave_prefix_sum
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));
  const int lane = threadIdx.x & 63;
  const int before = __builtin_amdgcn_ds_bpermute(4 * (lane - 1), v);
  return lane > 0 ? before : 0;
}

// Tile `id` of a group's tiles_m × tiles_n: column-major inside bands of tile rows, so that the
// tiles an XCD computes at one time share operand rows in its L2.  The bands are as near to
// `height` rows as equal bands can be (a thin last band would read the whole of B once more).
__device__ __forceinline__ void band_tile(int id, int tiles_m, int tiles_n, int height, int& tm, int& tn) {
  const int bands = max(1, (tiles_m + height / 2) / height);
  const int low = tiles_m / bands, more = tiles_m - low * bands;  // the first `more` bands have low + 1 rows
  const int split = more * (low + 1) * tiles_n;
  const int h = id < split ? low + 1 : low;
  const int rest = id < split ? id : id - split;
  const int band = rest / (h * tiles_n), in = rest - band * h * tiles_n;
  tm = (id < split ? 0 : more * (low + 1)) + band * h + in % h;
  tn = in / h;
}

struct RaggedTile {
  int group;
  int row0;  // first row of the tile
  int rows;  // rows from row0 to the end of the group (may exceed the tile's height)
  int tn;    // tile column
};

// Tiles of BM rows that hold `rows` (never negative) rows.
template <int BM>
__device__ __forceinline__ int tile_rows(int rows) {
  return (int)(((uint32_t)rows + BM - 1) / BM);
}

// Tiles of BM rows over the groups, and each lane's share of them.
struct RaggedPlan {
  int upto, mine;  // tile rows up to and with this lane's groups; in them
  int least;       // no row below this belongs to this lane's groups (0 where no offsets descend)
  int begin, end;  // the rows of this lane's group (up to 64 groups)
  int tiles;       // tiles of all groups
};

template <int BM>
__device__ __forceinline__ RaggedPlan ragged_plan(const int32_t* offsets, int groups, int rows, int tiles_n) {
  const int per = (groups + 63) >> 6, g0 = (threadIdx.x & 63) * per;
  RaggedPlan p;
  p.least = 0;
  // Lanes that met a descending pair: a scalar, as all lanes stay active (one without a group looks at
  // the last).  With the lanes' own flags and a branch a lane, 4 rows of 4 groups in 4 bits took 2.99 µs
  // against 2.85.
  uint64_t descends = 0;
  auto count = [&] {
    p.mine = p.begin = 0;
    p.end = p.least;
    for (int j = 0; j < per; ++j) {
      const int g = min(g0 + j, groups - 1);
      descends |= __ballot(offsets[g + 1] < offsets[g]);
      group_rows(offsets, g, p.end, rows, p.begin, p.end);
      p.mine += g0 + j < groups ? tile_rows<BM>(p.end - p.begin) : 0;
    }
  };
  count();
  if (__builtin_expect(descends != 0, 0)) {
    p.least = wave_max_before(p.end);
    count();
  }
  p.upto = wave_prefix_sum(p.mine);
  p.tiles = __builtin_amdgcn_readlane(p.upto, 63) * tiles_n;
  return p;
}

// Tile number `lid` (below plan.tiles): groups one after another, inside a group in band_tile's
// order, which keeps a group's operands in few L2 caches.
template <int BM>
__device__ __forceinline__ void ragged_find(const RaggedPlan& p, const int32_t* offsets, int groups, int rows,
                                            int tiles_n, int height, int lid, RaggedTile& t) {
  const int per = (groups + 63) >> 6, g0 = (threadIdx.x & 63) * per;
  int at = (p.upto - p.mine) * tiles_n;  // this lane's first tile
  int found = -1, fb = 0, fe = 0, fi = 0, begin = p.begin, end = per > 1 ? p.least : p.end;
  for (int j = 0; j < per; ++j) {
    if (g0 + j < groups) {
      if (per > 1) group_rows(offsets, g0 + j, end, rows, begin, end);
      const int n = tile_rows<BM>(end - begin) * tiles_n;
      if (lid >= at && lid < at + n) {
        found = g0 + j;
        fb = begin;
        fe = end;
        fi = lid - at;
      }
      at += n;
    }
  }
  const int src = __builtin_ctzll(__ballot(found >= 0));
  t.group = __builtin_amdgcn_readlane(found, src);
  const int b = __builtin_amdgcn_readlane(fb, src), e = __builtin_amdgcn_readlane(fe, src);
  int tm;
  band_tile(__builtin_amdgcn_readlane(fi, src), tile_rows<BM>(e - b), tiles_n, height, tm, t.tn);
  t.row0 = b + tm * BM;
  t.rows = e - t.row0;
}

// Workgroups are dealt round-robin to the 8 XCDs: XCD x takes the x-th eighth of `tiles`, and
// workgroup `bid` is the (bid / 8)-th on it.  Its XCD's first tile and number of tiles.
__device__ __forceinline__ void xcd_share(int tiles, int bid, int& first, int& count) {
  const int q = tiles >> 3, r = tiles & 7, x = bid & 7;
  count = x < r ? q + 1 : q;
  first = x < r ? x * (q + 1) : r * (q + 1) + (x - r) * q;
}

// The tile of workgroup `bid`, one tile each; false when there is none (the grid is an upper bound).
template <int BM>
__device__ __forceinline__ bool ragged_tile(const GroupedParams& g, int height, int bid, RaggedTile& t) {
  const RaggedPlan p = ragged_plan<BM>(g.offsets, g.groups, g.rows, g.tiles_n);
  int first, count;
  xcd_share(p.tiles, bid, first, count);
  if ((bid >> 3) >= count) return false;
  ragged_find<BM>(p, g.offsets, g.groups, g.rows, g.tiles_n, height, first + (bid >> 3), t);
  return true;
}

// The tile of workgroup `bid` of the weight gradient.
struct GradTile {
  int group, begin, rows;  // the group and its rows
  int tm, tn;
};

// Every group has the same tiles but its own number of rows, and so its own cost per tile.  Each
// XCD takes an eighth of every group's tiles (p.per_xcd consecutive ones, column-major within
// bands of tile rows, so that they share operand rows in its L2), so the XCDs stay level however
// the rows are split; and (p.by_rows, up to 64 groups) they run in the order of their rows, the
// longest first, so that the last workgroups to start are the short ones.  (One contiguous eighth of all tiles per
// XCD, as the products of equal tiles use, left the XCD of the longest group running alone: 381 µs
// against 248 for 8 groups of 16384 rows in all, 4096×2048.)
__device__ __forceinline__ bool grad_tile(const GroupedParams& p, int bid, GradTile& t) {
  const int lane = threadIdx.x & 63;
  const int per_group = p.tiles_m * p.tiles_n;
  const int x = bid & 7, i = bid >> 3, c = p.per_xcd;
  const int id = i / c * (8 * c) + x * c + i % c;
  const int place = id / per_group;
  if (place >= p.groups) return false;
  int g = place, begin, end;
  if (p.by_rows) {
    int b = 0, e = 0;
    if (lane < p.groups) group_rows(p.offsets, lane, 0, p.rows, b, e);
    const int rows = lane < p.groups ? e - b : -1;
    int rank = 0;  // groups that run before this lane's: more rows, or as many and an earlier number
    for (int j = 0; j < p.groups; ++j) {
      const int other = __builtin_amdgcn_readlane(rows, j);
      rank += other > rows || (other == rows && j < lane);
    }
    g = __builtin_ctzll(__ballot(rank == place && lane < p.groups));
    begin = __builtin_amdgcn_readlane(b, g);
    end = __builtin_amdgcn_readlane(e, g);
  } else {
    group_rows(p.offsets, g, 0, p.rows, begin, end);
    begin = __builtin_amdgcn_readfirstlane(begin);
    end = __builtin_amdgcn_readfirstlane(end);
  }
  const int in_group = id - place * per_group;
  band_tile(in_group, p.tiles_m, p.tiles_n, p.group_m, t.tm, t.tn);
  t.group = g;
  t.begin = begin;
  t.rows = end - begin;
  return true;
}

}  // namespace tbg
