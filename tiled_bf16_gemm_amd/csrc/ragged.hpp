// Ragged groups on the device: which rows belong to a group, and which tile of which group a
// workgroup computes.
//
// Group e holds rows offsets[e] .. offsets[e+1]-1.  The offsets stay in device memory (a router
// writes them there, and a captured graph replays with new ones), so the host only knows the
// number of rows and of groups: it launches as many workgroups as the worst split needs
// (ragged_grid) and each workgroup finds its tile from the offsets, every wave for itself: a lane
// counts the tiles of its share of the groups, one prefix sum over the lanes places them, and
// the lane whose range holds the workgroup's number answers.  That is one dependent load and ≈30
// vector instructions before the K loop, against a launch of its own (and a table in a workspace)
// for a planning kernel.  Offsets are clamped to the rows that exist and to ascending pairs, so
// no value in them takes an access outside the operands.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tbg {

constexpr int kMaxGroups = 4096;  // 64 per lane

// Rows of group g: begin .. end-1, inside 0 .. rows whatever the offsets hold.
__device__ __forceinline__ void group_rows(const int32_t* offsets, int g, int rows, int& begin, int& end) {
  begin = min(max(offsets[g], 0), rows);
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

struct RaggedTile {
  int group;
  int row0;  // first row of the tile
  int rows;  // rows from row0 to the end of the group (may exceed the tile's height)
  int tn;    // tile column
};

// The tile of workgroup `bid`, BM rows high, of `tiles_n` tile columns; false when there is none
// (the grid is an upper bound).  Workgroups are dealt round-robin to the 8 XCDs, so XCD x gets
// the x-th eighth of the tiles that exist, in order: groups one after another, and inside a group
// column-major within `group_m` tile rows, which keeps a group's operands in few L2 caches.
template <int BM>
__device__ __forceinline__ bool ragged_tile(const int32_t* offsets, int groups, int rows, int tiles_n, int group_m,
                                            int bid, RaggedTile& t) {
  const int lane = threadIdx.x & 63;
  const int per = (groups + 63) >> 6, g0 = lane * per;
  int mine = 0, begin = 0, end = 0;
  for (int j = 0; j < per; ++j) {
    if (g0 + j < groups) {
      group_rows(offsets, g0 + j, rows, begin, end);
      mine += (end - begin + BM - 1) / BM;
    }
  }
  const int upto = wave_prefix_sum(mine);
  const int total = __builtin_amdgcn_readlane(upto, 63) * tiles_n;
  const int q = total >> 3, r = total & 7, x = bid & 7, i = bid >> 3;
  if (i >= (x < r ? q + 1 : q)) return false;
  const int lid = x < r ? x * (q + 1) + i : r * (q + 1) + (x - r) * q + i;

  int at = (upto - mine) * tiles_n;  // this lane's first tile
  int found = -1, fb = 0, fe = 0, fi = 0;
  for (int j = 0; j < per; ++j) {
    if (g0 + j < groups) {
      if (per > 1) group_rows(offsets, g0 + j, rows, begin, end);
      const int n = (end - begin + BM - 1) / BM * tiles_n;
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
  const int in_group = __builtin_amdgcn_readlane(fi, src);
  const int tiles_m = (e - b + BM - 1) / BM;
  const int per_band = group_m * tiles_n;
  const int band = in_group / per_band, first = band * group_m;
  const int height = min(tiles_m - first, group_m), in_band = in_group - band * per_band;
  t.row0 = b + (first + in_band % height) * BM;
  t.rows = e - t.row0;
  t.tn = in_band / height;
  return true;
}

}  // namespace tbg
