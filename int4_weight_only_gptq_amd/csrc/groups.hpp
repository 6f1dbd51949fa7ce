// Rows grouped by expert: which group a workgroup's tile belongs to.
//
// offsets[0 .. groups] (device memory, non-decreasing) give group e the rows
// offsets[e] .. offsets[e + 1] of a [rows][...] matrix.  The counts are known
// only on the device, so the host launches as many workgroups as the worst
// distribution needs and every workgroup finds its own tile: one pass over the
// offsets, 64 groups at a time, a prefix sum over the wave's lanes.  All waves
// of a workgroup do the same lookup, so no LDS or barrier is needed.
#pragma once

#include "common.hpp"

namespace qg {

// Inclusive prefix sum over the 64 lanes of a wave (row shifts within 16 lanes,
// then the row totals broadcast to the rows above).
__device__ __forceinline__ int wave_prefix_sum(int v) {
#if defined(__HIP_DEVICE_COMPILE__)
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);    // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);    // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);    // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);    // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast:15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // row_bcast:31
#endif
  return v;
}

// Rows [*lo, *lo + return value) of group e; whatever the offsets hold, the
// range lies inside [0, rows).
__device__ __forceinline__ int group_rows(const int32_t* offsets, int e, int rows, int* lo) {
  const int a = min(max(offsets[e], 0), rows), b = min(max(offsets[e + 1], 0), rows);
  *lo = a;
  return max(b - a, 0);
}

struct GroupTile {
  int group;    // -1: no tile left for this workgroup
  int row0;     // first row of the group
  int rows;     // rows of the group
  int tm, tn;   // row tile within the group, column tile
};

// Tile of workgroup `block` among every group's ceil(rows / bm) x tiles_n tiles.
// The tiles are numbered group by group and dealt out so that each XCD (block
// mod 8) gets one contiguous run of them; within a group they go in bands of
// `band` row tiles, column by column, so that the about 32 tiles an XCD works on
// at a time share row and column panels in its L2.
__device__ __forceinline__ GroupTile find_group_tile(const int32_t* __restrict__ offsets, int groups, int rows,
                                                     int bm, int tiles_n, int band, int block, int lane) {
  int first_lo = 0, first_rows = 0, first_sum = 0, row_tiles = 0;
  for (int c = 0; c < groups; c += 64) {
    const int e = c + lane;
    int lo = 0;
    const int r = e < groups ? group_rows(offsets, e, rows, &lo) : 0;
    const int sum = wave_prefix_sum((r + bm - 1) / bm);
    if (c == 0) {
      first_lo = lo;
      first_rows = r;
      first_sum = sum;
    }
    row_tiles += __builtin_amdgcn_readlane(sum, 63);
  }
  GroupTile g{-1, 0, 0, 0, 0};
  const int64_t tiles = (int64_t)row_tiles * tiles_n;
  const int64_t per_xcd = (tiles + 7) >> 3;
  const int64_t item = (int64_t)(block & 7) * per_xcd + (block >> 3);
  if ((block >> 3) >= per_xcd || item >= tiles) return g;
  const int q = (int)(item / tiles_n);   // row tiles before it, over all groups
  int base = 0;
  for (int c = 0; c < groups; c += 64) {
    int lo = first_lo, r = first_rows, sum = first_sum;
    if (c > 0) {
      const int e = c + lane;
      lo = 0;
      r = e < groups ? group_rows(offsets, e, rows, &lo) : 0;
      sum = wave_prefix_sum((r + bm - 1) / bm);
    }
    const int total = __builtin_amdgcn_readlane(sum, 63);
    if (q < base + total) {
      // the first lane whose inclusive sum exceeds q
      const uint64_t before = __ballot(base + sum <= q);
      const int l = __popcll(before);
      g.group = c + l;
      g.row0 = __builtin_amdgcn_readlane(lo, l);
      g.rows = __builtin_amdgcn_readlane(r, l);
      const int rt = (g.rows + bm - 1) / bm;
      const int start = base + __builtin_amdgcn_readlane(sum, l) - rt;
      const int local = (int)(item - (int64_t)start * tiles_n);
      const int b = local / (band * tiles_n), in = local - b * band * tiles_n;
      const int height = min(band, rt - b * band);
      g.tn = in / height;
      g.tm = b * band + (in - g.tn * height);
      return g;
    }
    base += total;
  }
  return g;
}

// Workgroups that cover every distribution of `rows` rows over `groups` groups
// in tiles of bm rows: sum of ceil(r / bm) <= min(rows, rows / bm + groups),
// rounded up to whole rounds of the 8 XCDs.
inline int64_t group_tile_blocks(int64_t rows, int64_t groups, int64_t bm, int64_t tiles_n) {
  int64_t row_tiles = rows / bm + groups;
  if (row_tiles > rows) row_tiles = rows;
  return (row_tiles * tiles_n + 7) / 8 * 8;
}

}  // namespace qg
