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
  int group;    // -1: none
  int row0;     // first row of the group
  int rows;     // rows of the group
  int tm, tn;   // row tile within the group, column tile
};

// All groups' ceil(rows / bm) x tiles_n tiles, numbered group by group; within a
// group in bands of `band` row tiles, column by column, so that tiles worked on at
// the same time share row and column panels in an XCD's L2.
struct GroupTiles {
  const int32_t* offsets;
  int groups, rows, bm, tiles_n, band, lane;
  int lo0 = 0, rows0 = 0, sum0 = 0;     // this lane's group among the first 64
  int64_t tiles;            // of all groups

  __device__ __forceinline__ GroupTiles(const int32_t* offsets_, int groups_, int rows_, int bm_, int tiles_n_,
                                        int band_, int lane_)
      : offsets(offsets_), groups(groups_), rows(rows_), bm(bm_), tiles_n(tiles_n_), band(band_), lane(lane_) {
    int64_t row_tiles = 0;
    for (int c = 0; c < groups; c += 64) {
      int lo, r, sum;
      chunk(c, lo, r, sum);
      if (c == 0) {
        lo0 = lo;
        rows0 = r;
        sum0 = sum;
      }
      row_tiles += __builtin_amdgcn_readlane(sum, 63);
    }
    // (offsets in order never give more; others, whose groups may overlap, stop here)
    if (row_tiles > rows / bm + groups) row_tiles = rows / bm + groups;
    tiles = row_tiles * tiles_n;
  }

  // groups c .. c + 63, one a lane: first row, rows, inclusive sum of row tiles
  __device__ __forceinline__ void chunk(int c, int& lo, int& r, int& sum) const {
    lo = 0;
    r = c + lane < groups ? group_rows(offsets, c + lane, rows, &lo) : 0;
    sum = wave_prefix_sum((r + bm - 1) / bm);
  }

  // Rows and first row of one group (wave-uniform e).
  __device__ __forceinline__ int rows_of(int e, int* lo) const {
    if (e < 64) {
      *lo = __builtin_amdgcn_readlane(lo0, e);
      return __builtin_amdgcn_readlane(rows0, e);
    }
    return group_rows(offsets, e, rows, lo);
  }

  // Tile i of XCD x: each of the 8 XCDs has one contiguous run of the tiles.
  __device__ __forceinline__ GroupTile find(int x, int64_t i) const {
    GroupTile g{-1, 0, 0, 0, 0};
    const int64_t per_xcd = (tiles + 7) >> 3, item = x * per_xcd + i;
    if (i >= per_xcd || item >= tiles) return g;
    const uint32_t q = (uint32_t)(item / tiles_n);   // row tiles before it, over all groups (below 2^31)
    uint32_t base = 0;
    for (int c = 0; c < groups; c += 64) {
      int lo = lo0, r = rows0, sum = sum0;
      if (c > 0) chunk(c, lo, r, sum);
      const int total = __builtin_amdgcn_readlane(sum, 63);
      if (q < base + total) {
        const int l = __popcll(__ballot(base + sum <= q));   // the first lane whose sum exceeds q
        g.group = c + l;
        g.row0 = __builtin_amdgcn_readlane(lo, l);
        g.rows = __builtin_amdgcn_readlane(r, l);
        const int rt = (g.rows + bm - 1) / bm;
        const int start = (int)base + __builtin_amdgcn_readlane(sum, l) - rt;
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
};

// Tile of a workgroup that takes one.
__device__ __forceinline__ GroupTile find_group_tile(const int32_t* __restrict__ offsets, int groups, int rows,
                                                     int bm, int tiles_n, int band, int block, int lane) {
  return GroupTiles(offsets, groups, rows, bm, tiles_n, band, lane).find(block & 7, block >> 3);
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
