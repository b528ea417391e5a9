// groups.cuh -- the tile schedule of products grouped by expert.
//
// The rows of group g are offsets[g] .. offsets[g + 1] - 1 of a matrix of
// `rows` rows; the offsets live in device memory, since a router writes them
// there, so the host knows neither the groups' sizes nor the number of tiles.
// Each CTA builds the schedule for itself in shared memory: the groups' first
// rows and the running number of their row tiles.  Persistent CTAs then take
// every gridDim.x-th tile of the same global order, and find a tile's group
// by walking forward from the previous tile's.
//
// Offsets are clamped to [0, rows] and made non-decreasing (a running
// maximum), so that wrong ones give wrong groups but no access out of range.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace g12 {

constexpr int kMaxGroups = 1024;

struct GroupTable {
  int row[kMaxGroups + 1];   // first row of each group; [groups]: end of the last
  int tile[kMaxGroups + 1];  // row tiles before each group
};

// Fills the table; all 32 lanes of one warp.  offsets == nullptr: one group
// of all rows.  tile_rows: rows per row tile.
__device__ __forceinline__ void build_groups(GroupTable& t, const int32_t* offsets, int groups,
                                             int rows, int tile_rows) {
  const int lane = threadIdx.x & 31;
  if (offsets == nullptr) {
    if (lane == 0) {
      t.row[0] = 0;
      t.row[1] = rows;
      t.tile[0] = 0;
      t.tile[1] = (rows + tile_rows - 1) / tile_rows;
    }
    return;
  }
  int reach = min(max(offsets[0], 0), rows);  // largest offset so far
  int tiles = 0;
  if (lane == 0) {
    t.row[0] = reach;
    t.tile[0] = 0;
  }
  for (int base = 0; base < groups; base += 32) {
    const int g = base + lane;
    int end = g < groups ? min(max(offsets[g + 1], 0), rows) : 0;
    end = max(end, reach);
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, end, s);
      if (lane >= s) end = max(end, v);
    }
    int start = __shfl_up_sync(0xffffffffu, end, 1);
    if (lane == 0) start = reach;
    int n = (end - start + tile_rows - 1) / tile_rows;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, n, s);
      if (lane >= s) n += v;
    }
    if (g < groups) {
      t.row[g + 1] = end;
      t.tile[g + 1] = tiles + n;
    }
    reach = __shfl_sync(0xffffffffu, end, 31);
    tiles += __shfl_sync(0xffffffffu, n, 31);
  }
}

// One tile of the schedule.
struct GroupTile {
  int group;
  int row0;   // first row of the tile
  int rows;   // its rows that belong to the group
  int tn;     // column tile
};

// Tile t of the forward order: group after group; within a group, bands of
// `band` row tiles, column tile by column tile (neighbouring CTAs share the
// group's weights and a band of its rows in L2).  g: the caller's group so
// far, only ever moved forward.
__device__ __forceinline__ GroupTile group_tile(const GroupTable& tab, int t, int tiles_n,
                                                int band, int tile_rows, int& g) {
  while (t >= tab.tile[g + 1] * tiles_n) ++g;
  const int tiles_m = tab.tile[g + 1] - tab.tile[g];
  const int local = t - tab.tile[g] * tiles_n;
  const int per_band = band * tiles_n;
  const int b = local / per_band;
  const int high = min(tiles_m - b * band, band);
  const int in_band = local - b * per_band;
  GroupTile r;
  r.group = g;
  r.tn = high == 8 ? in_band >> 3 : in_band / high;  // whole bands are 8 high
  const int tm = b * band + in_band - r.tn * high;
  r.row0 = tab.row[g] + tm * tile_rows;
  r.rows = min(tile_rows, tab.row[g + 1] - r.row0);
  return r;
}

}  // namespace g12
