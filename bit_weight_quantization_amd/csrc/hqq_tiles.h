// hqq_tiles.h -- tiles of rows sorted into groups (experts or adapters), found on the device
// from the groups' row offsets, so that no count has to come back to the host.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hqq_internal.h"

namespace hqq {

// Upper bound of the tiles of `tile_rows` rows that `rows` rows in `groups` groups (and the
// rows of no group) can have: every group adds at most one tile that is not full.
inline int64_t max_row_tiles(int64_t rows, int64_t groups, int64_t tile_rows) {
  return rows / tile_rows + (groups + 1 < rows ? groups + 1 : rows);
}

struct RowTile {
  int group;       // in [0, groups], or -1: no such tile.  `groups`: rows of no group
  int64_t row0;    // first sorted row
  int rows;        // rows of the tile, 0 where there is none
  int index;       // index of the tile within its group
  int64_t group0;  // first sorted row of its group
  int64_t group_rows;
};

// Tile number `tile` of `tile_rows` rows, groups in order, the rows behind the last group
// last.  The whole wavefront calls it with equal arguments; a lane counts one group's tiles.
__device__ __forceinline__ RowTile find_row_tile(const int32_t* offsets, int groups, int64_t rows,
                                                 int tile_rows, int64_t tile) {
  const int lane = threadIdx.x & (kWave - 1);
  RowTile t = {-1, 0, 0, 0, 0, 0};
  int64_t before = 0;
  for (int g0 = 0; g0 <= groups; g0 += kWave) {
    const int g = g0 + lane;
    int start = 0, count = 0;
    if (g <= groups) {
      const int last = (int)rows;
      start = min(max(offsets[g], 0), last);  // (never outside the rows, whatever is stored)
      count = max((g < groups ? min(offsets[g + 1], last) : last) - start, 0);
    }
    const int tiles = (count + tile_rows - 1) / tile_rows;
    int upto = tiles;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int v = __shfl_up(upto, o, kWave);
      if (lane >= o) upto += v;
    }
    const uint64_t hit = __ballot(before + upto > tile);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      const int first = __builtin_amdgcn_readlane(upto - tiles, l);
      t.group = g0 + l;
      t.index = (int)(tile - before) - first;
      t.group0 = __builtin_amdgcn_readlane(start, l);
      t.group_rows = __builtin_amdgcn_readlane(count, l);
      t.row0 = t.group0 + (int64_t)t.index * tile_rows;
      const int64_t left = t.group_rows - (int64_t)t.index * tile_rows;
      t.rows = (int)(left < tile_rows ? left : tile_rows);
      return t;
    }
    before += __builtin_amdgcn_readlane(upto, kWave - 1);
  }
  return t;
}

// How many tiles there are in all.  As find_row_tile.
__device__ __forceinline__ int64_t count_row_tiles(const int32_t* offsets, int groups, int64_t rows,
                                                   int tile_rows) {
  const int lane = threadIdx.x & (kWave - 1), last = (int)rows;
  int64_t total = 0;
  for (int g0 = 0; g0 <= groups; g0 += kWave) {
    const int g = g0 + lane;
    int tiles = 0;
    if (g <= groups) {
      const int start = min(max(offsets[g], 0), last);
      tiles = (max((g < groups ? min(offsets[g + 1], last) : last) - start, 0) + tile_rows - 1) / tile_rows;
    }
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) tiles += __shfl_xor(tiles, o, kWave);
    total += tiles;
  }
  return total;
}

// Place of block `id` of a one-dimensional grid among tiles x cols output tiles, for blocks of
// which an XCD holds `slots` at a time (its 32 CUs times one or two).  Workgroups go to the 8 XCDs
// (each with an L2 of its own) in turn, so XCD id % 8 takes one contiguous eighth of an order in
// which 8 row tiles share a column tile before the next one comes: the blocks that run on one XCD
// at a time then read few distinct tiles of either operand.  The tiles of an XCD's share that would
// run alone after its last full round are each split over blocks along the inner size (units of it;
// at most 8 parts), whose partial sums a second kernel adds in order: a round that is not full
// costs as much time as a full one.
constexpr int kXcds = 8, kBand = 8;
constexpr int kMaxParts = 8;

struct TileShare {                 // one XCD's part of the order
  int64_t first, full;             // its first place, how many whole tiles
  int rest, parts;                 // tiles behind them, blocks for each
};
__host__ __device__ __forceinline__ TileShare tile_share(int xcd, int64_t total, int units, int slots) {
  TileShare s;
  s.first = total * xcd / kXcds;
  s.full = total * (xcd + 1) / kXcds - s.first;
  s.rest = (int)(s.full % slots);
  s.parts = 1;
  if (s.rest > 0) {
    const int most = units < kMaxParts ? units : kMaxParts, fit = slots / s.rest;
    s.parts = fit < most ? fit : most;
  }
  if (s.parts <= 1) s.rest = 0, s.parts = 1;
  s.full -= s.rest;
  return s;
}

struct TilePlace {
  int64_t tile, col;               // tile < 0: nothing for this block
  int part, parts, slot;           // parts > 1: part `part` of the sum, kept in slab `slot`
};
__device__ __forceinline__ TilePlace place_at(int64_t at, int64_t tiles, int64_t cols) {
  const int64_t band = at / (kBand * cols), in = at % (kBand * cols);
  const int64_t left = tiles - band * kBand, high = left < kBand ? left : kBand;
  return {band * kBand + in % high, in / high, 0, 1, 0};
}
__device__ __forceinline__ TilePlace place_tile(int64_t id, int64_t tiles, int64_t cols, int units,
                                                int slots, int xcd_slabs) {
  const int xcd = (int)(id % kXcds);
  const TileShare s = tile_share(xcd, tiles * cols, units, slots);
  const int64_t at = id / kXcds;
  if (at < s.full) return place_at(s.first + at, tiles, cols);
  const int64_t p = at - s.full;
  // (the second condition holds whenever offsets ascend; a slab is never outside, whatever is stored)
  if (p >= (int64_t)s.rest * s.parts || p >= xcd_slabs) return {-1, 0, 0, 1, 0};
  TilePlace t = place_at(s.first + s.full + p / s.parts, tiles, cols);
  t.part = (int)(p % s.parts);
  t.parts = s.parts;
  t.slot = xcd * xcd_slabs + (int)p;
  return t;
}
// Whether any of `total` tiles (the exact number) is split.
inline bool place_splits(int64_t total, int units, int slots) {
  for (int x = 0; x < kXcds; ++x)
    if (tile_share(x, total, units, slots).rest > 0) return true;
  return false;
}
// Blocks that at most `total` tiles need.
inline int64_t place_blocks(int64_t total, int slots) { return ((total + kXcds - 1) / kXcds + slots) * kXcds; }
// Slabs of one XCD's parts where there are at most `total` tiles (its split tiles: at most its share,
// at most a slot for each part): slab p of XCD x is number x place_slabs(..) + p.
inline int place_slabs(int64_t total, int slots) {
  const int64_t most = (total + kXcds - 1) / kXcds * kMaxParts;
  return most < slots ? (int)most : slots;
}

// The tiles of group `group`: number of its first tile, and how many.  As find_row_tile.
struct GroupTiles {
  int64_t first;
  int count;
};
__device__ __forceinline__ GroupTiles find_group_tiles(const int32_t* offsets, int64_t rows,
                                                       int tile_rows, int group) {
  const int lane = threadIdx.x & (kWave - 1), last = (int)rows;
  GroupTiles t = {0, 0};
  for (int g0 = 0; g0 <= group; g0 += kWave) {
    const int g = g0 + lane;
    int tiles = 0;
    if (g <= group) {
      const int start = min(max(offsets[g], 0), last);
      tiles = (max(min(offsets[g + 1], last) - start, 0) + tile_rows - 1) / tile_rows;
    }
    if (group < g0 + kWave) t.count = __builtin_amdgcn_readlane(tiles, group - g0);
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) tiles += __shfl_xor(tiles, o, kWave);
    t.first += tiles;
  }
  t.first -= t.count;
  return t;
}

}  // namespace hqq
