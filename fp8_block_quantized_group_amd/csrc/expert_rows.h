// Which expert and which of its rows a block works on, for the kernels over rows
// sorted by expert.
#pragma once

#include "grid_map.h"

namespace moe {

// Rows [r0, r0 + n) of expert e.  Offsets that are not what the sort writes
// give wrong rows, never rows outside [0, R).
struct ExpertRange {
  int r0, n;
};
__device__ __forceinline__ ExpertRange expert_range(const int32_t* off, int R, int e) {
  if (off == nullptr) return ExpertRange{0, R};
  const int a = min(max(off[e], 0), R), b = min(max(off[e + 1], a), R);
  return ExpertRange{a, b - a};
}

// The rows' tile for this block: the tiles of all experts with rows, in their
// order, are the tile rows.  Every wave finds it for itself: a lane adds up the
// tiles of E / 64 experts, a scan over the lanes gives the total and the lane
// that holds the tile.  Offsets that do not ascend can make the experts' rows add up to
// more than R, and their tiles to more than 31 bits: a tile that is not found then is
// none, and no row outside [0, R) is taken.
struct RowTile {
  int e, r0, n, m, nt;      // expert, its first row and rows, tile row in it, tile column
  bool live;
};
template <int BM>
__device__ __forceinline__ RowTile find_row_tile(const int32_t* off, int R, int E, int nts,
                                                 int64_t block) {
  RowTile t{0, 0, R, 0, 0, true};
  if (off == nullptr) {
    const int mts = row_tiles(R, BM);
    const int64_t at = tile_of_block(block, (int64_t)mts * nts);
    t.live = at >= 0;
    if (!t.live) return t;
    const TileAt w = tile_at(at, mts, nts);
    t.m = w.m;
    t.nt = w.n;
    return t;
  }
  const int lane = threadIdx.x & 63, per = (E + 63) / 64;
  const int e0 = min(lane * per, E), e1 = min(e0 + per, E);
  unsigned mine = 0;
  for (int e = e0; e < e1; ++e) mine += row_tiles(expert_range(off, R, e).n, BM);
  unsigned upto = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const unsigned v = __shfl_up(upto, d);
    if (lane >= d) upto += v;
  }
  const int mts = __builtin_amdgcn_readlane((int)upto, 63);
  const int64_t at = tile_of_block(block, (int64_t)mts * nts);
  t.live = at >= 0;
  if (!t.live) return t;
  const TileAt w = tile_at(at, mts, nts);
  t.nt = w.n;
  // the lane whose tiles hold row w.m, then the expert among its own
  const uint64_t past = __ballot((unsigned)w.m < upto);
  const int owner = past != 0 ? __builtin_ctzll(past) : 0;
  int left = w.m - (int)(upto - mine), he = -1, hr = 0, hn = 0;
  for (int e = e0; e < e1; ++e) {
    const ExpertRange r = expert_range(off, R, e);
    const int tiles = row_tiles(r.n, BM);
    if (left >= 0 && left < tiles) {
      he = e;
      hr = r.r0;
      hn = r.n;
      break;
    }
    left -= tiles;
  }
  t.e = __builtin_amdgcn_readlane(he, owner);
  t.live = t.e >= 0;
  t.r0 = __builtin_amdgcn_readlane(hr, owner);
  t.n = __builtin_amdgcn_readlane(hn, owner);
  t.m = __builtin_amdgcn_readlane(left, owner);
  return t;
}

template <int BM>
inline int64_t most_row_tiles(const int32_t* offsets, int rows, int experts) {
  return most_row_tiles(BM, offsets != nullptr, rows, experts);
}

}  // namespace moe
