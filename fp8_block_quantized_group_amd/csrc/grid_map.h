// Which tile a block of a launch works on.  Functions of whole numbers, for the
// kernels and for the host, where a walk over a whole grid checks them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// Grids in two dimensions: a dimension holds fewer than 2^32 lanes, 2^22
// blocks of 1024.  A kernel compares its block's index (at most 2^31 blocks,
// rounded up to rows of the grid) with what there is.
constexpr int64_t kGridX = 1 << 20;
inline dim3 grid_of(int64_t blocks) {
  return dim3((unsigned)(blocks < kGridX ? blocks : kGridX),
              (unsigned)((blocks + kGridX - 1) / kGridX));
}

// Block b's tile of `live` ones.  Consecutive blocks run on the 8 XCDs in turn;
// each takes a run of consecutive tiles, whose operands its L2 then shares.
// -1: none.
__host__ __device__ inline int64_t tile_of_block(int64_t b, int64_t live) {
  const int64_t run = (live + 7) / 8, t = (b & 7) * run + (b >> 3);
  return (b >> 3) < run && t < live ? t : -1;
}
constexpr int64_t blocks_of_tiles(int64_t tiles) { return (tiles + 7) / 8 * 8; }

// The same where every expert has `per` tiles: they differ in work, so each is shared
// by the XCDs, an eighth of its tiles in a run (a run of experts per XCD instead: 32
// experts of 1024 rows on average, 2 x 2048 by 7168, weights' gradient 2.8 against 2.1
// ms).  e -1: none.
struct ExpertTile {
  int e;
  int64_t t;
};
__host__ __device__ inline ExpertTile expert_tile_of_block(int64_t b, int64_t per, int experts) {
  const int64_t run = (per + 7) / 8, at8 = b >> 3, e = at8 / run;
  const int64_t t = (b & 7) * run + (at8 - e * run);
  return e < experts && t < per ? ExpertTile{(int)e, t} : ExpertTile{-1, 0};
}

// Tiles of `tile` rows (at most 256) that n rows take; n + 255 passes 31 bits, not 32.
__host__ __device__ constexpr int row_tiles(int n, int tile) {
  return (int)(((unsigned)n + (unsigned)tile - 1) / (unsigned)tile);
}
// ... that rows sorted by expert can have at most
constexpr int64_t most_row_tiles(int tile, bool sorted, int rows, int experts) {
  return sorted ? (int64_t)(rows / tile) + (experts < rows ? experts : rows)
                : (int64_t)row_tiles(rows, tile);
}

// Tile t of mts x nts, walked in bands of 8 rows of tiles, down each band first.
struct TileAt {
  int m, n;
};
constexpr int kBand = 8;
__host__ __device__ inline TileAt tile_at(int64_t t, int mts, int nts) {
  const int64_t per = (int64_t)kBand * nts;
  const int band = (int)(t / per), rest = (int)(t - band * per);
  const int left = mts - band * kBand, h = left < kBand ? left : kBand;
  return TileAt{band * kBand + rest % h, rest / h};
}

}  // namespace moe
