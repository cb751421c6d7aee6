// Walks every block of a launch, up to the last one of the rounded-up grid, and counts
// the tiles that the blocks take.  Arguments: "experts" per E, or "tiles" launched live.
// Prints one line: "ok", or the first block that goes wrong.  "rows" rows tile prints the
// tiles of so many rows, of one expert and at most of 1024.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "grid_map.h"

int main(int argc, char** argv) {
  if (argc != 4) return 2;
  if (std::strcmp(argv[1], "rows") == 0) {
    const int rows = std::atoi(argv[2]), tile = std::atoi(argv[3]);
    std::printf("%d %lld %lld\n", moe::row_tiles(rows, tile),
                (long long)moe::most_row_tiles(tile, false, rows, 1),
                (long long)moe::most_row_tiles(tile, true, rows, 1024));
    return 0;
  }
  const bool experts = std::strcmp(argv[1], "experts") == 0;
  const int64_t per = std::atoll(argv[2]), second = std::atoll(argv[3]);
  const int64_t tiles = experts ? per * second : second;
  const dim3 grid =
      moe::grid_of(experts ? moe::blocks_of_tiles(per) * second : moe::blocks_of_tiles(per));
  std::vector<bool> taken(tiles);
  int64_t count = 0;
  for (int64_t b = 0; b < (int64_t)grid.x * grid.y; ++b) {
    int64_t t;
    if (experts) {
      const moe::ExpertTile w = moe::expert_tile_of_block(b, per, (int)second);
      if (w.e == -1) continue;
      t = w.e < 0 || w.e >= second || w.t < 0 || w.t >= per ? -1 : w.e * per + w.t;
    } else {
      t = moe::tile_of_block(b, second);
      if (t == -1) continue;
    }
    if (t < 0 || t >= tiles || taken[t]) {
      std::printf("block %lld of %u x %u\n", (long long)b, grid.x, grid.y);
      return 1;
    }
    taken[t] = true;
    ++count;
  }
  if (count != tiles) {
    std::printf("%lld of %lld tiles\n", (long long)count, (long long)tiles);
    return 1;
  }
  std::puts("ok");
  return 0;
}
