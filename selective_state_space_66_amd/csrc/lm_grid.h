// lm_grid.h -- launch grids of many blocks.
//
// HIP refuses a launch with 2^32 threads or more along one dimension of its
// grid, for 256 threads a block that is 2^24 blocks.  A kernel that may need
// more takes its block number from x and from a second dimension (grid_of
// spreads n blocks over both) and returns where the number is past n.
#pragma once

#include <stdint.h>

namespace ssm66 {

struct Grid { uint32_t x, more; };

// n blocks of `threads`, as x * more >= n; x is a multiple of 8 where more > 1
inline Grid grid_of(int64_t n, int threads) {
  const int64_t most = 0xffffffffll / threads / 8 * 8;
  const int64_t more = (n + most - 1) / most;
  if (more <= 1) return Grid{(uint32_t)n, 1u};
  return Grid{(uint32_t)(((n + more - 1) / more + 7) / 8 * 8), (uint32_t)more};
}

}  // namespace ssm66
