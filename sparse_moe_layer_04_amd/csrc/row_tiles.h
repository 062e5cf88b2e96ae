// How a group's rows split into row tiles of the grouped products, for groups of
// up to 2^31 - 1 rows (nothing is added to n before it is divided).  Plain C++,
// which a check on the host compiles too.
#pragma once

namespace moe {

// blocks of 32 rows of a group of n
constexpr int row_blocks(int n) { return (n >> 5) + ((n & 31) > 0); }
// rows of each of mt tiles of n > 0 rows, the last one perhaps fewer
constexpr int tile_rows(int n, int mt) { return ((n - 1) / mt + 32) & ~31; }

}  // namespace moe
