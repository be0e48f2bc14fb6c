// Which of the 8-bit products' kernels takes a call: plain host arithmetic on
// the sizes alone, from times measured at N = 100 .. 5760, K = 128 .. 4096, 1
// to 128 experts, 1 to 16384 rows.
#pragma once

#include <stdint.h>

namespace mxfp8 {

struct Plan {
  bool few;        // the kernel whose waves split K, else the one with tiles in LDS
  int rows, cols;  // of a block's tile
};

// Blocks that evenly routed rows make.
inline int64_t blocks_of(int64_t rows, int64_t cols, int64_t experts, int tile_rows, int tile_cols) {
  const int64_t used = experts < rows ? experts : rows, mean = (rows + used - 1) / used;
  return used * ((mean + tile_rows - 1) / tile_rows) * ((cols + tile_cols - 1) / tile_cols);
}

// y: the smallest tile that leaves every CU one block at most: a block takes a
// time of its own, by its size, and a second one on its CU half of that again
// (us at N = K = 2880, dense; blocks in brackets: 32 rows in tiles of 16 x 16,
// 32 x 32 and 32 x 64: 6.7 [360], 7.3, 8.8; 64 rows: 8.9 [720], 7.4 [180], 9.2;
// 128 rows in 32 x 32, 32 x 64 and 32 x 128: 12.2 [360], 9.3 [180], 11.3; 256 rows
// in 32 x 64, 32 x 128, 64 x 128: 16.6 [360], 11.4 [184], 15.0; 512 in 32 x 128,
// 64 x 128 and 64 x 256: 17.9 [368], 15.3 [184], 19.1; 1024 in 64 x 128, 64 x 256
// and 128 x 256: 22.2 [368], 20.3 [192], 27.7; 2048 in the last two: 34.8 [384],
// 29.0 [192]).  The smallest of all may come twice.
//   Where no tile does that, few rows an expert take the 16-row kernel up to
// sixteen blocks a CU, then tiles of 128 weight rows, then of 256, as the
// weights have to arrive (16 x 16, 64 x 128 and 64 x 256, 32 experts, N = 2880:
// 16 rows 21.6, 27.2 and 25.9; 64 rows 49.8, 46.7 and 54.6; over 128 experts 64
// rows 90.7, 80.4 and 91.0; 1024 rows over 128: 282, 214 and 205; N = 5760, 256
// rows over 32: 137, 116 and 98), and from 64 rows an expert tiles of 128 rows
// (64 x 256 and 128 x 256, 128 experts: means of 32 rows 242 and 250, of 128 411
// and 333, with N = 5760 745 and 602).
inline Plan plan_forward(int64_t rows, int64_t n, int64_t experts, int64_t cus) {
  const int64_t used = experts < rows ? experts : rows;
  auto blocks = [&](int tile_rows, int tile_cols) { return blocks_of(rows, n, experts, tile_rows, tile_cols); };
  if (blocks(16, 16) <= 2 * cus) return {true, 16, 16};
  if (experts > 1 && rows <= 16 * used && blocks(16, 16) <= 16 * cus) return {true, 16, 16};
  if (blocks(32, 32) <= cus) return {true, 32, 32};
  if (blocks(32, 64) <= cus) return {true, 32, 64};
  if (blocks(32, 128) <= cus) return {false, 32, 128};
  if (blocks(64, 128) <= cus) return {false, 64, 128};
  if (blocks(64, 256) <= cus) return {false, 64, 256};
  if (experts > 1 && rows <= 4 * used) return {false, 64, 128};
  return experts > 1 && rows < 64 * used ? Plan{false, 64, 256} : Plan{false, 128, 256};
}

// dx: the 16-row kernel up to two blocks of it a CU, for a dense matrix, which
// stays in the caches for all its row tiles, four (us, 16 rows x 64 k and 64 x 256;
// dense, N = K = 2880: 64 rows 9.2 and 23.9, 256 rows [720 blocks] 20.4 and 24.2,
// 512 rows [1440] 33.9 and 24.4; 32 experts: 4 rows [180] 9.5 and 16.3, 16 rows
// [720] 27.1 and 23.4; 8 experts, N = 1000, K = 736: 512 rows [384] 8.0 and 12.0,
// 2048 rows [1536] 21.9 and 12.3; 128 experts, N = K = 736: 16 rows [192] 6.1 and
// 7.3, 64 rows [768] 13.5 and 9.0).
inline bool backward_has_few(int64_t rows, int64_t k, int64_t experts, int64_t cus) {
  return blocks_of(rows, k, experts, 16, 64) <= (experts > 1 ? 2 : 4) * cus;
}

}  // namespace mxfp8
