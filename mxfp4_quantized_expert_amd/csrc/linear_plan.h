// Which of the linear operators' kernels takes a call, and the rows of its
// tiles: plain host arithmetic on the sizes alone, from times measured at N,
// K = 736 .. 2880, 1 to 128 experts, 4 to 16384 rows, even and skewed loads.
#pragma once

#include <math.h>
#include <stdint.h>

namespace mxlinear {

struct Sizes {
  int64_t rows, n, k, experts;
  bool grouped;  // rows by expert (expert_offsets), else one dense matrix
  bool nv;       // NVFP4 weights
};

inline double used_experts(const Sizes& s) { return (double)(s.experts < s.rows ? s.experts : s.rows); }

// Bytes of one expert's codes and scales.
inline double weight_bytes(const Sizes& s) { return (double)s.n * s.k * (s.nv ? 0.5625 : 0.53125); }

// Row tiles of `tm` rows that a call has.  Evenly routed rows: an expert's
// count is Poisson distributed, and it has a tile for every multiple of tm that
// the count passes, one at least.  Where the counts spread over more than a
// tile, the last ones are half full in the mean.
inline double expected_tiles(const Sizes& s, int tm) {
  if (!s.grouped) return (double)((s.rows + tm - 1) / tm);
  const double experts = used_experts(s), mean = s.rows / experts, spread = sqrt(mean);
  if (4 * spread > tm) return s.rows / (double)tm + 0.5 * experts;
  double tiles = 1;
  for (int j = 1; j * tm < mean + 4 * spread; ++j) tiles += 0.5 * erfc((j * tm + 0.5 - mean) / (spread * sqrt(2.0)));
  return tiles * experts;
}

// A tile block takes a fixed time for each chunk of its loop, by its rows and
// by whether it has its CU to itself or shares it with another.  So few rows
// take small tiles, for more blocks, and many take large ones, which read
// fewer bytes of LDS for a product (2880 x 2880, tiles of 128, 64 and 32 rows:
// 512 dense rows 42, 25 and 19 us; 1024 rows 43, 27 and 30; 8192 rows 120, 136
// and 174; 16384 rows over 128 experts 365, 374 and 494).
struct TileCost {  // us of a chunk of tiles of 32, 64 and 128 rows
  double alone[3], shared[3];
};
constexpr TileCost kForward{{0.32, 0.49, 0.88}, {0.57, 0.83, 1.43}};
constexpr TileCost kBackward{{0.53, 0.64, 1.02}, {0.78, 1.0, 1.58}};

// ... and no tile is faster than its weights arrive, in bytes/us: from HBM for
// an expert's first tile (forward tiles of 128 rows have fewer stages of them
// on their way: 832 rows over 128 experts, 5760 x 2880, in tiles of 128, 64 and
// 32 rows: 292, 279 and 277 us), mostly from the caches for the others (1280
// rows over 32 experts, 5760 x 2880, 36 tiles of 64 or 60 of 32: 89 and 121 us).
constexpr double kFirstRead = 3.5e6, kFirstRead128 = 3.3e6, kNextRead = 7e6;

// The 16-row kernels read the weights once for each 16 rows: from HBM the
// first time, at `cold` bytes/us, from the caches then, at `hot`.
struct FewCost {
  double cold, hot;
};
constexpr FewCost kForwardFew{2.9e6, 3.7e6}, kBackwardFew{1.9e6, 5e6};

constexpr int kFewTileRows = 16;

struct TilePlan {
  bool pays;  // tiles, else the 16-row kernels
  int rows;   // of a tile
};

// col_tiles, chunks: blocks and loop steps of the other two axes.
inline TilePlan plan_tiles(const Sizes& s, bool forward, int most_rows, int64_t col_tiles, int chunks, double cus) {
  const TileCost& cost = forward ? kForward : kBackward;
  const FewCost& few = forward ? kForwardFew : kBackwardFew;
  const double experts = used_experts(s), bytes = weight_bytes(s);
  TilePlan p{false, 0};
  double best = 0;
  for (int r = 0; r < 3 && 32 << r <= most_rows; ++r) {
    const double tiles = expected_tiles(s, 32 << r), load = tiles * col_tiles / cus;  // blocks of a CU
    double chunk;
    if (load > 4) {  // full tiles, and an expert's last ones as a block of 32 rows
      const double even = s.rows / (double)(32 << r), full = even < tiles ? even : tiles;
      chunk = (full * cost.shared[r] + (tiles - full) * cost.shared[0]) * col_tiles / (2 * cus);
    } else {  // in rounds of two
      const int rounds = (int)(load / 2);
      const double rest = load - 2 * rounds;
      chunk = rounds * cost.shared[r] + (rest > 1 ? cost.shared[r] : rest > 0 ? cost.alone[r] : 0);
    }
    const double first = forward && r == 2 ? kFirstRead128 : kFirstRead;
    const double read_us = (experts / first + (tiles > experts ? tiles - experts : 0) / kNextRead) * bytes;
    const double us = chunk * chunks > read_us ? chunk * chunks : read_us;
    if (p.rows == 0 || us < best) p.rows = 32 << r, best = us;
  }
  const double reads = s.rows / (double)kFewTileRows + 0.5 * experts;  // of one expert's weights
  const double few_us = experts * bytes / few.cold + (reads > experts ? reads - experts : 0) * bytes / few.hot;
  p.pays = best < few_us;
  return p;
}

// Rows of the tiles of the kernel that streams the weights past rows kept in
// registers (4 or 8), or 0 for the other kernels: up to a mean of 2 rows an
// expert (dense: 4 rows) in tiles of 4, up to 6 (dense: 8) in tiles of 8 (us,
// MXFP4, 2880 x 2880, 32 experts, means of 2, 3, 6 and 8: 28, 33, 46 and 56 in
// tiles of 4 | 31, 32, 38 and 44 in tiles of 8 | 46, 47, 48 and 48 by the best of
// the others; 5760 x 2880, 8: 105 | 81 | 77).  Not where the 16-row kernel
// passes K in one round and there is little to stream, though two row groups
// and more for every CU (us, MXFP4, weights from HBM, streamed | 16-row kernel):
//   one row, K = 2880, N = 736, 1440, 2880, 4096, 8192, 12288 and 32768: 3.4, 4.5,
//     5.1, 5.7, 6.3, 7.4 and 13.2 | 4.0, 4.5, 4.6, 4.7, 6.4, 10.0 and 23.2
//   8 rows, K = 2880, N = 736, 2880, 5760 and 32768: 4.7, 8.5, 14.3 and 17.8 | 4.7,
//     5.4, 7.7 and 23.5
//   one row, K = 4096 and 8192, N = 736 and 2880: 4.1, 6.1, 5.3 and 7.0 | 5.7, 5.9,
//     9.1 and 9.5
//   16 rows over 16 experts and over 8, 736 x 736 (5 MB) and 1440 x 2880 (18 MB):
//     6.4 and 9.3 | 4.9 and 11.2
constexpr int kMeanOf4 = 2, kMeanOf8 = 6, kDenseOf4 = 4, kDenseOf8 = 8;
constexpr double kStreamBytes = 12.7e6;
constexpr int kFewRoundK = 8 * 3 * 128;  // of the 16-row kernel: eight waves, three chunks each

inline int stream_tile_rows(const Sizes& s, int64_t cus) {
  const int rows = s.rows <= (s.grouped ? kMeanOf4 * s.experts : kDenseOf4)   ? 4
                   : s.rows <= (s.grouped ? kMeanOf8 * s.experts : kDenseOf8) ? 8
                                                                              : 0;
  const bool little = used_experts(s) * weight_bytes(s) < kStreamBytes;
  const bool groups = used_experts(s) * ((s.n + 3) / 4) >= 2.0 * cus;
  return little && groups && s.k <= kFewRoundK ? 0 : rows;
}

}  // namespace mxlinear
