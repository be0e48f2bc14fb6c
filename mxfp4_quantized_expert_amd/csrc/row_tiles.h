// What the kernels of rows times weights share: the row tiles of the experts
// and the blocks that make them, buffers whose bounds drop what lies past a
// tile, LDS stages that the load unit fills.
//
// The kernels' argument structs have `offsets` (int32 [E + 1], or nullptr for
// one expert with every row), `R`, `E` and `max_tiles`.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "mx_device.h"

namespace mxtiles {

using mx::u32x4;

constexpr int kXcds = 8;
constexpr int kRawBuffer = 0x00020000;  // descriptor word 3: 32-bit data format, for untyped loads
// An offset past every buffer (they hold less than 2 GiB): the load returns zero.
constexpr uint32_t kDead = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, kRawBuffer);
}

struct Tile {
  int e, row0, rows;
};

// Row tile `idx` of at most tm rows, the experts' tiles one after another.
// Offsets are clamped to [0, R], so that no tile reaches outside the rows.
// Every lane of the wave returns the same; false past the last tile.
template <typename A>
__device__ bool find_tile(const A& a, int tm, int idx, Tile& t) {
  if (a.offsets == nullptr) {
    t.e = 0;
    t.row0 = idx * tm;
    t.rows = min(tm, a.R - t.row0);
    return idx < (int)(((int64_t)a.R + tm - 1) / tm);
  }
  const int lane = mx::lane_id();
  int before = 0;
  for (int e0 = 0; e0 < a.E; e0 += 64) {
    const int e = e0 + lane;
    int first = 0, count = 0;
    if (e < a.E) {
      first = min(max(a.offsets[e], 0), a.R);
      count = max(min(max(a.offsets[e + 1], 0), a.R) - first, 0);
    }
    const int n = (int)(((int64_t)count + tm - 1) / tm);
    const int last = before + mx::wave_inclusive_sum(n);
    const uint64_t hit = __ballot(idx >= last - n && idx < last);
    if (hit != 0) {
      const int l = __builtin_ctzll(hit);
      const int at = (idx - (__builtin_amdgcn_readlane(last, l) - __builtin_amdgcn_readlane(n, l))) * tm;
      t.e = e0 + l;
      t.row0 = __builtin_amdgcn_readlane(first, l) + at;
      t.rows = min(tm, __builtin_amdgcn_readlane(count, l) - at);
      return true;
    }
    before = __builtin_amdgcn_readlane(last, 63);
  }
  return false;
}

// Block -> (tile, chunk of the other axis): each XCD (blocks are dealt to
// them round robin) walks a contiguous range with the tile fastest, so that
// the tiles of an expert read its weights from one XCD's L2.
__device__ __forceinline__ bool map_block(int tiles, int chunks, int& tile, int& chunk) {
  const int64_t total = (int64_t)tiles * chunks;
  const int64_t per = (total + kXcds - 1) / kXcds;
  const int64_t b = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t w = (b % kXcds) * per + b / kXcds;
  if (b / kXcds >= per || w >= total) return false;
  chunk = (int)(w / tiles);
  tile = (int)(w - (int64_t)chunk * tiles);
  return true;
}

// The row tiles of all experts.
template <typename A>
__device__ int count_tiles(const A& a, int tm) {
  if (a.offsets == nullptr) return (int)(((int64_t)a.R + tm - 1) / tm);
  int total = 0;
  for (int e0 = 0; e0 < a.E; e0 += 64) {
    const int e = e0 + mx::lane_id();
    int count = 0;
    if (e < a.E) {
      const int first = min(max(a.offsets[e], 0), a.R);
      count = max(min(max(a.offsets[e + 1], 0), a.R) - first, 0);
    }
    total += __builtin_amdgcn_readlane(mx::wave_inclusive_sum((int)(((int64_t)count + tm - 1) / tm)), 63);
  }
  return min(total, a.max_tiles);
}

// Block -> (row tile, chunk of the other axis) of a kernel whose blocks share
// both operands: each XCD walks a contiguous range of the tiles that exist, in
// groups of kGroup row tiles with the tile fastest, so that the blocks that
// run together on it share weights and rows through its L2.
constexpr int kGroup = 4;
template <typename A>
__device__ __forceinline__ bool map_tile(const A& a, int tm, int chunks, int& tile, int& chunk) {
  const int tiles = count_tiles(a, tm);
  const int64_t total = (int64_t)tiles * chunks;
  const int64_t per = (total + kXcds - 1) / kXcds;
  const int64_t b = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t w = (b % kXcds) * per + b / kXcds;
  if (b / kXcds >= per || w >= total) return false;
  const int64_t span = (int64_t)kGroup * chunks;
  const int g = (int)(w / span), rem = (int)(w - g * span);
  const int gm = min(kGroup, tiles - g * kGroup);
  tile = g * kGroup + rem % gm;
  chunk = rem / gm;
  return true;
}

// Block -> (tile, chunk), as map_tile and find_tile, with groups that end with
// an expert: the blocks that run together on an XCD share one expert's weights.
// (A group of four tiles of two or three experts reads all their weights at a
// time: in 8 bits, us, 16384 rows over 32 experts, 5760 x 2880, 369, in groups
// that mix them 463, 2880 x 2880 196 and 238, over 128 experts, 5760 x 2880, 602
// and 616; the gradient of 1024 rows over 128, 2880 x 2880, 181 and 194.  Of one
// expert eight tiles share more rows' reads than two or four: 16384 rows 152 us,
// 163 and 158.  Over 8 to 64 experts with 64 to 384 rows each, N = 1440 to 4096,
// four batches of each size, this order takes 0.86 to 1.06 times the other's time
// and 0.98 times on the average.  A batch with a few blocks more than run at once
// can go either way by a tenth: 4096 rows over 32 experts, 2880 x 2880, 516 blocks,
// have 65 for the 64 places of an XCD, and the 65th starts when the first ends,
// after 47 to 57 us in mixed groups and 57 to 60 in these, and takes 35 to 45 more
// by itself: 94 us and 104.  544 blocks of 16 experts, N = 4096, take 98 mixed and
// 91 so.  What decides it is the counts, which are on the device.)
constexpr int kExpertGroup = 8;
template <typename A>
__device__ bool find_block(const A& a, int tm, int chunks, Tile& t, int& chunk) {
  const int tiles = count_tiles(a, tm);
  const int64_t total = (int64_t)tiles * chunks;
  const int64_t per = (total + kXcds - 1) / kXcds;
  const int64_t b = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t w = (b % kXcds) * per + b / kXcds;
  if (b / kXcds >= per || w >= total) return false;
  const int in = (int)(w / chunks);  // a tile of the block's expert
  int of = tiles, before = 0, e = 0, row0 = 0, rows = a.R;  // the expert's tiles, those before it, its rows
  if (a.offsets != nullptr) {
    const int lane = mx::lane_id();
    uint64_t hit = 0;
    for (int e0 = 0, seen = 0; e0 < a.E && hit == 0; e0 += 64) {
      const int at = e0 + lane;
      int first = 0, count = 0;
      if (at < a.E) {
        first = min(max(a.offsets[at], 0), a.R);
        count = max(min(max(a.offsets[at + 1], 0), a.R) - first, 0);
      }
      const int n = (int)(((int64_t)count + tm - 1) / tm);
      const int last = seen + mx::wave_inclusive_sum(n);
      hit = __ballot(in >= last - n && in < last);
      if (hit != 0) {
        const int l = __builtin_ctzll(hit);
        e = e0 + l;
        of = __builtin_amdgcn_readlane(n, l);
        before = __builtin_amdgcn_readlane(last, l) - of;
        row0 = __builtin_amdgcn_readlane(first, l);
        rows = __builtin_amdgcn_readlane(count, l);
      }
      seen = __builtin_amdgcn_readlane(last, 63);
    }
    if (hit == 0) return false;
  }
  const int64_t local = w - (int64_t)before * chunks, span = (int64_t)kExpertGroup * chunks;
  const int g = (int)(local / span), rem = (int)(local - g * span);
  const int gm = min(kExpertGroup, of - g * kExpertGroup);
  const int at = (g * kExpertGroup + rem % gm) * tm;
  chunk = rem / gm;
  t.e = e;
  t.row0 = row0 + at;
  t.rows = min(tm, rows - at);
  return true;
}

// Eight consecutive dy values of a row from element n on, zeros past N.
// kAligned: N is even, so that every row starts at a dword.
template <bool kAligned>
__device__ __forceinline__ u32x4 load_dy8(const __amdgpu_buffer_rsrc_t& r, const uint16_t* row, uint32_t row_bytes0,
                                          int n, int N, bool whole) {
  if constexpr (kAligned) {
    u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, n < N ? row_bytes0 + n * 2 : kDead, 0, 0);
#pragma unroll
    for (int i = 1; i < 4; ++i) v[i] = n + 2 * i < N ? v[i] : 0u;
    return v;
  } else {
    u32x4 v;
    if (whole) {  // uniform: no lane reaches past N
      __builtin_memcpy(&v, row + n, 16);
    } else {
      uint32_t e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = n + i < N ? row[n + i] : 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = e[2 * i] | (e[2 * i + 1] << 16);
    }
    return v;
  }
}

__device__ __forceinline__ int swizzle(int row) { return (row ^ (row >> 3)) & 7; }

__device__ __forceinline__ void load_lds16(const __amdgpu_buffer_rsrc_t& r, u32x4* lds, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, off, 0, 0, 0);
}

// f(0), f(1), ... as compile-time numbers until one returns false.
template <typename F, int... kP>
__device__ __forceinline__ bool each_of(F&& f, std::integer_sequence<int, kP...>) {
  return (f(std::integral_constant<int, kP>{}) && ...);
}

// Row tiles that a call may have (the experts' counts are on the device).
template <typename A>
int max_tiles(const A& a, int tm) {
  const int64_t full = (int64_t)a.R / tm;
  return (int)(a.offsets == nullptr ? ((int64_t)a.R + tm - 1) / tm : full + (a.E < a.R ? a.E : a.R));
}

// One block for every tile and chunk, for each XCD the same number; a launch
// holds fewer than 2^32 threads along x.
inline dim3 grid_of(int64_t tiles, int64_t chunks) {
  constexpr int64_t kMaxX = 1 << 22;
  const int64_t blocks = (tiles * chunks + kXcds - 1) / kXcds * kXcds;
  return blocks <= kMaxX ? dim3((unsigned)blocks) : dim3((unsigned)kMaxX, (unsigned)((blocks + kMaxX - 1) / kMaxX));
}

}  // namespace mxtiles
