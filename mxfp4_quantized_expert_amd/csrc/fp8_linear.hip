// Rows in 8 bits times 8-bit weights, dense or per expert, and the gradient to
// the rows.
//
//   y[r, n]  = sum_k x[r, k] W_e[n, k] + b_e[n]
//   dx[r, k] = sum_n dy[r, n] W_e[n, k]
// for the rows r of expert e (expert_offsets; one expert without them).  x and
// W are E4M3 codes; x has a float32 scale for each 128 k of a row, W one for
// each 128 n x 128 k.  The weights are frozen, so the rows are all that has a
// gradient; dy is bf16.
//
// Codes multiply exactly: two of them on the FP8 MFMA, a code (exact in bf16)
// and dy on the bf16 one.  Each block of 128 of the summed axis is added up by
// the MFMA, multiplied by its scales and added to the sum, in fp32; the bias
// follows and the result is rounded once.  The MFMA sums are fp32, except that
// the FP8 one adds eight neighbouring products as integers in steps of 2^-13
// of the largest's power of two, and cuts off what lies below (measured by
// pairs of products on MI355X; the older 16x16x32 form does the same).  That is
// its price for twice the rate of the bf16 MFMA, on which the same codes would
// be added in full; it is 2^-4 of the rounding of a bf16 result where products
// are within a few powers of two of each other, as normal data are.
#include "expert_device.h"
#include "fp8_device.h"
#include "fp8_plan.h"
#include "internal.h"
#include "mx_device.h"
#include "row_tiles.h"

namespace {

using namespace mxtiles;
using mx::bf16x8;
using mx::f32x4;
using mx::i32x8;
using mx::u32x4;

constexpr int kBlock = mx8::kBlock;
// Floats that every lane reads alike, through the scalar cache.
typedef const __attribute__((address_space(4))) float* ScalarFloats;

struct Fp8Args {
  const void* x;           // forward: x [R, K] codes; gradient: dy [R, N] bf16
  const float* x_scales;   // forward: [R, ceil(K / 128)]
  const uint8_t* w;        // [E, N, K] codes
  const float* w_scales;   // [E, ceil(N / 128), ceil(K / 128)]
  const uint16_t* bias;    // [E, N] or nullptr
  const int32_t* offsets;  // [E + 1] or nullptr (E == 1, every row)
  uint16_t* y;             // forward: y [R, N]; gradient: dx [R, K]
  int R, K, N, E;
  int max_tiles;           // row tiles, at most
  int tile_rows;           // rows of a tile of the kernels with tiles in LDS
};

// Sixteen rows of A times sixteen rows of B over 128 k of codes: a lane's 32
// bytes are k 16 q .. + 15 and 64 + 16 q .. + 15 of row lane & 15 (q = lane >>
// 4) on both sides; any agreed order of k gives the same sum.
__device__ __forceinline__ f32x4 multiply(u32x4 a0, u32x4 a1, u32x4 b0, u32x4 b1) {
  const i32x8 a = {(int)a0[0], (int)a0[1], (int)a0[2], (int)a0[3], (int)a1[0], (int)a1[1], (int)a1[2], (int)a1[3]};
  const i32x8 b = {(int)b0[0], (int)b0[1], (int)b0[2], (int)b0[3], (int)b1[0], (int)b1[1], (int)b1[2], (int)b1[3]};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{}, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ void take_up(f32x4& sum, const f32x4& part, float scale) {
#pragma unroll
  for (int c = 0; c < 4; ++c) sum[c] = __builtin_fmaf(part[c], scale, sum[c]);
}

// Four consecutive outputs of a row, `n` of them in range (`whole`: always four, 8-byte aligned).
__device__ __forceinline__ void store4(uint16_t* out, f32x4 v, const uint16_t* bias, int n, bool whole) {
  if (bias != nullptr) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (c < n) v[c] += mx::bf16_to_f32(bias[c]);
  }
  const uint2 packed = mxgemm::pack_bf16x4(v);
  if (whole) {
    *reinterpret_cast<uint2*>(out) = packed;
    return;
  }
  const uint32_t d[2] = {packed.x, packed.y};
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (c < n) out[c] = (uint16_t)(d[c >> 1] >> (16 * (c & 1)));
}

// ---------------------------------------------------------------- few rows

// y for row tiles of at most 16 kR rows: weights as the A operand, rows as B,
// both straight to registers.  The waves of a block split K, kC blocks of 128
// each at a time (all loads of a wave in flight before the first product), for
// kG * 16 weight rows, so a block has no barrier before its sums meet in LDS,
// added in wave order: one round of latency, 4.0 us for one row of 2880 x 2880,
// 8.9 for 128.  Weight row 4 kG (m / 4) + 4 i + m % 4 is operand row m
// of subtile i, so that a lane's outputs are neighbours.  Loads past K, N or
// the tile's rows return zero from the buffer's bounds.
template <int kC, int kG, int kR>
__global__ __launch_bounds__(512) void fp8_linear_few_kernel(Fp8Args a) {
  extern __shared__ f32x4 red[];  // [waves][kG kR][64]
  const int n_chunks = (a.N + 16 * kG - 1) / (16 * kG);
  int ti, nc;
  if (!map_block(a.max_tiles, n_chunks, ti, nc)) return;  // uniform per block
  Tile t;
  if (!find_tile(a, 16 * kR, ti, t)) return;
  const int K = a.K, N = a.N, n0 = nc * 16 * kG, kb = (K + kBlock - 1) / kBlock;
  const int lane = mx::lane_id(), lr = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const auto rx = buffer(static_cast<const uint8_t*>(a.x) + (size_t)t.row0 * K, (uint32_t)t.rows * K);
  const auto rw = buffer(a.w + ((size_t)t.e * N + n0) * K, (uint32_t)min(16 * kG, N - n0) * K);
  const auto rs = buffer(a.x_scales + (size_t)t.row0 * kb, (uint32_t)t.rows * kb * 4);
  const ScalarFloats ws = (ScalarFloats)(a.w_scales + ((size_t)t.e * mx8::blocks_of(N) + n0 / kBlock) * kb);
  const uint32_t woff = __umul24(4 * kG * (lr >> 2) + (lr & 3), K) + 16 * q;

  f32x4 acc[kG][kR] = {};
  for (int c0 = wave * kC; c0 < kb; c0 += waves * kC) {
    u32x4 x[kC][kR][2], w[kC][kG][2];
    float s[kC][kR], u[kC];
#pragma unroll
    for (int j = 0; j < kC; ++j) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = (c0 + j) * kBlock + 64 * h;
        const bool in = k + 16 * q < K;
#pragma unroll
        for (int i = 0; i < kG; ++i)
          w[j][i][h] = __builtin_amdgcn_raw_buffer_load_b128(rw, in ? woff + __umul24(4 * i, K) + k : kDead, 0, 0);
#pragma unroll
        for (int r = 0; r < kR; ++r)
          x[j][r][h] =
              __builtin_amdgcn_raw_buffer_load_b128(rx, in ? __umul24(16 * r + lr, K) + 16 * q + k : kDead, 0, 0);
      }
      const int c = min(c0 + j, kb - 1);
      u[j] = ws[c];
#pragma unroll
      for (int r = 0; r < kR; ++r)
        s[j][r] = __builtin_bit_cast(
            float, __builtin_amdgcn_raw_buffer_load_b32(rs, __umul24(16 * r + lr, 4 * kb) + 4 * c, 0, 0));
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      if (c0 + j >= kb) break;  // uniform
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        const float scale = s[j][r] * u[j];
#pragma unroll
        for (int i = 0; i < kG; ++i)
          take_up(acc[i][r], multiply(w[j][i][0], w[j][i][1], x[j][r][0], x[j][r][1]), scale);
      }
    }
  }
  // lane (row lr of subtile r, q): features n0 + 4 kG q + 4 i .. + 3 in acc[i][r]
  constexpr int kAll = kG * kR;
#pragma unroll
  for (int i = 0; i < kAll; ++i) red[(wave * kAll + i) * 64 + lane] = acc[i % kG][i / kG];
  __syncthreads();
  for (int i = wave; i < kAll; i += waves) {
    f32x4 v = red[i * 64 + lane];
    for (int u = 1; u < waves; ++u) v += red[(u * kAll + i) * 64 + lane];
    const int n = n0 + 4 * kG * q + 4 * (i % kG), row = 16 * (i / kG) + lr;
    if (row >= t.rows || n >= N) continue;
    const uint16_t* bias = a.bias != nullptr ? a.bias + (size_t)t.e * N + n : nullptr;
    store4(a.y + (size_t)(t.row0 + row) * N + n, v, bias, min(4, N - n), (N & 3) == 0);
  }
}

// Two codes (bytes 2 SEL and 2 SEL + 1 of `four`) as two bf16, exactly.
template <int SEL>
__device__ __forceinline__ uint32_t fp8x2_to_bf16x2(uint32_t four) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(four, 1.0f, SEL != 0));
}

// dx for row tiles of at most 16 rows.  The sum runs over weight rows, so the
// MFMA's A operand is the transposed weights: lane (m, q) loads four codes, k =
// 4 m .. 4 m + 3 of a block's 64, of eight weight rows n = 8 q .. 8 q + 7,
// converts them to pairs of k and exchanges halves between the rows of a pair
// (v_perm) into four operands of eight n, one for each k.  The waves of a block
// take every waves-th block of 128 n and add their sums in LDS in wave order: one
// row of 2880 x 2880 7.5 us, 64 rows 8.8.  (32 or 64 rows a block, to convert the
// weights for more rows at a time, gained nothing: 64 rows 12.4 and 19.8 us, 256
// rows 22.2 and 19.8, where sixteen rows a block take 18.8 to 20.4.)
constexpr int kBackFewK = 64;
constexpr int kBackFewRows = 16;
constexpr int kRedStride = 20;  // floats per lane in LDS: 16 and padding

template <bool kAligned>
__global__ __launch_bounds__(512) void fp8_linear_backward_few_kernel(Fp8Args a) {
  extern __shared__ float redf[];
  const int k_chunks = (a.K + kBackFewK - 1) / kBackFewK;
  int ti, kc;
  if (!map_block(a.max_tiles, k_chunks, ti, kc)) return;  // uniform per block
  Tile t;
  if (!find_tile(a, kBackFewRows, ti, t)) return;
  const int K = a.K, N = a.N, k0 = kc * kBackFewK, kb = (K + kBlock - 1) / kBlock, nb = (N + kBlock - 1) / kBlock;
  const int lane = mx::lane_id(), m = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const auto rw = buffer(a.w + (size_t)t.e * N * K, (uint32_t)N * K);
  const uint16_t* dy0 = static_cast<const uint16_t*>(a.x) + (size_t)t.row0 * N;
  const auto rd = buffer(dy0, (uint32_t)t.rows * N * 2);
  const float* ws = a.w_scales + (size_t)t.e * nb * kb + k0 / kBlock;
  const uint32_t col = k0 + 4 * m;

  const int row = min(m, t.rows - 1);  // columns past the tile's rows are dropped
  f32x4 acc[4] = {};
  for (int b = wave; b < nb; b += waves) {
    uint32_t w[4][8];
    u32x4 d[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int n = kBlock * b + 32 * u + 8 * q;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[u][i] = __builtin_amdgcn_raw_buffer_load_b32(
            rw, n + i < N && col < (uint32_t)K ? (uint32_t)(n + i) * K + col : kDead, 0, 0);
      d[u] = load_dy8<kAligned>(rd, dy0 + (size_t)row * N, (uint32_t)row * N * 2, n, N,
                                kBlock * b + 32 * u + 32 <= N);
    }
    const float s = ws[(size_t)b * kb];
    __builtin_amdgcn_sched_barrier(0);
    f32x4 part[4] = {};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      uint32_t r[8][2];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        r[i][0] = fp8x2_to_bf16x2<0>(w[u][i]);
        r[i][1] = fp8x2_to_bf16x2<1>(w[u][i]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u32x4 op;
#pragma unroll
        for (int p = 0; p < 4; ++p)
          op[p] = __builtin_amdgcn_perm(r[2 * p + 1][j >> 1], r[2 * p][j >> 1], (j & 1) ? 0x07060302u : 0x05040100u);
        part[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(mx::as_bf16x8(op), mx::as_bf16x8(d[u]), part[j], 0, 0, 0);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) take_up(acc[j], part[j], s);
  }
  // lane (row m of the tile, q) holds k = k0 + 16 q + 4 c + j in acc[j][c]
  float* mine = redf + (wave * 64 + lane) * kRedStride;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<f32x4*>(mine + 4 * c) = f32x4{acc[0][c], acc[1][c], acc[2][c], acc[3][c]};
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * 4; i += blockDim.x) {
    const int l = i >> 2, c = i & 3;
    f32x4 v = *reinterpret_cast<const f32x4*>(redf + l * kRedStride + 4 * c);
    for (int u = 1; u < waves; ++u) v += *reinterpret_cast<const f32x4*>(redf + (u * 64 + l) * kRedStride + 4 * c);
    const int k = k0 + 16 * (l >> 4) + 4 * c, r = l & 15;
    if (r < t.rows && k < K) *reinterpret_cast<uint2*>(a.y + (size_t)(t.row0 + r) * K + k) = mxgemm::pack_bf16x4(v);
  }
}

// --------------------------------------------------------------- many rows

// y for larger row tiles: 16x16x128 MFMA, a block of kWaves waves makes 64
// kWaves weight rows x kRows rows, each wave 64 x kRows, in chunks of 128 k, the
// span of a scale.  x travels into a ring of LDS stages by the load unit, with
// the chunk's scales.  No wave shares its weights: they come to registers in
// whole lines of 128 bytes, kAhead chunks before they are wanted, and from there
// through an LDS place of the wave's own into operands.  (Loaded as operands,
// sixteen rows of 16 bytes at a time, they arrive at 8.9 TB/s from the caches,
// whole lines at 25.)  Eight waves a CU.
//   us at N = K = 2880: 512 dense rows 15.2, 2048 29.4, 4096 47.7, 16384 152 to
// 156 (1790 to 1750 TFLOP/s); 128 experts: 256 rows 172 and 1024 rows 213 (1.06 GB
// of weights at 5.0 TB/s), 16384 rows with N = 5760 602 to 633 (903 to 858 TFLOP/s,
// 2.4 GB of weights, rows and results at 3.9 TB/s: HBM and the matrix cores take
// turns).
template <int kRows, int kWaves>
struct Tiles {
  static constexpr int kN = 64 * kWaves;
  static constexpr int kAhead = kRows > 64 ? 1 : 2, kStages = kRows > 64 || kWaves < 4 ? 2 : 4;
  // a stage: the scales of the rows and of the waves' weights, the rows' 16-byte pieces
  static constexpr int kScales = kRows / 4 + 16, kSlots = kScales + kRows * 8, kOwn = 64 * 8;
  static_assert(kStages % kAhead == 0, "register sets repeat with the stages");
  static_assert((kStages * kSlots + kWaves * kOwn) * 16 <= 20 * 1024 * kWaves, "eight waves a CU");
};

// Piece p of row r of a subtile of sixteen lies at slot p ^ swizzle16(r): no two lanes that the LDS serves together
// (0-3, 12-15, 20-27; 4-11, 16-19, 28-31; and so on) read the same banks.
__device__ __forceinline__ int swizzle16(int row) {
  const int h = row >> 1;
  return (h & 1) | ((h >> 1) & 2) | ((h ^ (h << 1)) & 4);
}

// chunk(0), chunk(1), ... (as compile-time numbers) of every period from c0 on, and of what is left.  Whole periods
// have no exit: from a loop with exits inside, the compiler's waits would count the loads that are in flight at any of
// them.
template <int kPeriod, typename F>
__device__ __forceinline__ void all_chunks(int chunks, int& c0, F&& chunk) {
  for (; c0 + kPeriod <= chunks; c0 += kPeriod)
    each_of([&](auto at) __attribute__((always_inline)) { return chunk(at), true; },
            std::make_integer_sequence<int, kPeriod>{});
  each_of([&](auto at) __attribute__((always_inline)) {
    if (c0 + decltype(at)::value >= chunks) return false;  // uniform
    chunk(at);
    return true;
  }, std::make_integer_sequence<int, kPeriod - 1>{});
}

struct TileBuffers {
  __amdgpu_buffer_rsrc_t x, w, s;  // w: the wave's weight rows; s: the scales that it loads, of the rows or the weights
};

// The rows of a wave's 64 weight rows nw .. leave.
template <int kLive>
__device__ __forceinline__ void leave(const Fp8Args& a, const Tile& t, int nw, const f32x4 (&acc)[4][2 * kLive]) {
  const int lane = threadIdx.x & 63, lr = lane & 15, q = lane >> 4, N = a.N;
  // lane (row lr of a subtile of rows, q): features 16 q + 4 i + j of the wave's 64 in acc[i][.][j]
  const int n = nw + 16 * q;
  if (n >= N) return;
  const int have = min(16, N - n);
  float bias[16];
#pragma unroll
  for (int i = 0; i < 16; ++i)
    bias[i] = a.bias != nullptr ? mx::bf16_to_f32(a.bias[(size_t)t.e * N + min(n + i, N - 1)]) : 0.f;
  const bool whole = (N & 7) == 0;
#pragma unroll
  for (int cb = 0; cb < 2 * kLive; ++cb) {
    const int row = 16 * cb + lr;
    if (row >= t.rows) continue;
    uint16_t* y = a.y + (size_t)(t.row0 + row) * N + n;
    uint32_t d[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      d[i] = mx::pack_bf16x2_rne(acc[i >> 1][cb][2 * (i & 1)] + bias[2 * i],
                                 acc[i >> 1][cb][2 * (i & 1) + 1] + bias[2 * i + 1]);
    if (whole) {
      *reinterpret_cast<u32x4*>(y) = u32x4{d[0], d[1], d[2], d[3]};
      if (have > 8) *reinterpret_cast<u32x4*>(y + 8) = u32x4{d[4], d[5], d[6], d[7]};
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < have) y[i] = (uint16_t)(d[i >> 1] >> (16 * (i & 1)));
    }
  }
}

// A wave's share of a tile with kLive blocks of 32 rows; kWork: with weight rows, else it only loads its share of x.
// (Each instance to its end: where they met again, the compiler moved and spilled their sums.)
template <int kRows, int kWaves, int kLive, bool kWork>
__device__ __forceinline__ void run_tile(const Fp8Args& args, const Tile& tile, int nw,
                                         u32x4* const (&st)[Tiles<kRows, kWaves>::kStages], u32x4* own, const TileBuffers& r,
                                         int kb, int wave) {
  const int K = args.K;
  f32x4 acc[4][2 * kLive] = {};
  using T = Tiles<kRows, kWaves>;
  constexpr int kStages = T::kStages, kAhead = T::kAhead, kRound = 8 * kWaves;
  const int t = threadIdx.x, lane = t & 63, lr = lane & 15, q = lane >> 4;
  // this thread's piece of a round of kRound rows of x
  const int xrow = t >> 3, xpiece = (t & 7) ^ swizzle16(xrow & 15);
  const uint32_t xoff = __umul24(xrow, K) + 16 * xpiece;
  const int xleft = K - 1 - 16 * xpiece;  // a negative number for k past K is an offset past the buffer
  // the first waves load the rows' scales, the last the weights' for the four waves; the others repeat
  constexpr int kScaleWaves = kRows / 64;
  const int scale_part = wave == kWaves - 1 ? kScaleWaves : wave % kScaleWaves;
  const uint32_t soff = wave < kWaves - 1 ? __umul24(64 * scale_part + lane, 4 * kb)
                        : lane < kWaves   ? (64 * lane / kBlock) * 4 * kb
                                          : kDead;
  static_assert(kScaleWaves < kWaves, "waves for the scales");
  constexpr int kXRounds = 32 * kLive / kRound, kXLoads = kXRounds + 1, kWLoads = kWork ? 8 : 0;
  // where chunk c starts, as a number that the compiler does not know: it would keep offsets of its own for each of a
  // loop's chunks, in registers that are not there
  auto start_of = [](int c) __attribute__((always_inline)) {
    int k = c * kBlock;
    asm("" : "+s"(k));
    return k;
  };
  auto issue_x = [&](int k, int load, u32x4* to) __attribute__((always_inline)) {
    if (load < kXRounds) {
      const uint32_t o = (xoff + k) | ((uint32_t)(xleft - k) & kDead);
      load_lds16(r.x, to + T::kScales + wave * 64 + load * 64 * kWaves, o + (uint32_t)(kRound * load) * K);
    } else {
      const uint32_t o = (soff + ((uint32_t)k >> 5)) | ((uint32_t)(kb - 1 - k / kBlock) & kDead);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r.s, (__attribute__((address_space(3))) void*)(to + 16 * scale_part), 4,
                                               o, 0, 0, 0);
    }
  };
  // load j of a chunk's weights: eight rows, 8 j + lane / 8, whole lines
  const int wrow = lane >> 3;
  const uint32_t woff = __umul24(wrow, K) + 16 * (lane & 7);
  const int wleft = K - 1 - 16 * (lane & 7);
  u32x4 w[kAhead][8];
  auto issue_w = [&](int k, int j, u32x4& to) __attribute__((always_inline)) {
    const uint32_t o = (woff + k) | ((uint32_t)(wleft - k) & kDead);
    to = __builtin_amdgcn_raw_buffer_load_b128(r.w, o + (uint32_t)(8 * j) * K, 0, 0);
  };
  // weight row n = 16 (m / 4) + 4 i + m % 4 of the wave's 64 is operand row m of subtile i, so that a lane's outputs are
  // sixteen neighbours; in LDS rows of 8 pieces, swizzled by m
  const int put = wrow * 8 + ((lane & 7) ^ ((wrow >> 1) & 1));
  auto put_w = [&](int j, const u32x4& from) __attribute__((always_inline)) {
    own[64 * j + (put ^ (swizzle16(4 * (j >> 1))))] = from;
  };
  const int take = (16 * (lr >> 2) + (lr & 3)) * 8 + (q ^ swizzle16(lr));
  // piece q of a row of a subtile; the other half's is 4 pieces on
  const int xat = T::kScales + lr * 8 + (q ^ swizzle16(lr));

#pragma unroll
  for (int c = 0; c < kStages - 1; ++c) {
#pragma unroll
    for (int j = 0; j < kXLoads; ++j) issue_x(c * kBlock, j, st[c]);
    __builtin_amdgcn_sched_barrier(0);  // the waits count on this order
  }
  if constexpr (kWork) {
    u32x4 first[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) issue_w(0, j, first[j]);
#pragma unroll
    for (int c = 0; c < kAhead; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) issue_w((c + 1) * kBlock, j, w[(c + 1) % kAhead][j]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < 8; ++j) put_w(j, first[j]);
  }

  // a product's sums are taken up kLag products later, when they are there, a chunk's last ones in the next chunk
  constexpr int kSteps = 8 * kLive, kLag = kRows > 64 ? 2 : 4;
  f32x4 part[kLag] = {};
  float s[2] = {};
  auto take_up_step = [&](auto at) __attribute__((always_inline)) {
    constexpr int n = decltype(at)::value;
    take_up(acc[n % 4][n / 4], part[n % kLag], s[(n / 4) & 1]);
  };
  int c0 = 0;
  auto chunk = [&](auto at_chunk) __attribute__((always_inline)) {
    constexpr int p = decltype(at_chunk)::value;
    const int next_x = start_of(c0 + p + kStages - 1), next_w = start_of(c0 + p + 1 + kAhead);
    // x of this chunk is there; loads of the later chunks' x and weights may be on their way
    mxgemm::wait_loads_then_barrier<kWLoads + (kStages - 2) * (kXLoads + kWLoads)>();
    u32x4* const to = st[(p + kStages - 1) % kStages];
    if constexpr (!kWork) {
#pragma unroll
      for (int j = 0; j < kXLoads; ++j) issue_x(next_x, j, to);
    } else {
      const u32x4* from = st[p];
      const float* sc = reinterpret_cast<const float*>(from);
      u32x4 a[4][2], b[2][2];
      float raw[2];
      int x0 = xat, x1 = xat ^ 4, row = lr;
      if constexpr (kRows <= 64) asm("" : "+v"(x0), "+v"(x1), "+v"(row));  // (as above: no addresses for each stage)
      auto read = [&](int cb) __attribute__((always_inline)) {
        b[cb & 1][0] = from[x0 + cb * 128];
        b[cb & 1][1] = from[x1 + cb * 128];
        raw[cb & 1] = sc[16 * cb + row];
      };
      read(0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i][0] = own[take + 32 * i];
        a[i][1] = own[(take ^ 4) + 32 * i];
      }
      const float wscale = sc[kRows + wave];
      __builtin_amdgcn_sched_barrier(0);
      // once the operands are read, the next chunk's weights take their place in LDS
      each_of([&](auto at) __attribute__((always_inline)) {
        constexpr int n = decltype(at)::value, i = n % 4, cb = n / 4;
        if constexpr (n % 4 == kLag % 4 && n >= kLag) s[((n - kLag) / 4) & 1] = raw[((n - kLag) / 4) & 1] * wscale;
        if constexpr (i == 0 && cb + 1 < 2 * kLive) read(cb + 1);
        take_up_step(std::integral_constant<int, n >= kLag ? n - kLag : kSteps - kLag + n>{});
        part[n % kLag] = multiply(a[i][0], a[i][1], b[cb & 1][0], b[cb & 1][1]);
        // (all of x before the weights: the wait above counts on it)
        constexpr int kFirstW = kLive > 1 ? kXLoads : 0;
        if constexpr (kLive == 1 && n == 0) {
#pragma unroll
          for (int j = 0; j < kXLoads; ++j) issue_x(next_x, j, to);
          __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (kLive > 1 && n < kXLoads) issue_x(next_x, n, to);
        if constexpr (n >= kFirstW && n < kFirstW + 8) {
          put_w(n - kFirstW, w[(p + 1) % kAhead][n - kFirstW]);
          issue_w(next_w, n - kFirstW, w[(p + 1) % kAhead][n - kFirstW]);
        }
        __builtin_amdgcn_sched_barrier(0);
        return true;
      }, std::make_integer_sequence<int, kSteps>{});
      if constexpr (kLag == 4) s[(2 * kLive - 1) & 1] = raw[(2 * kLive - 1) & 1] * wscale;
    }
  };
  if constexpr (kRows > 64) {
    // (two at least, and a copy for one more: with a loop that may not run the registers do not suffice; a chunk past K
    // adds zeros)
    do {
      each_of([&](auto at) __attribute__((always_inline)) { return chunk(at), true; },
              std::make_integer_sequence<int, kStages>{});
      c0 += kStages;
    } while (c0 + kStages <= kb);
    if (c0 < kb) chunk(std::integral_constant<int, 0>{});
  } else {
    all_chunks<kStages>(kb, c0, chunk);
  }
  if constexpr (kWork)
    each_of([&](auto at) __attribute__((always_inline)) {
      take_up_step(std::integral_constant<int, kSteps - kLag + decltype(at)::value>{});
      return true;
    }, std::make_integer_sequence<int, kLag>{});
  mxgemm::wait_loads_then_barrier<0>();  // no load still writes LDS
  if constexpr (kWork) leave<kLive>(args, tile, nw, acc);
}

template <int kRows, int kWaves>
__global__ __launch_bounds__(64 * kWaves, 2) void fp8_linear_tile_kernel(Fp8Args a) {
  using T = Tiles<kRows, kWaves>;
  __shared__ __attribute__((aligned(16))) u32x4 own[kWaves * T::kOwn];
  __shared__ __attribute__((aligned(16))) u32x4 st0[T::kSlots], st1[T::kSlots];
  const int n_tiles = (a.N + T::kN - 1) / T::kN;
  int nt;
  Tile t;
  if (!find_block(a, a.tile_rows, n_tiles, t, nt)) return;  // uniform per block
  const int K = a.K, N = a.N, n0 = nt * T::kN, kb = (K + kBlock - 1) / kBlock, nb = (N + kBlock - 1) / kBlock;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), nw = n0 + wave * 64;
  const bool work = nw < N;  // uniform
  const TileBuffers r{
      buffer(static_cast<const uint8_t*>(a.x) + (size_t)t.row0 * K, (uint32_t)t.rows * K),
      buffer(a.w + ((size_t)t.e * N + (work ? nw : 0)) * K, (uint32_t)min(64, N - (work ? nw : 0)) * K),
      wave == kWaves - 1
          ? buffer(a.w_scales + ((size_t)t.e * nb + n0 / kBlock) * kb, (uint32_t)(nb - n0 / kBlock) * kb * 4)
          : buffer(a.x_scales + (size_t)t.row0 * kb, (uint32_t)t.rows * kb * 4)};
  const int live = (t.rows + 31) >> 5;
  auto run = [&](u32x4* const (&st)[T::kStages]) __attribute__((always_inline)) {
    u32x4* const mine = own + wave * T::kOwn;
#define MX_CHUNKS(LIVE)                                                             \
  do {                                                                              \
    if (work) run_tile<kRows, kWaves, LIVE, true>(a, t, nw, st, mine, r, kb, wave); \
    else run_tile<kRows, kWaves, LIVE, false>(a, t, nw, st, mine, r, kb, wave);     \
  } while (0)
    if constexpr (kRows > 64) {
      if (live > 3) MX_CHUNKS(4);
      else if (live > 2) MX_CHUNKS(3);
    }
    if (live == 2) MX_CHUNKS(2);
    else if (live < 2) MX_CHUNKS(1);
#undef MX_CHUNKS
  };
  if constexpr (T::kStages == 2) {
    u32x4* const st[] = {st0, st1};
    run(st);
  } else {
    static_assert(T::kStages == 4, "stages are arrays of their own");
    __shared__ __attribute__((aligned(16))) u32x4 st2[T::kSlots], st3[T::kSlots];
    u32x4* const st[] = {st0, st1, st2, st3};
    run(st);
  }
}

template <int kRows, int kWaves>
hipError_t launch_tiles(Fp8Args a, int rows, hipStream_t stream) {
  using T = Tiles<kRows, kWaves>;
  a.tile_rows = rows;
  a.max_tiles = max_tiles(a, rows);
  fp8_linear_tile_kernel<kRows, kWaves>
      <<<grid_of(a.max_tiles, (a.N + T::kN - 1) / T::kN), 64 * kWaves, 0, stream>>>(a);
  return hipGetLastError();
}

// dx for row tiles of up to 64: 32x32x16 bf16 MFMA, a block of four waves makes
// 256 k x 64 rows, each wave 64 x 64, in chunks of 64 weight rows n; two of
// them are the span of a scale, added up in sums of their own.  The weights'
// bytes and dy travel into rings of LDS stages by the load unit.  The A operand
// needs eight n of one k, so the codes are read transposed: of a group of
// sixteen lanes each reads eight bytes of one of eight rows
// (ds_read_b64_tr_b8), and lane c gets byte c of the eight rows.  A half chunk's
// operands are read while the products of the other are made, and a product's A
// operand is converted while the one before runs.  Two blocks a CU.
//   us at N = K = 2880: 512 dense rows 24.8, 2048 43, 16384 267 (1020 TFLOP/s, the
// matrix cores busy for 52% of the cycles at 1.88 GHz); 128 experts: 256 rows 166
// and 1024 rows 187 (1.06 GB of weights at 5.7 TB/s), 16384 rows 404.  Rows of dy
// that no 16 bytes divide travel through registers, element by element: 2048
// rows at N = 2876 93 us.
constexpr int kBackK = 256, kBackRows = 64, kBackStages = 3;
constexpr int kCodeSlots = 1024, kDSlots = kBackRows * 8;  // 16-byte slots of a stage: 64 n x 256 codes, 64 rows x 64 n
constexpr int kWSlots = kCodeSlots + 4 * 16;              // ... and the codes' scale for each wave, 64 times

typedef __attribute__((__vector_size__(2 * sizeof(int)))) int i32x2;
using mx::f32x16;

__device__ __forceinline__ u32x4 fp8x8_to_bf16x8(i32x2 v) {
  return u32x4{fp8x2_to_bf16x2<0>(v[0]), fp8x2_to_bf16x2<1>(v[0]), fp8x2_to_bf16x2<0>(v[1]), fp8x2_to_bf16x2<1>(v[1])};
}

constexpr int kOutStride = 72;  // bf16 per row of a wave's outputs in LDS: 64 and padding

// The rows of a wave's 64 k leave through `out`, LDS that nothing else uses any more.
template <int kLive>
__device__ __forceinline__ void leave_back(const Fp8Args& a, const Tile& t, int kw, uint16_t* out, const f32x16 (&acc)[2][kLive]) {
  // lane (row lane & 31 of the block, half): k = 32 r + 8 i + 4 half + j of the wave's 64 in acc[r][.][4 i + j]
  const int lane = threadIdx.x & 63, half = lane >> 5, lrow = lane & 31, K = a.K;
#pragma unroll
  for (int cb = 0; cb < kLive; ++cb) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint2*>(out + lrow * kOutStride + 32 * r + 8 * i + 4 * half) = mxgemm::pack_bf16x4(
            f32x4{acc[r][cb][4 * i], acc[r][cb][4 * i + 1], acc[r][cb][4 * i + 2], acc[r][cb][4 * i + 3]});
    asm volatile("" ::: "memory");  // a wave's own LDS traffic is in order
    const int rows = min(32, t.rows - cb * 32);
    uint16_t* dx = a.y + (size_t)(t.row0 + cb * 32) * K + kw;
    for (int p = lane; p < rows * 8; p += 64) {
      const int r = p >> 3, col = (p & 7) * 8;
      if (kw + col < K)
        *reinterpret_cast<u32x4*>(dx + (size_t)r * K + col) = *reinterpret_cast<const u32x4*>(out + r * kOutStride + col);
    }
    asm volatile("" ::: "memory");
  }
}

// A wave's share of a tile with kLive blocks of 32 rows, as above.
template <int kLive, bool kAligned, bool kWork>
__device__ __forceinline__ void run_back(const Fp8Args& args, const Tile& tile, u32x4* const (&dst)[kBackStages],
                                         u32x4* const (&wst)[kBackStages], const __amdgpu_buffer_rsrc_t& rd,
                                         const __amdgpu_buffer_rsrc_t& rw, int k0, int wave) {
  const int K = args.K, N = args.N, kb = (K + kBlock - 1) / kBlock, kw = k0 + 64 * wave;
  f32x16 acc[2][kLive] = {};
  const int t = threadIdx.x, lane = t & 63, half = lane >> 5, lrow = lane & 31, mg = (lane >> 4) & 1, c16 = lane & 15;
  const int chunks = (N + 63) >> 6, nb = (chunks + 1) >> 1;
  const auto rs = buffer(args.w_scales + (size_t)tile.e * nb * kb, (uint32_t)nb * kb * 4);
  const uint32_t soff = 4 * (min(kw, K - 1) / kBlock);
  // this thread's pieces of a stage: of dy row pr (of 32), of weight row t / 16 (of 16)
  const int pr = t >> 3, part_d = (t & 7) ^ swizzle(pr);
  const uint32_t doff = (uint32_t)pr * N * 2 + 16 * part_d;
  const int dleft = N - 1 - 8 * part_d;  // a negative number for n past N is an offset past the buffer
  const uint32_t woff = (uint32_t)(t >> 4) * K + k0 + 16 * ((t & 15) ^ (((t >> 4) & 7) << 1));
  constexpr int kLoads = kAligned ? 5 + kLive : 5;
  u32x4 dreg[kLive];
  auto load_dy = [&](int c) __attribute__((always_inline)) {
    const int n = 64 * c + 8 * part_d;
#pragma unroll
    for (int k = 0; k < kLive; ++k) {
      uint32_t e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        e[i] = __builtin_amdgcn_raw_buffer_load_b16(rd, n + i < N ? ((uint32_t)(pr + 32 * k) * N + n + i) * 2 : kDead, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) dreg[k][i] = e[2 * i] | (e[2 * i + 1] << 16);
    }
  };
  auto store_dy = [&](u32x4* st) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < kLive; ++k) st[t + k * 256] = dreg[k];
  };
  auto issue = [&](int c, u32x4* d, u32x4* w) __attribute__((always_inline)) {  // past N: zeros
#pragma unroll
    for (int k = 0; k < 4; ++k) load_lds16(rw, w + wave * 64 + k * 256, woff + (uint32_t)(64 * c + 16 * k) * K);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(w + kCodeSlots + wave * 16), 4,
                                             soff + 4 * __umul24(c >> 1, kb), 0, 0, 0);
    if constexpr (kAligned) {
      const uint32_t o = (doff + 128 * c) | ((uint32_t)(dleft - 64 * c) & kDead);
#pragma unroll
      for (int k = 0; k < kLive; ++k) load_lds16(rd, d + wave * 64 + k * 256, o + (uint32_t)(k * 32) * N * 2);
    }
  };
  if (!kAligned) {
    load_dy(0);
    store_dy(dst[0]);
  }
#pragma unroll
  for (int c = 0; c < kBackStages; ++c) {
    __builtin_amdgcn_sched_barrier(0);  // the waits count on this order
    issue(c, dst[c], wst[c]);
  }
  int boff[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) boff[s] = lrow * 8 + ((2 * s + half) ^ swizzle(lrow));
  // codes: this lane's address for row i = c16 / 2 of the eight of a step, byte 8 (c16 & 1) of the wave's piece 2 r + mg
  const int ai = c16 >> 1;
  int aoff[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) aoff[r] = (8 * half + ai) * 256 + (((wave * 4 + 2 * r + mg) ^ (ai << 1)) * 16) + 8 * (c16 & 1);

  // operands of a half chunk, read while the other half's products are made
  u32x4 b[2][2][kLive];
  i32x2 w[2][2][2];
  auto read = [&](auto at_half, int stage) __attribute__((always_inline)) {
    constexpr int h = decltype(at_half)::value;
    const u32x4* base = dst[stage];
    const uint8_t* codes = reinterpret_cast<const uint8_t*>(wst[stage]);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
        w[h][s][r] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (__attribute__((address_space(3))) i32x2*)(codes + aoff[r] + (2 * h + s) * 16 * 256));
#pragma unroll
      for (int cb = 0; cb < kLive; ++cb) b[h][s][cb] = base[boff[2 * h + s] + cb * 256];
    }
  };
  f32x16 part[2][kLive] = {};
  float wscale = 0.f;
  auto take_up_block = [&](int r, int cb) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[r][cb][i] = __builtin_fmaf(part[r][cb][i], wscale, acc[r][cb][i]);
  };
  // The products of a half chunk; the next A operand is converted while one runs.  first: they open a block of 128 n, and
  // the sums of the last block are taken up.
  u32x4 op;
  auto multiply_half = [&](auto at_half, bool first) __attribute__((always_inline)) {
    constexpr int h = decltype(at_half)::value;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int s = j >> 1, r = j & 1;
      const bf16x8 now = mx::as_bf16x8(op);
#pragma unroll
      for (int cb = 0; cb < kLive; ++cb) {
        if (first && s == 0) take_up_block(r, cb);
        part[r][cb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(now, mx::as_bf16x8(b[h][s][cb]),
                                                              first && s == 0 ? f32x16{} : part[r][cb], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
        if (cb == 0) op = fp8x8_to_bf16x8(j < 3 ? w[h][(j + 1) >> 1][(j + 1) & 1] : w[1 - h][0][0]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr std::integral_constant<int, 0> kFirst{};
  constexpr std::integral_constant<int, 1> kSecond{};
  mxgemm::wait_loads_then_barrier<(kBackStages - 1) * kLoads>();
  if constexpr (kWork) {
    read(kFirst, 0);
    op = fp8x8_to_bf16x8(w[0][0][0]);
  }
  int c0 = 0;
  auto chunk = [&](auto at) __attribute__((always_inline)) {
    constexpr int p = decltype(at)::value, stage = p % kBackStages, next = (p + 1) % kBackStages;
    const int c = c0 + p;
    if constexpr (kWork) {
      read(kSecond, stage);
      __builtin_amdgcn_sched_barrier(0);
      multiply_half(kFirst, p % 2 == 0);
      if constexpr (p % 2 == 0) wscale = *reinterpret_cast<const float*>(wst[stage] + kCodeSlots + wave * 16);
    }
    if (!kAligned) {
      load_dy(c + 1);
      store_dy(dst[next]);
    }
    // the next chunk is there, and no wave still reads this one
    mxgemm::wait_loads_then_barrier<(kBackStages - 2) * kLoads>();
    if constexpr (kWork) {
      read(kFirst, next);
      __builtin_amdgcn_sched_barrier(0);
    }
    int ahead = __builtin_amdgcn_readfirstlane(c + kBackStages);
    asm("" : "+s"(ahead));  // (as above: no offsets for each of a period's chunks)
    issue(ahead, dst[stage], wst[stage]);
    if constexpr (kWork) multiply_half(kSecond, false);
  };
  all_chunks<2 * kBackStages>(chunks, c0, chunk);
  mxgemm::wait_loads_then_barrier<0>();  // no load still writes LDS, no wave still reads it
  if constexpr (kWork) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int cb = 0; cb < kLive; ++cb) take_up_block(r, cb);
    static_assert(32 * kOutStride * sizeof(uint16_t) <= kWSlots * 16, "a wave's rows fit in a stage");
    static_assert(32 * kOutStride * sizeof(uint16_t) <= kDSlots * 16, "... of dy as well");
    u32x4* const out = wave == 0 ? wst[0] : wave == 1 ? wst[1] : wave == 2 ? wst[2] : dst[0];
    leave_back<kLive>(args, tile, kw, reinterpret_cast<uint16_t*>(out), acc);
  }
}

template <bool kAligned>
__global__ __launch_bounds__(256, 2) void fp8_linear_backward_tile_kernel(Fp8Args a) {
  __shared__ __attribute__((aligned(16))) u32x4 w0[kWSlots], w1[kWSlots], w2[kWSlots];
  __shared__ __attribute__((aligned(16))) u32x4 d0[kDSlots], d1[kDSlots], d2[kDSlots];
  const int k_tiles = (a.K + kBackK - 1) / kBackK;
  int kt;
  Tile t;
  if (!find_block(a, kBackRows, k_tiles, t, kt)) return;  // uniform per block
  const int K = a.K, N = a.N, k0 = kt * kBackK;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool work = k0 + wave * 64 < K;  // uniform: a wave past K only loads its share
  const auto rd = buffer(static_cast<const uint16_t*>(a.x) + (size_t)t.row0 * N, (uint32_t)t.rows * N * 2);
  const auto rw = buffer(a.w + (size_t)t.e * N * K, (uint32_t)N * K);
  u32x4* const dst[] = {d0, d1, d2};
  u32x4* const wst[] = {w0, w1, w2};
  if (t.rows > 32) {
    if (work) run_back<2, kAligned, true>(a, t, dst, wst, rd, rw, k0, wave);
    else run_back<2, kAligned, false>(a, t, dst, wst, rd, rw, k0, wave);
  } else {
    if (work) run_back<1, kAligned, true>(a, t, dst, wst, rd, rw, k0, wave);
    else run_back<1, kAligned, false>(a, t, dst, wst, rd, rw, k0, wave);
  }
}

template <int kR, int kG>
hipError_t launch_few(Fp8Args a, hipStream_t stream) {
  a.max_tiles = max_tiles(a, 16 * kR);
  const int chunks = (a.K + kBlock - 1) / kBlock, waves = chunks < 8 ? chunks : 8, c = (chunks + waves - 1) / waves;
  constexpr int c_most = kG + kR > 5 ? 2 : 3;  // what the registers hold
  const dim3 grid = grid_of(a.max_tiles, ((int64_t)a.N + 16 * kG - 1) / (16 * kG));
  const size_t lds = (size_t)waves * kG * kR * 64 * sizeof(f32x4);  // 64 KB at most
  if (c == 1) fp8_linear_few_kernel<1, kG, kR><<<grid, waves * 64, lds, stream>>>(a);
  else if (c == 2) fp8_linear_few_kernel<2, kG, kR><<<grid, waves * 64, lds, stream>>>(a);
  else fp8_linear_few_kernel<c_most, kG, kR><<<grid, waves * 64, lds, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_back_tiles(Fp8Args a, hipStream_t stream) {
  a.max_tiles = max_tiles(a, kBackRows);
  const dim3 grid = grid_of(a.max_tiles, (a.K + kBackK - 1) / kBackK);
  if (a.N % 8 == 0) fp8_linear_backward_tile_kernel<true><<<grid, 256, 0, stream>>>(a);
  else fp8_linear_backward_tile_kernel<false><<<grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_back_few(Fp8Args a, hipStream_t stream) {
  a.max_tiles = max_tiles(a, kBackFewRows);
  const int blocks = (int)mx8::blocks_of(a.N), waves = blocks < 8 ? blocks : 8;
  const dim3 grid = grid_of(a.max_tiles, (a.K + kBackFewK - 1) / kBackFewK);
  const size_t lds = (size_t)waves * 64 * kRedStride * sizeof(float);
  if (a.N % 2 == 0) fp8_linear_backward_few_kernel<true><<<grid, waves * 64, lds, stream>>>(a);
  else fp8_linear_backward_few_kernel<false><<<grid, waves * 64, lds, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

namespace mxfp4moe {

hipError_t launch_fp8_linear(const uint8_t* x, const float* x_scales, const uint8_t* w, const float* w_scales,
                             const uint16_t* bias, const int32_t* offsets, int64_t R, int64_t K, int64_t N, int64_t E,
                             uint16_t* y, hipStream_t stream) {
  if (R == 0) return hipSuccess;
  Fp8Args a{x, x_scales, w, w_scales, bias, offsets, y, (int)R, (int)K, (int)N, (int)E, 0, 0};
  ProfileScope prof(kStageFp8Linear, stream);
  const mxfp8::Plan p = mxfp8::plan_forward(R, N, E, device_cu_count());
  if (p.few) {
    if (p.rows == 16) return launch_few<1, 1>(a, stream);
    return p.cols == 32 ? launch_few<2, 2>(a, stream) : launch_few<2, 4>(a, stream);
  }
  if (p.rows == 128) return launch_tiles<128, 4>(a, 128, stream);
  return p.cols == 256 ? launch_tiles<64, 4>(a, 64, stream) : launch_tiles<64, 2>(a, p.rows, stream);
}

hipError_t launch_fp8_linear_backward(const uint16_t* dy, const uint8_t* w, const float* w_scales,
                                      const int32_t* offsets, int64_t R, int64_t K, int64_t N, int64_t E, uint16_t* dx,
                                      hipStream_t stream) {
  if (R == 0) return hipSuccess;
  Fp8Args a{dy, nullptr, w, w_scales, nullptr, offsets, dx, (int)R, (int)K, (int)N, (int)E, 0, 0};
  ProfileScope prof(kStageFp8LinearBackward, stream);
  return mxfp8::backward_has_few(R, K, E, device_cu_count()) ? launch_back_few(a, stream) : launch_back_tiles(a, stream);
}

}  // namespace mxfp4moe
