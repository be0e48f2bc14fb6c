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
  int tile_rows;           // rows of a tile (the 128-row kernels: 128, 64 or 32)
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

// y for row tiles of at most 16 rows: weights as the A operand, straight to
// registers, x rows as B.  The waves of a block split K, kC blocks of 128 each
// at a time (all loads of a wave in flight before the first product), for kG *
// 16 weight rows; their sums meet in LDS, added in wave order.  Loads past K,
// N or the tile's rows return zero from the buffer's bounds.
constexpr int kFewRows = 16;

template <int kC, int kG>
__global__ __launch_bounds__(512) void fp8_linear_few_kernel(Fp8Args a) {
  extern __shared__ f32x4 red[];
  const int n_chunks = (a.N + 16 * kG - 1) / (16 * kG);
  int ti, nc;
  if (!map_block(a.max_tiles, n_chunks, ti, nc)) return;  // uniform per block
  Tile t;
  if (!find_tile(a, kFewRows, ti, t)) return;
  const int K = a.K, N = a.N, n0 = nc * 16 * kG, kb = (K + kBlock - 1) / kBlock;
  const int lane = mx::lane_id(), lr = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const auto rx = buffer(static_cast<const uint8_t*>(a.x) + (size_t)t.row0 * K, (uint32_t)t.rows * K);
  const auto rw = buffer(a.w + ((size_t)t.e * N + n0) * K, (uint32_t)min(16 * kG, N - n0) * K);
  const float* xs = a.x_scales + (size_t)(t.row0 + min(lr, t.rows - 1)) * kb;
  const float* ws = a.w_scales + ((size_t)t.e * mx8::blocks_of(N) + n0 / kBlock) * kb;

  f32x4 acc[kG] = {};
  for (int c0 = wave * kC; c0 < kb; c0 += waves * kC) {
    u32x4 x[kC][2], w[kG][kC][2];
    float s[kC];
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      const int k = (c0 + j) * kBlock + 16 * q;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = k + 64 * h < K;
#pragma unroll
        for (int i = 0; i < kG; ++i)
          w[i][j][h] = __builtin_amdgcn_raw_buffer_load_b128(rw, in ? (uint32_t)(lr + 16 * i) * K + k + 64 * h : kDead, 0, 0);
        x[j][h] = __builtin_amdgcn_raw_buffer_load_b128(rx, in ? (uint32_t)lr * K + k + 64 * h : kDead, 0, 0);
      }
      const int c = min(c0 + j, kb - 1);
      s[j] = xs[c] * ws[c];
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      if (c0 + j >= kb) break;  // uniform
#pragma unroll
      for (int i = 0; i < kG; ++i) {
        take_up(acc[i], multiply(w[i][j][0], w[i][j][1], x[j][0], x[j][1]), s[j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kG; ++i) red[(wave * kG + i) * 64 + lane] = acc[i];
  __syncthreads();
  for (int i = wave; i < kG; i += waves) {
    f32x4 v = red[i * 64 + lane];
    for (int u = 1; u < waves; ++u) v += red[(u * kG + i) * 64 + lane];
    const int n = n0 + 16 * i + 4 * q;  // lane (row lr of the tile, q): features n .. n + 3
    if (lr >= t.rows || n >= N) continue;
    const uint16_t* bias = a.bias != nullptr ? a.bias + (size_t)t.e * N + n : nullptr;
    store4(a.y + (size_t)(t.row0 + lr) * N + n, v, bias, min(4, N - n), (N & 3) == 0);
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
// take every waves-th block of 128 n and add their sums in LDS in wave order.
constexpr int kBackFewK = 64;
constexpr int kRedStride = 20;  // floats per lane in LDS: 16 and padding

template <bool kAligned>
__global__ __launch_bounds__(512) void fp8_linear_backward_few_kernel(Fp8Args a) {
  extern __shared__ float redf[];
  const int k_chunks = (a.K + kBackFewK - 1) / kBackFewK;
  int ti, kc;
  if (!map_block(a.max_tiles, k_chunks, ti, kc)) return;  // uniform per block
  Tile t;
  if (!find_tile(a, kFewRows, ti, t)) return;
  const int K = a.K, N = a.N, k0 = kc * kBackFewK, kb = (K + kBlock - 1) / kBlock, nb = (N + kBlock - 1) / kBlock;
  const int lane = mx::lane_id(), m = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const auto rw = buffer(a.w + (size_t)t.e * N * K, (uint32_t)N * K);
  const uint16_t* dy0 = static_cast<const uint16_t*>(a.x) + (size_t)t.row0 * N;
  const auto rd = buffer(dy0, (uint32_t)t.rows * N * 2);
  const float* ws = a.w_scales + (size_t)t.e * nb * kb + k0 / kBlock;
  const int row = min(m, t.rows - 1);  // columns past the tile's rows are dropped
  const uint32_t col = k0 + 4 * m;

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

// y for row tiles of up to 128: 16x16x128 MFMA, a block of four waves makes 256
// weight rows x 128 rows, each wave 64 x 128, in chunks of 128 k, the span of a
// scale.  No wave shares its weights, so they go straight to registers, two
// chunks ahead of their use; x travels into a ring of three LDS stages by the
// load unit, with the chunk's 128 row scales.  Two blocks a CU.
constexpr int kTileRows = 128, kTileN = 256, kStages = 4;
constexpr int kScaleSlots = kTileRows / 4;  // a stage: the scales of the rows, then their 16-byte pieces, swizzled
constexpr int kStageSlots = kScaleSlots + kTileRows * 8;

template <int kLive>
__device__ __forceinline__ void tile_chunks(f32x4 (&acc)[4][kTileRows / 16], u32x4* const (&xst)[kStages],
                                            const __amdgpu_buffer_rsrc_t& rx,
                                            const __amdgpu_buffer_rsrc_t (&rw)[4], const __amdgpu_buffer_rsrc_t& rs,
                                            const ScalarFloats ws, int K, int kb, int wave, bool work) {
  const int t = threadIdx.x, lane = t & 63, lr = lane & 15, q = lane >> 4;
  // this thread's piece of a round of 32 rows of x
  const int xr = t >> 3, xpart = (t & 7) ^ swizzle(xr & 15);
  const uint32_t xoff = __umul24(xr, K) + 16 * xpart;
  const uint32_t woff = __umul24(16 * (lr >> 2) + (lr & 3), K) + 16 * q;
  const uint32_t soff = __umul24(64 * (wave & 1) + lane, 4 * kb);  // (waves 2 and 3 repeat what 0 and 1 load)
  // a negative number for k past K is an offset past the buffer
  const int xleft = K - 1 - 16 * xpart, wleft = K - 1 - 16 * q;
  auto issue_x = [&](int c, u32x4* st) __attribute__((always_inline)) {
    const uint32_t o = (xoff + c * kBlock) | ((uint32_t)(xleft - c * kBlock) & kDead);
#pragma unroll
    for (int k = 0; k < kLive; ++k) load_lds16(rx, st + kScaleSlots + wave * 64 + k * 256, o + (uint32_t)(32 * k) * K);
    // (past the last chunk: the next row's, of no use)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(st + 16 * (wave & 1)), 4,
                                             soff + 4 * c, 0, 0, 0);
  };
  u32x4 w[2][4][2];
  auto issue_w = [&](int c, u32x4 (&r)[4][2]) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = c * kBlock + 64 * h;
      const uint32_t o = (woff + k) | ((uint32_t)(wleft - k) & kDead);
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i][h] = __builtin_amdgcn_raw_buffer_load_b128(rw[i], o, 0, 0);
    }
  };
  constexpr int kXLoads = kLive + 1, kWLoads = 8;
  issue_x(0, xst[0]);
  issue_w(0, w[0]);
  __builtin_amdgcn_sched_barrier(0);  // the waits count on this order
  issue_x(1, xst[1]);
  issue_w(1, w[1]);
  float wscale = ws[0];
  // piece q of row lr of a subtile; the other half's is 4 pieces on
  const int b0 = lr * 8 + (q ^ swizzle(lr)), b1 = b0 ^ 4;

  int c0 = 0;
  auto chunk = [&](auto at) __attribute__((always_inline)) {
    constexpr int p = decltype(at)::value;
    const int c = c0 + p;
    mxgemm::wait_loads_then_barrier<kXLoads + kWLoads>();
    issue_x(c + 2, xst[(p + 2) % kStages]);
    const float wnext = ws[min(c + 1, kb - 1)];
    const u32x4* xs = xst[p] + kScaleSlots;
    const float* sc = reinterpret_cast<const float*>(xst[p]);
    if (work && c < kb) {
      // a product's sums are taken up four products later, when they are there
      u32x4 b[2][2];
      f32x4 part[4];
      float s = 0.f, raw = sc[lr];
      b[0][0] = xs[b0];
      b[0][1] = xs[b1];
#pragma unroll
      for (int cb = 0; cb < 2 * kLive; ++cb) {
        const float before = s;
        s = raw * wscale;
        if (cb + 1 < 2 * kLive) {
          b[(cb + 1) & 1][0] = xs[b0 + (cb + 1) * 128];
          b[(cb + 1) & 1][1] = xs[b1 + (cb + 1) * 128];
          raw = sc[16 * (cb + 1) + lr];
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (cb > 0) take_up(acc[i][cb - 1], part[i], before);
          part[i] = multiply(w[p & 1][i][0], w[p & 1][i][1], b[cb & 1][0], b[cb & 1][1]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) take_up(acc[i][2 * kLive - 1], part[i], s);
    }
    wscale = wnext;
    __builtin_amdgcn_sched_barrier(0);
    issue_w(c + 2, w[p & 1]);
  };
  // Whole periods of the stages and the register sets, without an exit: from a loop with exits inside, the compiler's
  // waits would count the loads that are in flight at any of them.  Chunks past K load nothing and multiply nothing.
  for (; c0 < kb; c0 += kStages)
    each_of([&](auto at) __attribute__((always_inline)) { return chunk(at), true; },
            std::make_integer_sequence<int, kStages>{});
}

__global__ __launch_bounds__(256, 2) void fp8_linear_tile_kernel(Fp8Args a) {
  __shared__ __attribute__((aligned(16))) u32x4 x0[kStageSlots], x1[kStageSlots], x2[kStageSlots], x3[kStageSlots];
  const int n_tiles = (a.N + kTileN - 1) / kTileN;
  int ti, nt;
  if (!map_tile(a, a.tile_rows, n_tiles, ti, nt)) return;  // uniform per block
  Tile t;
  if (!find_tile(a, a.tile_rows, ti, t)) return;
  const int K = a.K, N = a.N, n0 = nt * kTileN, kb = (K + kBlock - 1) / kBlock;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, lr = lane & 15,
            q = lane >> 4;
  const int nw = n0 + wave * 64;
  const bool work = nw < N;  // uniform: a wave past N only loads its share of x
  const auto rx = buffer(static_cast<const uint8_t*>(a.x) + (size_t)t.row0 * K, (uint32_t)t.rows * K);
  // weight row of operand row lr and subtile i: 16 (lr / 4) + 4 i + lr % 4 of the wave's 64, so that a lane's outputs
  // are sixteen neighbours; a buffer for each i (a scalar offset could pass the bounds)
  __amdgpu_buffer_rsrc_t rw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int rows = max(min(64, N - nw) - 4 * i, 0);
    rw[i] = buffer(a.w + ((size_t)t.e * N + (rows > 0 ? nw + 4 * i : 0)) * K, (uint32_t)rows * K);
  }
  const auto rs = buffer(a.x_scales + (size_t)t.row0 * kb, (uint32_t)t.rows * kb * 4);
  const ScalarFloats ws =
      (ScalarFloats)(a.w_scales + ((size_t)t.e * mx8::blocks_of(N) + min(nw, N - 1) / kBlock) * kb);
  u32x4* const xst[] = {x0, x1, x2, x3};
  f32x4 acc[4][kTileRows / 16] = {};
  const int live = (t.rows + 31) >> 5;
  if (live == 4) tile_chunks<4>(acc, xst, rx, rw, rs, ws, K, kb, wave, work);
  else if (live == 3) tile_chunks<3>(acc, xst, rx, rw, rs, ws, K, kb, wave, work);
  else if (live == 2) tile_chunks<2>(acc, xst, rx, rw, rs, ws, K, kb, wave, work);
  else tile_chunks<1>(acc, xst, rx, rw, rs, ws, K, kb, wave, work);
  mxgemm::wait_loads_then_barrier<0>();  // no load still writes LDS
  if (!work) return;

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
  for (int cb = 0; cb < kTileRows / 16; ++cb) {
    if (cb >= 2 * live) break;
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

// dx for row tiles of up to 64: 32x32x16 bf16 MFMA, a block of four waves makes
// 256 k x 64 rows, each wave 64 x 64, in chunks of 64 weight rows n; two of
// them are the span of a scale, added up in sums of their own.  The weights'
// bytes and dy travel into rings of LDS stages by the load unit.  The A operand
// needs eight n of one k, so the codes are read transposed: of a group of
// sixteen lanes each reads eight bytes of one of eight rows
// (ds_read_b64_tr_b8), and lane c gets byte c of the eight rows.  Two blocks a
// CU.
constexpr int kBackK = 256, kBackRows = 64, kBackStages = 3;
constexpr int kWSlots = 1024, kDSlots = kBackRows * 8;  // 16-byte slots of a stage: 64 n x 256 codes, 64 rows x 64 n

typedef __attribute__((__vector_size__(2 * sizeof(int)))) int i32x2;
using mx::f32x16;

__device__ __forceinline__ u32x4 fp8x8_to_bf16x8(i32x2 v) {
  return u32x4{fp8x2_to_bf16x2<0>(v[0]), fp8x2_to_bf16x2<1>(v[0]), fp8x2_to_bf16x2<0>(v[1]), fp8x2_to_bf16x2<1>(v[1])};
}

template <int kLive, bool kAligned>
__device__ __forceinline__ void backward_chunks(f32x16 (&acc)[2][2], u32x4* const (&dst)[kBackStages],
                                                u32x4* const (&wst)[kBackStages], const __amdgpu_buffer_rsrc_t& rd,
                                                const uint16_t* dy, const __amdgpu_buffer_rsrc_t& rw,
                                                const ScalarFloats ws, int rows, int K, int N, int kb, int k0,
                                                int wave, bool work) {
  const int t = threadIdx.x, lane = t & 63, half = lane >> 5, lrow = lane & 31, mg = (lane >> 4) & 1, c16 = lane & 15;
  const int chunks = (N + 63) >> 6, nb = (chunks + 1) >> 1;
  // this thread's pieces of a stage: of dy row pr (of 32), of weight row t / 16 (of 16)
  const int pr = t >> 3, part_d = (t & 7) ^ swizzle(pr);
  const uint32_t doff = (uint32_t)pr * N * 2 + 16 * part_d;
  const uint32_t woff = (uint32_t)(t >> 4) * K + k0 + 16 * ((t & 15) ^ (((t >> 4) & 7) << 1));
  constexpr int kLoads = kAligned ? 4 + kLive : 4;
  u32x4 dreg[kLive];
  auto load_dy = [&](int c) __attribute__((always_inline)) {
    const int n = 64 * c + 8 * part_d;
#pragma unroll
    for (int k = 0; k < kLive; ++k)
      dreg[k] = load_dy8<false>(rd, dy + (size_t)min(pr + 32 * k, rows - 1) * N, 0, n, N, 64 * c + 64 <= N);
  };
  auto store_dy = [&](u32x4* st) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < kLive; ++k) st[t + k * 256] = dreg[k];
  };
  auto issue = [&](int c, u32x4* d, u32x4* w) __attribute__((always_inline)) {  // past N: zeros, or for dy the next row
#pragma unroll
    for (int k = 0; k < 4; ++k) load_lds16(rw, w + wave * 64 + k * 256, woff + (uint32_t)(64 * c + 16 * k) * K);
    if constexpr (kAligned) {
#pragma unroll
      for (int k = 0; k < kLive; ++k)
        load_lds16(rd, d + wave * 64 + k * 256, doff + (uint32_t)(k * 32) * N * 2 + c * 128);
    }
  };
  if (!kAligned) {
    load_dy(0);
    store_dy(dst[0]);
    load_dy(1);
  }
#pragma unroll
  for (int c = 0; c < kBackStages - 1; ++c) {
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

  f32x16 part[2][2];
  float wscale = ws[0];
  int c0 = 0;
  auto chunk = [&](auto at) __attribute__((always_inline)) {
    constexpr int p = decltype(at)::value, kOdd = p & 1;
    const int c = c0 + p;
    mxgemm::wait_loads_then_barrier<(kBackStages - 2) * kLoads>();
    if (!kAligned) {  // (every wave is past the stage that this one overwrites)
      store_dy(dst[(p + 1) % kBackStages]);
      load_dy(c + 2);
      __builtin_amdgcn_sched_barrier(0);
    }
    issue(c + kBackStages - 1, dst[(p + kBackStages - 1) % kBackStages], wst[(p + kBackStages - 1) % kBackStages]);
    if (kAligned && c == chunks - 1 && (N & 63) != 0) {  // uniform: dy past N becomes zeros as the weights there are
      uint16_t* stage = reinterpret_cast<uint16_t*>(dst[p % kBackStages]);
      for (int i = t; i < kLive * 32 * 64; i += 256) {
        const int r = i >> 6, col = i & 63;
        if (64 * c + col >= N) stage[r * 64 + 8 * ((col >> 3) ^ swizzle(r & 31)) + (col & 7)] = 0;
      }
      mxgemm::lds_reads_then_barrier();
    }
    if (work && c < chunks) {
      const u32x4* base = dst[p % kBackStages];
      const uint8_t* codes = reinterpret_cast<const uint8_t*>(wst[p % kBackStages]);
      u32x4 b[4][kLive];
      i32x2 w[4][2];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
          w[s][r] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
              (__attribute__((address_space(3))) i32x2*)(codes + aoff[r] + s * 16 * 256));
#pragma unroll
        for (int cb = 0; cb < kLive; ++cb) b[s][cb] = base[boff[s] + cb * 256];
      }
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const bf16x8 op = mx::as_bf16x8(fp8x8_to_bf16x8(w[s][r]));
#pragma unroll
          for (int cb = 0; cb < kLive; ++cb)
            part[r][cb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(op, mx::as_bf16x8(b[s][cb]),
                                                                  s == 0 && !kOdd ? f32x16{} : part[r][cb], 0, 0, 0);
        }
    }
    if constexpr (kOdd) {
      if (work && c - 1 < chunks) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int cb = 0; cb < kLive; ++cb)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[r][cb][i] = __builtin_fmaf(part[r][cb][i], wscale, acc[r][cb][i]);
      }
      wscale = ws[(size_t)min((c + 1) >> 1, nb - 1) * kb];
    }
  };
  // whole periods without an exit, as above
  for (; c0 < chunks; c0 += 2 * kBackStages)
    each_of([&](auto at) __attribute__((always_inline)) { return chunk(at), true; },
            std::make_integer_sequence<int, 2 * kBackStages>{});
}

constexpr int kOutStride = 72;  // bf16 per row of a wave's outputs in LDS: 64 and padding

template <bool kAligned>
__global__ __launch_bounds__(256, 2) void fp8_linear_backward_tile_kernel(Fp8Args a) {
  __shared__ __attribute__((aligned(16))) u32x4 w0[kWSlots], w1[kWSlots], w2[kWSlots];
  __shared__ __attribute__((aligned(16))) u32x4 d0[kDSlots], d1[kDSlots], d2[kDSlots];
  const int k_tiles = (a.K + kBackK - 1) / kBackK;
  int ti, kt;
  if (!map_tile(a, a.tile_rows, k_tiles, ti, kt)) return;  // uniform per block
  Tile t;
  if (!find_tile(a, a.tile_rows, ti, t)) return;
  const int K = a.K, N = a.N, k0 = kt * kBackK, kb = (K + kBlock - 1) / kBlock;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int kw = k0 + wave * 64;
  const bool work = kw < K;  // uniform: a wave past K only loads its share
  const uint16_t* dy = static_cast<const uint16_t*>(a.x) + (size_t)t.row0 * N;
  const auto rd = buffer(dy, (uint32_t)t.rows * N * 2);
  const auto rw = buffer(a.w + (size_t)t.e * N * K, (uint32_t)N * K);
  const ScalarFloats ws = (ScalarFloats)(a.w_scales + (size_t)t.e * mx8::blocks_of(N) * kb + min(kw, K - 1) / kBlock);
  u32x4* const dst[] = {d0, d1, d2};
  u32x4* const wst[] = {w0, w1, w2};
  f32x16 acc[2][2] = {};
  const int live = (t.rows + 31) >> 5;
  if (live == 2) backward_chunks<2, kAligned>(acc, dst, wst, rd, dy, rw, ws, t.rows, K, N, kb, k0, wave, work);
  else backward_chunks<1, kAligned>(acc, dst, wst, rd, dy, rw, ws, t.rows, K, N, kb, k0, wave, work);

  // lane (row lane & 31 of the block, half): k = 32 r + 8 i + 4 half + j of the wave's 64 in acc[r][.][4 i + j]
  mxgemm::wait_loads_then_barrier<0>();  // no load still writes LDS, no wave still reads it
  if (!work) return;                     // no barrier follows
  const int half = lane >> 5, lrow = lane & 31;
  static_assert(32 * kOutStride * sizeof(uint16_t) <= sizeof(w0), "a wave's rows fit in a stage");
  uint16_t* out = reinterpret_cast<uint16_t*>(wave == 0 ? w0 : wave == 1 ? w1 : wave == 2 ? w2 : d0);
#pragma unroll
  for (int cb = 0; cb < 2; ++cb) {
    if (cb >= live) break;
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

template <int kC>
hipError_t launch_few(Fp8Args a, int waves, hipStream_t stream) {
  // as many row groups to a block (x is read once for all) as leave two blocks for every CU
  a.max_tiles = max_tiles(a, kFewRows);
  const int64_t groups = ((int64_t)a.N + 15) / 16 * a.max_tiles, want = 2 * mxfp4moe::device_cu_count();
  const int g = groups >= 4 * want ? 4 : groups >= 2 * want ? 2 : 1;
  const dim3 grid = grid_of(a.max_tiles, ((int64_t)a.N + 16 * g - 1) / (16 * g));
  const size_t lds = (size_t)waves * g * 64 * sizeof(f32x4);
  if (g == 4) fp8_linear_few_kernel<kC, 4><<<grid, waves * 64, lds, stream>>>(a);
  else if (g == 2) fp8_linear_few_kernel<kC, 2><<<grid, waves * 64, lds, stream>>>(a);
  else fp8_linear_few_kernel<kC, 1><<<grid, waves * 64, lds, stream>>>(a);
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
  if (R > 16 * E) {
    a.tile_rows = 128;
    a.max_tiles = max_tiles(a, a.tile_rows);
    fp8_linear_tile_kernel<<<grid_of(a.max_tiles, (N + kTileN - 1) / kTileN), 256, 0, stream>>>(a);
    return hipGetLastError();
  }
  const int chunks = (int)mx8::blocks_of(K), waves = chunks < 8 ? chunks : 8;
  return (chunks + waves - 1) / waves <= 2 ? launch_few<2>(a, waves, stream) : launch_few<3>(a, waves, stream);
}

hipError_t launch_fp8_linear_backward(const uint16_t* dy, const uint8_t* w, const float* w_scales,
                                      const int32_t* offsets, int64_t R, int64_t K, int64_t N, int64_t E, uint16_t* dx,
                                      hipStream_t stream) {
  if (R == 0) return hipSuccess;
  Fp8Args a{dy, nullptr, w, w_scales, nullptr, offsets, dx, (int)R, (int)K, (int)N, (int)E, 0, 0};
  ProfileScope prof(kStageFp8LinearBackward, stream);
  if (R > 16 * E) {
    a.tile_rows = kBackRows;
    a.max_tiles = max_tiles(a, a.tile_rows);
    const dim3 grid = grid_of(a.max_tiles, (K + kBackK - 1) / kBackK);
    if (N % 2 == 0) fp8_linear_backward_tile_kernel<true><<<grid, 256, 0, stream>>>(a);
    else fp8_linear_backward_tile_kernel<false><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
  }
  a.max_tiles = max_tiles(a, kFewRows);
  const int blocks = (int)mx8::blocks_of(N), waves = blocks < 8 ? blocks : 8;
  const dim3 grid = grid_of(a.max_tiles, (K + kBackFewK - 1) / kBackFewK);
  const size_t lds = (size_t)waves * 64 * kRedStride * sizeof(float);
  if (N % 2 == 0) fp8_linear_backward_few_kernel<true><<<grid, waves * 64, lds, stream>>>(a);
  else fp8_linear_backward_few_kernel<false><<<grid, waves * 64, lds, stream>>>(a);
  return hipGetLastError();
}

}  // namespace mxfp4moe
