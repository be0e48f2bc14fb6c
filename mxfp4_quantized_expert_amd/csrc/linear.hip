// Rows times 4-bit weights with group scales, dense or per expert, and the
// gradient to the rows.
//
//   y[r, n]  = s2_e * sum_k x[r, k] W_e[n, k] + b_e[n]
//   dx[r, k] = s2_e * sum_n dy[r, n] W_e[n, k]
// for the rows r of expert e (expert_offsets; one expert without them), with
// W_e[n, k] = E2M1(code) * group scale: MXFP4 has an E8M0 scale per 32 k and
// s2 = 1, NVFP4 an E4M3 scale per 16 k and a float32 s2 per expert.  Formats
// and the order of scale and bias as in the fused layer ("feat(gguf): serve
// gpt-oss gguf checkpoints on gpt_oss", FreeToken PR #838, review item 3);
// the weights are frozen, so the rows are all that has a gradient.
//
// A code times its scale is exact in bf16 (two significant bits for MXFP4,
// at most six for NVFP4), so every product of the bf16 MFMA is exact and the
// sums are its fp32 accumulation; s2 and the bias follow in fp32 and the
// result is rounded once.
#include "expert_device.h"
#include "internal.h"
#include "linear_plan.h"
#include "mx_device.h"
#include "row_tiles.h"

namespace {

using namespace mxtiles;
using mx::bf16x8;
typedef __attribute__((__vector_size__(2 * sizeof(int)))) int i32x2;
using mx::f32x16;
using mx::f32x4;
using mx::u32x4;
using mxgemm::GroupScale;

struct LinearArgs {
  const uint16_t* x;        // forward: x [R, K]; gradient: dy [R, N]
  const uint8_t* blocks;    // [E, N, K/2]
  const uint8_t* scales;    // [E, N, K/32], NVFP4 [E, N, K/16]
  const float* scale2;      // [E] or nullptr
  const uint16_t* bias;     // [E, N] or nullptr
  const int32_t* offsets;   // [E + 1] or nullptr (E == 1, every row)
  uint16_t* y;              // forward: y [R, N]; gradient: dx [R, K]
  int R, K, N, E;
  int max_tiles;            // row tiles, at most
  int tile_rows;            // rows of a tile (the 128-row kernels: 128, 64 or 32)
};

// ---------------------------------------------------------------- few rows

// y for row tiles of at most 16 rows: 16x16x32 MFMA, weights as the A operand
// (16 weight rows), x rows as B.  A chunk is four groups (128 k): lane (r, q)
// holds group q of weight row r, one 16-byte load, whose dword s goes to step
// s with the x values of the same k; any agreed order of k gives the same
// sums.  The waves of a block split K, kC chunks each at a time (all loads of
// a wave in flight before the first product), and hold the sums of kG * 16
// weight rows; x stays in registers for those kG row groups.  The partial
// sums meet in LDS, added in wave order.  Loads past K, N or the tile's rows
// return zero from the buffer's bounds.  Bound: the weights' bytes from HBM,
// at 2.9 TB/s (224 rows over 32 experts, 2880 x 2880: 56 us, where tiles take
// 46), and for a single small matrix the latency of one pass (256 rows, N =
// 1024, K = 736: 4.6 us, of which an empty launch is 2.2; one row, 2880 x 2880:
// 4.6 us, where tiles of 4 rows take 5.0; 128 rows, 2880 x 2880: 14.6 us, where
// tiles take 17.5).
constexpr int kFewRows = mxlinear::kFewTileRows;

// Four consecutive outputs: s2 * v + bias, `n` of them in range (`whole`: always four, 8-byte aligned).
__device__ __forceinline__ void store4(uint16_t* out, f32x4 v, float s2, const uint16_t* bias, int n, bool whole) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    v[c] *= s2;
    if (bias != nullptr && c < n) v[c] += mx::bf16_to_f32(bias[c]);
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

template <bool kNv, int kC, int kG>
__global__ __launch_bounds__(512) void linear_few_kernel(LinearArgs a) {
  extern __shared__ f32x4 red[];
  const int n_chunks = (a.N + 16 * kG - 1) / (16 * kG);
  int ti, nc;
  if (!map_block(a.max_tiles, n_chunks, ti, nc)) return;  // uniform per block
  Tile t;
  if (!find_tile(a, kFewRows, ti, t)) return;
  const int K = a.K, N = a.N, kgroups = K >> 5, n0 = nc * 16 * kG;
  const int lane = mx::lane_id(), lr = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const size_t wrow0 = (size_t)t.e * N + n0;
  const int nrows = min(16 * kG, N - n0);
  const int kscales = kNv ? K >> 4 : kgroups;
  const auto rx = buffer(a.x + (size_t)t.row0 * K, (uint32_t)t.rows * K * 2);
  const auto rw = buffer(a.blocks + wrow0 * (K >> 1), (uint32_t)nrows * (K >> 1));
  const auto rs = buffer(a.scales + wrow0 * kscales, (uint32_t)nrows * kscales);

  f32x4 acc[kG] = {};
  const int per = waves * kC;
  for (int c0 = wave * kC; 4 * c0 < kgroups; c0 += per) {
    u32x4 xb[kC][4], w[kG][kC];
    uint32_t sc[kG][kC];
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      const int g = 4 * (c0 + j) + q;
#pragma unroll
      for (int i = 0; i < kG; ++i) {
        const uint32_t row = lr + 16 * i;
        w[i][j] = __builtin_amdgcn_raw_buffer_load_b128(rw, g < kgroups ? row * (K >> 1) + g * 16 : kDead, 0, 0);
        if (kNv)
          sc[i][j] = __builtin_amdgcn_raw_buffer_load_b16(rs, g < kgroups ? row * kscales + g * 2 : kDead, 0, 0);
        else
          sc[i][j] = __builtin_amdgcn_raw_buffer_load_b8(rs, g < kgroups ? row * kscales + g : kDead, 0, 0);
      }
#pragma unroll
      for (int s = 0; s < 4; ++s)
        xb[j][s] = __builtin_amdgcn_raw_buffer_load_b128(
            rx, g < kgroups ? (uint32_t)lr * K * 2 + g * 64 + 16 * s : kDead, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < kC; ++j)
#pragma unroll
      for (int i = 0; i < kG; ++i) {
        const GroupScale<kNv> gs(sc[i][j] & 255u, sc[i][j] >> 8);
#pragma unroll
        for (int s = 0; s < 4; ++s)
          acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(mx::as_bf16x8(gs.convert(w[i][j][s], s)),
                                                           mx::as_bf16x8(xb[j][s]), acc[i], 0, 0, 0);
      }
  }
#pragma unroll
  for (int i = 0; i < kG; ++i) red[(wave * kG + i) * 64 + lane] = acc[i];
  __syncthreads();
  const float s2 = kNv ? a.scale2[t.e] : 1.0f;
  for (int i = wave; i < kG; i += waves) {
    f32x4 v = red[i * 64 + lane];
    for (int u = 1; u < waves; ++u) v += red[(u * kG + i) * 64 + lane];
    const int n = n0 + 16 * i + 4 * q;  // lane (row lr of the tile, q): features n .. n+3
    if (lr >= t.rows || n >= N) continue;
    uint16_t* out = a.y + (size_t)(t.row0 + lr) * N + n;
    const uint16_t* bias = a.bias != nullptr ? a.bias + (size_t)t.e * N + n : nullptr;
    store4(out, v, s2, bias, min(4, N - n), (N & 3) == 0);
  }
}

// y for row tiles of at most 4 kT rows (decode: one token, or a few over many
// experts), where the weights' bytes and the latency of a pass are all there
// is.  4x4x4 MFMA, sixteen independent 4 x 4 products at once: lane (b, i) is
// weight row i of four and group 16u + b of unit u (512 k: a wave reads 256
// contiguous bytes of each row at a time), and row i of x (of each of kT
// times four) for the same k, so that x takes no registers for columns that
// 16 of them would leave empty.  x of a
// wave's kU units stays in registers while it streams the weights of its row
// groups (four weight rows each), the next group's loads in flight behind the
// current one's products.  The sixteen blocks' sums are added across lanes;
// lane block b keeps row group b of up to sixteen, which leave together.  A
// block's waves split K where it exceeds one wave's units and add their sums
// through LDS in wave order.  Row groups are dealt to the blocks in equal
// contiguous ranges, eight waves a CU.  13 of 32 NVFP4 experts, 5760 x 2880,
// 16 rows: 28 us = 4.3 TB/s of 121 MB (16-row tiles: 47); one row, 32768 x
// 2880: 13.2 us = 3.8 TB/s of 50 MB (23.2); 128 rows over 32 experts, 2880 x
// 2880: 34 us (50).
constexpr int kOneRows = 4;
constexpr int kBatch = 16;  // row groups that leave together

template <bool kNv, int kU, int kT>
__global__ __launch_bounds__(512, 2) void linear_one_kernel(LinearArgs a) {
  typedef __attribute__((__vector_size__(4 * sizeof(short)))) short s16x4;
  extern __shared__ f32x4 red[];  // [waves][kT][64], only with more than one wave
  const int K = a.K, N = a.N, kgroups = K >> 5;
  const int lane = mx::lane_id(), b = lane >> 2, i4 = lane & 3;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int kscales = kNv ? K >> 4 : kgroups;
  const int groups = (N + 3) >> 2;  // of a tile
  const int64_t total = (int64_t)count_tiles(a, kOneRows * kT) * groups;
  int64_t job = total * blockIdx.x / gridDim.x;
  const int64_t last = total * (blockIdx.x + 1) / gridDim.x;

  while (job < last) {  // uniform: the jobs of one tile at a time
    const int ti = (int)(job / groups);
    Tile t;
    if (!find_tile(a, kOneRows * kT, ti, t)) return;  // uniform, not reached: job < total
    const int g0 = (int)(job - (int64_t)ti * groups), g1 = (int)min((int64_t)groups, g0 + (last - job));
    job += g1 - g0;
    const auto rx = buffer(a.x + (size_t)t.row0 * K, (uint32_t)t.rows * K * 2);
    const size_t row0 = (size_t)t.e * N + 4 * (size_t)g0;
    const uint32_t nrows = min(4 * g1, N) - 4 * g0;
    const auto rw = buffer(a.blocks + row0 * (K >> 1), nrows * (K >> 1));
    const auto rs = buffer(a.scales + row0 * kscales, nrows * kscales);

    u32x4 x[kT][kU][4];
    uint32_t woff[kU], soff[kU];
    bool dead[kU];  // groups past K: zero x and zero weights
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int g = 16 * (wave * kU + u) + b;
      dead[u] = g >= kgroups;
#pragma unroll
      for (int p = 0; p < kT; ++p)
#pragma unroll
        for (int s = 0; s < 4; ++s)
          x[p][u][s] = __builtin_amdgcn_raw_buffer_load_b128(
              rx, dead[u] ? kDead : (uint32_t)(4 * p + i4) * K * 2 + g * 64 + 16 * s, 0, 0);
      woff[u] = (uint32_t)i4 * (K >> 1) + g * 16;
      soff[u] = (uint32_t)i4 * kscales + g * (kNv ? 2 : 1);
    }
    const float s2 = kNv ? a.scale2[t.e] : 1.0f;

    struct Group {
      u32x4 w[kU];
      uint32_t sc[kU];
    };
    auto load = [&](Group& r, int g) {  // past the last group: zeros
      const uint32_t wrow = (uint32_t)(4 * (g - g0)) * (K >> 1), srow = (uint32_t)(4 * (g - g0)) * kscales;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        r.w[u] = __builtin_amdgcn_raw_buffer_load_b128(rw, dead[u] ? kDead : woff[u] + wrow, 0, 0);
        const uint32_t so = dead[u] ? kDead : soff[u] + srow;
        r.sc[u] = kNv ? __builtin_amdgcn_raw_buffer_load_b16(rs, so, 0, 0) : __builtin_amdgcn_raw_buffer_load_b8(rs, so, 0, 0);
      }
    };
    f32x4 kept[kT] = {};
    auto multiply = [&](const Group& r, int g) {
      f32x4 acc[kT][2] = {};
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const GroupScale<kNv> gs(r.sc[u] & 255u, r.sc[u] >> 8);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const u32x4 wv = gs.convert(r.w[u][s], s);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint2 av{wv[2 * h], wv[2 * h + 1]};
#pragma unroll
            for (int p = 0; p < kT; ++p) {
              const uint2 bv{x[p][u][s][2 * h], x[p][u][s][2 * h + 1]};
              acc[p][h] = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(s16x4, av),
                                                                 __builtin_bit_cast(s16x4, bv), acc[p][h], 0, 0, 0);
            }
          }
        }
      }
      // lane (b, j): weight rows 0..3 of x row j over block b's k; add the blocks
#pragma unroll
      for (int i = 0; i < 4 * kT; ++i) {
        const int p = i >> 2, c = i & 3;
        float f = acc[p][0][c] + acc[p][1][c];
        f += __int_as_float(mx::dpp_i32<mx::kDppRowRor4>(__float_as_int(f)));
        f += __int_as_float(mx::dpp_i32<mx::kDppRowRor8>(__float_as_int(f)));
        const auto r16 = __builtin_amdgcn_permlane16_swap(__float_as_uint(f), __float_as_uint(f), false, false);
        f = __uint_as_float(r16[0]) + __uint_as_float(r16[1]);
        const auto r32 = __builtin_amdgcn_permlane32_swap(__float_as_uint(f), __float_as_uint(f), false, false);
        f = __uint_as_float(r32[0]) + __uint_as_float(r32[1]);
        if (b == ((g - g0) & (kBatch - 1))) kept[p][c] = f;
      }
    };
    auto leave = [&](int gb, int ge) {  // row groups gb .. ge - 1, at most kBatch
      f32x4 v[kT];
#pragma unroll
      for (int p = 0; p < kT; ++p) v[p] = kept[p];
      if (waves > 1) {  // uniform
#pragma unroll
        for (int p = 0; p < kT; ++p) red[(wave * kT + p) * 64 + lane] = kept[p];
        __syncthreads();
#pragma unroll
        for (int p = 0; p < kT; ++p) {
          v[p] = red[p * 64 + lane];
          for (int u = 1; u < waves; ++u) v[p] += red[(u * kT + p) * 64 + lane];
        }
        __syncthreads();
        if (wave > 0) return;
      }
      const int n = 4 * (gb + b);
      if (gb + b >= ge) return;
      const uint16_t* bias = a.bias != nullptr ? a.bias + (size_t)t.e * N + n : nullptr;
#pragma unroll
      for (int p = 0; p < kT; ++p)
        if (4 * p + i4 < t.rows)
          store4(a.y + (size_t)(t.row0 + 4 * p + i4) * N + n, v[p], s2, bias, min(4, N - n), (N & 3) == 0);
    };

    Group r0, r1;
    load(r0, g0);
    for (int gb = g0; gb < g1; gb += kBatch) {
      const int ge = min(gb + kBatch, g1);
      for (int g = gb; g < ge; g += 2) {
        load(r1, g + 1);
        __builtin_amdgcn_sched_barrier(0);
        multiply(r0, g);
        load(r0, g + 2);
        __builtin_amdgcn_sched_barrier(0);
        if (g + 1 < ge) multiply(r1, g + 1);  // uniform
      }
      leave(gb, ge);
    }
  }
}

// dx for row tiles of at most 16 rows.  The sum runs over weight rows, so the
// MFMA's A operand is the transposed weights: lane (m, q) loads kCodes codes k
// = kCodes m .. of eight weight rows n = 8q .. 8q+7, converts each to pairs of
// k, and exchanges halves between the rows of a pair (v_perm) into kCodes
// operands of eight n, one for each k: operand j multiplies with k = kCodes m
// + j as its row m.  Waves split N and add their sums in LDS in wave order.
// Bound: the weights' bytes, at 1.9 TB/s (128 rows over 32 experts, 2880 x
// 2880: 74 us, where tiles take 45), and for a small matrix the latency of a
// pass (300 rows over 8 experts, N = 1000, K = 736: 8.1 us MXFP4, 9.1 NVFP4, of
// which an empty launch is 2.2).  Not better: codes through LDS by the load
// unit, a quarter of the load instructions (9.3 and 10.2 us); 16 waves a block
// (8.6 and 9.6 us); row tiles of 32 (9.3 and 11.4 us).
constexpr int red_stride(int codes) { return 4 * codes + 4; }  // floats per lane in LDS, with padding

template <bool kNv, bool kAligned, int kCodes>
__global__ __launch_bounds__(512) void linear_backward_few_kernel(LinearArgs a) {
  extern __shared__ float redf[];
  constexpr int kFewK = 16 * kCodes, kRedStride = red_stride(kCodes);
  const int k_chunks = (a.K + kFewK - 1) / kFewK;
  int ti, kc;
  if (!map_block(a.max_tiles, k_chunks, ti, kc)) return;  // uniform per block
  Tile t;
  if (!find_tile(a, kFewRows, ti, t)) return;
  const int K = a.K, N = a.N, k0 = kc * kFewK;
  const int lane = mx::lane_id(), m = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int kscales = kNv ? K >> 4 : K >> 5;
  const auto rw = buffer(a.blocks + (size_t)t.e * N * (K >> 1), (uint32_t)N * (K >> 1));
  const auto rs = buffer(a.scales + (size_t)t.e * N * kscales, (uint32_t)N * kscales);
  const uint16_t* dy0 = a.x + (size_t)t.row0 * N;
  const auto rd = buffer(dy0, (uint32_t)t.rows * N * 2);
  const int row = min(m, t.rows - 1);  // columns past the tile's rows are dropped
  const uint32_t wcol = (k0 + kCodes * m) >> 1, scol = (k0 + kCodes * m) >> (kNv ? 4 : 5);

  f32x4 acc[kCodes] = {};
  const int steps = (N + 31) >> 5;
  for (int s0 = wave; s0 < steps; s0 += 2 * waves) {
    uint32_t w[2][8], sc[2][8];
    u32x4 d[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int s = s0 + u * waves;
      const int n = 32 * s + 8 * q;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t o = n + i < N ? (uint32_t)(n + i) * (K >> 1) + wcol : kDead;
        if constexpr (kCodes == 8) w[u][i] = __builtin_amdgcn_raw_buffer_load_b32(rw, o, 0, 0);
        else if constexpr (kCodes == 4) w[u][i] = __builtin_amdgcn_raw_buffer_load_b16(rw, o, 0, 0);
        else w[u][i] = __builtin_amdgcn_raw_buffer_load_b8(rw, o, 0, 0);
        sc[u][i] = __builtin_amdgcn_raw_buffer_load_b8(rs, n + i < N ? (uint32_t)(n + i) * kscales + scol : kDead, 0, 0);
      }
      d[u] = load_dy8<kAligned>(rd, dy0 + (size_t)row * N, (uint32_t)row * N * 2, n, N, 32 * s + 32 <= N);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      u32x4 r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        r[i] = kNv ? mx::fp4x8_to_bf16x8_any_scale(w[u][i], mx::e4m3x2_operands(sc[u][i]).x)
                   : mx::fp4x8_to_bf16x8(w[u][i], mx::e8m0_operand(sc[u][i]));
#pragma unroll
      for (int j = 0; j < kCodes; ++j) {
        u32x4 op;
#pragma unroll
        for (int p = 0; p < 4; ++p)
          op[p] = __builtin_amdgcn_perm(r[2 * p + 1][j >> 1], r[2 * p][j >> 1], (j & 1) ? 0x07060302u : 0x05040100u);
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(mx::as_bf16x8(op), mx::as_bf16x8(d[u]), acc[j], 0, 0, 0);
      }
    }
  }
  // lane (row m of the tile, q) holds k = k0 + 4 kCodes q + kCodes r + j in acc[j][r]
  float* mine = redf + (wave * 64 + lane) * kRedStride;
#pragma unroll
  for (int i = 0; i < kCodes; ++i) {
    f32x4 v;
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = acc[(4 * i + c) % kCodes][(4 * i + c) / kCodes];
    *reinterpret_cast<f32x4*>(mine + 4 * i) = v;
  }
  __syncthreads();
  const float s2 = kNv ? a.scale2[t.e] : 1.0f;
  for (int i = threadIdx.x; i < 64 * kCodes; i += blockDim.x) {
    const int l = i / kCodes, piece = i % kCodes;
    f32x4 v = *reinterpret_cast<const f32x4*>(redf + l * kRedStride + 4 * piece);
    for (int u = 1; u < waves; ++u)
      v += *reinterpret_cast<const f32x4*>(redf + (u * 64 + l) * kRedStride + 4 * piece);
    const int k = k0 + 4 * kCodes * (l >> 4) + 4 * piece, r = l & 15;
    if (r < t.rows && k < K) *reinterpret_cast<uint2*>(a.y + (size_t)(t.row0 + r) * K + k) = mxgemm::pack_bf16x4(v * s2);
  }
}

// --------------------------------------------------------------- many rows

// Scale bytes of one weight row, 24 at a time from byte offset `o` of the
// buffer: aligned dwords and a funnel shift, because a row of scales starts
// at any byte.  The buffer starts at a dword and ends with the dword that
// holds its last byte.
constexpr int kScaleDwords = 6;
struct ScaleBytes {
  uint32_t d[kScaleDwords + 1];
  __device__ __forceinline__ void load(const __amdgpu_buffer_rsrc_t& r, uint32_t o) {
    o &= ~3u;
    const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0);
    const auto u = __builtin_amdgcn_raw_buffer_load_b96(r, o + 16, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = v[i];
#pragma unroll
    for (int i = 0; i < 3; ++i) d[4 + i] = u[i];
  }
};

// y for row tiles of 128: 32x32x16 MFMA, a block of four waves makes 256
// weight rows x 128 rows, each wave 64 x 128.  K runs in chunks of 64: lane
// half h takes group 2c + h of its weight row, dword s of the group's 16
// bytes in step s, and the x values of the same k.  x travels from global
// memory into a ring of LDS stages of 64 k, the weights into one of stages of
// 128 k, by the load unit (16 bytes a lane), later chunks on their way while
// one is multiplied; one barrier a chunk.  x rows are 128 bytes a stage, their
// 16-byte pieces XOR-swizzled so that the 128-bit reads of consecutive rows
// hit distinct banks; scale bytes go straight to registers, 24 of a row at a
// time.  Two blocks a CU: one converts and waits while the other multiplies.
// Token blocks of 32 without rows are neither read nor multiplied.  Bound, by
// sizes at 2880 x 2880: many dense rows the bf16 MFMA rate (16384: 240 us = 1130
// TFLOP/s, as a large library product reaches); over experts also the weights,
// needed once each (128 experts of 128 rows: 296 us), the tiles' empty rows and
// XCDs with less to do (128 experts at random: 360 us = 750 TFLOP/s; 4096 rows
// over them: 170 us, the weights at 3.4 TB/s); few dense rows the chain of
// chunks of one block (256 and 512: 20 and 21 us).  NVFP4 266, 335, 421, 213, 26
// and 27 us: twice the vector instructions to convert a code.
//
// The stages are arrays of their own and the loop is unrolled over the period
// of both rings: the compiler waits for every load into an array that an LDS
// read may touch, so with one array and a stage counted at run time it waited
// for all loads in flight before each chunk (1024 rows 35 us instead of 30,
// 4096 over 128 experts 193 instead of 172).  For the same reason loads are
// issued outside the branch on `work`.
constexpr int kTileRows = 128, kTileN = 256;

// The rings of a kernel for up to kMax blocks of 32 rows: kX stages of x, kW
// of the weights, 80 KB in all (two blocks a CU).  The fewer rows share the
// weights, the more of them have to be on their way to keep HBM busy.  Weight
// stages hold 128 k because 64 bytes of a row at a time stream from HBM at 4.7
// TB/s, 32 bytes at 3.3 (565 MB in this pattern, no arithmetic).
template <int kMax>
struct Rings {
  static constexpr int kX = kMax > 2 ? 3 : 4, kW = kMax > 2 ? 2 : 3;
  static constexpr int kPeriod = 12;  // chunks: a multiple of kX and of 2 kW
  static_assert(kPeriod % kX == 0 && kPeriod % (2 * kW) == 0, "stages repeat with the period");
  static constexpr int kXStage = kMax * 256, kWStage = kTileN * 4;  // 16-byte slots
  static_assert(kX * kXStage + kW * kWStage <= 5120, "two blocks a CU");
  // Chunk c issues `live` loads of x of chunk c + kX - 1, even c also 4 loads of the weights of chunks c + 2 kW - 2 and
  // the next one.  Loads that may be in flight when chunk c is read: those of the chunks after the one that issued its
  // x, and for its weights.  Loads of scales are not counted: a wave without work makes none.
  static constexpr int after_x(int live, int odd) {
    int n = 0;
    for (int i = 1; i <= kX - 2; ++i) n += live + (((odd + i) & 1) == 0 ? 4 : 0);
    return n;
  }
  static constexpr int ahead(int live, int odd) {
    const int w = live * 2 * (kW - 1) + 4 * (kW - 2), x = after_x(live, odd);
    return odd || x < w ? x : w;
  }
};

// The chunk loop over kLive blocks of 32 rows.
template <bool kNv, int kLive, int kMax>
__device__ __forceinline__ void tile_chunks(f32x16 (&acc)[2][kMax], u32x4* const (&xst)[Rings<kMax>::kX],
                                            u32x4* const (&wst)[Rings<kMax>::kW], const __amdgpu_buffer_rsrc_t& rx,
                                            const __amdgpu_buffer_rsrc_t& rw, const __amdgpu_buffer_rsrc_t& rs,
                                            int K, uint32_t scale0, int kscales, int wave, bool work) {
  using Ring = Rings<kMax>;
  const int t = threadIdx.x, lane = t & 63, half = lane >> 5, lrow = lane & 31;
  const int chunks = (K + 63) >> 6, pairs = (chunks + 1) >> 1;
  // this thread's pieces of a stage
  const int xr = t >> 3, xpart = (t & 7) ^ swizzle(xr & 31);
  const uint32_t xoff = (uint32_t)xr * K * 2 + 16 * xpart;
  const uint32_t xlast = (K & 32) != 0 && xpart >= 4 ? kDead : 0u;  // the half chunk past K: zeros
  const uint32_t woff = (uint32_t)(t >> 2) * (K >> 1) + 16 * ((t & 3) ^ ((t >> 4) & 3));
  auto issue_x = [&](int c, u32x4* st, int k) __attribute__((always_inline)) {
    const uint32_t o = xoff + (uint32_t)(k * 32) * K * 2 + min(c, chunks - 1) * 128;
    load_lds16(rx, st + wave * 64 + k * 256, c >= chunks - 1 ? o | xlast : o);
  };
  auto issue_w = [&](int s, u32x4* st, int k) __attribute__((always_inline)) {
    load_lds16(rw, st + wave * 64 + k * 256, woff + (uint32_t)(k * 64) * (K >> 1) + min(s, pairs - 1) * 64);
  };

  // this lane's scale row (of the wave's 64): 24 bytes hold the groups of kSpan chunks
  constexpr int kSpan = kNv ? 6 : 12;
  const uint32_t so = scale0 + (uint32_t)(wave * 64 + lane) * kscales;
  ScaleBytes next;
  uint32_t sb[kScaleDwords];
  next.load(rs, so);
  // what chunks before the first would have issued
  constexpr int kPrologue = 2 * (Ring::kW - 1) > Ring::kX - 1 ? 2 * (Ring::kW - 1) : (Ring::kX / 2) * 2;
#pragma unroll
  for (int c = -kPrologue; c < 0; ++c) {
    if (c % 2 == 0 && c / 2 + Ring::kW - 1 >= 0) {
#pragma unroll
      for (int k = 0; k < 4; ++k) issue_w(c / 2 + Ring::kW - 1, wst[c / 2 + Ring::kW - 1], k);
    }
    if (c + Ring::kX - 1 >= 0) {
#pragma unroll
      for (int k = 0; k < kLive; ++k) issue_x(c + Ring::kX - 1, xst[c + Ring::kX - 1], k);
    }
    __builtin_amdgcn_sched_barrier(0);  // the waits count on this order
  }
  int boff[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) boff[s] = lrow * 8 + ((4 * half + s) ^ swizzle(lrow));
  const int arow = (wave * 64 + lrow) * 4, aswz = (lrow >> 2) & 3;

  int c0 = 0;
  auto chunk = [&](auto at) __attribute__((always_inline)) {
    constexpr int p = decltype(at)::value, kOdd = p & 1;
    const int c = c0 + p;
    mxgemm::wait_loads_then_barrier<Ring::ahead(kLive, kOdd)>();
    if constexpr (p % kSpan == 0) {
#pragma unroll
      for (int i = 0; i < kScaleDwords; ++i) sb[i] = __builtin_amdgcn_alignbit(next.d[i + 1], next.d[i], 8 * (so & 3u));
      next.load(rs, so + 4 * kScaleDwords * (c / kSpan + 1));
    }
    u32x4* const xnext = xst[(p + Ring::kX - 1) % Ring::kX];
    u32x4* const wnext = wst[(p / 2 + Ring::kW - 1) % Ring::kW];
    if constexpr (!kOdd) {
#pragma unroll
      for (int k = 0; k < 4; ++k) issue_w(c / 2 + Ring::kW - 1, wnext, k);
    }
#pragma unroll
    for (int k = 0; k < kLive; ++k) issue_x(c + Ring::kX - 1, xnext, k);
    if (!work) return;
    const u32x4* xbase = xst[p % Ring::kX];
    const u32x4* wbase = wst[p / 2 % Ring::kW] + arow + ((2 * kOdd + half) ^ aswz);
    u32x4 w[2];
    bf16x8 b[4][kLive];
#pragma unroll
    for (int rb = 0; rb < 2; ++rb) w[rb] = wbase[rb * 128];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int cb = 0; cb < kLive; ++cb) b[i][cb] = mx::as_bf16x8(xbase[boff[i] + cb * 256]);
    // the chunk's dword of scales, in row order: e[0] of the lane's first weight row, e[1] of its second
    constexpr int kDword = kNv ? p % kSpan : p % kSpan / 2;
    const auto e = __builtin_amdgcn_permlane32_swap(sb[kDword], sb[kDword], false, false);
    const uint32_t sh = kNv ? 16 * half : 16 * kOdd + 8 * half;
    uint32_t e0 = e[0] >> sh, e1 = e[1] >> sh;
    if (64 * c + 64 > K && half == 1) e0 = e1 = 0u;  // past K the rows are zeros: no NaN from a scale there
    const GroupScale<kNv> g0(e0 & 255u, (e0 >> 8) & 255u), g1(e1 & 255u, (e1 >> 8) & 255u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bf16x8 a0 = mx::as_bf16x8(g0.convert(w[0][i], i)), a1 = mx::as_bf16x8(g1.convert(w[1][i], i));
#pragma unroll
      for (int cb = 0; cb < kLive; ++cb) {
        acc[0][cb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a0, b[i][cb], acc[0][cb], 0, 0, 0);
        acc[1][cb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a1, b[i][cb], acc[1][cb], 0, 0, 0);
      }
    }
  };
  // Whole periods without an exit: from a loop with exits inside, the compiler's waits would count the loads that are
  // in flight at any of them.
  for (; c0 + Ring::kPeriod <= chunks; c0 += Ring::kPeriod)
    each_of([&](auto at) __attribute__((always_inline)) { return chunk(at), true; },
            std::make_integer_sequence<int, Ring::kPeriod>{});
  each_of([&](auto at) __attribute__((always_inline)) {
    if (c0 + decltype(at)::value >= chunks) return false;  // uniform
    chunk(at);
    return true;
  }, std::make_integer_sequence<int, Ring::kPeriod - 1>{});
}

// Rows of the wave's 64 outputs x 32 rows in LDS, before they leave in whole rows.
constexpr int kOutStride = 72;  // bf16 per row: 64 and padding

template <bool kNv, int kMax>
__global__ __launch_bounds__(256, 2) void linear_tile_kernel(LinearArgs a) {
  using Ring = Rings<kMax>;
  __shared__ __attribute__((aligned(16))) u32x4 x0[Ring::kXStage], x1[Ring::kXStage], x2[Ring::kXStage];
  __shared__ __attribute__((aligned(16))) u32x4 w0[Ring::kWStage], w1[Ring::kWStage];
  const int n_tiles = (a.N + kTileN - 1) / kTileN;
  int ti, nt;
  if (!map_tile(a, a.tile_rows, n_tiles, ti, nt)) return;  // uniform per block
  Tile t;
  if (!find_tile(a, a.tile_rows, ti, t)) return;
  const int K = a.K, N = a.N, n0 = nt * kTileN;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int nrows = min(kTileN, N - n0), kscales = kNv ? K >> 4 : K >> 5;
  const size_t wrow0 = (size_t)t.e * N + n0;
  const auto rx = buffer(a.x + (size_t)t.row0 * K, (uint32_t)t.rows * K * 2);
  const auto rw = buffer(a.blocks + wrow0 * (K >> 1), (uint32_t)nrows * (K >> 1));
  const uint8_t* sp = a.scales + wrow0 * kscales;
  const uint32_t shift = (uint32_t)((uintptr_t)sp & 3u);
  const auto rs = buffer(sp - shift, (shift + (uint32_t)nrows * kscales + 3u) & ~3u);

  f32x16 acc[2][kMax] = {};
  const int live = (t.rows + 31) >> 5;
  const bool work = n0 + wave * 64 < N;  // uniform: a wave past N only loads its share
  if constexpr (kMax > 2) {
    u32x4* const xst[] = {x0, x1, x2};
    u32x4* const wst[] = {w0, w1};
    if (live == 4) tile_chunks<kNv, 4, kMax>(acc, xst, wst, rx, rw, rs, K, shift, kscales, wave, work);
    else if (live == 3) tile_chunks<kNv, 3, kMax>(acc, xst, wst, rx, rw, rs, K, shift, kscales, wave, work);
    else if (live == 2) tile_chunks<kNv, 2, kMax>(acc, xst, wst, rx, rw, rs, K, shift, kscales, wave, work);
    else tile_chunks<kNv, 1, kMax>(acc, xst, wst, rx, rw, rs, K, shift, kscales, wave, work);
  } else {
    __shared__ __attribute__((aligned(16))) u32x4 x3[Ring::kXStage], w2[Ring::kWStage];
    u32x4* const xst[] = {x0, x1, x2, x3};
    u32x4* const wst[] = {w0, w1, w2};
    if (live == 2) tile_chunks<kNv, 2, kMax>(acc, xst, wst, rx, rw, rs, K, shift, kscales, wave, work);
    else tile_chunks<kNv, 1, kMax>(acc, xst, wst, rx, rw, rs, K, shift, kscales, wave, work);
  }

  // lane (row lane & 31 of the block, half): features 8i + 4 half .. + 3 in acc[.][.][4i ..]
  mxgemm::wait_loads_then_barrier<0>();  // no load still writes LDS, no wave still reads it
  const int nw = n0 + wave * 64, half = lane >> 5, lrow = lane & 31;
  if (!work) return;  // no barrier follows
  const float s2 = kNv ? a.scale2[t.e] : 1.0f;
  float bias[2][16];
#pragma unroll
  for (int rb = 0; rb < 2; ++rb)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int n = min(nw + rb * 32 + 8 * (i >> 2) + 4 * half + (i & 3), N - 1);
      bias[rb][i] = a.bias != nullptr ? mx::bf16_to_f32(a.bias[(size_t)t.e * N + n]) : 0.f;
    }
  static_assert(2 * 32 * kOutStride * sizeof(uint16_t) <= sizeof(w0), "two waves' rows fit in a stage");
  uint16_t* out = reinterpret_cast<uint16_t*>(wave < 2 ? w0 : w1) + (wave & 1) * 32 * kOutStride;
#pragma unroll
  for (int cb = 0; cb < kMax; ++cb) {
    if (cb >= live) break;
#pragma unroll
    for (int rb = 0; rb < 2; ++rb)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f32x4 v;
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = acc[rb][cb][4 * i + c] * s2 + bias[rb][4 * i + c];
        *reinterpret_cast<uint2*>(out + lrow * kOutStride + rb * 32 + 8 * i + 4 * half) = mxgemm::pack_bf16x4(v);
      }
    asm volatile("" ::: "memory");  // a wave's own LDS traffic is in order
    const int rows = min(32, t.rows - cb * 32);
    uint16_t* y = a.y + (size_t)(t.row0 + cb * 32) * N + nw;
    if ((N & 7) == 0) {
      for (int p = lane; p < rows * 8; p += 64) {
        const int r = p >> 3, col = (p & 7) * 8;
        if (nw + col < N)
          *reinterpret_cast<u32x4*>(y + (size_t)r * N + col) = *reinterpret_cast<const u32x4*>(out + r * kOutStride + col);
      }
    } else if (nw + lane < N) {
      for (int r = 0; r < rows; ++r) y[(size_t)r * N + lane] = out[r * kOutStride + lane];
    }
    asm volatile("" ::: "memory");
  }
}

// dx for row tiles of 128: a block of four waves makes 256 k x 128 rows, each
// wave 64 k x 128, over chunks of 64 weight rows n.  Stages and swizzles as
// above: dy pieces of 64 n a row, and the chunk's weight rows, 128 bytes of
// codes each.  The A operand needs eight n of one k, so the codes are read
// transposed: of a group of 16 lanes each reads eight bytes of one of eight
// rows (ds_read_b64_tr_b8), and lane c gets byte c of the eight rows, i.e. k
// = 2c and 2c + 1 of the group's 32 k for eight n.  Each byte is converted
// with its row's scale and the halves of neighbouring rows are exchanged
// (v_perm; NVFP4 rounds the pair itself, exactly) into an operand for the even
// and one for the odd k.  The chunk's scales lie transposed in LDS as bf16
// (exact), written one chunk ahead from bytes loaded one chunk before that.
// Bound: as the forward tiles.  16384 rows, 2880 x 2880: dense 245 us = 1110
// TFLOP/s, over 128 experts 352 us = 770; odd N (2883; dy through registers, in
// tiles of 64 rows) 460; 4096 rows over 128 experts 174 us (NVFP4 264, 394, 512
// and 194).
constexpr int kBackK = 256;

// The ring of a kernel for up to kMax blocks of 32 rows: as many stages as
// leave two blocks a CU.
template <int kMax>
struct BackRing {
  static constexpr int kStages = kMax > 2 ? 3 : 4;
  static constexpr int kDStage = kMax * 256, kWStage = 512;  // 16-byte slots
};

template <bool kNv, int kLive, int kMax, bool kAligned>
__device__ __forceinline__ void backward_chunks(f32x16 (&acc)[2][kMax], u32x4* const (&dst)[BackRing<kMax>::kStages],
                                                u32x4* const (&wst)[BackRing<kMax>::kStages], uint16_t* table,
                                                const __amdgpu_buffer_rsrc_t& rd, const uint16_t* dy,
                                                const __amdgpu_buffer_rsrc_t& rw, const __amdgpu_buffer_rsrc_t& rs,
                                                int rows, int K, int N, int k0, int wave, bool work) {
  constexpr int kStages = BackRing<kMax>::kStages;
  const int t = threadIdx.x, lane = t & 63, half = lane >> 5, lrow = lane & 31, mg = (lane >> 4) & 1, c16 = lane & 15;
  const int chunks = (N + 63) >> 6, kscales = kNv ? K >> 4 : K >> 5;
  constexpr int kGroups = kNv ? 16 : 8;  // of the block's 256 k
  const int pr = t >> 3, pc = t & 7;     // this thread's row (of 32) and place in a stage
  const int part = pc ^ swizzle(pr & 31);
  const uint32_t doff = (uint32_t)pr * N * 2 + 16 * part;
  // weight rows pr, pr + 32: the swizzle of the code pieces is the row's low bits
  const uint32_t woff = (uint32_t)pr * (K >> 1) + (k0 >> 1) + 16 * (pc ^ (pr & 7));
  // dy rows that start at a dword (N even) travel by the load unit, others through registers
  constexpr int kLoads = kAligned ? 2 + kLive : 2;
  u32x4 dreg[kLive];
  auto load_dy = [&](int c) __attribute__((always_inline)) {
    c = min(c, chunks - 1);
    const int n = 64 * c + 8 * part;
#pragma unroll
    for (int k = 0; k < kLive; ++k) {
      const uint16_t* row = dy + (size_t)min(pr + 32 * k, rows - 1) * N;
      dreg[k] = load_dy8<false>(rd, row, 0, n, N, 64 * c + 64 <= N);
    }
  };
  auto store_dy = [&](u32x4* st) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < kLive; ++k) st[t + k * 256] = dreg[k];
  };
  auto issue = [&](int c, u32x4* d, u32x4* w) __attribute__((always_inline)) {
    c = min(c, chunks - 1);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      load_lds16(rw, w + wave * 64 + k * 256, woff + (uint32_t)(64 * c + 32 * k) * (K >> 1));
    if constexpr (kAligned) {
#pragma unroll
      for (int k = 0; k < kLive; ++k)
        load_lds16(rd, d + wave * 64 + k * 256, doff + (uint32_t)(k * 32) * N * 2 + c * 128);
    }
  };
  // scales: thread -> row t / 4 of the chunk, a quarter of its groups
  const int sn = t >> 2, sq = t & 3;
  uint32_t sreg[2];
  auto load_scales = [&](int c) {
    const int n = 64 * c + sn;
    const uint32_t o = (uint32_t)n * kscales + (k0 >> (kNv ? 4 : 5)) + sq * (kGroups / 4);
    if (kNv) {  // a row holds an even number of them
      sreg[0] = __builtin_amdgcn_raw_buffer_load_b16(rs, n < N ? o : kDead, 0, 0);
      sreg[1] = __builtin_amdgcn_raw_buffer_load_b16(rs, n < N ? o + 2 : kDead, 0, 0);
    } else {
      sreg[0] = __builtin_amdgcn_raw_buffer_load_b8(rs, n < N ? o : kDead, 0, 0);
      sreg[1] = __builtin_amdgcn_raw_buffer_load_b8(rs, n < N ? o + 1 : kDead, 0, 0);
    }
  };
  auto store_scales = [&](int c) {
    uint16_t* dst = table + (c & 1) * kGroups * 64 + sq * (kGroups / 4) * 64 + sn;
#pragma unroll
    for (int i = 0; i < (kNv ? 2 : 1); ++i) {
      uint32_t two;
      if (kNv) {
        const mx::f32x2p v = mx::e4m3x2_operands(sreg[i]);
        two = mx::pack_bf16x2_rne(v.x, v.y);
      } else {
        two = (sreg[0] << 7) | (sreg[1] << 23);
      }
      dst[2 * i * 64] = (uint16_t)two;
      dst[(2 * i + 1) * 64] = (uint16_t)(two >> 16);
    }
  };

  load_scales(0);
  if (!kAligned) {
    load_dy(0);
    store_dy(dst[0]);
  }
  store_scales(0);
  load_scales(1);
  if (!kAligned) load_dy(1);
#pragma unroll
  for (int c = 0; c < kStages - 1; ++c) {
    __builtin_amdgcn_sched_barrier(0);  // the waits count on this order
    issue(c, dst[c], wst[c]);
  }

  int boff[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) boff[s] = lrow * 8 + ((2 * s + half) ^ swizzle(lrow));
  // codes: this lane's address for row i = c16 / 2 of the eight of a step, byte 8 (c16 & 1) of the wave's piece mg
  const int ai = c16 >> 1;
  const int aoff = (8 * half + ai) * 128 + (((wave * 2 + mg) ^ ai) * 16) + 8 * (c16 & 1);
  const int soff = (kNv ? wave * 4 + mg * 2 + (c16 >> 3) : wave * 2 + mg) * 64 + 8 * half;

  int c0 = 0;
  auto chunk = [&](auto at) __attribute__((always_inline)) {
    constexpr int p = decltype(at)::value;
    const int c = c0 + p;
    mxgemm::wait_loads_then_barrier<(kStages - 2) * kLoads>();
    // the next chunk's scales (and unaligned dy) into LDS, the one's after that on their way
    store_scales(c + 1);
    load_scales(c + 2);
    if (!kAligned) {
      store_dy(dst[(p + 1) % kStages]);
      load_dy(c + 2);
    }
    __builtin_amdgcn_sched_barrier(0);
    issue(c + kStages - 1, dst[(p + kStages - 1) % kStages], wst[(p + kStages - 1) % kStages]);
    if (kAligned && 64 * c + 64 > N) {  // uniform: dy past N, the next row's, becomes zeros as the weights there are
      uint16_t* stage = reinterpret_cast<uint16_t*>(dst[p]);
      for (int i = t; i < kLive * 32 * 64; i += 256) {
        const int r = i >> 6, col = i & 63;
        if (64 * c + col >= N) stage[r * 64 + 8 * ((col >> 3) ^ swizzle(r & 31)) + (col & 7)] = 0;
      }
      mxgemm::lds_reads_then_barrier();
    }
    if (!work) return;
    const u32x4* base = dst[p];
    const uint8_t* codes = reinterpret_cast<const uint8_t*>(wst[p]) + aoff;
    const uint16_t* sc = table + (c & 1) * kGroups * 64 + soff;
    u32x4 b[4][kLive], sv[4];
    i32x2 w[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      w[s] = __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2*)(codes + s * 16 * 128));
      sv[s] = *reinterpret_cast<const u32x4*>(sc + 16 * s);
#pragma unroll
      for (int cb = 0; cb < kLive; ++cb) b[s][cb] = base[boff[s] + cb * 256];
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      // From the second step on before the other block's loads and scales (16384 rows over 128 experts, 2880 x 2880: 356
      // us, without 380, from the first step on 369 and five registers spilled; dense 240, 262, 260; NVFP4 over 128
      // experts 388 and 404, dense 257 and 274; forward: none, or worse).
      if (s == 1) __builtin_amdgcn_s_setprio(1);
      u32x4 op[2];
#pragma unroll
      for (int p = 0; p < 4; ++p) {  // rows 2p, 2p + 1 of the eight
        const uint32_t d = (uint32_t)w[s][p >> 1];
        const float f0 = __uint_as_float(sv[s][p] << 16), f1 = __uint_as_float(sv[s][p] & 0xffff0000u);
        if (kNv) {
          const mx::f32x2e v0 = (p & 1) ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 2)
                                        : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 0);
          const mx::f32x2e v1 = (p & 1) ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 3)
                                        : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 1);
          op[0][p] = mx::pack_bf16x2_rne(v0.x * f0, v1.x * f1);
          op[1][p] = mx::pack_bf16x2_rne(v0.y * f0, v1.y * f1);
        } else {
          const uint32_t r0 = (p & 1) ? mx::fp4x2_to_bf16x2<2>(d, f0) : mx::fp4x2_to_bf16x2<0>(d, f0);
          const uint32_t r1 = (p & 1) ? mx::fp4x2_to_bf16x2<3>(d, f1) : mx::fp4x2_to_bf16x2<1>(d, f1);
          op[0][p] = __builtin_amdgcn_perm(r1, r0, 0x05040100u);
          op[1][p] = __builtin_amdgcn_perm(r1, r0, 0x07060302u);
        }
      }
#pragma unroll
      for (int cb = 0; cb < kLive; ++cb)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          acc[e][cb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(mx::as_bf16x8(op[e]), mx::as_bf16x8(b[s][cb]),
                                                               acc[e][cb], 0, 0, 0);
    }
    __builtin_amdgcn_s_setprio(0);
  };
  // whole periods without an exit, as above
  for (; c0 + kStages <= chunks; c0 += kStages)
    each_of([&](auto at) __attribute__((always_inline)) { return chunk(at), true; },
            std::make_integer_sequence<int, kStages>{});
  each_of([&](auto at) __attribute__((always_inline)) {
    if (c0 + decltype(at)::value >= chunks) return false;  // uniform
    chunk(at);
    return true;
  }, std::make_integer_sequence<int, kStages - 1>{});
}

template <bool kNv, int kMax, bool kAligned>
__global__ __launch_bounds__(256, 2) void linear_backward_tile_kernel(LinearArgs a) {
  using Ring = BackRing<kMax>;
  __shared__ __attribute__((aligned(16))) u32x4 d0[Ring::kDStage], d1[Ring::kDStage], d2[Ring::kDStage];
  __shared__ __attribute__((aligned(16))) u32x4 w0[Ring::kWStage], w1[Ring::kWStage], w2[Ring::kWStage];
  __shared__ __attribute__((aligned(16))) uint16_t table[2 * (kNv ? 16 : 8) * 64];
  const int k_tiles = (a.K + kBackK - 1) / kBackK;
  int ti, kt;
  if (!map_tile(a, a.tile_rows, k_tiles, ti, kt)) return;  // uniform per block
  Tile t;
  if (!find_tile(a, a.tile_rows, ti, t)) return;
  const int K = a.K, N = a.N, k0 = kt * kBackK;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int kscales = kNv ? K >> 4 : K >> 5;
  const uint16_t* dy = a.x + (size_t)t.row0 * N;
  const auto rd = buffer(dy, (uint32_t)t.rows * N * 2);
  const auto rw = buffer(a.blocks + (size_t)t.e * N * (K >> 1), (uint32_t)N * (K >> 1));
  const auto rs = buffer(a.scales + (size_t)t.e * N * kscales, (uint32_t)N * kscales);

  f32x16 acc[2][kMax] = {};
  const int live = (t.rows + 31) >> 5;
  const bool work = k0 + wave * 64 < K;  // uniform: a wave past K only loads its share
  if constexpr (kMax > 2) {
    u32x4* const dst[] = {d0, d1, d2};
    u32x4* const wst[] = {w0, w1, w2};
    if (live == 4)
      backward_chunks<kNv, 4, kMax, kAligned>(acc, dst, wst, table, rd, dy, rw, rs, t.rows, K, N, k0, wave, work);
    else if (live == 3)
      backward_chunks<kNv, 3, kMax, kAligned>(acc, dst, wst, table, rd, dy, rw, rs, t.rows, K, N, k0, wave, work);
    else if (live == 2)
      backward_chunks<kNv, 2, kMax, kAligned>(acc, dst, wst, table, rd, dy, rw, rs, t.rows, K, N, k0, wave, work);
    else
      backward_chunks<kNv, 1, kMax, kAligned>(acc, dst, wst, table, rd, dy, rw, rs, t.rows, K, N, k0, wave, work);
  } else {
    __shared__ __attribute__((aligned(16))) u32x4 d3[Ring::kDStage], w3[Ring::kWStage];
    u32x4* const dst[] = {d0, d1, d2, d3};
    u32x4* const wst[] = {w0, w1, w2, w3};
    if (live == 2)
      backward_chunks<kNv, 2, kMax, kAligned>(acc, dst, wst, table, rd, dy, rw, rs, t.rows, K, N, k0, wave, work);
    else
      backward_chunks<kNv, 1, kMax, kAligned>(acc, dst, wst, table, rd, dy, rw, rs, t.rows, K, N, k0, wave, work);
  }

  // lane (row lane & 31 of the block, half): k = 32 (b / 2) + 16 (b & 1) + 8 half + 2 r + e of the wave's 64 in
  // acc[e][.][4b + r]
  mxgemm::wait_loads_then_barrier<0>();  // no load still writes LDS, no wave still reads it
  if (!work) return;                     // no barrier follows
  const int kw = k0 + wave * 64, half = lane >> 5, lrow = lane & 31;
  const float s2 = kNv ? a.scale2[t.e] : 1.0f;
  static_assert(32 * kOutStride * sizeof(uint16_t) <= sizeof(w0), "a wave's rows fit in a stage");
  uint16_t* out = reinterpret_cast<uint16_t*>(wave == 0 ? w0 : wave == 1 ? w1 : wave == 2 ? w2 : d0);
#pragma unroll
  for (int cb = 0; cb < kMax; ++cb) {
    if (cb >= live) break;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      u32x4 v;
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = mx::pack_bf16x2_rne(acc[0][cb][4 * b + r] * s2, acc[1][cb][4 * b + r] * s2);
      *reinterpret_cast<u32x4*>(out + lrow * kOutStride + 32 * (b >> 1) + 16 * (b & 1) + 8 * half) = v;
    }
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

mxlinear::Sizes sizes_of(const LinearArgs& a, bool nv) { return {a.R, a.N, a.K, a.E, a.offsets != nullptr, nv}; }

// Blocks for `jobs` row groups: one each while they are few (one pass, no
// second latency), else as many as stay resident (per_cu waves to a CU).
unsigned stream_blocks(int64_t jobs, int waves, int per_cu) {
  const int64_t most = (int64_t)mxfp4moe::device_cu_count() * (per_cu / waves > 0 ? per_cu / waves : 1);
  return (unsigned)(jobs < 2 * most ? jobs : most);
}

template <bool kNv, int kC>
hipError_t launch_few_groups(const LinearArgs& a, int waves, hipStream_t stream) {
  // as many row groups to a block (x is read once for all) as leave two blocks for every CU
  const int64_t groups = ((int64_t)a.N + 15) / 16 * a.max_tiles, want = 2 * mxfp4moe::device_cu_count();
  const int g = groups >= 4 * want ? 4 : groups >= 2 * want ? 2 : 1;
  const dim3 grid = grid_of(a.max_tiles, ((int64_t)a.N + 16 * g - 1) / (16 * g));
  const size_t lds = (size_t)waves * g * 64 * sizeof(f32x4);
  if (g == 4) linear_few_kernel<kNv, kC, 4><<<grid, waves * 64, lds, stream>>>(a);
  else if (g == 2) linear_few_kernel<kNv, kC, 2><<<grid, waves * 64, lds, stream>>>(a);
  else linear_few_kernel<kNv, kC, 1><<<grid, waves * 64, lds, stream>>>(a);
  return hipGetLastError();
}

template <bool kNv>
hipError_t launch_few(LinearArgs a, hipStream_t stream) {
  a.max_tiles = max_tiles(a, kFewRows);
  const int chunks = (a.K + 127) / 128;
  const int waves = chunks <= 2 ? 1 : chunks <= 8 ? 4 : 8;
  const int c = (chunks + waves - 1) / waves;
  if (c <= 2) return launch_few_groups<kNv, 2>(a, waves, stream);
  return launch_few_groups<kNv, 3>(a, waves, stream);
}

template <bool kNv, int kT>
hipError_t launch_one(LinearArgs a, hipStream_t stream) {
  a.max_tiles = max_tiles(a, kOneRows * kT);
  const int units = (a.K + 511) / 512;
  const int waves = units <= 24 ? (units + 2) / 3 : 8, u = (units + waves - 1) / waves;
  const unsigned grid = stream_blocks((int64_t)a.max_tiles * ((a.N + 3) / 4), waves, u >= 3 || kT > 1 ? 8 : 16);
  const size_t lds = waves > 1 ? (size_t)waves * kT * 64 * sizeof(f32x4) : 0;
  switch (u) {
    case 1: linear_one_kernel<kNv, 1, kT><<<grid, waves * 64, lds, stream>>>(a); break;
    case 2: linear_one_kernel<kNv, 2, kT><<<grid, waves * 64, lds, stream>>>(a); break;
    default: linear_one_kernel<kNv, 3, kT><<<grid, waves * 64, lds, stream>>>(a); break;
  }
  return hipGetLastError();
}
constexpr int kOneMaxK = 3 * 8 * 512;  // three units for each of eight waves

template <bool kNv>
hipError_t linear(LinearArgs a, hipStream_t stream) {
  const int64_t n_tiles = (a.N + kTileN - 1) / kTileN;
  const mxlinear::Sizes sizes = sizes_of(a, kNv);
  if (a.K <= kOneMaxK) {
    const int rows = mxlinear::stream_tile_rows(sizes, mxfp4moe::device_cu_count());
    if (rows == 4) return launch_one<kNv, 1>(a, stream);
    if (rows == 8) return launch_one<kNv, 2>(a, stream);
  }
  const mxlinear::TilePlan plan =
      mxlinear::plan_tiles(sizes, true, kTileRows, n_tiles, (a.K + 63) / 64, mxfp4moe::device_cu_count());
  if (!plan.pays) return launch_few<kNv>(a, stream);
  a.tile_rows = plan.rows;
  a.max_tiles = max_tiles(a, plan.rows);
  const dim3 tile_grid = grid_of(a.max_tiles, n_tiles);
  if (plan.rows > 64) linear_tile_kernel<kNv, 4><<<tile_grid, 256, 0, stream>>>(a);
  else linear_tile_kernel<kNv, 2><<<tile_grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

template <bool kNv, int kCodes>
hipError_t launch_backward_few(LinearArgs a, hipStream_t stream) {
  a.max_tiles = max_tiles(a, kFewRows);
  const int steps = (a.N + 31) / 32, waves = steps < 8 ? steps : 8;
  const dim3 grid = grid_of(a.max_tiles, (a.K + 16 * kCodes - 1) / (16 * kCodes));
  const size_t lds = (size_t)waves * 64 * red_stride(kCodes) * sizeof(float);
  if (a.N % 2 == 0) linear_backward_few_kernel<kNv, true, kCodes><<<grid, waves * 64, lds, stream>>>(a);
  else linear_backward_few_kernel<kNv, false, kCodes><<<grid, waves * 64, lds, stream>>>(a);
  return hipGetLastError();
}

template <bool kNv>
hipError_t linear_backward(LinearArgs a, hipStream_t stream) {
  const int64_t k_tiles = (a.K + kBackK - 1) / kBackK;
  // odd N: dy through registers, which 128 rows leave none of
  const int most = a.N % 2 == 0 ? kTileRows : 64;
  const mxlinear::TilePlan plan = mxlinear::plan_tiles(sizes_of(a, kNv), false, most, k_tiles, (a.N + 63) / 64,
                                                       mxfp4moe::device_cu_count());
  if (plan.pays) {
    a.tile_rows = plan.rows;
    a.max_tiles = max_tiles(a, plan.rows);
    const dim3 tile_grid = grid_of(a.max_tiles, k_tiles);
    if (a.tile_rows > 64) linear_backward_tile_kernel<kNv, 4, true><<<tile_grid, 256, 0, stream>>>(a);
    else if (a.N % 2 == 0) linear_backward_tile_kernel<kNv, 2, true><<<tile_grid, 256, 0, stream>>>(a);
    else linear_backward_tile_kernel<kNv, 2, false><<<tile_grid, 256, 0, stream>>>(a);
    return hipGetLastError();
  }
  // 64 k a block instead of 128 while that leaves them a CU each (16 rows, 2880 x 2880, 24 or 45 blocks: 13.5 and 11 us;
  // 48 or 92 blocks of N = 2880, K = 736: 16 and 12 us; 184 or 360 blocks: 13.6 and 18 us)
  const int64_t blocks = (int64_t)max_tiles(a, kFewRows) * ((a.K + 127) / 128);
  return 2 * blocks <= mxfp4moe::device_cu_count() ? launch_backward_few<kNv, 4>(a, stream)
                                                   : launch_backward_few<kNv, 8>(a, stream);
}

LinearArgs args_of(const uint16_t* in, const uint8_t* blocks, const uint8_t* scales, const float* scale2,
                   const uint16_t* bias, const int32_t* offsets, int64_t R, int64_t K, int64_t N, int64_t E,
                   uint16_t* out) {
  return {in, blocks, scales, scale2, bias, offsets, out, (int)R, (int)K, (int)N, (int)E, 0, 0};
}

}  // namespace

namespace mxfp4moe {

hipError_t launch_linear(const uint16_t* x, const uint8_t* blocks, const uint8_t* scales, const float* scale2,
                         const uint16_t* bias, const int32_t* offsets, int64_t R, int64_t K, int64_t N, int64_t E,
                         uint16_t* y, hipStream_t stream) {
  if (R == 0) return hipSuccess;
  const LinearArgs a = args_of(x, blocks, scales, scale2, bias, offsets, R, K, N, E, y);
  ProfileScope prof(kStageLinear, stream);
  return scale2 != nullptr ? linear<true>(a, stream) : linear<false>(a, stream);
}

hipError_t launch_linear_backward(const uint16_t* dy, const uint8_t* blocks, const uint8_t* scales,
                                  const float* scale2, const int32_t* offsets, int64_t R, int64_t K, int64_t N,
                                  int64_t E, uint16_t* dx, hipStream_t stream) {
  if (R == 0) return hipSuccess;
  const LinearArgs a = args_of(dy, blocks, scales, scale2, nullptr, offsets, R, K, N, E, dx);
  ProfileScope prof(kStageLinearBackward, stream);
  return scale2 != nullptr ? linear_backward<true>(a, stream) : linear_backward<false>(a, stream);
}

}  // namespace mxfp4moe
