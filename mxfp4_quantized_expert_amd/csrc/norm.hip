// The root-mean-square norm of token rows with the residual's addition, its
// rows out in the input type or in 8 bits, and its gradients: what stands
// ahead of the router and the experts.
//
//   s = x + residual, rounded to the rows' type;  r = (mean_i s_i^2 + eps)^(-1/2)
//   y_i = s_i r w_i
//   dx_i = r (w_i dy_i - s_i r^2 mean_j(s_j w_j dy_j)) + d_s_i  (dx and the
//          residual's gradient alike), d_w_i = sum_t dy_ti s_ti r_t
// fp32 throughout, one rounding at the end.  A row lies in the registers of
// one wave (or of four or sixteen of one block), 8 elements a piece, so that
// each tensor moves once; HBM is the bound, and for a few rows the latency of
// a launch.  us and TB/s of launches in a row, bf16, with a residual: 4 x 2880
// 3.2 forward and 5.9 backward (two launches), 4096 x 2880 17.6 (5.4), in 8 bits
// 18.1 (4.6), backward 21.8 (4.3), 16384 x 2880 74 (5.1), 68 (4.9) and 80 (4.7),
// 512 x 16384 14.4 (4.7), 15.5 (3.8) and 28.3 (2.4: the largest form of four waves,
// whose registers leave eight waves a CU), 512 x 32768 23.9 (5.6), 24.9 (4.7) and
// 45.6 (2.9); float32 777 x 1001 4.6 and 8.7, 512 x 16384 24.8 (5.4), 21.7 (5.0) and
// 34.6 (3.9), 512 x 32768 52.7 (5.1), 38.8 (5.6) and 84 (3.2).
#include "fp8_device.h"
#include "internal.h"
#include "mx_device.h"
#include "row_device.h"

namespace {

using mx8::f32x8;
using mx8::kPiece;
using mxrow::Piece;

struct NormArgs {
  const void* x;
  const void* residual;  // or nullptr
  const void* weight;
  void* summed;          // with a residual
  void* y;               // or in 8 bits:
  uint8_t* codes;
  float* scales;
  float* rstd;
  float eps;
  int64_t T;
  int H;
};

// The sum over a row's waves, in every lane of them.  kWaves > 1: every wave of
// the block takes part, for its row.
template <int kWaves>
__device__ __forceinline__ float row_sum(float v, float* part) {
  v = mx::wave_sum_f32(v);
  if constexpr (kWaves > 1) {
    __syncthreads();  // the last row's sums have been read
    if (mx::lane_id() == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
    const int first = threadIdx.x / (64 * kWaves) * kWaves;
#pragma unroll
    for (int u = 0; u < kWaves; ++u) v += part[first + u];
  }
  return v;
}

// Sixteen waves have 128 registers each, which a row's own pieces fill: what is
// wanted after the row's sum alone (the norm's weight, the gradient's d_s) is
// loaded then, and the weight, which the caches hold, anew for every row and use.
// (All of it held, up to 155 registers spill: 512 x 16384 float32, forward and
// backward, 49 and 93 us, so 25 and 35; 512 x 32768 bf16 25 and 64, 24 and 46.)
template <int kWaves>
constexpr bool kLate = kWaves > 4;

// The weight's address and the lane as numbers that the compiler does not know:
// it would keep the weight, and where a lane's pieces lie, over all rows.
template <int kWaves, typename W>
__device__ __forceinline__ const W* fresh(const W* w) {
  if constexpr (kLate<kWaves>) asm volatile("" : "+s"(w));
  return w;
}
template <int kWaves>
__device__ __forceinline__ int fresh_lane() {
  int lane = mx::lane_id();
  if constexpr (kLate<kWaves>) asm volatile("" : "+v"(lane));
  return lane;
}

// kWaves waves a row, kP pieces of it a lane at most.
template <typename E, typename W, bool kFp8, int kWaves, int kP>
__global__ __launch_bounds__(kWaves > 4 ? 64 * kWaves : 256) void rms_norm_kernel(NormArgs a) {
  using Pc = Piece<E, kPiece>;
  constexpr int kRows = kWaves > 4 ? 1 : 4 / kWaves;  // of a block
  __shared__ float part[16];
  const int lane = mx::lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), sub = wave % kWaves;
  const int H = a.H, nv = (H + kPiece - 1) / kPiece;
  const E* xs = static_cast<const E*>(a.x);
  const E* rs = static_cast<const E*>(a.residual);
  const W* w = static_cast<const W*>(a.weight);
  for (int64_t t = (int64_t)blockIdx.x * kRows + wave / kWaves; t < a.T; t += (int64_t)gridDim.x * kRows) {
    typename Pc::vec h[kP], res[kP];
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const int v = (i * kWaves + sub) * 64 + lane;
      h[i] = v < nv ? mx8::load_piece(xs + t * H, v, H) : typename Pc::vec{};
      if (rs != nullptr) res[i] = v < nv ? mx8::load_piece(rs + t * H, v, H) : typename Pc::vec{};
    }
    auto weight = [&](int v) {
      return v < nv ? mx8::load_piece(fresh<kWaves>(w), v, H) : typename Piece<W, kPiece>::vec{};
    };
    typename Piece<W, kPiece>::vec wv[kP];
    if constexpr (!kLate<kWaves>) {
#pragma unroll
      for (int i = 0; i < kP; ++i) wv[i] = weight((i * kWaves + sub) * 64 + lane);
    }
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const int v = (i * kWaves + sub) * 64 + lane;
      if (rs != nullptr) {
        h[i] = mx8::from_f32<E>(mx8::to_f32<E>(h[i]) + mx8::to_f32<E>(res[i]));
        if (v < nv) mx8::store_piece(static_cast<E*>(a.summed) + t * H, v, H, h[i]);
      }
      const f32x8 f = mx8::to_f32<E>(h[i]);
#pragma unroll
      for (int c = 0; c < kPiece; ++c) sq = __builtin_fmaf(f[c], f[c], sq);
    }
    const float r = 1.0f / sqrtf(row_sum<kWaves>(sq, part) / (float)H + a.eps);
    if (lane == 0 && sub == 0) a.rstd[t] = r;
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const int v = (i * kWaves + sub) * 64 + lane;
      if ((v & ~15) >= nv) continue;  // whole rows of sixteen lanes
      if constexpr (kLate<kWaves>) wv[i] = weight(v);
      f32x8 y = mx8::to_f32<E>(h[i]) * r * mx8::to_f32<W>(wv[i]);
      if constexpr (kFp8) {
        if (r == __builtin_inff()) {  // uniform: zeros past the row's end count for nothing then too
#pragma unroll
          for (int c = 0; c < kPiece; ++c) y[c] = kPiece * v + c < H ? y[c] : 0.f;
        }
        mx8::store_quantized(y, v, H, a.codes + t * H, a.scales + t * mx8::blocks_of(H));
      } else if (v < nv) {
        mx8::store_piece(static_cast<E*>(a.y) + t * H, v, H, mx8::from_f32<E>(y));
      }
    }
  }
}

struct NormBackArgs {
  const void* dy;
  const void* d_summed;  // or nullptr
  const void* summed;
  const void* weight;
  const float* rstd;
  void* dx;
  float* part;  // [blocks][H] sums of d_weight over the block's rows
  int64_t T;
  int H;
};

// Pieces of a lane that the registers hold: 256 bytes of a row in each kernel's largest form.
template <typename E>
constexpr int kMostPieces = sizeof(E) == 4 ? 4 : 8;

// Rows of a block at a time: what sixteen waves a CU, two blocks, have registers
// for (4096 x 2880 bf16 21.7 us, with one row of four waves 24.3; 777 x 1001
// float32, in one round instead of two, 8.7 and 10.3).
constexpr int back_rows(int waves, int pieces, int most) { return waves == 1 ? 4 : waves == 4 && pieces < most ? 2 : 1; }

// A block takes every gridDim.x-th group of kRows rows and keeps its columns'
// sums of d_weight in registers; they meet in LDS in wave order and leave as
// one row of `part`.
template <typename E, typename W, int kWaves, int kP>
__global__ __launch_bounds__(64 * kWaves * back_rows(kWaves, kP, kMostPieces<E>)) void rms_norm_backward_kernel(
    NormBackArgs a) {
  using Pc = Piece<E, kPiece>;
  constexpr int kRows = back_rows(kWaves, kP, kMostPieces<E>);
  __shared__ float part[16];
  const int lane = mx::lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), sub = wave % kWaves;
  const int H = a.H, all = (H + kPiece - 1) / kPiece;
  const E* dys = static_cast<const E*>(a.dy);
  const E* ds = static_cast<const E*>(a.d_summed);
  const E* hs = static_cast<const E*>(a.summed);
  const W* w = static_cast<const W*>(a.weight);
  f32x8 dw[kP];
#pragma unroll
  for (int i = 0; i < kP; ++i) dw[i] = f32x8{};
  for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < a.T; t0 += (int64_t)gridDim.x * kRows) {
    const int64_t t = t0 + wave / kWaves;
    if (kWaves == 1 && t >= a.T) break;
    const int nv = t < a.T ? all : 0;  // (the block's barriers are for every wave)
    typename Pc::vec h[kP], g[kP], d[kP];
    auto stream_gradient = [&](int v) {
      return ds != nullptr && v < nv ? mx8::load_piece(ds + t * H, v, H) : typename Pc::vec{};
    };
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const int v = (i * kWaves + sub) * 64 + fresh_lane<kWaves>();
      h[i] = v < nv ? mx8::load_piece(hs + t * H, v, H) : typename Pc::vec{};
      g[i] = v < nv ? mx8::load_piece(dys + t * H, v, H) : typename Pc::vec{};
      if constexpr (!kLate<kWaves>) d[i] = stream_gradient(v);
    }
    const float r = t < a.T ? a.rstd[t] : 0.f;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const int v = (i * kWaves + sub) * 64 + fresh_lane<kWaves>();
      if (v >= nv) continue;
      const f32x8 s = mx8::to_f32<E>(h[i]), y = mx8::to_f32<E>(g[i]);
      const f32x8 f = y * mx8::to_f32<W>(mx8::load_piece(fresh<kWaves>(w), v, H));
#pragma unroll
      for (int c = 0; c < kPiece; ++c) {
        dot = __builtin_fmaf(f[c], s[c], dot);
        dw[i][c] = __builtin_fmaf(y[c], s[c] * r, dw[i][c]);
      }
    }
    // s r^2 mean(s w dy) as (s r) times what every element of the row shares
    const float mean = row_sum<kWaves>(dot, part) / (float)H * r;
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const int v = (i * kWaves + sub) * 64 + fresh_lane<kWaves>();
      if (v >= nv) continue;
      const f32x8 s = mx8::to_f32<E>(h[i]);
      const f32x8 f = mx8::to_f32<E>(g[i]) * mx8::to_f32<W>(mx8::load_piece(fresh<kWaves>(w), v, H));
      if constexpr (kLate<kWaves>) d[i] = stream_gradient(v);
      const f32x8 dx = r * (f - s * r * mean) + mx8::to_f32<E>(d[i]);
      mx8::store_piece(static_cast<E*>(a.dx) + t * H, v, H, mx8::from_f32<E>(dx));
    }
  }
  float* out = a.part + (size_t)blockIdx.x * H;
  extern __shared__ __attribute__((aligned(32))) float sums[];  // [all * kPiece] where kRows > 1
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    if (wave / kWaves == u) {
#pragma unroll
      for (int i = 0; i < kP; ++i) {
        const int v = (i * kWaves + sub) * 64 + lane;
        if (v >= all) continue;
        f32x8* at = reinterpret_cast<f32x8*>(sums + kPiece * v);
        if (u > 0) dw[i] += *at;
        if (u + 1 < kRows) *at = dw[i];
        else mx8::store_piece(out, v, H, dw[i]);
      }
    }
    if (u + 1 < kRows) __syncthreads();
  }
}

// d_weight[i] = sum of the blocks' rows of `part`: 32 columns a block, eight
// rows a wave at a time and sixteen bytes a lane, kJoinRows of them in flight;
// the lanes' sums meet in the wave, then the waves' in order.
constexpr int kJoinWaves = 16, kJoinCols = 32, kJoinRows = 4;
typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef f32x4v f32x4loose __attribute__((aligned(4)));

__global__ __launch_bounds__(64 * kJoinWaves) void rms_norm_join_kernel(const float* __restrict__ part, int rows,
                                                                        int H, float* __restrict__ d_weight) {
  __shared__ f32x4v sums[kJoinWaves][kJoinCols / 4];
  constexpr int kStep = 8 * kJoinWaves;
  const int lane = mx::lane_id(), wave = threadIdx.x >> 6, at = 4 * (lane & 7), col = blockIdx.x * kJoinCols + at;
  f32x4v s = {};
  for (int r0 = 8 * wave + (lane >> 3); r0 < rows; r0 += kJoinRows * kStep) {
    f32x4v v[kJoinRows];
#pragma unroll
    for (int i = 0; i < kJoinRows; ++i) {
      const int r = r0 + i * kStep;
      const float* from = part + (size_t)r * H + col;
      v[i] = f32x4v{};
      if (r < rows && col + 4 <= H) {
        v[i] = *reinterpret_cast<const f32x4loose*>(from);
      } else if (r < rows) {
#pragma unroll
        for (int c = 0; c < 3; ++c)
          if (col + c < H) v[i][c] = from[c];
      }
    }
#pragma unroll
    for (int i = 0; i < kJoinRows; ++i) s += v[i];
  }
#pragma unroll
  for (int m = 8; m < 64; m <<= 1)
#pragma unroll
    for (int c = 0; c < 4; ++c) s[c] += __shfl_xor(s[c], m);
  if (lane < 8) sums[wave][lane] = s;
  __syncthreads();
  const int out = blockIdx.x * kJoinCols + (int)threadIdx.x;
  if (threadIdx.x < kJoinCols && out < H) {
    float v = 0.f;
#pragma unroll
    for (int u = 0; u < kJoinWaves; ++u) v += sums[u][threadIdx.x >> 2][threadIdx.x & 3];
    d_weight[out] = v;
  }
}

// A launch holds fewer than 2^32 threads; the kernels loop past that.
constexpr int64_t kMaxBlocks = 1 << 20;

// A wave takes a row of few pieces alone; longer rows are four waves' (4096 x
// 2880 bf16, forward to 8 bits and backward: 18.1 and 21.8 us; a wave a row, of
// eight pieces a lane, 20.9 and 27.4; 256 rows 3.9 and 7.2, 7.4 and 11.1), the
// longest sixteen's.
template <typename F>
auto by_row(int64_t H, int most, F&& f) {
  // -> f(waves of a row, pieces of a lane)
  const int64_t nv = (H + kPiece - 1) / kPiece;
  const int few = most / 4;
  if (nv <= 64 * few) return f(1, few);
  if (nv <= 256 * few) return f(4, few);
  if (nv <= 256 * most) return f(4, most);
  return f(16, 4);
}

template <typename E, typename W, bool kFp8>
hipError_t norm(const NormArgs& a, hipStream_t stream) {
  constexpr int kMost = kMostPieces<E>, kFew = kMost / 4;
  return by_row(a.H, kMost, [&](int waves, int pieces) {
    const int64_t rows = waves > 4 ? 1 : 4 / waves, blocks = (a.T + rows - 1) / rows;
    const unsigned grid = (unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks);
    if (waves == 1) rms_norm_kernel<E, W, kFp8, 1, kFew><<<grid, 256, 0, stream>>>(a);
    else if (waves == 4 && pieces == kFew) rms_norm_kernel<E, W, kFp8, 4, kFew><<<grid, 256, 0, stream>>>(a);
    else if (waves == 4) rms_norm_kernel<E, W, kFp8, 4, kMost><<<grid, 256, 0, stream>>>(a);
    else rms_norm_kernel<E, W, kFp8, 16, 4><<<grid, 1024, 0, stream>>>(a);
    return hipGetLastError();
  });
}

// Blocks of the gradient's kernel, and rows of `part`: two for every CU at most.
int64_t back_blocks(int64_t T, int64_t H, int most) {
  return by_row(H, most, [&](int waves, int pieces) {
    const int64_t rows = back_rows(waves, pieces, most), blocks = (T + rows - 1) / rows;
    const int64_t full = 2 * mxfp4moe::device_cu_count();
    return blocks < full ? blocks : full;
  });
}

template <typename E, typename W>
hipError_t norm_backward(const NormBackArgs& a, float* d_weight, hipStream_t stream) {
  constexpr int kMost = kMostPieces<E>, kFew = kMost / 4;
  const unsigned grid = (unsigned)back_blocks(a.T, a.H, kMost);
  const size_t lds = (size_t)((a.H + kPiece - 1) / kPiece) * kPiece * sizeof(float);
  if (grid > 0) {
    by_row(a.H, kMost, [&](int waves, int pieces) {
      if (waves == 1) rms_norm_backward_kernel<E, W, 1, kFew><<<grid, 256, lds, stream>>>(a);
      else if (waves == 4 && pieces == kFew) rms_norm_backward_kernel<E, W, 4, kFew><<<grid, 512, lds, stream>>>(a);
      else if (waves == 4) rms_norm_backward_kernel<E, W, 4, kMost><<<grid, 256, 0, stream>>>(a);
      else rms_norm_backward_kernel<E, W, 16, 4><<<grid, 1024, 0, stream>>>(a);
      return 0;
    });
  }
  rms_norm_join_kernel<<<(unsigned)((a.H + kJoinCols - 1) / kJoinCols), 64 * kJoinWaves, 0, stream>>>(a.part, (int)grid, a.H, d_weight);
  return hipGetLastError();
}

}  // namespace

namespace mxfp4moe {

hipError_t launch_rms_norm(const void* x, const void* residual, const void* weight, int dtype, int weight_dtype,
                           float eps, int64_t T, int64_t H, void* summed, void* y, uint8_t* codes, float* scales,
                           float* rstd, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const NormArgs a{x, residual, weight, summed, y, codes, scales, rstd, eps, T, (int)H};
  ProfileScope prof(kStageRmsNorm, stream);
#define MX_NORM(E, W) (codes != nullptr ? norm<E, W, true>(a, stream) : norm<E, W, false>(a, stream))
  if (dtype == kF32) return MX_NORM(float, float);
  if (dtype == kF16) return weight_dtype == kF32 ? MX_NORM(_Float16, float) : MX_NORM(_Float16, _Float16);
  return weight_dtype == kF32 ? MX_NORM(__bf16, float) : MX_NORM(__bf16, __bf16);
#undef MX_NORM
}

size_t rms_norm_backward_workspace(int dtype, int64_t T, int64_t H) {
  return (size_t)back_blocks(T, H, dtype == kF32 ? kMostPieces<float> : kMostPieces<__bf16>) * H * sizeof(float);
}

hipError_t launch_rms_norm_backward(const void* dy, const void* d_summed, const void* summed, const void* weight,
                                    int dtype, int weight_dtype, const float* rstd, int64_t T, int64_t H, void* dx,
                                    float* d_weight, float* workspace, hipStream_t stream) {
  const NormBackArgs a{dy, d_summed, summed, weight, rstd, dx, workspace, T, (int)H};
  ProfileScope prof(kStageRmsNormBackward, stream);
  if (dtype == kF32) return norm_backward<float, float>(a, d_weight, stream);
  if (dtype == kF16)
    return weight_dtype == kF32 ? norm_backward<_Float16, float>(a, d_weight, stream)
                                : norm_backward<_Float16, _Float16>(a, d_weight, stream);
  return weight_dtype == kF32 ? norm_backward<__bf16, float>(a, d_weight, stream)
                              : norm_backward<__bf16, __bf16>(a, d_weight, stream);
}

}  // namespace mxfp4moe
