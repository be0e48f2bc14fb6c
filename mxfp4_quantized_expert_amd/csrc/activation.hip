// The experts' activation between the two products, its rows out in the input
// type or in 8 bits, and its gradient; and rows in 8 bits as they are.
//
//   g = min(gate, limit), u = clamp(up, -limit, limit)
//   a = g sigmoid(alpha g) (u + offset)
//   d_gate = da (u + offset) sigmoid(alpha g) (1 + alpha g (1 - sigmoid(alpha g))), 0 past the limit
//   d_up   = da g sigmoid(alpha g), 0 past the limits
// (gpt-oss: alpha 1.702, limit 7, offset 1; the plain gated SiLU: 1, infinity
// and 0.)  Gate and up lie side by side or in two halves of a row.  A lane
// takes eight outputs, sixteen lanes a scale's 128, so no block of threads
// waits for another; HBM is the bound.  us and TB/s of launches in a row, bf16 rows
// of 2880: 4096 rows 13.0 (5.5), to 8 bits 13.2 (4.5), gradient 21.1 (5.6), rows to 8
// bits as they are 7.3 (4.9); 16384 rows 44 (6.4), 38 (6.3), 84 (5.6) and 22.8 (6.3).
#include "fp8_device.h"
#include "internal.h"
#include "mx_device.h"
#include "row_device.h"

namespace {

using mx8::f32x8;
using mx8::kPiece;
using mxrow::Piece;

constexpr int kThreads = 256;

struct ActArgs {
  const void* h;   // [R, 2 I]
  const void* da;  // gradient: [R, I]
  void* a;         // [R, I], or in 8 bits:
  uint8_t* codes;
  float* scales;
  void* dh;
  int64_t R;
  int I;
  unsigned blocks;  // of 128 outputs in a row
  float alpha, limit, offset;
  bool split;
};

__device__ __forceinline__ float sigmoid(float alpha, float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-alpha * 1.4426950408889634f * g));
}

// Gates and ups of outputs 8v .. of a row.
template <typename E>
__device__ __forceinline__ void load_pairs(const ActArgs& a, const E* row, int v, f32x8& gate, f32x8& up) {
  if (a.split) {
    gate = mx8::to_f32<E>(mx8::load_piece(row, v, a.I));
    up = mx8::to_f32<E>(mx8::load_piece(row + a.I, v, a.I));
    return;
  }
  const f32x8 lo = mx8::to_f32<E>(mx8::load_piece(row, 2 * v, 2 * a.I));
  const f32x8 hi = mx8::to_f32<E>(mx8::load_piece(row, 2 * v + 1, 2 * a.I));
  gate = __builtin_shufflevector(lo, hi, 0, 2, 4, 6, 8, 10, 12, 14);
  up = __builtin_shufflevector(lo, hi, 1, 3, 5, 7, 9, 11, 13, 15);
}

// Every sixteen lanes a block of 128 outputs after another: body(row, piece of the row).
template <typename F>
__device__ __forceinline__ void each_block(int64_t rows, unsigned blocks, F&& body) {
  const uint64_t total = (uint64_t)rows * blocks, step = (uint64_t)gridDim.x * (kThreads / 16);
  for (uint64_t g = (uint64_t)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4); g < total; g += step) {
    const unsigned r = (unsigned)g / blocks;  // total < 2^31
    body((int64_t)r, (int)(((unsigned)g - r * blocks) * 16 + (threadIdx.x & 15)));
  }
}

template <typename E, bool kFp8>
__global__ __launch_bounds__(kThreads) void swiglu_kernel(ActArgs a) {
  each_block(a.R, a.blocks, [&](int64_t r, int v) {
    f32x8 out = {};
    if (kPiece * v < a.I) {
      f32x8 gate, up;
      load_pairs(a, static_cast<const E*>(a.h) + r * 2 * a.I, v, gate, up);
#pragma unroll
      for (int c = 0; c < kPiece; ++c) {
        // (IEEE minimum and maximum: a NaN stays one)
        const float g = __builtin_elementwise_minimum(gate[c], a.limit);
        const float u = __builtin_elementwise_maximum(__builtin_elementwise_minimum(up[c], a.limit), -a.limit);
        out[c] = g * sigmoid(a.alpha, g) * (u + a.offset);
      }
      if (!kFp8) mx8::store_piece(static_cast<E*>(a.a) + r * a.I, v, a.I, mx8::from_f32<E>(out));
      else if (kPiece * v + kPiece > a.I) {  // outputs past the row count for nothing
#pragma unroll
        for (int c = 0; c < kPiece; ++c) out[c] = kPiece * v + c < a.I ? out[c] : 0.f;
      }
    }
    if constexpr (kFp8) mx8::store_quantized(out, v, a.I, a.codes + r * a.I, a.scales + r * a.blocks);
  });
}

template <typename E>
__global__ __launch_bounds__(kThreads) void swiglu_backward_kernel(ActArgs a) {
  each_block(a.R, a.blocks, [&](int64_t r, int v) {
    if (kPiece * v >= a.I) return;
    f32x8 gate, up, dg, du;
    load_pairs(a, static_cast<const E*>(a.h) + r * 2 * a.I, v, gate, up);
    const f32x8 da = mx8::to_f32<E>(mx8::load_piece(static_cast<const E*>(a.da) + r * a.I, v, a.I));
#pragma unroll
    for (int c = 0; c < kPiece; ++c) {
      const float g = __builtin_elementwise_minimum(gate[c], a.limit);
      const float u = __builtin_elementwise_maximum(__builtin_elementwise_minimum(up[c], a.limit), -a.limit);
      const float s = sigmoid(a.alpha, g);
      // (past 128 either way s or 1 - s is 0 in fp32, and so is the product: the bound keeps it from being 0 times an
      // infinite alpha g; s is NaN where that is)
      const float x = __builtin_amdgcn_fmed3f(a.alpha * g, 128.0f, -128.0f);
      dg[c] = gate[c] <= a.limit ? da[c] * (u + a.offset) * s * (1.0f + x * (1.0f - s)) : 0.f;
      du[c] = fabsf(up[c]) <= a.limit ? da[c] * g * s : 0.f;
    }
    E* row = static_cast<E*>(a.dh) + r * 2 * a.I;
    if (a.split) {
      mx8::store_piece(row, v, a.I, mx8::from_f32<E>(dg));
      mx8::store_piece(row + a.I, v, a.I, mx8::from_f32<E>(du));
    } else {
      mx8::store_piece(row, 2 * v, 2 * a.I, mx8::from_f32<E>(__builtin_shufflevector(dg, du, 0, 8, 1, 9, 2, 10, 3, 11)));
      if (kPiece * (2 * v + 1) < 2 * a.I)
        mx8::store_piece(row, 2 * v + 1, 2 * a.I,
                         mx8::from_f32<E>(__builtin_shufflevector(dg, du, 4, 12, 5, 13, 6, 14, 7, 15)));
    }
  });
}

template <typename E>
__global__ __launch_bounds__(kThreads) void fp8_quantize_kernel(const E* __restrict__ x, int64_t R, int K,
                                                                unsigned blocks, uint8_t* __restrict__ codes,
                                                                float* __restrict__ scales) {
  each_block(R, blocks, [&](int64_t r, int v) {
    f32x8 f = {};
    if (kPiece * v < K) f = mx8::to_f32<E>(mx8::load_piece(x + r * K, v, K));
    mx8::store_quantized(f, v, K, codes + r * K, scales + r * blocks);
  });
}

// A launch holds fewer than 2^32 threads; the kernels loop past that.
unsigned grid_of(int64_t rows, int64_t blocks) {
  constexpr int64_t kMaxBlocks = 1 << 22;
  const int64_t n = (rows * blocks + kThreads / 16 - 1) / (kThreads / 16);
  return (unsigned)(n < kMaxBlocks ? n : kMaxBlocks);
}

}  // namespace

namespace mxfp4moe {

hipError_t launch_swiglu(const void* h, int dtype, int64_t R, int64_t I, float alpha, float limit, float offset,
                         bool split, void* out, uint8_t* codes, float* scales, hipStream_t stream) {
  if (R == 0) return hipSuccess;
  const ActArgs a{h, nullptr, out, codes, scales, nullptr, R, (int)I, (unsigned)mx8::blocks_of(I), alpha, limit, offset,
                  split};
  const unsigned grid = grid_of(R, a.blocks);
  ProfileScope prof(kStageSwiglu, stream);
#define MX_ACT(E)                                                              \
  do {                                                                         \
    if (codes != nullptr) swiglu_kernel<E, true><<<grid, kThreads, 0, stream>>>(a); \
    else swiglu_kernel<E, false><<<grid, kThreads, 0, stream>>>(a);            \
  } while (0)
  if (dtype == kF32) MX_ACT(float);
  else if (dtype == kF16) MX_ACT(_Float16);
  else MX_ACT(__bf16);
#undef MX_ACT
  return hipGetLastError();
}

hipError_t launch_swiglu_backward(const void* da, const void* h, int dtype, int64_t R, int64_t I, float alpha,
                                  float limit, float offset, bool split, void* dh, hipStream_t stream) {
  if (R == 0) return hipSuccess;
  const ActArgs a{h, da, nullptr, nullptr, nullptr, dh, R, (int)I, (unsigned)mx8::blocks_of(I), alpha, limit, offset,
                  split};
  const unsigned grid = grid_of(R, a.blocks);
  ProfileScope prof(kStageSwigluBackward, stream);
  if (dtype == kF32) swiglu_backward_kernel<float><<<grid, kThreads, 0, stream>>>(a);
  else if (dtype == kF16) swiglu_backward_kernel<_Float16><<<grid, kThreads, 0, stream>>>(a);
  else swiglu_backward_kernel<__bf16><<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_fp8_quantize(const void* x, int dtype, int64_t R, int64_t K, uint8_t* codes, float* scales,
                               hipStream_t stream) {
  if (R == 0) return hipSuccess;
  const unsigned blocks = (unsigned)mx8::blocks_of(K), grid = grid_of(R, blocks);
  ProfileScope prof(kStageFp8Quantize, stream);
  if (dtype == kF32)
    fp8_quantize_kernel<<<grid, kThreads, 0, stream>>>(static_cast<const float*>(x), R, (int)K, blocks, codes, scales);
  else if (dtype == kF16)
    fp8_quantize_kernel<<<grid, kThreads, 0, stream>>>(static_cast<const _Float16*>(x), R, (int)K, blocks, codes, scales);
  else
    fp8_quantize_kernel<<<grid, kThreads, 0, stream>>>(static_cast<const __bf16*>(x), R, (int)K, blocks, codes, scales);
  return hipGetLastError();
}

}  // namespace mxfp4moe
