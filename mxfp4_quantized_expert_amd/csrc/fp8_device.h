// Rows in 8 bits: E4M3 codes (OCP: finite only, largest 448) with a float32
// scale for each 128 elements of a row.
//
//   largest = max(max |v|, 2^-100);  scale = largest / 448
//   code = e4m3(v * (448 / largest)), to nearest, ties to even
// The smallest `largest` keeps 448 / largest finite and a block of zeros at
// zero.  A NaN makes its block's scale and codes NaN; with an infinity the
// scale is infinite, its code NaN and those of finite elements 0.  (The
// maximum is taken of the bits of |v|, which order as the values do, with NaN
// above infinity.)
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"
#include "row_device.h"

namespace mx8 {

constexpr int kBlock = 128;             // elements of a row that share a scale
constexpr int kPiece = 8;               // elements of a lane: sixteen lanes, one DPP row, hold a block
constexpr float kLargest = 448.0f;      // of E4M3
constexpr float kLeast = 0x1p-100f;

__host__ __device__ constexpr int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

typedef float f32x8 __attribute__((ext_vector_type(8)));

// Elements 8v .. 8v + 7 of a row of H elements as floats, zeros past its end.
// Rows start at any element.
template <typename E>
__device__ __forceinline__ typename mxrow::Piece<E, kPiece>::vec load_piece(const E* __restrict__ row, int v, int H) {
  using Pc = mxrow::Piece<E, kPiece>;
  if (kPiece * v + kPiece <= H) return Pc::load(row + kPiece * v);
  typename Pc::vec r = {};
#pragma unroll
  for (int c = 0; c < kPiece; ++c)
    if (kPiece * v + c < H) r[c] = row[kPiece * v + c];
  return r;
}
template <typename E>
__device__ __forceinline__ void store_piece(E* __restrict__ row, int v, int H,
                                            typename mxrow::Piece<E, kPiece>::vec x) {
  using Pc = mxrow::Piece<E, kPiece>;
  if (kPiece * v + kPiece <= H) {
    Pc::store(row + kPiece * v, x);
    return;
  }
#pragma unroll
  for (int c = 0; c < kPiece; ++c)
    if (kPiece * v + c < H) row[kPiece * v + c] = x[c];
}
template <typename E>
__device__ __forceinline__ f32x8 to_f32(typename mxrow::Piece<E, kPiece>::vec x) {
  return __builtin_convertvector(x, f32x8);
}
template <typename E>
__device__ __forceinline__ typename mxrow::Piece<E, kPiece>::vec from_f32(f32x8 x) {
  return __builtin_convertvector(x, typename mxrow::Piece<E, kPiece>::vec);
}

// The largest |v| (as bits) of the sixteen lanes of a DPP row, in every lane of
// it; all sixteen have to be active.
__device__ __forceinline__ uint32_t row_max_bits(uint32_t b) {
  b = max(b, (uint32_t)mx::dpp_i32<mx::kDppQuadXor1>((int)b));
  b = max(b, (uint32_t)mx::dpp_i32<mx::kDppQuadXor2>((int)b));
  b = max(b, (uint32_t)mx::dpp_i32<mx::kDppRowRor4>((int)b));
  return max(b, (uint32_t)mx::dpp_i32<mx::kDppRowRor8>((int)b));
}

// The codes of a lane's eight elements of a block that sixteen lanes hold, and
// the block's scale (the same in each of them).
__device__ __forceinline__ uint2 quantize(f32x8 v, float& scale) {
  uint32_t b = 0;
#pragma unroll
  for (int c = 0; c < kPiece; ++c) b = max(b, __float_as_uint(v[c]) & 0x7fffffffu);
  b = max(row_max_bits(b), __float_as_uint(kLeast));
  const float largest = __uint_as_float(b), up = kLargest / largest;
  scale = largest / kLargest;
  uint2 r{0u, 0u};
  r.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[0] * up, v[1] * up, (int)r.x, false);
  r.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2] * up, v[3] * up, (int)r.x, true);
  r.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4] * up, v[5] * up, (int)r.y, false);
  r.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[6] * up, v[7] * up, (int)r.y, true);
  return r;
}

// ... and stored: codes of elements 8v .. of the row, the scale by the first
// lane of the block's sixteen.
__device__ __forceinline__ void store_quantized(f32x8 x, int v, int H, uint8_t* __restrict__ codes,
                                                float* __restrict__ scales) {
  float scale;
  const uint2 q = quantize(x, scale);
  if (kPiece * v >= H) return;
  typedef uint8_t u8x8 __attribute__((ext_vector_type(8)));
  store_piece<uint8_t>(codes, v, H, __builtin_bit_cast(u8x8, q));
  if ((v & (kBlock / kPiece - 1)) == 0) scales[v / (kBlock / kPiece)] = scale;
}

}  // namespace mx8
