// Pieces of token rows, for the kernels that go through rows of any width.
#pragma once

#include <hip/hip_runtime.h>

namespace mxrow {

// Row pieces of kN elements (16 bytes, or one element for rows shorter than
// that).  A row starts at any element: the loads and stores assume no more
// alignment than an element's (the hardware takes 16 bytes at any address),
// and the last piece of a row ends with it, repeating some of the elements of
// the one before where kN does not divide H (both hold the same values).
template <typename E, int kN>
struct Piece {
  typedef E vec __attribute__((ext_vector_type(kN)));
  typedef vec loose __attribute__((aligned(sizeof(E))));
  typedef float fvec __attribute__((ext_vector_type(kN)));
  static __device__ __forceinline__ int at(int v, int H) { return min(v * kN, H - kN); }
  static __device__ __forceinline__ vec load(const E* p) { return *reinterpret_cast<const loose*>(p); }
  static __device__ __forceinline__ void store(E* p, vec x) { *reinterpret_cast<loose*>(p) = x; }
  static __device__ __forceinline__ void stream(E* p, vec x) {
    __builtin_nontemporal_store(x, reinterpret_cast<loose*>(p));
  }
};

}  // namespace mxrow
