// The router's balance loss with the experts' counts, and its gradient to the
// logits.
//
//   m_t = 1 for the tokens that count, V of them; p_t = softmax(logits_t)
//   c_e = picks of expert e by them;  density_e = E c_e / (sum_j c_j) / V
//   loss = sum_t m_t sum_e p_te density_e  (= E sum_e (share of picks)_e (mean probability)_e)
//   d_logits_te = d_loss m_t p_te (density_e - sum_j p_tj density_j)
// The counts have no gradient.  Sixteen lanes hold a token's logits (64 beyond
// 128 experts) and keep their experts' sums of probabilities over the tokens
// that they meet; sums are fp32 in an order fixed by the sizes, counts are
// whole numbers in LDS.  HBM is the bound, and for a few tokens a launch.
#include "../../include/mxfp4moe.h"
#include "internal.h"
#include "mx_device.h"

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;

typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef f32x4v f32x4loose __attribute__((aligned(4)));

// A token's logits over kLanes lanes, kPer of them each: chunk j of a lane is
// experts 4 (kLanes j + lane) .. + 3.
template <int kLanes, int kPer>
struct Token {
  static constexpr int kTokens = 64 / kLanes;  // of a wave
  static __device__ __forceinline__ int expert(int i) {
    return 4 * (kLanes * (i >> 2) + (int)(threadIdx.x & (kLanes - 1))) + (i & 3);
  }
  // row[expert], `rest` for experts past E
  static __device__ __forceinline__ void load(const float* __restrict__ row, int E, float rest, float (&v)[kPer]) {
#pragma unroll
    for (int j = 0; j < kPer; j += 4) {
      const int e = expert(j);
      if (e + 4 <= E) {
        const f32x4v q = *reinterpret_cast<const f32x4loose*>(row + e);
#pragma unroll
        for (int c = 0; c < 4; ++c) v[j + c] = q[c];
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) v[j + c] = e + c < E ? row[e + c] : rest;
      }
    }
  }
  static __device__ __forceinline__ float sum(float x) {
    if constexpr (kLanes == 64) return mx::wave_sum_f32(x);
    x += __int_as_float(mx::dpp_i32<mx::kDppQuadXor1>(__float_as_int(x)));
    x += __int_as_float(mx::dpp_i32<mx::kDppQuadXor2>(__float_as_int(x)));
    x += __int_as_float(mx::dpp_i32<mx::kDppRowRor4>(__float_as_int(x)));
    return x + __int_as_float(mx::dpp_i32<mx::kDppRowRor8>(__float_as_int(x)));
  }
  static __device__ __forceinline__ float largest(float x) {
    x = __builtin_elementwise_maximum(x, __int_as_float(mx::dpp_i32<mx::kDppQuadXor1>(__float_as_int(x))));
    x = __builtin_elementwise_maximum(x, __int_as_float(mx::dpp_i32<mx::kDppQuadXor2>(__float_as_int(x))));
    x = __builtin_elementwise_maximum(x, __int_as_float(mx::dpp_i32<mx::kDppRowRor4>(__float_as_int(x))));
    x = __builtin_elementwise_maximum(x, __int_as_float(mx::dpp_i32<mx::kDppRowRor8>(__float_as_int(x))));
    if constexpr (kLanes == 64) {
      float r[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) r[q] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 16 * q));
      x = __builtin_elementwise_maximum(__builtin_elementwise_maximum(r[0], r[1]),
                                        __builtin_elementwise_maximum(r[2], r[3]));
    }
    return x;
  }
  // Logits -> probabilities: all zeros for a token whose logits are all
  // -infinity (a mask that leaves none).  Every lane of the wave takes part.
  static __device__ __forceinline__ void softmax(float (&v)[kPer]) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) m = __builtin_elementwise_maximum(m, v[i]);
    m = largest(m);
    const bool none = m == -__builtin_inff();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      v[i] = __builtin_amdgcn_exp2f((v[i] - (none ? 0.f : m)) * 1.4426950408889634f);
      s += v[i];
    }
    s = sum(s);
    const float inv = none ? 0.f : 1.0f / s;
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] *= inv;
  }
};

struct BalanceArgs {
  const float* logits;
  const int32_t* ids;
  const uint8_t* mask;  // or nullptr
  int64_t T;
  int E, top_k;
  float* loss;
  int32_t* counts;
  float* density;
  // sums of the blocks, where there are several: [blocks][E] probabilities, [blocks][E] counts, [blocks] tokens
  float* part_p;
  int32_t* part_c;
  int32_t* part_live;
};

// Sum over the block's threads in a fixed order, in every thread.
template <typename V>
__device__ V block_sum(V v, V* lds) {
  __syncthreads();
  lds[threadIdx.x] = v;
  __syncthreads();
  for (int n = kThreads / 2; n > 0; n >>= 1) {
    if ((int)threadIdx.x < n) lds[threadIdx.x] += lds[threadIdx.x + n];
    __syncthreads();
  }
  return lds[0];
}

// Thread e < E has its expert's sum of probabilities and count.
__device__ void finish(const BalanceArgs& a, float p, int32_t count, int32_t live, float* lds) {
  const int e = threadIdx.x;
  const int32_t picks = block_sum<int32_t>(e < a.E ? count : 0, reinterpret_cast<int32_t*>(lds));
  const float density = (float)a.E * ((float)count / (float)max(picks, 1)) / (float)max(live, 1);
  if (e < a.E) {
    a.counts[e] = count;
    a.density[e] = density;
  }
  const float loss = block_sum<float>(e < a.E ? p * density : 0.f, lds);
  if (e == 0) *a.loss = loss;
}

template <int kLanes, int kPer>
__global__ __launch_bounds__(kThreads) void balance_kernel(BalanceArgs a) {
  using Tk = Token<kLanes, kPer>;
  constexpr int kRound = kThreads / kLanes;  // tokens of a block at a time
  __shared__ int32_t counts[MXFP4MOE_MAX_EXPERTS];
  __shared__ int32_t live;
  __shared__ float sums[kThreads > kWaves * kLanes * kPer ? kThreads : kWaves * kLanes * kPer];
  const int E = a.E;
  for (int e = threadIdx.x; e < E; e += kThreads) counts[e] = 0;
  if (threadIdx.x == 0) live = 0;
  __syncthreads();
  float p[kPer] = {};
  for (int64_t t0 = (int64_t)blockIdx.x * kRound; t0 < a.T; t0 += (int64_t)gridDim.x * kRound) {
    const int n = (int)min((int64_t)kRound, a.T - t0);
    const int at = threadIdx.x / kLanes;
    const bool counts_here = at < n && (a.mask == nullptr || a.mask[t0 + at] != 0);
    float v[kPer];
    if (counts_here) {
      Tk::load(a.logits + (t0 + at) * E, E, -__builtin_inff(), v);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = -__builtin_inff();
    }
    Tk::softmax(v);
#pragma unroll
    for (int i = 0; i < kPer; ++i) p[i] += v[i];
    if (counts_here && (threadIdx.x & (kLanes - 1)) == 0) atomicAdd(&live, 1);
    for (int i = threadIdx.x; i < n * a.top_k; i += kThreads) {
      const int32_t e = a.ids[t0 * a.top_k + i];
      if (e >= 0 && e < E && (a.mask == nullptr || a.mask[t0 + i / a.top_k] != 0)) atomicAdd(&counts[e], 1);
    }
  }
  // the tokens of a wave, then the waves
  const int lane = mx::lane_id(), wave = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if constexpr (kLanes == 16) {
      p[i] += __shfl_xor(p[i], 16);
      p[i] += __shfl_xor(p[i], 32);
    }
    if (lane < kLanes) sums[wave * kLanes * kPer + Tk::expert(i)] = p[i];
  }
  __syncthreads();
  const int e = threadIdx.x;
  float sum = 0.f;
  if (e < E) {
#pragma unroll
    for (int u = 0; u < kWaves; ++u) sum += sums[u * kLanes * kPer + e];
  }
  const int32_t count = e < E ? counts[e] : 0;
  if (gridDim.x == 1) {  // uniform
    finish(a, sum, count, live, sums);
    return;
  }
  if (e < E) {
    a.part_p[(size_t)blockIdx.x * E + e] = sum;
    a.part_c[(size_t)blockIdx.x * E + e] = count;
  }
  if (e == 0) a.part_live[blockIdx.x] = live;
}

// The blocks' sums joined, by one block: 512 / `slices` experts at a time.
__global__ __launch_bounds__(kThreads) void balance_join_kernel(BalanceArgs a, int blocks, int lg_experts) {
  __shared__ float sums[kThreads];
  __shared__ int32_t counts[kThreads];
  const int experts = 1 << lg_experts, e = threadIdx.x & (experts - 1), slice = threadIdx.x >> lg_experts;
  const int slices = kThreads >> lg_experts;
  float p = 0.f;
  int32_t c = 0, n = 0;
  if (e < a.E) {
#pragma unroll 8
    for (int b = slice; b < blocks; b += slices) {
      p += a.part_p[(size_t)b * a.E + e];
      c += a.part_c[(size_t)b * a.E + e];
    }
  }
  for (int b = threadIdx.x; b < blocks; b += kThreads) n += a.part_live[b];
  sums[threadIdx.x] = p;
  counts[threadIdx.x] = c;
  __syncthreads();
  if ((int)threadIdx.x < experts) {
    for (int s = 1; s < slices; ++s) {
      p += sums[s * experts + e];
      c += counts[s * experts + e];
    }
  }
  const int32_t live = block_sum<int32_t>(n, counts);
  __syncthreads();
  finish(a, p, c, live, sums);
}

template <int kLanes, int kPer>
__global__ __launch_bounds__(256) void balance_backward_kernel(const float* __restrict__ logits,
                                                               const float* __restrict__ density,
                                                               const float* __restrict__ d_loss,
                                                               const uint8_t* __restrict__ mask,
                                                               const float* add, int64_t T, int E,
                                                               float* d_logits) {  // may be `add`
  using Tk = Token<kLanes, kPer>;
  constexpr int kRound = 256 / kLanes;
  float d[kPer];
  Tk::load(density, E, 0.f, d);
  const float g = *d_loss;
  const int at = threadIdx.x / kLanes;
  for (int64_t t0 = (int64_t)blockIdx.x * kRound; t0 < T; t0 += (int64_t)gridDim.x * kRound) {
    const int64_t t = t0 + at;
    const bool here = t < T, counts_here = here && (mask == nullptr || mask[t] != 0);
    float v[kPer], out[kPer];
    if (here && add != nullptr) {
      Tk::load(add + t * E, E, 0.f, out);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) out[i] = 0.f;
    }
    if (counts_here) {
      Tk::load(logits + t * E, E, -__builtin_inff(), v);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = -__builtin_inff();
    }
    Tk::softmax(v);
    float mean = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) mean = __builtin_fmaf(v[i], d[i], mean);
    mean = Tk::sum(mean);
    if (!here) continue;  // (no lane of another token waits for this one's)
    if (counts_here) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) out[i] = __builtin_fmaf(g * v[i], d[i] - mean, out[i]);
    }
    float* row = d_logits + t * E;
#pragma unroll
    for (int j = 0; j < kPer; j += 4) {
      const int e = Tk::expert(j);
      if (e + 4 <= E) {
        *reinterpret_cast<f32x4loose*>(row + e) = f32x4v{out[j], out[j + 1], out[j + 2], out[j + 3]};
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (e + c < E) row[e + c] = out[j + c];
      }
    }
  }
}

// Blocks of the loss's kernel: one for every CU at most.
int64_t loss_blocks(int64_t T, int64_t E) {
  const int64_t round = kThreads / (E <= 128 ? 16 : 64), n = (T + round - 1) / round;
  const int64_t most = mxfp4moe::device_cu_count();
  return n < 1 ? 1 : n < most ? n : most;
}

}  // namespace

namespace mxfp4moe {

size_t balance_loss_workspace(int64_t T, int64_t E) {
  const int64_t blocks = loss_blocks(T, E);
  return blocks > 1 ? (size_t)blocks * (2 * (size_t)E + 1) * 4 : 0;
}

hipError_t launch_balance_loss(const float* logits, const int32_t* ids, const uint8_t* mask, int64_t T, int64_t E,
                               int64_t top_k, float* loss, int32_t* counts, float* density, void* workspace,
                               hipStream_t stream) {
  const int64_t blocks = loss_blocks(T, E);
  BalanceArgs a{logits, ids, mask, T, (int)E, (int)top_k, loss, counts, density, nullptr, nullptr, nullptr};
  if (blocks > 1) {
    a.part_p = static_cast<float*>(workspace);
    a.part_c = static_cast<int32_t*>(workspace) + blocks * E;
    a.part_live = a.part_c + blocks * E;
  }
  ProfileScope prof(kStageBalance, stream);
  if (E <= 64) balance_kernel<16, 4><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  else if (E <= 128) balance_kernel<16, 8><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  else balance_kernel<64, 8><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  if (blocks > 1) {
    int lg = 3;
    while ((1 << lg) < E) ++lg;
    balance_join_kernel<<<1, kThreads, 0, stream>>>(a, (int)blocks, lg);
  }
  return hipGetLastError();
}

hipError_t launch_balance_loss_backward(const float* logits, const float* density, const float* d_loss,
                                        const uint8_t* mask, const float* add, int64_t T, int64_t E, float* d_logits,
                                        hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const int64_t round = 256 / (E <= 128 ? 16 : 64), n = (T + round - 1) / round, most = 16 * device_cu_count();
  const unsigned grid = (unsigned)(n < most ? n : most);
  ProfileScope prof(kStageBalanceBackward, stream);
  if (E <= 64)
    balance_backward_kernel<16, 4><<<grid, 256, 0, stream>>>(logits, density, d_loss, mask, add, T, (int)E, d_logits);
  else if (E <= 128)
    balance_backward_kernel<16, 8><<<grid, 256, 0, stream>>>(logits, density, d_loss, mask, add, T, (int)E, d_logits);
  else
    balance_backward_kernel<64, 8><<<grid, 256, 0, stream>>>(logits, density, d_loss, mask, add, T, (int)E, d_logits);
  return hipGetLastError();
}

}  // namespace mxfp4moe
