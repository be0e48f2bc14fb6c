// The router's balance loss with the experts' counts, and its gradient to the
// logits.
//
//   m_t = 1 for the tokens that count, V of them; p_t = softmax(logits_t)
//   c_e = picks of expert e by them;  density_e = E c_e / (sum_j c_j) / V
//   loss = sum_t m_t sum_e p_te density_e  (= E sum_e (share of picks)_e (mean probability)_e)
//   d_logits_te = d_loss m_t p_te (density_e - sum_j p_tj density_j)
// The counts have no gradient.  Eight lanes hold a token's logits (sixteen beyond
// 32 experts, 64 beyond 128) and keep their experts' sums of probabilities over the tokens
// that they meet; sums are fp32 in an order fixed by the sizes, counts are
// whole numbers in LDS.  HBM is the bound, and for a few tokens a launch: 256
// tokens of 32 experts 4.4 us and 2.8 (the gradient), 32768 of 128 6.4 + 5.4 and
// 8.5 (50 MB of logits and gradients, 5.9 TB/s).
#include "../../include/mxfp4moe.h"
#include "internal.h"
#include "mx_device.h"

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kAlone = 4;  // rounds of tokens that one block takes alone

typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef f32x4v f32x4loose __attribute__((aligned(4)));
typedef int32_t i32x4v __attribute__((ext_vector_type(4)));
typedef i32x4v i32x4loose __attribute__((aligned(4)));

constexpr int kDppHalfMirror = 0x141;  // lane i of eight gets lane 7 - i's

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
    if constexpr (kLanes == 8) return x + __int_as_float(mx::dpp_i32<kDppHalfMirror>(__float_as_int(x)));
    x += __int_as_float(mx::dpp_i32<mx::kDppRowRor4>(__float_as_int(x)));
    return x + __int_as_float(mx::dpp_i32<mx::kDppRowRor8>(__float_as_int(x)));
  }
  static __device__ __forceinline__ float largest(float x) {
    x = __builtin_elementwise_maximum(x, __int_as_float(mx::dpp_i32<mx::kDppQuadXor1>(__float_as_int(x))));
    x = __builtin_elementwise_maximum(x, __int_as_float(mx::dpp_i32<mx::kDppQuadXor2>(__float_as_int(x))));
    if constexpr (kLanes == 8)
      return __builtin_elementwise_maximum(x, __int_as_float(mx::dpp_i32<kDppHalfMirror>(__float_as_int(x))));
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
  float* part;  // sums of the blocks, where there are several: rows of part_floats(E)
};

// E sums of probabilities, E counts and the tokens that count.
__host__ __device__ constexpr int padded(int E) { return (E + 3) & ~3; }
__host__ __device__ constexpr int part_floats(int E) { return 2 * padded(E) + 4; }

__device__ __forceinline__ int32_t wave_total(int32_t v) {
  return __builtin_amdgcn_readlane(mx::wave_inclusive_sum(v), 63);
}

// Thread e < E has its expert's sum of probabilities and count, each thread the tokens that it counted.  sums: LDS.
__device__ void finish(const BalanceArgs& a, float p, int32_t count, int32_t live, float* sums) {
  const int e = threadIdx.x, wave = threadIdx.x >> 6;
  int32_t* const picks_of = reinterpret_cast<int32_t*>(sums);  // [3][kWaves]: picks, tokens, loss
  const int32_t w_picks = wave_total(count), w_live = wave_total(live);
  __syncthreads();  // (sums is free)
  if (mx::lane_id() == 0) {
    picks_of[wave] = w_picks;
    picks_of[kWaves + wave] = w_live;
  }
  __syncthreads();
  int32_t picks = 0, tokens = 0;
#pragma unroll
  for (int u = 0; u < kWaves; ++u) {
    picks += picks_of[u];
    tokens += picks_of[kWaves + u];
  }
  const float density = (float)a.E * ((float)count / (float)max(picks, 1)) / (float)max(tokens, 1);
  if (e < a.E) {
    a.counts[e] = count;
    a.density[e] = density;
  }
  const float w_loss = mx::wave_sum_f32(p * density);
  if (mx::lane_id() == 0) sums[2 * kWaves + wave] = w_loss;
  __syncthreads();
  if (e == 0) {
    float loss = 0.f;
#pragma unroll
    for (int u = 0; u < kWaves; ++u) loss += sums[2 * kWaves + u];
    *a.loss = loss;
  }
}

template <int kLanes, int kPer>
__global__ __launch_bounds__(kThreads) void balance_kernel(BalanceArgs a) {
  using Tk = Token<kLanes, kPer>;
  constexpr int kRound = kThreads / kLanes;  // tokens of a block at a time
  __shared__ int32_t counts[MXFP4MOE_MAX_EXPERTS];
  __shared__ float sums[kWaves * kLanes * kPer];
  const int E = a.E, at = threadIdx.x / kLanes;
  const int64_t step = (int64_t)gridDim.x * kRound;
  bool next_counts;
  float next[kPer];
  auto load = [&](int64_t t0) __attribute__((always_inline)) {
    next_counts = t0 + at < a.T && (a.mask == nullptr || a.mask[t0 + at] != 0);
    if (next_counts) {
      Tk::load(a.logits + (t0 + at) * E, E, -__builtin_inff(), next);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) next[i] = -__builtin_inff();
    }
  };
  load((int64_t)blockIdx.x * kRound);
  for (int e = threadIdx.x; e < E; e += kThreads) counts[e] = 0;
  __syncthreads();
  float p[kPer] = {};
  int32_t live = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * kRound; t0 < a.T; t0 += step) {
    const int n = (int)min((int64_t)kRound, a.T - t0);
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = next[i];
    live += next_counts && (threadIdx.x & (kLanes - 1)) == 0;
    if (t0 + step < a.T) load(t0 + step);  // (uniform: past the last token there is nothing to load)
    for (int i = threadIdx.x; i < n * a.top_k; i += kThreads) {
      const int32_t e = a.ids[t0 * a.top_k + i];
      if (e >= 0 && e < E && (a.mask == nullptr || a.mask[t0 + i / a.top_k] != 0)) atomicAdd(&counts[e], 1);
    }
    Tk::softmax(v);
#pragma unroll
    for (int i = 0; i < kPer; ++i) p[i] += v[i];
  }
  // the tokens of a wave, then the waves
  const int lane = mx::lane_id(), wave = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if constexpr (kLanes == 8) p[i] += __shfl_xor(p[i], 8);
    if constexpr (kLanes <= 16) {
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
  float* const row = a.part + (size_t)blockIdx.x * part_floats(E);
  int32_t* const irow = reinterpret_cast<int32_t*>(row);
  if (e < padded(E)) {
    row[e] = sum;
    irow[padded(E) + e] = count;
  }
  const int32_t w_live = wave_total(live);
  __syncthreads();
  if (lane == 0) counts[wave] = w_live;
  __syncthreads();
  if (e < 4) {
    int32_t all = 0;
#pragma unroll
    for (int u = 0; u < kWaves; ++u) all += counts[u];
    irow[2 * padded(E) + e] = e == 0 ? all : 0;
  }
}

// The blocks' sums joined, by one block: 1 << lg_lanes lanes read a row of
// them, 16 bytes each, as many rows at a time as the block has lanes for, and
// their sums meet in LDS.  256 rows of 128 experts take 5.4 us, 2 of them the
// 266 KB that one CU reads.
constexpr int kJoinRows = 8;  // of a lane at a time
__global__ __launch_bounds__(kThreads) void balance_join_kernel(BalanceArgs a, int blocks, int lg_lanes) {
  __shared__ f32x4v sums[kThreads], counts[kThreads];
  const int lanes = 1 << lg_lanes, l = threadIdx.x & (lanes - 1), slice = threadIdx.x >> lg_lanes;
  const int slices = kThreads >> lg_lanes, stride = part_floats(a.E), E4 = padded(a.E);
  f32x4v p = {};
  i32x4v c = {};
  int32_t live = 0;
  for (int b = threadIdx.x; b < blocks; b += kThreads)
    live += reinterpret_cast<const int32_t*>(a.part)[(size_t)b * stride + 2 * E4];
  if (4 * l < E4) {
    for (int b0 = slice; b0 < blocks; b0 += kJoinRows * slices) {
      f32x4v pv[kJoinRows];
      i32x4v cv[kJoinRows];
#pragma unroll
      for (int i = 0; i < kJoinRows; ++i) {
        const int b = b0 + i * slices;
        const float* row = a.part + (size_t)(b < blocks ? b : b0) * stride + 4 * l;
        pv[i] = *reinterpret_cast<const f32x4loose*>(row);
        cv[i] = *reinterpret_cast<const i32x4loose*>(row + E4);
      }
      __builtin_amdgcn_sched_barrier(0);  // all loads on their way
#pragma unroll
      for (int i = 0; i < kJoinRows; ++i) {
        if (b0 + i * slices >= blocks) break;
        p += pv[i];
        c += cv[i];
      }
    }
  }
  sums[threadIdx.x] = p;
  counts[threadIdx.x] = __builtin_bit_cast(f32x4v, c);
  __syncthreads();
  const int e = threadIdx.x;
  float sum = 0.f;
  int32_t count = 0;
  if (e < a.E) {
#pragma unroll 8
    for (int s = 0; s < min(slices, blocks); ++s) {
      sum += reinterpret_cast<const float*>(sums)[4 * (s << lg_lanes) + e];
      count += reinterpret_cast<const int32_t*>(counts)[4 * (s << lg_lanes) + e];
    }
  }
  finish(a, sum, count, live, reinterpret_cast<float*>(sums));
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

int lanes_of(int64_t E) { return E <= 32 ? 8 : E <= 128 ? 16 : 64; }  // of a token

// Blocks of the loss's kernel: one for every CU at most, and a single one, which
// needs no second launch, up to four rounds of its tokens (us, four rounds in one
// block and in four with the join: 512 tokens of 32 experts 5.5 and 6.3, 256 of
// 128 6.7 and 6.7, 64 of 500 7.0 and 7.1; five rounds 6.0 and 6.5, 7.4 and 7.0,
// 8.1 and 7.5; the second launch costs the host 3.5 besides).
int64_t loss_blocks(int64_t T, int64_t E) {
  const int64_t round = kThreads / lanes_of(E), n = (T + round - 1) / round;
  const int64_t most = mxfp4moe::device_cu_count();
  return n <= kAlone ? 1 : n < most ? n : most;
}

}  // namespace

namespace mxfp4moe {

size_t balance_loss_workspace(int64_t T, int64_t E) {
  const int64_t blocks = loss_blocks(T, E);
  return blocks > 1 ? (size_t)blocks * part_floats((int)E) * sizeof(float) : 0;
}

hipError_t launch_balance_loss(const float* logits, const int32_t* ids, const uint8_t* mask, int64_t T, int64_t E,
                               int64_t top_k, float* loss, int32_t* counts, float* density, void* workspace,
                               hipStream_t stream) {
  const int64_t blocks = loss_blocks(T, E);
  const BalanceArgs a{logits, ids, mask, T, (int)E, (int)top_k, loss, counts, density, static_cast<float*>(workspace)};
  ProfileScope prof(kStageBalance, stream);
  if (E <= 32) balance_kernel<8, 4><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  else if (E <= 64) balance_kernel<16, 4><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  else if (E <= 128) balance_kernel<16, 8><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  else balance_kernel<64, 8><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  if (blocks > 1) {
    int lg = 3;
    while ((4 << lg) < E) ++lg;
    balance_join_kernel<<<1, kThreads, 0, stream>>>(a, (int)blocks, lg);
  }
  return hipGetLastError();
}

hipError_t launch_balance_loss_backward(const float* logits, const float* density, const float* d_loss,
                                        const uint8_t* mask, const float* add, int64_t T, int64_t E, float* d_logits,
                                        hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const int64_t round = 256 / lanes_of(E), n = (T + round - 1) / round, most = 16 * device_cu_count();
  const unsigned grid = (unsigned)(n < most ? n : most);
  ProfileScope prof(kStageBalanceBackward, stream);
  if (E <= 32)
    balance_backward_kernel<8, 4><<<grid, 256, 0, stream>>>(logits, density, d_loss, mask, add, T, (int)E, d_logits);
  else if (E <= 64)
    balance_backward_kernel<16, 4><<<grid, 256, 0, stream>>>(logits, density, d_loss, mask, add, T, (int)E, d_logits);
  else if (E <= 128)
    balance_backward_kernel<16, 8><<<grid, 256, 0, stream>>>(logits, density, d_loss, mask, add, T, (int)E, d_logits);
  else
    balance_backward_kernel<64, 8><<<grid, 256, 0, stream>>>(logits, density, d_loss, mask, add, T, (int)E, d_logits);
  return hipGetLastError();
}

}  // namespace mxfp4moe
