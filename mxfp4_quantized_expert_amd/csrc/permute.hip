// Token rows sorted by expert and summed back, with their gradients, and the
// gradient of the routing softmax.
//
// The fused layer gathers and combines inside its GEMM launches; these are
// the same two steps as operators of their own ("Restore GPT-OSS's
// router-masked expert-parallel plan", transformers PR #49431, description:
// experts take routing data and route their tokens themselves), for callers
// that run the experts in parts, train through them, or hold a share of them.
//
//   pair p = t * top_k + j is pick j of token t; sorted_pairs[i] is the pair
//   of row i (out of range: an empty row); pair_rows[p] is the row of pair p
//   (out of range: a pair without a row, e.g. of an expert held elsewhere).
//   permute:            rows[i] = x[sorted_pairs[i] / top_k], empty rows 0
//   permute_backward:   dx[t] = sum_j d_rows[row of (t, j)]
//   unpermute:          y[t] = sum_j w[t, j] rows[row of (t, j)]
//   unpermute_backward: d_rows[row of (t, j)] = w[t, j] dy[t]
//                       d_w[t, j] = <dy[t], rows[row of (t, j)]>
//   route_backward:     d_logits[t, id_j] = w_j (d_w_j - sum_i w_i d_w_i)
// Sums run in fp32 in ascending j (dot products in a fixed tree), each result
// is rounded once, and no result depends on the order of blocks.  Every
// kernel here moves each byte a few flops at most: HBM is the bound, and for
// a handful of tokens the latency of a launch.
#include "../../include/mxfp4moe.h"
#include "internal.h"
#include "mx_device.h"
#include "row_device.h"

namespace {

using mxrow::Piece;

constexpr int kThreads = 256;

// How lanes share a row: groups of 2^lg lanes (a power of two up to the
// wave, so that short rows do not idle most of a wave), `segs` groups to a
// row, a piece to a lane where there are enough of them.
struct RowSplit {
  int nv;    // pieces of a row
  int lg;    // log2 of the lanes of a group
  int segs;  // groups of a row
};

__device__ __forceinline__ bool in_range(int32_t i, int64_t n) { return i >= 0 && (int64_t)i < n; }

// pair_rows of the kPairChunk pairs from chunk * kPairChunk, by one block:
// every row's pair is read and those of the chunk are kept in LDS (the later
// row wins where a pair is listed twice), so that pairs without a row come
// out as -1 without a launch that clears first.
constexpr int kPairChunk = 2048;
__device__ void invert_chunk(const int32_t* __restrict__ sorted_pairs, int64_t R, int64_t P, int chunk,
                             int32_t* __restrict__ pair_rows) {
  __shared__ int32_t lds[kPairChunk];
  for (int i = threadIdx.x; i < kPairChunk; i += blockDim.x) lds[i] = -1;
  __syncthreads();
  const int64_t first = (int64_t)chunk * kPairChunk;
  // sixteen pairs of a thread in flight, four to a load
  typedef int32_t four __attribute__((ext_vector_type(4)));
  typedef four loose __attribute__((aligned(4)));
  const int64_t whole = R & ~(int64_t)3;
#pragma unroll 4
  for (int64_t i = 4 * (int64_t)threadIdx.x; i < whole; i += 4 * blockDim.x) {
    const four p = *reinterpret_cast<const loose*>(sorted_pairs + i);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t d = (uint32_t)p[c] - (uint32_t)first;
      if (d < (uint32_t)kPairChunk) atomicMax(&lds[d], (int)i + c);
    }
  }
  if (threadIdx.x < R - whole) {
    const uint32_t d = (uint32_t)sorted_pairs[whole + threadIdx.x] - (uint32_t)first;
    if (d < (uint32_t)kPairChunk) atomicMax(&lds[d], (int)(whole + threadIdx.x));
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kPairChunk; i += blockDim.x)
    if (first + i < P) pair_rows[first + i] = lds[i];
}

__global__ __launch_bounds__(1024) void invert_kernel(const int32_t* __restrict__ sorted_pairs, int64_t R, int64_t P,
                                                      int32_t* __restrict__ pair_rows) {
  invert_chunk(sorted_pairs, R, P, blockIdx.x, pair_rows);
}

// ... and for a batch of many pairs, where every block reading every row's
// pair would cost more than a second launch: clear, then enter the rows (the
// larger one wins, whatever the order).  us of a permute of 64 bf16, in blocks
// and in two launches: 16384 pairs 6.4 and 7.5, 32768 7.8 and 8.4, 65536 11.1
// and 11.1, 98304 15.2 and 13.7, 262144 44.0 and 29.4.
constexpr int64_t kInvertInBlocks = 65536;
__global__ __launch_bounds__(kThreads) void clear_pair_rows_kernel(int32_t* __restrict__ pair_rows, int64_t P) {
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < P; i += (int64_t)gridDim.x * kThreads)
    pair_rows[i] = -1;
}
__global__ __launch_bounds__(kThreads) void enter_pair_rows_kernel(const int32_t* __restrict__ sorted_pairs,
                                                                   int64_t R, int64_t P,
                                                                   int32_t* __restrict__ pair_rows) {
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < R; i += (int64_t)gridDim.x * kThreads)
    if (in_range(sorted_pairs[i], P)) atomicMax(&pair_rows[sorted_pairs[i]], (int)i);
}

// Small batches, one launch: rows[i] = x[sorted_pairs[i] / top_k], a piece to
// a lane; the blocks before copy_block0 write pair_rows meanwhile.  Bound by
// the launch: 4 tokens, top 4, 2880 bf16: 2.4 us.
template <typename E, int kN>
__global__ __launch_bounds__(kThreads) void permute_kernel(const E* __restrict__ x,
                                                           const int32_t* __restrict__ sorted_pairs,
                                                           E* __restrict__ rows, int32_t* __restrict__ pair_rows,
                                                           int64_t R, int64_t P, int H, int top_k, RowSplit sp,
                                                           int copy_block0) {
  using Pc = Piece<E, kN>;
  if ((int)blockIdx.x < copy_block0) {
    invert_chunk(sorted_pairs, R, P, blockIdx.x, pair_rows);
    return;
  }
  const int lanes = 1 << sp.lg;
  const unsigned blocks = gridDim.x - copy_block0;
  for (int64_t g = ((int64_t)(blockIdx.x - copy_block0) * kThreads + threadIdx.x) >> sp.lg; g < R * sp.segs;
       g += ((int64_t)blocks * kThreads) >> sp.lg) {
    const unsigned i = (unsigned)g / (unsigned)sp.segs;
    const int32_t p = sorted_pairs[i];
    const bool live = in_range(p, P);
    const E* src = x + (size_t)(live ? p / top_k : 0) * H;
    E* dst = rows + (size_t)i * H;
    for (int v = (int)((unsigned)g % (unsigned)sp.segs) * lanes + (threadIdx.x & (lanes - 1)); v < sp.nv;
         v += lanes * sp.segs) {
      const int e = Pc::at(v, H);
      Pc::store(dst + e, live ? Pc::load(src + e) : typename Pc::vec{});
    }
  }
}

// Clears the rows that hold no pair, a wave looking at kZeroRows of them (they
// lie together behind a rank's share of the rows): block `block` of `blocks`.
// With x, the earlier row of a pair listed twice gets its token's row instead.
constexpr int kZeroRows = 4;
template <typename E, int kN>
__device__ __forceinline__ void clear_empty_rows(E* __restrict__ rows, const E* __restrict__ x, int top_k,
                                                 const int32_t* __restrict__ sorted_pairs,
                                                 const int32_t* __restrict__ pair_rows, int64_t R, int64_t P, int H,
                                                 int nv, int block, int blocks) {
  using Pc = Piece<E, kN>;
  const int lane = mx::lane_id();
  const int64_t waves = (int64_t)blocks * (kThreads / 64);
  for (int64_t r0 = ((int64_t)block * (kThreads / 64) + (threadIdx.x >> 6)) * kZeroRows; r0 < R;
       r0 += waves * kZeroRows) {
    const int64_t r = r0 + lane;
    bool empty = false;
    int32_t p = -1;
    if (lane < kZeroRows && r < R) {
      p = sorted_pairs[r];
      empty = !in_range(p, P) || pair_rows[p] != (int32_t)r;
    }
    uint64_t todo = __ballot(empty);
    while (todo != 0) {
      const int b = __builtin_ctzll(todo);
      todo &= todo - 1;
      const int32_t pb = __builtin_amdgcn_readlane(p, b);
      const E* src = x != nullptr && in_range(pb, P) ? x + (size_t)(pb / top_k) * H : nullptr;
      for (int v = lane; v < nv; v += 64) {
        const int e = Pc::at(v, H);
        Pc::store(rows + (size_t)(r0 + b) * H + e, src != nullptr ? Pc::load(src + e) : typename Pc::vec{});
      }
    }
  }
}

// Large batches, with pair_rows written before: a token's pieces are read once
// and stored to its top_k rows, past the caches; the blocks from zero_block0 on
// clear the rows that hold no pair.  4096 tokens, top 4, 2880 bf16: 24 us = 4.9
// TB/s of 118 MB (row by row, x read four times: 32 us; a copy of 1 GiB reaches
// 5.2 TB/s).  Two, three or six pieces a lane were slower (37 to 40 us).
template <typename E, int kN>
__global__ __launch_bounds__(kThreads) void permute_by_token_kernel(const E* __restrict__ x,
                                                                    const int32_t* __restrict__ sorted_pairs,
                                                                    E* __restrict__ rows,
                                                                    const int32_t* __restrict__ pair_rows, int64_t T,
                                                                    int64_t R, int H, int top_k, RowSplit sp,
                                                                    int zero_block0) {
  using Pc = Piece<E, kN>;
  if ((int)blockIdx.x >= zero_block0) {
    clear_empty_rows<E, kN>(rows, x, top_k, sorted_pairs, pair_rows, R, T * top_k, H, sp.nv, blockIdx.x - zero_block0,
                            gridDim.x - zero_block0);
    return;
  }
  const int lanes = 1 << sp.lg;
  for (int64_t g = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> sp.lg; g < T * sp.segs;
       g += ((int64_t)zero_block0 * kThreads) >> sp.lg) {
    const unsigned t = (unsigned)g / (unsigned)sp.segs;
    const E* src = x + (size_t)t * H;
    for (int v = (int)((unsigned)g % (unsigned)sp.segs) * lanes + (threadIdx.x & (lanes - 1)); v < sp.nv;
         v += lanes * sp.segs) {
      const int e = Pc::at(v, H);
      const typename Pc::vec piece = Pc::load(src + e);
      for (int j = 0; j < top_k; ++j) {
        const int32_t r = pair_rows[(size_t)t * top_k + j];
        if (in_range(r, R)) Pc::stream(rows + (size_t)r * H + e, piece);
      }
    }
  }
}

// y[t] = sum_j w[t, j] rows[pair_rows[t, j]] (w == nullptr: 1), j ascending, four
// pairs' pieces in flight.  Bound by HBM: 4096 tokens, top 4, 2880 bf16: 22 us =
// 5.3 TB/s of 118 MB.
template <typename E, int kN>
__global__ __launch_bounds__(kThreads) void unpermute_kernel(const E* __restrict__ rows,
                                                             const int32_t* __restrict__ pair_rows,
                                                             const float* __restrict__ weights, E* __restrict__ y,
                                                             int64_t T, int64_t R, int H, int top_k, RowSplit sp) {
  using Pc = Piece<E, kN>;
  const int lanes = 1 << sp.lg;
  for (int64_t g = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> sp.lg; g < T * sp.segs;
       g += ((int64_t)gridDim.x * kThreads) >> sp.lg) {
    const unsigned t = (unsigned)g / (unsigned)sp.segs;
    for (int v = (int)((unsigned)g % (unsigned)sp.segs) * lanes + (threadIdx.x & (lanes - 1)); v < sp.nv;
         v += lanes * sp.segs) {
      const int e = Pc::at(v, H);
      typename Pc::fvec sum = {};
      for (int j0 = 0; j0 < top_k; j0 += 4) {  // four pairs' pieces in flight
        typename Pc::vec z[4];
        float w[4];
        bool live[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const size_t p = (size_t)t * top_k + min(j0 + u, top_k - 1);
          const int32_t r = pair_rows[p];
          live[u] = j0 + u < top_k && in_range(r, R);
          w[u] = weights != nullptr ? weights[p] : 1.0f;
          z[u] = live[u] ? Pc::load(rows + (size_t)r * H + e) : typename Pc::vec{};
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const typename Pc::fvec f = __builtin_convertvector(z[u], typename Pc::fvec);
#pragma unroll
          for (int c = 0; c < kN; ++c) sum[c] = live[u] ? __builtin_fmaf(w[u], f[c], sum[c]) : sum[c];
        }
      }
      Pc::store(y + (size_t)t * H + e, __builtin_convertvector(sum, typename Pc::vec));
    }
  }
}

// d_rows and d_w, kWaves waves per token (four for a batch too small to fill
// the chip with one each), four pairs at a time beside one read of dy; the
// blocks from zero_block0 on clear the rows that hold no pair.  Bound by HBM:
// 4096 tokens, top 4, 2880 bf16: 37 us = 5.7 TB/s of 212 MB; 777 tokens, top 2,
// 1001 float32, 5 of 8 experts: 4.7 us, of which an empty launch is 2.2.
template <typename E, int kN, int kWaves>
__global__ __launch_bounds__(kThreads) void unpermute_backward_kernel(
    const E* __restrict__ dy, const E* __restrict__ rows, const int32_t* __restrict__ sorted_pairs,
    const int32_t* __restrict__ pair_rows, const float* __restrict__ weights, E* __restrict__ d_rows,
    float* __restrict__ d_weights, int64_t T, int64_t R, int H, int top_k, int nv, int zero_block0) {
  using Pc = Piece<E, kN>;
  constexpr int kTokens = kThreads / (64 * kWaves);  // of a block
  __shared__ float part[4][4];                       // kWaves > 1: [wave][pair]
  const int lane = mx::lane_id();
  if ((int)blockIdx.x >= zero_block0) {
    clear_empty_rows<E, kN>(d_rows, nullptr, top_k, sorted_pairs, pair_rows, R, T * top_k, H, nv,
                            blockIdx.x - zero_block0, gridDim.x - zero_block0);
    return;
  }
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int64_t t = (int64_t)blockIdx.x * kTokens + wave / kWaves; t < T; t += (int64_t)zero_block0 * kTokens) {
    const E* g = dy + (size_t)t * H;
    for (int j0 = 0; j0 < top_k; j0 += 4) {
      size_t at[4];
      float w[4], dot[4];
      bool live[4], own[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const size_t p = (size_t)t * top_k + min(j0 + u, top_k - 1);
        const int32_t r = pair_rows[p];
        live[u] = j0 + u < top_k && in_range(r, R);
        own[u] = live[u] && (size_t)sorted_pairs[r] == p;
        w[u] = weights[p];
        at[u] = (size_t)(live[u] ? r : 0) * H;
        dot[u] = 0.f;
      }
      for (int v = (wave % kWaves) * 64 + lane; v < nv; v += 64 * kWaves) {
        const int e = Pc::at(v, H), again = v * kN - e;  // `again`: elements that the piece before this one has too
        typename Pc::vec zv[4];
        const typename Pc::fvec gv = __builtin_convertvector(Pc::load(g + e), typename Pc::fvec);
#pragma unroll
        for (int u = 0; u < 4; ++u) zv[u] = live[u] ? Pc::load(rows + at[u] + e) : typename Pc::vec{};
        typename Pc::fvec gd = gv;
        if (again > 0) {
#pragma unroll
          for (int c = 0; c < kN; ++c)
            if (c < again) {
              gd[c] = 0.f;
#pragma unroll
              for (int u = 0; u < 4; ++u) zv[u][c] = (E)0.f;
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const typename Pc::fvec f = __builtin_convertvector(zv[u], typename Pc::fvec);
          if (live[u]) {  // uniform
#pragma unroll
            for (int c = 0; c < kN; ++c) dot[u] = __builtin_fmaf(gd[c], f[c], dot[u]);
          }
          if (own[u]) Pc::store(d_rows + at[u] + e, __builtin_convertvector(gv * w[u], typename Pc::vec));
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) dot[u] = mx::wave_sum_f32(dot[u]);
      if constexpr (kWaves == 1) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (lane == u && j0 + u < top_k) d_weights[t * top_k + j0 + u] = dot[u];
      } else {
        if (lane == 0) {
#pragma unroll
          for (int u = 0; u < 4; ++u) part[wave][u] = dot[u];
        }
        __syncthreads();
        const int u = threadIdx.x;
        if (u < 4 && j0 + u < top_k)
          d_weights[t * top_k + j0 + u] = (part[0][u] + part[1][u]) + (part[2][u] + part[3][u]);
        __syncthreads();
      }
    }
  }
}

// A block takes `tokens` tokens (at most kRouteTokens, a multiple of 4): their
// rows lie in LDS, zeros into which a thread per token adds the gradients of
// its picks in order, and leave as one contiguous stretch, 16 bytes a thread.
// Bound by the bytes written: 32768 tokens, 128 experts, top 4: 6.1 us = 3.0
// TB/s of 18 MB, of which an empty launch is 2.2 (each logit compared with its
// token's picks instead: 7.4).
constexpr int kRouteTokens = 32;
__global__ __launch_bounds__(kThreads) void route_backward_kernel(const int32_t* __restrict__ ids,
                                                                  const float* __restrict__ weights,
                                                                  const float* __restrict__ d_weights,
                                                                  float* __restrict__ d_logits, int64_t T, int E,
                                                                  int top_k, int tokens) {
  using Pc = Piece<float, 4>;
  extern __shared__ __attribute__((aligned(16))) float rows[];  // [tokens][E]
  __shared__ int32_t id[kRouteTokens * MXFP4MOE_MAX_TOPK];
  __shared__ float w[kRouteTokens * MXFP4MOE_MAX_TOPK], dw[kRouteTokens * MXFP4MOE_MAX_TOPK];
  for (int64_t t0 = (int64_t)blockIdx.x * tokens; t0 < T; t0 += (int64_t)gridDim.x * tokens) {
    const int n = (int)min((int64_t)tokens, T - t0), pairs = n * top_k, floats = n * E;
    const size_t p0 = (size_t)t0 * top_k;
    for (int i = threadIdx.x; i < pairs; i += kThreads) {
      id[i] = ids[p0 + i];
      w[i] = weights[p0 + i];
      dw[i] = d_weights[p0 + i];
    }
    for (int i = threadIdx.x; 4 * i < floats; i += kThreads) *reinterpret_cast<Pc::vec*>(rows + 4 * i) = Pc::vec{};
    __syncthreads();
    if ((int)threadIdx.x < n) {
      const int q0 = threadIdx.x * top_k;
      float s = 0.f;
#pragma unroll 4
      for (int j = 0; j < top_k; ++j) s = __builtin_fmaf(w[q0 + j], dw[q0 + j], s);
#pragma unroll 4
      for (int j = 0; j < top_k; ++j) {
        const int e = id[q0 + j];
        if (e >= 0 && e < E) rows[threadIdx.x * E + e] += w[q0 + j] * (dw[q0 + j] - s);
      }
    }
    __syncthreads();
    float* out = d_logits + t0 * E;
    for (int i = threadIdx.x; 4 * i < floats; i += kThreads) {
      if (4 * i + 4 <= floats) {
        Pc::store(out + 4 * i, *reinterpret_cast<const Pc::vec*>(rows + 4 * i));
      } else {
        for (int c = 4 * i; c < floats; ++c) out[c] = rows[c];
      }
    }
    __syncthreads();
  }
}

// One piece a lane while the groups can be counted in 31 bits.
RowSplit row_split(int64_t rows, int64_t nv) {
  RowSplit s{(int)nv, 0, 1};
  while (s.lg < 6 && (1 << s.lg) < nv) ++s.lg;
  const int64_t segs = (nv + (1 << s.lg) - 1) >> s.lg;
  s.segs = rows * segs <= (int64_t)1 << 24 ? (int)segs : 1;
  return s;
}

// A launch holds fewer than 2^32 threads; the kernels loop past that.
constexpr int64_t kMaxBlocks = 1 << 22;

unsigned block_count(int64_t work, int64_t per_block) {
  const int64_t n = (work + per_block - 1) / per_block;
  return (unsigned)(n < kMaxBlocks ? n : kMaxBlocks);
}

unsigned split_blocks(int64_t rows, const RowSplit& s) { return block_count(rows * s.segs, kThreads >> s.lg); }

// Bytes of the rows from which a second launch, the pair list's, costs less
// than reading x once for each pick (us in one launch, and by token with the
// list before it: 512, 1024, 1456 and 4096 tokens, top 4, 2880 bf16 = 11, 22, 32
// and 90 MiB: 6.0 and 6.5, 9.2 and 8.8, 11.7 and 11.2, 29.5 and 24.1; 8192
// tokens, top 8, 512 bf16 = 64 MiB: 31.0 and 25.3; top 1 saves no read: 8192
// tokens of 2880 = 45 MiB 18.8 and 20.4).
constexpr int64_t kByTokenBytes = 32 << 20;

template <typename E, int kN>
hipError_t permute(const void* x, const int32_t* sorted_pairs, int64_t T, int64_t H, int64_t R, int top_k, void* rows,
                   int32_t* pair_rows, hipStream_t stream) {
  const int64_t P = T * top_k, nv = (H + kN - 1) / kN;
  const bool in_blocks = P <= kInvertInBlocks;
  const int chunks = in_blocks ? (int)((P + kPairChunk - 1) / kPairChunk) : 0;
  if (in_blocks && R * H * (int64_t)sizeof(E) < kByTokenBytes) {
    const RowSplit sp = row_split(R, nv);
    permute_kernel<E, kN><<<chunks + split_blocks(R, sp), kThreads, 0, stream>>>(
        static_cast<const E*>(x), sorted_pairs, static_cast<E*>(rows), pair_rows, R, P, (int)H, top_k, sp, chunks);
    return hipGetLastError();
  }
  if (in_blocks) {
    if (chunks > 0) invert_kernel<<<chunks, 1024, 0, stream>>>(sorted_pairs, R, P, pair_rows);
  } else {
    clear_pair_rows_kernel<<<block_count(P, kThreads), kThreads, 0, stream>>>(pair_rows, P);
    if (R > 0)
      enter_pair_rows_kernel<<<block_count(R, kThreads), kThreads, 0, stream>>>(sorted_pairs, R, P, pair_rows);
  }
  if (R == 0) return hipGetLastError();
  const RowSplit sp = row_split(T, nv);
  const unsigned token_blocks = split_blocks(T, sp);
  permute_by_token_kernel<E, kN><<<token_blocks + block_count(R, kZeroRows * kThreads / 64), kThreads, 0, stream>>>(
      static_cast<const E*>(x), sorted_pairs, static_cast<E*>(rows), pair_rows, T, R, (int)H, top_k, sp,
      (int)token_blocks);
  return hipGetLastError();
}

template <typename E, int kN>
hipError_t unpermute(const void* rows, const int32_t* pair_rows, const float* weights, int64_t T, int64_t H,
                     int64_t R, int top_k, void* y, hipStream_t stream) {
  const RowSplit sp = row_split(T, (H + kN - 1) / kN);
  unpermute_kernel<E, kN><<<split_blocks(T, sp), kThreads, 0, stream>>>(
      static_cast<const E*>(rows), pair_rows, weights, static_cast<E*>(y), T, R, (int)H, top_k, sp);
  return hipGetLastError();
}

// Tokens from which a wave each fills the chip; below, four waves take one
// token (us with four and with one: 256, 1024, 1536, 2048 and 4096 tokens, top
// 4, 2880 bf16: 6.2 and 8.9, 11.4 and 12.0, 15.2 and 15.9, 22.6 and 21.7, 48.0
// and 47.7; 1024 bf16, top 2, 512, 1536, 2048 and 4096 tokens: 4.2 and 4.4, 6.2
// and 6.0, 8.5 and 6.8, 12.3 and 9.7).  Rows of up to 64 pieces are one wave's.
constexpr int64_t kManyTokens = 2048;

template <typename E, int kN>
hipError_t unpermute_backward(const void* dy, const void* rows, const int32_t* sorted_pairs,
                              const int32_t* pair_rows, const float* weights, int64_t T, int64_t H, int64_t R,
                              int top_k, void* d_rows, float* d_weights, hipStream_t stream) {
  const int nv = (int)((H + kN - 1) / kN), row_blocks = (int)block_count(R, kZeroRows * kThreads / 64);
  const bool split = T < kManyTokens && nv > 64;
  const int token_blocks = (int)block_count(T, split ? 1 : kThreads / 64);
  const auto kernel = split ? unpermute_backward_kernel<E, kN, 4> : unpermute_backward_kernel<E, kN, 1>;
  kernel<<<token_blocks + row_blocks, kThreads, 0, stream>>>(
      static_cast<const E*>(dy), static_cast<const E*>(rows), sorted_pairs, pair_rows, weights,
      static_cast<E*>(d_rows), d_weights, T, R, (int)H, top_k, nv, token_blocks);
  return hipGetLastError();
}

}  // namespace

namespace mxfp4moe {

size_t element_bytes(int dtype) { return dtype == kF32 ? 4 : 2; }

// The call on 16-byte pieces, or on single elements for shorter rows.
#define MX_BY_PIECE(FN, E, ...) (H * (int64_t)sizeof(E) >= 16 ? FN<E, 16 / (int)sizeof(E)>(__VA_ARGS__) : FN<E, 1>(__VA_ARGS__))
#define MX_BY_TYPE(FN, ...)                               \
  (dtype == kF32   ? MX_BY_PIECE(FN, float, __VA_ARGS__)    \
   : dtype == kF16 ? MX_BY_PIECE(FN, _Float16, __VA_ARGS__) \
                   : MX_BY_PIECE(FN, __bf16, __VA_ARGS__))

hipError_t launch_permute(const void* x, int dtype, const int32_t* sorted_pairs, int64_t T, int64_t H, int64_t top_k,
                          int64_t R, void* rows, int32_t* pair_rows, hipStream_t stream) {
  if (R == 0 && T == 0) return hipSuccess;
  const int k = (int)top_k;
  ProfileScope prof(kStagePermute, stream);
  return dtype == kF32 ? MX_BY_PIECE(permute, uint32_t, x, sorted_pairs, T, H, R, k, rows, pair_rows, stream)
                       : MX_BY_PIECE(permute, uint16_t, x, sorted_pairs, T, H, R, k, rows, pair_rows, stream);
}

hipError_t launch_unpermute(const void* rows, int dtype, const int32_t* pair_rows, const float* weights, int64_t T,
                            int64_t H, int64_t top_k, int64_t R, void* y, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  ProfileScope prof(kStageUnpermute, stream);
  return MX_BY_TYPE(unpermute, rows, pair_rows, weights, T, H, R, (int)top_k, y, stream);
}

hipError_t launch_unpermute_backward(const void* dy, const void* rows, int dtype, const int32_t* sorted_pairs,
                                     const int32_t* pair_rows, const float* weights, int64_t T, int64_t H,
                                     int64_t top_k, int64_t R, void* d_rows, float* d_weights, hipStream_t stream) {
  if (T == 0 && R == 0) return hipSuccess;
  ProfileScope prof(kStageUnpermuteBackward, stream);
  return MX_BY_TYPE(unpermute_backward, dy, rows, sorted_pairs, pair_rows, weights, T, H, R, (int)top_k, d_rows,
                    d_weights, stream);
}

#undef MX_BY_TYPE
#undef MX_BY_PIECE

hipError_t launch_route_backward(const int32_t* ids, const float* weights, const float* d_weights, int64_t T,
                                 int64_t E, int64_t top_k, float* d_logits, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  // fewer tokens a block while two blocks a CU are not there, or a block writes more than 8 KB (tokens 32, 16 and 8: T =
  // 4096, E = 128, top 8: 4.0, 3.7 and 3.6 us; T = 32768, E = 128: 6.3, 6.2 and 7.2; E = 32: 3.8, 4.3 and 5.6)
  int tokens = kRouteTokens;
  while (tokens > 8 && ((T + tokens - 1) / tokens < 2 * device_cu_count() || (tokens > 16 && tokens * E > 2048)))
    tokens /= 2;
  ProfileScope prof(kStageRouteBackward, stream);
  route_backward_kernel<<<block_count(T, tokens), kThreads, ((size_t)tokens * E + 3) / 4 * 16, stream>>>(
      ids, weights, d_weights, d_logits, T, (int)E, (int)top_k, tokens);
  return hipGetLastError();
}

}  // namespace mxfp4moe
