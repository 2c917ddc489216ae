// Tokens to experts and back: the stable sort of routed pairs by expert, the
// row dispatch, the weighted combine, and their gradients.
//
//   sort      ids [T, K] -> position of every pair (t, k) in expert order
//             (equal experts in ascending t K + k), segment offsets, counts,
//             and the pairs' tokens and weights in that order.  Pairs whose
//             id is outside 0..E-1 belong to another rank: position -1, and
//             the entries behind the last pair say token -1, weight 0.
//   dispatch  xp[pos[t, k]] = x[t]
//   combine   y[t] = residual[t] + sum_k w[t, k] rows[pos[t, k]], k ascending,
//             in float32, rounded once; with w = 1 it is dispatch's gradient
//   combine's gradient   drows[pos[t, k]] = w[t, k] dy[t],
//             dw[t, k] = <dy[t], rows[pos[t, k]]>, float32 sums
//
// All of them go by token (not by pair): the K rows of a token meet in one
// wave, so x and dy are read once and a sum needs no atomics and has one
// order.  They are bound by memory traffic; a copy on this card moves 5.1 TB/s
// (32768 tokens, 8 slots, rows of 2048 bf16: dispatch 231 us, 5.2 TB/s; combine
// onto a residual 258 us, 5.2 TB/s; its gradient, 8191 tokens with rows of
// 4096, 225 us, 5.1 TB/s).  Narrow rows leave lanes idle: at 64 columns (32768
// tokens, 8 slots) dispatch and combine run at 2.1 and 1.9 TB/s, from 256 columns
// on at a copy's rate; combine's gradient, which gives a token a whole workgroup,
// at 1.7 TB/s with 256 columns, 2.6 with 512, 4.4 with 1024.  A position outside
// 0..P-1 is skipped.
#include "forward.h"

namespace lrmoe {
namespace {

// ------------------------------------------------------------------ sort
// A workgroup owns a run of ids, each of its 16 waves a contiguous part of
// it.  Counting fills one LDS histogram per wave; a scan over waves (and over
// the workgroups before this one, from their histograms in the workspace)
// turns them into the first position of each wave's pairs of each expert; a
// second walk over the ids, 64 at a time, ranks the lanes that hold the same
// expert by ballots over the bits of the id.  Bin E holds the pairs of other
// ranks.  Up to kOneBlock ids the one workgroup does it all in one launch
// (64 tokens, 8 slots: 4.2 us); more take a histogram launch first (262144 ids
// over 128 experts 12.6 us, of which the two launches are 5 and 8; 655360 ids 23
// us; with 8192 ids a workgroup instead of 2048 20.5 and 27 us).  Each workgroup
// reads the histograms of all, so past that their number squared counts: 2.4
// million ids take 68 us over 128 experts and 96 us over 256.
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kOneBlock = 4096;   // ids of a call that one workgroup sorts
constexpr int kBlockIds = 2048;   // ids of a workgroup otherwise
constexpr int kMaxBlocks = 1024;
constexpr int kMaxBins = kMaxSegs + 1;

struct SortShape {
  int blocks;
  int64_t per_block;   // ids of a workgroup, a multiple of its waves' part
  int64_t per_wave;    // a multiple of 64
};
SortShape sort_shape(int64_t n) {
  SortShape s;
  int64_t blocks = n <= kOneBlock ? 1 : (n + kBlockIds - 1) / kBlockIds;
  if (blocks > kMaxBlocks) blocks = kMaxBlocks;
  const int64_t per = (n + blocks - 1) / blocks;
  s.per_wave = (per + kSortThreads - 1) / kSortThreads * 64;
  if (s.per_wave == 0) s.per_wave = 64;
  s.per_block = s.per_wave * kSortWaves;
  s.blocks = (int)((n + s.per_block - 1) / s.per_block);
  if (s.blocks == 0) s.blocks = 1;
  return s;
}

__device__ __forceinline__ int bin_of(int id, int E) { return id >= 0 && id < E ? id : E; }

// Counts ids[i] of the wave's live lanes.  Bin E, which holds most pairs where
// most experts are on other ranks, is counted by a ballot: atomics of many
// lanes on one address go one after the other.
__device__ __forceinline__ void count(uint32_t* h, const int32_t* ids, int64_t i, int64_t hi,
                                      int E) {
  const bool live = i < hi;
  const int e = live ? bin_of(ids[i], E) : E;
  const unsigned long long others = __ballot(live && e == E);
  if (e < E) atomicAdd(&h[e], 1u);
  if ((threadIdx.x & 63) == 0 && others) atomicAdd(&h[E], (uint32_t)__popcll(others));
}

__global__ __launch_bounds__(kSortThreads) void sort_hist_kernel(const int32_t* __restrict__ ids,
                                                                 int64_t n, int E,
                                                                 int64_t per_block,
                                                                 uint32_t* __restrict__ hist) {
  __shared__ uint32_t h[kMaxBins];
  const int tid = threadIdx.x;
  for (int e = tid; e <= E; e += kSortThreads) h[e] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * per_block;
  const int64_t hi = lo + per_block < n ? lo + per_block : n;
  for (int64_t i0 = lo + (tid & ~63); i0 < hi; i0 += kSortThreads)
    count(h, ids, i0 + (tid & 63), hi, E);
  __syncthreads();
  for (int e = tid; e <= E; e += kSortThreads) hist[(int64_t)blockIdx.x * (E + 1) + e] = h[e];
}

__global__ __launch_bounds__(kSortThreads) void sort_kernel(
    const int32_t* __restrict__ ids, const float* __restrict__ weights, int64_t n, int K, int E,
    int64_t per_block, int64_t per_wave, const uint32_t* __restrict__ hist, int blocks, int bits,
    int64_t* __restrict__ counts, int32_t* __restrict__ seg_offsets,
    int32_t* __restrict__ row_index, int32_t* __restrict__ pos, float* __restrict__ alpha) {
  __shared__ uint32_t wave_h[kSortWaves][kMaxBins];
  __shared__ uint32_t total[kMaxBins];   // pairs of each bin, then its first position
  __shared__ uint32_t before[kMaxBins];  // ... those of the workgroups before this one
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int bins = E + 1;
  for (int i = tid; i < kSortWaves * kMaxBins; i += kSortThreads) (&wave_h[0][0])[i] = 0;
  for (int e = tid; e < bins; e += kSortThreads) total[e] = before[e] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * per_block + wave * per_wave;
  const int64_t hi = lo + per_wave < n ? lo + per_wave : n;
  for (int64_t i0 = lo; i0 < hi; i0 += 64) count(wave_h[wave], ids, i0 + lane, hi, E);
  if (blocks > 1) {
    // 4 groups of 256 threads add up every fourth workgroup's histogram
    for (int e = tid & 255; e < bins; e += 256) {
      uint32_t all = 0, early = 0;
#pragma unroll 8
      for (int b = tid >> 8; b < blocks; b += kSortThreads / 256) {
        const uint32_t c = hist[(int64_t)b * bins + e];
        all += c;
        early += b < (int)blockIdx.x ? c : 0u;
      }
      atomicAdd(&total[e], all);   // whole numbers: any order
      atomicAdd(&before[e], early);
    }
  }
  __syncthreads();
  for (int e = tid; e < bins; e += kSortThreads) {   // waves of this workgroup, in order
    uint32_t run = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = wave_h[w][e];
      wave_h[w][e] = run;
      run += c;
    }
    if (blocks == 1) total[e] = run;
  }
  __syncthreads();
  if (wave == 0) {   // first position of each bin: 5 bins a lane (257 at most)
    constexpr int per = (kMaxBins + 63) / 64;
    uint32_t c[per], sum = 0;
#pragma unroll
    for (int j = 0; j < per; ++j) {
      const int e = lane * per + j;
      c[j] = e < bins ? total[e] : 0u;
      sum += c[j];
    }
    uint32_t run = sum;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const uint32_t o = __shfl_up(run, m, 64);
      if (lane >= m) run += o;
    }
    run -= sum;
#pragma unroll
    for (int j = 0; j < per; ++j) {
      const int e = lane * per + j;
      if (e < bins) {
        total[e] = run;
        if (blockIdx.x == 0) {
          seg_offsets[e] = (int32_t)run;   // bin E starts where the last expert ends
          if (e < E) counts[e] = c[j];
        }
      }
      run += c[j];
    }
  }
  __syncthreads();
  for (int i = tid; i < kSortWaves * bins; i += kSortThreads) {
    const int w = i / bins, e = i - w * bins;
    wave_h[w][e] += total[e] + before[e];
  }
  __syncthreads();
  uint32_t* mine = wave_h[wave];   // next position of each bin, this wave's own
  for (int64_t i0 = lo; i0 < hi; i0 += 64) {
    const int64_t i = i0 + lane;
    const bool live = i < hi;
    const int e = live ? bin_of(ids[i], E) : -1;
    unsigned long long same = __ballot(live);
    for (int b = 0; b < bits; ++b) {
      const unsigned long long set = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? set : ~set;
    }
    if (live) {
      const int rank = __popcll(same & ((1ull << lane) - 1));
      const uint32_t p = mine[e] + rank;
      if (e < E) {
        row_index[p] = (int32_t)(i / K);
        pos[i] = (int32_t)p;
      } else {
        row_index[p] = -1;
        pos[i] = -1;
      }
      if (alpha != nullptr) alpha[p] = e < E ? weights[i] : 0.f;
      if (rank == 0) mine[e] = p + __popcll(same);   // the lowest lane of the bin
    }
    // LDS accesses of one wave stay in order: the next round reads the sums
    // written here
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// ------------------------------------------------------- rows and tokens
constexpr int kRowThreads = 256;
constexpr int kRowWaves = kRowThreads / 64;

// Jobs of a kernel are walked with the grid's stride: at most this many
// workgroups are launched (a launch holds fewer than 2^32 threads).
constexpr int64_t kMaxGrid = int64_t(1) << 22;
dim3 row_grid(int64_t blocks) { return dim3((uint32_t)(blocks < kMaxGrid ? blocks : kMaxGrid)); }

// Wave-uniform position of slot k of token t, or -1.
__device__ __forceinline__ int64_t place(const int32_t* pos, int64_t at, int64_t P) {
  const int32_t p = __builtin_amdgcn_readfirstlane(pos[at]);
  return p >= 0 && p < P ? p : -1;
}

// dispatch: a wave moves one 4 KiB piece of one token's row to the K places.
// Pieces are counted in 16-byte units (row length in units: W).
constexpr int kPiece = 4;   // 16-byte loads of a lane
__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(
    const vec4u* __restrict__ x, const int32_t* __restrict__ pos, int64_t tokens, int K, int W,
    int pieces, int64_t P, vec4u* __restrict__ xp) {
  const int lane = threadIdx.x & 63;
  const int64_t jobs = tokens * pieces;
  for (int64_t job = (int64_t)blockIdx.x * kRowWaves +
                     __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
       job < jobs; job += (int64_t)gridDim.x * kRowWaves) {
    const int64_t t = job / pieces;
    const int c0 = (int)(job - t * pieces) * (64 * kPiece) + lane;
    vec4u v[kPiece];
#pragma unroll
    for (int j = 0; j < kPiece; ++j)
      if (c0 + 64 * j < W) v[j] = x[t * W + c0 + 64 * j];
    for (int k = 0; k < K; ++k) {
      const int64_t p = place(pos, t * K + k, P);
      if (p < 0) continue;
#pragma unroll
      for (int j = 0; j < kPiece; ++j)
        if (c0 + 64 * j < W) xp[p * W + c0 + 64 * j] = v[j];
    }
  }
}

// combine: a wave sums one piece of 64 * N columns of one token's K rows.
template <typename TI, typename TO, int N, bool WEIGHTED>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(
    const TI* __restrict__ rows, const int32_t* __restrict__ pos,
    const float* __restrict__ weights, const TO* __restrict__ residual, int64_t tokens, int K,
    int D, int pieces, int64_t P, TO* __restrict__ y) {
  const int lane = threadIdx.x & 63;
  const int64_t jobs = tokens * pieces;
  for (int64_t job = (int64_t)blockIdx.x * kRowWaves +
                     __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
       job < jobs; job += (int64_t)gridDim.x * kRowWaves) {
    const int64_t t = job / pieces;
    const int c = ((int)(job - t * pieces) * 64 + lane) * N;
    if (c >= D) continue;
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
    if (residual != nullptr) load_vals(residual + t * D + c, acc);
    constexpr int U = 4;   // rows in flight
    for (int k0 = 0; k0 < K; k0 += U) {
      float v[U][N], w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t p = k0 + u < K ? place(pos, t * K + k0 + u, P) : -1;
        w[u] = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) v[u][i] = 0.f;
        if (p >= 0) {
          load_vals(rows + p * D + c, v[u]);
          if (WEIGHTED) w[u] = weights[t * K + k0 + u];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < N; ++i)
          acc[i] = WEIGHTED ? fmaf(w[u], v[u][i], acc[i]) : acc[i] + v[u][i];
    }
    store_vals(y + t * D + c, acc);
  }
}

// combine's gradient: a workgroup takes one token; its waves share the row's
// columns, the dot products meet in LDS.
constexpr int kSlots = 8;   // slots of one walk over the row
template <typename T, int N>
__global__ __launch_bounds__(kRowThreads) void combine_backward_kernel(
    const T* __restrict__ dy, const T* __restrict__ rows, const int32_t* __restrict__ pos,
    const float* __restrict__ weights, int64_t tokens, int K, int D, int64_t P,
    T* __restrict__ drows, float* __restrict__ dweights) {
  __shared__ float part[kRowWaves][kSlots];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
    for (int k0 = 0; k0 < K; k0 += kSlots) {
      int64_t p[kSlots];
      float w[kSlots], dot[kSlots];
#pragma unroll
      for (int k = 0; k < kSlots; ++k) {
        p[k] = k0 + k < K ? place(pos, t * K + k0 + k, P) : -1;
        w[k] = p[k] >= 0 ? weights[t * K + k0 + k] : 0.f;
        dot[k] = 0.f;
      }
      for (int c = tid * N; c < D; c += kRowThreads * N) {
        float g[N];
        load_vals(dy + t * D + c, g);
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
          if (p[k] < 0) continue;
          float v[N], o[N];
          load_vals(rows + p[k] * D + c, v);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            dot[k] = fmaf(g[i], v[i], dot[k]);
            o[i] = w[k] * g[i];
          }
          store_vals(drows + p[k] * D + c, o);
        }
      }
#pragma unroll
      for (int k = 0; k < kSlots; ++k) {
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) dot[k] += __shfl_xor(dot[k], m, 64);
        if (lane == 0) part[wave][k] = dot[k];
      }
      __syncthreads();
      if (tid < kSlots && k0 + tid < K) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kRowWaves; ++i) s += part[i][tid];
        dweights[t * K + k0 + tid] = s;   // 0 for a slot without a row
      }
      __syncthreads();
    }
  }
}

template <typename TI, typename TO, int N>
hipError_t combine(const void* rows, const int32_t* pos, const float* weights,
                   const void* residual, int64_t T, int K, int D, int64_t P, void* y,
                   hipStream_t s) {
  const int pieces = (D + 64 * N - 1) / (64 * N);
  const dim3 grid = row_grid((T * pieces + kRowWaves - 1) / kRowWaves), block(kRowThreads);
  const TI* r = static_cast<const TI*>(rows);
  const TO* res = static_cast<const TO*>(residual);
  if (weights != nullptr)
    hipLaunchKernelGGL((combine_kernel<TI, TO, N, true>), grid, block, 0, s, r, pos, weights, res,
                       T, K, D, pieces, P, static_cast<TO*>(y));
  else
    hipLaunchKernelGGL((combine_kernel<TI, TO, N, false>), grid, block, 0, s, r, pos, weights, res,
                       T, K, D, pieces, P, static_cast<TO*>(y));
  return hipGetLastError();
}

}  // namespace

size_t route_sort_workspace(int64_t n, int32_t E) {
  const SortShape sh = sort_shape(n);
  return sh.blocks > 1 ? (size_t)sh.blocks * (E + 1) * sizeof(uint32_t) : 0;
}

hipError_t launch_route_sort(const int32_t* ids, const float* weights, int64_t T, int32_t K,
                             int32_t E, int64_t* counts, int32_t* seg_offsets, int32_t* row_index,
                             int32_t* pos, float* alpha, uint32_t* ws, hipStream_t s) {
  const int64_t n = T * K;
  const SortShape sh = sort_shape(n);
  if (sh.blocks > 1) {
    hipLaunchKernelGGL(sort_hist_kernel, dim3(sh.blocks), dim3(kSortThreads), 0, s, ids, n, E,
                       sh.per_block, ws);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  int bits = 1;
  while ((1 << bits) < E + 1) ++bits;
  hipLaunchKernelGGL(sort_kernel, dim3(sh.blocks), dim3(kSortThreads), 0, s, ids, weights, n, K, E,
                     sh.per_block, sh.per_wave, ws, sh.blocks, bits, counts, seg_offsets,
                     row_index, pos, alpha);
  return hipGetLastError();
}

hipError_t launch_dispatch(int dtype, const void* x, const int32_t* pos, int64_t T, int32_t K,
                           int32_t D, int64_t P, void* xp, hipStream_t s) {
  if (T == 0) return hipSuccess;
  const int W = D / (dtype == LRMOE_BF16 ? 8 : 4);
  const int pieces = (W + 64 * kPiece - 1) / (64 * kPiece);
  hipLaunchKernelGGL(dispatch_kernel, row_grid((T * pieces + kRowWaves - 1) / kRowWaves),
                     dim3(kRowThreads), 0, s, static_cast<const vec4u*>(x), pos, T, K, W, pieces,
                     P, static_cast<vec4u*>(xp));
  return hipGetLastError();
}

hipError_t launch_combine(int in_dtype, int out_dtype, const void* rows, const int32_t* pos,
                          const float* weights, const void* residual, int64_t T, int32_t K,
                          int32_t D, int64_t P, void* y, hipStream_t s) {
  if (T == 0) return hipSuccess;
  if (in_dtype == LRMOE_BF16 && out_dtype == LRMOE_BF16)
    return combine<uint16_t, uint16_t, 8>(rows, pos, weights, residual, T, K, D, P, y, s);
  if (in_dtype == LRMOE_BF16)
    return combine<uint16_t, float, 8>(rows, pos, weights, residual, T, K, D, P, y, s);
  if (out_dtype == LRMOE_BF16)
    return combine<float, uint16_t, 8>(rows, pos, weights, residual, T, K, D, P, y, s);
  return combine<float, float, 4>(rows, pos, weights, residual, T, K, D, P, y, s);
}

hipError_t launch_combine_backward(int dtype, const void* dy, const void* rows, const int32_t* pos,
                                   const float* weights, int64_t T, int32_t K, int32_t D,
                                   int64_t P, void* drows, float* dweights, hipStream_t s) {
  if (T == 0) return hipSuccess;
  const dim3 grid = row_grid(T), block(kRowThreads);
  if (dtype == LRMOE_BF16)
    hipLaunchKernelGGL((combine_backward_kernel<uint16_t, 8>), grid, block, 0, s,
                       static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(rows), pos,
                       weights, T, K, D, P, static_cast<uint16_t*>(drows), dweights);
  else
    hipLaunchKernelGGL((combine_backward_kernel<float, 4>), grid, block, 0, s,
                       static_cast<const float*>(dy), static_cast<const float*>(rows), pos,
                       weights, T, K, D, P, static_cast<float*>(drows), dweights);
  return hipGetLastError();
}

}  // namespace lrmoe
