// Gradient of the grouped product's epilogue (bias and activation), ahead of
// the product's own gradients:
//
//   dz_u = dy_u act'(a_u)                          (a: saved pre-activations)
//   SwiGLU: dz_u = [ dy_u b_u SiLU'(a_u) | dy_u SiLU(a_u) ]
//   dbias_e = sum over the expert's rows of dz_u   (before dz's rounding)
//
//   SiLU'(a) = s (1 + a (1 - s)), s = sigmoid(a)
//   GELU'(a) = Phi(a) + a phi(a)
//
// Memory bound: dy, a (and b) are read once, dz written once.  A workgroup
// takes a run of kRows rows of one expert and LPR lanes' columns, its groups of
// LPR lanes take a row each in turn and keep the column sums in registers,
// which meet in LDS and go to the workspace, one row of sums for each run.  A second kernel
// adds an expert's runs in order, so the sums do not depend on timing.
// SwiGLU, 32768 x 768 bf16 (252 MB): 53 us, 4.7 TB/s, 47 of them in the first
// kernel; GELU, 32768 x 1536: 77 us, bound by the error function.
#include <algorithm>

#include "forward.h"

namespace lrmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 64;
constexpr int kBatch = 2;

// Runs of an expert with n rows.
__host__ __device__ inline int64_t runs_of(int64_t n) { return (n + kRows - 1) / kRows; }
// Bound of the runs of all experts.
int64_t max_runs(int64_t P, int E) { return P / kRows + (P < E ? P : E); }

// Segment e of the (untrusted) device offsets, inside [0, P].
__device__ __forceinline__ void segment(const int32_t* seg, int e, int64_t P, int64_t& lo,
                                        int64_t& hi) {
  lo = seg[e] < 0 ? 0 : seg[e] > P ? P : seg[e];
  hi = seg[e + 1] < lo ? lo : seg[e + 1] > P ? P : seg[e + 1];
}

// Expert of run r and the run's number inside it, or false past the last run.
// Every wave finds it for itself: lane l looks at experts 4 l .. 4 l + 3.
__device__ __forceinline__ bool find_run(const int32_t* seg, int E, int64_t P, int64_t r, int& e,
                                         int& sub) {
  const int lane = threadIdx.x & 63;
  int n[4], sum = 0;   // fewer than 2^31 / kRows + E runs in all
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    n[j] = 0;
    if (4 * lane + j < E) {
      int64_t lo, hi;
      segment(seg, 4 * lane + j, P, lo, hi);
      n[j] = (int)runs_of(hi - lo);
    }
    sum += n[j];
  }
  const int end = wave_scan(sum);
  const unsigned long long past = __ballot(end > r);
  if (past == 0) return false;
  const int owner = __ffsll(past) - 1;
  int at = (int)r - (end - sum), j = 0;   // meant for the owner lane
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (j == i && at >= n[i]) {
      at -= n[i];
      j = i + 1;
    }
  e = __builtin_amdgcn_readlane(4 * lane + j, owner);
  sub = __builtin_amdgcn_readlane(at, owner);
  return true;
}

// SiLU' or GELU'.
template <int ACT>
__device__ __forceinline__ float act_grad(float a) {
  static_assert(ACT == LRMOE_ACT_SILU || ACT == LRMOE_ACT_GELU, "the others have no function");
  if constexpr (ACT == LRMOE_ACT_SILU) {
    const float s = sigmoid_f32(a);
    return s + a * s * (1.f - s);
  } else {
    return 0.5f * (1.f + erff(a * 0.70710678f)) +
           a * (0.39894228f * __builtin_amdgcn_exp2f(-0.72134752f * a * a));   // exp(-a^2 / 2)
  }
}

template <typename T, typename TO, int N, int ACT, int LPR>
__global__ __launch_bounds__(kThreads) void act_backward_kernel(
    const int32_t* __restrict__ seg, const T* __restrict__ dy, const T* __restrict__ pa,
    const T* __restrict__ pb, int64_t P, int E, int F, TO* __restrict__ dz,
    float* __restrict__ sums, int64_t runs) {
  constexpr bool GLU = ACT == LRMOE_ACT_SWIGLU;
  constexpr int H = GLU ? 2 : 1;
  constexpr int kGroups = kThreads / LPR;   // rows at a time
  __shared__ float part[kGroups - 1][H * N][LPR];
  const int tid = threadIdx.x, lane = tid % LPR, group = tid / LPR;
  const int col = (int)blockIdx.y * (LPR * N) + lane * N;
  // runs go by the grid's stride: a launch holds fewer than 2^32 threads
  for (int64_t run = blockIdx.x; run < runs; run += gridDim.x) {
    int e, sub;
    if (!find_run(seg, E, P, run, e, sub)) return;   // the same answer in every wave
    int64_t lo, hi;
    segment(seg, e, P, lo, hi);
    if (sub < 0 || sub >= runs_of(hi - lo)) continue;   // offsets out of order: counts overflowed
    lo += (int64_t)sub * kRows;
    if (hi > lo + kRows) hi = lo + kRows;
    float acc[H][N];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int i = 0; i < N; ++i) acc[h][i] = 0.f;
    if (col < F) {
      // kBatch rows in flight: their loads go out before the first is used
      for (int64_t u0 = lo + group; u0 < hi; u0 += kBatch * kGroups) {
        float g[kBatch][N], a[kBatch][N], b[kBatch][N];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int64_t u = u0 + k * kGroups;
          if (u < hi) {
            load_vals(dy + u * F + col, g[k]);
            if (ACT != LRMOE_ACT_NONE) load_vals(pa + u * F + col, a[k]);
            if (GLU) load_vals(pb + u * F + col, b[k]);
          }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int64_t u = u0 + k * kGroups;
          if (u >= hi) break;
          float z[H][N];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            if constexpr (GLU) {
              const float s = sigmoid_f32(a[k][i]), as = a[k][i] * s;
              z[0][i] = g[k][i] * b[k][i] * (s + as * (1.f - s));
              z[H - 1][i] = g[k][i] * as;
            } else if constexpr (ACT == LRMOE_ACT_RELU) {
              z[0][i] = a[k][i] > 0.f ? g[k][i] : 0.f;
            } else if constexpr (ACT == LRMOE_ACT_NONE) {
              z[0][i] = g[k][i];
            } else {
              z[0][i] = g[k][i] * act_grad<ACT>(a[k][i]);
            }
          }
#pragma unroll
          for (int h = 0; h < H; ++h) {
            store_vals(dz + (u * H + h) * F + col, z[h]);
#pragma unroll
            for (int i = 0; i < N; ++i) acc[h][i] += z[h][i];
          }
        }
      }
    }
    if (sums == nullptr) continue;
    if (group > 0)
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int i = 0; i < N; ++i) part[group - 1][h * N + i][lane] = acc[h][i];
    __syncthreads();
    if (group == 0 && col < F) {
#pragma unroll
      for (int h = 0; h < H; ++h) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int w = 0; w < kGroups - 1; ++w) acc[h][i] += part[w][h * N + i][lane];
        store_vals(sums + (run * H + h) * F + col, acc[h]);
      }
    }
    __syncthreads();   // the next run writes the same LDS
  }
}

// dbias[e] = the expert's runs; 0 for an expert without rows.  A workgroup
// takes 64 columns; its 16 waves add a sixteenth of the runs each, in order, and
// the sixteen sums are added in order (one wave for all runs of an expert: 11.3
// us for 16 experts, 528 runs, 1536 columns; 5.4 us like this).
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(64 * kSumWaves) void dbias_kernel(const int32_t* __restrict__ seg,
                                                               int64_t P, int width, int64_t limit,
                                                               const float* __restrict__ sums,
                                                               float* __restrict__ dbias) {
  __shared__ float part[kSumWaves][64];
  const int e = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane;
  int64_t first = 0, lo, hi;
  for (int i = lane; i < e; i += 64) {
    segment(seg, i, P, lo, hi);
    first += runs_of(hi - lo);
  }
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) first += __shfl_xor(first, m, 64);
  segment(seg, e, P, lo, hi);
  // offsets that do not ascend may name more runs than there are: never read past them
  int64_t end = first + runs_of(hi - lo);
  if (end > limit) end = limit;
  const int64_t share = (end - first + kSumWaves - 1) / kSumWaves;
  const int64_t r0 = first + wave * share, r1 = r0 + share < end ? r0 + share : end;
  float s = 0.f;
  if (col < width)
#pragma unroll 8
    for (int64_t r = r0; r < r1; ++r) s += sums[r * width + col];
  part[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || col >= width) return;
#pragma unroll
  for (int w = 1; w < kSumWaves; ++w) s += part[w][lane];
  dbias[(int64_t)e * width + col] = s;
}

template <typename T, typename TO, int N, int LPR>
hipError_t run(int act, const int32_t* seg, const void* dy, const void* a, const void* b, int64_t P,
               int E, int F, void* dz, float* sums, hipStream_t s) {
  const int64_t runs = max_runs(P, E);
  if (runs == 0) return hipSuccess;
  const dim3 grid((uint32_t)std::min<int64_t>(runs, 1 << 22), (F + LPR * N - 1) / (LPR * N));
  const dim3 block(kThreads);
#define LRMOE_ACT(A)                                                                               \
  case A:                                                                                          \
    hipLaunchKernelGGL((act_backward_kernel<T, TO, N, A, LPR>), grid, block, 0, s, seg,            \
                       static_cast<const T*>(dy), static_cast<const T*>(a),                        \
                       static_cast<const T*>(b), P, E, F, static_cast<TO*>(dz), sums, runs);       \
    break
  switch (act) {
    LRMOE_ACT(LRMOE_ACT_NONE);
    LRMOE_ACT(LRMOE_ACT_RELU);
    LRMOE_ACT(LRMOE_ACT_SILU);
    LRMOE_ACT(LRMOE_ACT_GELU);
    LRMOE_ACT(LRMOE_ACT_SWIGLU);
  }
#undef LRMOE_ACT
  return hipGetLastError();
}

// Lanes of a row: as many as leave the fewest of them past its end (768 bf16
// columns: 64 lanes would idle in a quarter of their steps, 32 in none).
template <typename T, typename TO, int N>
hipError_t run(int act, const int32_t* seg, const void* dy, const void* a, const void* b, int64_t P,
               int E, int F, void* dz, float* sums, hipStream_t s) {
  const int units = (F + N - 1) / N;
  const int w64 = (units + 63) / 64 * 64, w32 = (units + 31) / 32 * 32;
  const int w16 = (units + 15) / 16 * 16;
  if (w64 <= w32) return run<T, TO, N, 64>(act, seg, dy, a, b, P, E, F, dz, sums, s);
  if (w32 <= w16) return run<T, TO, N, 32>(act, seg, dy, a, b, P, E, F, dz, sums, s);
  return run<T, TO, N, 16>(act, seg, dy, a, b, P, E, F, dz, sums, s);
}

}  // namespace

size_t act_backward_workspace(int64_t P, int32_t E, int32_t width) {
  return (size_t)max_runs(P, E) * width * sizeof(float);
}

hipError_t launch_act_backward(int dtype, int out_dtype, int act, const int32_t* seg,
                               const void* dy, const void* a, const void* b, int64_t P, int32_t E,
                               int32_t F, void* dz, float* dbias, float* ws, hipStream_t s) {
  float* sums = dbias != nullptr ? ws : nullptr;
  hipError_t err;
  if (dtype == LRMOE_BF16 && out_dtype == LRMOE_BF16)
    err = run<uint16_t, uint16_t, 8>(act, seg, dy, a, b, P, E, F, dz, sums, s);
  else if (dtype == LRMOE_BF16)
    err = run<uint16_t, float, 8>(act, seg, dy, a, b, P, E, F, dz, sums, s);
  else
    err = run<float, float, 4>(act, seg, dy, a, b, P, E, F, dz, sums, s);
  if (err != hipSuccess || dbias == nullptr) return err;
  const int width = F * (act == LRMOE_ACT_SWIGLU ? 2 : 1);
  hipLaunchKernelGGL(dbias_kernel, dim3((width + 63) / 64, E), dim3(64 * kSumWaves), 0, s,
                     seg, P, width, max_runs(P, E), sums, dbias);
  return hipGetLastError();
}

}  // namespace lrmoe
