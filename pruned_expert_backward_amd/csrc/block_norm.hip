// The norms around a block, with its gate and residual scale:
//
//   b = y  or  y rms(y) w_b,   s = c x + g b,   h = s rms(s) w
//   rms(v) = (mean(v^2) + eps)^-1/2
//
// and the gradient, with n = s rms(s), z = y rms(y), from ds and dh:
//
//   d   = ds + rms(s) (dh w - n mean(dh w n))        what arrives at s
//   dx  = c d
//   dy  = rms(y) (d g w_b - z mean(d g w_b z))       without w_b: d g
//   dw  = sum over rows dh n,  dw_b = sum d g z,  dg = sum d b (over rows or columns)
//
// Memory bound: the forward reads x and y and writes s and h, the gradient
// reads ds, dh, s and y and writes dx and dy; everything between stays in registers.
// A row belongs to WPR waves; each lane holds PIECES 16-byte pieces of it and of the
// weights, which stay in registers over the rows that the waves go through.  The sums
// over rows stay in registers too; every group of waves leaves its own in the
// workspace and a second kernel adds them in one order.
#include <algorithm>

#include "forward.h"
#include "row_norm.h"

namespace lrmoe {
namespace {

template <typename T>
constexpr int kPiece = 16 / (int)sizeof(T);   // values of a piece

// Sums of K values over the WPR waves of a row (uniform).  Two sets of slots in
// turn: a wave that is ahead does not write what another one still reads.
template <int WPR, int K>
struct RowSum {
  float (*slots)[K][WPR];   // [2] in LDS
  int turn = 0;
  __device__ __forceinline__ void operator()(float (&v)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
    if constexpr (WPR > 1) {
      const int wave = threadIdx.x >> 6;
      if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) slots[turn][k][wave] = v[k];
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float t = slots[turn][k][0];
#pragma unroll
        for (int w = 1; w < WPR; ++w) t += slots[turn][k][w];
        v[k] = t;
      }
      turn ^= 1;
    }
  }
};

// Piece i of this lane starts at column at(i).
template <typename T, int WPR, int PIECES>
struct Row {
  static constexpr int N = kPiece<T>;
  static constexpr int kWaves = WPR > 4 ? WPR : 4;      // waves of a workgroup
  static constexpr int kRows = kWaves / WPR;            // rows it works on at once
  static constexpr int kWidth = WPR * 64 * PIECES * N;  // columns it can hold
  __device__ __forceinline__ static int at(int i) {
    return (i * WPR * 64 + (int)(threadIdx.x % (WPR * 64))) * N;
  }
  __device__ __forceinline__ static void load(const void* p, int64_t row, int D,
                                              float (&v)[PIECES][N]) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
#pragma unroll
      for (int j = 0; j < N; ++j) v[i][j] = 0.f;
      if (at(i) < D) load_vals(static_cast<const T*>(p) + row * D + at(i), v[i]);
    }
  }
  __device__ __forceinline__ static void store(void* p, int64_t row, int D,
                                               const float (&v)[PIECES][N]) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
      if (at(i) < D) store_vals(static_cast<T*>(p) + row * D + at(i), v[i]);
  }
};

// A weight row, held as it is stored; all ones if there is none.
template <typename T, int PIECES>
struct Weight {
  vec4u w[PIECES];
  __device__ __forceinline__ void get(int i, float (&v)[kPiece<T>]) const {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(w[i][j] << 16);
        v[2 * j + 1] = __uint_as_float(w[i][j] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(w[i][j]);
    }
  }
  template <typename R>
  __device__ __forceinline__ void load(const void* p, int D) {
    constexpr uint32_t one = sizeof(T) == 2 ? 0x3F803F80u : 0x3F800000u;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      w[i] = vec4u{one, one, one, one};
      if (p != nullptr && R::at(i) < D)
        w[i] = *reinterpret_cast<const vec4u*>(static_cast<const T*>(p) + R::at(i));
    }
  }
};

__device__ __forceinline__ float inv_rms(float sumsq, int D, float eps) {
  return 1.f / sqrtf(sumsq / (float)D + eps);
}

template <typename T, int WPR, int PIECES>
__global__ __launch_bounds__(64 * (WPR > 4 ? WPR : 4)) void norm_kernel(NormArgs a, void* s,
                                                                        void* h) {
  typedef Row<T, WPR, PIECES> R;
  constexpr int N = R::N;
  __shared__ float slots[2][1][WPR];
  RowSum<WPR, 1> sum{slots};
  Weight<T, PIECES> wb, gc, w;
  wb.template load<R>(a.branch_weight, a.D);
  gc.template load<R>(a.gate_kind == LRMOE_BRANCH_GATE_CHANNEL ? a.gate : nullptr, a.D);
  w.template load<R>(a.weight, a.D);
  const int mine = WPR > 1 ? 0 : threadIdx.x >> 6;
  for (int64_t row = (int64_t)blockIdx.x * R::kRows + mine; row < a.T;
       row += (int64_t)gridDim.x * R::kRows) {
    float x[PIECES][N];
    R::load(a.x, row, a.D, x);
    if (a.y != nullptr) {
      float y[PIECES][N];
      R::load(a.y, row, a.D, y);
      float r = a.gate_kind == LRMOE_BRANCH_GATE_TOKEN ? static_cast<const float*>(a.gate)[row]
                                                       : 1.f;
      if (a.branch_weight != nullptr) {
        float q[1] = {0.f};
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
#pragma unroll
          for (int j = 0; j < N; ++j) q[0] += y[i][j] * y[i][j];
        sum(q);
        r *= inv_rms(q[0], a.D, a.eps);
      }
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        float u[N], g[N];
        wb.get(i, u);
        gc.get(i, g);
#pragma unroll
        for (int j = 0; j < N; ++j) x[i][j] = a.scale * x[i][j] + g[j] * (y[i][j] * r * u[j]);
      }
      R::store(s, row, a.D, x);
    }
    if (a.weight != nullptr) {
      float q[1] = {0.f};
#pragma unroll
      for (int i = 0; i < PIECES; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) q[0] += x[i][j] * x[i][j];
      sum(q);
      const float r = inv_rms(q[0], a.D, a.eps);
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        float u[N];
        w.get(i, u);
#pragma unroll
        for (int j = 0; j < N; ++j) x[i][j] = x[i][j] * r * u[j];
      }
      R::store(h, row, a.D, x);
    }
  }
}

// ---- gradient
// Groups of waves that a gradient call has (the workspace has a row of sums for
// each), and its sums over rows, in this order: dw, dw_b, dg.
constexpr int kGroups = 1024;
constexpr int kSums = 3;

template <typename T, int WPR, int PIECES>
__global__ __launch_bounds__(64 * (WPR > 4 ? WPR : 4)) void norm_grad_kernel(
    NormArgs a, const void* ds, const void* dh, void* dx, void* dy, float* dgate, float* ws,
    int sums) {
  typedef Row<T, WPR, PIECES> R;
  constexpr int N = R::N;
  __shared__ float slots3[2][3][WPR], slots1[2][1][WPR];
  RowSum<WPR, 3> sum3{slots3};
  RowSum<WPR, 1> sum1{slots1};
  const bool token = a.gate_kind == LRMOE_BRANCH_GATE_TOKEN;
  const bool norm = a.weight != nullptr, branch_norm = a.branch_weight != nullptr;
  Weight<T, PIECES> wb, gc, w;
  wb.template load<R>(a.branch_weight, a.D);
  gc.template load<R>(a.gate_kind == LRMOE_BRANCH_GATE_CHANNEL ? a.gate : nullptr, a.D);
  w.template load<R>(a.weight, a.D);
  float acc[kSums][PIECES][N];
#pragma unroll
  for (int k = 0; k < kSums; ++k)
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) acc[k][i][j] = 0.f;
  const int mine = WPR > 1 ? 0 : threadIdx.x >> 6;
  const int64_t group = (int64_t)blockIdx.x * R::kRows + mine;
  for (int64_t row = group; row < a.T; row += (int64_t)gridDim.x * R::kRows) {
    float d[PIECES][N], x[PIECES][N], y[PIECES][N], e[PIECES][N];
    if (ds != nullptr) R::load(ds, row, a.D, d);
    else
#pragma unroll
      for (int i = 0; i < PIECES; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) d[i][j] = 0.f;
    if (norm) {
      R::load(dh, row, a.D, e);
      R::load(a.x, row, a.D, x);
    }
    if (a.y != nullptr) R::load(a.y, row, a.D, y);
    float q[3] = {0.f, 0.f, 0.f};   // s^2, dh w s, y^2
    if (norm) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        float u[N];
        w.get(i, u);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          q[0] += x[i][j] * x[i][j];
          q[1] += e[i][j] * u[j] * x[i][j];
        }
      }
    }
    if (branch_norm) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) q[2] += y[i][j] * y[i][j];
    }
    if (norm || branch_norm) sum3(q);
    if (norm) {
      const float r = inv_rms(q[0], a.D, a.eps);
      const float c = r * q[1] / (float)a.D;
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        float u[N];
        w.get(i, u);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float n = x[i][j] * r;
          acc[0][i][j] += e[i][j] * n;
          d[i][j] += r * (e[i][j] * u[j] - n * c);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) e[i][j] = a.scale * d[i][j];
    R::store(dx, row, a.D, e);
    if (a.y == nullptr) continue;   // uniform
    const float r = branch_norm ? inv_rms(q[2], a.D, a.eps) : 1.f;
    float t[1] = {0.f};             // d g w_b z, without a token's gate
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      float u[N], g[N];
      wb.get(i, u);
      gc.get(i, g);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        y[i][j] *= r;
        t[0] += d[i][j] * g[j] * u[j] * y[i][j];
      }
    }
    if (branch_norm || token) sum1(t);
    const float tg = token ? static_cast<const float*>(a.gate)[row] : 1.f;
    if (token && dgate != nullptr && threadIdx.x % (WPR * 64) == 0) dgate[row] = t[0];
    const float c = branch_norm ? tg * t[0] / (float)a.D : 0.f;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      float u[N], g[N];
      wb.get(i, u);
      gc.get(i, g);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float dg = d[i][j] * g[j] * tg;
        acc[1][i][j] += dg * y[i][j];
        acc[2][i][j] += d[i][j] * y[i][j] * u[j];
        y[i][j] = r * (dg * u[j] - y[i][j] * c);
      }
    }
    R::store(dy, row, a.D, y);
  }
#pragma unroll
  for (int k = 0; k < kSums; ++k) {
    if (!(sums >> k & 1)) continue;
    float* out = ws + (group * kSums + k) * a.D;
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
      if (R::at(i) < a.D) store_vals(out + R::at(i), acc[k][i]);
  }
}

// Sums of all groups: a workgroup takes 64 columns of one sum, its 16 waves the
// groups in turn.
__global__ __launch_bounds__(1024) void norm_sums_kernel(const float* ws, int groups, int D,
                                                         float* dw, float* dwb, float* dg) {
  __shared__ float part[16][64];
  const int k = blockIdx.y;
  float* out = k == 0 ? dw : k == 1 ? dwb : dg;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane;
  float t = 0.f;
  if (col < D) {
#pragma unroll 8
    for (int g = wave; g < groups; g += 16) t += ws[((int64_t)g * kSums + k) * D + col];
  }
  part[wave][lane] = t;
  __syncthreads();
  if (wave != 0 || col >= D) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) t += part[w][lane];
  out[col] = t;
}

// Workgroups of a gradient call (each of them R::kRows groups).
template <typename R>
int grad_blocks(int64_t T) {
  return (int)std::min<int64_t>((T + R::kRows - 1) / R::kRows, kGroups / R::kRows);
}

template <typename T, int WPR, int PIECES>
hipError_t norm(const NormArgs& a, void* s, void* h, hipStream_t st) {
  typedef Row<T, WPR, PIECES> R;
  const int64_t blocks = std::min<int64_t>((a.T + R::kRows - 1) / R::kRows, 2048 * 4 / R::kWaves);
  hipLaunchKernelGGL((norm_kernel<T, WPR, PIECES>), dim3((uint32_t)blocks), dim3(64 * R::kWaves),
                     0, st, a, s, h);
  return hipGetLastError();
}

template <typename T, int WPR, int PIECES>
hipError_t norm_grad(const NormArgs& a, const void* ds, const void* dh, void* dx, void* dy,
                     float* dweight, float* dbranch_weight, float* dgate, float* ws,
                     hipStream_t st) {
  typedef Row<T, WPR, PIECES> R;
  float* dg = a.gate_kind == LRMOE_BRANCH_GATE_CHANNEL ? dgate : nullptr;
  const int sums = (dweight != nullptr) | (dbranch_weight != nullptr) << 1 | (dg != nullptr) << 2;
  const int blocks = grad_blocks<R>(a.T);   // no rows, no groups: the sums are zeros
  if (blocks > 0) {
    hipLaunchKernelGGL((norm_grad_kernel<T, WPR, PIECES>), dim3(blocks), dim3(64 * R::kWaves), 0,
                       st, a, ds, dh, dx, dy, dgate, ws, sums);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (sums == 0) return hipSuccess;
  hipLaunchKernelGGL(norm_sums_kernel, dim3((a.D + 63) / 64, kSums), dim3(1024), 0, st, ws,
                     blocks * R::kRows, a.D, dweight, dbranch_weight, dg);
  return hipGetLastError();
}

// The narrowest shape that holds the row (columns in bf16; float32 half of them).
template <typename T, typename F>
hipError_t by_width(int D, F&& f) {
  constexpr int N = kPiece<T>, P = 8 / N;   // float32 takes twice the pieces
  if (D <= 512) return f(std::integral_constant<int, 1>(), std::integral_constant<int, P>());
  if (D <= 2048) return f(std::integral_constant<int, 4>(), std::integral_constant<int, P>());
  if (D <= 8192) return f(std::integral_constant<int, 16>(), std::integral_constant<int, P>());
  return f(std::integral_constant<int, 16>(), std::integral_constant<int, 2 * P>());
}

}  // namespace

hipError_t launch_residual_norm(int dtype, const NormArgs& a, void* s, void* h, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  if (dtype == LRMOE_BF16)
    return by_width<uint16_t>(a.D, [&](auto w, auto p) {
      return norm<uint16_t, w, p>(a, s, h, st);
    });
  return by_width<float>(a.D, [&](auto w, auto p) { return norm<float, w, p>(a, s, h, st); });
}

size_t residual_norm_workspace(int64_t T, int32_t D) {
  return (size_t)std::min<int64_t>((T + 3) / 4 * 4, kGroups) * kSums * D * sizeof(float);
}

hipError_t launch_residual_norm_backward(int dtype, const NormArgs& a, const void* ds,
                                         const void* dh, void* dx, void* dy, float* dweight,
                                         float* dbranch_weight, float* dgate, float* ws,
                                         hipStream_t st) {
  if (dtype == LRMOE_BF16)
    return by_width<uint16_t>(a.D, [&](auto w, auto p) {
      return norm_grad<uint16_t, w, p>(a, ds, dh, dx, dy, dweight, dbranch_weight, dgate, ws, st);
    });
  return by_width<float>(a.D, [&](auto w, auto p) {
    return norm_grad<float, w, p>(a, ds, dh, dx, dy, dweight, dbranch_weight, dgate, ws, st);
  });
}

}  // namespace lrmoe
