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
// reads ds, dh, s and y and writes dx and dy.
// A row belongs to WPR waves; each lane holds PIECES 16-byte pieces of it and of the
// weights, which stay in registers over the rows that the waves go through.  The sums
// over rows stay with the lanes too; every group of waves leaves its own in the
// workspace and a second kernel adds them in one order.  The gradient loads a row ahead.
// All of that fits the registers in the forward, and in the gradient for rows up to
// 8192 columns in bfloat16 and 4096 in float32.  Beyond, 16 waves a row leave a lane of the
// gradient 128 registers, and it spills: in float32 29 of them up to 8192 columns, above
// 8192 columns 147 in bfloat16 and 338 in float32.
// bfloat16, TB/s: 32768 x 2048 104 us (5.2), its gradient with all sums 158 us (5.1);
// 32768 x 4096 209 and 294 us, 8192 x 8192 100 and 163, 32768 x 512 22 and 45.
// float32: 32768 x 2048 209 us (5.1) and 310 (5.2), 16384 x 4096 204 and 294 (5.5).  With
// spills: float32 8192 x 8192 203 and 367 us (4.4), 4096 x 16384 in bfloat16 101 and 669
// (1.2), in float32 198 and 1096 us (1.5).
// 16 rows 3.1 us, 512 rows' gradient 15.5 us: two launches and a few waits.
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

template <typename T>
__device__ __forceinline__ void unpack(const vec4u& w, float (&v)[kPiece<T>]) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(w[j]);
  }
}

// Piece i of this lane starts at column at(i).
template <typename T, int WPR, int PIECES>
struct Row {
  static constexpr int N = kPiece<T>;
  static constexpr int kWaves = WPR > 1 ? WPR : 4;      // waves of a workgroup: one row, or
                                                        // four rows without barriers
  static constexpr int kRows = kWaves / WPR;            // rows it works on at once
  static constexpr int kWidth = WPR * 64 * PIECES * N;  // columns it can hold
  __device__ __forceinline__ static int at(int i) {
    return (i * WPR * 64 + (int)(threadIdx.x % (WPR * 64))) * N;
  }
  // A row as it is stored (null: zeros), and its values.
  __device__ __forceinline__ static void load(const void* p, int64_t row, int D,
                                              vec4u (&w)[PIECES]) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      w[i] = vec4u{};
      if (p != nullptr && at(i) < D)
        w[i] = *reinterpret_cast<const vec4u*>(static_cast<const T*>(p) + row * D + at(i));
    }
  }
  __device__ __forceinline__ static void values(const vec4u (&w)[PIECES], float (&v)[PIECES][N]) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) unpack<T>(w[i], v[i]);
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
  __device__ __forceinline__ void get(int i, float (&v)[kPiece<T>]) const { unpack<T>(w[i], v); }
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
__global__ __launch_bounds__(64 * (WPR > 1 ? WPR : 4)) void norm_kernel(NormArgs a, void* s,
                                                                        void* h) {
  typedef Row<T, WPR, PIECES> R;
  constexpr int N = R::N;
  __shared__ float slots[2][1][WPR];
  RowSum<WPR, 1> sum{slots};
  Weight<T, PIECES> wb, gc, w;
  wb.template load<R>(a.branch_weight, a.D);
  gc.template load<R>(a.gate_kind == LRMOE_BRANCH_GATE_CHANNEL ? a.gate : nullptr, a.D);
  w.template load<R>(a.weight, a.D);
  const int mine = threadIdx.x / (WPR * 64);
  for (int64_t row = (int64_t)blockIdx.x * R::kRows + mine; row < a.T;
       row += (int64_t)gridDim.x * R::kRows) {
    float x[PIECES][N], y[PIECES][N];
    {
      vec4u wx[PIECES], wy[PIECES];
      R::load(a.x, row, a.D, wx);
      R::load(a.y, row, a.D, wy);
      R::values(wx, x);
      R::values(wy, y);
    }
    if (a.y != nullptr) {
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
// Groups of waves (one for a row) have a row of sums each in the workspace; its three
// kinds: dw, dw_b, dg.
constexpr int kSums = 3;

template <typename T, int WPR, int PIECES>
__global__ __launch_bounds__(64 * (WPR > 1 ? WPR : 4)) void norm_grad_kernel(
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
  const int mine = threadIdx.x / (WPR * 64);
  const int64_t group = (int64_t)blockIdx.x * R::kRows + mine;
  const int64_t stride = (int64_t)gridDim.x * R::kRows;
  vec4u wd[PIECES], we[PIECES], wx[PIECES], wy[PIECES];
  auto fetch = [&](int64_t row) __attribute__((always_inline)) {
    R::load(ds, row, a.D, wd);
    R::load(dh, row, a.D, we);
    R::load(norm ? a.x : nullptr, row, a.D, wx);
    R::load(a.y, row, a.D, wy);
  };
  if (group < a.T) fetch(group);
  for (int64_t row = group; row < a.T; row += stride) {
    float d[PIECES][N], x[PIECES][N], y[PIECES][N], e[PIECES][N];
    R::values(wd, d);
    R::values(we, e);
    R::values(wx, x);
    R::values(wy, y);
    if (row + stride < a.T) fetch(row + stride);   // under way while this row is worked on
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

// Sums of all groups: a workgroup takes 32 columns of one kind, its 32 half waves the
// groups in turn.  (512 rows of 2048: 15.5 us with the gradient, 20.6 with 16 columns, 16.1
// with 64.)
__global__ __launch_bounds__(1024) void norm_sums_kernel(const float* ws, int groups, int D,
                                                         float* dw, float* dwb, float* dg) {
  __shared__ float part[32][33];
  const int k = blockIdx.y;
  float* out = k == 0 ? dw : k == 1 ? dwb : dg;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float t = 0.f;
  if (col < D) {
#pragma unroll 8
    for (int g = row; g < groups; g += 32) t += ws[((int64_t)g * kSums + k) * D + col];
  }
  part[row][lane] = t;
  __syncthreads();
  if (threadIdx.x >= 32 || col >= D) return;
#pragma unroll
  for (int r = 1; r < 32; ++r) t += part[r][lane];
  out[col] = t;
}

// Most groups of a gradient call, for rows of `wpr` waves: those that 256 CUs hold at
// once, so that all rows are shared evenly.  12 waves a CU by their registers; of 8-wave
// workgroups one, of 16-wave ones (held to 128 registers) one.  (16 waves a CU
// throughout: 32768 x 2048 191 us, 163 like this; 32768 x 4096 310 and 294 us.)
int grad_groups(int wpr) { return 256 * (wpr <= 4 ? 12 : wpr == 8 ? 8 : 16) / wpr; }

// Workgroups of a gradient call (each of them R::kRows groups).
template <typename R>
int grad_blocks(int64_t T) {
  return (int)std::min<int64_t>((T + R::kRows - 1) / R::kRows,
                                grad_groups(R::kWaves / R::kRows) / R::kRows);
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
  hipLaunchKernelGGL(norm_sums_kernel, dim3((a.D + 31) / 32, kSums), dim3(1024), 0, st, ws,
                     blocks * R::kRows, a.D, dweight, dbranch_weight, dg);
  return hipGetLastError();
}

// Waves of a row and pieces of a lane: the narrowest shape that holds the row (512
// columns a wave in bf16 and, with twice the pieces, in float32; 16 waves and more pieces
// for the widest).
template <typename T, typename F>
hipError_t by_width(int D, F&& f) {
  constexpr int P = 8 / kPiece<T>;
  std::integral_constant<int, P> p;
  if (D <= 512) return f(std::integral_constant<int, 1>(), p);
  if (D <= 1024) return f(std::integral_constant<int, 2>(), p);
  if (D <= 2048) return f(std::integral_constant<int, 4>(), p);
  if (D <= 4096) return f(std::integral_constant<int, 8>(), p);
  if (D <= 8192) return f(std::integral_constant<int, 16>(), p);
  return f(std::integral_constant<int, 16>(), std::integral_constant<int, 2 * P>());
}
int waves_of_row(int D) {
  return D <= 512 ? 1 : D <= 1024 ? 2 : D <= 2048 ? 4 : D <= 4096 ? 8 : 16;
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
  return (size_t)std::min<int64_t>((T + 3) / 4 * 4, grad_groups(waves_of_row(D))) * kSums * D *
         sizeof(float);
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
