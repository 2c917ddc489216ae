// The router's top-k gate and its gradient.
//
//   forward   key_e = x_e (softmax; sigmoid without a selection bias), or
//             sigmoid(x_e) + bias_e in float64.  The K largest keys of a row,
//             best first, ties to the lower expert.  Weights over the chosen
//             set C, with scale s:
//               softmax, renorm  s exp(x_k) / sum_{j in C} exp(x_j)
//               softmax          s exp(x_k) / sum_e exp(x_e)
//               sigmoid, renorm  s sig(x_k) / sum_{j in C} sig(x_j)
//               sigmoid          s sig(x_k)
//             A logit that is -inf or NaN is never chosen (+inf counts as the
//             largest finite value); slots left over get id -1, weight 0.
//   backward  with v_k = x[id_k], dw the gradient of the weights:
//               softmax, renorm  dx_k = s p_k (dw_k - sum_j p_j dw_j)
//               softmax          dx_e = s p_e ([e in C] dw_e - sum_j p_j dw_j)
//               sigmoid, renorm  dx_k = s r_k (dw_k - sum_j r_j dw_j) sig(-v_k),
//                                r_k = sig(v_k) / sum_j sig(v_j)
//               sigmoid          dx_k = s dw_k sig(v_k) sig(-v_k)
//             All other entries of the dense row are 0.  Slots with an id
//             outside 0..E-1 carry nothing; an id that stands twice in a row
//             counts as two slots whose gradients add up.
//
// Sigmoid sums: where the largest chosen logit is below -30, sig(v) = exp(v)
// to float32, and the ratio is taken as a softmax of v: sig(v) itself would
// underflow below -103.
//
// Mapping: LANES lanes own one row, V values each.  Rows of up to 256 experts
// and 16 slots take 16 lanes, so a wave works on four rows and the argmax
// needs four exchange steps instead of six; wider ones take the whole wave.
// The K rounds are a running argmax over registers: no LDS, no sorting.  The
// choice with a selection bias compares float64 keys, since the order of two
// near values decides a whole number.
#include <algorithm>
#include <type_traits>

#include "forward.h"

namespace lrmoe {
namespace {

constexpr int kThreads = 256;
constexpr float kNegInf = -__builtin_inff();
constexpr float kMaxF32 = 3.402823466e38f;

// A logit as the gate reads it: NaN as -inf, +inf as the largest finite value.
__device__ __forceinline__ float clean(float x) {
  return x == x ? fminf(x, kMaxF32) : kNegInf;
}
__device__ __forceinline__ float logit(const float* p, int64_t i) { return clean(p[i]); }
__device__ __forceinline__ float logit(const uint16_t* p, int64_t i) {
  return clean(bf16_to_f32(p[i]));
}

// Expert of slot v of lane l: runs of four consecutive experts per lane
// (fewer where a lane holds fewer), ascending in v.
template <int LANES, int V>
__device__ __forceinline__ int expert_of(int l, int v) {
  constexpr int R = V < 4 ? V : 4;
  return (v / R) * (LANES * R) + l * R + v % R;
}

template <typename T, int LANES, int V>
__device__ __forceinline__ void load_row(const T* row, int E, int l, float (&x)[V]) {
  if (V >= 4 && (E & 3) == 0) {   // the run of four is in the row as a whole or not at all
#pragma unroll
    for (int v = 0; v < V; v += 4) {
      const int e = expert_of<LANES, V>(l, v);
      if (e < E) {
        if constexpr (sizeof(T) == 4) {
          const vec4f w = *reinterpret_cast<const vec4f*>(row + e);
#pragma unroll
          for (int j = 0; j < 4; ++j) if (v + j < V) x[v + j] = clean(w[j]);
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(row + e);
          const uint32_t d[2] = {w.x, w.y};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (v + j < V)
              x[v + j] = clean(__uint_as_float((j & 1) ? (d[j >> 1] & 0xFFFF0000u)
                                                       : (d[j >> 1] << 16)));
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) if (v + j < V) x[v + j] = kNegInf;
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = expert_of<LANES, V>(l, v);
      x[v] = e < E ? logit(row, e) : kNegInf;
    }
  }
}

template <int LANES>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int m = 1; m < LANES; m <<= 1) x += __shfl_xor(x, m, LANES);
  return x;
}
template <int LANES>
__device__ __forceinline__ float group_max(float x) {
#pragma unroll
  for (int m = 1; m < LANES; m <<= 1) x = fmaxf(x, __shfl_xor(x, m, LANES));
  return x;
}

__device__ __forceinline__ float ratio(float num, float den) { return den > 0.f ? num / den : 0.f; }

template <typename T, typename Key, int LANES, int V, bool SIGMOID>
__global__ __launch_bounds__(kThreads) void gate_kernel(
    const T* __restrict__ logits, const float* __restrict__ bias, int64_t rows, int E, int K,
    bool renorm, float scale, int32_t* __restrict__ ids, float* __restrict__ weights) {
  const int l = threadIdx.x % LANES;
  // whole groups of LANES lanes take a row or leave together
  for (int64_t t = (int64_t)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES; t < rows;
       t += (int64_t)gridDim.x * (kThreads / LANES)) {
    const T* row = logits + t * E;
    float x[V];
    load_row<T, LANES, V>(row, E, l, x);
    float top = kNegInf, all = 0.f;
    if (!SIGMOID && !renorm) {
#pragma unroll
      for (int v = 0; v < V; ++v) top = fmaxf(top, x[v]);
      top = fmaxf(group_max<LANES>(top), -kMaxF32);
#pragma unroll
      for (int v = 0; v < V; ++v) all += expf(x[v] - top);
      all = group_sum<LANES>(all);
    }
    Key key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (sizeof(Key) == 8) {
        const int e = expert_of<LANES, V>(l, v);
        const double k = 1.0 / (1.0 + exp(-(double)x[v])) + (e < E ? (double)bias[e] : 0.0);
        key[v] = x[v] > kNegInf && k == k ? k : -__builtin_inf();
      } else {
        key[v] = x[v];
      }
    }
    int mine = -1;   // lane k keeps the expert of slot k
    for (int k = 0; k < K; ++k) {
      Key best = key[0];
      int at = expert_of<LANES, V>(l, 0);
#pragma unroll
      for (int v = 1; v < V; ++v)   // experts ascend with v: the first of equals stays
        if (key[v] > best) {
          best = key[v];
          at = expert_of<LANES, V>(l, v);
        }
#pragma unroll
      for (int m = 1; m < LANES; m <<= 1) {
        const Key ob = __shfl_xor(best, m, LANES);
        const int oa = __shfl_xor(at, m, LANES);
        if (ob > best || (ob == best && oa < at)) {
          best = ob;
          at = oa;
        }
      }
      const bool some = best > (Key)kNegInf;
      if (l == k) mine = some ? at : -1;
      if (!some) break;   // the whole group agrees; later slots keep -1
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (expert_of<LANES, V>(l, v) == at) key[v] = (Key)kNegInf;
    }
    const float v = mine >= 0 ? logit(row, mine) : kNegInf;
    float w;
    if (!SIGMOID) {
      const float m = renorm ? fmaxf(group_max<LANES>(v), -kMaxF32) : top;
      w = expf(v - m);
      w = ratio(w, renorm ? group_sum<LANES>(w) : all);
    } else {
      const float m = fmaxf(group_max<LANES>(v), -kMaxF32);
      w = mine < 0 ? 0.f : renorm && m < -30.f ? expf(v - m) : sigmoid_f32(v);
      if (renorm) w = ratio(w, group_sum<LANES>(w));
    }
    if (l < K) {
      ids[t * K + l] = mine;
      weights[t * K + l] = mine >= 0 ? scale * w : 0.f;
    }
  }
}

template <typename T, int LANES, int V, bool SIGMOID>
__global__ __launch_bounds__(kThreads) void gate_backward_kernel(
    const T* __restrict__ logits, const int32_t* __restrict__ ids, const float* __restrict__ dw,
    int64_t rows, int E, int K, bool renorm, float scale, T* __restrict__ dlogits) {
  const int l = threadIdx.x % LANES;
  // whole groups of LANES lanes take a row or leave together
  for (int64_t t = (int64_t)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES; t < rows;
       t += (int64_t)gridDim.x * (kThreads / LANES)) {
    const T* row = logits + t * E;
    int id = -1;
    float d = 0.f, v = kNegInf;
    if (l < K) {
      id = ids[t * K + l];
      if (id < 0 || id >= E) id = -1;
      if (id >= 0) {
        d = dw[t * K + l];
        v = logit(row, id);
      }
    }
    const bool dense = !SIGMOID && !renorm;
    float x[V];
    if (dense) {
      load_row<T, LANES, V>(row, E, l, x);
      float m = kNegInf;
#pragma unroll
      for (int i = 0; i < V; ++i) m = fmaxf(m, x[i]);
      m = fmaxf(group_max<LANES>(m), -kMaxF32);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        x[i] = expf(x[i] - m);
        sum += x[i];
      }
      sum = group_sum<LANES>(sum);
      const float p = ratio(expf(v - m), sum);
      const float dot = group_sum<LANES>(p * d);
      d = scale * p * d;
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = -scale * ratio(x[i], sum) * dot;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = 0.f;
      const float m = fmaxf(group_max<LANES>(v), -kMaxF32);
      if (!SIGMOID) {
        const float e = expf(v - m);
        const float p = ratio(e, group_sum<LANES>(e));
        d = scale * p * (d - group_sum<LANES>(p * d));
      } else {
        const float sg = v > kNegInf ? sigmoid_f32(v) : 0.f;
        const float co = v > kNegInf ? sigmoid_f32(-v) : 0.f;
        if (renorm) {
          const float e = m < -30.f ? expf(v - m) : sg;
          const float r = ratio(e, group_sum<LANES>(e));
          d = scale * r * (d - group_sum<LANES>(r * d)) * co;
        } else {
          d = scale * d * sg * co;
        }
      }
    }
    for (int k = 0; k < K; ++k) {
      const int e = __shfl(id, k, LANES);
      const float dk = __shfl(d, k, LANES);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (expert_of<LANES, V>(l, i) == e) x[i] += dk;
    }
    T* out = dlogits + t * E;
    if (V >= 4 && (E & 3) == 0) {
#pragma unroll
      for (int i = 0; i + 3 < V; i += 4) {
        const int e = expert_of<LANES, V>(l, i);
        if (e < E) {
          if constexpr (sizeof(T) == 4)
            *reinterpret_cast<vec4f*>(out + e) = vec4f{x[i], x[i + 1], x[i + 2], x[i + 3]};
          else
            *reinterpret_cast<uint2*>(out + e) =
                uint2{pack_bf16(x[i], x[i + 1]), pack_bf16(x[i + 2], x[i + 3])};
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = expert_of<LANES, V>(l, i);
        if (e < E) {
          if constexpr (sizeof(T) == 4) out[e] = x[i];
          else out[e] = f32_to_bf16(x[i]);
        }
      }
    }
  }
}

// Rows are walked with the grid's stride: a launch holds fewer than 2^32 threads.
uint32_t blocks_for(int64_t rows, int lanes) {
  const int per = kThreads / lanes;
  return (uint32_t)std::min<int64_t>((rows + per - 1) / per, int64_t(1) << 22);
}

// Calls f(lanes, values a lane) with the launch shape as compile-time values.
template <typename F>
void with_shape(int E, int K, F&& f) {
  using std::integral_constant;
  if (E <= 256 && K <= 16) {
    constexpr integral_constant<int, 16> L;
    if (E <= 16) f(L, integral_constant<int, 1>());
    else if (E <= 32) f(L, integral_constant<int, 2>());
    else if (E <= 64) f(L, integral_constant<int, 4>());
    else if (E <= 128) f(L, integral_constant<int, 8>());
    else f(L, integral_constant<int, 16>());
  } else {
    constexpr integral_constant<int, 64> L;
    if (E <= 256) f(L, integral_constant<int, 4>());
    else if (E <= 512) f(L, integral_constant<int, 8>());
    else f(L, integral_constant<int, 16>());
  }
}

template <typename T>
hipError_t gate(int score, bool renorm, float scale, const T* logits, const float* bias, int64_t rows,
                int E, int K, int32_t* ids, float* w, hipStream_t s) {
  with_shape(E, K, [&](auto L, auto V) {
    constexpr int lanes = decltype(L)::value, vals = decltype(V)::value;
    const dim3 grid(blocks_for(rows, lanes)), block(kThreads);
    if (score == LRMOE_GATE_SOFTMAX)
      hipLaunchKernelGGL((gate_kernel<T, float, lanes, vals, false>), grid, block, 0, s, logits,
                         bias, rows, E, K, renorm, scale, ids, w);
    else if (bias == nullptr)
      hipLaunchKernelGGL((gate_kernel<T, float, lanes, vals, true>), grid, block, 0, s, logits,
                         bias, rows, E, K, renorm, scale, ids, w);
    else
      hipLaunchKernelGGL((gate_kernel<T, double, lanes, vals, true>), grid, block, 0, s, logits,
                         bias, rows, E, K, renorm, scale, ids, w);
  });
  return hipGetLastError();
}

template <typename T>
hipError_t gate_backward(int score, bool renorm, float scale, const T* logits, const int32_t* ids,
                         const float* dw, int64_t rows, int E, int K, T* dx, hipStream_t s) {
  with_shape(E, K, [&](auto L, auto V) {
    constexpr int lanes = decltype(L)::value, vals = decltype(V)::value;
    const dim3 grid(blocks_for(rows, lanes)), block(kThreads);
    if (score == LRMOE_GATE_SOFTMAX)
      hipLaunchKernelGGL((gate_backward_kernel<T, lanes, vals, false>), grid, block, 0, s, logits,
                         ids, dw, rows, E, K, renorm, scale, dx);
    else
      hipLaunchKernelGGL((gate_backward_kernel<T, lanes, vals, true>), grid, block, 0, s, logits,
                         ids, dw, rows, E, K, renorm, scale, dx);
  });
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gate_topk(int dtype, int score, bool renorm, float scale, const void* logits,
                            const float* select_bias, int64_t T, int32_t E, int32_t K,
                            int32_t* ids, float* weights, hipStream_t s) {
  if (T == 0) return hipSuccess;
  return dtype == LRMOE_BF16
             ? gate(score, renorm, scale, static_cast<const uint16_t*>(logits), select_bias, T, E,
                    K, ids, weights, s)
             : gate(score, renorm, scale, static_cast<const float*>(logits), select_bias, T, E, K,
                    ids, weights, s);
}

hipError_t launch_gate_topk_backward(int dtype, int score, bool renorm, float scale,
                                     const void* logits, const int32_t* ids, const float* dweights,
                                     int64_t T, int32_t E, int32_t K, void* dlogits,
                                     hipStream_t s) {
  if (T == 0) return hipSuccess;
  return dtype == LRMOE_BF16
             ? gate_backward(score, renorm, scale, static_cast<const uint16_t*>(logits), ids,
                             dweights, T, E, K, static_cast<uint16_t*>(dlogits), s)
             : gate_backward(score, renorm, scale, static_cast<const float*>(logits), ids, dweights,
                             T, E, K, static_cast<float*>(dlogits), s);
}

}  // namespace lrmoe
