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
// and 16 slots take 16 lanes, so a wave works on four rows and an exchange is
// four DPP instructions; wider ones take the whole wave.  The K rounds are a
// running argmax over registers: no LDS, no sorting (keys and experts packed
// into float64 numbers and sorted per lane were 1.7 to 4 times slower).  The order
// of two near keys decides a whole number, so with a selection bias it is float64's; but
// float64 sigmoids of every logit cost more than all else, so float32 keys
// choose first, and where neighbours among the best are within the float32
// error (one row in a thousand) their float64 keys put them in order.
//
// Bound by the selection's instructions, not by the logits' 16.8 MB (4 us at
// the rate of a copy): 32768 rows of 128 float32, 8 slots: softmax 11.6 us,
// sigmoid with a bias 18 us (26 us with float64 keys throughout), the
// gradient from bf16 logits 8.3 us.  One to 16 rows take 4.6 us, most of it the
// launch.
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

// The value of the lane that step S of an exchange over LANES lanes pairs this
// one with.  After steps 0 .. S every lane of a run of 2^(S + 1) has the run's
// result: inside a row of 16 lanes by DPP (neighbours, pairs, the mirrored
// half row, the mirrored row), across rows through the LDS crossbar.
template <int S>
__device__ __forceinline__ int partner(int x) {
  if constexpr (S == 0) return __builtin_amdgcn_mov_dpp(x, 0xB1, 0xF, 0xF, true);        // 1 0 3 2
  else if constexpr (S == 1) return __builtin_amdgcn_mov_dpp(x, 0x4E, 0xF, 0xF, true);   // 2 3 0 1
  else if constexpr (S == 2) return __builtin_amdgcn_mov_dpp(x, 0x141, 0xF, 0xF, true);
  else if constexpr (S == 3) return __builtin_amdgcn_mov_dpp(x, 0x140, 0xF, 0xF, true);
  else return __shfl_xor(x, 1 << S, 64);
}
template <int S>
__device__ __forceinline__ float partner(float x) {
  return __int_as_float(partner<S>(__float_as_int(x)));
}
template <int S>
__device__ __forceinline__ double partner(double x) {
  const long long b = __double_as_longlong(x);
  const uint32_t lo = (uint32_t)partner<S>((int)(uint32_t)b);
  const uint32_t hi = (uint32_t)partner<S>((int)(uint32_t)(b >> 32));
  return __longlong_as_double((long long)(((unsigned long long)hi << 32) | lo));
}
template <int LANES, int S = 0>
__device__ __forceinline__ float group_sum(float x) {
  if constexpr ((1 << S) < LANES) return group_sum<LANES, S + 1>(x + partner<S>(x));
  else return x;
}
template <int LANES, int S = 0>
__device__ __forceinline__ float group_max(float x) {
  if constexpr ((1 << S) < LANES) return group_max<LANES, S + 1>(fmaxf(x, partner<S>(x)));
  else return x;
}
template <int LANES, int S = 0>
__device__ __forceinline__ uint32_t group_max(uint32_t x) {
  if constexpr ((1 << S) < LANES)
    return group_max<LANES, S + 1>(max(x, (uint32_t)partner<S>((int)x)));
  else return x;
}
template <int LANES, int S = 0>
__device__ __forceinline__ uint32_t group_min(uint32_t x) {
  if constexpr ((1 << S) < LANES)
    return group_min<LANES, S + 1>(min(x, (uint32_t)partner<S>((int)x)));
  else return x;
}
// The largest key of all lanes, of equal ones the lower expert's.
template <int LANES, int S = 0>
__device__ __forceinline__ void group_best(double& best, int& at) {
  if constexpr ((1 << S) < LANES) {
    const double ob = partner<S>(best);
    const int oa = partner<S>(at);
    if (ob > best || (ob == best && oa < at)) {
      best = ob;
      at = oa;
    }
    group_best<LANES, S + 1>(best, at);
  }
}

// sigmoid with expf and the exact division: the weights' own accuracy
__device__ __forceinline__ float sigmoid_exact(float x) { return 1.f / (1.f + expf(-x)); }

// A float32 key as a whole number of the same order; 0 is no key (-inf).
__device__ __forceinline__ uint32_t ordered(float key) {
  if (!(key > kNegInf)) return 0u;
  const uint32_t b = __float_as_uint(key + 0.f);   // -0 counts as 0
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float(o >> 31 ? o & 0x7FFFFFFFu : ~o);
}

// The experts of the K largest keys of the group's row, lane k holding slot
// k's (-1 where nothing is left).  Spends the keys.  A round finds the largest
// key of all lanes first and then the lowest expert that has it: two chains of
// one-instruction steps, half the work of carrying both through one.  CHECK:
// keys that are only nearly exact.  Rounds go on past K while a key is within
// 2^-19 (1 + the larger magnitude) of the one before it, or not ordered with
// it; `close` tells whether there were such neighbours at all, and `found` how
// many experts the lanes hold (LANES + 1: more are near than there are lanes).
template <int LANES, int V, bool CHECK>
__device__ __forceinline__ int select(uint32_t (&key)[V], int l, int K, bool& close, int& found) {
  int mine = -1;   // lane k keeps the expert of round k
  float before = 0.f;
  const int first = expert_of<LANES, V>(l, 0);
  close = false;
  int k = 0;
  for (; k < (CHECK ? LANES + 1 : K); ++k) {
    uint32_t best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = max(best, key[v]);
    best = group_max<LANES>(best);
    if (best == 0u) break;   // the whole group agrees; later slots keep -1
    if (CHECK) {
      const float now = unordered(best);
      const bool clear = before - now > 0x1p-19f * (1.f + fmaxf(fabsf(before), fabsf(now)));
      if (k >= K && clear) break;
      close |= k > 0 && !clear;
      before = now;
    }
    uint32_t at = 0x7FFFFFFFu;
#pragma unroll
    for (int v = V - 1; v >= 0; --v)   // experts ascend with v
      if (key[v] == best) at = expert_of<LANES, V>(0, v);
    at = group_min<LANES>(at + first);
    if (l == k) mine = (int)at;
    at -= first;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (at == (uint32_t)expert_of<LANES, V>(0, v)) key[v] = 0u;
  }
  found = k;
  return mine;
}

// The lanes' experts in the order of their float64 keys, equal ones by expert:
// lane r gets the one with r others before it.  Lanes without an expert (-1)
// are last.
template <int LANES>
__device__ __forceinline__ int reorder(double key, int mine, int l, int found) {
  int rank = 0;
  for (int j = 0; j < found; ++j) {
    const double kj = __shfl(key, j, LANES);
    const int ej = __shfl(mine, j, LANES);
    rank += kj > key || (kj == key && ej < mine);
  }
  if (mine < 0) rank = LANES;
  int out = -1;
  for (int j = 0; j < found; ++j) {
    const int rj = __shfl(rank, j, LANES), ej = __shfl(mine, j, LANES);
    if (rj == l) out = ej;
  }
  return out;
}

// The selection key in float64.
__device__ __forceinline__ double exact_key(float x, float bias) {
  return 1.0 / (1.0 + exp(-(double)x)) + (double)bias;
}

// select() from float64 keys.
template <int LANES, int V>
__device__ __forceinline__ int select_exact(double (&key)[V], int l, int K) {
  int mine = -1;
  for (int k = 0; k < K; ++k) {
    double best = key[0];
    int at = expert_of<LANES, V>(l, 0);
#pragma unroll
    for (int v = 1; v < V; ++v)   // experts ascend with v: the first of equals stays
      if (key[v] > best) {
        best = key[v];
        at = expert_of<LANES, V>(l, v);
      }
    group_best<LANES>(best, at);
    if (!(best > -__builtin_inf())) break;
    if (l == k) mine = at;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (expert_of<LANES, V>(l, v) == at) key[v] = -__builtin_inf();
  }
  return mine;
}

__device__ __forceinline__ float ratio(float num, float den) { return den > 0.f ? num / den : 0.f; }

template <typename T, int LANES, int V, bool SIGMOID, bool BIASED>
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
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = expert_of<LANES, V>(l, v);
      float k = x[v];
      if constexpr (BIASED) {
        k = sigmoid_f32(x[v]) + (e < E ? bias[e] : 0.f);
        if (!(x[v] > kNegInf && k == k)) k = kNegInf;
      }
      key[v] = ordered(k);
    }
    bool close;
    int found;
    int mine = select<LANES, V, BIASED>(key, l, K, close, found);
    if (BIASED && close) {
      // float32 keys are within 2^-21 (1 + |key|) of the float64 ones (sigmoid
      // to 2^-22, the sum's rounding 2^-24 |key|): neighbours further apart
      // than that are in float64's order.  This row has some that are not.
      if (found <= LANES) {   // all that matter are here, one a lane
        double k = -__builtin_inf();
        if (mine >= 0) k = exact_key(logit(row, mine), bias[mine]);
        mine = reorder<LANES>(k, mine, l, found);
      } else {
        double all_keys[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int e = expert_of<LANES, V>(l, v);
          const double k = exact_key(x[v], e < E ? bias[e] : 0.f);
          all_keys[v] = x[v] > kNegInf && k == k ? k : -__builtin_inf();
        }
        mine = select_exact<LANES, V>(all_keys, l, K);
      }
    }
    if (BIASED && l >= K) mine = -1;   // near ones past the last slot
    const float v = mine >= 0 ? logit(row, mine) : kNegInf;
    float w;
    if (!SIGMOID) {
      const float m = renorm ? fmaxf(group_max<LANES>(v), -kMaxF32) : top;
      w = expf(v - m);
      w = ratio(w, renorm ? group_sum<LANES>(w) : all);
    } else {
      const float m = fmaxf(group_max<LANES>(v), -kMaxF32);
      w = mine < 0 ? 0.f : renorm && m < -30.f ? expf(v - m) : sigmoid_exact(v);
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
        const float sg = v > kNegInf ? sigmoid_exact(v) : 0.f;
        const float co = v > kNegInf ? sigmoid_exact(-v) : 0.f;
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
hipError_t gate(int score, bool renorm, float scale, const T* logits, const float* bias,
                int64_t rows, int E, int K, int32_t* ids, float* w, hipStream_t s) {
  with_shape(E, K, [&](auto L, auto V) {
    constexpr int lanes = decltype(L)::value, vals = decltype(V)::value;
    const dim3 grid(blocks_for(rows, lanes)), block(kThreads);
    if (score == LRMOE_GATE_SOFTMAX)
      hipLaunchKernelGGL((gate_kernel<T, lanes, vals, false, false>), grid, block, 0, s, logits,
                         bias, rows, E, K, renorm, scale, ids, w);
    else if (bias == nullptr)
      hipLaunchKernelGGL((gate_kernel<T, lanes, vals, true, false>), grid, block, 0, s, logits,
                         bias, rows, E, K, renorm, scale, ids, w);
    else
      hipLaunchKernelGGL((gate_kernel<T, lanes, vals, true, true>), grid, block, 0, s, logits,
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
