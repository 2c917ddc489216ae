// Shared declarations of the forward-side translation units (router gate,
// expert sort, dispatch and combine, grouped product with epilogue).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lrmoe.h"

namespace lrmoe {

constexpr int kMaxSegs = LRMOE_MAX_EXPERTS;

typedef unsigned int vec4u __attribute__((ext_vector_type(4)));
typedef float vec4f __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_to_f32(uint16_t h) {
  return __uint_as_float((uint32_t)h << 16);
}
// Round to nearest, ties to even (the hardware conversion; NaN stays NaN).
__device__ __forceinline__ uint16_t f32_to_bf16(float f) {
  return __builtin_bit_cast(uint16_t, (__bf16)f);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return (uint32_t)f32_to_bf16(lo) | ((uint32_t)f32_to_bf16(hi) << 16);
}

// Storage types by their element: load and store of N consecutive values
// (N * size a multiple of 16 bytes, 16-byte aligned).
template <typename T, int N>
__device__ __forceinline__ void load_vals(const T* p, float (&v)[N]) {
  if constexpr (sizeof(T) == 2) {
    static_assert(N % 8 == 0, "16-byte pieces");
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      const vec4u w = reinterpret_cast<const vec4u*>(p)[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
        v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
  } else {
    static_assert(N % 4 == 0, "16-byte pieces");
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const vec4f w = reinterpret_cast<const vec4f*>(p)[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * i + j] = w[j];
    }
  }
}
template <typename T, int N>
__device__ __forceinline__ void store_vals(T* p, const float (&v)[N]) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      vec4u w;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = pack_bf16(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
      reinterpret_cast<vec4u*>(p)[i] = w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      reinterpret_cast<vec4f*>(p)[i] = vec4f{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
  }
}

// Sum over lanes 0 .. this one, by DPP: inside rows of 16 lanes, then the last
// lane of a row into the next one, of two rows into the next two.
__device__ __forceinline__ int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);   // row_shr:1
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);   // row_bcast:15
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);   // row_bcast:31
  return x;
}

// ---- activations, float32
// Sigmoid from the hardware exp2 and reciprocal (about one ulp each; the
// rounded argument adds |x| 2^-24 relative to exp(-x), which is at most 2^-25
// of the result's scale).  exp(-x) = 2^(-x log2(e)); its overflow gives 0, as it
// should.  expf and the exact division take several times the instructions, and
// the elementwise kernels are near the point where those count.
__device__ __forceinline__ float sigmoid_f32(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * x));
}
__device__ __forceinline__ float gelu_f32(float x) {
  return 0.5f * x * (1.f + erff(x * 0.70710678f));
}

// ---- launchers (hipSuccess or the launch error)
hipError_t launch_gate_topk(int dtype, int score, bool renorm, float scale, const void* logits,
                            const float* select_bias, int64_t T, int32_t E, int32_t K,
                            int32_t* ids, float* weights, hipStream_t s);
hipError_t launch_gate_topk_backward(int dtype, int score, bool renorm, float scale,
                                     const void* logits, const int32_t* ids, const float* dweights,
                                     int64_t T, int32_t E, int32_t K, void* dlogits, hipStream_t s);

size_t route_sort_workspace(int64_t n, int32_t E);
hipError_t launch_route_sort(const int32_t* ids, const float* weights, int64_t T, int32_t K,
                             int32_t E, int64_t* counts, int32_t* seg_offsets, int32_t* row_index,
                             int32_t* pos, float* alpha, uint32_t* ws, hipStream_t s);
hipError_t launch_dispatch(int dtype, const void* x, const int32_t* pos, int64_t T, int32_t K,
                           int32_t D, int64_t P, void* xp, hipStream_t s);
// y[t] = residual[t] + sum_k weights[t, k] * rows[pos[t, k]]; weights null: 1
hipError_t launch_combine(int in_dtype, int out_dtype, const void* rows, const int32_t* pos,
                          const float* weights, const void* residual, int64_t T, int32_t K,
                          int32_t D, int64_t P, void* y, hipStream_t s);
hipError_t launch_combine_backward(int dtype, const void* dy, const void* rows, const int32_t* pos,
                                   const float* weights, int64_t T, int32_t K, int32_t D,
                                   int64_t P, void* drows, float* dweights, hipStream_t s);

struct ForwardArgs {
  const int32_t* seg;         // device [E + 1]
  const int32_t* row_index;   // device [P] or null
  const void* x;              // [T, d_in]
  const void* W;              // [E, d_out, d_in]
  const void* bias;           // [E, d_out] or null
  const void* residual;       // [P, F] or null
  void* y;                    // [P, F]
  void* pre_a;                // [P, F] or null
  void* pre_b;                // [P, F] or null (SwiGLU)
  int64_t P, T;
  int32_t E, d_out, d_in, act;
};
hipError_t launch_grouped_forward(int dtype, const ForwardArgs& a, hipStream_t s);

size_t act_backward_workspace(int64_t P, int32_t E, int32_t width);  // with bias sums
hipError_t launch_act_backward(int dtype, int out_dtype, int act, const int32_t* seg,
                               const void* dy, const void* a, const void* b, int64_t P, int32_t E,
                               int32_t F, void* dz, float* dbias, float* ws, hipStream_t s);

}  // namespace lrmoe
