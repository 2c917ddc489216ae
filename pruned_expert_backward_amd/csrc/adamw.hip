// AdamW over many tensors in one launch:
//
//   g' = s g,  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   p  = (1 - lr d) p - (lr / c1) m / (sqrt(v) / sqrt(c2) + eps),   ci = 1 - bi^step
//
// States in float32, or 8-bit blocks of 128 (fp8.h) that hold m and sqrt(v).  A
// launch takes up to 48 tensors of the same types through its arguments (no table
// in device memory, so a captured call needs none to outlive it); a workgroup takes a
// chunk of one tensor, a lane 8 consecutive elements, and so a row of 16 lanes
// one block of the states.
//
// Memory bound: 28 bytes an element in float32, 16 with 8-bit states, 2 more for a
// bfloat16 copy.  75.5 million float32 parameters, 8-bit states and copies (1.36 GB):
// 266 us, 5.1 TB/s; float32 states 398 us (5.3), with copies 428; bfloat16 parameters with
// float32 states 341 us (5.3), with float32 and with bfloat16 gradients and 8-bit states 215
// and 221 us (4.2 and 3.4 TB/s: arithmetic, three roundings and two hashes an element).
//
// sqrt(v) is what the step uses, and its range is half of v's: e4m3 with a scale
// a block then covers gradients from 1 to 2^-17 of the block's largest.  Rounding to
// nearest would freeze the states (a step changes v by 1 - b2 of its distance,
// far less than half of e4m3's step), so they are rounded stochastically.  The root then
// keeps its mean and its square gains the variance: a root of q steps of its code moves by
// about q (1 - b2) / 2 of a step, and so gains that many squared steps, which b2 lets add up
// to 1 / (2 q) of v: 4 % for q = 8 .. 16.
#include <cmath>

#include "forward.h"
#include "fp8.h"

// The states' codes follow from float32 values next to a border: the products and
// sums below stay as they are written, so that the definition decides.
#pragma clang fp contract(off)

namespace lrmoe {
namespace {

constexpr int kMost = 48;          // tensors of a launch: 3.6 KB of the 4 KB of arguments
constexpr int kLane = 8;           // elements of a lane
constexpr int kPass = 256 * kLane;

struct Tensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  uint8_t* ms;
  uint8_t* vs;
  uint16_t* copy;
  int64_t n;
};

struct Step {
  double lr, beta1, beta2;         // for scalars on the device
  const float* lr_at;
  const int64_t* step_at;
  const float* grad_scale;
  const float* skip;
  float b1, c1, b2, c2;            // beta, 1 - beta
  float keep, rate, root, eps;     // 1 - lr d, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  double decay;
  uint32_t seed, step;
  int32_t count, chunk;            // elements of a workgroup
};

struct Launch {
  Tensor t[kMost];
  uint32_t first[kMost];           // its first workgroup
  uint32_t ordinal[kMost];         // place in the caller's list
  Step s;
};
static_assert(sizeof(Launch) <= 4096, "kernel arguments");

// b^t by squaring: the same on the host and on the device.
__host__ __device__ inline double power(double b, int64_t t) {
  double r = 1.0;
  for (; t > 0; t >>= 1, b *= b)
    if (t & 1) r *= b;
  return r;
}
__host__ __device__ inline void corrections(double lr, double beta1, double beta2, double decay,
                                            int64_t t, float& keep, float& rate, float& root) {
  keep = (float)(1.0 - lr * decay);
  rate = (float)(lr / (1.0 - power(beta1, t)));
  root = (float)(1.0 / sqrt(1.0 - power(beta2, t)));
}

__host__ __device__ inline uint32_t mix(uint32_t a) {
  a ^= a >> 16;
  a *= 0x6A09E667u;
  a ^= a >> 15;
  a *= 0xBB67AE85u;
  return a ^ (a >> 16);
}

// Elements i .. i + 7 of a buffer of n (i a multiple of 8), 0 behind its end.
template <typename T>
__device__ __forceinline__ void load8(const void* p, int64_t i, int64_t n, float (&v)[kLane]) {
  const T* t = static_cast<const T*>(p) + i;
  if (i + kLane <= n) {
    if constexpr (sizeof(T) == 1) {
      const uint2 w = *reinterpret_cast<const uint2*>(t);
      float a[4], b[4];
      fp8_unpack4(w.x, a);
      fp8_unpack4(w.y, b);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = a[j];
        v[4 + j] = b[j];
      }
    } else {
      load_vals(t, v);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < kLane; ++j) {
    v[j] = 0.f;
    if (i + j < n) {
      if constexpr (sizeof(T) == 1) v[j] = __builtin_amdgcn_cvt_f32_fp8((int)t[j], 0);
      else if constexpr (sizeof(T) == 2) v[j] = bf16_to_f32(t[j]);
      else v[j] = t[j];
    }
  }
}

// Codes of elements i .. i + 7, as many as there are.
template <typename T, int N>
__device__ __forceinline__ void store_words(T* p, int64_t i, int64_t n, const uint32_t (&w)[N]) {
  constexpr int size = N * 4 / kLane;   // bytes of an element
  static_assert(size == sizeof(T), "whole elements");
  if (i + kLane <= n) {
#pragma unroll
    for (int j = 0; j < N / 2; ++j)
      reinterpret_cast<uint2*>(p + i)[j] = make_uint2(w[2 * j], w[2 * j + 1]);
    return;
  }
#pragma unroll
  for (int j = 0; j < kLane; ++j)
    if (i + j < n) p[i + j] = (T)(w[j * size / 4] >> (j * size % 4 * 8));
}

// Stochastic rounding of |x| / scale to a multiple of e4m3's step there (a power of
// two, at least 2^-9): the quotient is exact, and floor(quotient + r / 2^16) rounds
// up as often as the value lies beyond the lower neighbour.  At most 14 steps
// of 32 in the top binade, so nothing passes 448.
__device__ __forceinline__ float round_e4m3(float x, uint32_t r) {
  uint32_t lead = __float_as_uint(x) & 0x7F800000u;
  lead = lead < (121u << 23) ? 121u << 23 : lead;
  const float up = __uint_as_float((257u << 23) - lead), down = __uint_as_float(lead - (3u << 23));
  return floorf(fabsf(x) * up + (float)r * 0x1p-16f) * down;
}

// One row of 16 lanes' block: codes and scale byte.  ROOT: no sign, and what is
// not zero stays so.
template <bool ROOT>
__device__ __forceinline__ uint32_t encode(const float (&x)[kLane], const uint32_t (&r)[kLane],
                                           uint32_t (&w)[2]) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < kLane; ++j) top = umax(top, finite_bits(x[j]));
  const uint32_t byte = fp8_scale_byte(row16_max(top));
  const float inv = fp8_inverse(byte);
  float q[kLane];
#pragma unroll
  for (int j = 0; j < kLane; ++j) {
    const float z = fp8_scaled(x[j], inv);
    float c = round_e4m3(z, ROOT ? r[j] & 0xFFFFu : r[j] >> 16);
    if (ROOT) c = x[j] > 0.f && c == 0.f ? 0x1p-9f : c;
    q[j] = z != z ? z : ROOT ? c : copysignf(c, z);
  }
  w[0] = fp8_pack4(q[0], q[1], q[2], q[3]);
  w[1] = fp8_pack4(q[4], q[5], q[6], q[7]);
  return byte;
}

// P, G, S: storage of p, g and the states (1 byte: 8-bit blocks).
template <typename P, typename G, typename S>
__global__ __launch_bounds__(256) void adamw_kernel(Launch a) {
  const Step& s = a.s;
  if (s.skip != nullptr && *s.skip != 0.f) return;
  int k = 0;   // the last tensor that starts at or before this workgroup
  for (int half = 32; half > 0; half >>= 1)
    if (k + half < s.count && a.first[k + half] <= blockIdx.x) k += half;
  const Tensor t = a.t[k];
  float keep = s.keep, rate = s.rate, root = s.root;
  uint32_t step = s.step;
  if (s.step_at != nullptr || s.lr_at != nullptr) {
    const int64_t at = s.step_at != nullptr ? *s.step_at : (int64_t)s.step;
    step = (uint32_t)at;
    corrections(s.lr_at != nullptr ? (double)*s.lr_at : s.lr, s.beta1, s.beta2, s.decay, at, keep,
                rate, root);
  }
  const float gs = s.grad_scale != nullptr ? *s.grad_scale : 1.f;
  const uint32_t key = mix(mix(s.seed + step * 0x9E3779B9u) + (a.ordinal[k] + 1) * 0x3C6EF373u);
  constexpr bool wide = sizeof(S) == 4;
  const int64_t begin = (int64_t)(blockIdx.x - a.first[k]) * s.chunk;
  const int64_t end = begin + s.chunk < t.n ? begin + s.chunk : t.n;
  // whole rows of 16 lanes: the lanes behind a block's end take part in its maximum
  for (int64_t row = begin + (threadIdx.x & ~15) * kLane; row < end; row += kPass) {
    const int64_t i = row + (threadIdx.x & 15) * kLane;
    float p[kLane], g[kLane], m[kLane], v[kLane];
    load8<P>(t.p, i, t.n, p);
    load8<G>(t.g, i, t.n, g);
    load8<S>(t.m, i, t.n, m);
    load8<S>(t.v, i, t.n, v);
    if constexpr (!wide) {
      const float mz = fp8_scale(t.ms[i / kFp8Block]), vz = fp8_scale(t.vs[i / kFp8Block]);
#pragma unroll
      for (int j = 0; j < kLane; ++j) {
        m[j] *= mz;
        const float r = v[j] * vz;
        v[j] = r * r;
      }
    }
    float q[kLane];   // sqrt(v)
#pragma unroll
    for (int j = 0; j < kLane; ++j) {
      const float gj = g[j] * gs;
      m[j] = m[j] * s.b1 + gj * s.c1;
      v[j] = v[j] * s.b2 + (gj * gj) * s.c2;
      q[j] = sqrtf(v[j]);
      p[j] = p[j] * keep - (m[j] * __builtin_amdgcn_rcpf(q[j] * root + s.eps)) * rate;
    }
    uint32_t r[kLane];
    if constexpr (!wide || sizeof(P) == 2) {
#pragma unroll
      for (int j = 0; j < kLane; ++j) r[j] = mix((uint32_t)i + j + key);
    }
    if constexpr (sizeof(P) == 4) {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < kLane; ++j) w[j] = __float_as_uint(p[j]);
      store_words(static_cast<uint32_t*>(t.p), i, t.n, w);
      if (t.copy != nullptr) {
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = pack_bf16(p[2 * j], p[2 * j + 1]);
        store_words(t.copy, i, t.n, c);
      }
    } else {
      uint32_t c[4], h[kLane];
#pragma unroll
      for (int j = 0; j < kLane; ++j) {
        const uint32_t b = __float_as_uint(p[j]);
        h[j] = (b & 0x7F800000u) == 0x7F800000u
                   ? (uint32_t)f32_to_bf16(p[j])
                   : (b + (mix(r[j] + 0xA54FF53Bu) >> 16)) >> 16;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] = h[2 * j] | h[2 * j + 1] << 16;
      store_words(static_cast<uint16_t*>(t.p), i, t.n, c);
    }
    if constexpr (wide) {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < kLane; ++j) w[j] = __float_as_uint(m[j]);
      store_words(static_cast<uint32_t*>(t.m), i, t.n, w);
#pragma unroll
      for (int j = 0; j < kLane; ++j) w[j] = __float_as_uint(v[j]);
      store_words(static_cast<uint32_t*>(t.v), i, t.n, w);
    } else {
      // elements behind the end are zeros: they leave the block's scale alone
#pragma unroll
      for (int j = 0; j < kLane; ++j)
        if (i + j >= t.n) m[j] = q[j] = 0.f;
      uint32_t w[2];
      const uint32_t mb = encode<false>(m, r, w);
      store_words(static_cast<uint8_t*>(t.m), i, t.n, w);
      const uint32_t vb = encode<true>(q, r, w);
      store_words(static_cast<uint8_t*>(t.v), i, t.n, w);
      if ((threadIdx.x & 15) == 0) {
        t.ms[i / kFp8Block] = (uint8_t)mb;
        t.vs[i / kFp8Block] = (uint8_t)vb;
      }
    }
  }
}

template <typename P, typename G, typename S>
hipError_t launch(const Launch& a, uint32_t blocks, hipStream_t s) {
  hipLaunchKernelGGL((adamw_kernel<P, G, S>), dim3(blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

typedef hipError_t (*Launcher)(const Launch&, uint32_t, hipStream_t);
// [p bf16][g bf16][8-bit states]
const Launcher kLaunch[2][2][2] = {
    {{launch<float, float, float>, launch<float, float, uint8_t>},
     {launch<float, uint16_t, float>, launch<float, uint16_t, uint8_t>}},
    {{launch<uint16_t, float, float>, launch<uint16_t, float, uint8_t>},
     {launch<uint16_t, uint16_t, float>, launch<uint16_t, uint16_t, uint8_t>}}};

}  // namespace

hipError_t launch_adamw(const lrmoe_adamw* c, const lrmoe_adamw_tensor* t, int32_t count,
                        hipStream_t s) {
  Launch a;
  Step& st = a.s;
  st.lr = c->lr;
  st.beta1 = c->beta1;
  st.beta2 = c->beta2;
  st.decay = c->weight_decay;
  st.lr_at = c->lr_at;
  st.step_at = c->step_at;
  st.grad_scale = c->grad_scale;
  st.skip = c->skip;
  st.b1 = (float)c->beta1;
  st.c1 = (float)(1.0 - c->beta1);
  st.b2 = (float)c->beta2;
  st.c2 = (float)(1.0 - c->beta2);
  st.eps = (float)c->eps;
  st.seed = c->seed;
  st.step = (uint32_t)c->step;
  corrections(c->lr, c->beta1, c->beta2, c->weight_decay, c->step, st.keep, st.rate, st.root);
  int64_t total = 0;
  for (int32_t k = 0; k < count; ++k) total += t[k].n;
  // a chunk of four passes, of one where that would leave CUs idle
  st.chunk = total >= int64_t(256) * 4 * 4 * kPass ? 4 * kPass : kPass;
  for (int kind = 0; kind < 8; ++kind) {
    const int p = kind >> 2, g = kind >> 1 & 1, b = kind & 1;
    st.count = 0;
    int64_t blocks = 0;
    for (int32_t k = 0; k <= count; ++k) {
      const bool full = st.count == kMost;
      // at most 2^23: a tensor has less than 2^36 elements
      const int64_t need = k < count ? (t[k].n + st.chunk - 1) / st.chunk : 0;
      if (st.count > 0 && (k == count || full || blocks + need >= int64_t(1) << 24)) {
        const hipError_t e = kLaunch[p][g][b](a, (uint32_t)blocks, s);
        if (e != hipSuccess) return e;
        st.count = 0;
        blocks = 0;
      }
      if (k == count) break;
      if ((t[k].p_dtype == LRMOE_BF16) != (p != 0) || (t[k].g_dtype == LRMOE_BF16) != (g != 0) ||
          (t[k].m_scale != nullptr) != (b != 0) || t[k].n == 0)
        continue;
      a.t[st.count] = Tensor{t[k].p, t[k].g, t[k].m, t[k].v, t[k].m_scale, t[k].v_scale,
                             static_cast<uint16_t*>(t[k].copy), t[k].n};
      a.first[st.count] = (uint32_t)blocks;
      a.ordinal[st.count] = (uint32_t)k;
      ++st.count;
      blocks += need;
    }
  }
  return hipSuccess;
}

}  // namespace lrmoe
