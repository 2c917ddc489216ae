// Grouped expert product with its epilogue, over expert-sorted pairs:
//
//   z_u = W_e x_{row(u)} + bias_e,   y_u = act(z_u) + residual_u
//   SwiGLU: W_e stacks gate over up rows, z = [a | b], y = SiLU(a) * b + residual
//
// The segments are read from device memory, so nothing of the routing has to
// visit the host; the launch covers the most tiles that P rows over E experts
// can have, and workgroups without a tile leave at once.
//
// Both operands are rows along K (x rows, W rows), so they move to LDS as they
// are and fragments are 16-byte LDS reads; the same kernel serves bfloat16
// (v_mfma_f32_32x32x16_bf16, 8 values a fragment) and float32
// (v_mfma_f32_32x32x2_f32, 4 values a fragment, four products), float32
// accumulation in both.  Masked rows and the end of K read a page of zeros.
#include "forward.h"

namespace lrmoe {
namespace {

#define LDS_AS __attribute__((address_space(3)))

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ const vec4u zero_page[16] = {};

__device__ __forceinline__ float activate(int act, float x) {
  switch (act) {
    case LRMOE_ACT_RELU: return fmaxf(x, 0.f);
    case LRMOE_ACT_SILU: return x * sigmoid_f32(x);
    case LRMOE_ACT_GELU: return gelu_f32(x);
  }
  return x;
}

// ---------------------------------------------------------------- tiles
struct TileAt {
  int e;
  int64_t lo;    // first pair row of the tile
  int rows;      // rows of the tile (at least 1)
  int col;       // column tile
};

// Tile of this workgroup, or false.  Workgroup b runs on XCD b % 8, so each
// XCD takes a contiguous eighth of the tiles; inside it, group rows tiles
// share their W panels, column by column.  Each wave finds the tile for
// itself: lane l counts the tiles of experts 4 l .. 4 l + 3.
__device__ __forceinline__ bool find_tile(const int32_t* seg, int E, int64_t P, int tm, int cols,
                                          int group, TileAt& at) {
  const int lane = threadIdx.x & 63;
  int64_t off[5];
#pragma unroll
  for (int j = 0; j < 5; ++j) {
    const int e = 4 * lane + j;
    const int64_t o = seg[e < E ? e : E];
    off[j] = o < 0 ? 0 : o > P ? P : o;
  }
  int n[4], sum = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    n[j] = off[j + 1] > off[j] ? (int)((off[j + 1] - off[j] + tm - 1) / tm) : 0;
    sum += n[j];
  }
  int end = sum;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const int o = __shfl_up(end, m, 64);
    if (lane >= m) end += o;
  }
  const int all = __builtin_amdgcn_readlane(end, 63);
  const int64_t total = (int64_t)all * cols;
  const int64_t share = (total + 7) / 8;
  const int64_t t = (int64_t)(blockIdx.x & 7) * share + (blockIdx.x >> 3);
  if ((int64_t)(blockIdx.x >> 3) >= share || t >= total) return false;
  const int64_t per = (int64_t)group * cols;
  const int g = (int)(t / per);
  const int in = (int)(t - g * per);
  const int left = all - g * group;
  const int gr = left < group ? left : group;
  const int r = __builtin_amdgcn_readfirstlane(g * group + in % gr);
  at.col = __builtin_amdgcn_readfirstlane(in / gr);
  const int owner = __ffsll((unsigned long long)__ballot(end > r)) - 1;
  int sub = r - (end - sum), j = 0;   // meant for the owner lane
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (j == i && sub >= n[i]) {
      sub -= n[i];
      j = i + 1;
    }
  const int64_t lo = (j == 0 ? off[0] : j == 1 ? off[1] : j == 2 ? off[2] : off[3]) +
                     (int64_t)sub * tm;
  const int64_t hi = j == 0 ? off[1] : j == 1 ? off[2] : j == 2 ? off[3] : off[4];
  const int rows = (int)(hi - lo < tm ? hi - lo : tm);
  at.e = __builtin_amdgcn_readlane(4 * lane + j, owner);
  const uint32_t lo32 = __builtin_amdgcn_readlane((uint32_t)lo, owner);   // P < 2^31
  at.lo = lo32;
  at.rows = __builtin_amdgcn_readlane(rows, owner);
  return true;
}

// Row of x of pair row u: null when its index is out of range (a zero row).
template <typename T>
__device__ __forceinline__ const char* x_row(const ForwardArgs& a, int64_t u) {
  const int64_t r = a.row_index != nullptr ? (int64_t)a.row_index[u] : u;
  if (r < 0 || r >= a.T) return nullptr;
  return reinterpret_cast<const char*>(static_cast<const T*>(a.x) + r * a.d_in);
}

// 16-byte value of one lane times one lane's: four float32 products or one bf16.
template <typename T>
__device__ __forceinline__ f32x16 mfma32(vec4u a, vec4u b, f32x16 c) {
  if constexpr (sizeof(T) == 2) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[i]), __uint_as_float(b[i]), c, 0,
                                               0, 0);
    return c;
  }
}
template <typename T>
__device__ __forceinline__ f32x4 mfma16(vec4u a, vec4u b, f32x4 c) {
  if constexpr (sizeof(T) == 2) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]), c, 0,
                                               0, 0);
    return c;
  }
}

// ---- global -> LDS, 16 bytes a lane: lane i writes LDS bytes [lds + 16 i,
// lds + 16 i + 16).  Inline asm without outputs: the compiler then does not
// wait for it before LDS reads of other stages; the explicit waits below
// order the stages.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds16(uint32_t lds, const char* p) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds),
               "v"(p)
               : "memory", "m0");
}
#pragma clang diagnostic pop

template <int N>
__device__ __forceinline__ void wait_loads_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// T: storage.  MB x NB 32x32 blocks a wave, WM x WN waves.  RB: bytes of one
// row in one K step (64 or 128).  NS: LDS stages.
template <typename T, int MB, int NB, int WM, int WN, int RB, int NS, bool GLU>
struct Gemm {
  static constexpr int kMB = MB, kNB = NB;
  static constexpr int kWaves = WM * WN;
  static constexpr int kWavesPerSimd = MB * NB > 8 ? 1 : 2;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int TM = WM * MB * 32, TN = WN * NB * 32;
  static constexpr int kOut = GLU ? TN / 2 : TN;           // columns of y
  static constexpr int kSlices = RB / 32;                  // MFMA steps of a K step
  static constexpr int kChunks = RB / 16;
  static constexpr int kStage = (TM + TN) * RB;
  static constexpr int kPwA = TM * RB / 1024 / kWaves, kPwB = TN * RB / 1024 / kWaves;
  static constexpr int kLoads = kPwA + kPwB;               // load instructions a stage and wave
  static constexpr int kEpi = kWaves * NB * 4096;          // epilogue staging
  static constexpr int kMain = NS * kStage > kEpi ? NS * kStage : kEpi;
  static constexpr int kLds = kMain + kWaves * 1024;       // + a sink for loads past the end
  static_assert(TM * RB % (1024 * kWaves) == 0 && TN * RB % (1024 * kWaves) == 0, "whole loads");
  static_assert(!GLU || NB % 2 == 0, "gate and up blocks of a wave");
  static_assert(kSlices % 2 == 0, "fragment sets alternate");

  // Chunk c of row r sits at slot c ^ swz(r): 16 consecutive rows of one chunk
  // (one LDS cycle of a 16-byte read) fall on 16 distinct bank groups.
  __device__ __forceinline__ static int swz(int r) {
    return RB == 64 ? (r ^ (r >> 2)) & 3 : (r >> 1) & 7;
  }

  struct Frags {
    vec4u a[MB], b[NB];
  };

  const ForwardArgs& args;
  uint32_t lds;            // LDS byte address of stage 0
  int lane, wave, wm, wn;
  int kbytes, nk;
  const char* src[kLoads]; // this lane's next 16 bytes of each load
  int step[kLoads];        // bytes to the next K step (0 for masked rows)
  int chunk[kLoads];       // byte offset of the lane's chunk inside the step
  uint32_t fa, fb;         // fragment base addresses (A rows, B rows of the wave)
  uint32_t fs[kSlices];    // lane's offset of each slice

  __device__ __forceinline__ Gemm(const ForwardArgs& a, const TileAt& at, LDS_AS char* smem)
      : args(a) {
    lds = (uint32_t)(uintptr_t)smem;
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = wave / WN;
    wn = wave % WN;
    kbytes = a.d_in * (int)sizeof(T);
    nk = (kbytes + RB - 1) / RB;
    const char* zero = reinterpret_cast<const char*>(zero_page);
    const int F = GLU ? a.d_out / 2 : a.d_out;
    constexpr int rows_per = 1024 / RB;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const bool isA = j < kPwA;
      const int blk = isA ? wave * kPwA + j : wave * kPwB + j - kPwA;
      const int r = blk * rows_per + lane / kChunks;
      chunk[j] = ((lane % kChunks) ^ swz(r)) * 16;
      const char* p = nullptr;
      if (isA) {
        if (r < at.rows) p = x_row<T>(a, at.lo + r);
      } else {
        // LDS row r holds, for SwiGLU, of wave column w = r / (NB * 32) first
        // the gate rows and then the up rows of the wave's output columns
        int64_t n;
        bool ok;
        if constexpr (GLU) {
          constexpr int half = NB * 16;
          const int w = r / (NB * 32), i = r % (NB * 32);
          const int c = at.col * kOut + w * half + i % half;
          ok = c < F;
          n = (int64_t)(i / half) * F + c;
        } else {
          n = at.col * TN + r;
          ok = n < F;
        }
        if (ok)
          p = reinterpret_cast<const char*>(static_cast<const T*>(a.W) +
                                            ((int64_t)at.e * a.d_out + n) * a.d_in);
      }
      step[j] = p != nullptr ? RB : 0;
      src[j] = p != nullptr ? p + chunk[j] : zero;
    }
    const int fr = lane & 31;
#pragma unroll
    for (int s = 0; s < kSlices; ++s) fs[s] = fr * RB + (((2 * s + (lane >> 5)) ^ swz(fr)) << 4);
    fa = lds + wm * MB * 32 * RB;
    fb = lds + TM * RB + wn * NB * 32 * RB;
  }

  // Load j of the K step that starts `left` bytes before the end of K, into
  // stage buffer `buf`.  Past the end (left <= 0) it keeps its place in the
  // instruction stream and writes zeros into the wave's sink.
  __device__ __forceinline__ void issue(int j, int buf, int left) {
    const bool isA = j < kPwA;
    const uint32_t dst = isA ? (wave * kPwA + j) * 1024 : TM * RB + (wave * kPwB + j - kPwA) * 1024;
    const uint32_t to = left > 0 ? lds + buf * kStage + dst : lds + kMain + wave * 1024;
    const char* p = chunk[j] < left ? src[j] : reinterpret_cast<const char*>(zero_page);
    load_lds16(__builtin_amdgcn_readfirstlane(to), p);
    src[j] += step[j];
  }

  __device__ __forceinline__ vec4u read16(uint32_t addr) const {
    return *reinterpret_cast<LDS_AS const vec4u*>((LDS_AS char*)(uintptr_t)addr);
  }
  __device__ __forceinline__ void read_frag(Frags& f, int buf, int s, int i) const {
    const uint32_t so = buf * kStage + fs[s];
    if (i < MB) f.a[i] = read16(fa + so + i * 32 * RB);
    else f.b[i - MB] = read16(fb + so + (i - MB) * 32 * RB);
  }

  // The K loop.  In step kt (buffer S = kt % NS) the fragments of slice s + 1
  // are read while slice s is multiplied.  Before the last slice one barrier:
  // the next stage is in LDS (its loads are the oldest ones), and nobody
  // reads buffer S any more; the loads of step kt + NS then go out between
  // the products of the last slice and of the next step's first slices.
  __device__ __forceinline__ void mainloop(f32x16 (&acc)[MB][NB]) {
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.f;
#pragma unroll
    for (int d = 0; d < NS; ++d)
#pragma unroll
      for (int j = 0; j < kLoads; ++j) issue(j, d, kbytes - d * RB);
    wait_loads_barrier<(NS - 1) * kLoads>();
    Frags f[2];
#pragma unroll
    for (int i = 0; i < MB + NB; ++i) read_frag(f[0], 0, 0, i);
    constexpr int kHalf = (kLoads + 1) / 2;   // loads after the barrier; the rest a slice later
    for (int kt = 0, S = 0; kt < nk; ++kt) {
      const int SN = S + 1 == NS ? 0 : S + 1, SP = S == 0 ? NS - 1 : S - 1;
#pragma unroll
      for (int s = 0; s < kSlices; ++s) {
        const bool last = s == kSlices - 1;
        if (last) {
          wait_loads_barrier<(NS - 2) * kLoads>();
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < MB * NB; ++i) {
          const int a = i / NB, b = i % NB;
          acc[a][b] = mfma32<T>(f[s & 1].b[b], f[s & 1].a[a], acc[a][b]);
          // spread over the products: the next slice's fragments, one load
          for (int q = i * (MB + NB) / (MB * NB); q < (i + 1) * (MB + NB) / (MB * NB); ++q)
            read_frag(f[(s + 1) & 1], last ? SN : S, last ? 0 : s + 1, q);
          if (last) {
            for (int q = i * kHalf / (MB * NB); q < (i + 1) * kHalf / (MB * NB); ++q)
              issue(q, S, kbytes - (kt + NS) * RB);
          } else if (s == 0 && kt > 0) {
            for (int q = i * (kLoads - kHalf) / (MB * NB);
                 q < (i + 1) * (kLoads - kHalf) / (MB * NB); ++q)
              issue(kHalf + q, SP, kbytes - (kt + NS - 1) * RB);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      S = SN;
    }
    wait_loads_barrier<0>();   // the stages become the epilogue's staging
  }

  // Epilogue: 32 rows at a time through the wave's own LDS region, so that
  // rows leave in whole 16-byte pieces; bias, activation and residual in
  // float32, one rounding.
  static constexpr int UN = 16 / sizeof(T);   // values of a 16-byte piece
  __device__ __forceinline__ uint32_t epi_off(int r, int c) const {   // c: 16-byte chunk
    constexpr int cpr = NB * 8;
    if constexpr (NB % 2 == 0) return r * NB * 128 + ((c ^ (r & 15)) << 4);
    else return r * NB * 128 + ((c ^ ((r >> 1) & 7)) << 4);
  }
  __device__ __forceinline__ void read_vals(uint32_t base, int r, int col, float (&v)[UN]) const {
#pragma unroll
    for (int h = 0; h < UN / 4; ++h) {
      const vec4u w = read16(base + epi_off(r, col / 4 + h));
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * h + i] = __uint_as_float(w[i]);
    }
  }

  __device__ __forceinline__ void epilogue(const TileAt& at, const f32x16 (&acc)[MB][NB]) const {
    const int F = GLU ? args.d_out / 2 : args.d_out;
    constexpr int wave_cols = GLU ? NB * 16 : NB * 32;
    constexpr int lanes = wave_cols / UN;    // lanes of one row
    constexpr int per = 64 / lanes;          // rows of one pass
    const uint32_t base = lds + wave * NB * 4096;
    const int c = (lane % lanes) * UN;
    const int col = at.col * kOut + wn * wave_cols + c;
    const bool col_ok = col < F;
    const T* bias = static_cast<const T*>(args.bias);
    float ba[UN], bb[UN];
#pragma unroll
    for (int i = 0; i < UN; ++i) ba[i] = bb[i] = 0.f;
    if (bias != nullptr && col_ok) {
      load_vals(bias + (int64_t)at.e * args.d_out + col, ba);
      if (GLU) load_vals(bias + (int64_t)at.e * args.d_out + F + col, bb);
    }
#pragma unroll
    for (int a = 0; a < MB; ++a) {
      const int r0 = (wm * MB + a) * 32;
      if (r0 >= at.rows) break;   // wave-uniform
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int chunk16 = (b * 32 + 8 * g + 4 * (lane >> 5)) / 4;
          f32x4 q;
#pragma unroll
          for (int i = 0; i < 4; ++i) q[i] = acc[a][b][4 * g + i];
          *reinterpret_cast<LDS_AS f32x4*>(
              (LDS_AS char*)(uintptr_t)(base + epi_off(lane & 31, chunk16))) = q;
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      for (int p = 0; p < 32 / per; ++p) {
        const int r = p * per + lane / lanes;
        if (r0 + r < at.rows && col_ok) {
          const int64_t o = (at.lo + r0 + r) * F + col;
          float z[UN], v[UN];
          read_vals(base, r, c, z);
#pragma unroll
          for (int i = 0; i < UN; ++i) z[i] += ba[i];
          if (args.pre_a != nullptr) store_vals(static_cast<T*>(args.pre_a) + o, z);
          if constexpr (GLU) {
            float w[UN];
            read_vals(base, r, NB * 16 + c, w);
#pragma unroll
            for (int i = 0; i < UN; ++i) w[i] += bb[i];
            if (args.pre_b != nullptr) store_vals(static_cast<T*>(args.pre_b) + o, w);
#pragma unroll
            for (int i = 0; i < UN; ++i) v[i] = z[i] * sigmoid_f32(z[i]) * w[i];
          } else {
#pragma unroll
            for (int i = 0; i < UN; ++i) v[i] = activate(args.act, z[i]);
          }
          if (args.residual != nullptr) {
            float r8[UN];
            load_vals(static_cast<const T*>(args.residual) + o, r8);
#pragma unroll
            for (int i = 0; i < UN; ++i) v[i] += r8[i];
          }
          store_vals(static_cast<T*>(args.y) + o, v);
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  }
};

template <typename G>
__global__ __launch_bounds__(G::kThreads, G::kWavesPerSimd) void gemm_kernel(ForwardArgs args,
                                                                             int cols, int group) {
  __shared__ __attribute__((aligned(16))) char smem[G::kLds];
  TileAt at;
  if (!find_tile(args.seg, args.E, args.P, G::TM, cols, group, at)) return;
  G g(args, at, (LDS_AS char*)smem);
  f32x16 acc[G::kMB][G::kNB];
  g.mainloop(acc);
  g.epilogue(at, acc);
}

// ---------------------------------------------------------------- few rows
// With few rows an expert the product is bound by reading W once.  A workgroup
// takes 16 rows and 16 * NC rows of W; its four waves split K and read both
// operands straight into fragments (no LDS, nothing is reused), partial sums
// meet in LDS.
template <typename T, int NC, bool GLU>
__global__ __launch_bounds__(256) void few_rows_kernel(ForwardArgs args, int cols, int group) {
  constexpr int kOut = GLU ? NC * 8 : NC * 16;
  __shared__ float part[4][16][NC * 16 + 4];
  TileAt at;
  if (!find_tile(args.seg, args.E, args.P, 16, cols, group, at)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int F = GLU ? args.d_out / 2 : args.d_out;
  const int kbytes = args.d_in * (int)sizeof(T);
  const int steps = (kbytes + 63) / 64;
  const int share = (steps + 3) / 4;
  const int first = wave * share;
  const int end = first + share < steps ? first + share : steps;
  const char* zero = reinterpret_cast<const char*>(zero_page);
  const int off = (lane >> 4) * 16;
  const char* wp[NC];
  int wstep[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = lane & 15;
    int64_t n;
    bool ok;
    if constexpr (GLU) {
      const int o = at.col * kOut + (c % (NC / 2)) * 16 + i;
      ok = o < F;
      n = (int64_t)(c / (NC / 2)) * F + o;
    } else {
      n = at.col * kOut + c * 16 + i;
      ok = n < F;
    }
    wp[c] = ok ? reinterpret_cast<const char*>(static_cast<const T*>(args.W) +
                                               ((int64_t)at.e * args.d_out + n) * args.d_in) +
                     off + first * 64
               : zero;
    wstep[c] = ok ? 64 : 0;
  }
  const char* xp = (lane & 15) < at.rows ? x_row<T>(args, at.lo + (lane & 15)) : nullptr;
  const int xstep = xp != nullptr ? 64 : 0;
  xp = xp != nullptr ? xp + off + first * 64 : zero;
  f32x4 acc[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
  constexpr int U = 8;
  int s = first;
  const int whole = kbytes / 64 < end ? kbytes / 64 : end;   // steps without a K tail
  for (; s + U <= whole; s += U) {
    vec4u w[U][NC], x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
        w[u][c] = *reinterpret_cast<const vec4u*>(wp[c] + u * wstep[c]);
      x[u] = *reinterpret_cast<const vec4u*>(xp + u * xstep);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[c] = mfma16<T>(w[u][c], x[u], acc[c]);
#pragma unroll
    for (int c = 0; c < NC; ++c) wp[c] += U * wstep[c];
    xp += U * xstep;
  }
  for (; s < end; ++s) {
    const bool in = s * 64 + off < kbytes;
    const vec4u x = *reinterpret_cast<const vec4u*>(in ? xp : zero);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const vec4u w = *reinterpret_cast<const vec4u*>(in ? wp[c] : zero);
      acc[c] = mfma16<T>(w, x, acc[c]);
      wp[c] += wstep[c];
    }
    xp += xstep;
  }
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[wave][lane & 15][c * 16 + 4 * (lane >> 4) + i] = acc[c][i];
  __syncthreads();
  const T* bias = static_cast<const T*>(args.bias);
  T* y = static_cast<T*>(args.y);
  auto put = [](void* p, int64_t o, float v) {
    if constexpr (sizeof(T) == 2) static_cast<uint16_t*>(p)[o] = f32_to_bf16(v);
    else static_cast<float*>(p)[o] = v;
  };
  auto get = [](const void* p, int64_t o) {
    if constexpr (sizeof(T) == 2) return bf16_to_f32(static_cast<const uint16_t*>(p)[o]);
    else return static_cast<const float*>(p)[o];
  };
  for (int i = threadIdx.x; i < at.rows * kOut; i += 256) {
    const int r = i / kOut, c = i % kOut;
    const int col = at.col * kOut + c;
    if (col >= F) continue;
    const int64_t o = (at.lo + r) * F + col;
    float z = part[0][r][c] + part[1][r][c] + part[2][r][c] + part[3][r][c];
    if (bias != nullptr) z += get(bias, (int64_t)at.e * args.d_out + col);
    if (args.pre_a != nullptr) put(args.pre_a, o, z);
    float v;
    if constexpr (GLU) {
      const int cu = c + kOut;
      float b = part[0][r][cu] + part[1][r][cu] + part[2][r][cu] + part[3][r][cu];
      if (bias != nullptr) b += get(bias, (int64_t)at.e * args.d_out + F + col);
      if (args.pre_b != nullptr) put(args.pre_b, o, b);
      v = z * sigmoid_f32(z) * b;
    } else {
      v = activate(args.act, z);
    }
    if (args.residual != nullptr) v += get(args.residual, o);
    put(y, o, v);
  }
}

// ---------------------------------------------------------------- launch
int64_t grid_blocks(int64_t P, int E, int tm, int64_t cols) {
  const int64_t tiles = P / tm + (P < E ? P : E);   // most row tiles of P rows over E experts
  return (tiles * cols + 7) / 8 * 8;
}

template <typename G>
hipError_t launch_gemm(const ForwardArgs& a, int F, int group, hipStream_t s) {
  const int cols = (F + G::kOut - 1) / G::kOut;
  const int64_t blocks = grid_blocks(a.P, a.E, G::TM, cols);
  if (blocks * G::kThreads >= int64_t(1) << 32) return hipErrorInvalidValue;
  hipLaunchKernelGGL(gemm_kernel<G>, dim3((uint32_t)blocks), dim3(G::kThreads), 0, s, a, cols,
                     group);
  return hipGetLastError();
}

template <typename T, int NC, bool GLU>
hipError_t launch_few_rows(const ForwardArgs& a, int F, hipStream_t s) {
  constexpr int kOut = GLU ? NC * 8 : NC * 16;
  const int cols = (F + kOut - 1) / kOut;
  const int64_t blocks = grid_blocks(a.P, a.E, 16, cols);
  if (blocks * 256 >= int64_t(1) << 32) return hipErrorInvalidValue;
  hipLaunchKernelGGL((few_rows_kernel<T, NC, GLU>), dim3((uint32_t)blocks), dim3(256), 0, s, a,
                     cols, 8);
  return hipGetLastError();
}

template <bool GLU>
hipError_t forward_bf16(const ForwardArgs& a, int F, hipStream_t s) {
  const int64_t mean = a.P / a.E;
  if (mean <= 8) return launch_few_rows<uint16_t, 2, GLU>(a, F, s);
  if (mean < 256) return launch_gemm<Gemm<uint16_t, 2, 4, 2, 2, 64, 3, GLU>>(a, F, 4, s);
  return launch_gemm<Gemm<uint16_t, 4, 4, 2, 2, 64, 4, GLU>>(a, F, 8, s);
}

template <bool GLU>
hipError_t forward_f32(const ForwardArgs& a, int F, hipStream_t s) {
  if (a.P / a.E <= 8) return launch_few_rows<float, 2, GLU>(a, F, s);
  return launch_gemm<Gemm<float, 2, 2, 2, 2, 128, 2, GLU>>(a, F, 8, s);
}

}  // namespace

hipError_t launch_grouped_forward(int dtype, const ForwardArgs& a, hipStream_t s) {
  if (a.P == 0) return hipSuccess;
  const bool glu = a.act == LRMOE_ACT_SWIGLU;
  const int F = glu ? a.d_out / 2 : a.d_out;
  if (dtype == LRMOE_BF16) return glu ? forward_bf16<true>(a, F, s) : forward_bf16<false>(a, F, s);
  return glu ? forward_f32<true>(a, F, s) : forward_f32<false>(a, F, s);
}

}  // namespace lrmoe
