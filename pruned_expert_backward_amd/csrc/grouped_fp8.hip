// Grouped expert product on 8-bit blocks (fp8.h), with the epilogue of
// grouped_forward.hip:
//
//   z_u[n] = sum over blocks b of 128 columns
//              2^(sx[row(u), b] + sw[n / 128, b]) * sum_{k in b} xq[row(u), k] Wq[n, k]
//   y_u = act(z_u + bias) + residual_u
//
// A K step is one block: 128 bytes of every row, a cache line and the depth of
// one scaled matrix instruction (v_mfma_scale_f32_16x16x128_f8f6f4), which takes the
// two scale bytes of its rows as operands and adds the scaled products to float32
// accumulators.  So the scales cost no arithmetic; they wait in LDS, as dwords of four
// steps, and are shifted by a byte a step.
//
// The instruction adds the products of a run of 8 on one scale and cuts off what
// lies below 2^-13 of the largest (measured); the runs' sums and the accumulator are
// float32.  Over a row that is some 2^-16 of the sum of absolute terms, far below the
// rounding to bfloat16 at the end; exact products would take the bfloat16
// instructions, at half the rate.
#include "fp8.h"
#include "grouped_tiles.h"

namespace lrmoe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct Fp8Args {
  ForwardArgs f;
  const uint8_t* xs;   // [T, pitch]
  const uint8_t* ws;   // [E, ceil(d_out / 128), pitch]
};

// 32 of a row's 128 values of a step: chunks g and g + 4 of 16 bytes in lane group
// g, the same ones in both operands.
struct Frag {
  vec4u lo, hi;
};

__device__ __forceinline__ f32x4 mfma(const Frag& a, const Frag& b, f32x4 c, uint32_t sa,
                                      uint32_t sb) {
  const i32x8 va = {(int)a.lo[0], (int)a.lo[1], (int)a.lo[2], (int)a.lo[3],
                    (int)a.hi[0], (int)a.hi[1], (int)a.hi[2], (int)a.hi[3]};
  const i32x8 vb = {(int)b.lo[0], (int)b.lo[1], (int)b.lo[2], (int)b.lo[3],
                    (int)b.hi[0], (int)b.hi[1], (int)b.hi[2], (int)b.hi[3]};
  // e4m3 in both; the scales' low bytes
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, c, 0, 0, 0, (int)sa, 0, (int)sb);
}

__device__ __forceinline__ int scale_blocks(int d) { return (d + kFp8Block - 1) / kFp8Block; }

// Each column tile of each expert starts its K loop this many groups of four K steps
// after its neighbour's and goes round, so that they do not all read the same few
// memory channels.
constexpr int kStaggerGroups = 1;

template <int WR, int WC, int WM, int WN, int NS, bool GLU, bool FAR = false>
struct Gemm8 {
  static constexpr int MI = 16, RB = 128;
  static constexpr int MB = WR / MI, NB = WC / MI;
  static constexpr int kMB = MB, kNB = NB;
  static constexpr int kWaves = WM * WN;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kWavesPerSimd = 2;
  static constexpr int TM = WM * WR, TN = WN * WC;
  static constexpr int kOut = GLU ? TN / 2 : TN;
  static constexpr int kChunks = RB / 16;
  static constexpr int kStage = (TM + TN) * RB;
  static constexpr int kPwA = TM * RB / 1024 / kWaves, kPwB = TN * RB / 1024 / kWaves;
  static constexpr int kLoads = kPwA + kPwB;
  typedef Epilogue<uint16_t, WR, WC, WM, WN, GLU> Epi;
  static constexpr int kStages = NS * kStage > Epi::kLds ? NS * kStage : Epi::kLds;
  // scales: K steps that LDS holds at a time; dwords of a row, one more so that 16
  // rows fall on distinct banks
  static constexpr int kScaleSteps = 32;
  static constexpr int kScalePitch = kScaleSteps / 4 + 1;
  static constexpr int kLds = kStages + (TM + TN) * kScalePitch * 4;
  static constexpr int R = NB < 4 ? NB : 4;   // B fragments in registers
  // The scales of a wave's columns: one for all of them, which start at a multiple of
  // WC; the up rows of SwiGLU start at F plus that and may cross into the next 128
  // anywhere, so a lane looks at its own row of each block.
  static constexpr int kScales = GLU ? 1 + NB / 2 : 1;
  __device__ __forceinline__ static constexpr int scale_of(int b) {
    return GLU && b >= NB / 2 ? 1 + b - NB / 2 : 0;
  }
  static_assert(128 % WC == 0, "a wave's columns in one block of 128");
  static_assert(TM * RB % (1024 * kWaves) == 0 && TN * RB % (1024 * kWaves) == 0, "whole loads");
  static_assert(!GLU || NB % 2 == 0, "gate and up blocks of a wave");
  static_assert(NB % R == 0, "fragments keep their registers over the steps");

  __device__ __forceinline__ static int swz(int r) { return (r >> 1) & 7; }

  const Fp8Args& args;
  uint32_t lds, scales;    // LDS byte addresses
  int lane, wave, wm, wn;
  int kbytes, nk, k0;
  __amdgpu_buffer_rsrc_t xbuf, wbuf;
  uint32_t off[FAR ? 1 : kLoads];
  const char* src[FAR ? kLoads : 1];
  int step[FAR ? kLoads : 1];
  static constexpr int kRowsPer = 1024 / RB;
  static constexpr int kVar = 16 / kRowsPer;
  static constexpr int kVarA = std::min(kPwA, kVar), kVarB = std::min(kPwB, kVar);
  int cha[kVarA], chb[kVarB];
  uint32_t fa, fb;         // fragment base addresses (A rows, B rows of the wave)
  uint32_t fs[2];          // lane's offset of the halves of a fragment
  uint32_t sa, sb;         // the lane's rows in the scales

  // Row of the expert's weights in LDS row r of the B operand, or -1.
  __device__ __forceinline__ static int64_t w_row(const TileAt& at, int r, int F) {
    if constexpr (GLU) {
      // of wave column w = r / WC first the gate rows, then the up rows
      constexpr int half = WC / 2;
      const int w = r / WC, i = r % WC;
      const int c = at.col * kOut + w * half + i % half;
      return c < F ? (int64_t)(i / half) * F + c : -1;
    } else {
      const int64_t n = (int64_t)at.col * TN + r;
      return n < F ? n : -1;
    }
  }

  __device__ __forceinline__ Gemm8(const Fp8Args& a8, const TileAt& at, LDS_AS char* smem)
      : args(a8) {
    const ForwardArgs& a = a8.f;
    lds = (uint32_t)(uintptr_t)smem;
    scales = lds + kStages;
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = wave / WN;
    wn = wave % WN;
    kbytes = a.d_in;
    nk = (kbytes + RB - 1) / RB;
    k0 = 0;
    const int groups = nk / 4 < 16 ? nk / 4 : 16;
    if constexpr (!FAR)
      if (groups > 1) k0 = (at.e * 64 + at.col) * kStaggerGroups % groups * 4;
    const int F = GLU ? a.d_out / 2 : a.d_out;
    const char* W = static_cast<const char*>(a.W) + (int64_t)at.e * a.d_out * kbytes;
    const char* x = static_cast<const char*>(a.x);
    if (!FAR) {
      int64_t rows = a.T;
      if (a.row_index == nullptr) {   // the tile's own rows
        x += at.lo * kbytes;
        rows = at.rows;
      }
      xbuf = buffer(x, rows * kbytes);
      wbuf = buffer(W, (int64_t)a.d_out * kbytes);
    }
#pragma unroll
    for (int j = 0; j < kVarA; ++j)
      cha[j] = ((lane % kChunks) ^ swz((wave * kPwA + j) * kRowsPer + lane / kChunks)) * 16;
#pragma unroll
    for (int j = 0; j < kVarB; ++j)
      chb[j] = ((lane % kChunks) ^ swz((wave * kPwB + j) * kRowsPer + lane / kChunks)) * 16;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const bool isA = j < kPwA;
      const int blk = isA ? wave * kPwA + j : wave * kPwB + j - kPwA;
      const int r = blk * kRowsPer + lane / kChunks;
      const int ch = chunk_of(j);
      int64_t n;   // row of x or of the expert's weights
      bool ok;
      if (isA) {
        ok = r < at.rows;
        n = ok && a.row_index != nullptr ? (int64_t)a.row_index[at.lo + r]
                                         : (FAR ? at.lo + r : (int64_t)r);
        ok = ok && n >= 0 && n < (a.row_index != nullptr || FAR ? a.T : (int64_t)at.rows);
      } else {
        n = w_row(at, r, F);
        ok = n >= 0;
      }
      if constexpr (FAR) {
        step[j] = ok ? RB : 0;
        src[j] = ok ? (isA ? x : W) + n * kbytes + ch : reinterpret_cast<const char*>(zero_page);
      } else {
        off[j] = ok ? (uint32_t)n * (uint32_t)kbytes + ch : kOutOfRange;
      }
    }
    const int fr = lane % MI;
#pragma unroll
    for (int h = 0; h < 2; ++h) fs[h] = fr * RB + (((h * 4 + lane / MI) ^ swz(fr)) << 4);
    fa = lds + wm * WR * RB;
    fb = lds + TM * RB + wn * WC * RB;
    sa = scales + (wm * WR + fr) * kScalePitch * 4;
    sb = scales + (TM + wn * WC + fr) * kScalePitch * 4;
  }

  __device__ __forceinline__ int chunk_of(int j) const {
    return j < kPwA ? cha[j % kVarA] : chb[(j - kPwA) % kVarB];
  }

  // Load j of K step kt into stage buffer `buf`.  Past the end of K it writes
  // zeros (with scalar offset 0, which keeps the range check's difference positive).
  __device__ __forceinline__ void issue(int j, int buf, int kt) {
    const bool isA = j < kPwA;
    const int blk = isA ? wave * kPwA + j : wave * kPwB + j - kPwA;
    const uint32_t dst =
        __builtin_amdgcn_readfirstlane(lds + buf * kStage + (isA ? 0 : TM * RB) + blk * 1024);
    const int at = kt >= nk ? 0 : (kt + k0 < nk ? kt + k0 : kt + k0 - nk) * RB;
    const int left = kt < nk ? kbytes - at : 0;
    const bool in = chunk_of(j) < left;
    if constexpr (FAR) {
      load_lds16(dst, in ? src[j] : reinterpret_cast<const char*>(zero_page));
      src[j] += step[j];
    } else {
      load_lds16(dst, isA ? xbuf : wbuf, in ? off[j] : kOutOfRange, at);
    }
  }

  // The scales of K steps first .. first + kScaleSteps - 1 of all the tile's rows
  // into LDS; 1 for rows and steps that are not there (their values are zeros).
  __device__ __forceinline__ void fill_scales(const TileAt& at, int first) const {
    const ForwardArgs& a = args.f;
    constexpr int kDwords = kScaleSteps / 4;
    const int F = GLU ? a.d_out / 2 : a.d_out;
    const int pitch = fp8_scale_row(a.d_in);
    const uint8_t* ws = args.ws + (int64_t)at.e * scale_blocks(a.d_out) * pitch;
    for (int i = threadIdx.x; i < (TM + TN) * kDwords; i += kThreads) {
      const int r = i / kDwords, j = i % kDwords;
      const uint8_t* p = nullptr;
      if (first + 4 * j < nk) {
        if (r < TM) {
          if (r < at.rows) {
            const int64_t n = a.row_index != nullptr ? (int64_t)a.row_index[at.lo + r] : at.lo + r;
            if (n >= 0 && n < a.T) p = args.xs + n * pitch;
          }
        } else {
          const int64_t n = w_row(at, r - TM, F);
          if (n >= 0) p = ws + n / kFp8Block * pitch;
        }
      }
      const uint32_t w =
          p != nullptr ? *reinterpret_cast<const uint32_t*>(p + first + 4 * j) : 0x7F7F7F7Fu;
      *reinterpret_cast<LDS_AS uint32_t*>(
          (LDS_AS char*)(uintptr_t)(scales + (r * kScalePitch + j) * 4)) = w;
    }
  }
  __device__ __forceinline__ static uint32_t read_dword(uint32_t addr) {
    return *reinterpret_cast<LDS_AS const uint32_t*>((LDS_AS char*)(uintptr_t)addr);
  }

  __device__ __forceinline__ Frag frag(uint32_t base, int buf, int i) const {
    const uint32_t at = base + buf * kStage + i * MI * RB;
    return Frag{read_lds16(at + fs[0]), read_lds16(at + fs[1])};
  }

  // One K step.  Its A fragments and its first R B fragments are in registers.  First
  // the B blocks whose registers the step's other B blocks then take.  Then the
  // barrier: all of this stage is in registers, the next stage's loads (the oldest
  // ones) are in LDS; its fragments are read as registers come free, A row block
  // by A row block, and the loads of step kt + NS go out over the stage.
  static constexpr int kLate = MB * R;    // products behind the barrier
  __device__ __forceinline__ static constexpr int spread(int i, int n, int span) {
    return i >= span ? n : i * n / span;
  }
  __device__ __forceinline__ void round(int kt, int S, Frag (&a_)[MB], Frag (&b_)[R],
                                        uint32_t (&xs_)[MB], uint32_t (&ws_)[kScales],
                                        f32x4 (&acc)[MB][NB]) {
    const int SN = S + 1 == NS ? 0 : S + 1;
    __builtin_amdgcn_s_setprio(1);
    static_for<(NB - R) * MB>([&](auto i_) __attribute__((always_inline)) {
      constexpr int i = i_, b = i / MB, a = i % MB;
      acc[a][b] = mfma(b_[b % R], a_[a], acc[a][b], ws_[scale_of(b)], xs_[a]);
      if constexpr (a == MB - 1) b_[b % R] = frag(fb, S, b + R);
      __builtin_amdgcn_sched_barrier(0);
    });
    __builtin_amdgcn_s_setprio(0);
    wait_loads_barrier<(NS - 2) * kLoads>();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
    static_for<kLate>([&](auto i_) __attribute__((always_inline)) {
      constexpr int i = i_, a = i / R, q = i % R, b = NB - R + q;
      acc[a][b] = mfma(b_[q], a_[a], acc[a][b], ws_[scale_of(b)], xs_[a]);
      if constexpr (q == R - 1) a_[a] = frag(fa, SN, a);
      if constexpr (a == MB - 1) b_[q] = frag(fb, SN, q);
      constexpr int l0 = spread(i, kLoads, kLate), l1 = spread(i + 1, kLoads, kLate);
      static_for<l1 - l0>([&](auto l) __attribute__((always_inline)) {
        issue(l0 + l, S, kt + NS);
      });
      __builtin_amdgcn_sched_barrier(0);
    });
    __builtin_amdgcn_s_setprio(0);
#pragma unroll
    for (int a = 0; a < MB; ++a) xs_[a] >>= 8;
#pragma unroll
    for (int b = 0; b < kScales; ++b) ws_[b] >>= 8;
  }

  __device__ __forceinline__ void mainloop(const TileAt& at, f32x4 (&acc)[MB][NB]) {
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[a][b] = f32x4{};
#pragma unroll
    for (int d = 0; d < NS; ++d)
#pragma unroll
      for (int j = 0; j < kLoads; ++j) issue(j, d, d);
    fill_scales(at, k0 / kScaleSteps * kScaleSteps);
    wait_loads_barrier<(NS - 1) * kLoads>();
    Frag a_[MB], b_[R];
#pragma unroll
    for (int i = 0; i < MB; ++i) a_[i] = frag(fa, 0, i);
#pragma unroll
    for (int i = 0; i < R; ++i) b_[i] = frag(fb, 0, i);
    uint32_t xs_[MB], ws_[kScales];
    int S = 0, k = k0;   // k: the K step of this turn
    for (int kt = 0; kt < nk; ++kt) {
      if (k % 4 == 0) {
        if (k % kScaleSteps == 0 && nk > kScaleSteps && kt > 0) {
          // everybody has read the last of the old ones before the barrier of the
          // step that has just ended
          fill_scales(at, k);
          __syncthreads();
        }
        const uint32_t j = k % kScaleSteps / 4 * 4;
#pragma unroll
        for (int i = 0; i < MB; ++i) xs_[i] = read_dword(sa + i * MI * kScalePitch * 4 + j);
#pragma unroll
        for (int i = 0; i < kScales; ++i)
          ws_[i] = read_dword(sb + (i == 0 ? 0 : NB / 2 + i - 1) * MI * kScalePitch * 4 + j);
      }
      round(kt, S, a_, b_, xs_, ws_, acc);
      S = S + 1 == NS ? 0 : S + 1;
      k = k + 1 == nk ? 0 : k + 1;
    }
    wait_loads_barrier<0>();   // the stages become the epilogue's staging
  }
};

template <typename G>
__device__ __forceinline__ void run_tile(const Fp8Args& args, const TileAt& at,
                                         LDS_AS char* smem) {
  G g(args, at, smem);
  f32x4 acc[G::kMB][G::kNB];
  g.mainloop(at, acc);
  G::Epi::run(args.f, at, acc, g.lds, g.lane, g.wave);
}

template <typename G>
__global__ __launch_bounds__(G::kThreads, G::kWavesPerSimd) void gemm8_kernel(Fp8Args args,
                                                                              int cols) {
  __shared__ __attribute__((aligned(16))) char smem[G::kLds];
  TileAt at;
  if (!find_tile(args.f.seg, args.f.E, args.f.P, G::TM, cols, at)) return;
  run_tile<G>(args, at, (LDS_AS char*)smem);
}

template <bool GLU>
struct Ragged8 {
  typedef Gemm8<64, 128, 4, 2, 2, GLU> G256;
  typedef Gemm8<64, 64, 2, 4, 3, GLU> G128;
  typedef Gemm8<32, 64, 2, 4, 3, GLU> G64;
  static constexpr int kLds = std::max(std::max(G256::kLds, G128::kLds), G64::kLds);
  static constexpr int kThreads = G256::kThreads, kOut = G256::kOut;
};

template <bool GLU>
__global__ __launch_bounds__(512, 2) void ragged_gemm8_kernel(Fp8Args args, int cols) {
  typedef Ragged8<GLU> R;
  __shared__ __attribute__((aligned(16))) char smem[R::kLds];
  TileAt at;
  if (!find_ragged_tile(args.f.seg, args.f.E, args.f.P, cols, at)) return;
  if (at.rows > 128) run_tile<typename R::G256>(args, at, (LDS_AS char*)smem);
  else if (at.rows > 64) run_tile<typename R::G128>(args, at, (LDS_AS char*)smem);
  else run_tile<typename R::G64>(args, at, (LDS_AS char*)smem);
}

// ---------------------------------------------------------------- few rows
// 16 rows and 16 * NC rows of W a workgroup; its four waves split K in groups of
// four steps and read both operands straight into fragments, with the four scales of
// a group in one dword.  Partial sums meet in LDS.
template <int NC, bool GLU>
__global__ __launch_bounds__(256) void few_rows8_kernel(Fp8Args a8, int cols) {
  constexpr int kOut = GLU ? NC * 8 : NC * 16;
  __shared__ float part[4][16][NC * 16 + 4];
  const ForwardArgs& args = a8.f;
  TileAt at;
  if (!find_tile(args.seg, args.E, args.P, 16, cols, at)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int F = GLU ? args.d_out / 2 : args.d_out;
  const int K = args.d_in, pitch = fp8_scale_row(K);
  const int groups = (K + 4 * kFp8Block - 1) / (4 * kFp8Block);
  const int share = (groups + 3) / 4;
  const int first = wave * share;
  const int end = first + share < groups ? first + share : groups;
  const uint8_t* zero = reinterpret_cast<const uint8_t*>(zero_page);
  const int off = (lane >> 4) * 16;
  const uint8_t *wp[NC], *ws[NC];   // rows' first bytes, or null
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
    wp[c] = ok ? static_cast<const uint8_t*>(args.W) + ((int64_t)at.e * args.d_out + n) * K
               : nullptr;
    ws[c] = ok ? a8.ws + ((int64_t)at.e * scale_blocks(args.d_out) + n / kFp8Block) * pitch
               : nullptr;
  }
  int64_t row = -1;
  if ((lane & 15) < at.rows) {
    const int64_t u = at.lo + (lane & 15);
    row = args.row_index != nullptr ? (int64_t)args.row_index[u] : u;
    if (row >= args.T) row = -1;
  }
  const uint8_t* xp = row >= 0 ? static_cast<const uint8_t*>(args.x) + row * K : nullptr;
  const uint8_t* xs = row >= 0 ? a8.xs + row * pitch : nullptr;
  f32x4 acc[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto piece = [&](const uint8_t* p, int k) __attribute__((always_inline)) {
    return *reinterpret_cast<const vec4u*>(p != nullptr && k < K ? p + k : zero);
  };
  auto dword = [&](const uint8_t* p, int g) __attribute__((always_inline)) {
    return p != nullptr ? *reinterpret_cast<const uint32_t*>(p + 4 * g) : 0x7F7F7F7Fu;
  };
  for (int g = first; g < end; ++g) {
    Frag w[4][NC], x[4];
    uint32_t sw[NC], sx;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = (4 * g + u) * kFp8Block + off;
#pragma unroll
      for (int c = 0; c < NC; ++c) w[u][c] = Frag{piece(wp[c], k), piece(wp[c], k + 64)};
      x[u] = Frag{piece(xp, k), piece(xp, k + 64)};
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) sw[c] = dword(ws[c], g);
    sx = dword(xs, g);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int c = 0; c < NC; ++c)
        acc[c] = mfma(w[u][c], x[u], acc[c], sw[c] >> (8 * u), sx >> (8 * u));
  }
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[wave][lane & 15][c * 16 + 4 * (lane >> 4) + i] = acc[c][i];
  __syncthreads();
  few_rows_epilogue<uint16_t, NC, GLU>(args, at, part);
}

// ---------------------------------------------------------------- launch
template <typename G>
hipError_t launch_gemm(const Fp8Args& a, int F, hipStream_t s) {
  const int cols = (F + G::kOut - 1) / G::kOut;
  const int64_t blocks = grid_blocks(a.f.P, a.f.E, G::TM, cols);
  if (blocks * G::kThreads >= int64_t(1) << 32) return hipErrorInvalidValue;
  hipLaunchKernelGGL(gemm8_kernel<G>, dim3((uint32_t)blocks), dim3(G::kThreads), 0, s, a, cols);
  return hipGetLastError();
}

template <bool GLU>
hipError_t launch_ragged(const Fp8Args& a, int F, hipStream_t s) {
  typedef Ragged8<GLU> R;
  const int cols = (F + R::kOut - 1) / R::kOut;
  const int64_t blocks = ragged_blocks(a.f, cols);
  if (blocks * R::kThreads >= int64_t(1) << 32) return hipErrorInvalidValue;
  hipLaunchKernelGGL((ragged_gemm8_kernel<GLU>), dim3((uint32_t)blocks), dim3(R::kThreads), 0, s,
                     a, cols);
  return hipGetLastError();
}

template <int NC, bool GLU>
hipError_t launch_few_rows(const Fp8Args& a, int F, hipStream_t s) {
  constexpr int kOut = GLU ? NC * 8 : NC * 16;
  const int cols = (F + kOut - 1) / kOut;
  const int64_t blocks = grid_blocks(a.f.P, a.f.E, 16, cols);
  if (blocks * 256 >= int64_t(1) << 32) return hipErrorInvalidValue;
  hipLaunchKernelGGL((few_rows8_kernel<NC, GLU>), dim3((uint32_t)blocks), dim3(256), 0, s, a,
                     cols);
  return hipGetLastError();
}

template <bool GLU>
hipError_t forward(const Fp8Args& a, int F, bool far, hipStream_t s) {
  constexpr int h = GLU ? 2 : 1;   // W rows of an output column
  if (expected(a.f, F, 16, 32 / h) <= 320) return launch_few_rows<2, GLU>(a, F, s);
  if (far) return launch_gemm<Gemm8<32, 64, 2, 2, 3, GLU, true>>(a, F, s);
  if (a.f.P <= (int64_t)16 * a.f.E && expected(a.f, F, 32, 256 / h) >= 160)
    return launch_gemm<Gemm8<32, 64, 1, 4, 3, GLU>>(a, F, s);
  if (expected(a.f, F, 32, 64 / h) <= 320)
    return launch_gemm<Gemm8<32, 32, 1, 2, 4, GLU>>(a, F, s);
  if (expected(a.f, F, 64, 64 / h) <= 400)
    return launch_gemm<Gemm8<32, 32, 2, 2, 3, GLU>>(a, F, s);
  if (expected(a.f, F, 64, 128 / h) <= 512)
    return launch_gemm<Gemm8<32, 64, 2, 2, 3, GLU>>(a, F, s);
  return launch_ragged<GLU>(a, F, s);
}

}  // namespace

hipError_t launch_grouped_forward_fp8(const ForwardArgs& f, const uint8_t* x_scale,
                                      const uint8_t* W_scale, hipStream_t s) {
  if (f.P == 0) return hipSuccess;
  const Fp8Args a{f, x_scale, W_scale};
  const bool glu = f.act == LRMOE_ACT_SWIGLU;
  const int F = glu ? f.d_out / 2 : f.d_out;
  // beyond a buffer's reach: one expert's weights, or x where its rows are picked by
  // index
  const bool far = (int64_t)f.d_out * f.d_in >= kNearBytes ||
                   (f.row_index != nullptr && f.T * f.d_in >= kNearBytes);
  return glu ? forward<true>(a, F, far, s) : forward<false>(a, F, far, s);
}

}  // namespace lrmoe
