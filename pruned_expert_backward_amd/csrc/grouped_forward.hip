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
// (v_mfma_f32_16x16x32_bf16, 8 values a fragment) and float32
// (v_mfma_f32_16x16x4_f32, 4 values a fragment, four products), float32
// accumulation in both.  Masked rows and the end of K read zeros.
//
// What bounds it (one GPU's 16 experts, Zipf-shared pairs):
//   many rows      the matrix cores: 8192^3 on one segment 810 us, 1.36 PFLOP/s
//                  (torch.mm 1.41 to 1.55 on the same machines).  32768 pairs,
//                  2048 -> 1536 SwiGLU with pre-activations 215 us, 0.96 PFLOP/s:
//                  3.2 rounds of tiles, each with 6 us of tile search, row indices
//                  and first loads ahead of it, and 150 MB of rows to write
//   some rows      reading W: 2000 pairs over 369 MB of W 83 us (4.5 TB/s) when
//                  evenly shared, 112 us with one expert of 591 rows, whose tiles
//                  walk the same K with more to multiply
//   few rows       one workgroup's walk over K: 2048 values take 7 to 9 us for 1
//                  to 16 rows
//   float32        the float32 matrix rate (157 TFLOP/s): 4097 pairs, 768 -> 2048
//                  124 us, 104 TFLOP/s; few rows read W: 32 pairs over 201 MB of
//                  W 45 us, 4.5 TB/s
//   more capacity than pairs
//                  empty workgroups, and a variant for the capacity: 512 pairs,
//                  2048 -> 1536 SwiGLU 19.7 us at their own size, 21.1 at eight
//                  times that; 32768 pairs 218 and 228 us, 768 -> 2048 131 and 159
#include "grouped_tiles.h"

namespace lrmoe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
// Row of x of pair row u: null when its index is out of range (a zero row).
template <typename T>
__device__ __forceinline__ const char* x_row(const ForwardArgs& a, int64_t u) {
  const int64_t r = a.row_index != nullptr ? (int64_t)a.row_index[u] : u;
  if (r < 0 || r >= a.T) return nullptr;
  return reinterpret_cast<const char*>(static_cast<const T*>(a.x) + r * a.d_in);
}

// 16 x 16 products of 16-byte fragments: one bf16 product of 32 values of K, or
// four float32 products of 4 values.  (32 x 32 results, the same rate with half
// the fragments, were 5 to 8 % slower here: twice the accumulator traffic.)
template <typename T>
__device__ __forceinline__ f32x4 mfma(vec4u a, vec4u b, f32x4 c) {
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

// Each column tile of each expert starts its K loop this many K steps after
// its neighbour's and goes round: rows of W a power of two apart would else
// have all workgroups on the same few memory channels at a time (4096 columns:
// 87 us against 68 us for 369 MB of W; other strides are unchanged).
constexpr int kStagger = 3;

// Epilogue of a tile whose waves (WM x WN) hold WR x WC results each, in 16 x 16
// blocks: 32 rows at a time through the wave's own LDS region, so that rows leave
// in whole 16-byte pieces; bias, activation and residual in float32, one rounding
// to O.
template <typename O, int WR, int WC, int WM, int WN, bool GLU>
struct Epilogue {
  static constexpr int MI = 16;
  static constexpr int MB = WR / MI, NB = WC / MI;
  static constexpr int kOut = GLU ? WN * WC / 2 : WN * WC;
  static constexpr int kLds = WM * WN * WC * 128;
  static constexpr int UN = 16 / sizeof(O);   // values of a 16-byte piece
  __device__ __forceinline__ static uint32_t epi_off(int r, int c) {   // c: 16-byte chunk
    if constexpr (WC % 64 == 0) return r * WC * 4 + ((c ^ (r & 15)) << 4);
    else return r * WC * 4 + ((c ^ ((r >> 1) & 7)) << 4);
  }
  __device__ __forceinline__ static void read_vals(uint32_t base, int r, int col, float (&v)[UN]) {
#pragma unroll
    for (int h = 0; h < UN / 4; ++h) {
      const vec4u w = read_lds16(base + epi_off(r, col / 4 + h));
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * h + i] = __uint_as_float(w[i]);
    }
  }

  // lds: address of the staging of all waves
  __device__ __forceinline__ static void run(const ForwardArgs& args, const TileAt& at,
                                             const f32x4 (&acc)[MB][NB], uint32_t lds, int lane,
                                             int wave) {
    const int wm = wave / WN, wn = wave % WN;
    const int F = GLU ? args.d_out / 2 : args.d_out;
    constexpr int wave_cols = GLU ? WC / 2 : WC;
    constexpr int lanes = wave_cols / UN;    // lanes of one row
    constexpr int per = 64 / lanes;          // rows of one pass
    const uint32_t base = lds + wave * WC * 128;
    const int c = (lane % lanes) * UN;
    const int col = at.col * kOut + wn * wave_cols + c;
    const bool col_ok = col < F;
    const O* bias = static_cast<const O*>(args.bias);
    float ba[UN], bb[UN];
#pragma unroll
    for (int i = 0; i < UN; ++i) ba[i] = bb[i] = 0.f;
    if (bias != nullptr && col_ok) {
      load_vals(bias + (int64_t)at.e * args.d_out + col, ba);
      if (GLU) load_vals(bias + (int64_t)at.e * args.d_out + F + col, bb);
    }
    constexpr int G = 32 / MI;   // blocks of 32 rows
    static_for<MB / G>([&](auto a_) __attribute__((always_inline)) {
      constexpr int a = a_ * G;
      const int r0 = wm * WR + a * MI;
      if (r0 < at.rows) {   // wave-uniform
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int b = 0; b < NB; ++b)   // a lane holds 4 columns of one row
            *reinterpret_cast<LDS_AS f32x4*>((LDS_AS char*)(uintptr_t)(
                base + epi_off(g * MI + lane % MI, b * (MI / 4) + lane / 16))) = acc[a + g][b];
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
            if (args.pre_a != nullptr) store_vals(static_cast<O*>(args.pre_a) + o, z);
            if constexpr (GLU) {
              float w[UN];
              read_vals(base, r, WC / 2 + c, w);
#pragma unroll
              for (int i = 0; i < UN; ++i) w[i] += bb[i];
              if (args.pre_b != nullptr) store_vals(static_cast<O*>(args.pre_b) + o, w);
#pragma unroll
              for (int i = 0; i < UN; ++i) v[i] = z[i] * sigmoid_f32(z[i]) * w[i];
            } else {
#pragma unroll
              for (int i = 0; i < UN; ++i) v[i] = z[i];
              activate(args.act, v);
            }
            if (args.residual != nullptr) {
              float r8[UN];
              load_vals(static_cast<const O*>(args.residual) + o, r8);
#pragma unroll
              for (int i = 0; i < UN; ++i) v[i] += r8[i];
            }
            store_vals(static_cast<O*>(args.y) + o, v);
          }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
    });
  }
};

// T: storage.  A wave computes WR x WC, WM x WN waves a workgroup, NS LDS
// stages of one K step (128 bytes of every row) each.  128 bytes are a cache
// line: 64-byte steps with twice the stages were 5 to 15 % slower on every shape,
// 256-byte ones with half the stages 10 to 25 % on all but the smallest.  Two
// waves a SIMD: with one (128 x 128 a wave) the K loop ran 1.13 PFLOP/s on 8192^3.
template <typename T, int WR, int WC, int WM, int WN, int NS, bool GLU, bool FAR = false>
struct Gemm {
  static constexpr int MI = 16, RB = 128;                  // MFMA rows; row bytes of a K step
  static constexpr int MB = WR / MI, NB = WC / MI;
  static constexpr int kMB = MB, kNB = NB;
  static constexpr int kWaves = WM * WN;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kWavesPerSimd = 2;
  static constexpr int TM = WM * WR, TN = WN * WC;
  static constexpr int kOut = GLU ? TN / 2 : TN;           // columns of y
  static constexpr int kSliceBytes = 64;                   // K bytes of one MFMA
  static constexpr int kSlices = RB / kSliceBytes;         // MFMA steps of a K step
  static constexpr int kChunks = RB / 16;
  static constexpr int kStage = (TM + TN) * RB;
  static constexpr int kPwA = TM * RB / 1024 / kWaves, kPwB = TN * RB / 1024 / kWaves;
  static constexpr int kLoads = kPwA + kPwB;               // load instructions a stage and wave
  typedef Epilogue<T, WR, WC, WM, WN, GLU> Epi;
  static constexpr int kLds = NS * kStage > Epi::kLds ? NS * kStage : Epi::kLds;
  static_assert(TM * RB % (1024 * kWaves) == 0 && TN * RB % (1024 * kWaves) == 0, "whole loads");
  static_assert(!GLU || NB % 2 == 0, "gate and up blocks of a wave");
  static_assert(kSlices % 2 == 0, "fragment sets alternate");

  // Chunk c of row r sits at slot c ^ swz(r): 16 consecutive rows of one chunk
  // (one LDS cycle of a 16-byte read) fall on 16 distinct bank groups.
  __device__ __forceinline__ static int swz(int r) {
    return (r >> 1) & 7;
  }

  const ForwardArgs& args;
  uint32_t lds;            // LDS byte address of stage 0
  int lane, wave, wm, wn;
  int kbytes, nk, k0;
  // Where this lane reads each of its loads.  Near: byte offsets into the
  // buffers of x and of the expert's weights, fixed over K.  Far (x or one
  // expert's weights beyond 2 GiB): addresses, advanced with K.
  __amdgpu_buffer_rsrc_t xbuf, wbuf;
  uint32_t off[FAR ? 1 : kLoads];
  const char* src[FAR ? kLoads : 1];
  int step[FAR ? kLoads : 1];
  // Byte offset of the lane's chunk inside the step, which depends on the LDS
  // block of the load modulo kVar: a few values for each operand.
  static constexpr int kRowsPer = 1024 / RB;   // rows of a load
  static constexpr int kVar = 16 / kRowsPer;
  static constexpr int kVarA = std::min(kPwA, kVar), kVarB = std::min(kPwB, kVar);
  int cha[kVarA], chb[kVarB];
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
    k0 = 0;
    if constexpr (!FAR) k0 = (at.e * 64 + at.col) * kStagger % (nk < 64 ? nk : 64);
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
      } else if constexpr (GLU) {
        // LDS row r holds, of wave column w = r / WC, first the gate rows and
        // then the up rows of the wave's output columns
        constexpr int half = WC / 2;
        const int w = r / WC, i = r % WC;
        const int c = at.col * kOut + w * half + i % half;
        ok = c < F;
        n = (int64_t)(i / half) * F + c;
      } else {
        n = at.col * TN + r;
        ok = n < F;
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
    for (int s = 0; s < kSlices; ++s)
      fs[s] = fr * RB + (((s * (kSliceBytes / 16) + lane / MI) ^ swz(fr)) << 4);
    fa = lds + wm * WR * RB;
    fb = lds + TM * RB + wn * WC * RB;
  }

  __device__ __forceinline__ int chunk_of(int j) const {
    return j < kPwA ? cha[j % kVarA] : chb[(j - kPwA) % kVarB];
  }

  // Load j of K step kt into stage buffer `buf`.  Past the end of K it writes
  // zeros.
  __device__ __forceinline__ void issue(int j, int buf, int kt) {
    const bool isA = j < kPwA;
    const int blk = isA ? wave * kPwA + j : wave * kPwB + j - kPwA;
    const uint32_t dst =
        __builtin_amdgcn_readfirstlane(lds + buf * kStage + (isA ? 0 : TM * RB) + blk * 1024);
    // uniform: where the K step read starts (steps go round from k0), bytes left
    // from there.  Past the end of K it is 0: a load is out of range when its lane
    // offset reaches the buffer's size less the scalar offset, and a step behind nk
    // can lie past a buffer of one row, where that difference would be negative.
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

  __device__ __forceinline__ vec4u frag_a(int buf, int s, int i) const {
    return read_lds16(fa + buf * kStage + fs[s] + i * MI * RB);
  }
  __device__ __forceinline__ vec4u frag_b(int buf, int s, int i) const {
    return read_lds16(fb + buf * kStage + fs[s] + i * MI * RB);
  }

  // The K loop.  While slice s is multiplied, A row block by A row block, the
  // fragments of slice s + 1 are read: A's into the registers that their row
  // block has just left, B's into a second set.  Before the last slice one
  // barrier: the next stage is in LDS (its loads are the oldest ones), and
  // nobody reads buffer S any more; the loads of step kt + NS then go out
  // between the products.
  static constexpr int N = MB * NB;
  // The loads of a step go out over the first half of the products after the
  // barrier: over all of them they come too late for the next one (8192^3: 841
  // us, 948 us over all, 851 us over a quarter).
  static constexpr int kSpan = N * kSlices / 2;
  static_assert(kSpan <= N, "all loads of a step in its last slice");
  // Of n items spread over `span` slots, those before slot i.
  __device__ __forceinline__ static constexpr int spread(int i, int n, int span) {
    return i >= span ? n : i * n / span;
  }
  __device__ __forceinline__ void round(int kt, int S, vec4u (&fa_)[MB], vec4u (&fb_)[2][NB],
                                        f32x4 (&acc)[MB][NB]) {
    const int SN = S + 1 == NS ? 0 : S + 1;
    static_for<kSlices>([&](auto s_) __attribute__((always_inline)) {
      constexpr int s = s_, cur = s & 1;
      constexpr bool last = s == kSlices - 1;
      if (last) {
        wait_loads_barrier<(NS - 2) * kLoads>();
        __builtin_amdgcn_sched_barrier(0);
      }
      const int from = last ? SN : S;
      constexpr int at = last ? 0 : s + 1;
      __builtin_amdgcn_s_setprio(1);
      static_for<N>([&](auto i_) __attribute__((always_inline)) {
        constexpr int i = i_, a = i / NB, b = i % NB;
        acc[a][b] = mfma<T>(fb_[cur][b], fa_[a], acc[a][b]);
        if constexpr (b == NB - 1) fa_[a] = frag_a(from, at, a);
        // B fragments early, so that the next slice's first products have them
        constexpr int q0 = spread(i, NB, N / 2), q1 = spread(i + 1, NB, N / 2);
        static_for<q1 - q0>([&](auto q) __attribute__((always_inline)) {
          fb_[cur ^ 1][q0 + q] = frag_b(from, at, q0 + q);
        });
        if constexpr (last) {
          constexpr int l0 = spread(i, kLoads, kSpan), l1 = spread(i + 1, kLoads, kSpan);
          static_for<l1 - l0>([&](auto q) __attribute__((always_inline)) {
            issue(l0 + q, S, kt + NS);
          });
        }
        __builtin_amdgcn_sched_barrier(0);
      });
      __builtin_amdgcn_s_setprio(0);
    });
  }
  __device__ __forceinline__ void mainloop(f32x4 (&acc)[MB][NB]) {
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[a][b] = f32x4{};
#pragma unroll
    for (int d = 0; d < NS; ++d)
#pragma unroll
      for (int j = 0; j < kLoads; ++j) issue(j, d, d);
    wait_loads_barrier<(NS - 1) * kLoads>();
    vec4u fa_[MB], fb_[2][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i) fa_[i] = frag_a(0, 0, i);
#pragma unroll
    for (int i = 0; i < NB; ++i) fb_[0][i] = frag_b(0, 0, i);
    int S = 0;
    for (int kt = 0; kt < nk; ++kt) {
      round(kt, S, fa_, fb_, acc);
      S = S + 1 == NS ? 0 : S + 1;
    }
    wait_loads_barrier<0>();   // the stages become the epilogue's staging
  }

};

template <typename G>
__global__ __launch_bounds__(G::kThreads, G::kWavesPerSimd) void gemm_kernel(ForwardArgs args,
                                                                             int cols) {
  __shared__ __attribute__((aligned(16))) char smem[G::kLds];
  TileAt at;
  if (!find_tile(args.seg, args.E, args.P, G::TM, cols, at)) return;
  G g(args, at, (LDS_AS char*)smem);
  f32x4 acc[G::kMB][G::kNB];
  g.mainloop(acc);
  G::Epi::run(args, at, acc, g.lds, g.lane, g.wave);
}

// ---- 256-row tiles, ragged ends and the last round
// Tiles of 256 rows with one workgroup a CU: the ends of the segments get
// 128-row or 64-row code (an expert's last tile is half empty on average), and
// the last round of an XCD's 32 CUs, if it would fill half of them or fewer, is
// cut into 128-row or 64-row parts.  Whole tiles come first, then the ends,
// each list in eighths over the XCDs.  (The training shape above: 237 us with
// 256-row code alone, 215 us like this.)
template <typename G>
__device__ __forceinline__ void run_tile(const ForwardArgs& args, const TileAt& at,
                                         LDS_AS char* smem) {
  G g(args, at, smem);
  f32x4 acc[G::kMB][G::kNB];
  g.mainloop(acc);
  G::Epi::run(args, at, acc, g.lds, g.lane, g.wave);
}

template <typename T, bool GLU>
struct Ragged {
  typedef Gemm<T, 64, 128, 4, 2, 2, GLU> G256;
  typedef Gemm<T, 64, 64, 2, 4, 3, GLU> G128;
  typedef Gemm<T, 32, 64, 2, 4, 3, GLU> G64;
  static constexpr int kLds = std::max(std::max(G256::kLds, G128::kLds), G64::kLds);
  static constexpr int kThreads = G256::kThreads, kOut = G256::kOut;
};

template <typename T, bool GLU>
__global__ __launch_bounds__(512, 2) void ragged_gemm_kernel(ForwardArgs args, int cols) {
  typedef Ragged<T, GLU> R;
  __shared__ __attribute__((aligned(16))) char smem[R::kLds];
  TileAt at;
  if (!find_ragged_tile(args.seg, args.E, args.P, cols, at)) return;
  if (at.rows > 128) run_tile<typename R::G256>(args, at, (LDS_AS char*)smem);
  else if (at.rows > 64) run_tile<typename R::G128>(args, at, (LDS_AS char*)smem);
  else run_tile<typename R::G64>(args, at, (LDS_AS char*)smem);
}

// ---------------------------------------------------------------- few rows
// With few rows an expert the product is bound by reading W once.  A workgroup
// takes 16 rows and 16 * NC rows of W; its four waves split K and read both
// operands straight into fragments (no LDS, nothing is reused), partial sums
// meet in LDS.
template <typename T, int NC, bool GLU>
__global__ __launch_bounds__(256) void few_rows_kernel(ForwardArgs args, int cols) {
  constexpr int kOut = GLU ? NC * 8 : NC * 16;
  __shared__ float part[4][16][NC * 16 + 4];
  TileAt at;
  if (!find_tile(args.seg, args.E, args.P, 16, cols, at)) return;
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
      for (int c = 0; c < NC; ++c) acc[c] = mfma<T>(w[u][c], x[u], acc[c]);
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
      acc[c] = mfma<T>(w, x, acc[c]);
      wp[c] += wstep[c];
    }
    xp += xstep;
  }
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[wave][lane & 15][c * 16 + 4 * (lane >> 4) + i] = acc[c][i];
  __syncthreads();
  few_rows_epilogue<T, NC, GLU>(args, at, part);
}

// ---------------------------------------------------------------- launch
template <typename G>
hipError_t launch_gemm(const ForwardArgs& a, int F, hipStream_t s) {
  const int cols = (F + G::kOut - 1) / G::kOut;
  const int64_t blocks = grid_blocks(a.P, a.E, G::TM, cols);
  return launch_workgroups(gemm_kernel<G>, blocks, G::kThreads, s, a, cols);
}

template <typename T, bool GLU>
hipError_t launch_ragged(const ForwardArgs& a, int F, hipStream_t s) {
  typedef Ragged<T, GLU> R;
  const int cols = (F + R::kOut - 1) / R::kOut;
  const int64_t blocks = ragged_blocks(a, cols);
  return launch_workgroups(ragged_gemm_kernel<T, GLU>, blocks, R::kThreads, s, a, cols);
}

template <typename T, int NC, bool GLU>
hipError_t launch_few_rows(const ForwardArgs& a, int F, hipStream_t s) {
  constexpr int kOut = GLU ? NC * 8 : NC * 16;
  const int cols = (F + kOut - 1) / kOut;
  const int64_t blocks = grid_blocks(a.P, a.E, 16, cols);
  return launch_workgroups(few_rows_kernel<T, NC, GLU>, blocks, 256, s, a, cols);
}

// The smallest tiles whose workgroups the 256 CUs hold at once, or nearly:
// below that a product takes the time of one workgroup's walk over K, which
// grows with the tile; above it the operands' re-reads count.  Measured (us;
// W of 2048 columns and 1536 rows an expert, SwiGLU): 1 expert, 64 rows: 10.2
// without tiles, 12.3 with 32x64, 16.6 with 64x128, 34 with 256x256; 4
// experts, 64 rows each: 25.1, 13.3, 16.9, 34; 4 experts, 512 rows each: 147,
// 41, 24, 23; 16 experts, 512 rows each: 542, 149, 95, 71.
template <bool GLU>
hipError_t forward_bf16(const ForwardArgs& a, int F, bool far, hipStream_t s) {
  typedef uint16_t T;
  constexpr int h = GLU ? 2 : 1;   // W rows of an output column
  if (expected(a, F, 16, 32 / h) <= 320) return launch_few_rows<T, 2, GLU>(a, F, s);
  // 64-bit addresses, one shape: the 32768 pairs of a 2048 -> 1536 SwiGLU take 192
  // us from an x just within a buffer's reach and 294 us from one beyond it
  if (far) return launch_gemm<Gemm<T, 32, 64, 2, 2, 3, GLU, true>>(a, F, s);
  // few rows for much W: wide tiles keep more of W in flight (16 experts of
  // 4096 columns and 2816 rows, 8 rows each: 67 us, 76 with the tiles below)
  if (a.P <= (int64_t)16 * a.E && expected(a, F, 32, 256 / h) >= 160)
    return launch_gemm<Gemm<T, 32, 64, 1, 4, 4, GLU>>(a, F, s);
  if (expected(a, F, 32, 64 / h) <= 320)
    return launch_gemm<Gemm<T, 32, 32, 1, 2, 4, GLU>>(a, F, s);
  if (expected(a, F, 64, 64 / h) <= 400)
    return launch_gemm<Gemm<T, 32, 32, 2, 2, 3, GLU>>(a, F, s);
  if (expected(a, F, 64, 128 / h) <= 512)
    return launch_gemm<Gemm<T, 32, 64, 2, 2, 3, GLU>>(a, F, s);
  return launch_ragged<T, GLU>(a, F, s);
}

// float32 products are bound by the matrix units (a sixteenth of bf16's rate)
// from some 16 rows an expert on, so small tiles that spread evenly win
// throughout: 8 experts, 512 rows each, 768 columns and 2048 rows of W: 126 us
// with 64x64, 173 with 128x128, 216 with 256-row tiles.
template <bool GLU>
hipError_t forward_f32(const ForwardArgs& a, int F, bool far, hipStream_t s) {
  if (expected(a, F, 16, GLU ? 16 : 32) <= 800) return launch_few_rows<float, 2, GLU>(a, F, s);
  if (far) return launch_gemm<Gemm<float, 32, 32, 2, 2, 2, GLU, true>>(a, F, s);
  return launch_gemm<Gemm<float, 32, 32, 2, 2, 2, GLU>>(a, F, s);
}

}  // namespace

hipError_t launch_grouped_forward(int dtype, const ForwardArgs& a, hipStream_t s) {
  if (a.P == 0) return hipSuccess;
  const bool glu = a.act == LRMOE_ACT_SWIGLU;
  const int F = glu ? a.d_out / 2 : a.d_out;
  // beyond a buffer's reach: one expert's weights, or x where its rows are
  // picked by index
  const int64_t kbytes = (int64_t)a.d_in * (dtype == LRMOE_BF16 ? 2 : 4);
  const bool far = a.d_out * kbytes >= kNearBytes ||
                   (a.row_index != nullptr && a.T * kbytes >= kNearBytes);
  if (dtype == LRMOE_BF16)
    return glu ? forward_bf16<true>(a, F, far, s)
               : forward_bf16<false>(a, F, far, s);
  return glu ? forward_f32<true>(a, F, far, s) : forward_f32<false>(a, F, far, s);
}

}  // namespace lrmoe
