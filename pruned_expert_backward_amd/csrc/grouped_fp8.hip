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
// accumulators.  So the scales cost no arithmetic.  They wait in LDS, for each step and
// lane in one piece: a lane's row blocks are the bytes of a dword, which the
// instruction picks from.
//
// The instruction adds the products of a run of 8 on one scale and cuts off what
// lies below 2^-13 of the largest (measured); the runs' sums and the accumulator are
// float32.  Over a row that is some 2^-16 of the sum of absolute terms, far below the
// rounding to bfloat16 at the end; exact products would take the bfloat16
// instructions, at half the rate.
//
// What bounds it (one GPU's 16 experts, Zipf-shared pairs; the product alone, many in a row
// with two or three sets of inputs in turn.  Behind the quantisation of its rows, which
// leaves them in the caches and the clock higher, the training products take 140 and 151 us):
//   many rows   8192^3 on one segment 442 us, 2.5 PFLOP/s (the library's product with
//               one scale a tensor 355 us): of 820 thousand cycles the matrix units are busy
//               in 524.  A step of the loop loses some 15 % to LDS reads and loads at once
//               (80 thousand), a tile about 13 us ahead of the loop and behind it (100
//               thousand); the other 110 thousand are not accounted for.  32768 pairs, 2048 ->
//               1536 SwiGLU with pre-activations 148 us (151 MB of rows to write), 1536 ->
//               2048 in the gradient's direction 156 us: 16 and 12 steps a tile
//   some rows   reading W: 512 pairs over 184 MB of W 39 us, 4.7 TB/s; 1999 pairs with one
//               expert of 591 rows 68 us, whose tiles walk the same K with more to multiply
//   few rows    32 pairs over 50 MB of W 12.3 us, one row 5.2 us: a walk over K
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

// 32 of a row's 128 values of a step: two chunks of 16 bytes in each lane, the same
// ones in both operands.
struct Frag {
  vec4u lo, hi;
};

// c + 2^(x + y - 254) a b, with x in byte XA of sa and y in byte XB of sb.
template <int XA, int XB>
__device__ __forceinline__ f32x4 mfma(const Frag& a, const Frag& b, f32x4 c, uint32_t sa,
                                      uint32_t sb) {
  const i32x8 va = {(int)a.lo[0], (int)a.lo[1], (int)a.lo[2], (int)a.lo[3],
                    (int)a.hi[0], (int)a.hi[1], (int)a.hi[2], (int)a.hi[3]};
  const i32x8 vb = {(int)b.lo[0], (int)b.lo[1], (int)b.lo[2], (int)b.lo[3],
                    (int)b.hi[0], (int)b.hi[1], (int)b.hi[2], (int)b.hi[3]};
  // e4m3 in both
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, c, 0, 0, XA, (int)sa, XB,
                                                          (int)sb);
}

__device__ __forceinline__ int scale_blocks(int d) { return (d + kFp8Block - 1) / kFp8Block; }

// Each column tile of each expert starts its K loop this many K steps after its
// neighbour's and goes round, so that they do not all read the same few memory channels
// (128 pairs over 16 x 2816 x 4096: 37.6 us, 43.6 without); not with 256-row tiles, which
// share their rows of x in the L2 (32768 pairs, 2048 -> 1536: 145 us, 153 with).
constexpr int kStagger = 3;

// Byte q of four dwords into dword q, byte by byte (a 4 x 4 transpose).
__device__ __forceinline__ void flip_bytes(uint32_t (&w)[4]) {
  const uint32_t lo01 = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u);
  const uint32_t hi01 = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
  const uint32_t lo23 = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u);
  const uint32_t hi23 = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
  w[0] = __builtin_amdgcn_perm(lo23, lo01, 0x05040100u);
  w[1] = __builtin_amdgcn_perm(lo23, lo01, 0x07060302u);
  w[2] = __builtin_amdgcn_perm(hi23, hi01, 0x05040100u);
  w[3] = __builtin_amdgcn_perm(hi23, hi01, 0x07060302u);
}

// Eight consecutive columns a lane from two neighbouring 16 x 16 results, which hold
// four a lane: lane group g then has columns 8 g .. 8 g + 7 of the 32.
__device__ __forceinline__ void eight_columns(const f32x4& p, const f32x4& q, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // rows of lanes [p0 p1 q0 q1], [p2 p3 q2 q3], then [p0 p2 q0 q2], [p1 p3 q1 q3]
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(p[i]), __float_as_uint(q[i]),
                                                    false, false);
    const auto s = __builtin_amdgcn_permlane16_swap(r[0], r[1], false, false);
    v[i] = __uint_as_float(s[0]);
    v[4 + i] = __uint_as_float(s[1]);
  }
}

template <int WR, int WC, int WM, int WN, int NS, bool GLU, bool FAR = false>
struct Gemm8 {
  static constexpr int MI = 16, RB = 128;
  static constexpr int MB = WR / MI, NB = WC / MI;
  static constexpr int kMB = MB, kNB = NB;
  static constexpr int kWaves = WM * WN;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int TM = WM * WR, TN = WN * WC;
  static constexpr int kOut = GLU ? TN / 2 : TN;
  static constexpr int kChunks = RB / 16;
  static constexpr int kStage = (TM + TN) * RB;
  static constexpr int kPwA = TM * RB / 1024 / kWaves, kPwB = TN * RB / 1024 / kWaves;
  static constexpr int kLoads = kPwA + kPwB;
  // scales of a step in LDS: for each wave row and column, 16 lanes' dwords
  static constexpr int kA = (MB + 3) / 4, kB = (NB + 3) / 4;
  static constexpr int kUnitsA = WM * 16 * kA, kUnits = kUnitsA + WN * 16 * kB;
  // K steps whose scales LDS holds at a time
  static constexpr int kScaleSteps = TM < 256 ? 32 : 64;
  static constexpr int kLds = NS * kStage + kScaleSteps * kUnits * 4;
  static_assert(kLds <= 160 * 1024, "LDS of a CU");
  static constexpr int kWavesPerSimd = std::max(1, 160 * 1024 / kLds * kWaves / 4);
  static_assert(TM * RB % (1024 * kWaves) == 0 && TN * RB % (1024 * kWaves) == 0, "whole loads");
  static_assert(MB % 2 == 0 && NB % 2 == 0, "halves");

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
  uint32_t sa, sb;         // the lane's dwords in a step's scales

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
    scales = lds + NS * kStage;
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = wave / WN;
    wn = wave % WN;
    kbytes = a.d_in;
    nk = (kbytes + RB - 1) / RB;
    k0 = 0;
    // (a longer loop goes by runs of kScaleSteps, from the first one on)
    if constexpr (!FAR && TM < 256)
      if (nk <= kScaleSteps) k0 = (at.e * 64 + at.col) * kStagger % nk;
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
    sa = scales + (wm * 16 + fr) * kA * 4;
    sb = scales + (kUnitsA + (wn * 16 + fr) * kB) * 4;
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

  // Scales come into LDS four row blocks by four steps at a time.  A thread has four
  // rows of its own, the same ones for all its steps; null: not there (its values are
  // zeros, its scales 1).
  static constexpr int kSide = kThreads / kUnits;   // groups of four steps at once
  static_assert(kSide >= 1, "rows for every thread");
  struct ScaleRows {
    const uint8_t* p[4];
  };
  __device__ __forceinline__ ScaleRows scale_rows(const TileAt& at) const {
    const ForwardArgs& a = args.f;
    const int F = GLU ? a.d_out / 2 : a.d_out;
    const int pitch = fp8_scale_row(a.d_in);
    const int unit = threadIdx.x % kUnits;
    ScaleRows s;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      s.p[q] = nullptr;
      if (unit < kUnitsA) {
        const int b = unit % kA * 4 + q, r = unit / (16 * kA) * WR + b * MI + unit / kA % 16;
        if (b < MB && r < at.rows) {
          const int64_t n = a.row_index != nullptr ? (int64_t)a.row_index[at.lo + r] : at.lo + r;
          if (n >= 0 && n < a.T) s.p[q] = args.xs + n * pitch;
        }
      } else {
        const int u = unit - kUnitsA;
        const int b = u % kB * 4 + q, r = u / (16 * kB) * WC + b * MI + u / kB % 16;
        const int64_t n = b < NB ? w_row(at, r, F) : -1;
        if (n >= 0)
          s.p[q] = args.ws + ((int64_t)at.e * scale_blocks(a.d_out) + n / kFp8Block) * pitch;
      }
    }
    return s;
  }
  // Those of K steps first .. first + kScaleSteps - 1, kBatch groups under way together.
  __device__ __forceinline__ void fill_scales(const ScaleRows& s, int first) const {
    constexpr int kGroups = kScaleSteps / 4, kBatch = 4;
    const int unit = threadIdx.x % kUnits, j0 = threadIdx.x / kUnits;
    if (j0 >= kSide) return;
    const int groups = (nk - first + 3) / 4;
    for (int j = j0; j < kGroups && j < groups; j += kSide * kBatch) {
      uint32_t w[kBatch][4];
#pragma unroll
      for (int c = 0; c < kBatch; ++c)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          w[c][q] = 0x7F7F7F7Fu;
          if (s.p[q] != nullptr && j + c * kSide < groups)
            w[c][q] = *reinterpret_cast<const uint32_t*>(s.p[q] + first + 4 * (j + c * kSide));
        }
#pragma unroll
      for (int c = 0; c < kBatch; ++c) {
        flip_bytes(w[c]);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (j + c * kSide < kGroups)
            *reinterpret_cast<LDS_AS uint32_t*>((LDS_AS char*)(uintptr_t)(
                scales + ((4 * (j + c * kSide) + q) * kUnits + unit) * 4)) = w[c][q];
      }
    }
  }
  __device__ __forceinline__ static uint32_t read_dword(uint32_t addr) {
    return *reinterpret_cast<LDS_AS const uint32_t*>((LDS_AS char*)(uintptr_t)addr);
  }

  struct Scales {
    uint32_t x[kA], w[kB];
  };
  __device__ __forceinline__ Scales read_scales(int k) const {
    const uint32_t at = k % kScaleSteps * (kUnits * 4);
    Scales s;
#pragma unroll
    for (int i = 0; i < kA; ++i) s.x[i] = read_dword(sa + at + 4 * i);
#pragma unroll
    for (int i = 0; i < kB; ++i) s.w[i] = read_dword(sb + at + 4 * i);
    return s;
  }

  __device__ __forceinline__ Frag frag(uint32_t base, int buf, int i) const {
    const uint32_t at = base + buf * kStage + i * MI * RB;
    return Frag{read_lds16(at + fs[0]), read_lds16(at + fs[1])};
  }

  // One K step, in four quarters of the products: a half of the A blocks by a half of
  // the B blocks.  Even steps take (a0 b0) (a0 b1) (a1 b1) (a1 b0), odd ones (a0 b1)
  // (a0 b0) (a1 b0) (a1 b1), so that each quarter lacks one half of the fragments, which has
  // been read in the quarter before into registers that were free:
  //   quarter 0   the other half of B, of this stage
  //   quarter 1   a1, of this stage; then nobody reads it any more
  //   quarter 2   a0, of the next stage
  //   quarter 3   the half of B that the next step starts with
  // LDS reads are as even over the step as that.  (All of a step's fragments in
  // registers at its start, the next ones read in its last row of products: the reads
  // of the four SIMDs then come at once, and 8192^3 took 911 thousand cycles.)
  // Between quarters 1 and 2 the barrier: this stage is free for the loads of step kt +
  // NS, which go out over the second half, and the next stage's loads are in LDS.
  static constexpr int N = MB * NB, Q = N / 4;
  static constexpr int MH = MB / 2, NH = NB / 2;
  // Loads of a step that are out before product i.
  __device__ __forceinline__ static constexpr int issued(int i) {
    return i <= N / 2 ? 0 : (i - N / 2) * kLoads / (N / 2);
  }
  // The product of a quarter behind which fragment f of n is read: early enough to
  // be back when the next quarter starts.
  __device__ __forceinline__ static constexpr int read_at(int f, int n) { return f * Q * 3 / 4 / n; }

  template <int ODD>
  __device__ __forceinline__ void round(int kt, int next, int S, Frag (&a_)[MB], Frag (&b_)[NB],
                                        Scales& sc, f32x4 (&acc)[MB][NB]) {
    const int SN = S + 1 == NS ? 0 : S + 1;
    Scales ahead;
    static_for<N>([&](auto i_) __attribute__((always_inline)) {
      constexpr int i = i_, q = i / Q, r = i % Q;
      constexpr int bh = (q == 1 || q == 2) != (ODD != 0);
      constexpr int a = (q >= 2 ? MH : 0) + r / NH, b = bh * NH + r % NH;
      if constexpr (i == N / 2) {
        wait_loads_barrier<(NS - 2) * kLoads>();
        __builtin_amdgcn_sched_barrier(0);
      }
      acc[a][b] = mfma<b % 4, a % 4>(b_[b], a_[a], acc[a][b], sc.w[b / 4], sc.x[a / 4]);
      static_for<(q == 1 || q == 2) ? MH : NH>([&](auto f_) __attribute__((always_inline)) {
        constexpr int f = f_;
        if constexpr (r == read_at(f, (q == 1 || q == 2) ? MH : NH)) {
          if constexpr (q == 0) b_[(1 - ODD) * NH + f] = frag(fb, S, (1 - ODD) * NH + f);
          if constexpr (q == 1) a_[MH + f] = frag(fa, S, MH + f);
          if constexpr (q == 2) a_[f] = frag(fa, SN, f);
          if constexpr (q == 3) b_[(1 - ODD) * NH + f] = frag(fb, SN, (1 - ODD) * NH + f);
        }
      });
      if constexpr (i == N / 2) ahead = read_scales(next);
      static_for<issued(i + 1) - issued(i)>([&](auto l) __attribute__((always_inline)) {
        issue(issued(i) + l, S, kt + NS);
      });
      __builtin_amdgcn_sched_barrier(0);
    });
    sc = ahead;
  }

  __device__ __forceinline__ void mainloop(const TileAt& at, f32x4 (&acc)[MB][NB]) {
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[a][b] = f32x4{};
    // the scales' loads beside the first stage's, which the products wait for as well
    const ScaleRows rows = scale_rows(at);
#pragma unroll
    for (int j = 0; j < kLoads; ++j) issue(j, 0, 0);
    fill_scales(rows, 0);
#pragma unroll
    for (int d = 1; d < NS; ++d)
#pragma unroll
      for (int j = 0; j < kLoads; ++j) issue(j, d, d);
    wait_loads_barrier<(NS - 1) * kLoads>();
    Frag a_[MB], b_[NB];
#pragma unroll
    for (int i = 0; i < MH; ++i) a_[i] = frag(fa, 0, i);
#pragma unroll
    for (int i = 0; i < NH; ++i) b_[i] = frag(fb, 0, i);
    Scales sc = read_scales(k0);
    int S = 0, k = k0;   // k: the K step of this turn
    for (int kt = 0;;) {
      const int end = nk - kt < kScaleSteps ? nk : kt + kScaleSteps;
      for (; kt + 1 < end; kt += 2) {
        k = k + 1 == nk ? 0 : k + 1;
        round<0>(kt, k, NS == 2 ? 0 : S, a_, b_, sc, acc);
        S = S + 1 == NS ? 0 : S + 1;
        k = k + 1 == nk ? 0 : k + 1;
        round<1>(kt + 1, k, NS == 2 ? 1 : S, a_, b_, sc, acc);
        S = S + 1 == NS ? 0 : S + 1;
      }
      if (kt < end) {   // the last one of an odd number
        round<0>(kt, 0, NS == 2 ? 0 : S, a_, b_, sc, acc);
        ++kt;
      }
      if (kt >= nk) break;
      // everybody has read the last of the old ones before the last step's barrier
      fill_scales(scale_rows(at), kt);
      __syncthreads();
      sc = read_scales(kt);
    }
    // nobody reads LDS any more, and nothing is on its way there
    wait_loads_barrier<0>();
  }

  // Epilogue from registers: 16 rows and 32 columns at a time, 64 bytes of a row; bias,
  // activation and residual in float32, one rounding.  It is straight-line code, which the
  // instruction cache has to take in for each tile: one activation's at a time.
  static constexpr int kOutBlocks = GLU ? NB / 2 : NB;
  static constexpr int CW = kOutBlocks % 2 == 0 ? 8 : 4;   // columns of a lane
  static constexpr int kPieces = kOutBlocks * 4 / CW;      // lanes' pieces of a row
  typedef std::conditional_t<CW == 8, vec4u, uint2> Piece;
  // Columns CW * g .. of piece p in lane group g, from block `first` of the results on.
  __device__ __forceinline__ static void columns(const f32x4 (&row)[NB], int first, int p,
                                                 float (&v)[CW]) {
    if constexpr (CW == 8) {
      eight_columns(row[first + 2 * p], row[first + 2 * p + 1], v);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = row[first + p][i];
    }
  }
  __device__ __forceinline__ static void add(float (&v)[CW], const Piece& w) {
    const uint32_t* d = reinterpret_cast<const uint32_t*>(&w);
#pragma unroll
    for (int j = 0; j < CW / 2; ++j) {
      v[2 * j] += __uint_as_float(d[j] << 16);
      v[2 * j + 1] += __uint_as_float(d[j] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ static Piece piece(const void* p, int64_t o) {
    return *reinterpret_cast<const Piece*>(static_cast<const uint16_t*>(p) + o);
  }
  __device__ __forceinline__ static void put(void* p, int64_t o, const float (&v)[CW]) {
    Piece w;
    uint32_t* d = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int j = 0; j < CW / 2; ++j) d[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
    *reinterpret_cast<Piece*>(static_cast<uint16_t*>(p) + o) = w;
  }

  __device__ __forceinline__ void epilogue(const TileAt& at, const f32x4 (&acc)[MB][NB]) const {
    if constexpr (GLU) return finish<LRMOE_ACT_SWIGLU>(at, acc);
    switch (args.f.act) {
      case LRMOE_ACT_RELU: return finish<LRMOE_ACT_RELU>(at, acc);
      case LRMOE_ACT_SILU: return finish<LRMOE_ACT_SILU>(at, acc);
      case LRMOE_ACT_GELU: return finish<LRMOE_ACT_GELU>(at, acc);
      default: return finish<LRMOE_ACT_NONE>(at, acc);
    }
  }
  template <int ACT>
  __device__ __forceinline__ void finish(const TileAt& at, const f32x4 (&acc)[MB][NB]) const {
    const ForwardArgs& a = args.f;
    const int F = GLU ? a.d_out / 2 : a.d_out;
    const int col = at.col * kOut + wn * kOutBlocks * MI + lane / MI * CW;
    const int64_t bias = (int64_t)at.e * a.d_out + col;
    static_for<MB>([&](auto i_) __attribute__((always_inline)) {
      constexpr int i = i_;
      const int r0 = wm * WR + i * MI;
      if (r0 >= at.rows) return;   // wave-uniform
      const bool row_ok = r0 + lane % MI < at.rows;
      const int64_t o = (at.lo + r0 + lane % MI) * F + col;
      Piece res[kPieces];
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
        if (a.residual != nullptr && row_ok && col + 4 * CW * p < F)
          res[p] = piece(a.residual, o + 4 * CW * p);
      static_for<kPieces>([&](auto p_) __attribute__((always_inline)) {
        constexpr int p = p_, c = 4 * CW * p;
        const bool ok = row_ok && col + c < F;
        float z[CW], v[CW];
        columns(acc[i], 0, p, z);
        if (a.bias != nullptr && ok) add(z, piece(a.bias, bias + c));
        if (a.pre_a != nullptr && ok) put(a.pre_a, o + c, z);
        if constexpr (GLU) {
          float w[CW];
          columns(acc[i], NB / 2, p, w);
          if (a.bias != nullptr && ok) add(w, piece(a.bias, bias + F + c));
          if (a.pre_b != nullptr && ok) put(a.pre_b, o + c, w);
#pragma unroll
          for (int j = 0; j < CW; ++j) v[j] = z[j] * sigmoid_f32(z[j]) * w[j];
        } else {
#pragma unroll
          for (int j = 0; j < CW; ++j) v[j] = z[j];
          activate(ACT, v);
        }
        if (a.residual != nullptr && ok) add(v, res[p]);
        if (ok) put(a.y, o + c, v);
      });
    });
  }
};

template <typename G>
__device__ __forceinline__ void run_tile(const Fp8Args& args, const TileAt& at,
                                         LDS_AS char* smem) {
  G g(args, at, smem);
  f32x4 acc[G::kMB][G::kNB];
  g.mainloop(at, acc);
  g.epilogue(at, acc);
}

template <typename G>
__global__ __launch_bounds__(G::kThreads, G::kWavesPerSimd) void gemm8_kernel(Fp8Args args,
                                                                              int cols) {
  __shared__ __attribute__((aligned(16))) char smem[G::kLds];
  TileAt at;
  if (!find_tile(args.f.seg, args.f.E, args.f.P, G::TM, cols, at)) return;
  run_tile<G>(args, at, (LDS_AS char*)smem);
}

// Tiles of 256 x 256 in four waves, one a SIMD: a wave of 128 x 128 reads half as much
// LDS as two of 64 x 128 do (8192^3 in turns: 435 us, 440 with eight waves; 32768 pairs,
// 2048 -> 1536: 148 and 158 us, 4096 -> 2816: 407 and 421 us).
template <bool GLU>
struct Ragged8 {
  typedef Gemm8<128, 128, 2, 2, 2, GLU> G256;
  typedef Gemm8<64, 128, 2, 2, 3, GLU> G128;
  typedef Gemm8<32, 128, 2, 2, 3, GLU> G64;
  static constexpr int kLds = std::max(std::max(G256::kLds, G128::kLds), G64::kLds);
  static constexpr int kThreads = G256::kThreads, kOut = G256::kOut;
};

template <bool GLU>
__global__ __launch_bounds__(256, 1) void ragged_gemm8_kernel(Fp8Args args, int cols) {
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
    static_for<4>([&](auto u_) __attribute__((always_inline)) {
      constexpr int u = u_;
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[c] = mfma<u, u>(w[u][c], x[u], acc[c], sw[c], sx);
    });
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
  return launch_workgroups(gemm8_kernel<G>, blocks, G::kThreads, s, a, cols);
}

template <bool GLU>
hipError_t launch_ragged(const Fp8Args& a, int F, hipStream_t s) {
  typedef Ragged8<GLU> R;
  const int cols = (F + R::kOut - 1) / R::kOut;
  const int64_t blocks = ragged_blocks(a.f, cols);
  return launch_workgroups(ragged_gemm8_kernel<GLU>, blocks, R::kThreads, s, a, cols);
}

template <int NC, bool GLU>
hipError_t launch_few_rows(const Fp8Args& a, int F, hipStream_t s) {
  constexpr int kOut = GLU ? NC * 8 : NC * 16;
  const int cols = (F + kOut - 1) / kOut;
  const int64_t blocks = grid_blocks(a.f.P, a.f.E, 16, cols);
  return launch_workgroups(few_rows8_kernel<NC, GLU>, blocks, 256, s, a, cols);
}

// The smallest tiles whose workgroups the CUs hold at once, as for bfloat16: below
// that a product takes the time of one workgroup's walk over K, which grows with the
// tile.  Measured (us; columns: without tiles, 32 x 64, 64 x 64, 64 x 128, 128 x 256,
// and 32 x 256 for few rows of much W):
//   1 row, 1 x 1536 x 2048 SwiGLU             5.3   8.8   8.3  10.1  18.0
//   64 rows, 1 x 4096 x 4096                 15.8  14.4  14.0  17.4  32.5
//   256 rows, 4 x 1536 x 2048 SwiGLU         12.0   9.7   9.5  11.5  21.0
//   2048 rows, 4 x 1536 x 2048 SwiGLU        74    28.9  19.5  16.4  22.2
//   8192 rows, 16 x 1536 x 2048 SwiGLU      275   108    63.5  49.5  45.9  (256 rows: 36.8)
//   512 rows, 16 x 2816 x 4096 SwiGLU        82    45.6  50.5  45.1  43.1  (32 x 256: 39.1)
//   128 rows, 16 x 2816 x 4096 SwiGLU        41.7  44.6  45.6  41.7  40.4  (32 x 256: 37.8)
template <bool GLU>
hipError_t forward(const Fp8Args& a, int F, bool far, hipStream_t s) {
  constexpr int h = GLU ? 2 : 1;   // W rows of an output column
  if (expected(a.f, F, 16, 32 / h) <= 320) return launch_few_rows<2, GLU>(a, F, s);
  if (far) return launch_gemm<Gemm8<32, 64, 2, 2, 3, GLU, true>>(a, F, s);   // 64-bit addresses
  if (a.f.P <= (int64_t)32 * a.f.E && expected(a.f, F, 32, 256 / h) >= 160)
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
