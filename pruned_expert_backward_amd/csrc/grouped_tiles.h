// What the grouped products share, whatever they multiply: the search for a
// workgroup's tile, moves from global memory to LDS, and the end of the few-rows form.
#pragma once

#include <algorithm>
#include <type_traits>
#include <utility>

#include "forward.h"

namespace lrmoe {
namespace {

#define LDS_AS __attribute__((address_space(3)))

typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ const vec4u zero_page[16] = {};

// One (uniform) branch for N values.
template <int N>
__device__ __forceinline__ void activate(int act, float (&v)[N]) {
  switch (act) {
    case LRMOE_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];   // NaN stays
      break;
    case LRMOE_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] *= sigmoid_f32(v[i]);
      break;
    case LRMOE_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = gelu_f32(v[i]);
      break;
  }
}

// ---------------------------------------------------------------- tiles
// Row tiles that take their turns at each column tile together, and so share
// its panel of W in the L2 (32768 pairs, 768 -> 2048: 129 us, 131 with 2, 135 with
// 8; 8192^3: 807, 843 and 805 us).
constexpr int kGroup = 4;

struct TileAt {
  int e;
  int64_t lo;    // first pair row of the tile
  int rows;      // rows of the tile (at least 1)
  int col;       // column tile
};

constexpr int kXcds = 8, kXcdCus = 32;

// A launch of any number of workgroups: a dimension of a grid has less than 2^32
// threads, so its workgroups go by rows of 2^22, whole turns of the XCDs.  This
// workgroup's number among those of its XCD, which is blockIdx.x % kXcds.
constexpr int kGridRow = 22, kGridRows = 1 << 13;   // numbers of 32 bits
__device__ __forceinline__ uint32_t number_on_xcd() {
  return blockIdx.y * ((1u << kGridRow) / kXcds) + blockIdx.x / kXcds;
}

// Tile of this workgroup, or false.  Workgroup b runs on XCD b % 8, so each
// XCD takes a contiguous eighth of the tiles; inside it, kGroup row tiles go
// column by column.  Each wave finds the tile for itself: lane l counts the
// tiles of experts 4 l .. 4 l + 3.
__device__ __forceinline__ bool find_tile(const int32_t* seg, int E, int64_t P, int tm, int cols,
                                          TileAt& at) {
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
  const int end = wave_scan(sum);
  const int all = __builtin_amdgcn_readlane(end, 63);
  const int64_t total = (int64_t)all * cols;
  const int64_t share = (total + 7) / 8;
  const int64_t pos = number_on_xcd();
  const int64_t t = (int64_t)(blockIdx.x % kXcds) * share + pos;
  if (pos >= share || t >= total) return false;
  const int64_t per = (int64_t)kGroup * cols;
  const int g = (int)(t / per);
  const int in = (int)(t - g * per);
  const int left = all - g * kGroup;
  const int gr = left < kGroup ? left : kGroup;
  const int r = __builtin_amdgcn_readfirstlane(g * kGroup + in % gr);
  at.col = __builtin_amdgcn_readfirstlane(in / gr);
  const unsigned long long past = __ballot(end > r);
  if (past == 0) return false;
  const int owner = __ffsll(past) - 1;
  int sub = r - (end - sum), j = 0;   // meant for the owner lane
  const bool sane = sub >= 0;         // offsets out of order may overflow the counts
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (j == i && sub >= n[i]) {
      sub -= n[i];
      j = i + 1;
    }
  const int64_t lo = (j == 0 ? off[0] : j == 1 ? off[1] : j == 2 ? off[2] : off[3]) +
                     (int64_t)sub * tm;
  const int64_t hi = j == 0 ? off[1] : j == 1 ? off[2] : j == 2 ? off[3] : off[4];
  const int rows = sane ? (int)(hi - lo < tm ? hi - lo : tm) : 0;
  at.e = __builtin_amdgcn_readlane(4 * lane + j, owner);
  const uint32_t lo32 = __builtin_amdgcn_readlane((uint32_t)lo, owner);   // P < 2^31
  at.lo = lo32;
  at.rows = __builtin_amdgcn_readlane(rows, owner);
  return at.rows > 0;
}

// Tile of this workgroup, or false (behind the last one, or a piece of a cut tile
// without rows).
__device__ __forceinline__ bool find_ragged_tile(const int32_t* seg, int E, int64_t P, int cols,
                                                 TileAt& at) {
  const int lane = threadIdx.x & 63;
  int64_t off[5];
#pragma unroll
  for (int j = 0; j < 5; ++j) {
    const int e = 4 * lane + j;
    const int64_t o = seg[e < E ? e : E];
    off[j] = o < 0 ? 0 : o > P ? P : o;
  }
  // One round of 128-row tiles reads W at the rate of memory and ends sooner
  // than 256-row tiles on part of the CUs; else 256-row tiles.
  int halves = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (off[j + 1] > off[j]) halves += (int)((off[j + 1] - off[j] + 127) / 128);
  halves = __builtin_amdgcn_readlane(wave_scan(halves), 63);
  const int tm = (int64_t)halves * cols <= kXcds * kXcdCus ? 128 : 256;
  int n[4], full = 0, part = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    n[j] = off[j + 1] > off[j] ? (int)(off[j + 1] - off[j]) : 0;
    full += n[j] / tm;
    part += n[j] % tm != 0;
  }
  // whole tiles and ends up to this lane's experts
  const int fend = wave_scan(full), pend = wave_scan(part);
  const int fulls = __builtin_amdgcn_readlane(fend, 63);
  const int parts = __builtin_amdgcn_readlane(pend, 63);
  const int x = blockIdx.x % kXcds;
  const int64_t pos = number_on_xcd();
  const int64_t ft = (int64_t)fulls * cols, pt = (int64_t)parts * cols;
  const int64_t f0 = ft * x / kXcds, f1 = ft * (x + 1) / kXcds;   // this XCD's share
  const int64_t p0 = pt * x / kXcds, p1 = pt * (x + 1) / kXcds;
  const int64_t mine = f1 - f0 + p1 - p0;
  const int64_t rounds = mine / kXcdCus * kXcdCus;
  const int rem = (int)(mine - rounds);
  int64_t tile = pos;
  int piece = 0, cut = 1;
  if (pos >= rounds) {
    cut = rem * 4 <= kXcdCus ? 4 : rem * 2 <= kXcdCus ? 2 : 1;
    if (pos - rounds >= (int64_t)rem * cut) return false;
    const int q = (int)(pos - rounds);
    tile = rounds + q / cut;
    piece = q % cut;
  }
  const bool whole = tile < f1 - f0;
  int r;   // row tile in its list
  if (whole) {
    const int64_t t = f0 + tile, per = (int64_t)kGroup * cols;
    const int g = (int)(t / per), in = (int)(t - g * per);
    const int left = fulls - g * kGroup, gr = left < kGroup ? left : kGroup;
    r = g * kGroup + in % gr;
    at.col = in / gr;
  } else {
    const int64_t t = p0 + tile - (f1 - f0);
    r = (int)(t / cols);
    at.col = (int)(t - (int64_t)r * cols);
  }
  r = __builtin_amdgcn_readfirstlane(r);
  at.col = __builtin_amdgcn_readfirstlane(at.col);
  const unsigned long long past = whole ? __ballot(fend > r) : __ballot(pend > r);
  if (past == 0) return false;   // offsets out of order
  const int owner = __ffsll(past) - 1;
  int sub = whole ? r - (fend - full) : r - (pend - part), j = 0;   // meant for the owner lane
  const bool sane = sub >= 0;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int c = whole ? n[i] / tm : (int)(n[i] % tm != 0);
    if (j == i && sub >= c) {
      sub -= c;
      j = i + 1;
    }
  }
  const int nj = j == 0 ? n[0] : j == 1 ? n[1] : j == 2 ? n[2] : n[3];
  const int64_t oj = j == 0 ? off[0] : j == 1 ? off[1] : j == 2 ? off[2] : off[3];
  const int first = (whole ? sub : nj / tm) * tm + piece * (tm / cut);
  int rows = nj - first;
  if (rows > tm / cut) rows = tm / cut;
  if (!sane) rows = 0;
  at.e = __builtin_amdgcn_readlane(4 * lane + j, owner);
  at.lo = (uint32_t)__builtin_amdgcn_readlane((uint32_t)(oj + first), owner);   // P < 2^31
  at.rows = __builtin_amdgcn_readlane(rows, owner);
  return at.rows > 0;
}

// ---- global -> LDS, 16 bytes a lane: lane i writes LDS bytes [lds + 16 i,
// lds + 16 i + 16).  Inline asm without outputs: the compiler then does not
// wait for it before LDS reads of other stages; the explicit waits below
// order the stages.  The buffer form reads zeros past its range.
constexpr uint32_t kBufferFlags = 0x00020000u;   // gfx9 family: raw 32-bit data
constexpr uint32_t kOutOfRange = 0x80000000u;    // offset that is never in range
constexpr int64_t kNearBytes = int64_t(1) << 31; // what one buffer reaches
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0,
                                           (int)(bytes > 0x7FFFFFFF ? 0x7FFFFFFF : bytes),
                                           (int)kBufferFlags);
}
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds16(uint32_t lds, const char* p) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds),
               "v"(p)
               : "memory", "m0");
}
__device__ __forceinline__ void load_lds16(uint32_t lds, __amdgpu_buffer_rsrc_t r, uint32_t voff,
                                           uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds),
               "v"(voff), "s"(r), "s"(soff)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// f(0), f(1), ... f(N - 1), each with its index as a compile-time constant.
template <typename F, int... I>
__device__ __forceinline__ void static_for_(F& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_(f, std::make_integer_sequence<int, N>());
}

template <int N>
__device__ __forceinline__ void wait_loads_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

__device__ __forceinline__ vec4u read_lds16(uint32_t addr) {
  return *reinterpret_cast<LDS_AS const vec4u*>((LDS_AS char*)(uintptr_t)addr);
}

// Epilogue of 16 rows whose sums over K lie in four parts (256 threads).
template <typename O, int NC, bool GLU>
__device__ __forceinline__ void few_rows_epilogue(const ForwardArgs& args, const TileAt& at,
                                                  const float (&part)[4][16][NC * 16 + 4]) {
  constexpr int kOut = GLU ? NC * 8 : NC * 16;
  const int F = GLU ? args.d_out / 2 : args.d_out;
  const O* bias = static_cast<const O*>(args.bias);
  O* y = static_cast<O*>(args.y);
  auto put = [](void* p, int64_t o, float v) {
    if constexpr (sizeof(O) == 2) static_cast<uint16_t*>(p)[o] = f32_to_bf16(v);
    else static_cast<float*>(p)[o] = v;
  };
  auto get = [](const void* p, int64_t o) {
    if constexpr (sizeof(O) == 2) return bf16_to_f32(static_cast<const uint16_t*>(p)[o]);
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
      float one[1] = {z};
      activate(args.act, one);
      v = one[0];
    }
    if (args.residual != nullptr) v += get(args.residual, o);
    put(y, o, v);
  }
}

// ---------------------------------------------------------------- launch
// `kernel` in as many workgroups.
template <typename... A>
hipError_t launch_workgroups(void (*kernel)(A...), int64_t blocks, int threads, hipStream_t s,
                             const A&... args) {
  const int64_t row = int64_t(1) << kGridRow, rows = (blocks + row - 1) / row;
  if (rows > kGridRows) return hipErrorInvalidValue;   // 2^35: no memory holds their tiles
  hipLaunchKernelGGL(kernel, dim3((uint32_t)std::min(blocks, row), (uint32_t)rows), dim3(threads),
                     0, s, args...);
  return hipGetLastError();
}

int64_t grid_blocks(int64_t P, int E, int tm, int64_t cols) {
  const int64_t tiles = P / tm + (P < E ? P : E);   // most row tiles of P rows over E experts
  return (tiles * cols + 7) / 8 * 8;
}

// Workgroups of find_ragged_tile: the most tiles of an XCD, its share of the whole
// tiles and of the ends, and the parts of a cut round.
int64_t ragged_blocks(const ForwardArgs& a, int cols) {
  const int64_t ends = a.P < a.E ? a.P : a.E;
  return (a.P / 256 * cols / kXcds + ends * cols / kXcds + 2 + kXcdCus) * kXcds;
}

// Workgroups that a call is expected to have with tiles of tm rows and `out`
// columns: the segments live on the device, so half of the experts are taken
// to end in a tile of their own.
int64_t expected(const ForwardArgs& a, int F, int tm, int out) {
  const int64_t ends = a.P < a.E ? a.P : a.E;
  const int64_t tiles = std::max(ends, a.P / tm + ends / 2);
  return tiles * ((F + out - 1) / out);
}

}  // namespace
}  // namespace lrmoe
