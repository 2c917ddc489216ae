// Rows and weights to 8-bit blocks (fp8.h):
//
//   rows     blocks of 1 x 128: s = 2^e, e the smallest with max |x| <= 448 * 2^e,
//            q = e4m3(x / s)
//   weights  blocks of 128 x 128, and the same values transposed: a block is its own
//            transpose's block, so the gradient's product reads exactly the weights
//            that the forward product has read
//
// Memory bound: every value is read once and written once (twice with the
// transpose), 2 or 4 bytes in and 1 out.  The kernels' own times: 8191 x 4096 float32
// rows (168 MB) 30.4 us, 5.5 TB/s; 16 x 1536 x 2048 bfloat16 weights in both orders (201
// MB) 41.1 us, 4.9 TB/s.  bfloat16 rows stay below that: 32768 x 1536 35.4 us (4.3 TB/s),
// 8192 x 4096 27.2 (3.7), 8192 x 2048 15.2 (3.3), 501 x 4096 6.3; a lane has four 16-byte
// loads under way where a float32 one has eight, and stores 8 bytes at a time.
#include <algorithm>

#include "forward.h"
#include "fp8.h"

namespace lrmoe {
namespace {

// ---- rows: 16 lanes a block, 8 values a lane
constexpr int kPasses = 4;                  // blocks of a group of 16 lanes
constexpr int kPerGroup = 16 * kPasses;     // blocks of a workgroup

template <typename T>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const T* x, int64_t rows, int D,
                                                            int blocks, int pitch, uint8_t* q,
                                                            uint8_t* scale) {
  const int64_t first = (int64_t)blockIdx.x * kPerGroup;   // block number over all rows
  const int64_t r0 = first / blocks;
  const uint32_t b0 = (uint32_t)(first - r0 * blocks);
  const int lane = threadIdx.x & 15, group = threadIdx.x >> 4;
  float v[kPasses][8];
  int64_t at[kPasses];
  int blk[kPasses];
  int64_t row[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const uint32_t n = b0 + i * 16 + group;
    row[i] = r0 + n / (uint32_t)blocks;
    blk[i] = (int)(n % (uint32_t)blocks);
    const int c = blk[i] * kFp8Block + lane * 8;
    const bool in = row[i] < rows && c < D;
    at[i] = in ? row[i] * D + c : -1;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    if (in) load_vals(x + at[i], v[i]);
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = umax(top, finite_bits(v[i][j]));
    const uint32_t byte = fp8_scale_byte(row16_max(top));
    const float inv = fp8_inverse(byte);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = fp8_scaled(v[i][j], inv);
    if (at[i] >= 0)
      *reinterpret_cast<uint2*>(q + at[i]) =
          make_uint2(fp8_pack4(v[i][0], v[i][1], v[i][2], v[i][3]),
                     fp8_pack4(v[i][4], v[i][5], v[i][6], v[i][7]));
    if (row[i] < rows) {
      uint8_t* s = scale + row[i] * pitch + blk[i];
      if (lane == 0) *s = (uint8_t)byte;
      // the row's padding, up to three bytes, by its last block's lanes
      if (blk[i] == blocks - 1 && lane >= 1 && lane < pitch - blocks + 1) s[lane] = 127;
    }
  }
}

// ---- weights: a workgroup a block, a patch of 8 x 8 a thread
// LDS row of the transposed block.  Four of sixteen patches share a bank; that hides
// behind the memory traffic (the kernel takes 40.7 us where a copy would take 39).
constexpr int kPitch = kFp8Block + 8;

template <typename T>
__global__ __launch_bounds__(256) void quantize_weights_kernel(const T* W, int N, int K,
                                                               uint8_t* q, uint8_t* scale,
                                                               uint8_t* qt, uint8_t* scale_t) {
  __shared__ uint32_t tops[4];
  __shared__ __attribute__((aligned(16))) uint8_t flip[kFp8Block * kPitch];
  const int bk = blockIdx.x, bn = blockIdx.y;
  const int64_t e = blockIdx.z;
  const int pk = threadIdx.x & 15, pn = threadIdx.x >> 4;
  const int n0 = bn * kFp8Block + pn * 8, k0 = bk * kFp8Block + pk * 8;
  float v[8][8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    if (n0 + i < N && k0 < K) load_vals(W + (e * N + n0 + i) * K + k0, v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) top = umax(top, finite_bits(v[i][j]));
  }
  top = row16_max(top);
  top = umax(umax(__builtin_amdgcn_readlane(top, 0), __builtin_amdgcn_readlane(top, 16)),
             umax(__builtin_amdgcn_readlane(top, 32), __builtin_amdgcn_readlane(top, 48)));
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
  const uint32_t byte = fp8_scale_byte(umax(umax(tops[0], tops[1]), umax(tops[2], tops[3])));
  const float inv = fp8_inverse(byte);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = fp8_scaled(v[i][j], inv);
    if (n0 + i < N && k0 < K)
      *reinterpret_cast<uint2*>(q + (e * N + n0 + i) * K + k0) =
          make_uint2(fp8_pack4(v[i][0], v[i][1], v[i][2], v[i][3]),
                     fp8_pack4(v[i][4], v[i][5], v[i][6], v[i][7]));
  }
  // scales; the padding of a row of scales by its last block
  const int kb = gridDim.x, nb = gridDim.y;
  const int pitch = fp8_scale_row(K), pitch_t = fp8_scale_row(N);
  if (threadIdx.x < 4) {
    const int t = threadIdx.x;
    if (t == 0 || (bk == kb - 1 && bk + t < pitch))
      scale[(e * nb + bn) * pitch + bk + t] = t == 0 ? (uint8_t)byte : 127;
    if (scale_t != nullptr && (t == 0 || (bn == nb - 1 && bn + t < pitch_t)))
      scale_t[(e * kb + bk) * pitch_t + bn + t] = t == 0 ? (uint8_t)byte : 127;
  }
  if (qt == nullptr) return;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<uint2*>(flip + (pk * 8 + j) * kPitch + pn * 8) =
        make_uint2(fp8_pack4(v[0][j], v[1][j], v[2][j], v[3][j]),
                   fp8_pack4(v[4][j], v[5][j], v[6][j], v[7][j]));
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int k = pn + 16 * i, n = bn * kFp8Block + pk * 8;
    if (bk * kFp8Block + k < K && n < N)
      *reinterpret_cast<uint2*>(qt + (e * K + bk * kFp8Block + k) * N + n) =
          *reinterpret_cast<const uint2*>(flip + k * kPitch + pk * 8);
  }
}

template <typename T>
hipError_t quantize_rows(const void* x, int64_t rows, int D, uint8_t* q, uint8_t* scale,
                         hipStream_t s) {
  const int blocks = (D + kFp8Block - 1) / kFp8Block;
  // a grid has less than 2^32 threads: 2^30 blocks and more take several launches, of
  // whole rows each
  const int64_t most = ((int64_t(1) << 24) - 1) * kPerGroup / blocks;
  const int pitch = fp8_scale_row(D);
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t n = std::min(most, rows - r);
    hipLaunchKernelGGL(quantize_rows_kernel<T>,
                       dim3((uint32_t)((n * blocks + kPerGroup - 1) / kPerGroup)), dim3(256), 0, s,
                       static_cast<const T*>(x) + r * D, n, D, blocks, pitch, q + r * D,
                       scale + r * pitch);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_fp8_quantize(int dtype, const void* x, int64_t rows, int32_t D, uint8_t* q,
                               uint8_t* scale, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  return dtype == LRMOE_BF16 ? quantize_rows<uint16_t>(x, rows, D, q, scale, s)
                             : quantize_rows<float>(x, rows, D, q, scale, s);
}

hipError_t launch_fp8_quantize_weights(int dtype, const void* W, int32_t E, int32_t N, int32_t K,
                                       uint8_t* q, uint8_t* scale, uint8_t* qt, uint8_t* scale_t,
                                       hipStream_t s) {
  const dim3 grid((K + kFp8Block - 1) / kFp8Block, (N + kFp8Block - 1) / kFp8Block, E);
  if (dtype == LRMOE_BF16)
    hipLaunchKernelGGL(quantize_weights_kernel<uint16_t>, grid, dim3(256), 0, s,
                       static_cast<const uint16_t*>(W), N, K, q, scale, qt, scale_t);
  else
    hipLaunchKernelGGL(quantize_weights_kernel<float>, grid, dim3(256), 0, s,
                       static_cast<const float*>(W), N, K, q, scale, qt, scale_t);
  return hipGetLastError();
}

}  // namespace lrmoe
