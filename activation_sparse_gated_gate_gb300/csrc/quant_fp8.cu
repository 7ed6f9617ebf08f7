// Quantisation to e4m3 with an fp32 scale for each block of 128.
//
// A block is 1 x 128 (activations, gradients) or 128 x 128 (weights):
//   scale = max(max |v|, 2^-64) / 448,   q = e4m3(v 448 / max(max |v|, 2^-64)).
// The transpose, when asked for, is quantised by its own blocks: 128 x 1 of
// the source for 1 x 128 blocks (the operand of a product that sums over the
// source's rows), the same 128 x 128 blocks otherwise.
//
// Bound by memory.  One CTA takes a tile of 128 x 128: thread (g, c) of
// 16 x 16 holds rows 8 g .. 8 g + 7 of columns 8 c .. 8 c + 7 in registers, so
// the source is read once for both outputs; a row's maximum is taken over the
// 16 lanes of a half-warp, a column's over the thread's rows and then the 16
// row groups through shared memory, and a thread already holds eight rows of
// a column, the eight bytes it puts into the transposed tile.
#include "common.cuh"
#include "vec.cuh"

namespace twell {
namespace {

struct QuantParams {
  const void* src;
  int64_t ld, ldq, ldqt;
  int32_t R, C;
  uint8_t* q;        // optional, with scale
  float* scale;
  uint8_t* qt;       // optional, with scale_t
  float* scale_t;
};

constexpr int kPitch = 144;   // bytes of a row of the transposed tile in shared memory

// VEC: 16-byte aligned source rows, C % 8 == 0 and 8-byte aligned rows of q.
// WIDE_T: rows of qt on 16-byte boundaries.
template <typename T, bool VEC, bool SQUARE>
__global__ void __launch_bounds__(256) quant_fp8_kernel(const QuantParams p, const bool wide_t) {
  __shared__ float colmax[16][128 + 4];
  __shared__ __align__(16) uint8_t tile[128 * kPitch];
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 128 + 8 * g;
  const int c0 = blockIdx.x * 128 + 8 * c;
  const int nc = p.C - c0;
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    if (r0 + i < p.R && nc > 0)
      load8<VEC>(static_cast<const T*>(p.src) + (r0 + i) * p.ld + c0, nc, v[i]);
  }
  const int64_t nbc = (p.C + 127) / 128, nbr = (p.R + 127) / 128;
  float inv_all = 0.0f;
  if (SQUARE) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, amax8(v[i]));
    m = half_warp_max(m);
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
    if ((threadIdx.x & 31) == 0) colmax[0][threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, colmax[0][i]);
    m = fmaxf(m, kFp8AmaxMin);
    inv_all = kFp8Max / m;
    if (threadIdx.x == 0) {
      if (p.scale) p.scale[blockIdx.y * nbc + blockIdx.x] = m / kFp8Max;
      if (p.scale_t) p.scale_t[blockIdx.x * nbr + blockIdx.y] = m / kFp8Max;
    }
  }
  if (p.q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float inv = inv_all;
      if (!SQUARE) {
        const float m = fmaxf(half_warp_max(amax8(v[i])), kFp8AmaxMin);
        inv = kFp8Max / m;
        if (c == 0 && r0 + i < p.R) p.scale[(r0 + i) * nbc + blockIdx.x] = m / kFp8Max;
      }
      if (r0 + i < p.R && nc > 0) store8_e4m3<VEC>(p.q + (r0 + i) * p.ldq + c0, nc, v[i], inv);
    }
  }
  if (!p.qt) return;
  float inv[8];
  if (SQUARE) {
#pragma unroll
    for (int j = 0; j < 8; ++j) inv[j] = inv_all;
  } else {
    float m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m[j] = fmaxf(m[j], fabsf(v[i][j]));
    }
    *reinterpret_cast<float4*>(&colmax[g][8 * c]) = make_float4(m[0], m[1], m[2], m[3]);
    *reinterpret_cast<float4*>(&colmax[g][8 * c + 4]) = make_float4(m[4], m[5], m[6], m[7]);
    __syncthreads();
    if (threadIdx.x < 128) {
      float a = kFp8AmaxMin;
#pragma unroll
      for (int i = 0; i < 16; ++i) a = fmaxf(a, colmax[i][threadIdx.x]);
      const int64_t col = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
      if (col < p.C) p.scale_t[col * nbr + blockIdx.y] = a / kFp8Max;
      colmax[0][threadIdx.x] = kFp8Max / a;   // this thread's own column
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) inv[j] = colmax[0][8 * c + j];
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<uint2*>(tile + (8 * c + j) * kPitch + 8 * g) =
        make_uint2(e4m3x4(v[0][j] * inv[j], v[1][j] * inv[j], v[2][j] * inv[j], v[3][j] * inv[j]),
                   e4m3x4(v[4][j] * inv[j], v[5][j] * inv[j], v[6][j] * inv[j], v[7][j] * inv[j]));
  __syncthreads();
  // rows of the transposed tile: 8 threads of 16 bytes each
  const int64_t rt = static_cast<int64_t>(blockIdx.y) * 128;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int col = (threadIdx.x >> 3) + 32 * i, b = (threadIdx.x & 7) * 16;
    const int64_t gc = static_cast<int64_t>(blockIdx.x) * 128 + col;
    if (gc >= p.C) continue;
    const uint8_t* s = tile + col * kPitch + b;
    uint8_t* d = p.qt + gc * p.ldqt + rt + b;
    const int64_t left = p.R - (rt + b);
    if (wide_t && left >= 16) {
      *reinterpret_cast<uint4*>(d) = *reinterpret_cast<const uint4*>(s);
    } else {
      for (int k = 0; k < 16 && k < left; ++k) d[k] = s[k];
    }
  }
}

template <typename T>
twell_status launch(const QuantParams& p, int32_t block_rows, bool vec, bool wide_t,
                    cudaStream_t s) {
  const dim3 grid((p.C + 127) / 128, (p.R + 127) / 128);
  if (block_rows == 1) {
    if (vec) quant_fp8_kernel<T, true, false><<<grid, 256, 0, s>>>(p, wide_t);
    else quant_fp8_kernel<T, false, false><<<grid, 256, 0, s>>>(p, wide_t);
  } else {
    if (vec) quant_fp8_kernel<T, true, true><<<grid, 256, 0, s>>>(p, wide_t);
    else quant_fp8_kernel<T, false, true><<<grid, 256, 0, s>>>(p, wide_t);
  }
  return cudaGetLastError() == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}

}  // namespace
}  // namespace twell

extern "C" twell_status twell_quant_fp8(const void* src, int32_t type, int64_t ld, int32_t R,
                                        int32_t C, int32_t block_rows, uint8_t* q, int64_t ldq,
                                        float* scale, uint8_t* qt, int64_t ldqt, float* scale_t,
                                        void* stream) {
  using namespace twell;
  if (R < 0 || C < 0 || (block_rows != 1 && block_rows != kFp8Block) ||
      (type != TWELL_BF16 && type != TWELL_F32))
    return TWELL_ERR_INVALID;
  if ((q != nullptr) != (scale != nullptr) || (qt != nullptr) != (scale_t != nullptr))
    return TWELL_ERR_INVALID;
  if (R == 0 || C == 0) return TWELL_OK;
  if (!src || (!q && !qt) || ld < C || (q && ldq < C) || (qt && ldqt < R))
    return TWELL_ERR_INVALID;
  const int elem = type == TWELL_BF16 ? 2 : 4;
  const uintptr_t a = reinterpret_cast<uintptr_t>(src);
  if (a % elem != 0 || reinterpret_cast<uintptr_t>(scale) % 4 != 0 ||
      reinterpret_cast<uintptr_t>(scale_t) % 4 != 0)
    return TWELL_ERR_INVALID;
  if ((static_cast<int64_t>(R) + 127) / 128 > 65535) return TWELL_ERR_UNSUPPORTED;  // grid rows
  DeviceInfo dev;
  twell_status st;
  if ((st = require_sm103(&dev)) != TWELL_OK) return st;
  const QuantParams p{src, ld, ldq, ldqt, R, C, q, scale, qt, scale_t};
  const bool vec = C % 8 == 0 && a % 16 == 0 && (ld * elem) % 16 == 0 &&
                   (!q || (reinterpret_cast<uintptr_t>(q) % 8 == 0 && ldq % 8 == 0));
  const bool wide_t = qt && aligned16(qt) && ldqt % 16 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return type == TWELL_BF16 ? launch<uint16_t>(p, block_rows, vec, wide_t, s)
                            : launch<float>(p, block_rows, vec, wide_t, s);
}
