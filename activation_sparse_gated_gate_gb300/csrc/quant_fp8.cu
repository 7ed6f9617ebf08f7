// Quantisation to e4m3 with an fp32 scale for each block of 128.
//
// A block is 1 x 128 (activations, gradients) or 128 x 128 (weights):
//   scale = max(max |v|, 2^-64) / 448,   q = e4m3(v 448 / max(max |v|, 2^-64)).
// The transpose, when asked for, is quantised by its own blocks: 128 x 1 of
// the source for 1 x 128 blocks (the operand of a product that sums over the
// source's rows), the same 128 x 128 blocks otherwise.
//
// Bound by memory.  One CTA takes a tile of 128 columns by 128 rows (16 x 16
// threads, thread (g, c) holding rows 8 g .. 8 g + 7 of columns 8 c .. 8 c + 7) so
// that the source is read once for both outputs; a row's maximum is taken over
// the 16 lanes of a half-warp, a column's over the thread's rows and then the 16
// row groups through shared memory, and a thread already holds eight rows of a
// column, the eight bytes it puts into the transposed tile.  bf16 stays packed
// in registers until it is scaled (64 values in 32 registers: 4 CTAs per SM).
// Without the transpose there is no shared memory and a thread holds two rows,
// so that more of them are in flight.  Measured: 8192 x 2048 bf16 9.5 us (5.3 TB/s),
// 16384 x 2304 both ways 26.6 (5.8 TB/s; issue slots 57 % busy).
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

// Eight values of a row as they were loaded: neighbours, or every 16th (vec.cuh).
template <typename T>
struct Piece;

template <>
struct Piece<float> {
  float v[8];
  typedef float Max;  // largest |v| so far of one column
  static constexpr int MAXES = 8;
  template <bool VEC>
  __device__ __forceinline__ void load(const float* p, int n) {
    load8<VEC, 16>(p, n, v);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  }
  __device__ __forceinline__ float get(int j) const { return v[j]; }
  __device__ __forceinline__ float amax() const { return amax8(v); }
  __device__ __forceinline__ void fold(Max (&m)[MAXES]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = fmaxf(m[j], fabsf(v[j]));
  }
  static __device__ __forceinline__ float max_of(const Max (&m)[MAXES], int j) { return m[j]; }
};

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));  // of a number and a NaN: the number
  return r;
}

template <>
struct Piece<uint16_t> {
  uint32_t v[4];
  typedef uint32_t Max;  // of two columns
  static constexpr int MAXES = 4;
  template <bool VEC>
  __device__ __forceinline__ void load(const uint16_t* p, int n) {
    if (VEC) {
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[k] = (32 * k < n ? p[32 * k] : 0u) |
               (32 * k + 16 < n ? static_cast<uint32_t>(p[32 * k + 16]) << 16 : 0u);
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = 0u;
  }
  __device__ __forceinline__ float get(int j) const {
    return __uint_as_float(j & 1 ? v[j / 2] & 0xffff0000u : v[j / 2] << 16);
  }
  __device__ __forceinline__ float amax() const {
    Max m = 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) m = max_bf16x2(m, v[k] & 0x7fff7fffu);
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
  __device__ __forceinline__ void fold(Max (&m)[MAXES]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = max_bf16x2(m[k], v[k] & 0x7fff7fffu);
  }
  static __device__ __forceinline__ float max_of(const Max (&m)[MAXES], int j) {
    return __uint_as_float(j & 1 ? m[j / 2] & 0xffff0000u : m[j / 2] << 16);
  }
};

// The maxima of ROWS rows over the 16 lanes of a half-warp: the lanes halve the
// rows between them as long as there are several (ROWS - 1 shuffles, then one
// for each step left, where a butterfly for each row would take four).  Lane c
// ends with the maximum of row c / (16 / ROWS).
template <int ROWS>
__device__ __forceinline__ float rows_max(float (&m)[ROWS], int c) {
  int o = 8;
#pragma unroll
  for (int n = ROWS / 2; n > 0; n /= 2, o /= 2) {
    const bool upper = (c & o) != 0;
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const float away = upper ? m[k] : m[k + n];
      const float mine = upper ? m[k + n] : m[k];
      m[k] = fmaxf(mine, __shfl_xor_sync(0xffffffffu, away, o));
    }
  }
  for (; o > 0; o /= 2) m[0] = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
  return m[0];
}

// e4m3 of four values times their scales.
__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d, float inv) {
  return e4m3x4(a * inv, b * inv, c * inv, d * inv);
}

// VEC: 16-byte aligned source rows, C % 8 == 0 and 8-byte aligned rows of q.
// SQUARE: blocks of 128 x 128 (else 1 x 128).  TRANS: qt is written; with
// neither a thread holds two rows of a tile of 32.  wide_t: rows of qt on
// 16-byte boundaries.
template <typename T, bool VEC, bool SQUARE, bool TRANS>
__global__ void __launch_bounds__(256) quant_fp8_kernel(const QuantParams p, const bool wide_t) {
  constexpr int ROWS = SQUARE || TRANS ? 8 : 2;
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4;
  // (unsigned: a size within 127 of 2^31 rounds up past it)
  const int64_t nbc = (static_cast<uint32_t>(p.C) + 127u) / 128u,
                nbr = (static_cast<uint32_t>(p.R) + 127u) / 128u;
  const int bx = blockIdx.x % static_cast<unsigned>(nbc);  // the tile's columns and rows
  const int64_t by = blockIdx.x / static_cast<unsigned>(nbc);
  const int64_t r0 = (by * 16 + g) * ROWS;
  const int c0 = bx * 128 + (VEC ? 8 * c : c);
  const int nc = p.C - c0;
  Piece<T> v[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    if (r0 + i < p.R && nc > 0)
      v[i].template load<VEC>(static_cast<const T*>(p.src) + (r0 + i) * p.ld + c0, nc);
    else v[i].clear();
  }
  float inv_all = 0.0f;
  if constexpr (SQUARE) {
    __shared__ float wmax[8];
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) m = fmaxf(m, v[i].amax());
    m = half_warp_max(m);
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
    if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, wmax[i]);
    m = fmaxf(m, kFp8AmaxMin);
    inv_all = kFp8Max / m;
    if (threadIdx.x == 0) {
      if (p.scale) p.scale[by * nbc + bx] = m / kFp8Max;
      if (p.scale_t) p.scale_t[bx * nbr + by] = m / kFp8Max;
    }
  }
  if (p.q) {
    constexpr int SHARE = 16 / ROWS;  // lanes that end with the same row's maximum
    float inv_row = 0.0f;             // of row c / SHARE
    if (!SQUARE) {
      float m[ROWS];
#pragma unroll
      for (int i = 0; i < ROWS; ++i) m[i] = v[i].amax();
      const float a = fmaxf(rows_max(m, c), kFp8AmaxMin);
      inv_row = kFp8Max / a;
      const int64_t r = r0 + c / SHARE;
      if (c % SHARE == 0 && r < p.R) p.scale[r * nbc + bx] = a / kFp8Max;
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const float inv =
          SQUARE ? inv_all : __shfl_sync(0xffffffffu, inv_row, i * SHARE, 16);
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = v[i].get(j);
      uint8_t* to = p.q + (r0 + i) * p.ldq + c0;
      if constexpr (VEC) {
        if (r0 + i < p.R && nc > 0) store8_e4m3(to, f, inv);
      } else {
        store8_e4m3_lanes<16>(to, nc, r0 + i < p.R, f, inv, inv);
      }
    }
  }
  if constexpr (TRANS) {
    // the transposed tile: row = column of the source, 16 units of 8 bytes (one
    // per row group), unit u of row r at u ^ (r / 8): with VEC the 16 lanes of a
    // half-warp write one unit of 16 rows without bank conflicts
    const auto column = [&](int j) { return VEC ? 8 * c + j : 16 * j + c; };  // of value j
    __shared__ __align__(16) uint2 tile[128][16];
    float inv[8];
    if constexpr (SQUARE) {
#pragma unroll
      for (int j = 0; j < 8; ++j) inv[j] = inv_all;
    } else {
      typedef typename Piece<T>::Max Max;
      constexpr int MAXES = Piece<T>::MAXES;
      __shared__ __align__(16) Max colmax[16][16 * MAXES];
      __shared__ float colinv[128];
      Max m[MAXES];
#pragma unroll
      for (int k = 0; k < MAXES; ++k) m[k] = 0;
#pragma unroll
      for (int i = 0; i < ROWS; ++i) v[i].fold(m);
#pragma unroll
      for (int k = 0; k < MAXES; k += 4)
        *reinterpret_cast<uint4*>(&colmax[g][MAXES * c + k]) =
            *reinterpret_cast<const uint4*>(&m[k]);
      __syncthreads();
      if (threadIdx.x < 128) {
        constexpr int PER = 8 / MAXES;  // columns of a Max
        // the lane and the value that hold this thread's column
        const int cc = VEC ? threadIdx.x / 8 : threadIdx.x % 16;
        const int jj = VEC ? threadIdx.x % 8 : threadIdx.x / 16;
        float a = kFp8AmaxMin;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          Max m1[MAXES];
          m1[0] = colmax[i][MAXES * cc + jj / PER];
          a = fmaxf(a, Piece<T>::max_of(m1, jj % PER));
        }
        const int64_t col = static_cast<int64_t>(bx) * 128 + threadIdx.x;
        if (col < p.C) p.scale_t[col * nbr + by] = a / kFp8Max;
        colinv[threadIdx.x] = kFp8Max / a;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) inv[j] = colinv[column(j)];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      tile[column(j)][g ^ (column(j) >> 3)] =
          make_uint2(quant4(v[0].get(j), v[1].get(j), v[2].get(j), v[3].get(j), inv[j]),
                     quant4(v[4].get(j), v[5].get(j), v[6].get(j), v[7].get(j), inv[j]));
    __syncthreads();
    // rows of the transposed tile: 8 threads of 16 bytes (two units) each
    const int64_t rt = by * 128;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = (threadIdx.x >> 3) + 32 * i, b = threadIdx.x & 7;
      const int64_t gc = static_cast<int64_t>(bx) * 128 + row;
      if (gc >= p.C) continue;
      const int x = row >> 3, odd = row & 1;  // (odd rows take their units in the other order)
      const uint2 u0 = tile[row][(2 * b + odd) ^ x], u1 = tile[row][(2 * b + 1 - odd) ^ x];
      const uint4 w = odd ? make_uint4(u1.x, u1.y, u0.x, u0.y) : make_uint4(u0.x, u0.y, u1.x, u1.y);
      uint8_t* d = p.qt + gc * p.ldqt + rt + 16 * b;
      const int64_t left = p.R - (rt + 16 * b);
      if (wide_t && left >= 16) {
        *reinterpret_cast<uint4*>(d) = w;
      } else {
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (k < left) d[k] = static_cast<uint8_t>(ww[k / 4] >> (8 * (k % 4)));
      }
    }
  }
}

template <typename T, bool VEC>
twell_status launch(const QuantParams& p, int32_t block_rows, bool wide_t, cudaStream_t s) {
  const bool square = block_rows != 1, trans = p.qt != nullptr;
  const int rows = square || trans ? 128 : 32;
  const int64_t tiles =
      (static_cast<int64_t>(p.C) + 127) / 128 * ((static_cast<int64_t>(p.R) + rows - 1) / rows);
  if (tiles > 0x7fffffff) return TWELL_ERR_UNSUPPORTED;
  const unsigned grid = static_cast<unsigned>(tiles);
  if (square && trans) quant_fp8_kernel<T, VEC, true, true><<<grid, 256, 0, s>>>(p, wide_t);
  else if (square) quant_fp8_kernel<T, VEC, true, false><<<grid, 256, 0, s>>>(p, wide_t);
  else if (trans) quant_fp8_kernel<T, VEC, false, true><<<grid, 256, 0, s>>>(p, wide_t);
  else quant_fp8_kernel<T, VEC, false, false><<<grid, 256, 0, s>>>(p, wide_t);
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
  DeviceInfo dev;
  twell_status st;
  if ((st = require_sm103(&dev)) != TWELL_OK) return st;
  const QuantParams p{src, ld, ldq, ldqt, R, C, q, scale, qt, scale_t};
  const bool vec = C % 8 == 0 && a % 16 == 0 && (ld * elem) % 16 == 0 &&
                   (!q || (reinterpret_cast<uintptr_t>(q) % 8 == 0 && ldq % 8 == 0));
  const bool wide_t = qt && aligned16(qt) && ldqt % 16 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (type == TWELL_BF16)
    return vec ? launch<uint16_t, true>(p, block_rows, wide_t, s)
               : launch<uint16_t, false>(p, block_rows, wide_t, s);
  return vec ? launch<float, true>(p, block_rows, wide_t, s)
             : launch<float, false>(p, block_rows, wide_t, s);
}
