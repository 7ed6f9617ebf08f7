// Eight-element pieces of a row: loads widened to fp32, stores rounded once,
// and e4m3 with the scale of a block of 128.  With VEC a thread's piece is eight
// neighbours, whole and 16-byte aligned.  Without, rows may start anywhere: the
// piece is every STEP-th element (STEP lanes side by side cover a run of 8 STEP),
// so that each access of theirs is one run too, and those below n are touched.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace twell {

constexpr int kFp8Block = 128;                // elements of a row that share a scale
constexpr float kFp8Max = 448.0f;             // e4m3's largest value
constexpr float kFp8AmaxMin = 5.42101086e-20f;  // 2^-64: 448 / amax stays finite

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(uint16_t v) {
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

// bf16 of two values (round to nearest even), lo in the low half.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void narrow(float v, float& o) { o = v; }
__device__ __forceinline__ void narrow(float v, uint16_t& o) {
  o = static_cast<uint16_t>(bf16x2(v, 0.0f));
}

// e4m3 of four values (round to nearest even, saturating; NaN stays NaN), in
// order from the low byte.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

template <bool VEC, int STEP = 32>
__device__ __forceinline__ void load8(const float* p, int n, float (&f)[8]) {
  if (VEC) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = j * STEP < n ? p[j * STEP] : 0.0f;
  }
}

template <bool VEC, int STEP = 32>
__device__ __forceinline__ void load8(const uint16_t* p, int n, float (&f)[8]) {
  if (VEC) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(u[k] << 16);
      f[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = j * STEP < n ? widen(p[j * STEP]) : 0.0f;
  }
}

// Four values from an aligned place in shared memory (zeros without `have`), and
// to an aligned place in a row.
template <typename T>
__device__ __forceinline__ void quad(const uint8_t* at, bool have, float* f) {
  if (sizeof(T) == 4) {
    const float4 a = have ? *reinterpret_cast<const float4*>(at) : make_float4(0.f, 0.f, 0.f, 0.f);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  } else {
    const uint2 a = have ? *reinterpret_cast<const uint2*>(at) : make_uint2(0u, 0u);
    f[0] = __uint_as_float(a.x << 16), f[1] = __uint_as_float(a.x & 0xffff0000u);
    f[2] = __uint_as_float(a.y << 16), f[3] = __uint_as_float(a.y & 0xffff0000u);
  }
}

__device__ __forceinline__ void store4(float* p, const float* f) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void store4(uint16_t* p, const float* f) {
  *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]));
}

template <bool VEC, int STEP = 32>
__device__ __forceinline__ void store8(float* p, int n, const float (&f)[8]) {
  if (VEC) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j * STEP < n) p[j * STEP] = f[j];
  }
}

template <bool VEC, int STEP = 32>
__device__ __forceinline__ void store8(uint16_t* p, int n, const float (&f)[8]) {
  if (VEC) {
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]),
                                              bf16x2(f[4], f[5]), bf16x2(f[6], f[7]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j * STEP < n) narrow(f[j], p[j * STEP]);
  }
}

__device__ __forceinline__ void store8_e4m3(uint8_t* p, const float (&f)[8], float inv) {
  *reinterpret_cast<uint2*>(p) =
      make_uint2(e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                 e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
}

// Bytes j of four neighbouring lanes' words to lane j of them.
__device__ __forceinline__ uint32_t transpose4(uint32_t x) {
  uint32_t t = __shfl_xor_sync(0xffffffffu, x, 1);
  x = __byte_perm(x, t, threadIdx.x & 1 ? 0x3715 : 0x6240);
  t = __shfl_xor_sync(0xffffffffu, x, 2);
  return __byte_perm(x, t, threadIdx.x & 2 ? 0x3276 : 0x5410);
}

// e4m3 of elements STEP apart, f * inv (of the last four: f * inv2), by whole warps
// whose lanes have neighbouring elements: lane j of four writes their values j
// and j + 4, a word each where the row allows (128 x 128 blocks of 15823 x 1638 take
// 30 us, stored a byte at a time 42).  `live`: this lane's row is written.
template <int STEP>
__device__ __forceinline__ void store8_e4m3_lanes(uint8_t* p, int n, bool live,
                                                  const float (&f)[8], float inv, float inv2) {
  const int k = threadIdx.x & 3;
  const uint32_t w[2] = {
      transpose4(e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv)),
      transpose4(e4m3x4(f[4] * inv2, f[5] * inv2, f[6] * inv2, f[7] * inv2))};
  if (!live) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = (4 * h + k) * STEP - k, left = n - at;
    uint8_t* d = p + at;
    if (left >= 4 && (reinterpret_cast<uintptr_t>(d) & 3u) == 0) {
      *reinterpret_cast<uint32_t*>(d) = w[h];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < left) d[j] = static_cast<uint8_t>(w[h] >> (8 * j));
    }
  }
}

__device__ __forceinline__ float amax8(const float (&f)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
  return m;
}

// Maximum over the 16 lanes (a block of 128 elements) of each half-warp.
__device__ __forceinline__ float half_warp_max(float m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

__device__ __forceinline__ float warp_max(float m) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace twell
