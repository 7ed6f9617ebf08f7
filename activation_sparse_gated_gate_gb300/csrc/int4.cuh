// Weights in 4 bits with a scale (and a zero point) for each group of a row, and the
// tensor-core products of a few rows of activations with them or with bf16 weights.
//
// A row of K weights is stored in blocks of 128 columns, 64 bytes each.  Column
// 32 i + 8 c + 2 n + o of a block (i, c, n < 4, o < 2) is nibble n of the 16 bits at
// byte 8 (2 c + o) + 2 i.  What this order is for:
//   * lane c of four reads 16 bytes of a row and has the eight columns 8 c .. 8 c + 7 of
//     every 32, so that the four lanes' share of an m16n8k16 product always lies in one
//     group of 32, whatever the group's size, and the columns' order is the one of the
//     activations as they lie in memory;
//   * lane g of eight reads 8 bytes (or 4) of a row and has four columns of every 32: the
//     transposed product (a sum over rows) has its 16 outputs in one group as well.
// A 4-bit code becomes a bf16 without a conversion: 0x4300 | code is 128 + code, and
// subtracting 128 + zero is exact.  Products of bf16 and such integers are exact in the
// tensor core's fp32 sums; the group's scale multiplies the group's sum in fp32.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"

namespace twell {

constexpr int kInt4Block = 128;  // columns of a stored block
constexpr int kInt4Bytes = 64;   // its bytes

// A matrix of 4-bit rows as the kernels see it.
struct Int4View {
  const uint8_t* code;
  const uint16_t* scale;
  const uint8_t* zero;  // optional
  int64_t pitch;        // bytes of a row
  int32_t held;         // groups of a row, those behind K of the last block included
};

inline Int4View view_of(const twell_int4_t& w) {
  const int32_t nb = static_cast<int32_t>((static_cast<int64_t>(w.K) + kInt4Block - 1) / kInt4Block);
  return Int4View{w.code, w.scale, w.zero, static_cast<int64_t>(nb) * kInt4Bytes,
                  nb * (kInt4Block / w.group)};
}

// TWELL_OK if the descriptor may be used (its rows may be none).
inline twell_status check_int4(const twell_int4_t* w) {
  if (!w || w->rows < 0 || w->K < 1) return TWELL_ERR_INVALID;
  if (w->group != 32 && w->group != 64 && w->group != 128) return TWELL_ERR_INVALID;
  if (w->rows == 0) return TWELL_OK;
  // a block's scales and zero points are read at once
  const unsigned per = kInt4Block / w->group;
  if (!w->code || !w->scale || !aligned16(w->code) ||
      reinterpret_cast<uintptr_t>(w->scale) % (2 * per) != 0 ||
      reinterpret_cast<uintptr_t>(w->zero) % per != 0)
    return TWELL_ERR_INVALID;
  return TWELL_OK;
}

// Reads of what is used once: weights pass the first cache by.
__device__ __forceinline__ uint4 ld_stream16(const void* p) {
  uint4 v;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ld16(const void* p) {
  return __ldg(static_cast<const uint4*>(p));
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Of eight nibbles, those n and n + 4 (the halves' n-th) as bf16 less `bias`, which
// holds 128 + zero in each half.
__device__ __forceinline__ uint32_t nibbles(uint32_t p, int n, uint32_t bias) {
  return sub_bf16x2(((p >> (4 * n)) & 0x000f000fu) | 0x43004300u, bias);
}

// Scales and zero points of a row's block, groups of 32 G32 columns.
template <int G32>
struct BlockScales {
  uint32_t s[G32 == 1 ? 2 : 1];
  uint32_t z;
  // From the block's first scale and zero point (NULL: 8).
  __device__ __forceinline__ void load(const uint16_t* scale, const uint8_t* zero) {
    if constexpr (G32 == 1) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(scale));
      s[0] = v.x, s[1] = v.y;
      z = zero ? __ldg(reinterpret_cast<const uint32_t*>(zero)) : 0x08080808u;
    } else if constexpr (G32 == 2) {
      s[0] = __ldg(reinterpret_cast<const uint32_t*>(scale));
      z = zero ? __ldg(reinterpret_cast<const uint16_t*>(zero)) : 0x0808u;
    } else {
      s[0] = __ldg(scale);
      z = zero ? __ldg(zero) : 0x08u;
    }
  }
  __device__ __forceinline__ void load(const Int4View& w, int64_t at) {
    load(w.scale + at, w.zero ? w.zero + at : nullptr);
  }
  // Scales and zero points of 0.
  __device__ __forceinline__ void none() {
    s[0] = z = 0u;
    if constexpr (G32 == 1) s[1] = 0u;
  }
  // Those that another lane has loaded.
  __device__ __forceinline__ void from_lane(const BlockScales& o, int lane) {
    if constexpr (G32 == 4) {  // both in one word (the scale is its low half)
      s[0] = __shfl_sync(0xffffffffu, o.s[0] | o.z << 16, lane);
      z = s[0] >> 16;
      return;
    }
    s[0] = __shfl_sync(0xffffffffu, o.s[0], lane);
    if constexpr (G32 == 1) s[1] = __shfl_sync(0xffffffffu, o.s[1], lane);
    z = __shfl_sync(0xffffffffu, o.z, lane);
  }
  __device__ __forceinline__ float scale(int k) const {
    return __uint_as_float(k & 1 ? s[k / 2] & 0xffff0000u : s[k / 2] << 16);  // (k = 0 of 128)
  }
  // 128 + zero as bf16, in both halves (zero points are below 16)
  __device__ __forceinline__ uint32_t bias(int k) const {
    const uint32_t b = G32 == 4 ? z : (z >> (8 * k)) & 255u;
    return b * 0x00010001u + 0x43004300u;
  }
};

// d += a b of a 16 x 16 and a 16 x 8 tile.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

}  // namespace twell
