// The TwELL epilogue of the batch gate kernels ("Sparser, Faster, Lighter
// Transformer Language Models", section 2.B.1): a thread packs the 128 fp32
// gate pre-activations of its row and tile, held in registers.
#pragma once

#include "common.cuh"

namespace twell {

// Where the epilogue writes: a TwELL's buffers and the optional copy of z.
struct PackOut {
  int32_t F, n_t, W;
  float* val;
  uint8_t* col;
  uint8_t* cnt;
  int32_t* spill_slot;
  int32_t spill_cap;
  int32_t* spill_n;
  int32_t* spill_rt;
  float* spill_val;
  uint32_t* block_bits;  // optional [ceil(T / 128)][F / 32]
  float* z_debug;
  int32_t* status;
};

inline PackOut pack_out(const twell_t& h, float* z_debug, int32_t* status) {
  return PackOut{h.F,         h.F / TWELL_TILE, h.width,    h.val,        h.col,
                 h.cnt,       h.spill_slot,     h.spill_cap, h.spill_n,   h.spill_rt,
                 h.spill_val, h.block_bits,     z_debug,    status};
}

__device__ __forceinline__ void flag(int32_t* status, int32_t bit) {
  if (status) atomicOr(status, bit);
}

// Pack the slice r (row t, tile kt) into the TwELL: a 32-bit mask of z > 0
// per 32-column chunk, a walk over its set bits (ascending columns), the
// chunk staged in the thread's 128 bytes of shared memory `my_stage`
// (XOR-swizzled by 16-byte chunk with `row`, the thread's row of its 128)
// only when it has entries; a spilled slice is written from the registers.
// Called by whole warps, a row per lane; rows with `valid` false (past T)
// write nothing.
__device__ __forceinline__ void pack_row_slice(const PackOut& p, const float (&r)[4][32], int t,
                                               bool valid, int m_blk, int kt, int lane, int row,
                                               uint8_t* my_stage) {
  const size_t rt = static_cast<size_t>(valid ? t : 0) * p.n_t + kt;
  float* vrow = p.val + rt * p.W;
  uint8_t* crow = p.col + rt * p.W;
  // bitmask of the positive gates of each 32-column chunk of the row
  uint32_t mk[4];
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (r[ch][i] > 0.0f) m |= 1u << i;
    mk[ch] = valid ? m : 0u;
  }
  if (p.block_bits) {
    // OR over the warp's 32 rows, one atomic per word and warp
#pragma unroll
    for (int ch = 0; ch < 4; ++ch) {
      const uint32_t any = __reduce_or_sync(0xffffffffu, mk[ch]);
      if (lane == 0 && any)
        atomicOr(p.block_bits + static_cast<size_t>(m_blk) * (p.F / 32) + kt * 4 + ch, any);
    }
  }
  int c = 0;
  if (valid) {
    if (p.z_debug) {
      float4* zd = reinterpret_cast<float4*>(p.z_debug + static_cast<size_t>(t) * p.F +
                                             kt * TWELL_TILE);
#pragma unroll
      for (int ch = 0; ch < 4; ++ch)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          zd[ch * 8 + i] =
              make_float4(r[ch][4 * i], r[ch][4 * i + 1], r[ch][4 * i + 2], r[ch][4 * i + 3]);
    }
#pragma unroll
    for (int ch = 0; ch < 4; ++ch) {
      const uint32_t m = mk[ch];
      if (m == 0u) continue;
      const int n = __popc(m);
      if (c < p.W) {
        // stage the chunk, then store its actives in column order
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<float4*>(my_stage + ((j ^ (row & 7)) << 4)) =
              make_float4(r[ch][4 * j], r[ch][4 * j + 1], r[ch][4 * j + 2], r[ch][4 * j + 3]);
        uint32_t mm = m;
        for (int e = c; e < p.W && mm != 0u; ++e) {
          const int i = __ffs(mm) - 1;
          mm &= mm - 1u;
          vrow[e] = *reinterpret_cast<const float*>(
              my_stage + ((((i >> 2) ^ (row & 7)) << 4) | ((i & 3) << 2)));
          crow[e] = static_cast<uint8_t>(ch * 32 + i);
        }
      }
      c += n;
    }
    p.cnt[rt] = static_cast<uint8_t>(c);
  }
  const bool spill = valid && c > p.W;
  if (spill) {
    const int slot = atomicAdd(p.spill_n, 1);
    p.spill_slot[rt] = slot;
    if (slot < p.spill_cap) {
      p.spill_rt[slot] = static_cast<int32_t>(rt);
      float4* dst = reinterpret_cast<float4*>(p.spill_val +
                                              static_cast<size_t>(slot) * TWELL_TILE);
#pragma unroll
      for (int ch = 0; ch < 4; ++ch)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float e[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float v = r[ch][4 * i + k];
            e[k] = v > 0.0f ? v : 0.0f;
          }
          dst[ch * 8 + i] = make_float4(e[0], e[1], e[2], e[3]);
        }
    } else {
      flag(p.status, TWELL_FLAG_SPILL_FULL);
    }
  }
}

}  // namespace twell
