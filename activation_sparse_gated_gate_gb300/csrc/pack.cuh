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

// r[i] for an i that differs from lane to lane: the registers halved five times.
__device__ __forceinline__ float pick32(const float (&r)[32], int i) {
  float t[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) t[k] = i & 1 ? r[2 * k + 1] : r[2 * k];
#pragma unroll
  for (int k = 0; k < 8; ++k) t[k] = i & 2 ? t[2 * k + 1] : t[2 * k];
#pragma unroll
  for (int k = 0; k < 4; ++k) t[k] = i & 4 ? t[2 * k + 1] : t[2 * k];
  const float u0 = i & 8 ? t[1] : t[0], u1 = i & 8 ? t[3] : t[2];
  return i & 16 ? u1 : u0;
}

// The entries of chunk ch (mask m) to slots c and up, through shared memory.
__device__ __forceinline__ void pack_staged(const PackOut& p, const float (&r)[32], uint32_t m,
                                            int ch, int c, int row, uint8_t* my_stage,
                                            float* vrow, uint8_t* crow) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<float4*>(my_stage + ((j ^ (row & 7)) << 4)) =
        make_float4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
  for (int e = c; e < p.W && m != 0u; ++e) {
    const int i = __ffs(m) - 1;
    m &= m - 1u;
    vrow[e] = *reinterpret_cast<const float*>(my_stage +
                                              ((((i >> 2) ^ (row & 7)) << 4) | ((i & 3) << 2)));
    crow[e] = static_cast<uint8_t>(ch * 32 + i);
  }
}

// Pack the slice r (row t, tile kt) into the TwELL: a 32-bit mask of z > 0 per
// 32-column chunk and a walk over its set bits (ascending columns); a spilled
// slice is written from the registers.  Called by whole warps, a row per lane;
// rows with `valid` false (past T) write nothing.
//
// How the walk reads its values: a chunk with entries is staged in the thread's 128
// bytes of shared memory `my_stage` (XOR-swizzled by 16-byte piece with `row`, the
// thread's row of its 128).  With PICK, for a kernel whose shared memory is busy while
// this runs, they are read from the registers (pick32; `my_stage` is not used): a gate of
// 8192 x 1536 x 6144 with 64 slots takes 84 us at 0.5 % active, 92 at 2 %, 187 at 15 % and
// 456 at 50 %, staged 92, 99, 193 and 470.
template <bool PICK>
__device__ __forceinline__ void pack_row_slice(const PackOut& p, const float (&r)[4][32], int t,
                                               bool valid, int m_blk, int kt, int lane, int row,
                                               uint8_t* my_stage) {
  const size_t rt = static_cast<size_t>(valid ? t : 0) * p.n_t + kt;
  float* vrow = p.val + rt * p.W;
  uint8_t* crow = p.col + rt * p.W;
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
  if (PICK) {
#pragma unroll
    for (int ch = 0; ch < 4; ++ch) {
      uint32_t m = mk[ch];
      const int n = __popc(m);
      for (int e = c; e < p.W && m != 0u; ++e) {
        const int i = __ffs(m) - 1;
        m &= m - 1u;
        vrow[e] = pick32(r[ch], i);
        crow[e] = static_cast<uint8_t>(ch * 32 + i);
      }
      c += n;
    }
  } else if (valid) {
#pragma unroll
    for (int ch = 0; ch < 4; ++ch) {
      if (mk[ch] == 0u) continue;
      if (c < p.W) pack_staged(p, r[ch], mk[ch], ch, c, row, my_stage, vrow, crow);
      c += __popc(mk[ch]);
    }
  }
  if (!valid) return;
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
  p.cnt[rt] = static_cast<uint8_t>(c);
  if (c > p.W) {
    const int slot = atomicAdd(p.spill_n, 1);
    p.spill_slot[rt] = slot;
    if (slot < p.spill_cap) {
      p.spill_rt[slot] = static_cast<int32_t>(rt);
      float4* dst =
          reinterpret_cast<float4*>(p.spill_val + static_cast<size_t>(slot) * TWELL_TILE);
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
