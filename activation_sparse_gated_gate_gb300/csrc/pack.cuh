// The TwELL epilogue of the batch gate kernels ("Sparser, Faster, Lighter
// Transformer Language Models", section 2.B.1): a thread packs the 128 fp32
// gate pre-activations of its row and tile, held in registers.
#pragma once

#include "common.cuh"
#include "ptx.cuh"

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

// Bit masks of z > 0 of N chunks of 32 columns (0 where the row is past T).
template <int N>
__device__ __forceinline__ void pack_masks(const float (&r)[N][32], bool valid,
                                           uint32_t (&mk)[N]) {
#pragma unroll
  for (int ch = 0; ch < N; ++ch) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (r[ch][i] > 0.0f) m |= 1u << i;
    mk[ch] = valid ? m : 0u;
  }
}

// OR the masks of a warp's 32 rows (chunks ch0.. of tile kt) into the block's
// bitmap, one atomic per word and warp.
template <int N>
__device__ __forceinline__ void pack_bits(const PackOut& p, const uint32_t (&mk)[N], int m_blk,
                                          int kt, int ch0, int lane) {
  if (!p.block_bits) return;
#pragma unroll
  for (int ch = 0; ch < N; ++ch) {
    const uint32_t any = __reduce_or_sync(0xffffffffu, mk[ch]);
    if (lane == 0 && any)
      atomicOr(p.block_bits + static_cast<size_t>(m_blk) * (p.F / 32) + kt * 4 + ch0 + ch, any);
  }
}

// The optional copy of z.
template <int N>
__device__ __forceinline__ void pack_z(const PackOut& p, const float (&r)[N][32], int t, int kt,
                                       int ch0) {
  float4* zd = reinterpret_cast<float4*>(p.z_debug + static_cast<size_t>(t) * p.F +
                                         kt * TWELL_TILE + ch0 * 32);
#pragma unroll
  for (int ch = 0; ch < N; ++ch)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      zd[ch * 8 + i] =
          make_float4(r[ch][4 * i], r[ch][4 * i + 1], r[ch][4 * i + 2], r[ch][4 * i + 3]);
}

// The slots: a walk over each mask's set bits (ascending columns), the chunk
// staged in STAGE bytes of the thread's own shared memory (128: a whole chunk,
// 64: half of one) only when it has entries.  STAGE is also the distance to
// the next row's staging, whose 16-byte pieces are XOR-swizzled with `row`.
// `c` entries of the row and tile come before these chunks.
template <int N, int STAGE>
__device__ __forceinline__ void pack_slots(const PackOut& p, const float (&r)[N][32],
                                           const uint32_t (&mk)[N], size_t rt, int ch0, int c,
                                           int row, uint8_t* my_stage) {
  constexpr int COLS = STAGE / 4, PIECES = STAGE / 16;
  const int sw = STAGE == 128 ? row & 7 : (row >> 1) & 3;
  float* vrow = p.val + rt * p.W;
  uint8_t* crow = p.col + rt * p.W;
#pragma unroll
  for (int part = 0; part < N * 32 / COLS; ++part) {
    const int ch = part * COLS / 32, first = part * COLS % 32;
    uint32_t m = mk[ch];
    if (COLS < 32) m = (m >> first) & ((1u << (COLS & 31)) - 1u);
    if (m == 0u) continue;
    const int n = __popc(m);
    if (c < p.W) {
#pragma unroll
      for (int j = 0; j < PIECES; ++j)
        *reinterpret_cast<float4*>(my_stage + ((j ^ sw) << 4)) =
            make_float4(r[ch][first + 4 * j], r[ch][first + 4 * j + 1], r[ch][first + 4 * j + 2],
                        r[ch][first + 4 * j + 3]);
      for (int e = c; e < p.W && m != 0u; ++e) {
        const int i = __ffs(m) - 1;
        m &= m - 1u;
        vrow[e] = *reinterpret_cast<const float*>(my_stage + ((((i >> 2) ^ sw) << 4) |
                                                              ((i & 3) << 2)));
        crow[e] = static_cast<uint8_t>((ch0 + ch) * 32 + first + i);
      }
    }
    c += n;
  }
}

// A slot of the spill list for (row, tile) rt; >= spill_cap when it is full.
__device__ __forceinline__ int pack_spill_slot(const PackOut& p, size_t rt) {
  const int slot = atomicAdd(p.spill_n, 1);
  p.spill_slot[rt] = slot;
  if (slot < p.spill_cap) p.spill_rt[slot] = static_cast<int32_t>(rt);
  else flag(p.status, TWELL_FLAG_SPILL_FULL);
  return slot;
}

// ReLU(z) of the chunks into spill slice `slot` (< spill_cap).
template <int N>
__device__ __forceinline__ void pack_spill(const PackOut& p, const float (&r)[N][32], int slot,
                                           int ch0) {
  float4* dst = reinterpret_cast<float4*>(p.spill_val + static_cast<size_t>(slot) * TWELL_TILE +
                                          ch0 * 32);
#pragma unroll
  for (int ch = 0; ch < N; ++ch)
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
}

// A whole slice (row t, tile kt) held by one thread, 128 bytes of staging
// each.  Called by whole warps, a row per lane; rows with `valid` false
// (past T) write nothing.
__device__ __forceinline__ void pack_row_slice(const PackOut& p, const float (&r)[4][32], int t,
                                               bool valid, int m_blk, int kt, int lane, int row,
                                               uint8_t* my_stage) {
  const size_t rt = static_cast<size_t>(valid ? t : 0) * p.n_t + kt;
  uint32_t mk[4];
  pack_masks(r, valid, mk);
  pack_bits(p, mk, m_blk, kt, 0, lane);
  if (!valid) return;
  if (p.z_debug) pack_z(p, r, t, kt, 0);
  pack_slots<4, 128>(p, r, mk, rt, 0, 0, row, my_stage);
  const int c = __popc(mk[0]) + __popc(mk[1]) + __popc(mk[2]) + __popc(mk[3]);
  p.cnt[rt] = static_cast<uint8_t>(c);
  if (c > p.W) {
    const int slot = pack_spill_slot(p, rt);
    if (slot < p.spill_cap) pack_spill(p, r, slot, 0);
  }
}

// Half a slice (64 columns, half h of tile kt) held by one thread, 64 bytes of
// staging each; the other half's thread has the same row of another warp.  The
// 256 threads of a tile's two halves meet at named barrier `bar`; `cnt`
// [2][128] and `slots` [128] are theirs in shared memory.
__device__ __forceinline__ void pack_row_half(const PackOut& p, const float (&r)[2][32], int t,
                                              bool valid, int m_blk, int kt, int h, int lane,
                                              int row, uint8_t* my_stage, uint8_t* cnt,
                                              int32_t* slots, uint32_t bar) {
  const size_t rt = static_cast<size_t>(valid ? t : 0) * p.n_t + kt;
  uint32_t mk[2];
  pack_masks(r, valid, mk);
  pack_bits(p, mk, m_blk, kt, 2 * h, lane);
  const int mine = __popc(mk[0]) + __popc(mk[1]);
  cnt[h * 128 + row] = static_cast<uint8_t>(mine);
  ptx::bar_sync(bar, 256);
  const int c = mine + cnt[(h ^ 1) * 128 + row];
  const bool spill = valid && c > p.W;
  if (valid) {
    if (p.z_debug) pack_z(p, r, t, kt, 2 * h);
    pack_slots<2, 64>(p, r, mk, rt, 2 * h, h ? c - mine : 0, row, my_stage);
    if (h == 0) {
      p.cnt[rt] = static_cast<uint8_t>(c);
      if (spill) slots[row] = pack_spill_slot(p, rt);
    }
  }
  // also: nobody writes cnt again before every count has been read
  if (ptx::bar_any(bar, 256, spill)) {
    if (spill && slots[row] < p.spill_cap) pack_spill(p, r, slots[row], 2 * h);
    ptx::bar_sync(bar, 256);
  }
}

}  // namespace twell
