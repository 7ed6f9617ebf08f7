// Sums over the columns of weight rows (bf16, or 4 bits with group scales) times a few
// rows of activations, by one warp: 16 MT rows at a time as the A operand of m16n8k16
// products, up to 8 NT activations as B.
//
// The weights come through a ring in shared memory that is the warp's own: each lane
// copies with cp.async the two 16-byte pieces of a row tile that it will use itself (rows g
// and g + 8, its share c of the columns; lane = 4 g + c), so that a copy is waited for by the thread
// that made it and by nobody else.  A slot holds 128 columns of 4-bit rows or 32 of bf16,
// 1 KB a tile either way.  The loops are kept rolled: a decode step runs each instruction a
// few times only, and code fetched from memory may cost more than what it does.
#pragma once

#include "common.cuh"
#include "int4.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace twell {

constexpr int kSlotBytes = 1024;  // 16 rows of a block of 128 columns in 4 bits, or of 32 in bf16

// As ptx::cp_async16, with the rest of the 256 bytes on its way to the second cache: for a
// stream of rows whose neighbouring pieces come next (64 tokens in bf16: 175 us of the layer
// without, 170 with; of 4-bit rows it makes no difference).
__device__ __forceinline__ void cp_async16_ahead(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// The activations of a row tile's product: B operands of 32 columns each, loaded DIST pieces of
// 32 ahead of their use (a load from the second cache takes longer than a piece does).
// x(t, k) loads columns k .. k + 7 of activation 8 t + g (it clamps k to the last eight there
// are); what lies behind K is masked where a block is not whole.  Activations that are
// absent may hold anything: a column of B is a column of the result and nothing else.
template <int NT>
struct Ahead {
  static constexpr int DIST = NT == 1 ? 4 : 2;
  uint4 v[DIST][NT];
  template <typename X>
  __device__ __forceinline__ void load(int at, int k, int nt, X x) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (t < nt) v[at][t] = x(t, k);
  }
  __device__ __forceinline__ void none(int at) {
#pragma unroll
    for (int t = 0; t < NT; ++t) v[at][t] = make_uint4(0u, 0u, 0u, 0u);
  }
};

// acc[m][t] += row tile m times activations t, over the blocks b0 to b1 of 128 columns, of K.
// at[m][h]: this lane's rows of bf16 (g + 8 h of tile m); nt tiles of activations are
// used.  A sum of 32 columns is taken by the tensor core and added in fp32: its own additions
// truncate, and a long chain of them would be felt in an fp32 result.
template <int MT, int NT, int S, typename X>
__device__ __forceinline__ void bf16_rows(const uint16_t* const (&at)[MT][2], int K, int b0, int b1,
                                          uint32_t ring, int nt, X x, float (&acc)[MT][NT][4]) {
  constexpr int DIST = Ahead<NT>::DIST, SLOT = MT * kSlotBytes;
  const int lane = threadIdx.x & 31, c8 = 8 * (lane & 3);
  const uint32_t mine = ring + 16 * lane;
  int put = 0, get = 0, k_put = b0 * kInt4Block + c8;
  const int k_end = min(K, b1 * kInt4Block);
  const auto issue = [&] {  // the next 32 columns
    const bool in = k_put < k_end;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        cp_async16_ahead(mine + put * SLOT + (2 * m + h) * 512, at[m][h] + (in ? k_put : 0),
                         in ? 16 : 0);
    ptx::cp_async_commit();
    k_put += 32;
    put = put + 1 == S ? 0 : put + 1;
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue();
  Ahead<NT> b;
#pragma unroll
  for (int i = 0; i < DIST; ++i) b.load(i, b0 * kInt4Block + 32 * i + c8, nt, x);
#pragma unroll 1
  for (int blk = b0; blk < b1; ++blk) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      issue();
      ptx::cp_async_wait<S - 1>();
      uint4 u[MT], v[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        u[m] = lds16(mine + get * SLOT + m * 1024);
        v[m] = lds16(mine + get * SLOT + m * 1024 + 512);
      }
      get = get + 1 == S ? 0 : get + 1;
      if ((blk + 1) * kInt4Block > K && blk * kInt4Block + 32 * i + c8 >= K) b.none(i % DIST);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (t >= nt) break;
        const uint4 w = b.v[i % DIST][t];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma16816(part, u[m].x, v[m].x, u[m].y, v[m].y, w.x, w.y);
          mma16816(part, u[m].z, v[m].z, u[m].w, v[m].w, w.z, w.w);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[m][t][j] += part[j];
        }
      }
      if (i + DIST < 4 || blk + 1 < b1)
        b.load(i % DIST, blk * kInt4Block + 32 * (i + DIST) + c8, nt, x);
    }
  }
  ptx::cp_async_wait<0>();
}

// The same of 4-bit rows; at[m][h]: the indexes of this lane's rows in w[m].  Of the sums'
// HELD tiles of activations the first NT are used: instructions bound this loop, and a test
// for each tile cost a layer of 64 tokens 196 us instead of 169 (with those of its other sums).
// The four lanes of a row have the scales of four blocks between them, the next four on their way.
template <int G32, int MT, int NT, int HELD, int S, typename X>
__device__ __forceinline__ void int4_rows(const Int4View* const (&w)[MT],
                                          const int64_t (&at)[MT][2], int K, int b0, int b1,
                                          uint32_t ring, X x, float (&acc)[MT][HELD][4]) {
  constexpr int GROUPS = 4 / G32, DIST = Ahead<NT>::DIST, SLOT = MT * kSlotBytes;
  const int lane = threadIdx.x & 31, c = lane & 3;
  const int nb = (K + kInt4Block - 1) / kInt4Block;
  const int n = b1 - b0;
  const uint32_t mine = ring + 16 * lane;
  const uint8_t* code[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) code[m][h] = w[m]->code + at[m][h] * w[m]->pitch + 16 * c;
  int put = 0, get = 0, b_put = b0;
  const auto issue = [&] {
    if (b_put < b1) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          ptx::cp_async<16>(mine + put * SLOT + (2 * m + h) * 512,
                             code[m][h] + b_put * kInt4Bytes);
    }
    ptx::cp_async_commit();
    ++b_put;
    put = put + 1 == S ? 0 : put + 1;
  };
  BlockScales<G32> next[MT][2];
  const auto scales = [&](int i) {  // of the blocks i .. i + 3 of this warp's
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        next[m][h].load(*w[m], at[m][h] * w[m]->held + min(b0 + i + c, nb - 1) * GROUPS);
  };
#pragma unroll 1
  for (int i = 0; i < S - 1; ++i) issue();
  if (n > 0) scales(0);
  Ahead<NT> b;
#pragma unroll
  for (int i = 0; i < DIST; ++i) b.load(i, b0 * kInt4Block + 32 * i + 8 * c, NT, x);
  int blk = b0;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += 4) {
    BlockScales<G32> four[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) four[m][0] = next[m][0], four[m][1] = next[m][1];
    if (i0 + 4 < n) scales(i0 + 4);
    const int last = min(4, n - i0);
#pragma unroll 1
    for (int i = 0; i < last; ++i, ++blk) {
      issue();
      BlockScales<G32> sc[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) sc[m][h].from_lane(four[m][h], (lane & 28) + i);
      ptx::cp_async_wait<S - 1>();
      uint4 raw[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) raw[m][h] = lds16(mine + get * SLOT + (2 * m + h) * 512);
      get = get + 1 == S ? 0 : get + 1;
      float part[MT][NT][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int k = q / G32;
        if (q % G32 == 0) {
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int j = 0; j < 4; ++j) part[m][t][j] = 0.0f;
        }
        const int k0 = blk * kInt4Block + 32 * q + 8 * c;
        if ((blk + 1) * kInt4Block > K && k0 >= K) b.none(q % DIST);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          uint32_t v[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t bias = sc[m][h].bias(k);
            const uint4 r = raw[m][h];
            const uint32_t pr = q < 2 ? __byte_perm(r.x, r.z, q & 1 ? 0x7632 : 0x5410)
                                      : __byte_perm(r.y, r.w, q & 1 ? 0x7632 : 0x5410);
#pragma unroll
            for (int z = 0; z < 4; ++z) v[h][z] = nibbles(pr, z, bias);
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint4 u = b.v[q % DIST][t];
            mma16816(part[m][t], v[0][0], v[1][0], v[0][1], v[1][1], u.x, u.y);
            mma16816(part[m][t], v[0][2], v[1][2], v[0][3], v[1][3], u.z, u.w);
          }
        }
        if (q + DIST < 4 || blk + 1 < b1)
          b.load(q % DIST, blk * kInt4Block + 32 * (q + DIST) + 8 * c, NT, x);
        // (a group behind K has sums of zero, and whatever scale is stored for it)
        if (q % G32 == G32 - 1 && (k == 0 || blk * kInt4Block + 32 * G32 * k < K)) {
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                acc[m][t][j] = fmaf(sc[m][j / 2].scale(k), part[m][t][j], acc[m][t][j]);
        }
      }
    }
  }
  ptx::cp_async_wait<0>();
}

}  // namespace twell
