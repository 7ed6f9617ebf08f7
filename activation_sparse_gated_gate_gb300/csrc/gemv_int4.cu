// y = x W^T for a few rows x and W in 4 bits with group scales.
//
// A decode step is the stream of its weights: N K / 2 bytes and 2 or 3 for each group.
// What a 4-bit weight costs apart from its half byte decides whether the stream is kept
// up: 13.5e12 weights a second leave a thread 2.7 issue slots a weight.  So the products run
// on the tensor cores even for a single row: an m16n8k16 takes 16 rows of W by 16 columns as
// its A operand, eight rows of x as B.  mma.sync and not tcgen05: its operands come from
// registers, where the codes are unpacked anyway, and its rate (measured: 8 cycles a warp) is
// above what the stream needs at these T.  What bounds it is the integer pipe: shifts,
// logic and byte permutations issue every other cycle, so that unpacking (8 of them for 8
// weights, 4 bf16 subtractions beside) takes 2 of the 2.7 cycles.  So the loop does little
// else: codes and scales go to registers, a step while the last one is used, at fixed
// offsets from one pointer a row, and bounds are looked at once a block.
// A CTA takes 16 rows of W, its 2 to 16 warps an equal part of the blocks of 128 columns
// each; their sums meet in shared memory, in a fixed order.  More than 32 rows of x are taken 32
// at a time, each reading W again (from the second cache).  All 8 NT rows are computed, whether x
// has them or repeats its last: a test for each tile cost 64 x 9216 x 2304 10 % of its time.
//   Measured, weights from memory: 1 x 8192 x 2048 5.6 us (8.7 MB, 1.5 TB/s; a kernel that only
// reads them 2.8 to 4.7), 5 x 2048 x 8192 6.9, 64 x 9216 x 2304 16.2, 1 x 32768 x 8192 42.6
// (3.3 TB/s).
#include <type_traits>

#include "common.cuh"
#include "int4.cuh"
#include "vec.cuh"

namespace twell {
namespace {

struct GemvParams {
  const uint16_t* x;
  int64_t ldx;
  Int4View w;
  int32_t T, N, K, nb;
  void* y;
  int64_t ldy;
  int32_t y_f32;
};

constexpr int kMaxWarps = 16;

// Rows 8 t + g of x from column 8 c on: load(t, i, left) gives this lane's columns of the i-th
// 32 behind the place that advance() moves, of `left` that there are.  Aligned rows, read 16
// bytes at a time (K is a multiple of 8),
template <int NT>
struct Rows16 {
  const uint16_t* p[NT];
  __device__ __forceinline__ uint4 load(int t, int i, int left) const {
    return 32 * i < left ? ld16(p[t] + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void advance(int k) {
#pragma unroll
    for (int t = 0; t < NT; ++t) p[t] += k;
  }
};
// or any rows.
template <int NT>
struct RowsAny {
  const uint16_t* p[NT];
  __device__ __forceinline__ uint4 load(int t, int i, int left) const {
    uint32_t u[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (32 * i + j < left)
        u[j / 2] |= static_cast<uint32_t>(__ldg(p[t] + 32 * i + j)) << (16 * (j % 2));
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
  __device__ __forceinline__ void advance(int k) {
#pragma unroll
    for (int t = 0; t < NT; ++t) p[t] += k;
  }
};

template <int NT, int G32, bool XV>
__global__ void __launch_bounds__(32 * kMaxWarps, 1)
    gemv_int4_kernel(const __grid_constant__ GemvParams p) {
  constexpr int GROUPS = 4 / G32;  // of a block
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int warps = blockDim.x / 32;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int t0 = blockIdx.y * (8 * NT);
  // this warp's blocks, and where its rows and x stand for them (rows behind the last
  // repeat it)
  const int b0 = static_cast<int>(static_cast<int64_t>(p.nb) * warp / warps),
            b1 = static_cast<int>(static_cast<int64_t>(p.nb) * (warp + 1) / warps);
  const uint8_t* code[2];
  const uint16_t* scale[2];
  const uint8_t* zero[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t r = min(row0 + 8 * h + g, static_cast<int64_t>(p.N - 1));
    code[h] = p.w.code + r * p.w.pitch + b0 * kInt4Bytes + 16 * c;
    scale[h] = p.w.scale + r * p.w.held + b0 * GROUPS;
    // (without zero points it is never read)
    zero[h] = (p.w.zero ? p.w.zero : p.w.code) + r * p.w.held + b0 * GROUPS;
  }
  typename std::conditional<XV, Rows16<NT>, RowsAny<NT>>::type x;
#pragma unroll
  for (int n = 0; n < NT; ++n)
    x.p[n] = p.x + static_cast<int64_t>(min(t0 + 8 * n + g, p.T - 1)) * p.ldx + b0 * kInt4Block +
             8 * c;

  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[n][j] = 0.0f;

  uint4 now[2], next[2];
  BlockScales<G32> s_now[2], s_next[2];
  const auto fetch = [&] {  // the block where the pointers stand
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      next[h] = ld_stream16(code[h]);
      s_next[h].load(scale[h], p.w.zero ? zero[h] : nullptr);
      code[h] += kInt4Bytes;
      scale[h] += GROUPS;
      zero[h] += GROUPS;
    }
  };
  // A block's rows of x at once, or where they would not fit in registers, those of 32 columns
  // while the 32 before are used.
  constexpr int HELD = NT <= 2 ? 4 : 2;
  uint4 u[HELD][NT];
  int left = p.K - b0 * kInt4Block - 8 * c;  // columns before K
  const auto load_x = [&](int q) {
    if (left + 8 * c >= (q < 4 ? kInt4Block : kInt4Block + 32)) {
#pragma unroll
      for (int t = 0; t < NT; ++t) u[q % HELD][t] = x.load(t, q, 2 * kInt4Block);
    } else {
#pragma unroll
      for (int t = 0; t < NT; ++t) u[q % HELD][t] = x.load(t, q, left);
    }
  };
  if (b0 < b1) fetch();
  if (HELD == 2) load_x(0);
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
#pragma unroll
    for (int h = 0; h < 2; ++h) now[h] = next[h], s_now[h] = s_next[h];
    if (b + 1 < b1) fetch();
    if (HELD == 4) {
#pragma unroll
      for (int q = 0; q < 4; ++q) load_x(q);
    }
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) {
      float part[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[t][j] = 0.0f;
#pragma unroll
      for (int q = k * G32; q < (k + 1) * G32; ++q) {
        if (HELD == 2) load_x(q + 1);
        uint32_t v[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t bias = s_now[h].bias(k);
          const uint4 r = now[h];
          const uint32_t pr = q < 2 ? __byte_perm(r.x, r.z, q & 1 ? 0x7632 : 0x5410)
                                    : __byte_perm(r.y, r.w, q & 1 ? 0x7632 : 0x5410);
#pragma unroll
          for (int z = 0; z < 4; ++z) v[h][z] = nibbles(pr, z, bias);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint4 o = u[q % HELD][t];
          mma16816(part[t], v[0][0], v[1][0], v[0][1], v[1][1], o.x, o.y);
          mma16816(part[t], v[0][2], v[1][2], v[0][3], v[1][3], o.z, o.w);
        }
      }
      // (a group behind K has sums of zero, and whatever scale is stored for it)
      if (k > 0 && left + 8 * c <= 32 * G32 * k) continue;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[t][j] = fmaf(s_now[j / 2].scale(k), part[t][j], acc[t][j]);
      }
    }
    x.advance(kInt4Block);
    left -= kInt4Block;
  }

  // the warps' sums
  extern __shared__ float sum[];  // [warps][NT 4][32]
  constexpr int VALUES = NT * 128;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[warp * VALUES + (n * 4 + j) * 32 + lane] = acc[n][j];
  __syncthreads();
#pragma unroll 1
  for (int i = tid; i < 16 * min(8 * NT, p.T - t0); i += blockDim.x) {
    const int r = i % 16, t = i / 16;
    const int from = ((t >> 3) * 4 + (r >> 3) * 2 + (t & 1)) * 32 + (r & 7) * 4 + (t >> 1 & 3);
    float v = 0.0f;
#pragma unroll 4
    for (int q = 0; q < warps; ++q) v += sum[q * VALUES + from];
    if (row0 + r >= p.N) continue;
    const int64_t to = static_cast<int64_t>(t0 + t) * p.ldy + row0 + r;
    if (p.y_f32) static_cast<float*>(p.y)[to] = v;
    else narrow(v, static_cast<uint16_t*>(p.y)[to]);
  }
}

template <int NT>
twell_status launch(const GemvParams& p, int32_t group, bool xv, int sms, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.N + 15LL) / 16),
                  static_cast<unsigned>((static_cast<int64_t>(p.T) + 8 * NT - 1) / (8 * NT)));
  // As many warps as run at once (20 an SM; 16 where more than eight rows of x take the
  // registers): what a warp does once takes as long as one or two blocks do (8192 x 2048: 4
  // warps a CTA 5.8 us, 8 6.2; 2048 x 8192: 16 6.4, 8 7.4; 16 rows, 11000 x 4096: 2 15.7, 4 17.9).
  // CTAs that run one after the other are better shorter, up to eight rows with 4 warps at
  // least (32768 x 8192: 42 us, 50 with 2; 12288 x 4096 12.1 and 13.9), of more rows with 4
  // where that leaves clearly less of the last round idle (32 rows, 20000 x 4096: 40 us, 49
  // with 2; 12288 x 4096, one round: 27 and 23).
  const int64_t ctas = static_cast<int64_t>(grid.x) * grid.y;
  const int most = (NT == 1 ? 20 : 16) * sms, least = NT == 1 && p.nb >= 8 ? 4 : 2;
  int warps = kMaxWarps;
  while (warps > least && (warps > p.nb || warps * ctas > most)) warps /= 2;
  if (NT > 1 && warps == 2 && p.nb >= 8 && ctas > 8 * sms) {
    const auto busy = [&](int64_t at_once) {  // percent, of the rounds
      return 100 * ctas / ((ctas + at_once - 1) / at_once * at_once);
    };
    if (busy(4 * sms) > busy(8 * sms) + 10) warps = 4;
  }
  const size_t smem = warps * NT * 512;
#define TWELL_GO(G32)                                                      \
  (xv ? gemv_int4_kernel<NT, G32, true><<<grid, 32 * warps, smem, s>>>(p)  \
      : gemv_int4_kernel<NT, G32, false><<<grid, 32 * warps, smem, s>>>(p))
  if (group == 32) TWELL_GO(1);
  else if (group == 64) TWELL_GO(2);
  else TWELL_GO(4);
#undef TWELL_GO
  return cudaGetLastError() == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}

}  // namespace
}  // namespace twell

extern "C" twell_status twell_gemv_int4(const uint16_t* x, int64_t ldx, const twell_int4_t* w,
                                        int32_t T, void* y, int32_t y_type, int64_t ldy,
                                        void* stream) {
  using namespace twell;
  twell_status st = check_int4(w);
  if (st != TWELL_OK) return st;
  if (T < 0 || (y_type != TWELL_BF16 && y_type != TWELL_F32)) return TWELL_ERR_INVALID;
  if (T == 0 || w->rows == 0) return TWELL_OK;
  if (!x || !y || ldx < w->K || ldy < w->rows || reinterpret_cast<uintptr_t>(x) % 2 != 0 ||
      reinterpret_cast<uintptr_t>(y) % (y_type == TWELL_BF16 ? 2 : 4) != 0)
    return TWELL_ERR_INVALID;
  if (w->rows > 0x7fffffffLL || T > (1 << 20)) return TWELL_ERR_UNSUPPORTED;
  DeviceInfo dev;
  if ((st = require_sm103(&dev)) != TWELL_OK) return st;
  const Int4View v = view_of(*w);
  const GemvParams p{x, ldx, v, T, static_cast<int32_t>(w->rows), w->K,
                     static_cast<int32_t>(v.pitch / kInt4Bytes), y, ldy, y_type == TWELL_F32};
  const bool xv = w->K % 8 == 0 && aligned16(x) && ldx % 8 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T <= 8) return launch<1>(p, w->group, xv, dev.sm_count, s);
  if (T <= 16) return launch<2>(p, w->group, xv, dev.sm_count, s);
  return launch<4>(p, w->group, xv, dev.sm_count, s);
}
