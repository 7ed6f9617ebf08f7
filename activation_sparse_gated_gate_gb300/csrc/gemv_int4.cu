// y = x W^T for a few rows x and W in 4 bits with group scales.
//
// A decode step is the stream of its weights: N K / 2 bytes and 2 or 3 for each group.
// What a 4-bit weight costs apart from its half byte decides whether the stream is kept
// up: 13.5e12 weights a second leave a thread 2.7 issue slots a weight.  So the products run
// on the tensor cores even for a single row: an m16n8k16 takes 16 rows of W by 16 columns as
// its A operand, eight tokens as B, and unpacking is 1.5 instructions a weight (int4.cuh).
// mma.sync and not tcgen05: its operands come from registers, where the codes are
// unpacked anyway, and its rate is far above what the stream needs at these T.
//
// A warp takes MT tiles of 16 rows and every WK-th block of 128 columns; lane (g, c) = (lane
// / 4, lane % 4) reads 16 bytes of rows g and g + 8 of a tile, a row's four lanes a block of
// it.  The group's sums are scaled in fp32.  The WK warps of the same rows add up through shared
// memory in a fixed tree; WR row sets share a CTA and x through the first cache.
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

template <int MT, int NT, int WK, int WR, int G32, bool XV>
__global__ void __launch_bounds__(32 * WK * WR) gemv_int4_kernel(const GemvParams p) {
  constexpr int GROUPS = 4 / G32;             // of a block
  constexpr int AHEAD = MT == 1 ? 4 : 2;      // blocks of codes in registers
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wk = warp % WK, wr = warp / WK;
  const int g = lane >> 2, c = lane & 3;
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * WR + wr) * (16 * MT);
  const int t0 = blockIdx.y * (8 * NT);
  int64_t at[MT][2];  // this lane's rows (those behind the last repeat it)
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t r = row0 + 16 * m + 8 * h + g;
      at[m][h] = r < p.N ? r : p.N - 1;
    }
  const uint16_t* xt[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
    xt[n] = t0 + 8 * n + g < p.T ? p.x + static_cast<int64_t>(t0 + 8 * n + g) * p.ldx : nullptr;

  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[m][n][j] = 0.0f;

  const auto load_x = [&](const uint16_t* row, int k) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (XV) {
      if (row && k < p.K) v = ld16(row + k);
    } else if (row) {
      uint32_t u[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (k + j < p.K) u[j / 2] |= static_cast<uint32_t>(__ldg(row + k + j)) << (16 * (j % 2));
      v = make_uint4(u[0], u[1], u[2], u[3]);
    }
    return v;
  };

  for (int b0 = wk; b0 < p.nb; b0 += WK * AHEAD) {
    uint4 raw[AHEAD][MT][2];
    BlockScales<G32> sc[AHEAD][MT][2];
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      const int b = b0 + a * WK;
      if (b >= p.nb) break;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          raw[a][m][h] = ld_stream16(p.w.code + at[m][h] * p.w.pitch + b * kInt4Bytes + 16 * c);
    }
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      const int b = b0 + a * WK;
      if (b >= p.nb) break;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          sc[a][m][h].load(p.w, at[m][h] * p.w.held + b * GROUPS);
    }
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      const int b = b0 + a * WK;
      if (b >= p.nb) break;
#pragma unroll
      for (int k = 0; k < GROUPS; ++k) {
        uint32_t w[MT][G32][2][4];  // bf16 pairs of rows g, g + 8
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t bias = sc[a][m][h].bias(k);
            const uint4 r = raw[a][m][h];
#pragma unroll
            for (int q = 0; q < G32; ++q) {
              const int i = k * G32 + q;
              const uint32_t pr = i < 2 ? __byte_perm(r.x, r.z, i & 1 ? 0x7632 : 0x5410)
                                        : __byte_perm(r.y, r.w, i & 1 ? 0x7632 : 0x5410);
#pragma unroll
              for (int n = 0; n < 4; ++n) w[m][q][h][n] = nibbles(pr, n, bias);
            }
          }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float part[MT][4];
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) part[m][j] = 0.0f;
#pragma unroll
          for (int q = 0; q < G32; ++q) {
            const uint4 x = load_x(xt[n], b * kInt4Block + 32 * (k * G32 + q) + 8 * c);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              mma16816(part[m], w[m][q][0][0], w[m][q][1][0], w[m][q][0][1], w[m][q][1][1], x.x,
                       x.y);
              mma16816(part[m], w[m][q][0][2], w[m][q][1][2], w[m][q][0][3], w[m][q][1][3], x.z,
                       x.w);
            }
          }
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[m][n][j] = fmaf(sc[a][m][j / 2].scale(k), part[m][j], acc[m][n][j]);
        }
      }
    }
  }

  // the WK warps of the same rows, halves onto halves
  if constexpr (WK > 1) {
    __shared__ float4 sum[WK / 2][WR][MT][NT][32];
#pragma unroll
    for (int half = WK / 2; half > 0; half /= 2) {
      if (half < WK / 2) __syncthreads();
      if (wk >= half && wk < 2 * half) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            sum[wk - half][wr][m][n][lane] =
                make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
      }
      __syncthreads();
      if (wk < half) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float4 o = sum[wk][wr][m][n][lane];
            acc[m][n][0] += o.x, acc[m][n][1] += o.y, acc[m][n][2] += o.z, acc[m][n][3] += o.w;
          }
      }
    }
  }
  if (wk != 0) return;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = t0 + 8 * n + 2 * c + (j & 1);
        const int64_t r = row0 + 16 * m + 8 * (j >> 1) + g;
        if (t >= p.T || r >= p.N) continue;
        const int64_t to = static_cast<int64_t>(t) * p.ldy + r;
        if (p.y_f32) static_cast<float*>(p.y)[to] = acc[m][n][j];
        else narrow(acc[m][n][j], static_cast<uint16_t*>(p.y)[to]);
      }
}

template <int MT, int NT, int WK, int WR>
twell_status launch(const GemvParams& p, int32_t group, bool xv, cudaStream_t s) {
  const int64_t rows = 16 * MT * WR;
  const dim3 grid(static_cast<unsigned>((p.N + rows - 1) / rows),
                  static_cast<unsigned>((static_cast<int64_t>(p.T) + 8 * NT - 1) / (8 * NT)));
  const dim3 block(32 * WK * WR);
#define TWELL_GO(G32)                                                              \
  (xv ? gemv_int4_kernel<MT, NT, WK, WR, G32, true><<<grid, block, 0, s>>>(p)      \
      : gemv_int4_kernel<MT, NT, WK, WR, G32, false><<<grid, block, 0, s>>>(p))
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
  if (w->rows > 0x7fffffffLL || T > (1 << 22) - 64) return TWELL_ERR_UNSUPPORTED;
  DeviceInfo dev;
  if ((st = require_sm103(&dev)) != TWELL_OK) return st;
  const Int4View v = view_of(*w);
  const GemvParams p{x, ldx, v, T, static_cast<int32_t>(w->rows), w->K,
                     static_cast<int32_t>(v.pitch / kInt4Bytes), y, ldy, y_type == TWELL_F32};
  const bool xv = w->K % 8 == 0 && aligned16(x) && ldx % 8 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T <= 8) return launch<1, 1, 8, 1>(p, w->group, xv, s);
  if (T <= 16) return launch<1, 2, 8, 1>(p, w->group, xv, s);
  if (T <= 32) return launch<2, 4, 4, 2>(p, w->group, xv, s);
  return launch<2, 8, 4, 2>(p, w->group, xv, s);
}
