// Residual addition with root-mean-square norm, forward and backward.
//
// Forward, row t of width D:  s = x + r,  rstd = 1 / sqrt(mean(s^2) + eps),
// y = s rstd w.  The sum and the statistics stay in fp32; the stream `total`
// is s rounded once to its own type and y is formed from the unrounded s, so
// a bf16 stream costs y nothing.  y leaves as bf16 and / or as e4m3 with one
// fp32 scale per 128 columns (max |y| / 448, from the unrounded y).
//
// Backward, with n = s rstd and g = dy w:
//   dx = rstd (g - n mean(g n)) + dtotal,   dw = sum_t dy n.
//
// Both are bound by memory: every input is read once and every output
// written once, a row held in registers between its two uses.  A row belongs
// to L threads (a multiple of 32) in pieces of eight elements, piece i of
// thread l being piece l + i L of the row, so the 16 pieces of a scale's block
// lie in 16 neighbouring lanes and its maximum takes four shuffles.
#include "common.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace twell {
namespace {

constexpr int kMaxD = 16384;   // 1024 threads of two pieces

struct NormParams {
  const void* x;
  const void* r;      // optional
  const void* w;
  int64_t ldx, ldr, ldt, ldy, ldq;
  int32_t T, D, w_bf16;
  float eps;
  void* total;        // with r
  uint16_t* y;        // optional
  uint8_t* q;         // optional, with scale
  float* scale;
  float* rstd;        // optional
};

template <bool VEC>
__device__ __forceinline__ void load_w(const void* w, int32_t w_bf16, int e, int n,
                                       float (&f)[8]) {
  if (w_bf16) load8<VEC>(static_cast<const uint16_t*>(w) + e, n, f);
  else load8<VEC>(static_cast<const float*>(w) + e, n, f);
}

// blockDim = (L, rows); rows > 1 only where L is one warp.
template <typename XT, typename RT, bool VEC, int MAXC>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const NormParams p) {
  __shared__ float red[32];
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (t >= p.T) return;  // whole warps, and blocks of one row never take it
  const int L = blockDim.x;
  const XT* xr = static_cast<const XT*>(p.x) + t * p.ldx;
  const RT* rr = p.r ? static_cast<const RT*>(p.r) + t * p.ldr : nullptr;
  float v[MAXC][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < MAXC; ++i) {
    const int e = (threadIdx.x + i * L) * 8;
    const int n = p.D - e;
    if (n > 0) {
      load8<VEC>(xr + e, n, v[i]);
      if (rr) {
        float f[8];
        load8<VEC>(rr + e, n, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += f[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < MAXC; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    const int e = (threadIdx.x + i * L) * 8;
    if (rr && e < p.D)
      store8<VEC>(static_cast<RT*>(p.total) + t * p.ldt + e, p.D - e, v[i]);
  }
  ss = warp_sum(ss);
  if (L > 32) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[warp] = ss;
    __syncthreads();
    ss = warp_sum(lane < (L >> 5) ? red[lane] : 0.0f);
  }
  const float rstd = 1.0f / sqrtf(ss / static_cast<float>(p.D) + p.eps);
  if (p.rstd && threadIdx.x == 0) p.rstd[t] = rstd;
  const int nb = (p.D + kFp8Block - 1) / kFp8Block;
#pragma unroll
  for (int i = 0; i < MAXC; ++i) {
    const int e = (threadIdx.x + i * L) * 8;
    const int n = p.D - e;
    if (n > 0) {
      float w[8];
      load_w<VEC>(p.w, p.w_bf16, e, n, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * w[j];
      if (p.y) store8<VEC>(p.y + t * p.ldy + e, n, v[i]);
    }
    if (p.q) {
      const float amax = fmaxf(half_warp_max(amax8(v[i])), kFp8AmaxMin);
      if (n > 0) {
        store8_e4m3<VEC>(p.q + t * p.ldq + e, n, v[i], kFp8Max / amax);
        if ((threadIdx.x & 15) == 0) p.scale[t * nb + e / kFp8Block] = amax / kFp8Max;
      }
    }
  }
}

struct NormBwdParams {
  const void* s;
  const void* w;
  const float* rstd;
  const void* dy;
  const void* dt;     // optional
  int64_t lds, lddy, lddt, lddx;
  int32_t T, D, w_bf16;
  void* dx;
  float* part;        // [gridDim.x][D]
};

// blockDim = (L, G): G groups of L threads, a row each at a time, each group
// with named barrier 1 + group.  A thread's columns are the same in every
// row, so its share of dw stays in registers until the block's last row; the
// groups' shares are then added in order in shared memory (no atomics: the
// same inputs give the same dw bit for bit).  With two pieces a thread
// (D > 8192) w and dtotal are read where they are used, not held.
template <typename ST, typename GT, bool VEC, int MAXC>
__global__ void __launch_bounds__(1024) rms_norm_bwd_kernel(const NormBwdParams p) {
  constexpr bool kHold = MAXC == 1;
  extern __shared__ float join[];             // [D] when G > 1
  __shared__ float red[2][32];
  const int L = blockDim.x, G = blockDim.y, grp = threadIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = L >> 5;
  float w[8], acc[MAXC][8];
#pragma unroll
  for (int i = 0; i < MAXC; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
  if (kHold && static_cast<int>(threadIdx.x) * 8 < p.D)
    load_w<VEC>(p.w, p.w_bf16, threadIdx.x * 8, p.D - threadIdx.x * 8, w);
  const float inv_d = 1.0f / static_cast<float>(p.D);
  int par = 0;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * G + grp; t < p.T;
       t += static_cast<int64_t>(gridDim.x) * G, par ^= 1) {
    const ST* sr = static_cast<const ST*>(p.s) + t * p.lds;
    const GT* gr = static_cast<const GT*>(p.dy) + t * p.lddy;
    const ST* tr = p.dt ? static_cast<const ST*>(p.dt) + t * p.lddt : nullptr;
    const float rstd = p.rstd[t];
    float n[MAXC][8], g[MAXC][8], d[8];
#pragma unroll
    for (int i = 0; i < MAXC; ++i) {
      const int e = (threadIdx.x + i * L) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) n[i][j] = g[i][j] = 0.0f;
      if (e < p.D) {
        load8<VEC>(sr + e, p.D - e, n[i]);
        load8<VEC>(gr + e, p.D - e, g[i]);
        if (kHold && tr) load8<VEC>(tr + e, p.D - e, d);
      }
    }
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < MAXC; ++i) {
      const int e = (threadIdx.x + i * L) * 8;
      if (e < p.D) {
        if (!kHold) load_w<VEC>(p.w, p.w_bf16, e, p.D - e, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          n[i][j] *= rstd;
          acc[i][j] = fmaf(g[i][j], n[i][j], acc[i][j]);
          g[i][j] *= w[j];
          dot = fmaf(g[i][j], n[i][j], dot);
        }
      }
    }
    dot = warp_sum(dot);
    if (nw > 1) {
      // two buffers in turn: a warp writes one again only after the barrier
      // of the row between, which every reader of it has reached
      if (lane == 0) red[par][grp * nw + warp] = dot;
      ptx::bar_sync(1 + grp, L);
      dot = warp_sum(lane < nw ? red[par][grp * nw + lane] : 0.0f);
    }
    dot *= inv_d;
    ST* dxr = static_cast<ST*>(p.dx) + t * p.lddx;
#pragma unroll
    for (int i = 0; i < MAXC; ++i) {
      const int e = (threadIdx.x + i * L) * 8;
      if (e < p.D) {
        if (!kHold && tr) load8<VEC>(tr + e, p.D - e, d);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          n[i][j] = fmaf(rstd, g[i][j] - n[i][j] * dot, tr ? d[j] : 0.0f);
        store8<VEC>(dxr + e, p.D - e, n[i]);
      }
    }
  }
  if (G > 1) {
    for (int k = 0; k < G; ++k) {
      if (grp == k) {
#pragma unroll
        for (int i = 0; i < MAXC; ++i) {
          const int e = (threadIdx.x + i * L) * 8;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (e + j < p.D) {
              if (k > 0) acc[i][j] += join[e + j];
              join[e + j] = acc[i][j];
            }
        }
      }
      __syncthreads();
    }
  }
  if (grp == G - 1) {
    float* o = p.part + static_cast<size_t>(blockIdx.x) * p.D;
#pragma unroll
    for (int i = 0; i < MAXC; ++i) {
      const int e = (threadIdx.x + i * L) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (e + j < p.D) o[e + j] = acc[i][j];
    }
  }
}

// dw[c] = sum over the P blocks' shares, in a fixed order.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* part, int32_t P, int32_t D,
                                                       float* dw) {
  __shared__ float red[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float a = 0.0f;
  if (c < D)
    for (int i = threadIdx.y; i < P; i += 32) a += part[static_cast<size_t>(i) * D + c];
  red[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  a = warp_sum(red[threadIdx.x][threadIdx.y]);
  const int o = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && o < D) dw[o] = a;
}

bool rows_aligned(const void* p, int64_t ld, int elem) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * elem) % 16 == 0;
}

int elem_bytes(int32_t type) { return type == TWELL_BF16 ? 2 : 4; }
bool type_ok(int32_t type) { return type == TWELL_BF16 || type == TWELL_F32; }
bool elem_aligned(const void* p, int elem) {
  return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(elem - 1)) == 0;
}

// Threads of a row for pieces of eight elements, `per` pieces a thread.
int threads_for(int32_t D, int per) {
  const int pieces = (D + 7) / 8;
  return ((pieces + per - 1) / per + 31) / 32 * 32;
}

template <typename XT, typename RT, bool VEC>
twell_status launch_fwd(const NormParams& p, cudaStream_t s) {
  const int pieces = (p.D + 7) / 8;
  const int per = pieces <= 32 ? 1 : 2;
  const int L = threads_for(p.D, per);
  const dim3 block(L, L == 32 ? 4 : 1);
  const unsigned grid = (static_cast<unsigned>(p.T) + block.y - 1) / block.y;
  if (per == 1) rms_norm_kernel<XT, RT, VEC, 1><<<grid, block, 0, s>>>(p);
  else rms_norm_kernel<XT, RT, VEC, 2><<<grid, block, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}

struct BwdShape {
  int per, L, G, grid;
};

BwdShape bwd_shape(int32_t T, int32_t D, int sms) {
  BwdShape b;
  const int pieces = (D + 7) / 8;
  b.per = pieces <= 1024 ? 1 : 2;
  b.L = threads_for(D, b.per);
  b.G = 1024 / b.L;
  if (b.G > 15) b.G = 15;                 // named barriers
  if (b.G < 1) b.G = 1;
  const int64_t want = (static_cast<int64_t>(T) + b.G - 1) / b.G;
  b.grid = static_cast<int>(want < sms ? want : sms);
  return b;
}

template <typename ST, typename GT, bool VEC>
twell_status launch_bwd(const NormBwdParams& p, const BwdShape& b, cudaStream_t s) {
  const dim3 block(b.L, b.G);
  const size_t smem = b.G > 1 ? static_cast<size_t>(p.D) * sizeof(float) : 0;
  if (b.per == 1) rms_norm_bwd_kernel<ST, GT, VEC, 1><<<b.grid, block, smem, s>>>(p);
  else rms_norm_bwd_kernel<ST, GT, VEC, 2><<<b.grid, block, smem, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}

}  // namespace
}  // namespace twell

extern "C" twell_status twell_rms_norm(const void* x, int32_t x_type, int64_t ldx, const void* r,
                                       int32_t r_type, int64_t ldr, const void* w, int32_t w_type,
                                       int32_t T, int32_t D, float eps, void* total, int64_t ldt,
                                       uint16_t* y, int64_t ldy, uint8_t* q, int64_t ldq,
                                       float* scale, float* rstd, void* stream) {
  using namespace twell;
  if (T < 0 || D <= 0 || !(eps >= 0.0f) || !type_ok(x_type) || !type_ok(w_type))
    return TWELL_ERR_INVALID;
  if (r && !type_ok(r_type)) return TWELL_ERR_INVALID;
  if ((r != nullptr) != (total != nullptr) || (q != nullptr) != (scale != nullptr))
    return TWELL_ERR_INVALID;
  if (D > kMaxD) return TWELL_ERR_UNSUPPORTED;
  if (T == 0) return TWELL_OK;
  if (!x || !w || (!y && !q)) return TWELL_ERR_INVALID;
  if (ldx < D || (r && (ldr < D || ldt < D)) || (y && ldy < D) || (q && ldq < D))
    return TWELL_ERR_INVALID;
  const int xe = elem_bytes(x_type), re = elem_bytes(r_type), we = elem_bytes(w_type);
  if (!elem_aligned(x, xe) || !elem_aligned(w, we) || (y && !elem_aligned(y, 2)) ||
      (r && (!elem_aligned(r, re) || !elem_aligned(total, re))) ||
      (scale && !elem_aligned(scale, 4)) || (rstd && !elem_aligned(rstd, 4)))
    return TWELL_ERR_INVALID;
  DeviceInfo dev;
  twell_status st;
  if ((st = require_sm103(&dev)) != TWELL_OK) return st;
  NormParams p{x, r, w, ldx, ldr, ldt, ldy, ldq, T, D, w_type == TWELL_BF16, eps, total, y, q,
               scale, rstd};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // whole pieces on 16-byte boundaries everywhere, or element by element
  const bool vec = D % 8 == 0 && rows_aligned(x, ldx, xe) && rows_aligned(w, 0, we) &&
                   (!r || (rows_aligned(r, ldr, re) && rows_aligned(total, ldt, re))) &&
                   (!y || rows_aligned(y, ldy, 2)) &&
                   (!q || ((reinterpret_cast<uintptr_t>(q) & 7u) == 0 && ldq % 8 == 0));
  const bool xb = x_type == TWELL_BF16, rb = r && r_type == TWELL_BF16;
  if (xb && rb)
    return vec ? launch_fwd<uint16_t, uint16_t, true>(p, s)
               : launch_fwd<uint16_t, uint16_t, false>(p, s);
  if (xb) return vec ? launch_fwd<uint16_t, float, true>(p, s)
                     : launch_fwd<uint16_t, float, false>(p, s);
  if (rb) return vec ? launch_fwd<float, uint16_t, true>(p, s)
                     : launch_fwd<float, uint16_t, false>(p, s);
  return vec ? launch_fwd<float, float, true>(p, s) : launch_fwd<float, float, false>(p, s);
}

extern "C" size_t twell_rms_norm_bwd_workspace(int32_t T, int32_t D) {
  using namespace twell;
  if (T < 0 || D <= 0 || D > kMaxD) return 0;
  DeviceInfo dev;
  // (without a device: the most blocks a call would use on the part this is for)
  const int sms = current_device(&dev) ? dev.sm_count : 152;
  const BwdShape b = bwd_shape(T > 0 ? T : 1, D, sms);
  return static_cast<size_t>(b.grid) * D * sizeof(float);
}

extern "C" twell_status twell_rms_norm_bwd(const void* total, int32_t type, int64_t ld,
                                           const void* w, int32_t w_type, const float* rstd,
                                           const void* dy, int32_t dy_type, int64_t lddy,
                                           const void* dtotal, int64_t lddt, int32_t T, int32_t D,
                                           void* dx, int64_t lddx, float* dw, void* ws,
                                           size_t ws_bytes, void* stream) {
  using namespace twell;
  if (T < 0 || D <= 0 || !type_ok(type) || !type_ok(w_type) || !type_ok(dy_type) || !dw ||
      !elem_aligned(dw, 4))
    return TWELL_ERR_INVALID;
  if (D > kMaxD) return TWELL_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  DeviceInfo dev;
  twell_status st;
  if (T == 0) {  // no rows: the weight's gradient is an empty sum
    if ((st = require_sm103(&dev)) != TWELL_OK) return st;
    return cudaMemsetAsync(dw, 0, static_cast<size_t>(D) * sizeof(float), s) == cudaSuccess
               ? TWELL_OK
               : TWELL_ERR_CUDA;
  }
  if (!total || !w || !rstd || !dy || !dx || !ws) return TWELL_ERR_INVALID;
  if (ld < D || lddy < D || lddx < D || (dtotal && lddt < D)) return TWELL_ERR_INVALID;
  const int se = elem_bytes(type), ge = elem_bytes(dy_type), we = elem_bytes(w_type);
  if (!elem_aligned(total, se) || !elem_aligned(dx, se) || !elem_aligned(dy, ge) ||
      !elem_aligned(w, we) || !elem_aligned(rstd, 4) || !elem_aligned(ws, 4) ||
      (dtotal && !elem_aligned(dtotal, se)))
    return TWELL_ERR_INVALID;
  if ((st = require_sm103(&dev)) != TWELL_OK) return st;
  const BwdShape b = bwd_shape(T, D, dev.sm_count);
  if (ws_bytes < static_cast<size_t>(b.grid) * D * sizeof(float)) return TWELL_ERR_INVALID;
  NormBwdParams p{total, w, rstd, dy, dtotal, ld, lddy, lddt, lddx, T, D, w_type == TWELL_BF16,
                  dx, static_cast<float*>(ws)};
  const bool vec = D % 8 == 0 && rows_aligned(total, ld, se) && rows_aligned(w, 0, we) &&
                   rows_aligned(dy, lddy, ge) && rows_aligned(dx, lddx, se) &&
                   (!dtotal || rows_aligned(dtotal, lddt, se));
  const bool sb = type == TWELL_BF16, gb = dy_type == TWELL_BF16;
  if (sb && gb)
    st = vec ? launch_bwd<uint16_t, uint16_t, true>(p, b, s)
             : launch_bwd<uint16_t, uint16_t, false>(p, b, s);
  else if (sb)
    st = vec ? launch_bwd<uint16_t, float, true>(p, b, s)
             : launch_bwd<uint16_t, float, false>(p, b, s);
  else if (gb)
    st = vec ? launch_bwd<float, uint16_t, true>(p, b, s)
             : launch_bwd<float, uint16_t, false>(p, b, s);
  else
    st = vec ? launch_bwd<float, float, true>(p, b, s) : launch_bwd<float, float, false>(p, b, s);
  if (st != TWELL_OK) return st;
  norm_dw_kernel<<<(D + 31) / 32, dim3(32, 32), 0, s>>>(p.part, b.grid, D, dw);
  return cudaGetLastError() == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}
