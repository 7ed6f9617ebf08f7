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
// lie in 16 neighbouring lanes and its maximum takes four shuffles.  Rows off
// 16-byte boundaries are read and written element by element, a warp's 256
// elements 32 side by side at a time (two scale blocks, four elements of each in
// a lane).  At 16384 x 2304 with an fp32 stream the forward takes 77 us and the
// backward 79, both 6.7-6.8 TB/s, the rate of a copy; 8192 x 1536 with e4m3 too takes
// 30 us (6.2 TB/s); four rows of 2048 take 2.8, the latency of a launch.
#include "common.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace twell {
namespace {

constexpr int kPipeThreads = 640; // of the pipelined backward (96 registers each: no spills)
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

// First element of piece i of a thread (the others: vec.cuh).
template <bool VEC>
__device__ __forceinline__ int piece_at(int i) {
  const int l = threadIdx.x + i * blockDim.x;
  return VEC ? l * 8 : (l & ~31) * 8 + (l & 31);
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
    const int e = piece_at<VEC>(i);
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
    const int e = piece_at<VEC>(i);
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
    const int e = piece_at<VEC>(i);
    const int n = p.D - e;
    if (n > 0) {
      float w[8];
      load_w<VEC>(p.w, p.w_bf16, e, n, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * w[j];
      if (p.y) store8<VEC>(p.y + t * p.ldy + e, n, v[i]);
    }
    if (p.q && VEC) {
      const float amax = fmaxf(half_warp_max(amax8(v[i])), kFp8AmaxMin);
      if (n > 0) {
        const float inv = kFp8Max / amax;
        store8_e4m3(p.q + t * p.ldq + e, v[i], inv);
        if ((threadIdx.x & 15) == 0) p.scale[t * nb + e / kFp8Block] = amax / kFp8Max;
      }
    }
    if (p.q && !VEC) {
      float a[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        a[k] = kFp8AmaxMin;
#pragma unroll
        for (int j = 4 * k; j < 4 * k + 4; ++j) a[k] = fmaxf(a[k], fabsf(v[i][j]));
        a[k] = warp_max(a[k]);
      }
      store8_e4m3_lanes<32>(p.q + t * p.ldq + e, n, true, v[i], kFp8Max / a[0], kFp8Max / a[1]);
      const int lane = threadIdx.x & 31, b = e / kFp8Block + lane;  // (lanes 0 and 1)
      if (lane < 2 && b < nb) p.scale[t * nb + b] = (lane ? a[1] : a[0]) / kFp8Max;
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

// The groups' shares of dw, added in order in shared memory (`join` [D], used
// when there are several groups), into this block's row of the partial sums.
template <bool VEC, int MAXC>
__device__ __forceinline__ void join_dw(const NormBwdParams& p, float (&acc)[MAXC][8],
                                        float* join) {
  constexpr int step = VEC ? 1 : 32;
  const int G = blockDim.y, grp = threadIdx.y;
  if (G > 1) {
    for (int k = 0; k < G; ++k) {
      if (grp == k) {
#pragma unroll
        for (int i = 0; i < MAXC; ++i) {
          const int e = piece_at<VEC>(i);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (e + j * step < p.D) {
              if (k > 0) acc[i][j] += join[e + j * step];
              join[e + j * step] = acc[i][j];
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
      const int e = piece_at<VEC>(i);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (e + j * step < p.D) o[e + j * step] = acc[i][j];
    }
  }
}

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
  if (kHold && piece_at<VEC>(0) < p.D)
    load_w<VEC>(p.w, p.w_bf16, piece_at<VEC>(0), p.D - piece_at<VEC>(0), w);
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
      const int e = piece_at<VEC>(i);
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
      const int e = piece_at<VEC>(i);
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
      const int e = piece_at<VEC>(i);
      if (e < p.D) {
        if (!kHold && tr) load8<VEC>(tr + e, p.D - e, d);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          n[i][j] = fmaf(rstd, g[i][j] - n[i][j] * dot, tr ? d[j] : 0.0f);
        store8<VEC>(dxr + e, p.D - e, n[i]);
      }
    }
  }
  join_dw<VEC, MAXC>(p, acc, join);
}

// The same for rows on 16-byte boundaries of at most eight elements a thread:
// each thread copies its own elements of the next P rows into shared memory
// (cp.async), so several rows of every group are on their way while one is
// worked on and nobody waits for another thread's copies.  A thread has two
// quads, L quads apart, so that a warp's copy or store of one is a contiguous
// run (with eight neighbours per thread, copies that bypass L1 fetch every
// 32-byte sector of an fp32 row twice).
template <typename ST, typename GT, int P>
__global__ void __launch_bounds__(kPipeThreads) rms_norm_bwd_pipe_kernel(const NormBwdParams p) {
  constexpr int SB = 4 * sizeof(ST), GB = 4 * sizeof(GT);  // bytes of a quad
  extern __shared__ __align__(16) uint8_t ring[];  // [P][2 of s, 2 of dtotal, 2 of dy][threads]
  __shared__ float red[2][32];
  const int L = blockDim.x, G = blockDim.y, grp = threadIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = L >> 5;
  const int nt = L * G, tid = grp * L + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * G;
  const int slot_bytes = nt * (4 * SB + 2 * GB);
  const int e[2] = {4 * static_cast<int>(threadIdx.x), 4 * (L + static_cast<int>(threadIdx.x))};
  float w[8], acc[8];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      acc[4 * k + j] = 0.0f;
      w[4 * k + j] = e[k] >= p.D ? 0.0f
                     : p.w_bf16 ? widen(static_cast<const uint16_t*>(p.w)[e[k] + j])
                                : static_cast<const float*>(p.w)[e[k] + j];
    }
  const uint32_t ring0 = ptx::smem_u32(ring);
  const auto fetch = [&](int64_t t, int slot) {
    if (t < p.T) {
      const uint32_t to = ring0 + slot * slot_bytes + tid * SB;
      const uint32_t tg = ring0 + slot * slot_bytes + 4 * nt * SB + tid * GB;
      const ST* s = static_cast<const ST*>(p.s) + t * p.lds;
      const GT* g = static_cast<const GT*>(p.dy) + t * p.lddy;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (e[k] < p.D) {
          ptx::cp_async<SB>(to + k * nt * SB, s + e[k]);
          if (p.dt)
            ptx::cp_async<SB>(to + (2 + k) * nt * SB,
                              static_cast<const ST*>(p.dt) + t * p.lddt + e[k]);
          ptx::cp_async<GB>(tg + k * nt * GB, g + e[k]);
        }
    }
    ptx::cp_async_commit();  // (a group for every row, empty ones past T)
  };
  const float inv_d = 1.0f / static_cast<float>(p.D);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * G + grp;
#pragma unroll
  for (int k = 0; k < P; ++k) fetch(t0 + k * step, k);
  int par = 0, slot = 0;
  const auto rstd_of = [&](int64_t t) { return t < p.T ? p.rstd[t] : 0.0f; };
  float rstd1 = rstd_of(t0), rstd2 = rstd_of(t0 + step);  // this row's and the next's
  for (int64_t t = t0; t < p.T; t += step, par ^= 1) {
    const float rstd = rstd1;
    rstd1 = rstd2;
    rstd2 = rstd_of(t + 2 * step);
    ptx::cp_async_wait<P - 1>();
    const uint8_t* at = ring + slot * slot_bytes + tid * SB;
    const uint8_t* ag = ring + slot * slot_bytes + 4 * nt * SB + tid * GB;
    float n[8], g[8], d[8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const bool have = e[k] < p.D;
      quad<ST>(at + k * nt * SB, have, n + 4 * k);
      quad<GT>(ag + k * nt * GB, have, g + 4 * k);
      quad<ST>(at + (2 + k) * nt * SB, have && p.dt, d + 4 * k);
    }
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      n[j] *= rstd;
      acc[j] = fmaf(g[j], n[j], acc[j]);
      g[j] *= w[j];
      dot = fmaf(g[j], n[j], dot);
    }
    dot = warp_sum(dot);
    fetch(t + P * step, slot);  // (this thread's values of the slot are in registers)
    if (++slot == P) slot = 0;
    if (nw > 1) {
      // two buffers in turn, as above
      if (lane == 0) red[par][grp * nw + warp] = dot;
      ptx::bar_sync(1 + grp, L);
      dot = warp_sum(lane < nw ? red[par][grp * nw + lane] : 0.0f);
    }
    dot *= inv_d;
    ST* dxr = static_cast<ST*>(p.dx) + t * p.lddx;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int j = 4 * k; j < 4 * k + 4; ++j) n[j] = fmaf(rstd, g[j] - n[j] * dot, d[j]);
      if (e[k] < p.D) store4(dxr + e[k], n + 4 * k);
    }
  }
  ptx::cp_async_wait<0>();
  // the groups' shares of dw, added in order in the ring
  float* join = reinterpret_cast<float*>(ring);
  for (int i = 0; i < G; ++i) {
    __syncthreads();
    if (grp == i) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (e[k] < p.D) {
          float4* o = reinterpret_cast<float4*>(join + e[k]);
          float4 v = make_float4(acc[4 * k], acc[4 * k + 1], acc[4 * k + 2], acc[4 * k + 3]);
          if (i > 0) {
            const float4 u = *o;
            v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
          }
          if (i + 1 == G)
            o = reinterpret_cast<float4*>(p.part + static_cast<size_t>(blockIdx.x) * p.D + e[k]);
          *o = v;
        }
    }
  }
}

// The same for wider rows, one row at a time per block.  Nothing would run
// while a row's sum is joined: so a row is read from the ring twice, for its sum
// while the row before it is finished and once more for dx, with one barrier a
// row between.  The ring holds s and dy only (dtotal is needed once, and is
// loaded where it has the next row's sum to arrive): P rows of it, one in use, one
// summed, with P > 2 others on their way.  A warp has Q x 128 elements of the row
// side by side, quad k of lane l at 128 k + 4 l, so that a thread's places are
// constants from its first.  What is left is bound by issue slots where all is
// bf16 (5000 x 8192, against the kernel above with two pieces a thread: fp32
// stream and bf16 dy 119 -> 87 us, 0.98 of the HBM rate; all bf16 80 -> 74;
// 3000 x 12288: 123 -> 88).
template <typename ST, typename GT, int P, int Q>
__global__ void __launch_bounds__(1024) rms_norm_bwd_wide_kernel(const NormBwdParams p) {
  extern __shared__ __align__(16) uint8_t ring[];  // [P][s of the row, dy of the row]
  __shared__ float red[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  const int e0 = warp * 128 * Q + lane * 4;
  const uint32_t s_bytes = blockDim.x * 4 * Q * sizeof(ST);
  const uint32_t slot_bytes = s_bytes + blockDim.x * 4 * Q * sizeof(GT);
  const uint32_t last = (P - 1) * slot_bytes;
  bool have[Q];
  float w[4 * Q], acc[4 * Q];
#pragma unroll
  for (int k = 0; k < Q; ++k) {
    have[k] = e0 + 128 * k < p.D;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = e0 + 128 * k + j;
      acc[4 * k + j] = 0.0f;
      w[4 * k + j] = !have[k]   ? 0.0f
                     : p.w_bf16 ? widen(static_cast<const uint16_t*>(p.w)[e])
                                : static_cast<const float*>(p.w)[e];
    }
  }
  // This thread's place in the rows, advanced a row of this block at a time.
  const uint32_t T = p.T, step = gridDim.x;  // (t + P step stays below 2^32)
  const ST* s_at = static_cast<const ST*>(p.s) + blockIdx.x * p.lds + e0;
  const GT* g_at = static_cast<const GT*>(p.dy) + blockIdx.x * p.lddy + e0;
  const ST* d_at = static_cast<const ST*>(p.dt) + (p.dt ? blockIdx.x * p.lddt + e0 : 0);
  ST* dx_at = static_cast<ST*>(p.dx) + blockIdx.x * p.lddx + e0;
  const int64_t s_step = step * p.lds, g_step = step * p.lddy, d_step = step * p.lddt,
                dx_step = step * p.lddx;
  const uint8_t* const own = ring + e0 * sizeof(ST);
  const uint8_t* const own_g = ring + s_bytes + e0 * sizeof(GT);
  const uint32_t to = ptx::smem_u32(own), to_g = ptx::smem_u32(own_g);
  const auto fetch = [&](uint32_t t, uint32_t slot) {
    if (t < T) {
#pragma unroll
      for (int k = 0; k < Q; ++k)
        if (have[k]) {
          ptx::cp_async<4 * sizeof(ST)>(to + slot + 128 * k * sizeof(ST), s_at + 128 * k);
          ptx::cp_async<4 * sizeof(GT)>(to_g + slot + 128 * k * sizeof(GT), g_at + 128 * k);
        }
    }
    ptx::cp_async_commit();  // (a group for every row, empty ones past T)
    s_at += s_step;
    g_at += g_step;
  };
  // n = s rstd and dy of quad k of the row in a slot
  const auto read = [&](uint32_t slot, int k, float rstd, float (&n)[4], float (&g)[4]) {
    quad<ST>(own + slot + 128 * k * sizeof(ST), have[k], n);
    quad<GT>(own_g + slot + 128 * k * sizeof(GT), have[k], g);
#pragma unroll
    for (int j = 0; j < 4; ++j) n[j] *= rstd;
  };
  // a row's share of dw and this warp's of its sum
  const auto sum = [&](uint32_t slot, float rstd, int par) {
    float dot = 0.0f;
#pragma unroll
    for (int k = 0; k < Q; ++k) {
      float n[4], g[4];
      read(slot, k, rstd, n, g);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[4 * k + j] = fmaf(g[j], n[j], acc[4 * k + j]);
        dot = fmaf(g[j] * w[4 * k + j], n[j], dot);
      }
    }
    dot = warp_sum(dot);
    if (lane == 0) red[par][warp] = dot;
  };
  const float inv_d = 1.0f / static_cast<float>(p.D);
  uint32_t t = blockIdx.x;
  float rstd = p.rstd[t], rstd1 = t + step < T ? p.rstd[t + step] : 0.0f;  // this row's, the next's
#pragma unroll
  for (int k = 0; k < P; ++k) fetch(t + k * step, k * slot_bytes);
  ptx::cp_async_wait<P - 1>();
  sum(0, rstd, 0);
  __syncthreads();
  uint32_t slot = 0;
  int par = 0;
  for (; t < T; t += step, par ^= 1) {
    float d[4 * Q];
#pragma unroll
    for (int k = 0; k < Q; ++k)
      quad<ST>(reinterpret_cast<const uint8_t*>(d_at + 128 * k), p.dt && have[k], d + 4 * k);
    d_at += d_step;
    const float rstd2 = t + 2 * step < T ? p.rstd[t + 2 * step] : 0.0f;
    const uint32_t ahead = slot == last ? 0 : slot + slot_bytes;
    ptx::cp_async_wait<P - 2>();
    if (t + step < T) sum(ahead, rstd1, par ^ 1);
    // (the row's sum was published by the barrier of the row before)
    const float dot = warp_sum(lane < nw ? red[par][lane] : 0.0f) * inv_d;
#pragma unroll
    for (int k = 0; k < Q; ++k) {
      float n[4], g[4];
      read(slot, k, rstd, n, g);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        n[j] = fmaf(rstd, g[j] * w[4 * k + j] - n[j] * dot, d[4 * k + j]);
      if (have[k]) store4(dx_at + 128 * k, n);
    }
    dx_at += dx_step;
    fetch(t + P * step, slot);  // (this thread is done with the slot)
    slot = ahead;
    rstd = rstd1;
    rstd1 = rstd2;
    __syncthreads();
  }
  ptx::cp_async_wait<0>();
#pragma unroll
  for (int k = 0; k < Q; ++k)
    if (have[k])
      store4(p.part + static_cast<size_t>(blockIdx.x) * p.D + e0 + 128 * k, acc + 4 * k);
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

enum class BwdForm { kPlain, kPipe, kWide };
struct BwdShape {
  BwdForm form;
  int per;   // pieces (plain), quads (wide) of a thread
  int L, G, grid;
  int rows;  // in flight per group
};

// `vec`: every row on 16-byte boundaries; se, ge: bytes of an element of s and dy.
// The wide form's limit is 1024 threads of three quads (64 registers each).
BwdShape bwd_shape(int32_t T, int32_t D, bool vec, int se, int ge, const DeviceInfo& dev) {
  BwdShape b;
  const int pieces = (D + 7) / 8;
  // rows in flight are what fits beside the static shared memory
  const int budget = dev.max_smem_optin - 2048;
  if (vec && pieces <= kPipeThreads) {
    b.form = BwdForm::kPipe;
    b.per = 1;
    b.L = threads_for(D, 1);
    b.G = kPipeThreads / b.L < 15 ? kPipeThreads / b.L : 15;  // named barriers
    const int fit = budget / (b.L * b.G * 8 * (2 * se + ge));
    b.rows = fit < 4 ? fit : 4;
  } else if (vec && D <= 3 * 4096) {
    b.form = BwdForm::kWide;
    b.per = D <= 2 * 4096 ? 2 : 3;
    b.L = (D / 4 + 32 * b.per - 1) / (32 * b.per) * 32;
    b.G = 1;
    const int fit = budget / (b.L * b.per * 4 * (se + ge));
    b.rows = fit < 4 ? fit : 4;
  } else {
    b.form = BwdForm::kPlain;
    b.per = pieces <= 1024 ? 1 : 2;
    b.L = threads_for(D, b.per);
    b.G = 1024 / b.L < 15 ? 1024 / b.L : 15;
    b.rows = 1;
  }
  const int64_t want = (static_cast<int64_t>(T) + b.G - 1) / b.G;
  b.grid = static_cast<int>(want < dev.sm_count ? want : dev.sm_count);
  return b;
}

// Q: quads of a thread in the wide form, 0 for the other.
template <typename ST, typename GT, int P, int Q>
twell_status launch_pipe(const NormBwdParams& p, const BwdShape& b, const DeviceInfo& dev,
                         cudaStream_t s) {
  static std::atomic<uint64_t> set{0};
  void (*kern)(NormBwdParams);
  if constexpr (Q > 0) kern = rms_norm_bwd_wide_kernel<ST, GT, P, Q>;
  else kern = rms_norm_bwd_pipe_kernel<ST, GT, P>;
  const int per = Q > 0 ? 4 * Q * (sizeof(ST) + sizeof(GT)) : 8 * (2 * sizeof(ST) + sizeof(GT));
  return launch_large(kern, dev.max_smem_optin - 1024,
                      launch_config(dim3(b.grid), dim3(b.L, b.G), P * b.L * b.G * per, s), dev,
                      set, p);
}

template <typename ST, typename GT, bool VEC>
twell_status launch_bwd(const NormBwdParams& p, const BwdShape& b, const DeviceInfo& dev,
                        cudaStream_t s) {
  const dim3 block(b.L, b.G);
  // (two rows always fit, three of a wide form's narrower rows)
  if (VEC && b.form == BwdForm::kWide) {
    if (b.per == 2)
      return b.rows == 4 ? launch_pipe<ST, GT, 4, 2>(p, b, dev, s)
                         : launch_pipe<ST, GT, 3, 2>(p, b, dev, s);
    return b.rows == 4   ? launch_pipe<ST, GT, 4, 3>(p, b, dev, s)
           : b.rows == 3 ? launch_pipe<ST, GT, 3, 3>(p, b, dev, s)
                         : launch_pipe<ST, GT, 2, 3>(p, b, dev, s);
  }
  if (VEC && b.form == BwdForm::kPipe)
    return b.rows == 4   ? launch_pipe<ST, GT, 4, 0>(p, b, dev, s)
           : b.rows == 3 ? launch_pipe<ST, GT, 3, 0>(p, b, dev, s)
                         : launch_pipe<ST, GT, 2, 0>(p, b, dev, s);
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
  if (!current_device(&dev)) {
    dev.sm_count = 152;
    dev.max_smem_optin = 232448;
  }
  // (other types and the element-by-element form have as many blocks or fewer)
  const BwdShape b = bwd_shape(T > 0 ? T : 1, D, true, 2, 2, dev);
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
    return cuda_ok(cudaMemsetAsync(dw, 0, static_cast<size_t>(D) * sizeof(float), s))
               ? TWELL_OK
               : TWELL_ERR_CUDA;
  }
  if (!total || !w || !rstd || !dy || !dx || !ws) return TWELL_ERR_INVALID;
  if (ld < D || lddy < D || lddx < D || (dtotal && lddt < D)) return TWELL_ERR_INVALID;
  const int se = elem_bytes(type), ge = elem_bytes(dy_type), we = elem_bytes(w_type);
  if (!elem_aligned(total, se) || !elem_aligned(dx, se) || !elem_aligned(dy, ge) ||
      !elem_aligned(w, we) || !elem_aligned(rstd, 4) || !aligned16(ws) ||
      (dtotal && !elem_aligned(dtotal, se)))
    return TWELL_ERR_INVALID;
  if ((st = require_sm103(&dev)) != TWELL_OK) return st;
  NormBwdParams p{total, w, rstd, dy, dtotal, ld, lddy, lddt, lddx, T, D, w_type == TWELL_BF16,
                  dx, static_cast<float*>(ws)};
  const bool vec = D % 8 == 0 && rows_aligned(total, ld, se) && rows_aligned(w, 0, we) &&
                   rows_aligned(dy, lddy, ge) && rows_aligned(dx, lddx, se) &&
                   (!dtotal || rows_aligned(dtotal, lddt, se));
  const BwdShape b = bwd_shape(T, D, vec, se, ge, dev);
  if (ws_bytes < static_cast<size_t>(b.grid) * D * sizeof(float)) return TWELL_ERR_INVALID;
  const bool sb = type == TWELL_BF16, gb = dy_type == TWELL_BF16;
  if (sb && gb)
    st = vec ? launch_bwd<uint16_t, uint16_t, true>(p, b, dev, s)
             : launch_bwd<uint16_t, uint16_t, false>(p, b, dev, s);
  else if (sb)
    st = vec ? launch_bwd<uint16_t, float, true>(p, b, dev, s)
             : launch_bwd<uint16_t, float, false>(p, b, dev, s);
  else if (gb)
    st = vec ? launch_bwd<float, uint16_t, true>(p, b, dev, s)
             : launch_bwd<float, uint16_t, false>(p, b, dev, s);
  else
    st = vec ? launch_bwd<float, float, true>(p, b, dev, s) : launch_bwd<float, float, false>(p, b, dev, s);
  if (st != TWELL_OK) return st;
  norm_dw_kernel<<<(D + 31) / 32, dim3(32, 32), 0, s>>>(p.part, b.grid, D, dw);
  return cudaGetLastError() == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}
