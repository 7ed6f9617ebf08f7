// A mixture-of-experts layer for a few tokens: the router's logits and choice, the chosen
// experts' gated FFNs (bf16 or 4-bit weights) and their weighted sum, in two kernels.
//
//   logits = x W_r^T;  the k largest of a token (ties: the lowest expert), p = softmax
//   y[t] = sum over the token's k slots of p sum_j a(x . Wg[e][j]) (x . Wu[e][j]) Wd[e][j]
//
// Bound by the stream of the chosen experts' weights, and at one token by the chain of
// dependent steps behind it.  The first kernel computes the logits (a warp an expert
// pair, eight tokens, fp32 FMAs: a choice must not hang on a tensor core's rounding).  In the second
// every CTA makes the same choice from them, so that nothing waits for a third.  Then a cluster
// of eight CTAs takes a part of an expert's neurons.  Each CTA computes the gate and up sums of its own
// neurons for all the expert's tokens, writes h = a(gate) up into all eight CTAs' shared
// memory, and after one cluster barrier sums h Wd over the cluster's neurons for its own
// eighth of the D columns.  So no sum of D columns leaves the cluster before an expert's part is
// complete: what goes through memory is a row of D for each (token, slot, part), read once
// by whoever completes a token's columns (a counter for each token and eighth), in slot
// order: results do not depend on the order in which clusters finish.
//   With ReLU a neuron whose gate is not positive for any token is dropped after its gate
// sum: its rows of Wu and Wd are not read.
//   The sums over D run on mma.sync with 16 neurons as A and up to 8 NT tokens as B; the
// sums over neurons with 16 columns of Wd as A (int4.cuh's order lets either way read whole
// sectors) and h as B in three bf16 parts, whose sum is h's 24 bits: one part would cost
// y 2^-9 of an element's size.
#include <atomic>

#include "common.cuh"
#include "int4.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace twell {
namespace {

constexpr int kRanks = 8;        // CTAs of a cluster
constexpr int kThreads = 256;
constexpr int kWarps = 8;
constexpr int kMaxExperts = 512, kMaxTokens = 256, kMaxPairs = 2048, kMaxTop = 32;
constexpr int kMaxWidth = 16384;

// ------------------------------------------------------------------- router

struct RouterParams {
  const uint16_t* x;
  const void* w;
  int32_t T, D, E;
  float* logits;
  int32_t* count;  // [T][kRanks], zeroed here for the experts' kernel
};

template <typename W, int EX, int TT>
__global__ void __launch_bounds__(128) router_kernel(const RouterParams p) {
  ptx::grid_launch_next();
  for (int i = blockIdx.x * 128 + threadIdx.x; i < p.T * kRanks; i += gridDim.x * 128)
    p.count[i] = 0;
  if (!p.w) return;
  const int lane = threadIdx.x & 31;
  const int eg = (p.E + EX - 1) / EX, tg = (p.T + TT - 1) / TT;
  const int job = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (job >= eg * tg) return;
  const int e0 = job % eg * EX, t0 = job / eg * TT;
  float acc[EX][TT];
#pragma unroll
  for (int e = 0; e < EX; ++e)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[e][t] = 0.0f;
  const W* w = static_cast<const W*>(p.w);
#pragma unroll(EX* TT == 1 ? 4 : 1)
  for (int k = 8 * lane; k < p.D; k += 256) {
    float wf[EX][8];
#pragma unroll
    for (int e = 0; e < EX; ++e)
      load8<true>(w + static_cast<int64_t>(min(e0 + e, p.E - 1)) * p.D + k, 8, wf[e]);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      float xf[8];
      load8<true>(p.x + static_cast<int64_t>(min(t0 + t, p.T - 1)) * p.D + k, 8, xf);
#pragma unroll
      for (int e = 0; e < EX; ++e)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[e][t] = fmaf(wf[e][j], xf[j], acc[e][t]);
    }
  }
#pragma unroll
  for (int e = 0; e < EX; ++e)
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const float v = warp_sum(acc[e][t]);
      if (lane == 0 && e0 + e < p.E && t0 + t < p.T)
        p.logits[static_cast<int64_t>(t0 + t) * p.E + e0 + e] = v;
    }
}

// ------------------------------------------------------------------ experts

struct MoeParams {
  const uint16_t* x;
  int32_t T, D, F, E, k;
  const float* logits;     // NULL: ids and weights are given
  int32_t* ids;            // [T][k]
  float* weights;
  int32_t renormalise, act;
  const uint16_t* w[3];    // gate, up, down: bf16,
  Int4View q[3];           // or 4 bits
  float* part;             // [T k][parts][D]
  int32_t parts_cap;
  int32_t* count;
  void* y;
  int32_t y_f32;
};

struct Bf16 {
  static constexpr bool FOUR = false;
};
template <int G>
struct Four {
  static constexpr bool FOUR = true;
  static constexpr int G32 = G;
};

// A value as three bf16 whose sum it is (to its 24 bits), for two values.
__device__ __forceinline__ void split3(float a, float b, uint32_t (&o)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    o[i] = bf16x2(a, b);
    a -= __uint_as_float(o[i] << 16);
    b -= __uint_as_float(o[i] & 0xffff0000u);
  }
}

// acc += rows g, g + 8 of `mat` (given by ra, rb) times the tokens' rows of x, over the
// blocks of 128 columns wk, wk + WK, ...
template <typename F, int NT>
__device__ __forceinline__ void row_sums(const MoeParams& p, int mat, int64_t ra, int64_t rb,
                                         const uint16_t* const (&xt)[NT], int wk, int WK,
                                         float (&acc)[NT][4]) {
  const int lane = threadIdx.x & 31, c = lane & 3;
  const int nb = (p.D + kInt4Block - 1) / kInt4Block;
  const auto load_x = [&](int n, int k) {
    return xt[n] && k < p.D ? ld16(xt[n] + k) : make_uint4(0u, 0u, 0u, 0u);
  };
  if constexpr (!F::FOUR) {
    const uint16_t* a = p.w[mat] + ra * p.D;
    const uint16_t* b = p.w[mat] + rb * p.D;
    constexpr int AHEAD = NT == 1 ? 2 : 1;
    for (int b0 = wk; b0 < nb; b0 += AHEAD * WK) {
      uint4 wa[AHEAD][4], wb[AHEAD][4];
#pragma unroll
      for (int s = 0; s < AHEAD; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = (b0 + s * WK) * kInt4Block + 32 * i + 8 * c;
          const bool in = k < p.D;
          wa[s][i] = in ? ld_stream16(a + k) : make_uint4(0u, 0u, 0u, 0u);
          wb[s][i] = in ? ld_stream16(b + k) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
      for (int s = 0; s < AHEAD; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = (b0 + s * WK) * kInt4Block + 32 * i + 8 * c;
          const uint4 u = wa[s][i], v = wb[s][i];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint4 x = load_x(n, k);
            mma16816(acc[n], u.x, v.x, u.y, v.y, x.x, x.y);
            mma16816(acc[n], u.z, v.z, u.w, v.w, x.z, x.w);
          }
        }
    }
  } else {
    const Int4View& q = p.q[mat];
    constexpr int G32 = F::G32, GROUPS = 4 / G32, AHEAD = 4;
    const uint8_t* code[2] = {q.code + ra * q.pitch + 16 * c, q.code + rb * q.pitch + 16 * c};
    const int64_t at[2] = {ra * q.held, rb * q.held};
    for (int b0 = wk; b0 < nb; b0 += AHEAD * WK) {
      uint4 raw[AHEAD][2];
      BlockScales<G32> sc[AHEAD][2];
#pragma unroll
      for (int s = 0; s < AHEAD; ++s) {
        const int blk = b0 + s * WK;
        if (blk >= nb) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) raw[s][h] = ld_stream16(code[h] + blk * kInt4Bytes);
      }
#pragma unroll
      for (int s = 0; s < AHEAD; ++s) {
        const int blk = b0 + s * WK;
        if (blk >= nb) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) sc[s][h].load(q, at[h] + blk * GROUPS);
      }
#pragma unroll
      for (int s = 0; s < AHEAD; ++s) {
        const int blk = b0 + s * WK;
        if (blk >= nb) break;
#pragma unroll
        for (int k = 0; k < GROUPS; ++k) {
          uint32_t w[G32][2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t bias = sc[s][h].bias(k);
            const uint4 r = raw[s][h];
#pragma unroll
            for (int j = 0; j < G32; ++j) {
              const int i = k * G32 + j;
              const uint32_t pr = i < 2 ? __byte_perm(r.x, r.z, i & 1 ? 0x7632 : 0x5410)
                                        : __byte_perm(r.y, r.w, i & 1 ? 0x7632 : 0x5410);
#pragma unroll
              for (int n = 0; n < 4; ++n) w[j][h][n] = nibbles(pr, n, bias);
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < G32; ++j) {
              const uint4 x = load_x(n, blk * kInt4Block + 32 * (k * G32 + j) + 8 * c);
              mma16816(part, w[j][0][0], w[j][1][0], w[j][0][1], w[j][1][1], x.x, x.y);
              mma16816(part, w[j][0][2], w[j][1][2], w[j][0][3], w[j][1][3], x.z, x.w);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[n][j] = fmaf(sc[s][j / 2].scale(k), part[j], acc[n][j]);
          }
        }
      }
    }
  }
}

// One step of the sums over neurons: 16 of them (this lane's four: rows r[0..3] of Wd at
// neurons 2 c, 2 c + 1, 2 c + 8, 2 c + 9, absent ones < 0) by the 64 columns from d0 on.
struct Bf16Step {
  uint4 v[4];
  __device__ __forceinline__ void load(const MoeParams& p, const int64_t (&r)[4], int d0) {
    const int d = d0 + 8 * ((threadIdx.x & 31) >> 2);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = r[i] >= 0 && d < p.D ? ld_stream16(p.w[2] + r[i] * p.D + d)
                                  : make_uint4(0u, 0u, 0u, 0u);
  }
};
template <int G32>
struct FourStep {
  static constexpr int GROUPS = G32 == 1 ? 2 : 1;  // of the 64 columns
  uint32_t v[4];
  uint16_t s[4][GROUPS];
  uint8_t z[4][GROUPS];
  __device__ __forceinline__ void load(const MoeParams& p, const int64_t (&r)[4], int d0) {
    const Int4View& q = p.q[2];
    const int b = d0 / kInt4Block, half = d0 / 64 % 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = 0u;
#pragma unroll
      for (int k = 0; k < GROUPS; ++k) s[i][k] = 0, z[i][k] = 8;
      if (r[i] < 0) continue;
      v[i] = __ldg(reinterpret_cast<const uint32_t*>(q.code + r[i] * q.pitch + b * kInt4Bytes +
                                                     8 * ((threadIdx.x & 31) >> 2) + 4 * half));
#pragma unroll
      for (int k = 0; k < GROUPS; ++k) {
        const int64_t at = r[i] * q.held + b * (4 / G32) + 2 * half / G32 + k;
        s[i][k] = __ldg(q.scale + at);
        if (q.zero) z[i][k] = __ldg(q.zero + at) & 15u;
      }
    }
  }
};

struct Shared {
  int32_t hcnt[2][kRanks];
  int32_t n_active, n_pairs, n_act;
  int32_t total;
  int16_t act[32];               // active rows of this CTA's round
  int16_t alist[kMaxExperts];    // experts with tokens
  int32_t hist[kMaxExperts];
  int32_t live[kMaxTokens];      // slots of a token that have an expert
  uint8_t last[32];              // pairs whose token this CTA completes
};

template <typename F, int NT>
__global__ void __cluster_dims__(kRanks, 1, 1) __launch_bounds__(kThreads, 2)
    experts_kernel(const __grid_constant__ MoeParams p) {
  constexpr int SP = 8 * NT;               // pairs (token, slot) of an expert at a time
  constexpr int UR = NT == 1 ? 2 : 1;      // units of 16 neurons of a CTA at a time
  constexpr int RM = 16 * UR;
  constexpr int SLOTS = kRanks * RM;
  extern __shared__ __align__(16) uint8_t raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int rank = static_cast<int>(ptx::cluster_ctarank());
  const int cluster = blockIdx.x / kRanks, clusters = gridDim.x / kRanks;
  const int P = p.T * p.k;
  const int tiles = (p.D + 63) / 64;                  // of 64 columns
  const int per_rank = (tiles + kRanks - 1) / kRanks;
  const int cols = 64 * per_rank;
  const int col0 = rank * cols;
  const int my_tiles = max(0, min(per_rank, tiles - rank * per_rank));

  float* yacc = reinterpret_cast<float*>(raw);        // [SP][cols]
  float* hb = yacc + SP * cols;                       // [2][SLOTS][SP]
  float4* red = reinterpret_cast<float4*>(hb + 2 * SLOTS * SP);  // [8][NT][32]
  float* zb = reinterpret_cast<float*>(red + 8 * NT * 32);       // [RM][SP]
  int32_t* hidx = reinterpret_cast<int32_t*>(zb + RM * SP);      // [2][SLOTS]
  int32_t* list = hidx + 2 * SLOTS;                   // [SLOTS]
  float* pw = reinterpret_cast<float*>(list + SLOTS);  // [P]
  int16_t* pid = reinterpret_cast<int16_t*>(pw + P);  // [P]
  int16_t* plist = pid + P;                           // [P]
  __shared__ Shared sh;

  ptx::cluster_arrive_relaxed();  // waited for before the first remote store
  bool started = false;
  for (int i = tid; i < p.E; i += kThreads) sh.hist[i] = 0;
  for (int i = tid; i < p.T; i += kThreads) sh.live[i] = 0;
  ptx::grid_wait();

  // ---- the choice, the same in every CTA
  if (p.logits) {
    for (int t = warp; t < p.T; t += kWarps) {
      float v[kMaxExperts / 32];
      uint32_t key[kMaxExperts / 32];  // ordered as the logits are; 0: taken, NaN or none
      bool nan = false;
#pragma unroll
      for (int j = 0; j < kMaxExperts / 32; ++j) {
        const int e = 32 * j + lane;
        v[j] = 0.0f;
        key[j] = 0u;
        if (32 * j < p.E && e < p.E) {
          v[j] = __ldcg(p.logits + static_cast<int64_t>(t) * p.E + e) + 0.0f;
          const uint32_t b = __float_as_uint(v[j]);
          nan |= v[j] != v[j];
          key[j] = v[j] != v[j] ? 1u : (b & 0x80000000u ? ~b : b | 0x80000000u) ;
        }
      }
      nan = __any_sync(0xffffffffu, nan);
      float top = 0.0f, mine = 0.0f;  // the largest logit; that of slot `lane`
      int chosen = -1;
      for (int s = 0; s < p.k; ++s) {
        uint32_t best = 0u;
        int at = 0x7fffffff;
        float val = 0.0f;
#pragma unroll
        for (int j = 0; j < kMaxExperts / 32; ++j)
          if (32 * j < p.E && key[j] > best) best = key[j], at = 32 * j + lane, val = v[j];
        const uint32_t most = __reduce_max_sync(0xffffffffu, best);
        const int e = __reduce_min_sync(0xffffffffu, best == most ? at : 0x7fffffff);
        val = __shfl_sync(0xffffffffu, val, e & 31);
        if (s == 0) top = val;
        if (lane == s) chosen = e, mine = val;
#pragma unroll
        for (int j = 0; j < kMaxExperts / 32; ++j)
          if (32 * j + lane == e) key[j] = 0u;
      }
      float w = lane < p.k ? expf(mine - top) : 0.0f;
      float sum = w;
      if (!p.renormalise) {
        sum = 0.0f;
#pragma unroll
        for (int j = 0; j < kMaxExperts / 32; ++j)
          if (32 * j < p.E && 32 * j + lane < p.E) sum += expf(v[j] - top);
      }
      w /= warp_sum(sum);
      if (nan) w = __uint_as_float(0x7fc00000u);
      if (lane < p.k) {
        pid[t * p.k + lane] = static_cast<int16_t>(chosen);
        pw[t * p.k + lane] = w;
        if (blockIdx.x == 0) {
          p.ids[static_cast<int64_t>(t) * p.k + lane] = chosen;
          p.weights[static_cast<int64_t>(t) * p.k + lane] = w;
        }
      }
    }
  } else {
    for (int i = tid; i < P; i += kThreads) {
      const int e = p.ids[i];
      pid[i] = static_cast<int16_t>(e >= 0 && e < p.E ? e : -1);
      pw[i] = p.weights[i];
    }
  }
  __syncthreads();
  for (int i = tid; i < P; i += kThreads) {
    const int e = pid[i];
    if (e >= 0) {
      atomicAdd(&sh.hist[e], 1);
      atomicAdd(&sh.live[i / p.k], 1);
    }
  }
  __syncthreads();
  if (warp == 0) {
    int n = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const bool on = e0 + lane < p.E && sh.hist[e0 + lane] > 0;
      const uint32_t m = __ballot_sync(0xffffffffu, on);
      if (on) sh.alist[n + __popc(m & ((1u << lane) - 1u))] = static_cast<int16_t>(e0 + lane);
      n += __popc(m);
    }
    if (lane == 0) sh.n_active = n;
  }
  __syncthreads();
  // tokens without an expert
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    if (sh.live[t]) continue;
    for (int d = tid; d < p.D; d += kThreads) {
      const int64_t to = static_cast<int64_t>(t) * p.D + d;
      if (p.y_f32) static_cast<float*>(p.y)[to] = 0.0f;
      else static_cast<uint16_t*>(p.y)[to] = 0;
    }
  }

  const int active = sh.n_active;
  const int units = (p.F + 15) / 16;
  const int parts = active ? max(1, min(clusters / active, p.parts_cap)) : 1;

  for (int item = cluster; item < active * parts; item += clusters) {
    const int e = sh.alist[item / parts], part = item % parts;
    const int u0 = static_cast<int>(static_cast<int64_t>(units) * part / parts);
    const int nu = static_cast<int>(static_cast<int64_t>(units) * (part + 1) / parts) - u0;
    const int rounds = ((nu + kRanks - 1) / kRanks + UR - 1) / UR;
    const int r0 = u0 + nu * rank / kRanks, r1 = u0 + nu * (rank + 1) / kRanks;  // own units
    const int64_t base = static_cast<int64_t>(e) * p.F;
    __syncthreads();
    if (warp == 0) {  // the expert's pairs, in order
      int n = 0;
      for (int i0 = 0; i0 < P; i0 += 32) {
        const bool on = i0 + lane < P && pid[i0 + lane] == e;
        const uint32_t m = __ballot_sync(0xffffffffu, on);
        if (on) plist[n + __popc(m & ((1u << lane) - 1u))] = static_cast<int16_t>(i0 + lane);
        n += __popc(m);
      }
      if (lane == 0) sh.n_pairs = n;
    }
    __syncthreads();
    const int n_pairs = sh.n_pairs;
    for (int s0 = 0; s0 < n_pairs; s0 += SP) {
      const int ns = min(SP, n_pairs - s0);  // pairs of this slab
      const uint16_t* xt[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n)
        xt[n] = 8 * n + g < ns
                    ? p.x + static_cast<int64_t>(plist[s0 + 8 * n + g] / p.k) * p.D
                    : nullptr;
      for (int i = tid; i < SP * cols; i += kThreads) yacc[i] = 0.0f;
      for (int round = 0; round < rounds; ++round) {
        const int buf = round & 1;
        const int ua = r0 + round * UR;
        const int j0 = ua * 16;                                  // first neuron
        const int nj = max(0, min(min(ua + UR, r1) * 16, p.F) - j0);  // neurons of this round
        const int nt = (nj + 15) / 16;                           // tiles of them
        // sums of the tiles of rows `row_of(tile, r)` of `mats` matrices from `mat` on
        const auto sums = [&](int mat, int mats, int tiles_m, auto row_of) {
          const int all = mats * tiles_m;   // 1, 2 or 4 of the eight warps' shares
          const int share = all == 3 ? 4 : all;
          const int WK = kWarps / share;
          const int tile = warp % share, wk = warp / share;
          float acc[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[n][j] = 0.0f;
          if (tile < all) {
            const int m = tile / tiles_m, tl = tile % tiles_m;
            row_sums<F, NT>(p, mat + m, base + row_of(16 * tl + g), base + row_of(16 * tl + g + 8),
                            xt, wk, WK, acc);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
            red[(warp * NT + n) * 32 + lane] =
                make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
          __syncthreads();
          return share;
        };
        // the sum of tile `tile`, row r of it, pair n
        const auto sum_at = [&](int share, int tile, int r, int n) {
          const float* f = reinterpret_cast<const float*>(red);
          const int at = ((n >> 3) * 32 + (r & 7) * 4 + (n & 7) / 2) * 4 + (r >> 3) * 2 + (n & 1);
          float v = 0.0f;
          for (int w = tile; w < kWarps; w += share) v += f[w * (NT * 128) + at];
          return v;
        };
        const auto plain_row = [&](int r) { return static_cast<int64_t>(min(j0 + r, p.F - 1)); };
        int n_act = 0;
        int share = 0, up_tile = 0;
        if (nt > 0) {
          if (p.act == TWELL_SILU) {
            share = sums(0, 2, nt, plain_row);
            up_tile = nt;
            n_act = nj;
          } else {
            share = sums(0, 1, nt, plain_row);
            for (int i = tid; i < nj * SP; i += kThreads) {
              const int r = i / SP, n = i % SP;
              zb[i] = n < ns ? sum_at(share, r >> 4, r & 15, n) : 0.0f;
            }
            __syncthreads();
            if (warp == 0) {
              bool on = false;
              if (lane < nj)
                for (int n = 0; n < ns; ++n) on |= !(zb[lane * SP + n] <= 0.0f);
              const uint32_t m = __ballot_sync(0xffffffffu, on);
              if (on) sh.act[__popc(m & ((1u << lane) - 1u))] = static_cast<int16_t>(lane);
              if (lane == 0) sh.n_act = __popc(m);
            }
            __syncthreads();
            n_act = sh.n_act;
            if (n_act > 0)
              share = sums(1, 1, (n_act + 15) / 16, [&](int r) {
                return static_cast<int64_t>(j0 + sh.act[min(r, n_act - 1)]);
              });
          }
        }
        if (!started) {
          ptx::cluster_wait();
          started = true;
        }
        const uint32_t to = ptx::smem_u32(hb + (buf * SLOTS + rank * RM) * SP);
        for (int i = tid; i < n_act * SP; i += kThreads) {
          const int r = i / SP, n = i % SP;
          float h = 0.0f;
          if (n < ns) {
            const float u = sum_at(share, up_tile + (r >> 4), r & 15, n);
            if (p.act == TWELL_SILU) {
              const float z = sum_at(share, r >> 4, r & 15, n);
              h = z / (1.0f + expf(-z)) * u;
            } else {
              const float z = zb[sh.act[r] * SP + n];
              h = z <= 0.0f ? 0.0f : z * u;
            }
          }
#pragma unroll
          for (int d = 0; d < kRanks; ++d)
            ptx::st_cluster_u32(ptx::mapa(to + 4u * i, d), __float_as_uint(h));
        }
        if (tid < n_act) {
          const uint32_t ix = ptx::smem_u32(hidx + buf * SLOTS + rank * RM + tid);
          const uint32_t j = j0 + (p.act == TWELL_SILU ? tid : sh.act[tid]);
#pragma unroll
          for (int d = 0; d < kRanks; ++d) ptx::st_cluster_u32(ptx::mapa(ix, d), j);
        }
        if (tid < kRanks)
          ptx::st_cluster_u32(ptx::mapa(ptx::smem_u32(&sh.hcnt[buf][rank]), tid), n_act);
        ptx::cluster_arrive();
        ptx::cluster_wait();

        // ---- the cluster's neurons times Wd, this CTA's columns
        if (tid < SLOTS) {
          const int q = tid / RM, s = tid % RM;
          int before = 0, total = 0;
#pragma unroll
          for (int d = 0; d < kRanks; ++d) {
            if (d < q) before += sh.hcnt[buf][d];
            total += sh.hcnt[buf][d];
          }
          if (s < sh.hcnt[buf][q]) list[before + s] = tid;
          if (tid == 0) sh.total = total;
        }
        __syncthreads();
        const int total = sh.total;
        const int steps = (total + 15) / 16;
        const int lanes_ct = min(kWarps, max(1, my_tiles));  // column tiles side by side
        const int NS = kWarps / lanes_ct;                    // warps that share a tile's neurons
        const int ct_w = warp % lanes_ct, ns_w = warp / lanes_ct;
        for (int cb = 0; cb < my_tiles && steps > 0; cb += lanes_ct) {
          const int ct = cb + ct_w;
          const bool on = ct < my_tiles && ns_w < NS;
          float acc[4][NT][4];
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int j = 0; j < 4; ++j) acc[q][n][j] = 0.0f;
          const float* h0 = hb + buf * SLOTS * SP;
          if (on) {
            const int d0 = col0 + 64 * ct;
            for (int st = ns_w; st < steps; st += NS) {
              int slot[4];
              int64_t row[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int s = 16 * st + 2 * c + (i & 1) + 8 * (i >> 1);
                slot[i] = s < total ? list[s] : -1;
                row[i] = s < total ? base + hidx[buf * SLOTS + slot[i]] : -1;
              }
              const auto h_of = [&](int i, int n) {
                return slot[i] >= 0 ? h0[slot[i] * SP + 8 * n + g] : 0.0f;
              };
              if constexpr (!F::FOUR) {
                Bf16Step w;
                w.load(p, row, d0);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  if (8 * n >= ns) break;
                  uint32_t b0[3], b1[3];
                  split3(h_of(0, n), h_of(1, n), b0);
                  split3(h_of(2, n), h_of(3, n), b1);
                  const uint32_t* v0 = &w.v[0].x;
                  const uint32_t* v1 = &w.v[1].x;
                  const uint32_t* v2 = &w.v[2].x;
                  const uint32_t* v3 = &w.v[3].x;
#pragma unroll
                  for (int q = 0; q < 4; ++q) {
                    const uint32_t a0 = __byte_perm(v0[q], v1[q], 0x5410),
                                   a1 = __byte_perm(v0[q], v1[q], 0x7632),
                                   a2 = __byte_perm(v2[q], v3[q], 0x5410),
                                   a3 = __byte_perm(v2[q], v3[q], 0x7632);
#pragma unroll
                    for (int i = 0; i < 3; ++i) mma16816(acc[q][n], a0, a1, a2, a3, b0[i], b1[i]);
                  }
                }
              } else {
                FourStep<F::G32> w;
                w.load(p, row, d0);
#pragma unroll
                for (int k = 0; k < 2; ++k) {  // the 32 columns' groups
                  constexpr int GR = FourStep<F::G32>::GROUPS;
                  const int gk = GR == 2 ? k : 0;
                  const uint32_t sel = k ? 0x7632 : 0x5410;
                  const uint32_t p01 = __byte_perm(w.v[0], w.v[1], sel),
                                 p23 = __byte_perm(w.v[2], w.v[3], sel);
                  const uint32_t z01 = 0x43004300u + w.z[0][gk] + (w.z[1][gk] << 16),
                                 z23 = 0x43004300u + w.z[2][gk] + (w.z[3][gk] << 16);
                  uint32_t a[2][4];
#pragma unroll
                  for (int q = 0; q < 2; ++q) {
                    a[q][0] = nibbles(p01, 2 * q, z01);
                    a[q][1] = nibbles(p01, 2 * q + 1, z01);
                    a[q][2] = nibbles(p23, 2 * q, z23);
                    a[q][3] = nibbles(p23, 2 * q + 1, z23);
                  }
#pragma unroll
                  for (int n = 0; n < NT; ++n) {
                    if (8 * n >= ns) break;
                    uint32_t b0[3], b1[3];
                    split3(h_of(0, n) * widen(w.s[0][gk]), h_of(1, n) * widen(w.s[1][gk]), b0);
                    split3(h_of(2, n) * widen(w.s[2][gk]), h_of(3, n) * widen(w.s[3][gk]), b1);
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                      for (int i = 0; i < 3; ++i)
                        mma16816(acc[2 * k + q][n], a[q][0], a[q][1], a[q][2], a[q][3], b0[i],
                                 b1[i]);
                  }
                }
              }
            }
          }
          for (int turn = 0; turn < NS; ++turn) {
            if (on && ns_w == turn) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    // column of m-row (j / 2, g) of tile q
                    const int d = F::FOUR ? 32 * (q >> 1) + 8 * (g >> 1) + 2 * (2 * (q & 1) + j / 2) +
                                                (g & 1)
                                          : 8 * g + 2 * q + j / 2;
                    yacc[(8 * n + 2 * c + (j & 1)) * cols + 64 * ct + d] += acc[q][n][j];
                  }
            }
            __syncthreads();
          }
        }
      }
      // ---- the slab's rows of this part, and the tokens that they complete
      __syncthreads();
      const int width = max(0, min(cols, p.D - col0));
      for (int i = tid; i < ns * (width / 4); i += kThreads) {
        const int n = i / (width / 4), d = i % (width / 4) * 4;
        const int pair = plist[s0 + n];
        const float w = pw[pair];
        float4 v = *reinterpret_cast<const float4*>(yacc + n * cols + d);
        v.x *= w, v.y *= w, v.z *= w, v.w *= w;
        __stcg(reinterpret_cast<float4*>(
                   p.part + (static_cast<int64_t>(pair) * parts + part) * p.D + col0 + d),
               v);
      }
      __threadfence();
      __syncthreads();
      if (tid < ns) {
        const int t = plist[s0 + tid] / p.k;
        const int before = width > 0 ? atomicAdd(p.count + t * kRanks + rank, 1) : -1;
        sh.last[tid] = before + 1 == sh.live[t] * parts && width > 0;
      }
      __syncthreads();
      for (int n = 0; n < ns; ++n) {
        if (!sh.last[n]) continue;
        __threadfence();
        const int t = plist[s0 + n] / p.k;
        for (int d = tid; d < width; d += kThreads) {
          float v = 0.0f;
          for (int s = 0; s < p.k; ++s) {
            const int pair = t * p.k + s;
            if (pid[pair] < 0) continue;
            const float* from = p.part + static_cast<int64_t>(pair) * parts * p.D + col0 + d;
#pragma unroll 4
            for (int q = 0; q < parts; ++q) v += __ldcg(from + static_cast<int64_t>(q) * p.D);
          }
          const int64_t at = static_cast<int64_t>(t) * p.D + col0 + d;
          if (p.y_f32) static_cast<float*>(p.y)[at] = v;
          else narrow(v, static_cast<uint16_t*>(p.y)[at]);
        }
      }
      __syncthreads();
    }
  }
  if (!started) ptx::cluster_wait();
  ptx::cluster_arrive();  // (nobody leaves while another CTA may still write to it)
  ptx::cluster_wait();
}

// -------------------------------------------------------------------- host

struct Layout {
  size_t logits, count, part, total;
  int32_t parts_cap;
};

// Clusters of the experts' kernel: two CTAs on each SM.
int clusters_of(const DeviceInfo& dev) { return dev.sm_count * 2 / kRanks; }

Layout layout_of(const DeviceInfo& dev, int32_t T, int32_t D, int32_t F, int32_t E, int32_t k) {
  Layout l;
  const int C = clusters_of(dev);
  // parts of an expert: a unit of 16 neurons for each CTA of its cluster at the least, and no
  // more than leave every slot of a token a cluster
  const int by_units = (F + 16 * kRanks - 1) / (16 * kRanks);
  l.parts_cap = by_units < C / k ? by_units : C / k;
  if (l.parts_cap < 1) l.parts_cap = 1;
  const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  l.logits = 0;
  l.count = up(sizeof(float) * T * E);
  l.part = l.count + up(sizeof(int32_t) * T * kRanks);
  l.total = l.part + sizeof(float) * T * k * l.parts_cap * D;
  return l;
}

size_t shared_bytes(int NT, int32_t D, int32_t P) {
  const size_t SP = 8 * NT, RM = NT == 1 ? 32 : 16, slots = kRanks * RM;
  const size_t cols = 64 * (((D + 63) / 64 + kRanks - 1) / kRanks);
  return 4 * (SP * cols + 2 * slots * SP + 8 * NT * 128 + RM * SP + 3 * slots + P) + 4 * P;
}

template <typename F, int NT>
twell_status launch_experts(const MoeParams& p, const DeviceInfo& dev, cudaStream_t s) {
  static std::atomic<uint64_t> set{0};
  const size_t smem = shared_bytes(NT, p.D, p.T * p.k);
  const int64_t most = static_cast<int64_t>(p.T) * p.k < p.E ? p.T * p.k : p.E;
  int64_t clusters = most * p.parts_cap;
  if (clusters > clusters_of(dev)) clusters = clusters_of(dev);
  cudaLaunchConfig_t cfg =
      launch_config(dim3(static_cast<unsigned>(clusters * kRanks)), dim3(kThreads), smem, s);
  cudaLaunchAttribute attr = overlapped();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return launch_large(experts_kernel<F, NT>, dev.max_smem_optin - 8192, cfg, dev, set, p);
}

template <typename F>
twell_status launch_experts(const MoeParams& p, const DeviceInfo& dev, cudaStream_t s) {
  // (the sums of a slab's columns are held in shared memory)
  return p.T <= 8 || p.D > 8192 ? launch_experts<F, 1>(p, dev, s)
                                : launch_experts<F, 4>(p, dev, s);
}

bool sizes_ok(int32_t T, int32_t D, int32_t F, int32_t E, int32_t k) {
  return T >= 0 && D >= 8 && D % 8 == 0 && F >= 1 && E >= 1 && k >= 1;
}
bool within_limits(int32_t T, int32_t D, int32_t E, int32_t k) {
  return T <= kMaxTokens && D <= kMaxWidth && E <= kMaxExperts && k <= kMaxTop &&
         static_cast<int64_t>(T) * k <= kMaxPairs;
}

}  // namespace
}  // namespace twell

extern "C" size_t twell_moe_decode_workspace(int32_t T, int32_t D, int32_t F, int32_t E,
                                             int32_t top_k) {
  using namespace twell;
  if (!sizes_ok(T, D, F, E, top_k) || !within_limits(T, D, E, top_k)) return 0;
  DeviceInfo dev;
  if (!current_device(&dev)) return 0;
  return layout_of(dev, T, D, F, E, top_k).total;
}

extern "C" twell_status twell_moe_decode(const uint16_t* x, int32_t T, const void* router,
                                         int32_t router_type, const twell_experts_t* w,
                                         int32_t top_k, int32_t act, int32_t renormalise,
                                         int32_t* ids, float* weights, void* y, int32_t y_type,
                                         void* ws, size_t ws_bytes, void* stream) {
  using namespace twell;
  if (!w || !sizes_ok(T, w->D, w->F, w->E, top_k) || (router && top_k > w->E))
    return TWELL_ERR_INVALID;
  if ((act != TWELL_RELU && act != TWELL_SILU) ||
      (y_type != TWELL_BF16 && y_type != TWELL_F32) ||
      (router && router_type != TWELL_BF16 && router_type != TWELL_F32))
    return TWELL_ERR_INVALID;
  const bool four = w->Wg4 != nullptr;
  const int32_t D = w->D, F = w->F, E = w->E;
  if (four) {
    const twell_int4_t* m[3] = {w->Wg4, w->Wu4, w->Wd4};
    for (const twell_int4_t* q : m) {
      const twell_status st = check_int4(q);
      if (st != TWELL_OK) return st;
      if (q->rows != static_cast<int64_t>(E) * F || q->K != D || q->group != m[0]->group)
        return TWELL_ERR_INVALID;
    }
    if (w->Wg_t || w->Wu_t || w->Wd) return TWELL_ERR_INVALID;
  } else if (w->Wu4 || w->Wd4 || !w->Wg_t || !w->Wu_t || !w->Wd || !aligned16(w->Wg_t) ||
             !aligned16(w->Wu_t) || !aligned16(w->Wd)) {
    return TWELL_ERR_INVALID;
  }
  if (T == 0) return TWELL_OK;
  if (!x || !aligned16(x) || !ids || !weights || !y || !aligned16(y) || !ws ||
      reinterpret_cast<uintptr_t>(ws) % 16 != 0 || reinterpret_cast<uintptr_t>(ids) % 4 != 0 ||
      reinterpret_cast<uintptr_t>(weights) % 4 != 0 || (router && !aligned16(router)))
    return TWELL_ERR_INVALID;
  if (!within_limits(T, D, E, top_k)) return TWELL_ERR_UNSUPPORTED;
  DeviceInfo dev;
  twell_status st;
  if ((st = require_sm103(&dev)) != TWELL_OK) return st;
  const Layout l = layout_of(dev, T, D, F, E, top_k);
  if (ws_bytes < l.total) return TWELL_ERR_INVALID;
  uint8_t* base = static_cast<uint8_t*>(ws);
  float* logits = reinterpret_cast<float*>(base + l.logits);
  int32_t* count = reinterpret_cast<int32_t*>(base + l.count);
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  const RouterParams r{x, router, T, D, E, logits, count};
  const int64_t jobs = !router  ? 1
                       : T == 1 ? E
                                : static_cast<int64_t>((E + 1) / 2) * ((T + 7) / 8);
  const unsigned grid = static_cast<unsigned>((jobs + 3) / 4);
  if (router_type == TWELL_F32 && router) {
    if (T == 1) router_kernel<float, 1, 1><<<grid, 128, 0, s>>>(r);
    else router_kernel<float, 2, 8><<<grid, 128, 0, s>>>(r);
  } else {
    if (T == 1) router_kernel<uint16_t, 1, 1><<<grid, 128, 0, s>>>(r);
    else router_kernel<uint16_t, 2, 8><<<grid, 128, 0, s>>>(r);
  }
  if (cudaGetLastError() != cudaSuccess) return TWELL_ERR_CUDA;

  MoeParams p{};
  p.x = x;
  p.T = T, p.D = D, p.F = F, p.E = E, p.k = top_k;
  p.logits = router ? logits : nullptr;
  p.ids = ids, p.weights = weights;
  p.renormalise = renormalise, p.act = act;
  p.part = reinterpret_cast<float*>(base + l.part);
  p.parts_cap = l.parts_cap;
  p.count = count;
  p.y = y, p.y_f32 = y_type == TWELL_F32;
  if (!four) {
    p.w[0] = w->Wg_t, p.w[1] = w->Wu_t, p.w[2] = w->Wd;
    return launch_experts<Bf16>(p, dev, s);
  }
  p.q[0] = view_of(*w->Wg4), p.q[1] = view_of(*w->Wu4), p.q[2] = view_of(*w->Wd4);
  return w->Wg4->group == 32   ? launch_experts<Four<1>>(p, dev, s)
         : w->Wg4->group == 64 ? launch_experts<Four<2>>(p, dev, s)
                               : launch_experts<Four<4>>(p, dev, s);
}
