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
// neurons for all the expert's tokens, writes h = a(gate) up into all CTAs' shared
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
#include "rows.cuh"
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
  float* part;             // [T k][parts_cap + 1][D]
  int32_t parts_cap;
  int32_t* count;
  void* y;
  int32_t y_f32;
};

// What is left of a value behind its upper half (nothing of an infinity).
__device__ __forceinline__ float behind(float a) {
  const float hi = __uint_as_float(__float_as_uint(a) & 0xffff0000u);
  return fabsf(a) == __uint_as_float(0x7f800000u) ? 0.0f : a - hi;
}

// Two values as three bf16 each, whose sum they are (to their 24 bits).  Two hold 16 bits:
// enough where y is rounded to bf16.
__device__ __forceinline__ void split(float a, float b, bool three, uint32_t (&o)[3]) {
  o[0] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
  a = behind(a), b = behind(b);
  o[2] = 0u;
  if (three) {
    o[1] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
    o[2] = bf16x2(behind(a), behind(b));
  } else {
    o[1] = bf16x2(a, b);
  }
}

// d += a times the values that b0, b1 are split into, the small ones first.
__device__ __forceinline__ void mma_split(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, bool three, const uint32_t (&b0)[3],
                                          const uint32_t (&b1)[3]) {
  if (three) mma16816(d, a0, a1, a2, a3, b0[2], b1[2]);
  mma16816(d, a0, a1, a2, a3, b0[1], b1[1]);
  mma16816(d, a0, a1, a2, a3, b0[0], b1[0]);
}

// A step of the sums over neurons: 16 of them by a tile of columns.  Lane (g, c) has the
// neurons 2 c, 2 c + 1, 2 c + 8, 2 c + 9 (row[i]; absent ones < 0), 16 bytes of bf16 each or 8 or 4 of
// 4-bit codes, which it copies into its own part of a ring slot.  Of 4-bit rows lanes 0 to 15
// also load the scales of one neuron each, a step or two ahead.
struct Bf16Step {
  static constexpr int BYTES = 2 * kSlotBytes;
  struct Scales {
    __device__ __forceinline__ void load(const MoeParams&, int64_t, int) {}
  };
  static __device__ __forceinline__ void copy(const MoeParams& p, const int64_t (&row)[4], int d0,
                                              uint32_t slot) {
    const int lane = threadIdx.x & 31, d = d0 + 8 * (lane >> 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = row[i] >= 0 && d < p.D;
      cp_async16_or_zero(slot + 512 * i + 16 * lane, p.w[2] + (in ? row[i] * p.D + d : 0), in);
    }
  }
  template <int NT, typename H>
  static __device__ __forceinline__ void add(uint32_t slot, const Scales&, int, H h_of, int nt,
                                             bool three, float (&acc)[4][NT][4]) {
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = lds16(slot + 512 * i + 16 * (threadIdx.x & 31));
    const uint32_t* v0 = &v[0].x;
    const uint32_t* v1 = &v[1].x;
    const uint32_t* v2 = &v[2].x;
    const uint32_t* v3 = &v[3].x;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (n >= nt) break;
      uint32_t b0[3], b1[3];
      split(h_of(0, n), h_of(1, n), three, b0);
      split(h_of(2, n), h_of(3, n), three, b1);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        mma_split(acc[q][n], __byte_perm(v0[q], v1[q], 0x5410), __byte_perm(v0[q], v1[q], 0x7632),
                  __byte_perm(v2[q], v3[q], 0x5410), __byte_perm(v2[q], v3[q], 0x7632), three, b0,
                  b1);
    }
  }
};
// SUB: 32s of columns, 4 (a block) or 2 (half of one).
template <int G32, int SUB>
struct FourStep {
  static constexpr int BYTES = kSlotBytes * SUB / 4;
  typedef BlockScales<G32> One;
  struct Scales {
    One one;  // of neuron `lane & 15`
    __device__ __forceinline__ void load(const MoeParams& p, int64_t row, int d0) {
      one.load(p.q[2], (row >= 0 ? row : 0) * p.q[2].held + d0 / kInt4Block * (4 / G32));
      if (row < 0) one.clear();  // (no product with a scale that is not finite)
    }
  };
  static __device__ __forceinline__ void copy(const MoeParams& p, const int64_t (&row)[4], int d0,
                                              uint32_t slot) {
    const Int4View& q = p.q[2];
    const int lane = threadIdx.x & 31;
    const uint8_t* from = q.code + d0 / kInt4Block * kInt4Bytes + 8 * (lane >> 2) +
                          (SUB == 2 ? 4 * (d0 / 64 % 2) : 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = row[i] >= 0;
      if constexpr (SUB == 4)
        cp_async8_or_zero(slot + 256 * i + 8 * lane, from + (in ? row[i] * q.pitch : 0), in);
      else
        cp_async4_or_zero(slot + 128 * i + 4 * lane, from + (in ? row[i] * q.pitch : 0), in);
    }
  }
  template <int NT, typename H>
  static __device__ __forceinline__ void add(uint32_t slot, const Scales& sc, int d0, H h_of, int nt,
                                             bool three, float (&acc)[2 * SUB][NT][4]) {
    const int lane = threadIdx.x & 31, c = lane & 3;
    uint32_t v[4][SUB / 2];
    One s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (SUB == 4)
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                     : "=r"(v[i][0]), "=r"(v[i][SUB / 2 - 1])
                     : "r"(slot + 256 * i + 8 * lane)
                     : "memory");
      else
        asm volatile("ld.shared.u32 %0, [%1];"
                     : "=r"(v[i][0])
                     : "r"(slot + 128 * i + 4 * lane)
                     : "memory");
      s[i].from_lane(sc.one, 2 * c + (i & 1) + 8 * (i >> 1));
      if (SUB == 2 && d0 / 64 % 2) {  // the half's groups to the front
        if constexpr (G32 == 1) s[i].s[0] = s[i].s[1], s[i].z >>= 16;
        else if constexpr (G32 == 2) s[i].s[0] >>= 16, s[i].z >>= 8;
      }
    }
    uint32_t b0[NT][3], b1[NT][3];
#pragma unroll
    for (int k = 0; k < SUB; ++k) {
      const int gk = k / G32;
      if (k % G32 == 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (n >= nt) break;
          split(h_of(0, n) * s[0].scale(gk), h_of(1, n) * s[1].scale(gk), three, b0[n]);
          split(h_of(2, n) * s[2].scale(gk), h_of(3, n) * s[3].scale(gk), three, b1[n]);
        }
      }
      const uint32_t sel = k & 1 ? 0x7632 : 0x5410;
      const uint32_t p01 = __byte_perm(v[0][k / 2], v[1][k / 2], sel),
                     p23 = __byte_perm(v[2][k / 2], v[3][k / 2], sel);
      const uint32_t z01 = __byte_perm(s[0].bias(gk), s[1].bias(gk), 0x5410),
                     z23 = __byte_perm(s[2].bias(gk), s[3].bias(gk), 0x5410);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t a0 = nibbles(p01, 2 * q, z01), a1 = nibbles(p01, 2 * q + 1, z01),
                       a2 = nibbles(p23, 2 * q, z23), a3 = nibbles(p23, 2 * q + 1, z23);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (n >= nt) break;
          mma_split(acc[2 * k + q][n], a0, a1, a2, a3, three, b0[n], b1[n]);
        }
      }
    }
  }
};

// The two forms of weights: the sums over the columns of two tiles of rows (at[m][h]: this
// lane's of matrix mat[m]), the step above, and the column of a tile that row (h, g) (g of the upper or lower eight) of its q-th
// 16 outputs is.
struct Bf16 {
  static constexpr bool FOUR = false;
  template <int TW>
  using Step = Bf16Step;
  template <int NT, int S, typename X>
  static __device__ __forceinline__ void rows(const MoeParams& p, const int (&mat)[2],
                                              const int64_t (&at)[2][2], int wk, int WK,
                                              uint32_t ring, int nt, X x, float (&acc)[2][NT][4]) {
    const uint16_t* const from[2][2] = {
        {p.w[mat[0]] + at[0][0] * p.D, p.w[mat[0]] + at[0][1] * p.D},
        {p.w[mat[1]] + at[1][0] * p.D, p.w[mat[1]] + at[1][1] * p.D}};
    bf16_rows<2, NT, S>(from, p.D, wk, WK, ring, nt, x, acc);
  }
  static __device__ __forceinline__ int column(int q, int h, int g) { return 8 * g + 2 * q + h; }
  // `width` columns (a multiple of 8) of a row of Wd towards the second cache.
  static __device__ __forceinline__ void ahead(const MoeParams& p, int64_t row, int d0, int width) {
    ptx::prefetch_l2_bulk(p.w[2] + row * p.D + d0, 2 * width);
  }
};
template <int G>
struct Four {
  static constexpr bool FOUR = true;
  template <int TW>
  using Step = FourStep<G, TW / 32>;
  template <int NT, int S, typename X>
  static __device__ __forceinline__ void rows(const MoeParams& p, const int (&mat)[2],
                                              const int64_t (&at)[2][2], int wk, int WK,
                                              uint32_t ring, int nt, X x, float (&acc)[2][NT][4]) {
    const Int4View* const from[2] = {&p.q[mat[0]], &p.q[mat[1]]};
    int4_rows<G, 2, NT, S>(from, at, p.D, wk, WK, ring, nt, x, acc);
  }
  static __device__ __forceinline__ void ahead(const MoeParams& p, int64_t row, int d0, int width) {
    ptx::prefetch_l2_bulk(p.q[2].code + row * p.q[2].pitch + d0 / kInt4Block * kInt4Bytes,
                          (width + kInt4Block - 1) / kInt4Block * kInt4Bytes);
  }
  static __device__ __forceinline__ int column(int q, int h, int g) {
    return 32 * (q >> 1) + 8 * (g >> 1) + 2 * (2 * (q & 1) + h) + (g & 1);
  }
};

template <int NT>
struct Sizes {
  static constexpr int SP = 8 * NT;              // pairs (token, slot) of an expert at a time
  static constexpr int UR = NT <= 2 ? 4 : 2;     // units of 16 neurons of a CTA at a time
  static constexpr int RM = 16 * UR;
  static constexpr int SLOTS = kRanks * RM;
  static constexpr int HS = SP + 4;              // floats between rows of h (no bank twice)
  static constexpr int RING = 6;                 // KB of a warp's ring
};

// Columns of a step's tile of the sums over neurons.
template <typename F, int NT>
struct Tile {
  static constexpr int COLS = F::FOUR && NT <= 2 ? 128 : 64;
};

struct Shared {
  int32_t hcnt[kRanks];
  int32_t n_slabs, n_act, total, n_rows;
  int16_t act[64];               // active rows of this CTA's round
  int32_t count[kMaxExperts];    // pairs of an expert
  int32_t first[kMaxExperts];    // its first in the sorted list, below its first slab
  int32_t live[kMaxTokens];      // rows of `part` that a token is the sum of
  int32_t rows[128];             // those of the token that is being completed
  uint8_t last[32];              // pairs whose token this CTA completes
};

// The k largest of a token's logits and their weights, by a warp: slot `lane` of them.
// `key`: E words of shared memory of the warp's own.
__device__ __forceinline__ void choose(const MoeParams& p, int t, uint32_t* key, int& chosen,
                                       float& weight) {
  const int lane = threadIdx.x & 31;
  const float* logits = p.logits + static_cast<int64_t>(t) * p.E;
  const auto float_of = [](uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
  };
  bool nan = false;
  uint32_t best = 0u;  // keys are ordered as the logits are; 1: NaN, 0: taken
#pragma unroll 1
  for (int e = lane; e < p.E; e += 32) {
    const float v = __ldcg(logits + e) + 0.0f;  // (adding zero makes one zero of two)
    const uint32_t b = __float_as_uint(v);
    const bool bad = v != v;
    nan |= bad;
    key[e] = bad ? 1u : b & 0x80000000u ? ~b : b | 0x80000000u;
    best = max(best, key[e]);
  }
  nan = __any_sync(0xffffffffu, nan);
  const float top = float_of(__reduce_max_sync(0xffffffffu, best));
  float sum = 0.0f, mine = 0.0f;
  if (!p.renormalise)
#pragma unroll 1
    for (int e = lane; e < p.E; e += 32) sum += expf(float_of(key[e]) - top);
#pragma unroll 1
  for (int s = 0; s < p.k; ++s) {
    best = 0u;
    int at = 0x7fffffff;
#pragma unroll 1
    for (int e = lane; e < p.E; e += 32)
      if (key[e] > best) best = key[e], at = e;
    const uint32_t most = __reduce_max_sync(0xffffffffu, best);
    const int e = __reduce_min_sync(0xffffffffu, best == most ? at : 0x7fffffff);
    if (lane == s) chosen = e, mine = float_of(most);
    if ((e & 31) == lane) key[e] = 0u;
  }
  weight = lane < p.k ? expf(mine - top) : 0.0f;
  weight /= warp_sum(p.renormalise ? weight : sum);
  if (nan) weight = __uint_as_float(0x7fc00000u);
}

template <typename F, int NT>
__global__ void __cluster_dims__(kRanks, 1, 1) __launch_bounds__(kThreads, 2)
    experts_kernel(const __grid_constant__ MoeParams p) {
  typedef Sizes<NT> Z;
  constexpr int SP = Z::SP, UR = Z::UR, RM = Z::RM, SLOTS = Z::SLOTS, HS = Z::HS;
  constexpr int TW = Tile<F, NT>::COLS;
  typedef typename F::template Step<TW> Step;
  extern __shared__ __align__(16) uint8_t raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int rank = static_cast<int>(ptx::cluster_ctarank());
  const int cluster = blockIdx.x / kRanks;
  const int P = p.T * p.k;
  const int tiles = (p.D + TW - 1) / TW;              // of TW columns
  const int per_rank = (tiles + kRanks - 1) / kRanks;
  const int cols = TW * per_rank;
  const int ystride = cols + 1;                       // (rows of a pair on other banks)
  const int col0 = rank * cols;
  const int my_tiles = max(0, min(per_rank, tiles - rank * per_rank));
  const int width = max(0, min(cols, p.D - col0));    // a multiple of 8

  // Each warp's ring, which also holds what it hands to the others: its sums (`red`), the
  // keys of its choice.
  constexpr int RING = Z::RING * kSlotBytes;
  uint8_t* ring = raw + warp * RING;
  float* hb = reinterpret_cast<float*>(raw + kWarps * RING);      // [SLOTS][HS]
  int2* list = reinterpret_cast<int2*>(hb + SLOTS * HS);          // [SLOTS] (slot, neuron)
  int32_t* hidx = reinterpret_cast<int32_t*>(list + SLOTS);       // [SLOTS]
  float* zb = reinterpret_cast<float*>(hidx + SLOTS);             // [RM][SP + 1]
  float* yacc = zb + RM * (SP + 1);                   // [SP][ystride]
  float* pw = yacc + SP * ystride;                    // [P] (from an even word on)
  int32_t* pid = reinterpret_cast<int32_t*>(pw + P);  // [P]
  int32_t* plist = pid + P;                           // [P] pairs by expert
  int32_t* place = plist + P;                         // [P] a pair's among its expert's
  int2* slab = reinterpret_cast<int2*>(place + P);    // [E + P / SP]
  __shared__ Shared sh;
  const uint32_t ring_at = ptx::smem_u32(ring);

  ptx::cluster_arrive_relaxed();  // this CTA's shared memory may be written
  for (int i = tid; i < p.E; i += kThreads) sh.count[i] = 0;
  for (int i = tid; i < p.T; i += kThreads) sh.live[i] = 0;
  ptx::grid_wait();
  ptx::cluster_wait();

  // ---- the choice.  Of a few tokens every CTA makes it for itself, a token a warp; of more
  // each warp of the cluster makes it for a token and tells the cluster's CTAs.
  const bool alone = p.T <= kWarps;
  if (p.logits) {
#pragma unroll 1
    for (int t = alone ? warp : rank + kRanks * warp; t < p.T; t += kRanks * kWarps) {
      int e = -1;
      float w = 0.0f;
      __syncwarp();
      choose(p, t, reinterpret_cast<uint32_t*>(ring), e, w);
      const int at = t * p.k + lane;
      if (lane < p.k) {
        if (alone) {
          pid[at] = e, pw[at] = w;
        } else {
#pragma unroll 1
          for (int d = 0; d < kRanks; ++d) {
            ptx::st_cluster_u32(ptx::mapa(ptx::smem_u32(pid + at), d), e);
            ptx::st_cluster_u32(ptx::mapa(ptx::smem_u32(pw + at), d), __float_as_uint(w));
          }
        }
        if (cluster == 0 && (!alone || rank == 0)) p.ids[at] = e, p.weights[at] = w;
      }
    }
  } else {
#pragma unroll 1
    for (int i = tid; i < P; i += kThreads) {
      const int e = p.ids[i];
      pid[i] = e >= 0 && e < p.E ? e : -1;
      pw[i] = p.weights[i];
    }
  }
  if (p.logits && !alone) {
    ptx::cluster_arrive();
    ptx::cluster_wait();
  } else {
    __syncthreads();
  }
  ptx::cluster_arrive();  // (waited for before h is written to another CTA)

  // The pairs sorted by expert, in order, and cut into slabs of at most SP pairs of one
  // expert (slab[]: its expert and its first pair in the sorted list).
  if (warp == 0) {
#pragma unroll 1
    for (int i0 = 0; i0 < P; i0 += 32) {
      const int e = i0 + lane < P ? pid[i0 + lane] : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, e);
      const int before = __popc(same & ((1u << lane) - 1u));
      if (e >= 0) place[i0 + lane] = sh.count[e] + before;
      __syncwarp();
      if (e >= 0 && before == 0) sh.count[e] += __popc(same);
      __syncwarp();
    }
    int pairs = 0, slabs = 0;
#pragma unroll 1
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int n = e0 + lane < p.E ? sh.count[e0 + lane] : 0;
      int up = n | ((n + SP - 1) / SP) << 16, mine = up;  // both sums at once
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += v;
      }
      const int first = pairs + ((up - mine) & 0xffff), s = slabs + ((up - mine) >> 16);
      if (e0 + lane < p.E) sh.first[e0 + lane] = first | s << 16;
#pragma unroll 1
      for (int q = 0; q < n; q += SP) slab[s + q / SP] = make_int2(e0 + lane, first + q);
      const int all = __shfl_sync(0xffffffffu, up, 31);
      pairs += all & 0xffff, slabs += all >> 16;
    }
    if (lane == 0) sh.n_slabs = slabs;
  }
  __syncthreads();

  // The slabs' units of 16 neurons in a row, U of them, are divided evenly among C
  // clusters: cluster i has those from U i / C on.  A part is what one cluster has of one
  // slab; a slab has at most parts_cap + 1 (C / slabs is at most parts_cap).
  const uint32_t slabs = sh.n_slabs;
  const uint32_t units = (p.F + 15u) / 16u;
  const uint32_t U = units * slabs;
  const uint32_t C = max(1u, min(min(gridDim.x / kRanks, U / kRanks), slabs * p.parts_cap));
  const auto cluster_of = [&](uint32_t u) { return static_cast<int>(((u + 1u) * C - 1u) / U); };
  const auto parts_of = [&](uint32_t s, int& first) {
    first = cluster_of(s * units);
    return cluster_of(s * units + units - 1u) - first + 1;
  };
  const auto slab_of = [&](int pair) {
    return (sh.first[pid[pair]] >> 16) + place[pair] / SP;
  };
#pragma unroll 1
  for (int i = tid; i < P; i += kThreads) {
    if (pid[i] < 0) continue;
    plist[(sh.first[pid[i]] & 0xffff) + place[i]] = i;
    int first;
    atomicAdd(&sh.live[i / p.k], parts_of(slab_of(i), first));
  }
  __syncthreads();
  // tokens without an expert
#pragma unroll 1
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    if (sh.live[t]) continue;
#pragma unroll 1
    for (int d = tid; d < p.D; d += kThreads) {
      const int64_t to = static_cast<int64_t>(t) * p.D + d;
      if (p.y_f32) static_cast<float*>(p.y)[to] = 0.0f;
      else static_cast<uint16_t*>(p.y)[to] = 0;
    }
  }

  const bool silu = p.act == TWELL_SILU;
  const bool three = p.y_f32 != 0;
  const uint32_t u_last = cluster < C ? U * (cluster + 1) / C : 0u;
#pragma unroll 1
  for (uint32_t ub = cluster < C ? U * cluster / C : 0u; ub < u_last;) {
    const uint32_t a = ub / units;
    const int e = slab[a].x, s0 = slab[a].y;
    const int ns = min(SP, (sh.first[e] & 0xffff) + sh.count[e] - s0);  // pairs of the slab
    const int nt_used = (ns + 7) / 8;
    const int u0 = ub - a * units;
    const int nu = min(u_last - a * units, units) - u0;
    int part;
    parts_of(a, part);
    part = cluster - part;
    ub += nu;
    const int rounds = ((nu + kRanks - 1) / kRanks + UR - 1) / UR;
    const int r0 = u0 + nu * rank / kRanks, r1 = u0 + nu * (rank + 1) / kRanks;  // own units
    const int64_t base = static_cast<int64_t>(e) * p.F;
    {
      const uint16_t* xt[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n)
        xt[n] = p.x + static_cast<int64_t>(plist[s0 + min(8 * n + g, ns - 1)] / p.k) * p.D;
      for (int i = tid; i < SP * ystride; i += kThreads) yacc[i] = 0.0f;
#pragma unroll 1
      for (int round = 0; round < rounds; ++round) {
        const int ua = r0 + round * UR;
        const int j0 = ua * 16;                                  // first neuron
        const int nj = max(0, min(min(ua + UR, r1) * 16, p.F) - j0);  // neurons of this round

        // (SiLU: the rows of Wd that the cluster's neurons of this round need, on their way)
        if (silu && width > 0) {
#pragma unroll 1
          for (int i = tid; i < SLOTS; i += kThreads) {
            const int q = i / RM, first = (u0 + nu * q / kRanks + round * UR) * 16 + i % RM;
            if (first < min((u0 + nu * (q + 1) / kRanks) * 16, p.F))
              F::ahead(p, base + first, col0, width);
          }
        }

        // ---- gate and up sums (with ReLU the gate's, then up of the active neurons):
        // `share` warps side by side on tiles of 16 rows, the others on their columns
        int n_act = silu ? nj : 0, share = 1;
        // the sum of a tile of pairs of tiles, its half m, row r of it, pair n
        const auto sum_at = [&](int tile, int m, int r, int n) {
          const int at = (((m * NT + (n >> 3)) * 32 + (r & 7) * 4 + (n & 7) / 2) * 4) +
                         (r >> 3) * 2 + (n & 1);
          float v = 0.0f;
#pragma unroll 1
          for (int w = tile; w < kWarps; w += share)
            v += reinterpret_cast<const float*>(raw + w * RING)[at];
          return v;
        };
#pragma unroll 1
        for (int stage = 0; stage < (silu ? 1 : 2); ++stage) {
          const int count = stage ? n_act : nj;
          if (count == 0) break;
          // a warp's two tiles: the gate and up rows of the same 16 neurons, or 32 rows of one
          const int n_tiles = silu ? (count + 15) / 16 : (count + 31) / 32;
          share = n_tiles <= 2 ? n_tiles : 4;
          const int tile = warp & (share - 1);
          float acc[2][NT][4];
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int j = 0; j < 4; ++j) acc[m][n][j] = 0.0f;
          const int mat[2] = {stage, silu ? 1 : stage};
          const int row0 = silu ? 16 * tile : 32 * tile;
          int64_t at[2][2];
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = min(row0 + (silu ? 0 : 16 * m) + 8 * h + g, count - 1);
              at[m][h] = base + j0 + (stage ? sh.act[r] : r);
            }
          if (tile < n_tiles)
            F::template rows<NT, Z::RING / 2>(
                p, mat, at, warp / share, kWarps / share, ring_at, nt_used,
                [&](int n, int k) { return ld16(xt[n] + min(k, p.D - 8)); }, acc);
          __syncwarp();
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
              reinterpret_cast<float4*>(ring)[(m * NT + n) * 32 + lane] =
                  make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
          __syncthreads();
          if (silu || stage) break;
#pragma unroll 1
          for (int i = tid; i < nj * SP; i += kThreads) {
            const int r = i / SP, n = i % SP;
            if (n < ns) zb[r * (SP + 1) + n] = sum_at(r >> 5, (r >> 4) & 1, r & 15, n);
          }
          __syncthreads();
          if (warp == 0) {
            int n = 0;
#pragma unroll 1
            for (int q = lane; q - lane < nj; q += 32) {
              bool on = false;
              if (q < nj)
#pragma unroll 1
                for (int i = 0; i < ns; ++i) on |= !(zb[q * (SP + 1) + i] <= 0.0f);
              const uint32_t m = __ballot_sync(0xffffffffu, on);
              if (on) sh.act[n + __popc(m & ((1u << lane) - 1u))] = static_cast<int16_t>(q);
              n += __popc(m);
            }
            if (lane == 0) sh.n_act = n;
          }
          __syncthreads();
          n_act = sh.n_act;
        }

        // ---- h of the active neurons to all CTAs, once they are done with the last round's
        ptx::cluster_wait();
        {
          const uint32_t to = ptx::smem_u32(hb + (rank * RM) * HS);
#pragma unroll 1
          for (int i = tid; i < n_act * (SP / 4); i += kThreads) {
            const int r = i / (SP / 4), n4 = i % (SP / 4) * 4;
            if (n4 >= 8 * nt_used) continue;
            float h[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
            for (int n = n4; n < min(ns, n4 + 4); ++n) {
              const float u = silu ? sum_at(r >> 4, 1, r & 15, n)
                                   : sum_at(r >> 5, (r >> 4) & 1, r & 15, n);
              const float z = silu ? sum_at(r >> 4, 0, r & 15, n) : zb[sh.act[r] * (SP + 1) + n];
              const float v = silu ? z / (1.0f + expf(-z)) * u : z <= 0.0f ? 0.0f : z * u;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (n == n4 + j) h[j] = v;
            }
#pragma unroll
            for (int d = 0; d < kRanks; ++d)
              ptx::st_cluster_f32x4(ptx::mapa(to + 4u * (r * HS + n4), d),
                                    make_float4(h[0], h[1], h[2], h[3]));
          }
          if (tid < n_act) {
            const uint32_t ix = ptx::smem_u32(hidx + rank * RM + tid);
            const uint32_t j = j0 + (silu ? tid : sh.act[tid]);
#pragma unroll
            for (int d = 0; d < kRanks; ++d) ptx::st_cluster_u32(ptx::mapa(ix, d), j);
          }
          if (tid < kRanks)
            ptx::st_cluster_u32(ptx::mapa(ptx::smem_u32(&sh.hcnt[rank]), tid), n_act);
        }
        ptx::cluster_arrive();
        ptx::cluster_wait();

        // ---- the cluster's neurons times Wd, this CTA's columns
#pragma unroll 1
        for (int i = tid; i < SLOTS; i += kThreads) {
          const int q = i / RM, s = i % RM;
          int before = 0, total = 0;
#pragma unroll
          for (int d = 0; d < kRanks; ++d) {
            const int n = sh.hcnt[d];
            before += d < q ? n : 0;
            total += n;
          }
          if (s < sh.hcnt[q]) list[before + s] = make_int2(i, hidx[i]);
          if (i == 0) sh.total = total;
        }
        __syncthreads();
        const int total = sh.total;
        const int steps = (total + 15) / 16;
        const int side = min(kWarps, max(1, my_tiles));      // tiles side by side
        const int NS = kWarps / side;                        // warps that share a tile's neurons
        const int ct_w = warp % side, ns_w = warp / side;
        const float* h0 = hb;
#pragma unroll 1
        for (int cb = 0; cb < my_tiles && steps > 0; cb += side) {
          const int ct = cb + ct_w;
          const bool on = ct < my_tiles && ns_w < NS;
          constexpr int MT = TW / 16;
          float acc[MT][NT][4];
#pragma unroll
          for (int q = 0; q < MT; ++q)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int j = 0; j < 4; ++j) acc[q][n][j] = 0.0f;
          if (on) {
            constexpr int SB = RING / Step::BYTES;  // steps in the ring
            const int d0 = col0 + TW * ct;
            int put = 0, get = 0, st_put = ns_w;
            const auto issue = [&] {
              int64_t row[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int s = 16 * st_put + 2 * c + (i & 1) + 8 * (i >> 1);
                row[i] = s < total ? base + list[s].y : -1;
              }
              Step::copy(p, row, d0, ring_at + put * Step::BYTES);
              cp_async_commit_group();
              st_put += NS;
              put = put + 1 == SB ? 0 : put + 1;
            };
            const auto scales = [&](int st, typename Step::Scales& s) {
              const int i = 16 * st + (lane & 15);
              s.load(p, i < total ? base + list[i].y : -1, d0);
            };
            typename Step::Scales s_now, s_next, s_then;
            scales(ns_w, s_now);
            scales(ns_w + NS, s_next);
#pragma unroll 1
            for (int i = 0; i < SB - 1; ++i) issue();
#pragma unroll 1
            for (int st = ns_w; st < steps; st += NS) {
              issue();
              scales(st + 2 * NS, s_then);
              int slot[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int s = 16 * st + 2 * c + (i & 1) + 8 * (i >> 1);
                slot[i] = s < total ? list[s].x : -1;
              }
              cp_async_wait_for<SB - 1>();
              Step::template add<NT>(
                  ring_at + get * Step::BYTES, s_now, d0,
                  [&](int i, int n) {
                    return slot[i] >= 0 ? h0[slot[i] * HS + 8 * n + g] : 0.0f;
                  },
                  nt_used, three, acc);
              get = get + 1 == SB ? 0 : get + 1;
              s_now = s_next, s_next = s_then;
            }
            cp_async_wait_for<0>();
          }
#pragma unroll 1
          for (int turn = 0; turn < NS; ++turn) {
            if (on && ns_w == turn) {
#pragma unroll
              for (int q = 0; q < MT; ++q) {
                float* to[NT][4];
                float v[NT][4];  // (all loads before the stores, which might alias them)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    const int pair = 8 * n + 2 * c + (j & 1);
                    to[n][j] = yacc + pair * ystride + TW * ct + F::column(q, j / 2, g);
                    v[n][j] = *to[n][j];
                  }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                  for (int j = 0; j < 4; ++j) *to[n][j] = v[n][j] + acc[q][n][j];
              }
            }
            __syncthreads();
          }
        }
        ptx::cluster_arrive();
      }
      // ---- the slab's rows of this part, and the tokens that they complete
      __syncthreads();
#pragma unroll 1
      for (int i = tid; i < ns * (width / 4); i += kThreads) {
        const int n = i / (width / 4), d = i % (width / 4) * 4;
        const int pair = plist[s0 + n];
        const float w = pw[pair];
        const float* v = yacc + n * ystride + d;
        __stcg(reinterpret_cast<float4*>(
                   p.part + (static_cast<int64_t>(pair) * (p.parts_cap + 1) + part) * p.D + col0 +
                   d),
               make_float4(v[0] * w, v[1] * w, v[2] * w, v[3] * w));
      }
      __threadfence();
      __syncthreads();
      if (tid < ns) {
        const int t = plist[s0 + tid] / p.k;
        sh.last[tid] =
            width > 0 && atomicAdd(p.count + t * kRanks + rank, 1) + 1 == sh.live[t];
      }
      __syncthreads();
#pragma unroll 1
      for (int n = 0; n < ns; ++n) {
        if (!sh.last[n]) continue;
        __threadfence();
        const int t = plist[s0 + n] / p.k;
        if (warp == 0) {  // the token's rows of `part`, by slot and part
          const int pair = t * p.k + lane;
          int first, mine = lane < p.k && pid[pair] >= 0 ? parts_of(slab_of(pair), first) : 0;
          int upto = mine;
#pragma unroll
          for (int o = 1; o < 32; o *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
          }
#pragma unroll 1
          for (int q = 0; q < mine; ++q)
            sh.rows[upto - mine + q] = pair * (p.parts_cap + 1) + q;
          if (lane == 31) sh.n_rows = upto;
        }
        __syncthreads();
        // four groups of threads have every fourth row each
        float4* quarter = reinterpret_cast<float4*>(raw);
        const int at = tid & 63, gr = tid >> 6, n_rows = sh.n_rows;
#pragma unroll 1
        for (int d = 4 * at; d - 4 * at < width; d += 256) {
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          if (d < width) {
#pragma unroll 8
            for (int r = gr; r < n_rows; r += 4) {
              const float4 o = __ldcg(reinterpret_cast<const float4*>(
                  p.part + static_cast<int64_t>(sh.rows[r]) * p.D + col0 + d));
              v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
            }
          }
          quarter[gr * 64 + at] = v;
          __syncthreads();
          if (gr == 0 && d < width) {
#pragma unroll
            for (int i = 1; i < 4; ++i) {
              const float4 o = quarter[i * 64 + at];
              v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
            }
            const float f[4] = {v.x, v.y, v.z, v.w};
            const int64_t to = static_cast<int64_t>(t) * p.D + col0 + d;
            if (p.y_f32) store4(static_cast<float*>(p.y) + to, f);
            else store4(static_cast<uint16_t*>(p.y) + to, f);
          }
          __syncthreads();
        }
      }
      __syncthreads();
    }
  }
  ptx::cluster_wait();  // (nobody leaves while another CTA may still write to it)
}

// -------------------------------------------------------------------- host

struct Layout {
  size_t logits, count, part, total;
  int32_t parts_cap;
};

// Clusters of the experts' kernel at the most: two CTAs on each SM.
int clusters_of(const DeviceInfo& dev) {
  const int n = dev.sm_count * 2 / kRanks;
  return n < 80 ? n : 80;  // (a token is the sum of at most that many rows and top_k more)
}
constexpr size_t kTwoCtas = 107 * 1024;  // dynamic shared memory that leaves room for two

Layout layout_of(const DeviceInfo& dev, int32_t T, int32_t D, int32_t F, int32_t E, int32_t k) {
  Layout l;
  const int C = clusters_of(dev);
  // clusters an expert is divided among on average at the most: a unit of 16 neurons for
  // each CTA, and no more than leave every slot of a token one
  const int by_units = (F + 16 * kRanks - 1) / (16 * kRanks);
  l.parts_cap = by_units < C / k ? by_units : C / k;
  if (l.parts_cap < 1) l.parts_cap = 1;
  const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  l.logits = 0;
  l.count = up(sizeof(float) * T * E);
  l.part = l.count + up(sizeof(int32_t) * T * kRanks);
  l.total = l.part + sizeof(float) * T * k * (l.parts_cap + 1) * D;
  return l;
}

template <typename F, int NT>
size_t shared_bytes(int32_t D, int32_t E, int32_t P) {
  typedef Sizes<NT> Z;
  constexpr int TW = Tile<F, NT>::COLS;
  const size_t cols = TW * (((D + TW - 1) / TW + kRanks - 1) / kRanks);
  return kWarps * Z::RING * kSlotBytes +
         4 * (Z::SLOTS * Z::HS + 3 * Z::SLOTS + Z::RM * (Z::SP + 1) + Z::SP * (cols + 1) +
              4 * P + 2 * (E + P / Z::SP));
}

template <typename F, int NT>
twell_status launch_experts(const MoeParams& p, const DeviceInfo& dev, cudaStream_t s) {
  static std::atomic<uint64_t> set{0};
  static DeviceValue resident[2];
  const int limit = dev.max_smem_optin - 8192;
  const int64_t pairs = static_cast<int64_t>(p.T) * p.k;
  const size_t smem = shared_bytes<F, NT>(p.D, p.E, static_cast<int32_t>(pairs));
  cudaLaunchConfig_t cfg =
      launch_config(dim3(kRanks * clusters_of(dev)), dim3(kThreads), smem, s);
  // as many clusters as run at once: with two CTAs on an SM, or one where its shared
  // memory holds no more
  const bool big = smem > kTwoCtas;
  const int most = resident[big].get(dev, [&]() -> int {
    int n = 0;
    cudaLaunchConfig_t ask = cfg;
    ask.dynamicSmemBytes = big ? limit : kTwoCtas;
    if (!cuda_ok(cudaFuncSetAttribute(reinterpret_cast<const void*>(experts_kernel<F, NT>),
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, limit)) ||
        !cuda_ok(cudaOccupancyMaxActiveClusters(&n, experts_kernel<F, NT>, &ask)))
      return -1;
    return n;
  });
  if (most < 0) return TWELL_ERR_CUDA;
  const int64_t units = ((pairs < p.E ? pairs : p.E) + pairs / Sizes<NT>::SP) *
                        ((static_cast<int64_t>(p.F) + 15) / 16);
  int64_t clusters = units / kRanks;  // one unit a CTA at the least
  if (clusters > most) clusters = most;
  if (clusters > clusters_of(dev)) clusters = clusters_of(dev);
  if (clusters < 1) clusters = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * kRanks));
  cudaLaunchAttribute attr = overlapped();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return launch_large(experts_kernel<F, NT>, limit, cfg, dev, set, p);
}

template <typename F>
twell_status launch_experts(const MoeParams& p, const DeviceInfo& dev, cudaStream_t s) {
  // tiles of eight pairs that an expert's weights are read once for: all its tokens
  // where they are eight at most, else by the pairs an expert has on average (one with
  // more reads its weights again, from the second cache); h and the sums of a slab's columns
  // are held in shared memory, which bounds them for wide rows
  const int64_t mean = static_cast<int64_t>(p.T) * p.k / p.E;
  if (p.T <= 8 || p.D > 8192) return launch_experts<F, 1>(p, dev, s);
  return mean <= 12 ? launch_experts<F, 2>(p, dev, s) : launch_experts<F, 4>(p, dev, s);
}

bool sizes_ok(int32_t T, int32_t D, int32_t F, int32_t E, int32_t k) {
  return T >= 0 && D >= 8 && D % 8 == 0 && F >= 1 && E >= 1 && k >= 1;
}
bool within_limits(int32_t T, int32_t D, int32_t E, int32_t k) {
  return T <= kMaxTokens && D <= kMaxWidth && E <= kMaxExperts && k <= kMaxTop &&
         static_cast<int64_t>(T) * k <= kMaxPairs;
}
// (units of 16 neurons of every slab of eight pairs, times the clusters, are counted in 32 bits)
bool neurons_ok(int32_t F, int32_t E) {
  return static_cast<int64_t>(E + kMaxPairs / 8) * ((static_cast<int64_t>(F) + 15) / 16) <= 1 << 25;
}

}  // namespace
}  // namespace twell

extern "C" size_t twell_moe_decode_workspace(int32_t T, int32_t D, int32_t F, int32_t E,
                                             int32_t top_k) {
  using namespace twell;
  if (!sizes_ok(T, D, F, E, top_k) || !within_limits(T, D, E, top_k) || !neurons_ok(F, E))
    return 0;
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
  if (!within_limits(T, D, E, top_k) || !neurons_ok(F, E)) return TWELL_ERR_UNSUPPORTED;
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
