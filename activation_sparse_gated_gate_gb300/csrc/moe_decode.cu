// A mixture-of-experts layer for a few tokens: the router's logits and choice, the chosen
// experts' gated FFNs (bf16 or 4-bit weights) and their weighted sum.
//
//   logits = x W_r^T;  the k largest of a token (ties: the lowest expert), p = softmax
//   y[t] = sum over the token's k slots of p sum_j a(x . Wg[e][j]) (x . Wu[e][j]) Wd[e][j]
//
// Three kernels, each launched while the one before runs:
//   router   the logits in fp32 FMAs (a choice must not hang on a tensor core's rounding), and
//            the counters of the last kernel set to zero (without a router that alone).  More
//            tokens than eight: a fourth kernel makes the choice, a warp a token; of fewer
//            every CTA of the next makes it (a launch costs 2 us, the choice 3 in either)
//   neurons  the (token, slot) pairs sorted by expert into slabs of up to 8 NT; the slabs'
//            neurons divided evenly among the CTAs, a CTA's columns among its warps; h = a(gate) up
//            to memory.  With ReLU a neuron whose gate is not positive for any token of the
//            slab is dropped after its gate sum: its rows of Wu and Wd are not read
//   down     a CTA a slab, a tile of columns and a part of the neurons: h Wd, its eight warps
//            side by side on columns or on every second, fourth or eighth step of 16 neurons,
//            and the token's sum by whoever completes a tile of it (a counter), in slot order:
//            results do not depend on who it is
// The sums over D run on mma.sync with 16 neurons as A and up to 8 NT pairs as B (rows.cuh);
// those over neurons with 16 columns of Wd as A and h as B in three bf16 parts, whose
// sum is h's 24 bits: one part would cost y 2^-9 of an element's size.  mma.sync and not tcgen05:
// 4-bit codes are unpacked in registers, where its operands come from, and eight to sixteen
// pairs of an expert leave the tensor pipe idle either way (17 to 25 % of its cycles).
//   What bounds it (E = 64, D = 2048, F = 1024, 8 experts a token, weights from memory):
//   * one token: the chain of launches, dependent reads and barriers, 25 us in bf16 with
//     1 % of the neurons active (34 MB read, 5 us of the stream), 26 in 4 bits with all
//   * 64 tokens, bf16: the stream, 805 MB in 173 us (4.65 TB/s; neurons 5.1, down 4.1 by themselves)
//   * 64 tokens, 4 bits: instructions, 5 to 8 a weight for unpacking, split parts, addresses and the
//     fp32 additions, with registers for 16 warps an SM (a few more are wanted and spilled, up
//     to 108 bytes a thread with groups of 128, 276 of 32), which issue in half of the cycles: 149 us
//     (with SiLU 135; groups of 64 145, of 32 163)
//   Figures below that weigh one form against another are of the time of the choice.
//   A form in two kernels (clusters of 8 CTAs that exchanged h through shared memory and
// summed their columns) took as long for a token and 364 us (bf16) and 407 (4 bits) for 64: its
// phases waited for one another.
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "int4.cuh"
#include "ptx.cuh"
#include "rows.cuh"
#include "vec.cuh"

namespace twell {
namespace {

template <int N>
using Count = std::integral_constant<int, N>;

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
  int32_t* count;  // counters of the down kernel, zeroed here
  int32_t counters;
};

// The logits of EX experts for TT tokens: its four warps take every fourth 256 columns.
template <typename W, int EX, int TT>
__global__ void __launch_bounds__(128) router_kernel(const RouterParams p) {
  constexpr int N = EX * TT;
  ptx::grid_launch_next();
  for (int i = blockIdx.x * 128 + threadIdx.x; i < p.counters; i += gridDim.x * 128)
    p.count[i] = 0;
  if (!p.w) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int eg = (p.E + EX - 1) / EX;
  const int e0 = blockIdx.x % eg * EX, t0 = blockIdx.x / eg * TT;
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.0f;
  const W* w = static_cast<const W*>(p.w);
#pragma unroll(N == 1 ? 2 : 1)
  for (int k = 256 * warp + 8 * lane; k < p.D; k += 1024) {
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
        for (int j = 0; j < 8; ++j)
          acc[e * TT + t] = fmaf(wf[e][j], xf[j], acc[e * TT + t]);
    }
  }
  __shared__ float sum[4][N];
  const float v = over_warp(acc, [](float a, float b) { return a + b; });
  if (lane % (32 / N) == 0) sum[warp][lane / (32 / N)] = v;
  __syncthreads();
  const int e = e0 + threadIdx.x / TT, t = t0 + threadIdx.x % TT;
  if (threadIdx.x < N && e < p.E && t < p.T)
    p.logits[static_cast<int64_t>(t) * p.E + e] = sum[0][threadIdx.x] + sum[1][threadIdx.x] +
                                                  sum[2][threadIdx.x] + sum[3][threadIdx.x];
}

// ------------------------------------------------------------------ experts

// What the neurons kernel leaves for the down kernel, in the workspace: the slabs
// (expert, first pair in the sorted list, pairs, first tile of h) and the list.
struct Plan {
  int32_t* n_slabs;
  int4* slab;
  int32_t* list;      // [T k] pairs, sorted by expert
  int32_t* live;      // [T] slots that have an expert
  uint16_t* masks;    // [slabs][units] ReLU: a bit for each active neuron of a unit of 16
  // h of each eight pairs of a slab, one after the other ([tile][16 units][8]): fp32 (4-bit
  // weights), or three planes of bf16 whose sum it is, `plane` elements apart
  void* h;
  int64_t plane;
};

struct MoeParams {
  const uint16_t* x;
  int32_t T, D, F, E, k;
  const float* logits;     // NULL: ids and weights are given
  int32_t* ids;            // [T][k]
  float* weights;
  int32_t renormalise, act;
  const uint16_t* w[3];    // gate, up, down: bf16,
  Int4View q[3];           // or 4 bits
  Plan plan;
  float* part;             // [T k][splits][D]
  int32_t side;            // warps side by side on columns in the down kernel: 1, 2, 4 or 8
  int32_t* count;          // [T][tiles]
  void* y;
  int32_t y_f32;
};

// What is left of a value behind its upper half.
__device__ __forceinline__ float behind(float a) {
  return a - __uint_as_float(__float_as_uint(a) & 0xffff0000u);
}

// Two values as three bf16 each, whose sum they are (to their 24 bits).
__device__ __forceinline__ void split(float a, float b, uint32_t (&o)[3]) {
  o[0] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
  const float inf = __uint_as_float(0x7f800000u);
  a = fabsf(a) == inf ? 0.0f : behind(a), b = fabsf(b) == inf ? 0.0f : behind(b);
  o[1] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
  o[2] = bf16x2(behind(a), behind(b));
}

// The same for weights that may be infinite: a part of zero times an infinity would be NaN where
// the value times it is an infinity, so that no part of a value is zero unless the value is: it
// is the least bf16, 2^-133, of its sign instead, a step of the grid that the parts lie on.
__device__ __forceinline__ void split_nonzero(float a, float b, uint32_t (&o)[3]) {
  split(a, b, o);
  const uint32_t lo = a != 0.0f ? (__float_as_uint(a) >> 16 & 0x8000u) | 1u : 0u;
  const uint32_t hi = b != 0.0f ? (__float_as_uint(b) & 0x80000000u) | 0x10000u : 0u;
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    if ((o[q] & 0x7fffu) == 0u) o[q] = (o[q] & 0xffff0000u) | lo;
    if ((o[q] & 0x7fff0000u) == 0u) o[q] = (o[q] & 0xffffu) | hi;
  }
}

// d += a times the values that b0, b1 are split into, the small ones first.  The tensor core's
// additions truncate: its sums are of 16 neurons each, and fp32 additions that round take them
// further (one chain of it through all of F = 14336 was up to 1.1e-4 off, this 4e-6).
__device__ __forceinline__ void mma_split(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, const uint32_t (&b0)[3],
                                          const uint32_t (&b1)[3]) {
  float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  mma16816(part, a0, a1, a2, a3, b0[2], b1[2]);
  mma16816(part, a0, a1, a2, a3, b0[1], b1[1]);
  mma16816(part, a0, a1, a2, a3, b0[0], b1[0]);
#pragma unroll
  for (int j = 0; j < 4; ++j) d[j] += part[j];
}

__device__ __forceinline__ uint64_t offset(int row, int64_t pitch) {
  return static_cast<uint64_t>(static_cast<uint32_t>(row)) * static_cast<uint32_t>(pitch);
}
__device__ __forceinline__ float lds_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
// 8 x 8 tiles of bf16, transposed: rows of 16 bytes at the addresses of lanes 0 to 7, 8 to 15 ...
__device__ __forceinline__ void ldmatrix_x2_t(uint32_t at, uint32_t& a, uint32_t& b) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];"
               : "=r"(a), "=r"(b)
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_t(uint32_t at, uint32_t& a, uint32_t& b, uint32_t& c,
                                              uint32_t& d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(at)
               : "memory");
}

// A step of the sums over neurons: 16 of them by a tile of columns.  Lane (g, c) uses the
// neurons 2 c, 2 c + 1, 2 c + 8, 2 c + 9, 16 bytes of bf16 each or 8 of 4-bit codes.  The warp
// copies them into a slot of its ring by whole lines (row_of(r): row of the r-th neuron; lanes that
// are neighbours have neighbouring pieces), 16-byte pieces swizzled so that the lanes' reads
// meet no bank twice.  Of 4-bit rows lanes 0 to 15 also load the scales of one neuron each, a
// step or two ahead.  Of neurons behind the last, as of h, zeros are copied (4-bit codes repeat
// the last one's, with a scale of 0: a scale of its own may be an infinity); columns behind D
// repeat some of the row and are left out at the end.
struct Bf16Step {
  static constexpr int BYTES = 2 * kSlotBytes;
  // where the warp's columns begin in row `base`
  struct Origin {
    const uint16_t* w;
    __device__ __forceinline__ Origin(const MoeParams& p, int64_t base, int d0)
        : w(p.w[2] + base * p.D + min(d0 + 8 * static_cast<int>(threadIdx.x & 7), p.D - 8)) {}
  };
  struct Scales {
    __device__ __forceinline__ void load(const MoeParams&, const Origin&, int) {}
    __device__ __forceinline__ void none() {}
  };
  // piece g of neuron r
  static __device__ __forceinline__ uint32_t at(int r, int g) {
    return 128 * r + 16 * (g ^ (r & 6));
  }
  // (of a step's neurons there are the first `have`)
  template <typename R>
  static __device__ __forceinline__ void copy(const MoeParams& p, const Origin& o, R row_of,
                                              int have, uint32_t slot) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * i + (lane >> 3);
      ptx::cp_async16(slot + at(r, lane & 7), o.w + offset(row_of(r), p.D), r < have ? 16 : 0);
    }
  }
  // h of a chunk in shared memory: [part][tile][neuron][8 pairs] of bf16
  static constexpr int H_ROW = 16;
  template <int NU, int NT, int CHUNK>
  static __device__ __forceinline__ void add(uint32_t slot, const Scales&, uint32_t hs, int st,
                                             float (&acc)[4][NT][4]) {
    const int lane = threadIdx.x & 31;
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = lds16(slot + at(2 * (lane & 3) + (i & 1) + 8 * (i >> 1), lane >> 2));
    const uint32_t* v0 = &v[0].x;
    const uint32_t* v1 = &v[1].x;
    const uint32_t* v2 = &v[2].x;
    const uint32_t* v3 = &v[3].x;
    uint32_t b0[NU][3], b1[NU][3];
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      // (lanes 16 to 31: the rows of the second part)
      const uint32_t from = hs + ((lane >> 4) * NT * CHUNK + n * CHUNK + 16 * st + (lane & 15)) * H_ROW;
      ldmatrix_x4_t(from, b0[n][0], b1[n][0], b0[n][1], b1[n][1]);
      ldmatrix_x2_t(from + 2 * NT * CHUNK * H_ROW, b0[n][2], b1[n][2]);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t a0 = __byte_perm(v0[q], v1[q], 0x5410), a1 = __byte_perm(v0[q], v1[q], 0x7632),
                     a2 = __byte_perm(v2[q], v3[q], 0x5410), a3 = __byte_perm(v2[q], v3[q], 0x7632);
#pragma unroll
      for (int n = 0; n < NU; ++n) {
        mma_split(acc[q][n], a0, a1, a2, a3, b0[n], b1[n]);
      }
    }
  }
};
template <int G32>
struct FourStep {
  static constexpr int BYTES = kSlotBytes;
  typedef BlockScales<G32> One;
  struct Origin {
    const uint8_t* code;
    const uint16_t* scale;
    const uint8_t* zero;
    __device__ __forceinline__ Origin(const MoeParams& p, int64_t base, int d0) {
      const Int4View& w = p.q[2];
      const int block = d0 < p.D ? d0 / kInt4Block : 0;
      code = w.code + base * w.pitch + block * kInt4Bytes + 16 * (threadIdx.x & 3);
      const int64_t at = base * w.held + block * (4 / G32);
      scale = w.scale + at;
      zero = (w.zero ? w.zero : w.code) + at;
    }
  };
  struct Scales {
    One one;  // of neuron `lane & 15`
    __device__ __forceinline__ void load(const MoeParams& p, const Origin& o, int row) {
      const uint64_t at = offset(row, p.q[2].held);
      one.load(o.scale + at, p.q[2].zero ? o.zero + at : nullptr);
    }
    __device__ __forceinline__ void none() { one.none(); }
  };
  // where a neuron's h is: those of the four lanes of a quarter warp in different banks
  static __device__ __forceinline__ int place(int r) { return r ^ (r >> 2 & 1); }
  // 16-byte piece q of neuron r: even neurons in the slot's first half
  static __device__ __forceinline__ uint32_t at(int r, int q) {
    const int pos = (r >> 1) + 8 * (r & 1);
    return 64 * pos + 16 * (q ^ (pos & 2));
  }
  template <typename R>
  static __device__ __forceinline__ void copy(const MoeParams& p, const Origin& o, R row_of,
                                              int, uint32_t slot) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 8 * i + (lane >> 2);
      ptx::cp_async<16>(slot + at(r, lane & 3), o.code + offset(row_of(r), p.q[2].pitch));
    }
  }
  // h of a chunk in shared memory: [tile][place(neuron)][8 pairs] of fp32
  static constexpr int H_ROW = 32;
  template <int NU, int NT, int CHUNK>
  static __device__ __forceinline__ void add(uint32_t slot, const Scales& sc, uint32_t hs, int st,
                                             float (&acc)[8][NT][4]) {
    const int lane = threadIdx.x & 31, c = lane & 3;
    const uint32_t h0 = hs + 16 * st * H_ROW + (lane >> 2) * 4;
    const auto h_of = [&](int i, int n) {
      return lds_f32(h0 + (n * CHUNK + place(2 * c + (i & 1)) + 8 * (i >> 1)) * H_ROW);
    };
    uint32_t v[4][2];
    One s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                   : "=r"(v[i][0]), "=r"(v[i][1])
                   : "r"(slot + at(2 * c + (i & 1) + 8 * (i >> 1), lane >> 3) + (lane >> 2 & 1) * 8)
                   : "memory");
      s[i].from_lane(sc.one, 2 * c + (i & 1) + 8 * (i >> 1));
    }
    uint32_t b0[NU][3], b1[NU][3];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int gk = k / G32;
      if (k % G32 == 0) {
#pragma unroll
        for (int n = 0; n < NU; ++n) {
          split(h_of(0, n) * s[0].scale(gk), h_of(1, n) * s[1].scale(gk), b0[n]);
          split(h_of(2, n) * s[2].scale(gk), h_of(3, n) * s[3].scale(gk), b1[n]);
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
        for (int n = 0; n < NU; ++n) {
          mma_split(acc[2 * k + q][n], a0, a1, a2, a3, b0[n], b1[n]);
        }
      }
    }
  }
};

// The two forms of weights: the sums over the blocks b0 to b1 of two tiles of rows (at[m][h]:
// this lane's of matrix mat[m]), the step above, and where in a warp's sums of eight pairs
// ([16 outputs q][2 h + pair & 1][4 g + pair / 2]; row g + 8 h of the q-th 16) columns are.
struct Bf16 {
  static constexpr bool FOUR = false;
  static constexpr int COLS = 64;  // of a step's tile
  typedef Bf16Step Step;
  template <int NT, int S, typename X>
  static __device__ __forceinline__ void rows(const MoeParams& p, const int (&mat)[2],
                                              const int64_t (&at)[2][2], int b0, int b1,
                                              uint32_t ring, int nt, X x, float (&acc)[2][NT][4]) {
    const uint16_t* const from[2][2] = {
        {p.w[mat[0]] + at[0][0] * p.D, p.w[mat[0]] + at[0][1] * p.D},
        {p.w[mat[1]] + at[1][0] * p.D, p.w[mat[1]] + at[1][1] * p.D}};
    bf16_rows<2, NT, S>(from, p.D, b0, b1, ring, nt, x, acc);
  }
  // the t-th four columns, the first of them of pair 0, and how far on the others are
  static __device__ __forceinline__ int columns(int t) { return 8 * (t & 7) + 4 * (t >> 3); }
  static __device__ __forceinline__ int first_of(int t) { return 256 * (t >> 3) + 4 * (t & 7); }
  static __device__ __forceinline__ int next(int j) { return 64 * j; }
};
template <int G>
struct Four {
  static constexpr bool FOUR = true;
  static constexpr int COLS = 128;
  typedef FourStep<G> Step;
  template <int NT, int S, typename X>
  static __device__ __forceinline__ void rows(const MoeParams& p, const int (&mat)[2],
                                              const int64_t (&at)[2][2], int b0, int b1,
                                              uint32_t ring, int nt, X x, float (&acc)[2][NT][4]) {
    const Int4View* const from[2] = {&p.q[mat[0]], &p.q[mat[1]]};
    if (NT > 1 && nt == 1) int4_rows<G, 2, 1, NT, S>(from, at, p.D, b0, b1, ring, x, acc);
    else int4_rows<G, 2, NT, NT, S>(from, at, p.D, b0, b1, ring, x, acc);
  }
  static __device__ __forceinline__ int columns(int t) {
    return 32 * (t >> 3) + 8 * (t & 3) + (t & 4);
  }
  static __device__ __forceinline__ int first_of(int t) { return 128 * (t >> 2) + 8 * (t & 3); }
  static __device__ __forceinline__ int next(int j) { return 64 * (j >> 1) + 4 * (j & 1); }
};

// The k largest of a token's logits and their weights, by a warp: slot `lane` of them.  EJ: 32s
// of experts in a lane's registers.
template <int EJ>
__device__ __forceinline__ void choose(const MoeParams& p, int t, int& chosen, float& weight) {
  const int lane = threadIdx.x & 31;
  const float* logits = p.logits + static_cast<int64_t>(t) * p.E;
  const auto float_of = [](uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
  };
  bool nan = false;
  uint32_t key[EJ], best = 0u;  // ordered as the logits are; 1: NaN, 0: taken or none
#pragma unroll
  for (int j = 0; j < EJ; ++j) {
    const int e = 32 * j + lane;
    key[j] = 0u;
    if (e < p.E) {
      const float v = __ldcg(logits + e) + 0.0f;  // (adding zero makes one zero of two)
      const uint32_t b = __float_as_uint(v);
      const bool bad = v != v;
      nan |= bad;
      key[j] = bad ? 1u : b & 0x80000000u ? ~b : b | 0x80000000u;
    }
    best = max(best, key[j]);
  }
  nan = __any_sync(0xffffffffu, nan);
  float top = 0.0f, sum = 0.0f, mine = 0.0f;
#pragma unroll 1
  for (int s = 0; s < p.k; ++s) {
    const uint32_t most = __reduce_max_sync(0xffffffffu, best);
    if (s == 0) {
      top = float_of(most);
      if (!p.renormalise)
#pragma unroll
        for (int j = 0; j < EJ; ++j)
          if (32 * j + lane < p.E) sum += expf(float_of(key[j]) - top);
    }
    // the lowest expert that has it is taken
    int at = 0x7fffffff;
    if (best == most)
#pragma unroll
      for (int j = EJ - 1; j >= 0; --j)
        if (key[j] == most) at = 32 * j + lane;
    const int e = __reduce_min_sync(0xffffffffu, at);
    if (lane == s) chosen = e, mine = float_of(most);
    if (at == e) {
      best = 0u;
#pragma unroll
      for (int j = 0; j < EJ; ++j) {
        if (32 * j + lane == e) key[j] = 0u;
        best = max(best, key[j]);
      }
    }
  }
  weight = lane < p.k ? expf(mine - top) : 0.0f;
  weight /= warp_sum(p.renormalise ? weight : sum);
  if (nan) weight = __uint_as_float(0x7fc00000u);
}
__device__ __forceinline__ void choose(const MoeParams& p, int t, int& chosen, float& weight) {
  if (p.E <= 64) choose<2>(p, t, chosen, weight);
  else if (p.E <= 128) choose<4>(p, t, chosen, weight);
  else choose<kMaxExperts / 32>(p, t, chosen, weight);
}

// More tokens than a CTA has warps: their choice, a warp a token.
__global__ void __launch_bounds__(kThreads) choose_kernel(const __grid_constant__ MoeParams p) {
  ptx::grid_launch_next();
  ptx::grid_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = blockIdx.x * kWarps + warp;
  if (t >= p.T) return;
  int e = -1;
  float w = 0.0f;
  choose(p, t, e, w);
  if (lane < p.k) p.ids[t * p.k + lane] = e, p.weights[t * p.k + lane] = w;
}

template <bool FOUR, int NT>
struct Sizes {
  static constexpr int SP = 8 * NT;              // pairs (token, slot) of an expert at a time
  static constexpr int UR = 8;                   // units of 16 neurons of a CTA at a time
  static constexpr int RM = 16 * UR;
  static constexpr int ZP = NT == 1 ? 8 : 24;    // between neurons' gate sums (no bank twice)
  // of a warp, neurons kernel (4-bit rows, bound by instructions, want no more on its way: 64
  // tokens 166 us, 169 with 6)
  static constexpr int RING = (FOUR ? 4 : 6) * kSlotBytes;
  static constexpr int CHUNK = 1024 / NT;        // neurons of h in shared memory
  // of a warp, down kernel (64 tokens, 4 bits: 144.8 us, 145.8 with 4, 149.1 with 6; bf16 170,
  // 173 with 4)
  static constexpr int RING2 = (FOUR ? 2 : 6) * kSlotBytes;
};

template <typename F, int NT>
__global__ void __launch_bounds__(kThreads, 2)
    neurons_kernel(const __grid_constant__ MoeParams p) {
  typedef Sizes<F::FOUR, NT> Z;
  constexpr int SP = Z::SP, UR = Z::UR, RM = Z::RM, RING = Z::RING, ZP = Z::ZP;
  extern __shared__ __align__(16) uint8_t raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2;
  const int P = p.T * p.k;
  // Each warp's ring, which also holds the sums that it hands to the others (those of a
  // first of two tiles: `firsts`).
  uint8_t* ring = raw + warp * RING;
  const uint32_t ring_at = ptx::smem_u32(ring);
  constexpr int FIRST = 1024 * NT;
  static_assert(FIRST <= RING, "a warp's sums");
  uint8_t* firsts = raw + kWarps * RING;
  int4* slab = reinterpret_cast<int4*>(firsts + kWarps * FIRST);  // [E + P / SP]
  float* zb = reinterpret_cast<float*>(slab + p.E + P / SP);      // [RM][ZP] gate sums (ReLU)
  int32_t* count = reinterpret_cast<int32_t*>(zb + RM * ZP);      // [E] pairs of an expert
  int32_t* pid = count + p.E;                         // [P]
  int32_t* plist = pid + P;                           // [P] pairs by expert
  int32_t* place = plist + P;                         // [P] a pair's among its expert's
  int32_t* live = place + P;                          // [T]
  __shared__ int16_t act[RM];                         // active rows of this round
  __shared__ uint32_t sh_mask[kWarps];                // those of a unit
  __shared__ int32_t sh_slabs, sh_full;

  ptx::grid_launch_next();
  for (int i = tid; i < p.E; i += kThreads) count[i] = 0;
  for (int i = tid; i < p.T; i += kThreads) live[i] = 0;
  ptx::grid_wait();

  // ---- the choice (of a few tokens: every CTA for itself), and the pairs by expert
  if (p.logits && p.T <= kWarps) {
    if (warp < p.T) {
      int e = -1;
      float w = 0.0f;
      choose(p, warp, e, w);
      if (lane < p.k) {
        const int at = warp * p.k + lane;
        pid[at] = e;
        if (blockIdx.x == 0) p.ids[at] = e, p.weights[at] = w;
      }
    }
  } else {
#pragma unroll 1
    for (int i = tid; i < P; i += kThreads) {
      const int e = __ldcg(p.ids + i);
      pid[i] = e >= 0 && e < p.E ? e : -1;
    }
  }
  __syncthreads();
  if (warp == 0) {
#pragma unroll 1
    for (int i0 = 0; i0 < P; i0 += 32) {
      const int e = i0 + lane < P ? pid[i0 + lane] : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, e);
      const int before = __popc(same & ((1u << lane) - 1u));
      if (e >= 0) place[i0 + lane] = count[e] + before;
      __syncwarp();
      if (e >= 0 && before == 0) count[e] += __popc(same);
      __syncwarp();
    }
    // the slabs; of two tiles, those that need both first (what is left for the end is short)
    const auto both = [](int n) { return NT == 1 ? (n + SP - 1) / SP : n / SP + (n % SP > SP / 2); };
    int full = 0;
    if (NT > 1) {
#pragma unroll 1
      for (int e = lane; e < p.E; e += 32) full += both(count[e]);
      full = __reduce_add_sync(0xffffffffu, full);
    }
    int sums = 0;  // of pairs, full slabs (from bit 12) and others (from bit 20)
#pragma unroll 1
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane, n = e < p.E ? count[e] : 0;
      const int f = both(n), o = n > f * SP;
      const int mine = n | f << 12 | o << 20;
      int up = mine;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, up, d);
        if (lane >= d) up += v;
      }
      const int before = sums + up - mine;
      const int first = before & 0xfff, af = NT == 1 ? before >> 12 : before >> 12 & 0xff,
                ao = full + (before >> 20);
      if (e < p.E) count[e] = first;
#pragma unroll 1
      for (int q = 0; q < f; ++q)
        slab[af + q] = make_int4(e, first + q * SP, min(SP, n - q * SP), NT * (af + q));
      if (o) slab[ao] = make_int4(e, first + f * SP, n - f * SP, NT * full + ao - full);
      sums += __shfl_sync(0xffffffffu, up, 31);
    }
    const int slabs = NT == 1 ? sums >> 12 : full + (sums >> 20);
    if (lane == 0) sh_slabs = slabs, sh_full = NT == 1 ? slabs : full;
  }
  __syncthreads();
#pragma unroll 1
  for (int i = tid; i < P; i += kThreads)
    if (pid[i] >= 0) {
      plist[count[pid[i]] + place[i]] = i;
      atomicAdd(&live[i / p.k], 1);
    }
  __syncthreads();
  const int slabs = sh_slabs;
  if (blockIdx.x == 0) {  // for the down kernel
#pragma unroll 1
    for (int i = tid; i < slabs; i += kThreads) p.plan.slab[i] = slab[i];
#pragma unroll 1
    for (int i = tid; i < P; i += kThreads) p.plan.list[i] = plist[i];
#pragma unroll 1
    for (int i = tid; i < p.T; i += kThreads) p.plan.live[i] = live[i];
    if (tid == 0) *p.plan.n_slabs = slabs;
  }
  // tokens without an expert
#pragma unroll 1
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    if (live[t]) continue;
#pragma unroll 1
    for (int d = tid; d < p.D; d += kThreads) {
      const int64_t to = static_cast<int64_t>(t) * p.D + d;
      if (p.y_f32) static_cast<float*>(p.y)[to] = 0.0f;
      else static_cast<uint16_t*>(p.y)[to] = 0;
    }
  }

  // ---- the slabs' units of 16 neurons in a row, divided evenly among the CTAs
  const bool silu = p.act == TWELL_SILU;
  const uint32_t units = (p.F + 15u) / 16u, U = units * slabs, C = min(gridDim.x, U);
  const auto first_unit = [&](uint32_t i) {  // of CTA i
    // what a unit of a slab of two tiles costs, and of one (4 bits, 64 tokens: 149 us, 156 where
    // both count the same; bf16 170 and 172)
    constexpr uint32_t FULL = F::FOUR ? 4 : 8, OTHER = F::FOUR ? 3 : 7;
    const uint32_t full = units * sh_full, all = full * FULL + (U - full) * OTHER;
    const uint32_t at = static_cast<uint32_t>(static_cast<uint64_t>(all) * i / C);
    return at <= full * FULL ? at / FULL : full + (at - full * FULL) / OTHER;
  };
  const uint32_t u_last = blockIdx.x < C ? first_unit(blockIdx.x + 1u) : 0u;
#pragma unroll 1
  for (uint32_t ub = blockIdx.x < C ? first_unit(blockIdx.x) : 0u; ub < u_last;) {
    const uint32_t a = ub / units;
    const int e = slab[a].x, s0 = slab[a].y, ns = slab[a].z, tile0 = slab[a].w;
    const int u0 = ub - a * units;
    const int nu = min(min(u_last - a * units, units) - u0, static_cast<uint32_t>(UR));
    ub += nu;
    const int nt_used = (ns + 7) / 8;
    const int64_t base = static_cast<int64_t>(e) * p.F;
    const int j0 = u0 * 16, nj = min(nu * 16, p.F - j0);  // neurons of this round
    const uint16_t* xt[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
      xt[n] = p.x + static_cast<int64_t>(plist[s0 + min(8 * n + g, ns - 1)] / p.k) * p.D;

    // ---- gate and up sums (with ReLU the gate's, then up of the active neurons): tiles of
    // two times 16 rows, their blocks of 128 columns divided evenly among the warps
    int n_act = silu ? nj : 0, n_tiles = 1, jobs = 0;
    const int nb = (p.D + kInt4Block - 1) / kInt4Block, c = lane & 3;
    // The sum of a tile's half m for the eight pairs n: rows g and g + 8 (x, y and z, w) of
    // its 16, pairs 2 c and 2 c + 1.  Warp w looks after the w-th 16 rows.
    const auto sum_of = [&](int tile, int m, int n) {
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
      for (int w = kWarps * tile / n_tiles; w * n_tiles < kWarps * (tile + 1); ++w) {
        const int from = jobs * w / kWarps, to = jobs * (w + 1) / kWarps;
        if (from == to || from >= (tile + 1) * nb || to <= tile * nb) continue;
        const uint8_t* at = to > (tile + 1) * nb ? firsts + w * FIRST : raw + w * RING;
        const float4 u = reinterpret_cast<const float4*>(at)[(m * NT + n) * 32 + lane];
        v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
      }
      return v;
    };
#pragma unroll 1
    for (int stage = 0;; ++stage) {
      const int rows = stage ? n_act : nj;
      // a warp's two tiles: the gate and up rows of the same 16 neurons, or 32 rows of one
      n_tiles = silu ? (rows + 15) / 16 : (rows + 31) / 32;
      jobs = n_tiles * nb;
      // (a warp's share may be the end of a tile and the beginning of the next)
      const int last = jobs * (warp + 1) / kWarps;
#pragma unroll 1
      for (int job = jobs * warp / kWarps; job < last;) {
        const int tile = job / nb, b0 = job - tile * nb, b1 = min(nb, b0 + last - job);
        job += b1 - b0;
        float acc[2][NT][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[m][n][j] = 0.0f;
        const int mat[2] = {stage, silu ? 1 : stage};
        int64_t at[2][2];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = min((silu ? 16 * tile : 32 * tile + 16 * m) + 8 * h + g, rows - 1);
            at[m][h] = base + j0 + (stage ? act[r] : r);
          }
        F::template rows<NT, RING / (2 * kSlotBytes)>(
            p, mat, at, b0, b1, ring_at, nt_used,
            [&](int n, int k) { return ld16(xt[n] + min(k, p.D - 8)); }, acc);
        __syncwarp();
        float4* to = reinterpret_cast<float4*>(job < last ? firsts + warp * FIRST : ring);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            to[(m * NT + n) * 32 + lane] =
                make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
      }
      __syncthreads();
      if (silu || stage) break;
      uint32_t mask = 0u;
      if (16 * warp < nj) {
        bool lo = false, hi = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (n >= nt_used) break;
          const float4 z = sum_of(warp >> 1, warp & 1, n);
          const bool one = 8 * n + 2 * c < ns, two = 8 * n + 2 * c + 1 < ns;
          lo |= (one && !(z.x <= 0.0f)) || (two && !(z.y <= 0.0f));
          hi |= (one && !(z.z <= 0.0f)) || (two && !(z.w <= 0.0f));
          float2* to = reinterpret_cast<float2*>(zb + (16 * warp + g) * ZP + 8 * n + 2 * c);
          to[0] = make_float2(z.x, z.y);
          to[8 * ZP / 2] = make_float2(z.z, z.w);
        }
        // (ballots: the four lanes of a row beside one another)
        const uint32_t b_lo = __ballot_sync(0xffffffffu, lo), b_hi = __ballot_sync(0xffffffffu, hi);
        const uint32_t of = (lane & 8 ? b_hi : b_lo) >> (4 * (lane & 7)) & 15u;
        mask = __ballot_sync(0xffffffffu, lane < 16 && 16 * warp + lane < nj && of != 0u);
        if (lane == 0)
          p.plan.masks[static_cast<int64_t>(a) * units + u0 + warp] = static_cast<uint16_t>(mask);
      }
      if (lane == 0) sh_mask[warp] = mask;
      __syncthreads();
      n_act = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w == warp && (mask >> lane & 1u))
          act[n_act + __popc(mask & ((1u << lane) - 1u))] = static_cast<int16_t>(16 * warp + lane);
        n_act += __popc(sh_mask[w]);
      }
      __syncthreads();
      if (n_act == 0) break;
    }

    // ---- h
    const int rows = silu ? nj : n_act;
    if (16 * warp < rows) {
      const int r[2] = {16 * warp + g, 16 * warp + g + 8};
      int j[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) j[i] = silu || r[i] >= rows ? min(r[i], nj - 1) : act[r[i]];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n >= nt_used) break;
        float z[4], h[4];
        if (silu) {
          const float4 s = sum_of(warp, 0, n), v = sum_of(warp, 1, n);
          z[0] = s.x, z[1] = s.y, z[2] = s.z, z[3] = s.w;
          h[0] = v.x, h[1] = v.y, h[2] = v.z, h[3] = v.w;
#pragma unroll
          for (int i = 0; i < 4; ++i) h[i] *= z[i] / (1.0f + expf(-z[i]));
        } else {
          const float4 v = sum_of(warp >> 1, warp & 1, n);
          h[0] = v.x, h[1] = v.y, h[2] = v.z, h[3] = v.w;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            z[i] = zb[j[i >> 1] * ZP + 8 * n + 2 * c + (i & 1)];
            h[i] = z[i] <= 0.0f ? 0.0f : z[i] * h[i];
          }
        }
        if (8 * n + 2 * c >= ns) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (r[i] >= rows) continue;
          const int64_t at =
              (static_cast<int64_t>(tile0 + n) * (16 * units) + (j0 + j[i])) * 8 + 2 * c;
          if constexpr (F::FOUR) {
            *reinterpret_cast<float2*>(static_cast<float*>(p.plan.h) + at) =
                make_float2(h[2 * i], h[2 * i + 1]);
          } else {
            uint32_t o[3];
            split_nonzero(h[2 * i], h[2 * i + 1], o);
            uint16_t* to = static_cast<uint16_t*>(p.plan.h) + at;
#pragma unroll
            for (int q = 0; q < 3; ++q)
              *reinterpret_cast<uint32_t*>(to + q * p.plan.plane) = o[q];
          }
        }
      }
    }
    __syncthreads();
  }
}

template <typename F, int NT>
__global__ void __launch_bounds__(kThreads, 2)
    down_kernel(const __grid_constant__ MoeParams p) {
  typedef Sizes<F::FOUR, NT> Z;
  typedef typename F::Step Step;
  constexpr int SP = Z::SP, CHUNK = Z::CHUNK, TW = F::COLS, MT = TW / 16, HR = Step::H_ROW;
  constexpr int SB = Z::RING2 / Step::BYTES;  // steps in a warp's ring
  extern __shared__ __align__(16) uint8_t raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int WC = p.side, WN = kWarps / WC, CW = TW * WC;  // (WC a power of two)
  const int wc = warp & (WC - 1), wn = warp / WC;
  // The rings and h of a chunk; at the end the warps' sums [warp][NT MT 4][32].
  const uint32_t ring_at = ptx::smem_u32(raw + warp * Z::RING2);
  const uint32_t hs = ptx::smem_u32(raw + kWarps * Z::RING2);
  float* red = reinterpret_cast<float*>(raw);
  __shared__ int16_t list[CHUNK];  // ReLU: the chunk's active neurons
  __shared__ int32_t sh_n, sh_done, done[SP], pairs[SP], expect[SP];
  __shared__ float share[SP];
  __shared__ uint8_t in[SP][kMaxTop];

  const int a = blockIdx.z, part = blockIdx.y, splits = gridDim.y, ct = blockIdx.x;
  const int tiles = gridDim.x, units = (p.F + 15) / 16, d0 = CW * ct + TW * wc;
  const int ub = static_cast<int>(static_cast<int64_t>(units) * part / splits),
            ue = static_cast<int>(static_cast<int64_t>(units) * (part + 1) / splits);
  const bool relu = p.act == TWELL_RELU;
  ptx::grid_wait();
  // (reads that depend on one another are few: under load each waits behind all that is
  // on its way)
  const int slabs = __ldcg(p.plan.n_slabs);
  const int4 sl = __ldcg(p.plan.slab + a);
  const uint16_t* masks = p.plan.masks + static_cast<int64_t>(a) * units;
  constexpr int PER = CHUNK / 16 / 32;  // units of a chunk that a lane of warp 0 compacts
  uint32_t mask[PER];
  const auto load_masks = [&](int u0) {
    const int nu = min(CHUNK / 16, ue - u0);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int q = PER * lane + i;
      mask[i] = q < nu ? __ldcg(masks + u0 + q) : 0u;
    }
  };
  if (relu && warp == 0) load_masks(ub);
  if (a >= slabs) return;
  const int e = sl.x, s0 = sl.y, ns = sl.z, nt_used = (ns + 7) / 8;
  const int64_t base = static_cast<int64_t>(e) * p.F;
  float acc[MT][NT][4];
#pragma unroll
  for (int q = 0; q < MT; ++q)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[q][n][j] = 0.0f;
#pragma unroll 1
  for (int u0 = ub; u0 < ue; u0 += CHUNK / 16) {
    const int nu = min(CHUNK / 16, ue - u0), whole = min(16 * nu, p.F - 16 * u0);
    int total = whole;
    if (relu) {  // compact
      if (warp == 0) {
        int mine = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) mine += __popc(mask[i]);
        int up = mine;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const int v = __shfl_up_sync(0xffffffffu, up, o);
          if (lane >= o) up += v;
        }
        int at = up - mine;
#pragma unroll
        for (int i = 0; i < PER; ++i)
#pragma unroll 1
          for (uint32_t m = mask[i]; m; m &= m - 1)
            list[at++] = static_cast<int16_t>(16 * (PER * lane + i) + __ffs(m) - 1);
        if (lane == 31) sh_n = up;
        if (u0 + CHUNK / 16 < ue) load_masks(u0 + CHUNK / 16);
      }
      __syncthreads();
      total = sh_n;
    }
    const bool some = total < whole;  // (else the list is 0, 1, 2 ...)
    const int steps = (total + 15) / 16;
    const int64_t row0 = base + 16 * u0;
    const auto neuron = [&](int s) { return some ? list[s] : s; };
    const auto first = [&] {  // what the end needs
      if (u0 == ub && tid < ns) {
        const int pair = __ldcg(p.plan.list + s0 + tid);
        pairs[tid] = pair;
        expect[tid] = __ldcg(p.plan.live + pair / p.k) * splits;
        share[tid] = __ldcg(p.weights + pair);
      }
    };
    if (total == 0) {
      first();
      __syncthreads();
      continue;
    }

    // h of the chunk, up to a whole step (of absent pairs: anything, each pair is a column of
    // its own)
    const int64_t tile = static_cast<int64_t>(16 * units) * HR;
    const uint8_t* from =
        static_cast<const uint8_t*>(p.plan.h) + sl.w * tile + 16 * u0 * HR;
#pragma unroll 1
    for (int s = tid; s < 16 * steps; s += kThreads) {
      const bool on = s < total;
      const uint8_t* src = from + (on ? neuron(s) : 0) * HR;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n >= nt_used) break;
        if constexpr (F::FOUR) {
          const uint32_t to = hs + (n * CHUNK + Step::place(s)) * HR;
          ptx::cp_async16(to, src + n * tile, on ? 16 : 0);
          if (8 * n + 4 < ns) ptx::cp_async16(to + 16, src + n * tile + 16, on ? 16 : 0);
        } else {
          const uint32_t to = hs + (n * CHUNK + s) * HR;
#pragma unroll
          for (int q = 0; q < 3; ++q)
            ptx::cp_async16(to + q * NT * CHUNK * HR, src + n * tile + q * 2 * p.plan.plane,
                            on ? 16 : 0);
        }
      }
    }
    ptx::cp_async_commit();

    int put = 0, get = 0, st_put = wn;
    const typename Step::Origin origin(p, row0, d0);
    const auto issue = [&] {
      if (st_put < steps)
        Step::copy(
            p, origin, [&](int r) { return neuron(min(16 * st_put + r, total - 1)); },
            total - 16 * st_put, ring_at + put * Step::BYTES);
      ptx::cp_async_commit();
      st_put += WN;
      put = put + 1 == SB ? 0 : put + 1;
    };
    const auto scales = [&](int st, typename Step::Scales& s) {
      if (16 * st + (lane & 15) < total) s.load(p, origin, neuron(16 * st + (lane & 15)));
      else s.none();  // (a test of what is loaded would wait for it)
    };
    typename Step::Scales s_now, s_next, s_then;
#pragma unroll 1
    for (int i = 0; i < SB - 1; ++i) issue();
    scales(wn, s_now);
    scales(wn + WN, s_next);
    first();
    ptx::cp_async_wait<SB - 1>();
    __syncthreads();
    // (for the tiles of pairs that there are: a test for each would cost as much as what it
    // leaves out)
    const auto run = [&](auto used) {
#pragma unroll 1
      for (int st = wn; st < steps; st += WN) {
        issue();
        scales(st + 2 * WN, s_then);
        ptx::cp_async_wait<SB - 1>();
        __syncwarp();
        Step::template add<decltype(used)::value, NT, CHUNK>(
            ring_at + get * Step::BYTES, s_now, hs, st, acc);
        __syncwarp();  // (the next copy but SB - 2 goes where this step was)
        get = get + 1 == SB ? 0 : get + 1;
        s_now = s_next, s_next = s_then;
      }
    };
    if (NT > 1 && nt_used == 1) run(Count<1>());
    else run(Count<NT>());
    ptx::cp_async_wait<0>();
    __syncthreads();
  }

  // ---- the warps' sums, then the token's where this part completes it
  constexpr int VALUES = MT * NT * 4 * 32;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int q = 0; q < MT; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        red[warp * VALUES + ((n * MT + q) * 4 + j) * 32 + lane] = acc[q][n][j];
  __syncthreads();
  constexpr int QUADS = 2 * TW;  // fours of columns of eight pairs
#pragma unroll 1
  for (int i = tid; i < WC * nt_used * QUADS; i += kThreads) {
    const int w0 = i / QUADS & (WC - 1), n = i >= WC * QUADS, t = i % QUADS / 8;
    const int pair = 8 * n + i % 8, d = CW * ct + TW * w0 + F::columns(t);
    if (pair >= ns || d >= p.D) continue;
    const float* at = red + w0 * VALUES + n * (MT * 128) + F::first_of(t) + 32 * (i & 1) + (i >> 1 & 3);
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
    for (int w = w0; w < kWarps; w += WC, at += WC * VALUES)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += at[F::next(j)];
    const float a = share[pair];
    __stcg(reinterpret_cast<float4*>(
               p.part + (static_cast<int64_t>(pairs[pair]) * splits + part) * p.D + d),
           make_float4(v[0] * a, v[1] * a, v[2] * a, v[3] * a));
  }
  __threadfence();
  __syncthreads();
  if (warp == 0) {
    bool last = false;
    int t = 0;
    if (lane < ns) {
      t = pairs[lane] / p.k;
      last = atomicAdd(p.count + static_cast<int64_t>(t) * tiles + ct, 1) + 1 == expect[lane];
    }
    const uint32_t m = __ballot_sync(0xffffffffu, last);
    if (last) done[__popc(m & ((1u << lane) - 1u))] = t;
    if (lane == 0) sh_done = __popc(m);
  }
  __syncthreads();
  const int n_done = sh_done;
  if (n_done == 0) return;
  __threadfence();
#pragma unroll 1
  for (int i = tid; i < n_done * p.k; i += kThreads) {  // the slots that have an expert
    const int id = __ldcg(p.ids + static_cast<int64_t>(done[i / p.k]) * p.k + i % p.k);
    in[i / p.k][i % p.k] = id >= 0 && id < p.E;
  }
  __syncthreads();
#pragma unroll 1
  for (int i = tid; i < n_done * (CW / 4); i += kThreads) {
    const int o = i / (CW / 4), t = done[o], d = CW * ct + i % (CW / 4) * 4;
    if (d >= p.D) continue;
    const float* from = p.part + static_cast<int64_t>(t) * p.k * splits * p.D + d;
    float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
    for (int q = 0; q < splits; ++q) {
#pragma unroll 8
      for (int s = 0; s < p.k; ++s) {
        if (!in[o][s]) continue;
        const float4 v = __ldcg(reinterpret_cast<const float4*>(
            from + (static_cast<int64_t>(s) * splits + q) * p.D));
        f[0] += v.x, f[1] += v.y, f[2] += v.z, f[3] += v.w;
      }
    }
    const int64_t to = static_cast<int64_t>(t) * p.D + d;
    if (p.y_f32) store4(static_cast<float*>(p.y) + to, f);
    else store4(static_cast<uint16_t*>(p.y) + to, f);
  }
}

// -------------------------------------------------------------------- host

// Tiles of eight pairs that an expert's weights are read once for: two where most experts
// have more than one tile's (an expert with more than a slab reads its weights again, from the
// second cache).  4 bits, E = 64, 8 experts a token: 32 tokens 112 us with one and 123 with two,
// 48 119 and 135, 64 192 and 166; bf16 169 and 170, 177 and 179, 222 and 187.
int pair_tiles(int32_t T, int32_t E, int32_t k) { return T <= 8 || T * k < 7 * E ? 1 : 2; }

// The down kernel: warps side by side on columns, tiles of a CTA's columns, slabs at the most,
// and parts of a slab's neurons.  The widest CTAs that still give every SM four, so that
// an SM's last ones leave little of it idle (64 tokens, 4 bits: 166 us, 172 with two, 239 with
// one, 177 with eight; bf16 187, 191, 192, 197).  Neurons are divided where CTAs of one
// warp's width leave SMs without two, into parts of 128 neurons at least (a token, 4 bits:
// 26.2 us, 29.3 where they are divided for one an SM, 30.6 for four).
struct Down {
  int32_t side, tiles, slabs, splits;
};
Down down_of(const DeviceInfo& dev, int32_t T, int32_t D, int32_t F, int32_t E, int32_t k,
             bool four) {
  const int nt = pair_tiles(T, E, k), tw = four ? 128 : 64, P = T * k;
  Down o;
  o.slabs = (P < E ? P : E) + P / (8 * nt);
  if (o.slabs > P) o.slabs = P;
  if (o.slabs < 1) o.slabs = 1;  // (no tokens)
  for (o.side = kWarps;; o.side /= 2) {
    o.tiles = (D + o.side * tw - 1) / (o.side * tw);
    if (o.side == 1 || o.tiles * o.slabs >= 4 * dev.sm_count) break;
  }
  const int fill = 2 * dev.sm_count / (o.tiles * o.slabs), most = (F + 15) / 16 / 8;
  o.splits = most < fill ? most : fill;
  o.splits = o.splits < 1 ? 1 : o.splits > 8 ? 8 : o.splits;
  return o;
}

struct Layout {
  size_t logits, count, slab, list, live, masks, h, part, total;
  int64_t plane;
  int32_t counters;
};

Layout layout_of(const DeviceInfo& dev, int32_t T, int32_t D, int32_t F, int32_t E, int32_t k) {
  Layout l;
  const size_t P = static_cast<size_t>(T) * k, units = (static_cast<size_t>(F) + 15) / 16;
  size_t slabs = 0, splits = 0, tiles = 0;  // of whichever form asks for most
  for (int four = 0; four < 2; ++four) {
    const Down o = down_of(dev, T, D, F, E, k, four);
    slabs = slabs > static_cast<size_t>(o.slabs) ? slabs : o.slabs;
    splits = splits > static_cast<size_t>(o.splits) ? splits : o.splits;
    tiles = tiles > static_cast<size_t>(o.tiles) ? tiles : o.tiles;
  }
  l.counters = static_cast<int32_t>(T * tiles);
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  l.logits = take(4 * static_cast<size_t>(T) * E);
  l.count = take(4 * static_cast<size_t>(l.counters));
  l.slab = take(16 * (slabs + 1));  // (the first: how many)
  l.list = take(4 * P);
  l.live = take(4 * static_cast<size_t>(T));
  l.masks = take(2 * slabs * units);
  // (tiles: an expert's last may not be whole)
  const size_t used = P < static_cast<size_t>(E) ? P : E;
  l.plane = static_cast<int64_t>((P + 7 * used) / 8 * 16 * units * 8);
  l.h = take(6 * static_cast<size_t>(l.plane));
  l.part = take(4 * P * splits * D);
  l.total = at;
  return l;
}

template <typename F, int NT>
twell_status launch_experts(MoeParams p, const DeviceInfo& dev, cudaStream_t s) {
  typedef Sizes<F::FOUR, NT> Z;
  static std::atomic<uint64_t> set[2] = {{0}, {0}};
  const int limit = dev.max_smem_optin - 8192;
  const int64_t P = static_cast<int64_t>(p.T) * p.k;
  const Down o = down_of(dev, p.T, p.D, p.F, p.E, p.k, F::FOUR);
  p.side = o.side;
  const int64_t units = o.slabs * ((static_cast<int64_t>(p.F) + 15) / 16);
  const int most = 2 * dev.sm_count;
  cudaLaunchAttribute attr = overlapped();
  size_t smem = kWarps * (Z::RING + 1024 * NT) + 16 * (p.E + P / Z::SP) +
                4 * (Z::RM * Z::ZP + p.E + 3 * P + p.T);
  cudaLaunchConfig_t cfg = launch_config(dim3(static_cast<unsigned>(units < most ? units : most)),
                                         dim3(kThreads), smem, s);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  twell_status st = launch_large(neurons_kernel<F, NT>, limit, cfg, dev, set[0], p);
  if (st != TWELL_OK) return st;
  const size_t rings =
      kWarps * Z::RING2 + (F::FOUR ? 1 : 3) * NT * Z::CHUNK * F::Step::H_ROW;
  const size_t sums = 4 * kWarps * (F::COLS / 16) * NT * 4 * 32;
  cfg = launch_config(dim3(o.tiles, o.splits, o.slabs), dim3(kThreads),
                      rings > sums ? rings : sums, s);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return launch_large(down_kernel<F, NT>, limit, cfg, dev, set[1], p);
}

template <typename F>
twell_status launch_experts(const MoeParams& p, const DeviceInfo& dev, cudaStream_t s) {
  return pair_tiles(p.T, p.E, p.k) == 1 ? launch_experts<F, 1>(p, dev, s)
                                        : launch_experts<F, 2>(p, dev, s);
}

bool sizes_ok(int32_t T, int32_t D, int32_t F, int32_t E, int32_t k) {
  return T >= 0 && D >= 8 && D % 8 == 0 && F >= 1 && E >= 1 && k >= 1;
}
bool within_limits(int32_t T, int32_t D, int32_t E, int32_t k) {
  return T <= kMaxTokens && D <= kMaxWidth && E <= kMaxExperts && k <= kMaxTop &&
         static_cast<int64_t>(T) * k <= kMaxPairs;
}
// (units of 16 neurons of every slab of eight pairs, times the CTAs, are counted in 32 bits)
bool neurons_ok(int32_t F, int32_t E) {
  return static_cast<int64_t>(E + kMaxPairs / 8) * ((static_cast<int64_t>(F) + 15) / 16) <= 1 << 23;
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
  // A layout may need more than that of a larger batch, whose neurons are in fewer parts: the
  // workspace is enough for any up to T.
  size_t most = 0;
  for (int32_t t = 0; t <= T; ++t) {
    const size_t total = layout_of(dev, t, D, F, E, top_k).total;
    most = most > total ? most : total;
  }
  return most;
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
  if (four && (w->Wg_t || w->Wu_t || w->Wd)) return TWELL_ERR_INVALID;
  if (four) {
    const twell_int4_t* m[3] = {w->Wg4, w->Wu4, w->Wd4};
    for (const twell_int4_t* q : m) {
      const twell_status st = check_int4(q);
      if (st != TWELL_OK) return st;
      if (q->rows != static_cast<int64_t>(E) * F || q->K != D || q->group != m[0]->group)
        return TWELL_ERR_INVALID;
    }
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

  const RouterParams r{x, router, T, D, E, logits, count, l.counters};
  const unsigned grid = !router ? 1u : T == 1 ? E : (E + 1) / 2 * ((T + 7) / 8);
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
  p.plan.n_slabs = reinterpret_cast<int32_t*>(base + l.slab);
  p.plan.slab = reinterpret_cast<int4*>(base + l.slab) + 1;
  p.plan.list = reinterpret_cast<int32_t*>(base + l.list);
  p.plan.live = reinterpret_cast<int32_t*>(base + l.live);
  p.plan.masks = reinterpret_cast<uint16_t*>(base + l.masks);
  p.plan.h = base + l.h;
  p.plan.plane = l.plane;
  p.part = reinterpret_cast<float*>(base + l.part);
  p.count = count;
  p.y = y, p.y_f32 = y_type == TWELL_F32;
  if (router && T > kWarps) {
    cudaLaunchConfig_t cfg = launch_config(dim3((T + kWarps - 1) / kWarps), dim3(kThreads), 0, s);
    cudaLaunchAttribute attr = overlapped();
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (!cuda_ok(cudaLaunchKernelEx(&cfg, choose_kernel, p))) return TWELL_ERR_CUDA;
  }
  if (!four) {
    p.w[0] = w->Wg_t, p.w[1] = w->Wu_t, p.w[2] = w->Wd;
    return launch_experts<Bf16>(p, dev, s);
  }
  p.q[0] = view_of(*w->Wg4), p.q[1] = view_of(*w->Wu4), p.q[2] = view_of(*w->Wd4);
  return w->Wg4->group == 32   ? launch_experts<Four<1>>(p, dev, s)
         : w->Wg4->group == 64 ? launch_experts<Four<2>>(p, dev, s)
                               : launch_experts<Four<4>>(p, dev, s);
}
