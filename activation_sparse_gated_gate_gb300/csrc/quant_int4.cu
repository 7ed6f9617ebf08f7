// Quantisation of weights to 4 bits with a scale (and a zero point) for each group of 32,
// 64 or 128 columns of a row, and the values that such weights stand for.
//
// Without zero points   s = bf16(max |v| / 7),  code = clamp(rint(v / s), -8, 7) + 8;
// with them, lo = min(v, 0) and hi = max(v, 0) over the group,
//   s = bf16((hi - lo) / 15),  z = clamp(rint(-lo / s), 0, 15),
//   code = clamp(rint(v / s) + z, 0, 15).
// rint is of the exact quotient, ties to even: v times 1 / s in fp32 gives a code that is
// at most one off, and the remainder v - code s, exact in one fused operation, says
// whether it is (an IEEE division for each value would double the kernel's instructions):
// eight values whose remainders are all below s / 2 have their codes, others are looked at
// one by one.  Of bf16 values one in some hundred is a tie, but a quotient of two 8-bit numbers
// that is none is 2^-9 or more away from any (2 v - (2 q + 1) s is a multiple of the last place of
// one of them): rounded to multiples of 2^-11 first, ties are exact and others stay where
// they are.
// The stored order is int4.cuh's.
//
// Bound by memory (8192 x 2048 bf16 and back in two launches, 76 MB: 16.4 us, 4.6 TB/s; fp32 32.8) and
// of ragged rows by instructions (1001 x 1999 with zero points and back: 10.8 us).  Half a
// warp takes a block of 128 columns of a row, 16 bytes (bf16) or 32 a lane; a group's maximum is taken over its 4, 8 or 16 lanes; a lane's eight
// codes are two runs of 16 bits, which a pair of lanes exchanges into words.  Rows off 16-byte
// boundaries: a warp a block, lane l with columns l, l + 32, l + 64, l + 96.
#include "common.cuh"
#include "int4.cuh"
#include "vec.cuh"

namespace twell {
namespace {

constexpr float kMagic = 12582912.0f;  // 1.5 2^23: adding it leaves the nearest integer
constexpr float kSnap = 6144.0f;       // 1.5 2^12: the nearest multiple of 2^-11
constexpr float kSmall = 7.88860905e-31f, kLift = 1.2676506e30f;  // 2^-100, 2^100

struct Scale {
  float s, inv, half;  // the scale (lifted where it is small), about 1 / s, s / 2
  float zero;          // the zero point
  uint16_t stored;
  bool none;           // a scale of zero or NaN: every code is the zero point
  bool small;
};

template <bool ZERO>
__device__ __forceinline__ float code_of(float v, const Scale& k) {
  const float t = fmaf(v, k.inv, kMagic);
  float q = t - kMagic;
  const float r = fmaf(-q, k.s, v);
  if (fabsf(r) >= k.half && (fabsf(r) > k.half || (__float_as_uint(t) & 1u)))
    q += copysignf(1.0f, r);
  return ZERO ? fminf(fmaxf(q + k.zero, 0.0f), 15.0f) : fminf(fmaxf(q, -8.0f), 7.0f) + 8.0f;
}

// From a group's largest |v| (as its bits, above infinity's where there is a NaN), and its
// least and largest value.
template <bool ZERO>
__device__ __forceinline__ Scale scale_of(uint32_t top, float lo, float hi) {
  Scale k;
  // a / 7 or a / 15, rounded as the division is: a quotient that is an ulp or two off,
  // corrected once by its exact remainder times the rounded reciprocal (Markstein 1990); where
  // the remainder might be subnormal, the division itself
  constexpr float D = ZERO ? 15.0f : 7.0f, Y = 1.0f / D;
  const float a = ZERO ? hi - lo : __uint_as_float(top);
  const float near = a * Y;
  float s = fmaf(fmaf(-near, D, a), Y, near);
  if (a < kSmall * 1024.0f) s = a / D;
  uint16_t b;
  narrow(s, b);
  s = widen(b);
  // a NaN, an infinity, or values whose scale is beyond bf16: the group is NaN
  const bool bad = top >= 0x7f800000u || !(s < __uint_as_float(0x7f800000u));
  k.stored = bad ? 0x7fc0u : b;
  k.none = bad || s == 0.0f;
  k.small = !k.none && s < kSmall;
  k.s = k.small ? s * kLift : s;
  asm("rcp.approx.f32 %0, %1;" : "=f"(k.inv) : "f"(k.s));  // (an ulp does not matter)
  k.half = 0.5f * k.s;
  k.zero = 8.0f;
  if (ZERO && !k.none) {
    Scale z = k;
    z.zero = 0.0f;
    k.zero = code_of<true>(k.small ? -lo * kLift : -lo, z);
  }
  return k;
}

// The codes of N values, the j-th at nibble `order` has it.  A code is the low end of the
// bits of 1.5 2^23 + code, so that the codes are put together by multiply-adds of these bits (one
// a value, where masks and shifts would be three on the slower integer pipe); what the
// constant adds up to is known.
template <bool ZERO, bool BF16, int N>
__device__ __forceinline__ uint32_t quantise(const float (&v)[N], const Scale& k,
                                             const int (&order)[N]) {
  static_assert(N == 8 || N == 1, "a word, or one code");
  constexpr uint32_t ONES = N == 8 ? 0x11111111u : 1u;
  if (k.none) return 8u * ONES;
  uint32_t x = 0u;
  float worst = 0.0f;
#pragma unroll
  for (int i = N - 1; i >= 0; --i) {
    const float w = v[order[i]];
    float t;
    if (BF16) {
      t = fmaf(w, k.inv, kSnap) + (kMagic - kSnap);
    } else {
      t = fmaf(w, k.inv, kMagic);
      worst = fmaxf(worst, fabsf(fmaf(kMagic - t, k.s, w)));
    }
    if (ZERO) t = fminf(t, kMagic + 15.0f - k.zero);
    x = x * 16u + __float_as_uint(t);
  }
  // (a scale that rounding has not left far from the group's extent keeps the others in range)
  if ((BF16 || worst < k.half) && !k.small)
    return x + (static_cast<uint32_t>(k.zero) - 0x4b400000u) * ONES;
  x = 0u;
#pragma unroll 1
  for (int i = N - 1; i >= 0; --i) {
    float w = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (i == j) w = v[order[j]];
    x = x * 16u + (__float_as_uint(code_of<ZERO>(k.small ? w * kLift : w, k) + kMagic) & 15u);
  }
  return x;
}

// Division of a number below 2^31 by a divisor that the host knows.
struct Divisor {
  uint32_t d, m, shift;
};
Divisor divisor(uint32_t d) {
  uint32_t l = 0;
  while (l < 31 && (1ull << l) < d) ++l;
  return Divisor{d, static_cast<uint32_t>((1ull << (31 + l)) / d + 1), l};
}
__device__ __forceinline__ uint32_t over(uint32_t n, const Divisor& v) {
  return v.d == 1 ? n : __umulhi(n, v.m) >> (v.shift - 1);
}

struct QuantParams {
  const void* src;
  int64_t ld;
  uint32_t K, items;  // items: blocks, nb a row
  Divisor nb;
  uint8_t* code;
  uint16_t* scale;
  uint8_t* zero;
};

// Eight values as they were loaded, and over LANES lanes the largest |v| (its bits; a NaN is
// above all) and the least and largest value.
template <typename T>
struct Eight;

template <>
struct Eight<float> {
  float v[8];
  __device__ __forceinline__ void load(const float* p, bool have) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    if (have) load8<true>(p, 8, v);
  }
  __device__ __forceinline__ float get(int j) const { return v[j]; }
  template <bool ZERO, int LANES>
  __device__ __forceinline__ void extent(uint32_t& top, float& lo, float& hi) const {
    top = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
      if (ZERO) lo = fminf(lo, v[j]), hi = fmaxf(hi, v[j]);
    }
#pragma unroll
    for (int o = 1; o < LANES; o *= 2) {
      top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (ZERO) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      }
    }
  }
};

__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <>
struct Eight<uint16_t> {
  uint32_t v[4];
  __device__ __forceinline__ void load(const uint16_t* p, bool have) {
    const uint4 a = have ? *reinterpret_cast<const uint4*>(p) : make_uint4(0u, 0u, 0u, 0u);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  }
  __device__ __forceinline__ float get(int j) const {
    return __uint_as_float(j & 1 ? v[j / 2] & 0xffff0000u : v[j / 2] << 16);
  }
  template <bool ZERO, int LANES>
  __device__ __forceinline__ void extent(uint32_t& top, float& lo, float& hi) const {
    // two columns at a time; a NaN stays one
    uint32_t t = 0u, least = 0u, most = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (ZERO) least = min_nan_bf16x2(least, v[j]), most = max_nan_bf16x2(most, v[j]);
      else t = max_nan_bf16x2(t, v[j] & 0x7fff7fffu);
    }
#pragma unroll
    for (int o = 1; o < LANES; o *= 2) {
      if (ZERO) {
        least = min_nan_bf16x2(least, __shfl_xor_sync(0xffffffffu, least, o));
        most = max_nan_bf16x2(most, __shfl_xor_sync(0xffffffffu, most, o));
      } else {
        t = max_nan_bf16x2(t, __shfl_xor_sync(0xffffffffu, t, o));
      }
    }
    if (ZERO) {
      least = min_nan_bf16x2(least, least >> 16), most = max_nan_bf16x2(most, most >> 16);
      lo = __uint_as_float(least << 16), hi = __uint_as_float(most << 16);
      top = max(__float_as_uint(lo) & 0x7fffffffu, __float_as_uint(hi) & 0x7fffffffu);
    } else {
      top = max_nan_bf16x2(t, t >> 16) << 16;
    }
  }
};

// G32: groups of 32 columns in a group.
template <typename T, int G32, bool ZERO>
__global__ void __launch_bounds__(256) quant_int4_kernel(const QuantParams p) {
  constexpr int ITEMS = sizeof(T) == 2 ? 4 : 2;  // 64 bytes a thread in flight
  const int l = threadIdx.x & 15, i = l >> 2, c = l & 3;
  const uint32_t first = blockIdx.x * (16u * ITEMS) + (threadIdx.x >> 4);
  Eight<T> raw[ITEMS];
#pragma unroll
  for (int m = 0; m < ITEMS; ++m) {
    const uint32_t item = first + 16u * m;
    const uint32_t row = over(item, p.nb), b = item - row * p.nb.d;
    const uint32_t c0 = b * kInt4Block + 8u * l;
    raw[m].load(static_cast<const T*>(p.src) + static_cast<int64_t>(row) * p.ld + c0,
                item < p.items && c0 < p.K);
  }
#pragma unroll
  for (int m = 0; m < ITEMS; ++m) {
    const uint32_t item = first + 16u * m;
    uint32_t top;
    float lo = 0.0f, hi = 0.0f;
    raw[m].template extent<ZERO, 4 * G32>(top, lo, hi);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = raw[m].get(j);
    const Scale k = scale_of<ZERO>(top, lo, hi);
    const uint32_t row = over(item, p.nb), b = item - row * p.nb.d;
    const bool held = b * kInt4Block + 8u * l < p.K;  // (K is a multiple of 8 here)
    // even columns in the low half, odd ones in the high
    const int order[8] = {0, 2, 4, 6, 1, 3, 5, 7};
    const uint32_t x = held ? quantise<ZERO, sizeof(T) == 2>(v, k, order) : 0x88888888u;
    const uint32_t t = __shfl_xor_sync(0xffffffffu, x, 4);
    const uint32_t w = i & 1 ? __byte_perm(t, x, 0x7632) : __byte_perm(x, t, 0x5410);
    if (item >= p.items) continue;
    // lane i of four: word 0 (even columns of i = 0, 1), 2 (odd), 1 (even of 2, 3), 3
    reinterpret_cast<uint32_t*>(p.code + static_cast<int64_t>(item) * kInt4Bytes)
        [4 * c + 2 * (i & 1) + (i >> 1)] = w;
    if (l % (4 * G32) == 0) {
      const int64_t at = static_cast<int64_t>(item) * (4 / G32) + l / (4 * G32);
      p.scale[at] = held ? k.stored : static_cast<uint16_t>(0);
      if (ZERO) p.zero[at] = held ? static_cast<uint8_t>(k.zero) : static_cast<uint8_t>(8);
    }
  }
}

// Any K and any pitch.
template <typename T, int G32, bool ZERO>
__global__ void __launch_bounds__(256) quant_int4_lanes_kernel(const QuantParams p) {
  constexpr int ITEMS = 2, GROUPS = 4 / G32;
  const int l = threadIdx.x & 31;
  const int n = (l >> 1) & 3, g = 2 * (l >> 3) + (l & 1);  // its nibble and its 8 bytes
  const uint32_t first = blockIdx.x * (8u * ITEMS) + (threadIdx.x >> 5);
  float v[ITEMS][4];
#pragma unroll
  for (int m = 0; m < ITEMS; ++m) {
    const uint32_t item = first + 8u * m;
    const uint32_t row = over(item, p.nb), b = item - row * p.nb.d;
    const T* src = static_cast<const T*>(p.src) + static_cast<int64_t>(row) * p.ld;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t col = b * kInt4Block + 32u * i + l;
      v[m][i] = item < p.items && col < p.K ? widen(src[col]) : 0.0f;
    }
  }
#pragma unroll
  for (int m = 0; m < ITEMS; ++m) {
    const uint32_t item = first + 8u * m;
    const uint32_t row = over(item, p.nb), b = item - row * p.nb.d;
    uint32_t top[GROUPS];
    float lo[GROUPS], hi[GROUPS];
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) {
      top[k] = 0u, lo[k] = hi[k] = 0.0f;
#pragma unroll
      for (int i = k * G32; i < (k + 1) * G32; ++i) {
        top[k] = max(top[k], __float_as_uint(v[m][i]) & 0x7fffffffu);
        if (ZERO) lo[k] = fminf(lo[k], v[m][i]), hi[k] = fmaxf(hi[k], v[m][i]);
      }
    }
    const uint32_t t = over_warp(top, [](uint32_t a, uint32_t c) { return max(a, c); });
    float least = 0.0f, most = 0.0f;
    if (ZERO) {
      least = over_warp(lo, [](float a, float c) { return fminf(a, c); });
      most = over_warp(hi, [](float a, float c) { return fmaxf(a, c); });
    }
    // each lane the scale of one group
    const int mine = l / (32 / GROUPS);
    const Scale own = scale_of<ZERO>(t, least, most);
    if (l % (32 / GROUPS) == 0 && item < p.items) {
      const int64_t at = static_cast<int64_t>(item) * GROUPS + mine;
      const bool some = b * kInt4Block + 32u * G32 * mine < p.K;
      p.scale[at] = some ? own.stored : static_cast<uint16_t>(0);
      if (ZERO) p.zero[at] = some ? static_cast<uint8_t>(own.zero) : static_cast<uint8_t>(8);
    }
    const uint32_t bits =
        static_cast<uint32_t>(own.zero) | (own.none ? 32u : 0u) | (own.small ? 64u : 0u);
    uint32_t word[2] = {0u, 0u};
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) {
      const int from = k * (32 / GROUPS);
      Scale sc;
      sc.s = __shfl_sync(0xffffffffu, own.s, from);
      sc.inv = __shfl_sync(0xffffffffu, own.inv, from);
      const uint32_t f = __shfl_sync(0xffffffffu, bits, from);
      sc.half = 0.5f * sc.s;
      sc.zero = static_cast<float>(f & 15u);
      sc.none = f & 32u, sc.small = f & 64u;
#pragma unroll
      for (int i = k * G32; i < (k + 1) * G32; ++i) {
        const bool held = b * kInt4Block + 32u * i + l < p.K;
        const float one[1] = {v[m][i]};
        const int order[1] = {0};
        const uint32_t q = held ? quantise<ZERO, sizeof(T) == 2>(one, sc, order) & 15u : 8u;
        word[i / 2] |= q << (4 * n + 16 * (i % 2));
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // the four lanes of the same 8 bytes
      word[h] |= __shfl_xor_sync(0xffffffffu, word[h], 2);
      word[h] |= __shfl_xor_sync(0xffffffffu, word[h], 4);
    }
    if (n == 0 && item < p.items)
      *reinterpret_cast<uint2*>(p.code + static_cast<int64_t>(item) * kInt4Bytes + 8 * g) =
          make_uint2(word[0], word[1]);
  }
}

struct DequantParams {
  Int4View w;
  uint32_t K, items;
  Divisor nb;
  void* out;
  int64_t ld;
};

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Nibble n of the low half as a float less the zero point, times the scale: the nibble is
// taken where it stands, as 2^23 + code 16^n, so that nothing is shifted or converted (code - zero
// and its products with the scale are exact).
struct Scaled {
  float minus[4], times[4];  // 2^23 + zero 16^n, scale / 16^n
  __device__ __forceinline__ Scaled(float zero, float scale) {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      minus[n] = fmaf(zero, static_cast<float>(1 << (4 * n)), 8388608.0f);
      times[n] = scale * (1.0f / static_cast<float>(1 << (4 * n)));
    }
  }
  __device__ __forceinline__ float of(uint32_t p, int n) const {
    return (__uint_as_float((p & (15u << (4 * n))) | 0x4b000000u) - minus[n]) * times[n];
  }
};

// A thread takes 16 bytes, the columns 8 c .. 8 c + 7 of each 32 of a block.
template <typename T, int G32>
__global__ void __launch_bounds__(256) dequant_int4_kernel(const DequantParams p) {
  constexpr int ITEMS = 2;
  const int c = threadIdx.x & 3;
  const uint32_t first = blockIdx.x * (64u * ITEMS) + (threadIdx.x >> 2);
  uint4 w[ITEMS];
  uint16_t s[ITEMS][4 / G32];
  uint8_t z[ITEMS][4 / G32];
#pragma unroll
  for (int m = 0; m < ITEMS; ++m) {
    const uint32_t item = first + 64u * m;
    if (item >= p.items) continue;
    w[m] = ld_stream16(p.w.code + static_cast<int64_t>(item) * kInt4Bytes + 16 * c);
#pragma unroll
    for (int k = 0; k < 4 / G32; ++k) {
      s[m][k] = __ldg(p.w.scale + static_cast<int64_t>(item) * (4 / G32) + k);
      z[m][k] = p.w.zero ? __ldg(p.w.zero + static_cast<int64_t>(item) * (4 / G32) + k)
                         : static_cast<uint8_t>(8);
    }
  }
#pragma unroll
  for (int m = 0; m < ITEMS; ++m) {
    const uint32_t item = first + 64u * m;
    if (item >= p.items) continue;
    const uint32_t row = over(item, p.nb), b = item - row * p.nb.d;
    T* out = static_cast<T*>(p.out) + static_cast<int64_t>(row) * p.ld;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t col = b * kInt4Block + 32u * i + 8u * c;
      const uint32_t e = i < 2 ? w[m].x : w[m].y, o = i < 2 ? w[m].z : w[m].w;
      if (col >= p.K) continue;
      if constexpr (sizeof(T) == 2) {  // two at a time, rounded once by the product
        const uint32_t both = __byte_perm(e, o, i & 1 ? 0x7632 : 0x5410);
        const uint32_t bias = z[m][i / G32] * 0x00010001u + 0x43004300u,
                       sc = s[m][i / G32] * 0x00010001u;
        *reinterpret_cast<uint4*>(out + col) =
            make_uint4(mul_bf16x2(nibbles(both, 0, bias), sc), mul_bf16x2(nibbles(both, 1, bias), sc),
                       mul_bf16x2(nibbles(both, 2, bias), sc), mul_bf16x2(nibbles(both, 3, bias), sc));
      } else {
        const Scaled k(static_cast<float>(z[m][i / G32]), widen(s[m][i / G32]));
        float f[8];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          f[2 * n] = k.of(i & 1 ? e >> 16 : e, n);
          f[2 * n + 1] = k.of(i & 1 ? o >> 16 : o, n);
        }
        store8<true>(out + col, 8, f);
      }
    }
  }
}

template <typename T, int G32>
__global__ void __launch_bounds__(256) dequant_int4_lanes_kernel(const DequantParams p) {
  constexpr int ITEMS = 4;
  const int l = threadIdx.x & 31;
  const int n = (l >> 1) & 3, g = 2 * (l >> 3) + (l & 1);
  const uint32_t first = blockIdx.x * (8u * ITEMS) + (threadIdx.x >> 5);
  uint2 w[ITEMS];
#pragma unroll
  for (int m = 0; m < ITEMS; ++m) {
    const uint32_t item = first + 8u * m;
    w[m] = item < p.items ? __ldg(reinterpret_cast<const uint2*>(
                                p.w.code + static_cast<int64_t>(item) * kInt4Bytes + 8 * g))
                          : make_uint2(0u, 0u);
  }
#pragma unroll
  for (int m = 0; m < ITEMS; ++m) {
    const uint32_t item = first + 8u * m;
    if (item >= p.items) continue;
    const uint32_t row = over(item, p.nb), b = item - row * p.nb.d;
    T* out = static_cast<T*>(p.out) + static_cast<int64_t>(row) * p.ld;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t col = b * kInt4Block + 32u * i + l;
      const int64_t at = static_cast<int64_t>(item) * (4 / G32) + i / G32;
      const float sc = widen(__ldg(p.w.scale + at));
      const float zf = p.w.zero ? static_cast<float>(__ldg(p.w.zero + at)) : 8.0f;
      const uint32_t q = ((i < 2 ? w[m].x : w[m].y) >> (16 * (i % 2) + 4 * n)) & 15u;
      const float f = (__uint_as_float(q | 0x4b000000u) - (8388608.0f + zf)) * sc;
      if (col < p.K) narrow(f, out[col]);
    }
  }
}

template <typename K, typename P>
twell_status enqueue(K kernel, const P& p, uint32_t per_cta, cudaStream_t s) {
  kernel<<<(p.items + per_cta - 1) / per_cta, 256, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}

template <typename T, int G32, bool ZERO>
twell_status quant(const QuantParams& p, bool vec, cudaStream_t s) {
  return vec ? enqueue(quant_int4_kernel<T, G32, ZERO>, p, sizeof(T) == 2 ? 64 : 32, s)
             : enqueue(quant_int4_lanes_kernel<T, G32, ZERO>, p, 16, s);
}

template <typename T>
twell_status quant(const QuantParams& p, int32_t group, bool vec, cudaStream_t s) {
  if (p.zero)
    return group == 32   ? quant<T, 1, true>(p, vec, s)
           : group == 64 ? quant<T, 2, true>(p, vec, s)
                         : quant<T, 4, true>(p, vec, s);
  return group == 32   ? quant<T, 1, false>(p, vec, s)
         : group == 64 ? quant<T, 2, false>(p, vec, s)
                       : quant<T, 4, false>(p, vec, s);
}

template <typename T, int G32>
twell_status dequant(const DequantParams& p, bool vec, cudaStream_t s) {
  return vec ? enqueue(dequant_int4_kernel<T, G32>, p, 128, s)
             : enqueue(dequant_int4_lanes_kernel<T, G32>, p, 32, s);
}

template <typename T>
twell_status dequant(const DequantParams& p, int32_t group, bool vec, cudaStream_t s) {
  return group == 32   ? dequant<T, 1>(p, vec, s)
         : group == 64 ? dequant<T, 2>(p, vec, s)
                       : dequant<T, 4>(p, vec, s);
}

// Blocks of the matrix, or 0 where there are more than the kernels index.
uint32_t blocks_of(const twell_int4_t& w) {
  const int64_t nb = (static_cast<int64_t>(w.K) + kInt4Block - 1) / kInt4Block;
  return w.rows > 0x7fffffffLL / nb ? 0u : static_cast<uint32_t>(w.rows * nb);
}

}  // namespace
}  // namespace twell

extern "C" twell_status twell_quant_int4(const void* src, int32_t type, int64_t ld,
                                         const twell_int4_t* out, void* stream) {
  using namespace twell;
  twell_status st = check_int4(out);
  if (st != TWELL_OK) return st;
  if (type != TWELL_BF16 && type != TWELL_F32) return TWELL_ERR_INVALID;
  if (out->rows == 0) return TWELL_OK;
  const int elem = type == TWELL_BF16 ? 2 : 4;
  if (!src || reinterpret_cast<uintptr_t>(src) % elem != 0 || ld < out->K)
    return TWELL_ERR_INVALID;
  DeviceInfo dev;
  if ((st = require_sm103(&dev)) != TWELL_OK) return st;
  const uint32_t items = blocks_of(*out);
  if (items == 0) return TWELL_ERR_UNSUPPORTED;
  const uint32_t nb = items / static_cast<uint32_t>(out->rows);
  const QuantParams p{src,   ld,          static_cast<uint32_t>(out->K),
                      items, divisor(nb), out->code, out->scale, out->zero};
  const bool vec = out->K % 8 == 0 && aligned16(src) && (ld * elem) % 16 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return type == TWELL_BF16 ? quant<uint16_t>(p, out->group, vec, s)
                            : quant<float>(p, out->group, vec, s);
}

extern "C" twell_status twell_dequant_int4(const twell_int4_t* w, void* out, int32_t type,
                                           int64_t ld, void* stream) {
  using namespace twell;
  twell_status st = check_int4(w);
  if (st != TWELL_OK) return st;
  if (type != TWELL_BF16 && type != TWELL_F32) return TWELL_ERR_INVALID;
  if (w->rows == 0) return TWELL_OK;
  const int elem = type == TWELL_BF16 ? 2 : 4;
  if (!out || reinterpret_cast<uintptr_t>(out) % elem != 0 || ld < w->K) return TWELL_ERR_INVALID;
  DeviceInfo dev;
  if ((st = require_sm103(&dev)) != TWELL_OK) return st;
  const uint32_t items = blocks_of(*w);
  if (items == 0) return TWELL_ERR_UNSUPPORTED;
  const uint32_t nb = items / static_cast<uint32_t>(w->rows);
  const DequantParams p{view_of(*w), static_cast<uint32_t>(w->K), items, divisor(nb), out, ld};
  const bool vec = w->K % 8 == 0 && aligned16(out) && (ld * elem) % 16 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return type == TWELL_BF16 ? dequant<uint16_t>(p, w->group, vec, s)
                            : dequant<float>(p, w->group, vec, s);
}
