// Products of 8-bit floating-point operands with a scale for each block of
// 128:  C[m][n] = sum_kb a_scale[m][kb] b_scale[n or n/128][kb]
//                 sum_{k in block kb} a[m][k] b[n][k],
// a, b e4m3, and the gate product that ends in the TwELL epilogue.
//
// The scales change every 128 of K and along M, so a tile's sum cannot stay
// in the tensor core's accumulator: each K block is one set of four 128 x BN x 32
// MMAs into a TMEM buffer of its own, and the epilogue warps add it, scaled,
// to fp32 sums in registers while the next block's MMAs run into another
// buffer.  e4m3 products are exact in fp32, so the rounding is that of the
// fp32 sums alone.
//
// Persistent kernel, one CTA per SM, 2 + BN / 32 warps:
//   warp 0    TMA producer: tiles of 128 (K) bytes by 128 rows of a and BN rows
//             of b, 128-byte swizzle, through a ring of stages
//   warp 1    TMEM allocator and MMA issuer
//   the rest  BN / 128 sets of four warps; a thread owns a row and 128 columns:
//             128 fp32 sums in registers (packed fp32 pairs), read from TMEM in
//             pieces of 16 columns, two in flight
//
// Waits are bounded as in the bf16 gate kernel: a role whose wait runs out sets
// TWELL_FLAG_TIMEOUT, and the CTA drains its TMA loads and MMAs before it frees
// the TMEM.
#include "common.cuh"
#include "gate.cuh"
#include "pack.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace twell {
namespace {

constexpr int BM = 128;
constexpr int BK = 128;             // e4m3 of a 128-byte row: one scale block
constexpr int kTmemCols = 512;
constexpr uint64_t kDefaultWaitNs = 1000000000ull;

struct GemmFp8Params {
  int32_t M, N;
  int32_t num_n, num_kb, num_tiles;
  const float* a_scale;   // [M][num_kb]
  const float* b_scale;   // [N or ceil(N / 128)][num_kb]
  void* c;
  int64_t ldc;
  int32_t c_bf16, c_vec;  // c_vec: rows of C on 16-byte boundaries
  PackOut out;
  int32_t* status;
  uint64_t wait_ns;
};

template <int BN>
struct Fp8Cfg {
  static constexpr int STAGES = BN == 256 ? 4 : 6;
  static constexpr int A_BYTES = BM * BK;
  static constexpr int B_BYTES = BN * BK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int SETS = BN / 128;
  static constexpr int BUFS = kTmemCols / BN;
  static constexpr int STAGING = SETS * 128 * 128;  // 128 bytes per epilogue thread
  static constexpr int BAR_BYTES = 256;
  static constexpr int SMEM = STAGES * STAGE_BYTES + STAGING + BAR_BYTES + 1024;
  static constexpr int THREADS = 64 + 128 * SETS;
};

// A pipeline wait under the call's bound (short bounds are checked on every
// retry, the default one every 64).
__device__ __forceinline__ bool pipe_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  return limit_ns >= kDefaultWaitNs ? ptx::mbar_wait(bar, parity, limit_ns)
                                    : ptx::mbar_wait_strict(bar, parity, limit_ns);
}

typedef unsigned long long f32x2;

__device__ __forceinline__ f32x2 pack2(uint32_t lo, uint32_t hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ void fma2(f32x2& d, f32x2 a, f32x2 b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// BROWS: b has a scale per row (of 1 x 128 blocks), else per 128 x 128 block.
// PACK: the sums are gate pre-activations and go to a TwELL.
template <int BN, bool BROWS, bool PACK>
__global__ void __launch_bounds__(Fp8Cfg<BN>::THREADS, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmap_a,
                    const __grid_constant__ CUtensorMap tmap_b, const GemmFp8Params p) {
  using Cfg = Fp8Cfg<BN>;
  constexpr int STAGES = Cfg::STAGES;
  constexpr int BUFS = Cfg::BUFS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = ptx::smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES * Cfg::A_BYTES;
  uint8_t* staging = smem + STAGES * Cfg::STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + Cfg::STAGING);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + BUFS;
  uint64_t* drain = tempty + BUFS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile uint32_t* aborted = tmem_slot + 1;
  uint32_t n_loads = 0;  // stage fills issued (producer thread)

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&tmap_a);
    ptx::prefetch_tmap(&tmap_b);
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < BUFS; ++b) {
      ptx::mbar_init(&tfull[b], 1);
      ptx::mbar_init(&tempty[b], 4 * Cfg::SETS);
    }
    ptx::mbar_init(drain, 1);
    *aborted = 0u;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_slot, kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (int tile = blockIdx.x; tile < p.num_tiles; tile += gridDim.x) {
        const int m0 = tile / p.num_n * BM;
        const int n0 = tile % p.num_n * BN;
        for (int kb = 0; kb < p.num_kb; ++kb) {
          if (!pipe_wait(&empty[stage], phase ^ 1u, p.wait_ns)) {
            flag(p.status, TWELL_FLAG_TIMEOUT);
            *aborted = 1u;
            goto done;
          }
          ptx::mbar_arrive_expect_tx(&full[stage], Cfg::STAGE_BYTES);
          ptx::tma_load_2d(sA + stage * Cfg::A_BYTES, &tmap_a, &full[stage], kb * BK, m0);
          ptx::tma_load_2d(sB + stage * Cfg::B_BYTES, &tmap_b, &full[stage], kb * BK, n0);
          ++n_loads;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = ptx::idesc_e4m3_f32(BM, BN);
      int stage = 0, buf = 0;
      uint32_t phase = 0, bphase = 0;
      for (int tile = blockIdx.x; tile < p.num_tiles; tile += gridDim.x) {
        for (int kb = 0; kb < p.num_kb; ++kb) {
          if (!pipe_wait(&tempty[buf], bphase ^ 1u, p.wait_ns) ||
              !pipe_wait(&full[stage], phase, p.wait_ns)) {
            flag(p.status, TWELL_FLAG_TIMEOUT);
            *aborted = 1u;
            goto done;
          }
          ptx::tc_fence_after();
          const uint32_t a_addr = ptx::smem_u32(sA + stage * Cfg::A_BYTES);
          const uint32_t b_addr = ptx::smem_u32(sB + stage * Cfg::B_BYTES);
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            ptx::mma_f8(tmem_base + static_cast<uint32_t>(buf * BN),
                        ptx::sdesc_kmajor_sw128(a_addr + kk * 32),
                        ptx::sdesc_kmajor_sw128(b_addr + kk * 32), idesc, kk > 0 ? 1u : 0u);
          ptx::mma_commit(&empty[stage]);
          ptx::mma_commit(&tfull[buf]);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
          if (++buf == BUFS) {
            buf = 0;
            bphase ^= 1u;
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;                // TMEM lane quarter this warp may read
    const int set = (warp - 2) >> 2;       // its 128 columns of the tile
    const int row = q * 32 + lane;         // its thread's row
    const int tid = (threadIdx.x - 64) & 127;
    uint8_t* my_stage = staging + set * 128 * 128 + row * 128;
    // b's row scales of two K blocks (the staging area is the packing's)
    float* sb = reinterpret_cast<float*>(staging + set * 128 * 128);
    int buf = 0, par = 0;
    uint32_t bphase = 0;
    for (int tile = blockIdx.x; tile < p.num_tiles; tile += gridDim.x) {
      const int m_blk = tile / p.num_n;
      const int t = m_blk * BM + row;
      const int col0 = tile % p.num_n * BN + set * 128;
      const bool valid = t < p.M;
      const float* as = p.a_scale + static_cast<size_t>(valid ? t : 0) * p.num_kb;
      const int bcol = BROWS ? col0 + tid : col0;
      const bool bvalid = bcol < p.N;
      const float* bs =
          p.b_scale + static_cast<size_t>(bvalid ? (BROWS ? bcol : bcol / 128) : 0) * p.num_kb;
      float sa = valid ? as[0] : 0.0f;
      float sbv = bvalid ? bs[0] : 0.0f;
      f32x2 acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0ull;
      for (int kb = 0; kb < p.num_kb; ++kb) {
        const float s = BROWS ? sa : sa * sbv;
        // two buffers of b's scales in turn: whoever writes one again has
        // passed the barrier that follows its last reads
        if (BROWS) sb[par * 128 + tid] = sbv;
        if (kb + 1 < p.num_kb) {
          sa = valid ? as[kb + 1] : 0.0f;
          sbv = bvalid ? bs[kb + 1] : 0.0f;
        }
        // the decision must be the same in the whole warp (tcgen05.ld below is
        // warp-collective), and in the whole set where it meets at a barrier
        const bool late = !pipe_wait(&tfull[buf], bphase, p.wait_ns);
        if (BROWS ? ptx::bar_any(1 + set, 128, late) : __any_sync(0xffffffffu, late)) {
          if (lane == 0) {
            flag(p.status, TWELL_FLAG_TIMEOUT);
            *aborted = 1u;
          }
          goto done;
        }
        ptx::tc_fence_after();
        const uint32_t taddr = tmem_base + static_cast<uint32_t>(buf * BN + set * 128) +
                               (static_cast<uint32_t>(q * 32) << 16);
        const f32x2 s2 = pack2(__float_as_uint(s), __float_as_uint(s));
        uint32_t r[2][16];
        ptx::tmem_ld_32x32b_x16(taddr, r[0]);
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          ptx::tmem_wait_ld();
          if (ch < 7) {
            ptx::tmem_ld_32x32b_x16(taddr + (ch + 1) * 16, r[(ch + 1) & 1]);
          } else {
            ptx::tc_fence_before();
            if (lane == 0) ptx::mbar_arrive(&tempty[buf]);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            f32x2 f = s2;
            if (BROWS)
              f = mul2(s2, *reinterpret_cast<const f32x2*>(sb + par * 128 + ch * 16 + 2 * i));
            fma2(acc[ch * 8 + i], pack2(r[ch & 1][2 * i], r[ch & 1][2 * i + 1]), f);
          }
        }
        par ^= 1;
        if (++buf == BUFS) {
          buf = 0;
          bphase ^= 1u;
        }
      }
      float z[4][32];
#pragma unroll
      for (int i = 0; i < 64; ++i)
        unpack2(acc[i], z[i / 16][2 * (i % 16)], z[i / 16][2 * (i % 16) + 1]);
      if (PACK) {
        if (col0 < p.N)
          pack_row_slice(p.out, z, t, valid, m_blk, col0 / TWELL_TILE, lane, row, my_stage);
      } else if (valid) {
        const size_t o = static_cast<size_t>(t) * p.ldc + col0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int left = p.N - (col0 + 8 * i);
          if (left <= 0) break;
          float f[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = z[i / 4][(i % 4) * 8 + j];
          if (p.c_bf16) {
            uint16_t* c = static_cast<uint16_t*>(p.c) + o + 8 * i;
            if (p.c_vec && left >= 8) store8<true>(c, 8, f);
            else store8<false>(c, left, f);
          } else {
            float* c = static_cast<float*>(p.c) + o + 8 * i;
            if (p.c_vec && left >= 8) store8<true>(c, 8, f);
            else store8<false>(c, left, f);
          }
        }
      }
    }
  }

done:
  __syncwarp();  // lanes idle during the producer / MMA loops rejoin lane 0
  ptx::tc_fence_before();
  __syncthreads();
  if (*aborted) {  // read after the barrier: the same value in every thread
    if (warp == 0 && lane == 0) {
      // the last fill of each stage: fills went round the ring in order
      for (int s = 0; s < STAGES; ++s) {
        const uint32_t n_s = (n_loads + STAGES - 1 - s) / STAGES;
        if (n_s > 0 && !ptx::mbar_wait(&full[s], (n_s - 1) & 1u)) break;
      }
    }
    if (warp == 1 && lane == 0) {
      ptx::tc_fence_after();
      ptx::mma_commit(drain);  // arrives once every MMA this thread issued is done
      ptx::mbar_wait(drain, 0);
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
  }
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, kTmemCols);
  }
}

template <int BN, bool BROWS, bool PACK>
twell_status launch(const DeviceInfo& dev, const CUtensorMap& ma, const CUtensorMap& mb,
                    const GemmFp8Params& p, cudaStream_t s) {
  using Cfg = Fp8Cfg<BN>;
  static_assert(Cfg::SMEM <= 232448, "shared memory budget");
  auto kern = gemm_fp8_kernel<BN, BROWS, PACK>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM) !=
      cudaSuccess)
    return TWELL_ERR_CUDA;
  const int grid = p.num_tiles < dev.sm_count ? p.num_tiles : dev.sm_count;
  kern<<<grid, Cfg::THREADS, Cfg::SMEM, s>>>(ma, mb, p);
  return cudaGetLastError() == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}

// Operand checks shared by the entry points: e4m3 rows on 16-byte boundaries.
bool operand_ok(const uint8_t* v, int64_t ld, int32_t K, const float* scale) {
  return v && scale && aligned16(v) && ld >= K && ld % 16 == 0 &&
         reinterpret_cast<uintptr_t>(scale) % 4 == 0;
}

template <bool PACK>
twell_status run(const DeviceInfo& dev, const uint8_t* a, int64_t lda, const uint8_t* b,
                 int64_t ldb, int32_t b_block, int32_t K, GemmFp8Params p, cudaStream_t s) {
  const int64_t num_m = (static_cast<int64_t>(p.M) + BM - 1) / BM;
  p.num_kb = (K + BK - 1) / BK;
  // Wide tiles (N = 256) when they still give every SM work; N = 128 otherwise.
  const bool wide = num_m * ((p.N + 255) / 256) >= dev.sm_count;
  const int BN = wide ? 256 : 128;
  p.num_n = (p.N + BN - 1) / BN;
  const int64_t tiles = num_m * p.num_n;
  if (tiles > 0x7fffffff - dev.sm_count) return TWELL_ERR_UNSUPPORTED;
  p.num_tiles = static_cast<int32_t>(tiles);
  CUtensorMap ma, mb;
  twell_status st;
  if ((st = make_tmap_2d(&ma, 1, a, K, p.M, BK, BM, lda, 128)) != TWELL_OK) return st;
  if ((st = make_tmap_2d(&mb, 1, b, K, p.N, BK, BN, ldb, 128)) != TWELL_OK) return st;
  if (PACK || b_block == 128)
    return wide ? launch<256, false, PACK>(dev, ma, mb, p, s)
                : launch<128, false, PACK>(dev, ma, mb, p, s);
  return wide ? launch<256, true, false>(dev, ma, mb, p, s)
              : launch<128, true, false>(dev, ma, mb, p, s);
}

}  // namespace
}  // namespace twell

extern "C" twell_status twell_gemm_fp8(const uint8_t* a, int64_t lda, const float* a_scale,
                                       const uint8_t* b, int64_t ldb, const float* b_scale,
                                       int32_t b_block, int32_t M, int32_t N, int32_t K, void* c,
                                       int32_t c_type, int64_t ldc, int32_t* status_dev,
                                       void* stream) {
  using namespace twell;
  if (M < 0 || N < 0 || K <= 0 || (b_block != 1 && b_block != 128) ||
      (c_type != TWELL_BF16 && c_type != TWELL_F32))
    return TWELL_ERR_INVALID;
  if (M == 0 || N == 0) return TWELL_OK;
  if (!operand_ok(a, lda, K, a_scale) || !operand_ok(b, ldb, K, b_scale)) return TWELL_ERR_INVALID;
  const int ce = c_type == TWELL_BF16 ? 2 : 4;
  if (!c || ldc < N || reinterpret_cast<uintptr_t>(c) % ce != 0) return TWELL_ERR_INVALID;
  DeviceInfo dev;
  twell_status st;
  if ((st = require_sm103(&dev)) != TWELL_OK) return st;
  GemmFp8Params p{};
  p.M = M;
  p.N = N;
  p.a_scale = a_scale;
  p.b_scale = b_scale;
  p.c = c;
  p.ldc = ldc;
  p.c_bf16 = c_type == TWELL_BF16;
  p.c_vec = aligned16(c) && (ldc * ce) % 16 == 0;
  p.status = status_dev;
  p.wait_ns = gate_wait_ns();
  return run<false>(dev, a, lda, b, ldb, b_block, K, p, static_cast<cudaStream_t>(stream));
}

extern "C" twell_status twell_gate_pack_fp8(const uint8_t* xq, int64_t ldx, const float* x_scale,
                                            const uint8_t* wq, int64_t ldw, const float* w_scale,
                                            int32_t T, int32_t D, int32_t F, const twell_t* out,
                                            float* z_debug, int32_t* status_dev, void* stream) {
  using namespace twell;
  if (T < 0 || D <= 0 || F <= 0 || F % TWELL_TILE != 0) return TWELL_ERR_INVALID;
  twell_status st = check_twell(out, T, F, true);
  if (st != TWELL_OK) return st;
  if (T == 0) return TWELL_OK;
  if (!operand_ok(xq, ldx, D, x_scale) || !operand_ok(wq, ldw, D, w_scale))
    return TWELL_ERR_INVALID;
  if (z_debug && !aligned16(z_debug)) return TWELL_ERR_INVALID;
  DeviceInfo dev;
  if ((st = require_sm103(&dev)) != TWELL_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(out->spill_n, 0, sizeof(int32_t), s) != cudaSuccess) return TWELL_ERR_CUDA;
  const size_t words = (static_cast<size_t>(T) + BM - 1) / BM * (F / 32);
  if (out->block_bits &&
      cudaMemsetAsync(out->block_bits, 0, words * sizeof(uint32_t), s) != cudaSuccess)
    return TWELL_ERR_CUDA;
  GemmFp8Params p{};
  p.M = T;
  p.N = F;
  p.a_scale = x_scale;
  p.b_scale = w_scale;
  p.out = pack_out(*out, z_debug, status_dev);
  p.status = status_dev;
  p.wait_ns = gate_wait_ns();
  return run<true>(dev, xq, ldx, wq, ldw, 128, D, p, s);
}
