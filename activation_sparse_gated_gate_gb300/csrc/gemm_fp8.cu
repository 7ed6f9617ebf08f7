// Products of 8-bit floating-point operands with a scale for each block of
// 128:  C[m][n] = sum_kb a_scale[m][kb] b_scale[n or n/128][kb]
//                 sum_{k in block kb} a[m][k] b[n][k],
// a, b e4m3, and the gate product that ends in the TwELL epilogue.
//
// The scales change every 128 of K and along M, so a tile's sum cannot stay
// in the tensor core's accumulator: each K block is one set of four MMAs (32
// along K) into a TMEM buffer of its own, and the epilogue warps add it,
// scaled, to fp32 sums in registers while the next block's MMAs run into
// another buffer.  e4m3 products are exact in fp32, so the rounding is that of
// the fp32 sums alone.
//
// Persistent kernel, one CTA per SM, warps:
//   0         TMA producer: tiles of 128 bytes (K) by 128 rows, 128-byte
//             swizzle, through a ring of stages
//   1         TMEM allocator and MMA issuer
//   2, 3      copy the scales, a round of eight K blocks at a time, into shared
//             memory (lanes along the K blocks: a row's scales are neighbours)
//   4 ..      sets of four epilogue warps; a thread owns a row and 128 columns (64
//             without PAIR, where two sets share the 128 and halve the time a K
//             block's sums take): fp32 sums in registers (packed pairs), read
//             from TMEM in pieces of 16 columns, two in flight
// With PAIR two CTAs of a cluster share a tile of 256 x 256 (cta_group::2): each
// loads its 128 rows of a and half of b's 256 rows, the even CTA issues MMAs of
// M = 256, and each CTA's TMEM and epilogue hold its own 128 rows by 256
// columns.  A K block then costs a CTA 32 KB of loads for the MMA work that
// takes 48 KB in a 128 x 256 tile of its own.  Without PAIR the tile is
// 128 x 128.
//
// TMEM holds two K blocks of a tile, so in the steady state a block's sums have
// to be in registers 512 cycles after the block before it: the epilogue's
// chain (wait, read, multiply-add, hand the buffer back) is kept short and
// in registers: the scales are other warps' work, a block's barrier is tried
// before the block before is done, and the pair kernel's epilogue warps take
// registers from the others.  (The shared memory leaves so little L1 that a
// spilled register comes back from L2: at 8192 x 6144 x 1536 the same loop took
// 147 us with about 300 bytes of spills in 168 registers, 88 us with 30, and
// takes 73 us with none in 224: 2.1 PFLOP/s.)  At 8192 x 8192 x 8192 it takes 390-430 us
// (up to 2.8 PFLOP/s) as the power limit allows.
//
// Without PAIR TMEM holds four blocks and the MMAs themselves are the bound: 250
// cycles a block alone, 134 more while the copies fill the stages' shared memory,
// 570 with the epilogue's reads (512 x 4096 x 4096: 12.7 us).
//
// C leaves through shared memory: a warp stages 32 rows of 64 bytes (64-byte
// swizzle) and stores them with TMA, two such pieces in flight, which also
// clips the tile to M x N.
//
// With SPLIT (few tiles: few rows of a) the K blocks of a 128 x 128 tile are
// shared by the CTAs of a cluster; each leaves its sums in its stages' shared
// memory, and each then adds its share of the rows over all of them, in order.
//
// Waits are bounded as in the bf16 gate kernel: a role whose wait runs out sets
// TWELL_FLAG_TIMEOUT and leaves its loop, the others' waits then run out too; the
// CTA drains its TMA loads and stores and its MMAs before it frees the TMEM, and both
// CTAs of a pair meet once more before either leaves.
#include "common.cuh"
#include "gate.cuh"
#include "pack.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace twell {
namespace {

constexpr int BM = 128;
constexpr int BK = 128;             // e4m3 of a 128-byte row: one scale block
constexpr int kPiece = 16;            // columns of a TMEM read
constexpr int kTmemCols = 512;
constexpr int kSplitBlocks = 8;       // K blocks from which a ragged last round is split
// The pair kernel's 384 threads start with 168 registers each; its epilogue
// threads take 224 and the others keep 56 (4 x 56 + 8 x 224 = 12 x 168).  (With
// 208 and 88 nothing spills either, but the loop is scheduled less well: 403
// against 385 us at 8192^3.)
constexpr int kRegsStart = 168, kRegsEpi = 224, kRegsOther = 56;
constexpr uint64_t kDefaultWaitNs = 1000000000ull;
// rows of c and b: what a tile of 256 rounds up to stays in 32 bits
constexpr int32_t kMaxRows = 0x7fffffff - 255;

struct GemmFp8Params {
  int32_t M, N;
  int32_t num_n, num_kb;
  int32_t first_tile, num_tiles;   // this launch's tiles, of num_n to a row of them
  int32_t quarters;  // without PAIR: the tiles are quarters of 256 x 256 tiles
  int32_t split;     // SPLIT: CTAs of a cluster
  const float* a_scale;   // [M][num_kb]
  const float* b_scale;   // [N or ceil(N / 128)][num_kb]
  void* c;
  int64_t ldc;
  int32_t c_bf16, c_vec;  // c_vec: rows of C on 16-byte boundaries
  PackOut out;
  int32_t* status;
  uint64_t wait_ns;
};

template <bool PAIR, bool BROWS, bool PACK>
struct Fp8Cfg {
  static constexpr int CTAS = PAIR ? 2 : 1;
  static constexpr int BN = PAIR ? 256 : 128;   // columns of a tile
  static constexpr int STAGES = 5;
  static constexpr int A_BYTES = BM * BK;
  static constexpr int B_ROWS = BN / CTAS;      // rows of b a CTA loads
  static constexpr int B_BYTES = B_ROWS * BK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  // columns of an epilogue thread (packing wants a row's 128)
  static constexpr int COLS = PAIR || PACK ? 128 : 64;
  static constexpr int SETS = BN / COLS;
  static constexpr int EPI = 128 * SETS;        // epilogue threads
  static constexpr int BUFS = kTmemCols / BN;
  static constexpr int STAGING = PACK ? 0 : EPI * 128;  // of C: 128 bytes per epilogue thread
  // scales of a round of K blocks, [K block][row], two rounds; rows padded so
  // that the lanes, along K blocks first, hit different banks
  static constexpr int ROUND = 8;
  static constexpr int A_PITCH = 128 + 32 / ROUND;
  static constexpr int B_PER = BROWS ? BN : BN / 128;
  static constexpr int B_PITCH = B_PER + 32 / ROUND;
  static constexpr int SCALES = 2 * ROUND * (A_PITCH + B_PITCH) * 4;
  static constexpr int BAR_BYTES = 256;
  static constexpr int SMEM =
      STAGES * STAGE_BYTES + STAGING + SCALES + BAR_BYTES + 1024;
  static constexpr int THREADS = 128 + EPI;
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

// Where a launch's tile starts, in units of 128 rows and of 128 columns.
struct TileAt {
  int m, n;
};

template <bool PAIR>
__device__ __forceinline__ TileAt tile_at(const GemmFp8Params& p, int tile) {
  if (!PAIR && p.quarters) {
    const int big = p.first_tile + (tile >> 2);
    return {big / p.num_n * 2 + ((tile >> 1) & 1), big % p.num_n * 2 + (tile & 1)};
  }
  constexpr int S = PAIR ? 2 : 1;
  return {tile / p.num_n * S, tile % p.num_n * S};
}

// BROWS: b has a scale per row (of 1 x 128 blocks), else per 128 x 128 block.
// PACK: the sums are gate pre-activations and go to a TwELL.
// SPLIT: a cluster per tile.
template <bool PAIR, bool BROWS, bool PACK, bool SPLIT>
__global__ void __launch_bounds__(Fp8Cfg<PAIR, BROWS, PACK>::THREADS, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmap_a,
                    const __grid_constant__ CUtensorMap tmap_b,
                    const __grid_constant__ CUtensorMap tmap_c, const GemmFp8Params p) {
  using Cfg = Fp8Cfg<PAIR, BROWS, PACK>;
  constexpr int BN = Cfg::BN;
  constexpr int STAGES = Cfg::STAGES;
  constexpr int BUFS = Cfg::BUFS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = ptx::smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES * Cfg::A_BYTES;
  uint8_t* staging = smem + STAGES * Cfg::STAGE_BYTES;
  float* a_sc = reinterpret_cast<float*>(staging + Cfg::STAGING);  // [2][ROUND][A_PITCH]
  float* b_sc = a_sc + 2 * Cfg::ROUND * Cfg::A_PITCH;               // [2][ROUND][B_PITCH]
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + Cfg::STAGING + Cfg::SCALES);
  uint64_t* empty = full + STAGES;
  // Without PAIR a stage's barrier also says that its block's sums are there: one
  // commit a block, not two, for MMAs of N = 128, which a second one holds up (66 of
  // 570 cycles a block; of a pair's N = 256 none, and there the shared barrier's
  // second counter costs the epilogue 3 %).  A stage comes round no sooner than its
  // sums' TMEM buffer.
  static_assert(PAIR || STAGES >= BUFS, "a barrier that producer and epilogue wait for");
  uint64_t* tfull = PAIR ? empty + STAGES : empty;
  uint64_t* tempty = empty + STAGES + (PAIR ? BUFS : 0);
  uint64_t* sfull = tempty + BUFS;
  uint64_t* sempty = sfull + 2;
  uint64_t* drain = sempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile uint32_t* aborted = tmem_slot + 1;
  volatile uint32_t* peer_state = tmem_slot + 2;  // PAIR: the other CTA's fills and abort flag
  uint32_t n_loads = 0;  // TMA stage fills issued (producer thread)

  if (PAIR) ptx::grid_launch_next();  // (of a last round's quarters)
  const uint32_t crank = PAIR || SPLIT ? ptx::cluster_ctarank() : 0u;
  const uint32_t rank = PAIR ? crank : 0u;                    // this CTA's half of the tile
  const int ctas = PAIR ? 2 : SPLIT ? p.split : 1;
  const int unit = static_cast<int>(blockIdx.x) / ctas;
  const int units = static_cast<int>(gridDim.x) / ctas;
  // SPLIT: this CTA's K blocks
  const int kb_lo = SPLIT ? p.num_kb * static_cast<int>(crank) / ctas : 0;
  const int kb_hi = SPLIT ? p.num_kb * (static_cast<int>(crank) + 1) / ctas : p.num_kb;
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
      if (PAIR) ptx::mbar_init(&tfull[b], 1);
      ptx::mbar_init(&tempty[b], 4 * Cfg::SETS * Cfg::CTAS);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&sfull[i], 64);
      ptx::mbar_init(&sempty[i], 4 * Cfg::SETS);
    }
    ptx::mbar_init(drain, 1);
    *aborted = 0u;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    if (PAIR) {
      ptx::tmem_alloc_pair(tmem_slot, kTmemCols);
    } else {
      ptx::tmem_alloc(tmem_slot, kTmemCols);
      ptx::tmem_relinquish();
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (PAIR) ptx::cluster_sync();  // both CTAs' barriers and TMEM are there
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp < 4) {
    if (PAIR) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      if (lane == 0) {
        int stage = 0;
        uint32_t phase = 0;
        for (int tile = unit; tile < p.num_tiles; tile += units) {
          const TileAt at = tile_at<PAIR>(p, tile);
          const int m0 = (at.m + static_cast<int>(rank)) * BM;
          const int n0 = at.n * 128 + static_cast<int>(rank) * Cfg::B_ROWS;
          for (int kb = kb_lo; kb < kb_hi; ++kb) {
            if (!pipe_wait(&empty[stage], phase ^ 1u, p.wait_ns)) {
              flag(p.status, TWELL_FLAG_TIMEOUT);
              *aborted = 1u;
              goto done;
            }
            uint8_t* a_dst = sA + stage * Cfg::A_BYTES;
            uint8_t* b_dst = sB + stage * Cfg::B_BYTES;
            if (PAIR) {
              // the even CTA's barrier counts the bytes of both; the odd CTA's loads
              // of the same phase may be counted before it expects them
              if (rank == 0) ptx::mbar_arrive_expect_tx(&full[stage], 2 * Cfg::STAGE_BYTES);
              const uint32_t bar = ptx::mapa(ptx::smem_u32(&full[stage]), 0);
              ptx::tma_load_2d_pair(a_dst, &tmap_a, bar, kb * BK, m0);
              ptx::tma_load_2d_pair(b_dst, &tmap_b, bar, kb * BK, n0);
            } else {
              ptx::mbar_arrive_expect_tx(&full[stage], Cfg::STAGE_BYTES);
              ptx::tma_load_2d(a_dst, &tmap_a, &full[stage], kb * BK, m0);
              ptx::tma_load_2d(b_dst, &tmap_b, &full[stage], kb * BK, n0);
            }
            ++n_loads;
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        // every stage released: no commit of the even CTA is still on its way to
        // this CTA's barriers when the two part
        for (int i = 0; PAIR && i < STAGES; ++i) {
          if (!pipe_wait(&empty[stage], phase ^ 1u, p.wait_ns)) {
            flag(p.status, TWELL_FLAG_TIMEOUT);
            *aborted = 1u;
            goto done;
          }
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      // (the whole warp walks the loop, so that addresses and descriptors stay in
      // uniform registers; one elected lane issues)
      if (rank == 0) {
        constexpr uint32_t idesc = ptx::idesc_e4m3_f32(BM * Cfg::CTAS, BN);
        const uint64_t desc_a = ptx::sdesc_kmajor_sw128(ptx::smem_u32(sA));
        const uint64_t desc_b = ptx::sdesc_kmajor_sw128(ptx::smem_u32(sB));
        int stage = 0, buf = 0;
        uint32_t phase = 0, bphase = 0;
        for (int tile = unit; tile < p.num_tiles; tile += units) {
          for (int kb = kb_lo; kb < kb_hi; ++kb) {
            // (both barriers are asked before either answer is needed)
            const bool loaded = ptx::mbar_test_wait(&full[stage], phase);
            const bool room = ptx::mbar_test_wait(&tempty[buf], bphase ^ 1u);
            const bool late = (!loaded && !pipe_wait(&full[stage], phase, p.wait_ns)) ||
                              (!room && !pipe_wait(&tempty[buf], bphase ^ 1u, p.wait_ns));
            if (__any_sync(0xffffffffu, late)) {
              if (lane == 0) {
                flag(p.status, TWELL_FLAG_TIMEOUT);
                *aborted = 1u;
              }
              goto done;
            }
            ptx::tc_fence_after();
            const uint64_t da = desc_a + static_cast<uint32_t>(stage * (Cfg::A_BYTES / 16));
            const uint64_t db = desc_b + static_cast<uint32_t>(stage * (Cfg::B_BYTES / 16));
            const uint32_t d = tmem_base + static_cast<uint32_t>(buf * BN);
            if (ptx::elect_one_sync()) {
#pragma unroll
              for (int kk = 0; kk < BK / 32; ++kk) {  // 32 bytes along the swizzled row
                if (PAIR) ptx::mma_f8_pair(d, da + 2 * kk, db + 2 * kk, idesc, kk > 0 ? 1u : 0u);
                else ptx::mma_f8(d, da + 2 * kk, db + 2 * kk, idesc, kk > 0 ? 1u : 0u);
              }
              if (PAIR) {
                ptx::mma_commit_pair(&tfull[buf]);
                ptx::mma_commit_pair(&empty[stage]);
              } else {
                ptx::mma_commit(&empty[stage]);
              }
            }
            __syncwarp();
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
      // -------------------------------------------------------------- scales
      // thread (r, k) of 8 x 8 copies every eighth row's scale of K block k of a
      // round (zeros past M, N and the last block); a round has the time of the
      // eight K blocks before it to arrive
      constexpr int R = Cfg::ROUND, STEP = 64 / R;
      const int lt = threadIdx.x - 64, k = lt % R, r = lt / R;
      const int nb = BROWS ? p.N : (p.N + 127) / 128;
      int par = 0;
      uint32_t phase = 0;
      for (int tile = unit; tile < p.num_tiles; tile += units) {
        const TileAt at = tile_at<PAIR>(p, tile);
        const int a0 = (at.m + static_cast<int>(rank)) * BM + r;
        const int b0 = at.n * (BROWS ? 128 : 1) + r;
        for (int kb = kb_lo + k; kb < kb_hi + k; kb += R) {
          if (!pipe_wait(&sempty[par], phase ^ 1u, p.wait_ns)) {
            flag(p.status, TWELL_FLAG_TIMEOUT);
            *aborted = 1u;
            goto done;
          }
          const uint32_t a_to = ptx::smem_u32(a_sc + (par * R + k) * Cfg::A_PITCH + r);
          const uint32_t b_to = ptx::smem_u32(b_sc + (par * R + k) * Cfg::B_PITCH + r);
          for (int j = 0; j < 128; j += STEP) {
            const bool in = a0 + j < p.M && kb < p.num_kb;
            ptx::cp_async4(a_to + j * 4,
                           p.a_scale + (in ? static_cast<size_t>(a0 + j) * p.num_kb + kb : 0),
                           in ? 4u : 0u);
          }
          for (int j = 0; r + j < Cfg::B_PER; j += STEP) {
            const bool in = b0 + j < nb && kb < p.num_kb;
            ptx::cp_async4(b_to + j * 4,
                           p.b_scale + (in ? static_cast<size_t>(b0 + j) * p.num_kb + kb : 0),
                           in ? 4u : 0u);
          }
          ptx::cp_async_commit();
          ptx::cp_async_wait<0>();
          ptx::mbar_arrive(&sfull[par]);
          par ^= 1;
          if (par == 0) phase ^= 1u;
        }
      }
    }
  } else {
    if (PAIR) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;                // TMEM lane quarter this warp may read
    constexpr int COLS = Cfg::COLS, kPieces = COLS / kPiece;
    const int set = (warp - 4) >> 2;       // its COLS columns of the tile
    // A thread's sums: of row 32 q + lane, all COLS columns; or with FRAG, of rows
    // 32 q + 8 i + lane / 4, i = 0..3, columns 8 j + 2 (lane mod 4) and the next: it
    // needs the scales of a quarter of the columns only.  Reading those of all of
    // them from shared memory costs a pair more than the slower TMEM reads of 16
    // lanes (345 against 368 us at dW's 9216 x 2304 x 16384), a single CTA less
    // (47.9 against 44.8 us at 283 x 3424 x 15616).
    constexpr bool FRAG = PAIR && BROWS;
    const int row = FRAG ? q * 32 + (lane >> 2) : q * 32 + lane;
    constexpr int kRound = Cfg::ROUND;
    int buf = 0, par = 0, stage = 0;
    const int& next = PAIR ? buf : stage;  // of tfull
    uint32_t phase = 0, sphase = 0;
    const uint32_t tempty0 = ptx::mapa(ptx::smem_u32(tempty), PAIR ? 0 : crank);
    const uint32_t taddr0 =
        tmem_base + static_cast<uint32_t>(set * COLS) + (static_cast<uint32_t>(q * 32) << 16);
    bool ready = false;  // the next block's barrier has been seen complete
    // PACK, for a warp that gives up: its slices of this tile and of those it would have
    // come to hold nothing, so that whoever reads the TwELL finds them empty
    const auto leave_empty = [&](int tile) {
      if constexpr (PACK) {
        for (; tile < p.num_tiles; tile += units) {
          const TileAt at = tile_at<PAIR>(p, tile);
          const int t = (at.m + static_cast<int>(rank)) * BM + row, kt = at.n + set;
          if (t < p.M && kt < p.out.n_t) p.out.cnt[static_cast<size_t>(t) * p.out.n_t + kt] = 0;
        }
      }
    };
    for (int tile = unit; tile < p.num_tiles; tile += units) {
      f32x2 acc[COLS / 2];
#pragma unroll
      for (int i = 0; i < COLS / 2; ++i) acc[i] = 0ull;
      for (int kb0 = kb_lo; kb0 < kb_hi; kb0 += kRound) {
        // the decisions to leave must be warp-uniform: tcgen05.ld is warp-collective
        if (__any_sync(0xffffffffu, !pipe_wait(&sfull[par], sphase, p.wait_ns))) {
          if (lane == 0) {
            flag(p.status, TWELL_FLAG_TIMEOUT);
            *aborted = 1u;
          }
          leave_empty(tile);
          goto done;
        }
        const float* as = a_sc + par * kRound * Cfg::A_PITCH + row;
        const float* bs =
            b_sc + par * kRound * Cfg::B_PITCH +
            (BROWS ? set * COLS + (FRAG ? 2 * (lane & 3) : 0) : set * COLS / 128);
        const int left = kb_hi - kb0;
        const float* as_end = as + (left < kRound ? left : kRound) * Cfg::A_PITCH;
        for (; as != as_end; as += Cfg::A_PITCH, bs += Cfg::B_PITCH) {
          if (!__all_sync(0xffffffffu, ready) &&
              __any_sync(0xffffffffu, !pipe_wait(&tfull[next], phase, p.wait_ns))) {
            if (lane == 0) {
              flag(p.status, TWELL_FLAG_TIMEOUT);
              *aborted = 1u;
            }
            leave_empty(tile);
            goto done;
          }
          ptx::tc_fence_after();
          const uint32_t taddr = taddr0 + static_cast<uint32_t>(buf * BN);
          uint32_t r[2][kPiece];
          // piece ch's sums and b's scales, the latter in pairs of columns
          f32x2 b2[2][BROWS ? (FRAG ? 2 : kPiece / 2) : 1];
          const auto read = [&](int ch) {
            const uint32_t at = taddr + static_cast<uint32_t>(ch * kPiece);
            if (FRAG) {
              ptx::tmem_ld_16x256b_x2(at, r[ch & 1]);
              ptx::tmem_ld_16x256b_x2(at + (16u << 16), r[ch & 1] + 8);
            } else {
              ptx::tmem_ld_32x32b_x16(at, r[ch & 1]);
            }
            const float* b = bs + ch * kPiece;
#pragma unroll
            for (int j = 0; BROWS && j < (FRAG ? 2 : kPiece / 4); ++j) {
              if (FRAG) {
                b2[ch & 1][j] = *reinterpret_cast<const f32x2*>(b + 8 * j);
              } else {
                const ulonglong2 b4 = *reinterpret_cast<const ulonglong2*>(b + 4 * j);
                b2[ch & 1][2 * j] = b4.x;
                b2[ch & 1][2 * j + 1] = b4.y;
              }
            }
          };
          read(0);
          f32x2 s2[FRAG ? 4 : 1];
#pragma unroll
          for (int i = 0; i < (FRAG ? 4 : 1); ++i) {
            const float s = BROWS ? as[8 * i] : as[0] * bs[0];
            s2[i] = pack2(__float_as_uint(s), __float_as_uint(s));
          }
          const uint32_t done_bar = tempty0 + buf * 8;
          if (++buf == BUFS) {
            buf = 0;
            if (PAIR) phase ^= 1u;
          }
          if (!PAIR && ++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
#pragma unroll
          for (int ch = 0; ch < kPieces; ++ch) {
            ptx::tmem_wait_ld();
            if (ch < kPieces - 1) {
              read(ch + 1);
              if (ch == kPieces - 2) ready = ptx::mbar_test_wait(&tfull[next], phase);
            } else {
              ptx::tc_fence_before();
              // (predicated; with b's row scales a branch is the faster: 45.0 against
              // 47.3 us at 283 x 3424 x 15616)
              if (!BROWS) ptx::mbar_arrive_cluster_relaxed(done_bar, lane == 0);
              else if (lane == 0) ptx::mbar_arrive_cluster_relaxed(done_bar, true);
            }
            const uint32_t* rr = r[ch & 1];
#pragma unroll
            for (int i = 0; i < kPiece / 2; ++i) {
              // FRAG: row i mod 4, columns 8 (i / 4)
              const uint32_t* v = FRAG ? rr + (i & 2) * 4 + (i >> 2) * 4 + (i & 1) * 2 : rr + 2 * i;
              fma2(acc[ch * (kPiece / 2) + i], pack2(v[0], v[1]),
                   FRAG    ? mul2(s2[i & 3], b2[ch & 1][i >> 2])
                   : BROWS ? mul2(s2[0], b2[ch & 1][i])
                           : s2[0]);
            }
          }
        }
        // the round's scales are read
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sempty[par]);
        par ^= 1;
        if (par == 0) sphase ^= 1u;
      }
      const TileAt at = tile_at<PAIR>(p, tile);
      const int m_blk = at.m + static_cast<int>(rank);
      const int col0 = at.n * 128 + set * COLS;
      // FRAG: f(row, column, its sum, the next column's) of the thread's sums in piece ch
      const auto each_pair = [&](int ch, auto&& f) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float lo, hi;
            unpack2(acc[ch * (kPiece / 2) + 4 * j + i], lo, hi);
            f(8 * i + (lane >> 2), 8 * j + 2 * (lane & 3), lo, hi);
          }
      };
      float z[COLS / 32][32];
      if (!FRAG) {
#pragma unroll
        for (int i = 0; i < COLS / 2; ++i)
          unpack2(acc[i], z[i / 16][2 * (i % 16)], z[i / 16][2 * (i % 16) + 1]);
      }
      if constexpr (PACK) {
        const int t = m_blk * BM + row;
        if (col0 < p.N)
          pack_row_slice<true>(p.out, z, t, t < p.M, m_blk, col0 / TWELL_TILE, lane, row, nullptr);
      } else if constexpr (SPLIT) {
        // (every stage has been read: the last block's barrier has been seen)
#pragma unroll
        for (int j = 0; j < COLS / 4; ++j) {
          const int c = set * (COLS / 4) + j;
          *reinterpret_cast<float4*>(smem + row * 512 + ((c ^ (row & 31)) << 4)) =
              make_float4(z[j / 8][j % 8 * 4], z[j / 8][j % 8 * 4 + 1], z[j / 8][j % 8 * 4 + 2],
                          z[j / 8][j % 8 * 4 + 3]);
        }
      } else {
        // pieces of 32 rows by 64 bytes, two in flight
        const int sw = (lane >> 1) & 3;
        uint8_t* mine = staging + (warp - 4) * 4096;
        const int t0 = m_blk * BM + q * 32;
        const int cols = p.c_bf16 ? 32 : 16;  // of a piece
        const auto store_piece = [&](int i, auto&& fill) {
          uint8_t* piece = mine + (i & 1) * 2048;
          const int col = col0 + i * cols;
          if (lane == 0) ptx::bulk_wait_read<1>();  // the piece before last has left
          __syncwarp();
          fill(piece);
          if (p.c_vec) {
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (t0 < p.M && col < p.N) ptx::tma_store_2d(&tmap_c, piece, col, t0);
              ptx::bulk_commit();
            }
          } else {
            // rows of C off 16-byte boundaries: element by element
            __syncwarp();
            for (int e = lane; e < 32 * cols; e += 32) {
              const int rr = e / cols, cc = e % cols, b = cc * (64 / cols);
              if (t0 + rr >= p.M || col + cc >= p.N) continue;
              const uint8_t* at = piece + rr * 64 + (((b >> 4) ^ ((rr >> 1) & 3)) << 4) + (b & 15);
              const size_t o = static_cast<size_t>(t0 + rr) * p.ldc + col + cc;
              if (p.c_bf16)
                static_cast<uint16_t*>(p.c)[o] = *reinterpret_cast<const uint16_t*>(at);
              else
                static_cast<float*>(p.c)[o] = *reinterpret_cast<const float*>(at);
            }
            __syncwarp();
          }
        };
        // byte b of row r of a piece
        const auto place = [&](uint8_t* piece, int r, int b) {
          return piece + r * 64 + (((b >> 4) ^ ((r >> 1) & 3)) << 4) + (b & 15);
        };
        const auto row_of = [&](int i, const uint32_t (&v)[16]) {
          store_piece(i, [&](uint8_t* piece) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<uint4*>(piece + lane * 64 + ((j ^ sw) << 4)) =
                  make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          });
        };
        if (p.c_bf16) {
#pragma unroll
          for (int i = 0; i < COLS / 32; ++i) {
            if constexpr (FRAG) {
              store_piece(i, [&](uint8_t* piece) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  each_pair(2 * i + h, [&](int r, int c, float lo, float hi) {
                    *reinterpret_cast<uint32_t*>(place(piece, r, 32 * h + 2 * c)) = bf16x2(lo, hi);
                  });
              });
            } else {
              uint32_t v[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] = bf16x2(z[i][2 * j], z[i][2 * j + 1]);
              row_of(i, v);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < COLS / 16; ++i) {
            if constexpr (FRAG) {
              store_piece(i, [&](uint8_t* piece) {
                each_pair(i, [&](int r, int c, float lo, float hi) {
                  *reinterpret_cast<float2*>(place(piece, r, 4 * c)) = make_float2(lo, hi);
                });
              });
            } else {
              uint32_t v[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(z[i / 2][i % 2 * 16 + j]);
              row_of(i, v);
            }
          }
        }
      }
    }
  }

done:
  __syncwarp();  // lanes idle during the producer / MMA loops rejoin lane 0
  if (!PACK && !SPLIT && warp >= 4 && lane == 0) ptx::bulk_wait_all();
  ptx::tc_fence_before();
  __syncthreads();
  bool drain_it = *aborted != 0u;  // read after the barrier: the same value in every thread
  // PAIR: the two tell each other what they issued; neither issues anything from here
  // on, and unless there is something to drain neither uses the other's barriers or TMEM.
  if (PAIR) {
    if (warp == 0 && lane == 0)
      ptx::st_cluster_u32(ptx::mapa(ptx::smem_u32(const_cast<uint32_t*>(peer_state)), crank ^ 1u),
                          (n_loads << 1) | *aborted);
    ptx::cluster_sync();
    drain_it |= (*peer_state & 1u) != 0u;
  }
  if (drain_it) {
    if (warp == 0 && lane == 0 && rank == 0) {
      // the last fill of each stage: the fills went round the ring in order, so stage s
      // got (n - s + STAGES - 1) / STAGES of them.  A pair's CTAs differ by one at
      // most (a stage's next fill waits for MMAs that read both CTAs' last): where the
      // other CTA's bytes will not come they are counted as arrived, where only its
      // bytes are on their way they are all that is expected.
      for (int s = 0; s < STAGES; ++s) {
        const uint32_t own = (n_loads + STAGES - 1 - s) / STAGES;
        const uint32_t other = PAIR ? ((*peer_state >> 1) + STAGES - 1 - s) / STAGES : own;
        if (own > other) ptx::mbar_complete_tx(&full[s], Cfg::STAGE_BYTES);
        if (own < other) ptx::mbar_arrive_expect_tx(&full[s], Cfg::STAGE_BYTES);
        const uint32_t n_s = own > other ? own : other;
        if (n_s > 0 && !ptx::mbar_wait(&full[s], (n_s - 1) & 1u)) break;
      }
    }
    if (warp == 1 && rank == 0 && ptx::elect_one_sync()) {
      ptx::tc_fence_after();
      // arrives once every MMA this thread issued is done
      if (PAIR) ptx::mma_commit_pair(drain);
      else ptx::mma_commit(drain);
      ptx::mbar_wait(drain, 0);
    }
    __syncwarp();
    ptx::tc_fence_before();
    if (PAIR) ptx::cluster_sync();
    else __syncthreads();
  }
  if (SPLIT) {
    ptx::cluster_sync();  // every CTA's sums of the tile are in its shared memory
    const TileAt at = tile_at<PAIR>(p, unit);
    const int left = p.M - at.m * BM, rows = left < BM ? left : BM;
    const uint32_t part = ptx::smem_u32(smem);
    // this CTA's rows: every ctas-th
    for (int i = threadIdx.x;; i += Cfg::THREADS) {
      const int row = (i >> 5) * ctas + static_cast<int>(crank), c = i & 31;
      if (row >= rows) break;
      const uint32_t off = static_cast<uint32_t>(row * 512 + ((c ^ (row & 31)) << 4));
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < ctas; ++k) {
        const float4 u = ptx::ld_cluster_f32x4(ptx::mapa(part, k) + off);
        v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
      }
      const int col = at.n * 128 + 4 * c, n = p.N - col;
      if (n <= 0) continue;
      const size_t o = static_cast<size_t>(at.m * BM + row) * p.ldc + col;
      const float f[4] = {v.x, v.y, v.z, v.w};
      uint16_t* c16 = static_cast<uint16_t*>(p.c) + o;
      float* c32 = static_cast<float*>(p.c) + o;
      if (p.c_vec && n >= 4) {
        if (p.c_bf16) store4(c16, f);
        else store4(c32, f);
      } else {
        for (int j = 0; j < 4 && j < n; ++j) {
          if (p.c_bf16) narrow(f[j], c16[j]);
          else c32[j] = f[j];
        }
      }
    }
    ptx::cluster_sync();  // nobody leaves while its sums are read
  }
  if (warp == 1) {
    ptx::tc_fence_after();
    if (PAIR) ptx::tmem_dealloc_pair(tmem_base, kTmemCols);
    else ptx::tmem_dealloc(tmem_base, kTmemCols);
  }
  if (!PAIR && !SPLIT && p.quarters) ptx::grid_wait();  // the call ends with both launches
}

template <bool PAIR, bool BROWS, bool PACK, bool SPLIT>
twell_status launch(const DeviceInfo& dev, const CUtensorMap& ma, const CUtensorMap& mb,
                    const CUtensorMap& mc, const GemmFp8Params& p, cudaStream_t s) {
  using Cfg = Fp8Cfg<PAIR, BROWS, PACK>;
  static_assert(Cfg::SMEM <= 232448, "shared memory budget");
  auto kern = gemm_fp8_kernel<PAIR, BROWS, PACK, SPLIT>;
  static std::atomic<uint64_t> set{0};
  const int ctas = SPLIT ? p.split : Cfg::CTAS;
  const int most = dev.sm_count / ctas;
  const int units = SPLIT || p.num_tiles < most ? p.num_tiles : most;
  cudaLaunchConfig_t cfg = launch_config(dim3(units * ctas), dim3(Cfg::THREADS), Cfg::SMEM, s);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  // quarters start as the full rounds' CTAs leave
  attr[1] = overlapped();
  cfg.attrs = attr;
  cfg.numAttrs = p.quarters ? 2 : 1;
  return launch_large(kern, Cfg::SMEM, cfg, dev, set, ma, mb, mc, p);
}

// Whether a pair's kernel may be launched: its register split draws on what the
// block starts with, which must not be less.
template <bool BROWS, bool PACK>
bool pair_ok(const DeviceInfo& dev) {
  static DeviceValue regs;
  return regs.get(dev, [] {
           cudaFuncAttributes at;
           return cuda_ok(cudaFuncGetAttributes(
                      &at, reinterpret_cast<const void*>(gemm_fp8_kernel<true, BROWS, PACK, false>)))
                      ? at.numRegs
                      : -1;
         }) == kRegsStart;
}

// CTAs of a cluster that share a tile's K blocks: as many as let every cluster run
// at once (the part holds 76 clusters of two of these CTAs, 36 of four and 15 of
// eight: they have to lie within a GPC) and leave each CTA four K blocks or more.
template <bool BROWS>
int split_for(const DeviceInfo& dev, int64_t tiles, int32_t num_kb) {
  static DeviceValue fit[3];
  int split = 1;
  for (int i = 0; i < 3; ++i) {
    const int n = 2 << i;
    if (num_kb < 4 * n) break;
    const int have = fit[i].get(dev, [n] {
      using Cfg = Fp8Cfg<false, BROWS, false>;
      cudaLaunchConfig_t cfg = launch_config(dim3(n), dim3(Cfg::THREADS), Cfg::SMEM, nullptr);
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = n;
      attr.val.clusterDim.y = 1;
      attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      const void* kern =
          reinterpret_cast<const void*>(gemm_fp8_kernel<false, BROWS, false, true>);
      int clusters;
      return cuda_ok(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          Cfg::SMEM)) &&
                     cuda_ok(cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg))
                 ? clusters
                 : -1;
    });
    if (tiles <= have) split = n;
  }
  return split;
}

// Whether few rows of a take the decode form: the tokens as the MMA's N, and K split
// over a cluster of two CTAs for each 128 rows of b.  It is the faster where all its
// clusters run at once: with the part's 76 a gate of 16 tokens, D 2048, takes 11.0
// against 15.3 us, and a product 9.1 against 9.5; with 80 16.8 against 15.7, and 14.7
// against 9.8.  And up to `most` rows, from where its epilogue, 16 of them a step,
// outweighs what the split gains.  Gate, D 512, F 8192: 9.6 against 10.7 us at 128
// tokens, 11.3 as either at 192, 12.8 against 10.4 at 256.  Product, N 8192: with K 512
// 5.5 against 5.4 at 32 rows, 6.0 against 5.4 at 64; with K 1024 6.9 against 7.7 at 32;
// with K 2048 8.5 against 9.3 for one row, 8.9 against 9.0 at 32, 9.6 against 9.5 at 64.
// (In a graph, b not in L2.)
constexpr int32_t kDecodeTokens = 128, kDecodeRows = 32;

bool decode_form(const DeviceInfo& dev, int32_t M, int32_t N, int32_t K, int32_t most) {
  return M <= most && 2 * ((static_cast<int64_t>(N) + 127) / 128) <= dev.sm_count &&
         decode_fp8_supported(M, K);
}

// Operand checks shared by the entry points: e4m3 rows on 16-byte boundaries.
bool operand_ok(const uint8_t* v, int64_t ld, int32_t K, const float* scale) {
  return v && scale && aligned16(v) && ld >= K && ld % 16 == 0 &&
         reinterpret_cast<uintptr_t>(scale) % 4 == 0;
}

template <bool PACK>
twell_status run(const DeviceInfo& dev, const uint8_t* a, int64_t lda, const uint8_t* b,
                 int64_t ldb, int32_t b_block, int32_t K, GemmFp8Params p, cudaStream_t s) {
  p.num_kb = static_cast<int32_t>((static_cast<int64_t>(K) + BK - 1) / BK);
  const bool brows = !PACK && b_block == 1;
  // Pairs of CTAs on 256 x 256 tiles when they still give every SM work, tiles
  // of 128 x 128 otherwise.  Pairs against single CTAs, K 2048: 1024 x 4864 (76 tiles, the
  // first with pairs) 13.2 against 13.5 us, with row scales 15.8 against 16.4, packed 19.6
  // against 20.6; 1024 x 4608 (72) 13.3 against 13.7, and at 40 to 64 tiles pairs would gain
  // 3 to 9 % (K 4096: 10 to 14 %), below 37 they lose to clusters over K (1536 x 1536: 12.4
  // against 8.7).  A few tiles into a second round they lose, 1024 x 5120 (80) 20.3
  // against 18.2, and from about 1536 x 5120 (120) they win: 20.6 against 22.6.
  const int64_t wide_m = (static_cast<int64_t>(p.M) + 255) / 256;
  const bool pair = 2 * wide_m * ((p.N + 255) / 256) >= dev.sm_count &&
                    (brows ? pair_ok<true, false>(dev) : pair_ok<false, PACK>(dev));
  const int64_t num_m = pair ? wide_m : (static_cast<int64_t>(p.M) + 127) / 128;
  p.num_n = pair ? (p.N + 255) / 256 : (p.N + 127) / 128;
  const int64_t tiles = num_m * p.num_n;
  if (tiles > 0x7fffffff / 4 - dev.sm_count) return TWELL_ERR_UNSUPPORTED;
  p.num_tiles = static_cast<int32_t>(tiles);
  CUtensorMap ma, mb, mc = {};
  twell_status st;
  if ((st = make_tmap_2d(&ma, 1, a, K, p.M, BK, BM, lda, 128)) != TWELL_OK) return st;
  if ((st = make_tmap_2d(&mb, 1, b, K, p.N, BK, 128, ldb, 128)) != TWELL_OK) return st;
  const int ce = p.c_bf16 ? 2 : 4;
  if (!PACK && p.c_vec &&
      (st = make_tmap_2d(&mc, ce, p.c, p.N, p.M, 64 / ce, 32, p.ldc * ce, 64)) != TWELL_OK)
    return st;
  if (pair) {
    // A last round of tiles that leaves most pairs idle runs as quarters, one per
    // CTA, in a launch of its own that starts as the full rounds' CTAs leave, where K
    // is long enough to pay for it (8192 x 6144 x 1536 with 12 blocks 72.9 -> 72.3 us,
    // with 8 blocks there is no difference; started early, 8192 x 2560 x 4096 takes 71.4,
    // else 73.5).  Packed, gate 8192 x D x 6144: D 1536 86.4 -> 84.3 us, 4096 170 -> 165,
    // 8192 317 -> 295; the most quarters at few blocks lose, 2500 x 1536 x 2560 24.3 -> 24.7.
    const int32_t pairs = dev.sm_count / 2;
    const int32_t rest = p.num_tiles % pairs;
    const bool split = p.num_kb >= kSplitBlocks && p.num_tiles > pairs && rest > 0 &&
                       4 * rest <= dev.sm_count;
    GemmFp8Params q = p;
    q.num_tiles = split ? p.num_tiles - rest : p.num_tiles;
    st = brows ? launch<true, true, false, false>(dev, ma, mb, mc, q, s)
               : launch<true, false, PACK, false>(dev, ma, mb, mc, q, s);
    if (st != TWELL_OK || !split) return st;
    p.first_tile = p.num_tiles - rest;
    p.num_tiles = 4 * rest;
    p.quarters = 1;
  }
  if constexpr (!PACK) {
    p.split = p.quarters ? 1
              : brows    ? split_for<true>(dev, p.num_tiles, p.num_kb)
                         : split_for<false>(dev, p.num_tiles, p.num_kb);
    if (p.split > 1)
      return brows ? launch<false, true, false, true>(dev, ma, mb, mc, p, s)
                   : launch<false, false, false, true>(dev, ma, mb, mc, p, s);
  }
  return brows ? launch<false, true, false, false>(dev, ma, mb, mc, p, s)
               : launch<false, false, PACK, false>(dev, ma, mb, mc, p, s);
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
  if (M > kMaxRows || N > kMaxRows) return TWELL_ERR_UNSUPPORTED;
  DeviceInfo dev;
  twell_status st;
  if ((st = require_sm103(&dev)) != TWELL_OK) return st;
  // Few rows: the decode form, unless the tiles are so few that larger clusters share
  // K (16 rows, N 2048, K 8192 with 16 tiles: 15.9 against 9.1 us).
  if (b_block == 128 && decode_form(dev, M, N, K, kDecodeRows) &&
      split_for<false>(dev,
                       (static_cast<int64_t>(M) + 127) / 128 * ((static_cast<int64_t>(N) + 127) / 128),
                       static_cast<int32_t>((static_cast<int64_t>(K) + 127) / 128)) < 4)
    return launch_gemm_decode_fp8(dev, a, lda, a_scale, b, ldb, b_scale, M, N, K, c,
                                  c_type == TWELL_BF16, ldc, status_dev, gate_wait_ns(),
                                  static_cast<cudaStream_t>(stream));
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
  // (a spilled slice is noted by its row and tile in 32 bits)
  if (T > kMaxRows || F > kMaxRows || static_cast<int64_t>(T) * (F / TWELL_TILE) > 0x7fffffff)
    return TWELL_ERR_UNSUPPORTED;
  DeviceInfo dev;
  if ((st = require_sm103(&dev)) != TWELL_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (decode_form(dev, T, F, D, kDecodeTokens))  // (it zeroes and stores all its counters and words itself)
    return launch_gate_decode_fp8(dev, xq, ldx, x_scale, wq, ldw, w_scale, T, D, F, out, z_debug,
                                  status_dev, gate_wait_ns(), s);
  if (!cuda_ok(cudaMemsetAsync(out->spill_n, 0, sizeof(int32_t), s))) return TWELL_ERR_CUDA;
  const size_t words = (static_cast<size_t>(T) + BM - 1) / BM * (F / 32);
  if (out->block_bits &&
      !cuda_ok(cudaMemsetAsync(out->block_bits, 0, words * sizeof(uint32_t), s)))
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
