/*
 * twell.h - C ABI of the GB300 (sm_103a) activation-sparse gated FFN library.
 *
 * The library computes the gated feed-forward block of a ReLU Transformer,
 *     z = x W_g,   h = ReLU(z),   u = x W_u,   y = (h * u) W_d,
 * with the gate activation h held in TwELL (Tile-wise ELLPACK), and the
 * training step over the hybrid (ELL + dense backup) format.
 *
 * Sources ("Sparser, Faster, Lighter Transformer Language Models", summary
 * at gist.science, and the news article "Sakana AI and NVIDIA TwELL boosts
 * LLM training speed by 21.9%"):
 *   - ReLU replaces SiLU so the gate has exact zeros; an L1 term with
 *     coefficient 2e-5 on the FFN activations (news article, recipe list;
 *     paper section 2.A).
 *   - TwELL splits the gate columns into horizontal tiles the width of the
 *     matmul tile and is written in the epilogue of the gate matmul
 *     h_g = ReLU(x W_g), with no separate conversion kernel (paper section
 *     2.B.1; news article, epilogue paragraph).
 *   - One fused kernel does the up and down projections from the TwELL gate,
 *     computing dot products only for nonzeros (paper section 2.B.2).
 *   - Training converts TwELL to a hybrid format (compact ELL rows plus a
 *     dense backup for overflow rows) and runs sparse-to-dense and
 *     dense-to-sparse matmuls forward and backward (paper section 2.B.3).
 *
 * Conventions (every entry point):
 *   - bf16 tensors are passed as uint16_t bit patterns.  Pointers are device
 *     pointers unless stated otherwise.  The caller owns all memory; the
 *     library allocates nothing and never synchronises: all work is enqueued
 *     on `stream` (a cudaStream_t; NULL is the legacy default stream).
 *   - Weights are stored neuron-major, [F][D] row-major: Wg_t = W_g^T,
 *     Wu_t = W_u^T, Wd = W_d.  Activations x, y are [T][D] row-major.
 *   - Arguments are validated on the host before anything is enqueued.  A
 *     failure returns TWELL_ERR_INVALID (or TWELL_ERR_UNSUPPORTED) and
 *     enqueues nothing.  TWELL_ERR_CUDA means a CUDA call failed while
 *     enqueuing; cudaGetLastError() then holds the CUDA error.
 *   - Data-dependent conditions found on the device (a full spill list, a
 *     full dense backup, a wait that timed out) never trap: the kernels OR a
 *     TWELL_FLAG_* bit into *status_dev (a caller-owned device int32 the
 *     library never clears) and the outputs of the affected rows are then
 *     undefined.  Read it after synchronising the stream.
 *   - Alignment: every pointer 16-byte aligned; D % 8 == 0 (rows of 16-byte
 *     multiples); F % 128 == 0; tile == 128.
 */
#ifndef TWELL_H
#define TWELL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  TWELL_OK = 0,
  TWELL_ERR_INVALID = 1,      /* bad argument; nothing enqueued */
  TWELL_ERR_UNSUPPORTED = 2,  /* device is not sm_103 or a size limit is exceeded */
  TWELL_ERR_CUDA = 3          /* a CUDA runtime call failed while enqueuing */
} twell_status;

/* Bits OR-ed into *status_dev by the kernels. */
enum {
  TWELL_FLAG_SPILL_FULL = 1,  /* more (row, tile) slices overflowed W than spill_cap */
  TWELL_FLAG_DENSE_FULL = 2,  /* more overflow rows than the hybrid's max_dense */
  TWELL_FLAG_TIMEOUT = 4,     /* a pipeline wait exceeded its bound (about 1 s by default) */
  TWELL_FLAG_RANGE = 8,       /* a value exceeded the fp16 range of an fp16 operand */
  TWELL_FLAG_BOUNDS = 16      /* bounds-checking build only: a gathered or scattered
                                 index fell outside its buffer (access skipped) */
};

#define TWELL_TILE 128

/*
 * TwELL gate activation of a [T][F] matrix (paper section 2.B.1).
 * n_t = F / tile column tiles.  For row t and tile k (columns
 * [k*tile, (k+1)*tile)):
 *   cnt[t*n_t + k]            number of active entries (z > 0), 0..tile
 *   col[(t*n_t + k)*W + s]    local column of slot s (ascending), s < min(cnt, W)
 *   val[(t*n_t + k)*W + s]    z at that column, fp32 (the accumulator's value)
 * Slots at or beyond min(cnt, W) are not written and hold anything.
 * When cnt > W the (row, tile) keeps its first W actives in the slots and its
 * whole fp32 slice ReLU(z) (tile values) in the spill list:
 *   spill_slot[t*n_t + k]     index of that slice, meaningful only where cnt > W;
 *                             an index >= spill_cap means the list was full
 *   spill_rt[s]               t*n_t + k of slice s
 *   spill_val[s*tile + c]     fp32 ReLU(z) of column k*tile + c
 *   *spill_n                  slices requested by the last pack (device int32;
 *                             may exceed spill_cap, then TWELL_FLAG_SPILL_FULL)
 *   block_bits[b*(F/32) + w] optional (may be NULL): bit i of word w is set
 *                             iff column 32*w + i is active (z > 0) in some row
 *                             of the block of rows [128 b, 128 b + 128)
 *                             (every active column counts, spilled or not)
 * Sizes: val [T][n_t][W] float, col [T][n_t][W] uint8, cnt [T][n_t] uint8,
 * spill_slot [T][n_t] int32, spill_rt [spill_cap] int32,
 * spill_val [spill_cap][tile] float, block_bits [ceil(T/128)][F/32] uint32.
 * spill_* may be NULL when spill_cap = 0.  A reader trusts block_bits to
 * describe the same gate as the rest of the TwELL.
 * (The pages leave the value precision open; fp32 keeps the stored gate
 * exact to the accumulator, where bf16 alone would cost up to ~2% of RMS(y).)
 */
typedef struct {
  int32_t T;          /* rows (tokens) */
  int32_t F;          /* columns (d_ff), a multiple of tile */
  int32_t tile;       /* column tile width; must be TWELL_TILE */
  int32_t width;      /* W: slots per (row, tile), 1..tile */
  float* val;
  uint8_t* col;
  uint8_t* cnt;
  int32_t* spill_slot;
  int32_t spill_cap;
  int32_t* spill_n;
  int32_t* spill_rt;
  float* spill_val;
  uint32_t* block_bits;
} twell_t;

/*
 * Gate GEMM with the TwELL epilogue (paper section 2.B.1; news article,
 * epilogue paragraph): z = x W_g with fp32 accumulation on the tensor cores,
 * then, in the same kernel, every (row, tile) slice of z is packed into
 * `*out`.  No dense h is written.
 *   x        [T][D] bf16            Wg_t  [F][D] bf16 (= W_g^T)
 *   out      TwELL with out->T == T, out->F == F; the kernel resets
 *            *out->spill_n to 0 first (stream-ordered) and, when
 *            out->block_bits is not NULL, fills every word of it
 *   z_debug  optional [T][F] fp32 copy of z (NULL to skip), for checking
 *   status_dev  device int32, see TWELL_FLAG_*
 * T may be 0 (nothing enqueued).
 */
twell_status twell_gate_pack(const uint16_t* x, const uint16_t* Wg_t, int32_t T, int32_t D,
                             int32_t F, const twell_t* out, float* z_debug,
                             int32_t* status_dev, void* stream);

/*
 * Decode-sized forward in one call (paper sections 2.B.1 and 2.B.2
 * together): the gate GEMM z = x W_g with its TwELL epilogue, exactly as
 * twell_gate_pack (same `out`, same z_debug), then y = sum over the active
 * entries (t, j) of (h u) W_d[j, :] with u = x_t . W_u[:, j] (fp32).  Up to 8
 * tokens (or d_model > 3072) the projection runs inside the gate kernel: every
 * active entry of z -- slots and spill alike, so nothing is dropped when the
 * spill list is full -- adds its row to y with fp32 atomics.  With more
 * tokens the gate kernel prefetches the active neurons' W_u and W_d rows
 * into L2 and zeroes y while it streams W_g, and the call then runs
 * twell_ffn_fwd's kernel on the TwELL it wrote (whose rules then hold: a
 * missing spill slice is skipped and flagged).  Rows with no active entry
 * get y_t = 0.
 *   x   [T][D] bf16   Wg_t, Wu_t, Wd  [F][D] bf16   y  [T][D] fp32 (written;
 *   zeroed by the call, stream-ordered)   status_dev  device int32 (required)
 * Supports 1 <= T <= 256 with D > 64 (TWELL_ERR_UNSUPPORTED otherwise:
 * use twell_gate_pack + twell_ffn_fwd); D % 8 == 0, all pointers 16-byte
 * aligned.  Repeats agree to fp32 rounding, not bit for bit (atomics).
 */
twell_status twell_ffn_decode(const uint16_t* x, const uint16_t* Wg_t, const uint16_t* Wu_t,
                              const uint16_t* Wd, int32_t T, int32_t D, int32_t F,
                              const twell_t* out, float* y, float* z_debug, int32_t* status_dev,
                              void* stream);

/*
 * Bound, in nanoseconds, on each pipeline wait of the kernels launched by
 * later twell_gate_pack, twell_gate_pack_fp8 and twell_gemm_fp8 calls
 * (process-wide; 0 restores the default of 1e9 ns); returns the previous
 * bound.  A wait that runs out sets TWELL_FLAG_TIMEOUT; the kernel then waits
 * (up to 1 s each) for the TMA loads and MMAs it already issued, frees its
 * tensor memory and returns, so the context stays usable.  The slices of the
 * TwELL that were not packed are then empty (count 0).  Meant
 * for exercising that path (the paper has no counterpart); a bound of a
 * few nanoseconds makes every call time out.
 */
uint64_t twell_gate_pack_wait_limit(uint64_t ns);

/*
 * Fused up + down projection from a TwELL gate (paper section 2.B.2): for
 * each row t and each stored active entry (j, h), u = x_t . W_u[:, j]
 * (fp32), and y_t += (h u) W_d[j, :] (fp32 accumulation).  Rows with no
 * active entry get y_t = 0.
 *   x   [T][D] bf16, T = h->T      Wu_t, Wd  [F][D] bf16, F = h->F
 *   y   [T][D] fp32 (written; fp32 because a bf16 output alone can exceed a
 *       2e-2 * RMS(y) error where |y| reaches 10 * RMS)
 * A (row, tile) whose spill slice is missing (index >= spill_cap) is skipped
 * and TWELL_FLAG_SPILL_FULL is set.  With few rows (decode batches) a row is
 * split over several warps whose partial sums are added with float atomics
 * into y (zeroed first), so repeated calls agree to fp32 rounding, not bit
 * for bit; with many rows each row is summed by one warp in a fixed order.
 */
twell_status twell_ffn_fwd(const uint16_t* x, const twell_t* h, const uint16_t* Wu_t,
                           const uint16_t* Wd, int32_t D, float* y, int32_t* status_dev,
                           void* stream);

/*
 * Tensor-core variant of twell_ffn_fwd (paper section 2.B.2: up and down
 * projections of the active neurons only, built to keep the tensor cores
 * busy).  Same function, different arithmetic: for each block of 128 rows
 * the union U of the rows' active neurons (h->block_bits when it is not
 * NULL, else built from the slots and spill slices) is gathered, u = x W_u[:, U] is
 * one tcgen05 GEMM (bf16 in, fp32 out), a = h u is rounded to fp16 at each
 * row's own active neurons (0 at the union's other positions), and
 * y = a W_d[U, :] is a second tcgen05 GEMM on fp16 operands (W_d converted
 * from bf16 into the workspace, exactly for |w| >= 2^-14) with fp32
 * accumulation.  The fp16 rounding of h u adds up to 2^-11 |h u| (+ 2^-25)
 * per term to y; fp16 rather than bf16 keeps y within the 2e-2 * RMS bar
 * where a bf16 a (2^-8) did not (30-40 active terms of one row).  A |h u|
 * beyond the fp16 range (65504) sets TWELL_FLAG_RANGE.
 *   x [T][D] bf16, T = h->T, D a multiple of 64;  Wu_t, Wd [F][D] bf16,
 *   F = h->F <= 32768;  y [T][D] fp32 (every row written)
 *   Wd_f16  optional [F][D] fp16 copy of Wd (twell_to_f16); NULL: the call
 *           makes one in the workspace (one extra pass over W_d)
 *   ws: twell_workspace_size(TWELL_WS_FFN_FWD_TC, T, D, F, 0, 0) bytes,
 *       256-byte aligned (per-block unions and position prefixes, the
 *       [T][F] fp16 matrix of a in union order and the fp16 copy of W_d:
 *       about 2 (T + D) F bytes)
 * A (row, tile) whose spill slice is missing is skipped and
 * TWELL_FLAG_SPILL_FULL is set.  Results do not depend on how the work is
 * scheduled: repeated calls agree bit for bit.  T may be 0.
 * Returns TWELL_ERR_UNSUPPORTED for F > 32768, TWELL_ERR_INVALID for a D
 * that is not a multiple of 64 or a workspace that is too small.
 */
twell_status twell_ffn_fwd_tc(const uint16_t* x, const twell_t* h, const uint16_t* Wu_t,
                              const uint16_t* Wd, const uint16_t* Wd_f16, int32_t D, float* y,
                              void* ws, size_t ws_bytes, int32_t* status_dev, void* stream);

/*
 * twell_ffn_fwd_tc over blocks of rows grouped by activity: the rows are
 * first ordered by their count of active neurons (a stable sort into eight
 * buckets per octave of the count), then every block of 128 rows in that
 * order is processed as in twell_ffn_fwd_tc (h->block_bits is not read; the
 * blocks' unions are built from the slots and spill slices) and each y row
 * is written to its own token.  A block's union grows with its rows'
 * summed activity in a concave way, so when the per-row activity varies
 * widely (a heavy-tailed batch) the sorted blocks have a much smaller total
 * union and the GEMMs less work; when every row is about equally active
 * the sort and the copy of x in sorted order only add time.  Same
 * arguments, results and errors as twell_ffn_fwd_tc; the workspace is
 * twell_workspace_size(TWELL_WS_FFN_FWD_TC_SORTED, T, D, F, 0, 0) bytes (that
 * of twell_ffn_fwd_tc plus the row order and a copy of x: + 2 T D + 5 T
 * bytes and a little more).  Rows are summed in an order fixed by the data,
 * so repeated calls agree bit for bit.
 */
twell_status twell_ffn_fwd_tc_sorted(const uint16_t* x, const twell_t* h, const uint16_t* Wu_t,
                                     const uint16_t* Wd, const uint16_t* Wd_f16, int32_t D,
                                     float* y, void* ws, size_t ws_bytes, int32_t* status_dev,
                                     void* stream);

/*
 * fp16 copy of bf16 values (for the W_d operand of twell_ffn_fwd_tc, made
 * once for weights that do not change between calls): dst[i] = fp16(src[i]),
 * round to nearest; exact for |v| >= 2^-14 (bf16 has fewer significant
 * bits); |v| > 65504 becomes inf and sets TWELL_FLAG_RANGE.
 *   src, dst  device arrays of n elements, 16-byte aligned, n a multiple of 8
 */
twell_status twell_to_f16(const uint16_t* src, uint16_t* dst, size_t n, int32_t* status_dev,
                          void* stream);

/*
 * Hybrid training format (paper section 2.B.3): rows whose every tile count
 * is at most the ELL capacity C stay in a compact ELL matrix; the other
 * ("overflow") rows go to a dense backup.  Both lists are in ascending token
 * order.  Reading: a row overflows iff some tile count exceeds C (a count of
 * exactly C stays in ELL).
 *   *n_ell, *n_dense          device int32 row counts (n_dense is the true
 *                             number of overflow rows; rows past max_dense get
 *                             no dense row and TWELL_FLAG_DENSE_FULL is set)
 *   row_map[t]                i >= 0: ELL row i;  i < 0: dense row -(i+1)
 *   ell_rows[i]               token of ELL row i, i < n_ell
 *   ell_cnt[i*n_t + k]        count of ELL row i in tile k (<= C)
 *   ell_col/ell_val[(i*n_t + k)*C + s]   its entries, ascending, s < count;
 *                             padding slots (s >= count) hold column 0xFF
 *   dense_rows[i]             token of dense row i, i < min(n_dense, max_dense)
 *   dense_h[i*F + j]          fp32 ReLU(z) of that token (zeros where inactive)
 * Sizes: row_map, ell_rows [T] int32; ell_cnt [T][n_t] uint8;
 * ell_col [T][n_t][C] uint8; ell_val [T][n_t][C] float (T rows reserved since
 * every row may be an ELL row); dense_rows [max_dense] int32;
 * dense_h [max_dense][F] float.
 */
typedef struct {
  int32_t T;
  int32_t F;
  int32_t tile;       /* must be TWELL_TILE */
  int32_t cap;        /* C: ELL slots per (row, tile), 1..tile */
  int32_t max_dense;  /* rows reserved for the dense backup, >= 0 */
  int32_t* n_ell;
  int32_t* n_dense;
  int32_t* row_map;
  int32_t* ell_rows;
  float* ell_val;
  uint8_t* ell_col;
  uint8_t* ell_cnt;
  int32_t* dense_rows;
  float* dense_h;
} hybrid_t;

/*
 * TwELL -> hybrid conversion (paper section 2.B.3: a custom kernel converts
 * TwELL to the hybrid format).  Reads the TwELL `h` (slots and spill) and
 * fills `out` (out->T == h->T, out->F == h->F; C = out->cap may differ from
 * h->width: entries beyond W come from the spill slices).  Row lists and
 * counts are produced on the device; nothing is read back.  A (row, tile)
 * that needs its spill slice when the TwELL's spill list had no room for it
 * is stored empty (ELL count 0, every slot padding; zeros in a dense row)
 * and TWELL_FLAG_SPILL_FULL is set.
 */
twell_status twell_to_hybrid(const twell_t* h, const hybrid_t* out, int32_t* status_dev,
                             void* stream);

/* Workspace operations for twell_workspace_size. */
enum {
  TWELL_WS_HYBRID_FWD = 1,
  TWELL_WS_HYBRID_BWD = 2,
  TWELL_WS_HYBRID_FWD_TC = 3,
  TWELL_WS_HYBRID_BWD_TC = 4,
  TWELL_WS_FFN_FWD_TC = 5,        /* twell_ffn_fwd_tc; cap and max_dense are ignored */
  TWELL_WS_FFN_FWD_TC_SORTED = 6  /* twell_ffn_fwd_tc_sorted; cap and max_dense ignored */
};

/*
 * Bytes of device workspace `op` needs for a hybrid of T rows, width d_model
 * D, F columns, ELL capacity C and max_dense dense rows (0 on bad
 * arguments).  The workspace is scratch the call overwrites; it must be
 * 256-byte aligned and not shared by calls that may overlap on the GPU.
 */
size_t twell_workspace_size(int32_t op, int32_t T, int32_t D, int32_t F, int32_t cap,
                            int32_t max_dense);

/*
 * Hybrid training forward (paper section 2.B.3: dense-to-sparse and
 * sparse-to-dense matmuls over the hybrid format).
 *   ELL rows (CUDA cores): u = x_t . W_u[:, j] at every ELL entry, saved in
 *     u_ell (same layout as ell_val), and y_t = sum_j (h u) W_d[j, :].
 *   Dense rows (tensor cores): U = X_ov W_u, saved in U_dense [max_dense][F]
 *     fp32; y_ov = (H_ov * U) W_d with the fp32 product split into bf16 hi
 *     and lo halves (two MMAs), so the bf16 operand adds no rounding beyond
 *     about 2^-17 relative.
 *   x [T][D] bf16; Wu_t, Wd [F][D] bf16; y [T][D] fp32 (every row written,
 *   dense rows past max_dense excepted); u_ell [T][n_t][C] fp32;
 *   ws: twell_workspace_size(TWELL_WS_HYBRID_FWD, ...) bytes (may be NULL
 *   when max_dense == 0).  Dense rows of y sum split-K partial products with
 *   atomics, so they agree across calls to fp32 rounding, not bit for bit.
 */
twell_status hybrid_ffn_fwd(const uint16_t* x, const hybrid_t* h, const uint16_t* Wu_t,
                            const uint16_t* Wd, int32_t D, float* y, float* u_ell,
                            float* U_dense, void* ws, size_t ws_bytes, int32_t* status_dev,
                            void* stream);

/*
 * Hybrid training backward with the L1 term (paper section 2.B.3; L1
 * coefficient from the news article's recipe list).  For the loss
 * L(y) + l1_coeff * sum(h), with dy = dL/dy [T][D] fp32 and a = h * u:
 *   da = dy W_d^T;  du = da h;  dz = da u + l1_coeff at active entries;
 *   dx = dz W_g^T + du W_u^T;  dW_g^T = dz^T x;  dW_u^T = du^T x;
 *   dW_d = a^T dy.
 * ELL rows run on the CUDA cores (dense-to-sparse da, sparse-to-dense dx,
 * per-neuron records for the weight gradients); dense rows run on the tensor
 * cores with fp32 operands split into bf16 hi and lo halves.
 *   u_ell, U_dense   as written by hybrid_ffn_fwd for the same hybrid
 *   dx [T][D] fp32 (written);  dWg_t, dWu_t, dWd [F][D] fp32 (overwritten,
 *   not accumulated, in the weights' neuron-major layout)
 *   ws: twell_workspace_size(TWELL_WS_HYBRID_BWD, ...) bytes
 * The weight gradients sum per-neuron records in an order set by atomics,
 * and dense rows sum split-K partial products with atomics, so repeated
 * calls agree to fp32 rounding, not bit for bit.
 */
twell_status hybrid_ffn_bwd(const uint16_t* x, const hybrid_t* h, const float* u_ell,
                            const float* U_dense, const uint16_t* Wg_t, const uint16_t* Wu_t,
                            const uint16_t* Wd, int32_t D, const float* dy, float l1_coeff,
                            float* dx, float* dWg_t, float* dWu_t, float* dWd, void* ws,
                            size_t ws_bytes, int32_t* status_dev, void* stream);

/*
 * Tensor-core variants of hybrid_ffn_fwd / hybrid_ffn_bwd (the paper's
 * hybrid matmuls of section 2.B.3 mapped onto tcgen05 for activation
 * densities at which every 128-token block touches every 128-neuron tile, so
 * CUDA-core gathers of neuron rows cost more than dense tiles).  Same
 * arguments, outputs and dense-row handling as the CUDA-core entry points;
 * the ELL rows change:
 *   dense-to-sparse products (u, and da in the backward) are full tensor-core
 *   tiles X_ell W_u and dY_ell W_d^T of which only the ELL entries are kept;
 *   sparse-to-dense products (y, dx, dW_g^T, dW_u^T, dW_d) expand the ELL
 *   values tile by tile in shared memory into fp16 operands.
 * Apart from x and W_u in u (bf16, exact), every tensor-core operand of the
 * ELL rows is fp16 (relative rounding up to 2^-11): h u, W_d in y; and in
 * the backward x, the weights and, multiplied by a power of two s that puts
 * max(max |dy|, 2^-14 l1_coeff) in [0.5, 1), dy, dz and du (the fp32
 * products are divided by s again, which rounds nothing); dy in da and dz in
 * dx also carry an fp16 low half (a bias-like column of W_g sums a token's
 * dz, and every da of a token shares the token's dy rounding, into one
 * element of dx).  Weights and the
 * gathered rows are converted into the workspace by each call.  A value
 * beyond the fp16 range sets TWELL_FLAG_RANGE (the results are then not
 * meaningful).  Accumulation is fp32; results differ from the CUDA-core
 * entry points by that rounding.  Requires
 * D % 64 == 0 and C in {16, 32}; other shapes return TWELL_ERR_UNSUPPORTED.
 * Deterministic for the ELL rows (no atomics); dense rows as above.
 *   ws: twell_workspace_size(TWELL_WS_HYBRID_FWD_TC / _BWD_TC, ...) bytes.
 */
twell_status hybrid_ffn_fwd_tc(const uint16_t* x, const hybrid_t* h, const uint16_t* Wu_t,
                               const uint16_t* Wd, int32_t D, float* y, float* u_ell,
                               float* U_dense, void* ws, size_t ws_bytes, int32_t* status_dev,
                               void* stream);
twell_status hybrid_ffn_bwd_tc(const uint16_t* x, const hybrid_t* h, const float* u_ell,
                               const float* U_dense, const uint16_t* Wg_t, const uint16_t* Wu_t,
                               const uint16_t* Wd, int32_t D, const float* dy, float l1_coeff,
                               float* dx, float* dWg_t, float* dWu_t, float* dWd, void* ws,
                               size_t ws_bytes, int32_t* status_dev, void* stream);

/*
 * hybrid_ffn_fwd with no workspace argument, for callers that cannot
 * allocate device memory themselves (a loop whose memory budget is fixed up
 * front, a host program without access to a device allocator, code that must
 * not call cudaMalloc because it can synchronise the device).  The paper has
 * no counterpart: this is a packaging of hybrid_ffn_fwd, with the same
 * arguments, results and errors apart from the workspace.
 *   The workspace is a 64 MiB device array inside this library, held on
 *   every GPU that loads it until the process exits.  A hybrid whose
 *   forward workspace (twell_workspace_size(TWELL_WS_HYBRID_FWD, ...)) is
 *   larger returns TWELL_ERR_UNSUPPORTED and enqueues nothing.
 *   The first call on a device looks up the array's device address (with
 *   that device current) and caches it with the device's current context;
 *   make that first call before any stream capture.  After the context is
 *   destroyed and created again (cudaDeviceReset), the array lives at a new
 *   address: the next call sees the new context and looks it up again, so
 *   it too belongs outside stream capture.  The entry point allocates
 *   nothing.
 *   All calls share the array: calls that may overlap on the GPU race.
 */
twell_status hybrid_ffn_fwd_noalloc(const uint16_t* x, const hybrid_t* h, const uint16_t* Wu_t,
                                    const uint16_t* Wd, int32_t D, float* y, float* u_ell,
                                    float* U_dense, int32_t* status_dev, void* stream);

/* Element types of the operands below that may have either. */
typedef enum {
  TWELL_BF16 = 0,
  TWELL_F32 = 1
} twell_dtype;

/*
 * Residual addition and root-mean-square norm, the operator in front of a
 * (sparse) FFN:  s = x + r,  rstd = 1 / sqrt(mean(s^2) + eps),
 * y = s rstd w.  s and the statistics are fp32; y comes from the unrounded s.
 * (The pages leave the block around the FFN open.)
 *   x [T][D] of x_type, rows ldx elements apart (the other ld's likewise)
 *   r, total  [T][D] of r_type: the residual stream before and after (total = s
 *             rounded to r_type; may be r itself).  Both NULL: s = x
 *   w [D] of w_type
 *   y         [T][D] bf16, or NULL
 *   q, scale  [T][D] e4m3 and [T][ceil(D/128)] fp32: y with a scale for each
 *             128 columns as twell_quant_fp8 gives them, from the unrounded y; or
 *             both NULL.  At least one of y and q is written
 *   rstd      [T] fp32 for the backward, or NULL
 * Any D up to 16384 (TWELL_ERR_UNSUPPORTED above) and any row pitch; pointers
 * aligned to their elements.  Rows and pitches on 16-byte boundaries with
 * D % 8 == 0 are read and written 16 bytes at a time, others element by
 * element.  T may be 0.
 */
twell_status twell_rms_norm(const void* x, int32_t x_type, int64_t ldx, const void* r,
                            int32_t r_type, int64_t ldr, const void* w, int32_t w_type, int32_t T,
                            int32_t D, float eps, void* total, int64_t ldt, uint16_t* y,
                            int64_t ldy, uint8_t* q, int64_t ldq, float* scale, float* rstd,
                            void* stream);

/*
 * Its backward.  With n = total rstd and g = dy w:
 *   dx = rstd (g - n mean(g n)) + dtotal      dw = sum over rows of dy n
 * dx is the gradient of x and of r alike.
 *   total [T][D] of `type` and rstd [T] as the forward left them (without a
 *   residual, total is x);  dy [T][D] of dy_type;  dtotal, dx [T][D] of `type`
 *   (dtotal NULL: the stream ends here; dtotal may be dx itself);
 *   dw [D] fp32 (overwritten; zeros when T is 0)
 *   ws: twell_rms_norm_bwd_workspace(T, D) bytes, 16-byte aligned
 * dw is summed in a fixed order: repeated calls agree bit for bit.
 */
twell_status twell_rms_norm_bwd(const void* total, int32_t type, int64_t ld, const void* w,
                                int32_t w_type, const float* rstd, const void* dy,
                                int32_t dy_type, int64_t lddy, const void* dtotal, int64_t lddt,
                                int32_t T, int32_t D, void* dx, int64_t lddx, float* dw, void* ws,
                                size_t ws_bytes, void* stream);

/* Bytes of workspace of twell_rms_norm_bwd on the current device (0 on bad
 * arguments). */
size_t twell_rms_norm_bwd_workspace(int32_t T, int32_t D);

/*
 * Quantisation to 8-bit floating point (e4m3: 4 exponent and 3 mantissa bits,
 * largest value 448) with an fp32 scale for each block of block_rows x 128
 * elements, block_rows 1 (activations, gradients) or 128 (weights):
 *   amax = max(max |v| over the block, 2^-64),
 *   q = e4m3(v (448 / amax)) (nearest, ties to even),  scale = amax / 448,
 * so that v is about q scale.  448 / amax and its product with v are rounded to
 * fp32: what is a tie in exact arithmetic only may go either way.  A NaN becomes e4m3's NaN and does not enter
 * the block's maximum; infinities give an infinite scale and NaN.
 *   src       [R][C] of `type`, rows ld elements apart
 *   q, scale  [R][C] (rows ldq bytes apart), [ceil(R/block_rows)][ceil(C/128)]
 *   qt, scale_t  the transpose [C][R] (rows ldqt bytes apart),
 *             [ceil(C/block_rows)][ceil(R/128)]; with block_rows 1 its blocks are
 *             128 rows of one column of src, with 128 they are q's own
 * Either pair may be NULL.  R or C may be 0 (nothing is written).
 */
twell_status twell_quant_fp8(const void* src, int32_t type, int64_t ld, int32_t R, int32_t C,
                             int32_t block_rows, uint8_t* q, int64_t ldq, float* scale,
                             uint8_t* qt, int64_t ldqt, float* scale_t, void* stream);

/*
 * Product of two e4m3 operands with block scales on the tensor cores:
 *   c[m][n] = sum_k (a[m][k] a_scale[m][k/128]) (b[n][k] b_scale[n/b_block][k/128])
 * Sums are fp32: in the tensor core within a block of 128, in registers
 * across blocks, rounded once to c's type.
 *   a [M][K], a_scale [M][ceil(K/128)]
 *   b [N][K], b_scale [ceil(N/b_block)][ceil(K/128)], b_block 1 or 128
 *   lda, ldb  bytes between rows, multiples of 16;  a and b 16-byte aligned
 *   c [M][N] of c_type, rows ldc elements apart
 * Any K >= 1, M and N up to 2^31 - 256 (TWELL_ERR_UNSUPPORTED above; M or N 0:
 * nothing to do).  Bytes past K of a row are not
 * used.  A wait that runs out (twell_gate_pack_wait_limit's bound) sets
 * TWELL_FLAG_TIMEOUT in *status_dev (may be NULL), c then being undefined.
 * Repeated calls agree bit for bit.
 * A linear layer y = x W^T trains on the same product: dx takes (dy, W^T),
 * dW takes (dy^T, x^T) with b_block 1.
 */
twell_status twell_gemm_fp8(const uint8_t* a, int64_t lda, const float* a_scale, const uint8_t* b,
                            int64_t ldb, const float* b_scale, int32_t b_block, int32_t M,
                            int32_t N, int32_t K, void* c, int32_t c_type, int64_t ldc,
                            int32_t* status_dev, void* stream);

/*
 * twell_gate_pack from 8-bit operands: z = x W_g as twell_gemm_fp8 computes
 * it, packed into `out` in the same kernel.
 *   xq [T][D], x_scale [T][ceil(D/128)]        rows ldx bytes apart
 *   wq [F][D] (= W_g^T), w_scale [F/128][ceil(D/128)]   rows ldw bytes apart
 * Any D >= 1; T and F as M and N of twell_gemm_fp8 and T F / 128 below 2^31; the
 * operands' alignment as in twell_gemm_fp8, the rest as in twell_gate_pack.
 */
twell_status twell_gate_pack_fp8(const uint8_t* xq, int64_t ldx, const float* x_scale,
                                 const uint8_t* wq, int64_t ldw, const float* w_scale, int32_t T,
                                 int32_t D, int32_t F, const twell_t* out, float* z_debug,
                                 int32_t* status_dev, void* stream);

/*
 * Weights in 4 bits with a scale (and, where they are given, a zero point) for each
 * group of 32, 64 or 128 columns of a row:
 *   w[r][k] = (code[r][k] - zero[r][k/group]) scale[r][k/group],  code, zero in 0..15
 * A row is stored in blocks of 128 columns, 64 bytes each: column 32 i + 8 c + 2 n + o
 * of a block (i, c, n < 4, o < 2) is nibble n (from the lowest) of the 16 bits at byte
 * 8 (2 c + o) + 2 i.  With nb = ceil(K/128) blocks and G = nb 128/group groups a row:
 *   code   [rows][64 nb] bytes, 16-byte aligned
 *   scale  [rows][G] bf16
 *   zero   [rows][G] uint8 (values 0..15), or NULL: 8 everywhere
 * scale and zero aligned to what a block has of them (8, 4 or 2 and 4, 2 or 1 bytes).
 * What belongs to columns behind K is stored (codes 8, scales of whole groups 0, their
 * zero points 8) but not used.
 */
typedef struct {
  int64_t rows;
  int32_t K;
  int32_t group;
  uint8_t* code;
  uint16_t* scale;
  uint8_t* zero;
} twell_int4_t;

/*
 * Quantisation into that form.  Without zero points (out->zero NULL):
 *   scale = bf16(fl32(max |w| / 7)),  code = clamp(rint(w / scale), -8, 7) + 8
 * with them, lo = min(0, w) and hi = max(0, w) over the group:
 *   scale = bf16(fl32(fl32(hi - lo) / 15)),  zero = clamp(rint(-lo / scale), 0, 15),
 *   code = clamp(rint(w / scale) + zero, 0, 15)
 * rint is of the exact quotient, ties to even.  A group whose scale is 0 has codes (and
 * zero points) of 8; one with a NaN, an infinity or a scale beyond bf16 gets a NaN
 * as its scale.
 *   src  [rows][K] of `type`, rows ld elements apart
 * rows may be 0.  More than 2^31 - 1 blocks: TWELL_ERR_UNSUPPORTED.
 */
twell_status twell_quant_int4(const void* src, int32_t type, int64_t ld, const twell_int4_t* out,
                              void* stream);

/* The values of such weights: out [rows][K] of `type` (fp32 is exact, bf16 rounds once),
 * rows ld elements apart; limits as above. */
twell_status twell_dequant_int4(const twell_int4_t* w, void* out, int32_t type, int64_t ld,
                                void* stream);

/*
 * Product of a few rows with such weights, y = x W^T:
 *   y[t][n] = sum over groups g of scale[n][g] sum over k in g of (code - zero) x[t][k]
 * Sums are fp32 and rounded once to y's type.
 *   x  [T][K] bf16, rows ldx elements apart (on 16-byte boundaries with K % 8 == 0 they
 *      are read 16 bytes at a time)
 *   y  [T][w->rows] of y_type, rows ldy elements apart
 * Any T: every 32 rows of x read W once, so that it is an operator for decode batches
 * (twell_dequant_int4 gives the operand of a prompt's product).  T and w->rows may be 0.
 * w->rows up to 2^31 - 1, T up to 2^20 (TWELL_ERR_UNSUPPORTED above).  Repeated calls
 * agree bit for bit.
 */
twell_status twell_gemv_int4(const uint16_t* x, int64_t ldx, const twell_int4_t* w, int32_t T,
                             void* y, int32_t y_type, int64_t ldy, void* stream);

/* Activations of twell_moe_decode's gates. */
typedef enum {
  TWELL_RELU = 0,
  TWELL_SILU = 1
} twell_activation;

/*
 * Experts of a mixture: E gated FFNs of F neurons over D features, neuron-major as
 * everywhere ([E][F][D]): either three bf16 matrices, or three of 4 bits (rows = E F,
 * K = D, the same group); the other three pointers NULL.
 */
typedef struct {
  int32_t E, F, D;
  const uint16_t* Wg_t;
  const uint16_t* Wu_t;
  const uint16_t* Wd;
  const twell_int4_t* Wg4;
  const twell_int4_t* Wu4;
  const twell_int4_t* Wd4;
} twell_experts_t;

/*
 * A mixture-of-experts layer for a few tokens:
 *   logits = x router^T (fp32);  of each token the top_k largest, ties to the lowest
 *   expert, in falling order;  weight = softmax over the chosen (renormalise != 0) or over
 *   all E
 *   y[t] = sum over the slots of weight sum_j a(x . Wg[e][j]) (x . Wu[e][j]) Wd[e][j]
 * with a = SiLU or ReLU (a neuron whose gate is not positive for a token contributes nothing
 * to it, whatever its row of Wu holds; its rows of Wu and Wd are not read where that is so
 * for all of the expert's tokens, and where it is not, its row of Wd enters times 0).
 *   x        [T][D] bf16
 *   router   [E][D] of router_type, or NULL: ids and weights are given
 *   ids      [T][top_k] int32, weights [T][top_k] fp32: the choice, written with a router
 *            and read without one.  An id outside 0..E-1 is no expert (a padded row, an
 *            expert elsewhere); an expert may stand in several slots of a token.  A token
 *            without any gets y = 0
 *   y        [T][D] of y_type
 *   ws       twell_moe_decode_workspace(T, D, F, E, top_k) bytes, 16-byte aligned; calls
 *            that may overlap have their own
 * A NaN logit makes the token's weights NaN.  Sums and h are fp32 (h enters the last product
 * in three bf16 parts, all of its bits); y_type decides how y is rounded and nothing else.
 * An infinity in Wd (or a scale of it) times an h that is not zero is one, times zero a NaN.
 * Repeated calls agree bit for bit; a token's y may differ in its last bits with the tokens beside it, which
 * decide how sums are divided.
 * D % 8 == 0, any F.  Limits (TWELL_ERR_UNSUPPORTED above): T 256, T top_k 2048, top_k 32,
 * E 512, D 16384, (E + 256) ceil(F/16) 2^23.  T may be 0.
 */
twell_status twell_moe_decode(const uint16_t* x, int32_t T, const void* router,
                              int32_t router_type, const twell_experts_t* w, int32_t top_k,
                              int32_t act, int32_t renormalise, int32_t* ids, float* weights,
                              void* y, int32_t y_type, void* ws, size_t ws_bytes, void* stream);

/* Bytes of workspace of twell_moe_decode on the current device (0 on bad arguments), enough
 * for T tokens and for any fewer. */
size_t twell_moe_decode_workspace(int32_t T, int32_t D, int32_t F, int32_t E, int32_t top_k);

/*
 * FP32 FMA throughput probe (a measurement helper; the paper has no
 * counterpart).  Launches, on `stream`, one grid of two 512-thread CTAs per
 * SM in which every thread runs 16 independent register-resident chains
 * acc = acc * a + b for `iters` rounds: scalar fp32 FMAs (packed = 0) or
 * packed two-lane fma.rn.f32x2 (packed != 0, the form the CUDA-core kernels
 * use).  The caller times the launch with CUDA events; the work is
 * 2 * 16 * iters * (*threads) flops.  `out` (device, 16-byte aligned,
 * out_len >= *threads floats) receives one sum per thread; `*threads` (host)
 * is set before the launch.  TWELL_ERR_INVALID if out_len is too small.
 */
twell_status twell_probe_fma(int32_t packed, int32_t iters, float* out, size_t out_len,
                             int64_t* threads, void* stream);

/* Human-readable name of a status code (static storage). */
const char* twell_status_string(twell_status s);

/* Library version, (major << 16) | minor. */
int32_t twell_version(void);

#ifdef __cplusplus
}
#endif

#endif /* TWELL_H */
