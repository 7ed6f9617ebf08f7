// Internal interface between the gate entry point and its decode-size
// kernel (gate_decode.cu).
#pragma once

#include "common.cuh"

namespace twell {

// Bound on each pipeline wait, in nanoseconds (twell_gate_pack_wait_limit).
uint64_t gate_wait_ns();

// True when the decode-size gate kernel handles T tokens of width D
// (1 <= T <= 256 and at least two K blocks of 64 to split).
bool gate_decode_supported(int32_t T, int32_t D);

// The up + down projection of twell_ffn_decode: with y, fused into the
// decode-size gate kernel (y [T][D] fp32, zeroed by the caller on the
// stream); with y NULL the kernel only prefetches the active neurons' W_u
// and W_d rows into L2 for the CUDA-core forward that follows it.
struct DecodeFfn {
  const uint16_t* Wu_t;  // [F][D] bf16
  const uint16_t* Wd;    // [F][D] bf16
  float* y;
  // with y NULL: [T][D] fp32 the kernel zeroes (NULL: none) for the forward
  // that follows, which adds into it
  float* y_zero;
};

// Enqueue the decode-size gate kernel (the caller has validated the
// arguments and zeroed out->spill_n on `s`; the kernel stores every word of
// out->block_bits itself).  With `ffn` not NULL the kernel also prefetches
// the active neurons' W_u and W_d rows into L2 and, when ffn->y is not NULL,
// adds every active entry's (h u) W_d[j, :] into it.
twell_status launch_gate_decode(const DeviceInfo& dev, const uint16_t* x, const uint16_t* Wg_t,
                                int32_t T, int32_t D, int32_t F, const twell_t* out,
                                float* z_debug, int32_t* status_dev, uint64_t wait_ns,
                                const DecodeFfn* ffn, cudaStream_t s);

// The same kernel on e4m3 operands with scales for each 128 of K (x per row, W
// per 128 x 128 block): true when it handles T tokens and K = D (all of a CTA's K
// blocks have their own TMEM columns).
bool decode_fp8_supported(int32_t T, int32_t K);

twell_status launch_gate_decode_fp8(const DeviceInfo& dev, const uint8_t* xq, int64_t ldx,
                                    const float* x_scale, const uint8_t* wq, int64_t ldw,
                                    const float* w_scale, int32_t T, int32_t D, int32_t F,
                                    const twell_t* out, float* z_debug, int32_t* status_dev,
                                    uint64_t wait_ns, cudaStream_t s);

// c [M][N] = a b^T of such operands (twell_gemm_fp8 with b_block 128).
twell_status launch_gemm_decode_fp8(const DeviceInfo& dev, const uint8_t* a, int64_t lda,
                                    const float* a_scale, const uint8_t* b, int64_t ldb,
                                    const float* b_scale, int32_t M, int32_t N, int32_t K,
                                    void* c, bool c_bf16, int64_t ldc, int32_t* status_dev,
                                    uint64_t wait_ns, cudaStream_t s);

}  // namespace twell
