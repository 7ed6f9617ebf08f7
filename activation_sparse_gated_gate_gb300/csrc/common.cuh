// Host-side helpers shared by the library's translation units: device
// properties, argument checks and tensor-map encoding.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/twell.h"

namespace twell {

constexpr int kMaxDevices = 64;  // ordinals below it

// Properties of the current device, cached per device ordinal.
struct DeviceInfo {
  int ordinal = -1;
  int sm_count = 0;
  int cc_major = 0;
  int cc_minor = 0;
  int max_smem_optin = 0;
};

// Returns false if the current device cannot be queried.
bool current_device(DeviceInfo* out);

// TWELL_OK if the current device is an sm_103 part, else
// TWELL_ERR_UNSUPPORTED (or TWELL_ERR_CUDA if it cannot be queried).
twell_status require_sm103(DeviceInfo* info);

// Whether a call succeeded.  The error of one that did not is consumed, so that a
// later launch that asks for the last error does not take it for its own.
inline bool cuda_ok(cudaError_t e) {
  if (e == cudaSuccess) return true;
  cudaGetLastError();
  return false;
}

// A number that the runtime is asked for once on each device (a static of the code
// that needs it).  `ask` returns it, or a negative value where the question failed:
// that is returned but not kept, and the next call asks again.
class DeviceValue {
 public:
  template <typename Ask>
  int get(const DeviceInfo& dev, Ask ask) {
    int v = known_[dev.ordinal].load(std::memory_order_relaxed) - 1;
    if (v < 0) {
      v = ask();
      if (v >= 0) known_[dev.ordinal].store(v + 1, std::memory_order_relaxed);
    }
    return v;
  }

 private:
  std::atomic<int> known_[kMaxDevices] = {};  // the value + 1, 0 unknown
};

inline cudaLaunchConfig_t launch_config(dim3 grid, dim3 block, size_t smem, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  return cfg;
}

// For a kernel that may start before the stream's last kernel is done and waits for
// it by itself (ptx::grid_wait before the first use of what it wrote).  Everything
// before that kernel is done when this one starts.
inline cudaLaunchAttribute overlapped() {
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}

// Launches a kernel that uses more dynamic shared memory than kernels may by
// themselves: its limit is raised to `limit` before the first launch on each device
// (`set`: one bit per device, a static of the launching code).  A context created
// again after a reset has forgotten that, and a launch in it fails without enqueuing
// anything: the limit is then raised again and the launch repeated.
template <typename T>
struct Same {
  typedef T type;
};

template <typename... P>
twell_status launch_large(void (*kern)(P...), int limit, const cudaLaunchConfig_t& cfg,
                          const DeviceInfo& dev, std::atomic<uint64_t>& set,
                          const typename Same<P>::type&... args) {
  const uint64_t bit = 1ull << dev.ordinal;
  const void* k = reinterpret_cast<const void*>(kern);
  for (;;) {
    const bool known = (set.load(std::memory_order_relaxed) & bit) != 0;
    if (!known) {
      if (!cuda_ok(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, limit)))
        return TWELL_ERR_CUDA;
      set.fetch_or(bit, std::memory_order_relaxed);
    }
    void* at[] = {const_cast<void*>(static_cast<const void*>(&args))...};
    if (cuda_ok(cudaLaunchKernelExC(&cfg, k, at))) return TWELL_OK;
    set.fetch_and(~bit, std::memory_order_relaxed);
    if (!known) return TWELL_ERR_CUDA;
  }
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Validate a TwELL descriptor against the expected T and F.
twell_status check_twell(const twell_t* h, int32_t T, int32_t F, bool need_spill_n);

// Validate a hybrid descriptor against the expected T and F.
twell_status check_hybrid(const hybrid_t* h, int32_t T, int32_t F);

// 2-D bf16 tensor map over a row-major [outer][inner] array whose rows are
// `pitch` elements apart (pitch = inner when 0), box [box_outer][box_inner],
// 128-byte swizzle, zero fill out of bounds.
twell_status make_tmap_bf16_2d(CUtensorMap* map, const void* base, uint64_t inner,
                               uint64_t outer, uint32_t box_inner, uint32_t box_outer,
                               uint64_t pitch = 0);

// 2-D tensor map of 1-byte (u8), 2-byte (bf16) or 4-byte (fp32) elements over a row-major
// [outer][inner] array with rows `pitch_bytes` apart (a multiple of 16), box
// [box_outer][box_inner], zero fill out of bounds.  `swizzle` = 0 (none) or
// the span in bytes (32, 64, 128): in shared memory, the 16-byte chunk index
// within each span is XORed with address bits 7 and up (as many bits as the
// span has chunk-index bits); the inner box must fit in the span.
twell_status make_tmap_2d(CUtensorMap* map, int elem_bytes, const void* base, uint64_t inner,
                          uint64_t outer, uint32_t box_inner, uint32_t box_outer,
                          uint64_t pitch_bytes, int swizzle);

}  // namespace twell
