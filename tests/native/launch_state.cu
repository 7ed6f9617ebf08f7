// Checks of what the launching code keeps from call to call, against a runtime whose
// calls fail when told to (linked without the CUDA runtime; needs no GPU).
#include <cstdio>
#include <cstdlib>

#include "../../activation_sparse_gated_gate_gb300/csrc/common.cuh"

namespace {
int g_fail = 0;                      // the next calls that fail
cudaError_t g_last = cudaSuccess;    // what cudaGetLastError would return
int g_limit = 0;                     // the kernel's shared memory limit, 0 in a new context
int g_set = 0, g_launched = 0;       // limits set, kernels launched
int g_args[2];                       // the arguments of the last of them

cudaError_t result(bool ok) {
  if (ok && g_fail == 0) return cudaSuccess;
  if (g_fail > 0) --g_fail;
  g_last = cudaErrorInvalidValue;
  return g_last;
}
}  // namespace

extern "C" cudaError_t cudaGetLastError() {
  const cudaError_t e = g_last;
  g_last = cudaSuccess;
  return e;
}
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int bytes) {
  ++g_set;
  const cudaError_t e = result(true);
  if (e == cudaSuccess) g_limit = bytes;
  return e;
}
extern "C" cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* cfg, const void*, void** at) {
  const cudaError_t e = result(static_cast<int>(cfg->dynamicSmemBytes) <= g_limit);
  if (e == cudaSuccess) {
    ++g_launched;
    g_args[0] = *static_cast<int*>(at[0]);
    g_args[1] = *static_cast<char*>(at[1]);
  }
  return e;
}

#define CHECK(x)                                              \
  do {                                                        \
    if (!(x)) {                                               \
      std::printf("line %d: %s\n", __LINE__, #x);             \
      std::exit(1);                                           \
    }                                                         \
  } while (0)

void kernel(int, char) {}

void device_value() {
  using namespace twell;
  static DeviceValue v;
  DeviceInfo a, b;
  a.ordinal = 0;
  b.ordinal = kMaxDevices - 1;
  int asked = 0;
  const auto ask = [&](int answer) {
    return [&asked, answer] {
      ++asked;
      return answer;
    };
  };
  CHECK(v.get(a, ask(-1)) < 0);   // a failure is not kept
  CHECK(v.get(a, ask(7)) == 7);
  CHECK(v.get(a, ask(9)) == 7);   // an answer is
  CHECK(v.get(b, ask(0)) == 0);   // of its own device, and 0 is an answer
  CHECK(v.get(b, ask(5)) == 0);
  CHECK(v.get(a, ask(9)) == 7);
  CHECK(asked == 3);
}

void launches() {
  using namespace twell;
  DeviceInfo dev;
  dev.ordinal = 3;
  std::atomic<uint64_t> set{0};
  const cudaLaunchConfig_t cfg = launch_config(dim3(1), dim3(32), 90000, nullptr);
  const auto launch = [&] { return launch_large(kernel, 100000, cfg, dev, set, 5, 'c'); };
  g_fail = 1;  // the limit cannot be raised
  CHECK(launch() == TWELL_ERR_CUDA && g_launched == 0);
  CHECK(cudaGetLastError() == cudaSuccess);  // (the error is consumed)
  CHECK(launch() == TWELL_OK && g_launched == 1 && g_set == 2);
  CHECK(g_args[0] == 5 && g_args[1] == 'c');
  CHECK(launch() == TWELL_OK && g_launched == 2 && g_set == 2);  // raised once
  g_limit = 0;                                                   // a new context
  CHECK(launch() == TWELL_OK && g_launched == 3 && g_set == 3);
  CHECK(cudaGetLastError() == cudaSuccess);
  g_fail = 2;  // a launch that fails however the limit stands is not repeated for ever
  CHECK(launch() == TWELL_ERR_CUDA && g_launched == 3);
  CHECK(cudaGetLastError() == cudaSuccess);
  g_fail = 3;
  CHECK(launch() == TWELL_ERR_CUDA && g_fail == 2);  // (at the limit, not known any more)
  g_fail = 0;
  CHECK(launch() == TWELL_OK && g_launched == 4);
  // an error that somebody else left behind is not this launch's
  g_last = cudaErrorInvalidValue;
  CHECK(launch() == TWELL_OK && g_launched == 5);
}

int main() {
  device_value();
  launches();
  std::puts("ok");
  return 0;
}
