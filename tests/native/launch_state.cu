// Checks of what the launching code keeps from call to call, against a runtime whose
// calls fail when told to (linked without the CUDA runtime; needs no GPU).
#include <cstdio>
#include <cstdlib>

#include "../../activation_sparse_gated_gate_gb300/csrc/common.cuh"

namespace {
int g_fail = 0;                      // the next calls that fail
cudaError_t g_last = cudaSuccess;    // what cudaGetLastError would return
int g_set = 0;                       // cudaFuncSetAttribute calls

cudaError_t result() {
  if (g_fail == 0) return cudaSuccess;
  --g_fail;
  g_last = cudaErrorInvalidValue;
  return g_last;
}
}  // namespace

extern "C" cudaError_t cudaGetLastError() {
  const cudaError_t e = g_last;
  g_last = cudaSuccess;
  return e;
}
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) {
  ++g_set;
  return result();
}

#define CHECK(x)                                              \
  do {                                                        \
    if (!(x)) {                                               \
      std::printf("line %d: %s\n", __LINE__, #x);             \
      std::exit(1);                                           \
    }                                                         \
  } while (0)

void kernel() {}

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

void errors_are_consumed() {
  using namespace twell;
  DeviceInfo dev;
  dev.ordinal = 3;
  std::atomic<uint64_t> set{0};
  g_fail = 1;
  CHECK(!smem_limit(kernel, 100000, dev, set));
  CHECK(cudaGetLastError() == cudaSuccess && set.load() == 0);
  CHECK(smem_limit(kernel, 100000, dev, set) && g_set == 2);
  CHECK(smem_limit(kernel, 100000, dev, set) && g_set == 2);
  g_last = cudaErrorInvalidValue;
  CHECK(smem_launched(cudaErrorInvalidValue, dev, set) == TWELL_ERR_CUDA);
  CHECK(cudaGetLastError() == cudaSuccess && set.load() == 0);
}

int main() {
  device_value();
  errors_are_consumed();
  std::puts("ok");
  return 0;
}
