// Host threads that launch kernels with different sizes of shared memory, against a runtime made up here: its limit of a
// kernel on a device is what cudaFuncSetAttribute set last.  Built with the library's hq_smem.cu as C++.
#include <atomic>
#include <chrono>
#include <cstdio>
#include <cstring>
#include <thread>
#include <vector>

#include "hq_internal.h"

namespace {
constexpr int kKernels = 40, kDevices = 8, kOptin = 232448, kStatic = 2048;
std::atomic<int> limit[kKernels][kDevices];
std::atomic<int> sets{0};
std::atomic<bool> small_set{false};
std::atomic<int> hold{0};  // a call that sets this size takes until a smaller one is set, or 200 ms
thread_local int device = 0;
const char kernels[kKernels] = {};
int index_of(const void* fn) { return static_cast<int>(static_cast<const char*>(fn) - kernels); }
}  // namespace

extern "C" {
cudaError_t cudaGetDevice(int* d) {
  *d = device;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) {
  *v = kOptin;
  return cudaSuccess;
}
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) {
  std::memset(a, 0, sizeof *a);
  a->sharedSizeBytes = kStatic;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* fn, cudaFuncAttribute, int bytes) {
  if (bytes > kOptin - kStatic) return cudaErrorInvalidValue;
  limit[index_of(fn)][device] = bytes;
  ++sets;
  if (bytes < hold) small_set = true;
  if (hold != 0 && bytes >= hold)
    for (int i = 0; i < 200 && !small_set; ++i) std::this_thread::sleep_for(std::chrono::milliseconds(1));
  return cudaSuccess;
}
}

unsigned long long hq::context_id() { return 7 + static_cast<unsigned long long>(device); }

#define CHECK(x) \
  if (!(x)) return std::printf("failed: %s (line %d)\n", #x, __LINE__), 1

int main() {
  // One thread has the limit raised, and before that is recorded another asks for less.
  hold = 200000;
  const void* const fn = &kernels[0];
  std::thread large([&] { hq::allow_smem(fn, 200000); });
  std::this_thread::sleep_for(std::chrono::milliseconds(20));
  std::thread little([&] { hq::allow_smem(fn, 60000); });
  large.join();
  little.join();
  hold = 0;
  CHECK(hq::allow_smem(fn, 200000) == cudaSuccess);
  CHECK(limit[0][0] >= 200000);  // the launch that follows would run
  // Every kernel on every device is set once, and asked about again costs the runtime nothing.
  for (int pass = 0; pass < 2; ++pass) {
    const int before = sets;
    for (device = 0; device < kDevices; ++device)
      for (int k = 1; k < kKernels; ++k) {
        CHECK(hq::allow_smem(&kernels[k], 50000 + 1000 * (k + pass)) == cudaSuccess);
        CHECK(limit[k][device] >= 50000 + 1000 * (k + pass));
      }
    if (pass) CHECK(sets == before);
  }
  device = 0;
  // More than there is: refused, and nothing is lowered.
  CHECK(hq::allow_smem(fn, kOptin - kStatic + 1) != cudaSuccess);
  CHECK(limit[0][0] >= 200000);
  // Many threads at once.
  std::atomic<int> bad{0};
  std::vector<std::thread> all;
  for (int t = 0; t < 8; ++t)
    all.emplace_back([&, t] {
      for (int i = 0; i < 20000; ++i) {
        device = (t + i) % kDevices;
        const int k = (t * 7 + i) % kKernels, bytes = 50000 + (i * 97 + t * 31) % 150000;
        if (hq::allow_smem(&kernels[k], bytes) != cudaSuccess || limit[k][device] < bytes) ++bad;
      }
    });
  for (auto& t : all) t.join();
  CHECK(bad == 0);
  std::puts("ok");
  return 0;
}
