// hq_smem.cu -- how much dynamic shared memory a kernel may be launched with (host code only).
#include <cuda_runtime.h>

#include <mutex>

#include "hq_internal.h"

// The attribute belongs to the kernel, the device and the context, and host threads launch one kernel with different
// sizes at the same time: set to a call's own size it could be lowered under another thread's launch.  So it is set
// once, to the most that the kernel can have, with the lock held until it is recorded.
cudaError_t hq::allow_smem(const void* fn, int bytes) {
  constexpr int kKernels = 128, kDevices = 64;
  struct Entry {
    const void* fn;
    int most[kDevices];                // by device: its limit less the kernel's static shared memory
    unsigned long long ctx[kDevices];  // and the context it is set in
  };
  static std::mutex mu;
  static Entry entries[kKernels];
  static int n = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  int at = 0;
  while (at < n && entries[at].fn != fn) ++at;
  const bool kept = at < kKernels && dev < kDevices;  // (else it is set to the same value again)
  unsigned long long ctx = hq::context_id();
  if (kept && at < n && ctx != 0 && entries[at].ctx[dev] == ctx)
    return bytes <= entries[at].most[dev] ? cudaSuccess : cudaErrorInvalidValue;
  cudaFuncAttributes attr;
  int most = 0;
  if ((e = cudaFuncGetAttributes(&attr, fn)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess) return e;
  most -= static_cast<int>(attr.sharedSizeBytes);
  if (bytes > most) return cudaErrorInvalidValue;
  if ((e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, most)) != cudaSuccess) return e;
  ctx = hq::context_id();  // (the calls may have made the context)
  if (kept && ctx != 0) {
    if (at == n) entries[n++].fn = fn;
    entries[at].most[dev] = most;
    entries[at].ctx[dev] = ctx;
  }
  return cudaSuccess;
}
