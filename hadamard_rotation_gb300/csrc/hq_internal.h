// hq_internal.h -- library-private helpers shared by the translation units of libhq.
#pragma once

#include <cuda_runtime.h>

#include "hq.h"

namespace hq {

// Record `e` as the calling thread's last CUDA error (read by hq_last_cuda_error())
// and return HQ_ERR_CUDA.
hq_status cuda_fail(cudaError_t e);

// The device fault word of the int8 translation unit (hq_int8.cu has its own copy
// of g_hq_fault): read it into *fault and, when `clear`, reset it.  The caller has
// synchronised the device.
cudaError_t int8_fault_word(unsigned int* fault, bool clear);

// The same for the FP4 products' translation unit (hq_gemm.cu).
cudaError_t gemm_fault_word(unsigned int* fault, bool clear);
// And for the norms' (hq_norm.cu).
cudaError_t norm_fault_word(unsigned int* fault, bool clear);

// Allow `fn` `bytes` of dynamic shared memory on the current device (hq_smem.cu); remembered per kernel, device and
// context, so that a call of a few microseconds asks the runtime once.  Host threads may call it at the same time.
cudaError_t allow_smem(const void* fn, int bytes);

// How many clusters of `ranks` CTAs, each alone on its SM, run at a time (not sms / ranks: the SMs of a cluster
// lie in one part of the chip); asked for once per device, context and size.  `cfg`: a launch of them.
cudaError_t clusters_at_a_time(const void* fn, const cudaLaunchConfig_t& cfg, int ranks, int* n);

// Multiprocessors of the current device, asked for once per device.
cudaError_t sm_count(int* sms);

// Launch the bounded-wait self-test kernel of the int8 translation unit on `stream`.
cudaError_t int8_selftest_bounded_wait(cudaStream_t stream);

// Unique ID of the CUDA context current on the calling thread (the driver's cuCtxGetId, which
// never repeats within a process), or 0 when no context is current or the driver does not
// report one.  Per-device caches of context state (a symbol's device address, a kernel's
// shared-memory attribute) key on it: after cudaDeviceReset the device's primary context is a
// new one with a new ID, so a cache entry of the old context no longer matches.
unsigned long long context_id();

}  // namespace hq
