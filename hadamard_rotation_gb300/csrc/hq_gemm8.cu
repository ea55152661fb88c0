// hq_gemm8.cu -- C ABI of the product of INT8 codes (include/hq.h) and its launch logic.  The kernel is in
// hq_gemm8.cuh.
#include <cuda_runtime.h>

#include <cstdint>

#include "hq.h"
#include "hq_gemm8.cuh"
#include "hq_internal.h"

namespace {

using hq::cuda_fail;

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxExtent = (int64_t{1} << 31) - 1024;  // sizes and row indexes are ints in the kernel
constexpr int64_t kMaxK = int64_t{1} << 17;

}  // namespace

cudaError_t hq::gemm8_fault_word(unsigned int* fault, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(fault, g_hq_fault, sizeof(unsigned int));
  if (e == cudaSuccess && clear && *fault) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_hq_fault, &zero, sizeof(unsigned int));
  }
  return e;
}

extern "C" hq_status hq_gemm_int8(const int8_t* xq, const float* x_scales, const int8_t* wq, const float* w_scales,
                                  int64_t M, int64_t N, int64_t K, void* out, hq_dtype out_dtype, hq_stream stream) {
  if (out_dtype != HQ_F32 && out_dtype != HQ_BF16) return HQ_ERR_DTYPE;
  if (M < 0 || N < 0 || K < 0 || K % 16 != 0 || K >= kMaxK || M > kMaxExtent || N > kMaxExtent) return HQ_ERR_SHAPE;
  if (M == 0 || N == 0) return HQ_OK;
  if (!out || !x_scales || !w_scales || (K > 0 && (!xq || !wq))) return HQ_ERR_NULL;
  if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4) ||
      !aligned(out, out_dtype == HQ_F32 ? 4 : 2))
    return HQ_ERR_ALIGN;
  hq::Gemm8Params p = {};
  p.x = xq;
  p.w = wq;
  p.xs = x_scales;
  p.ws = w_scales;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.out = out;
  p.out_f32 = out_dtype == HQ_F32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((N + 63) / 64), static_cast<unsigned>((M + 63) / 64));
  cfg.blockDim = dim3(256);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, hq::k_gemm8, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? HQ_OK : cuda_fail(e);
}
