// hq_tensor_map.h -- tensor maps of the products' launches (host code).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "hq.h"

namespace hq {

// cuTensorMapEncodeTiled through the runtime's driver entry points (the library does not link
// the driver library).
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return static_cast<EncodeTiledFn>(nullptr);
    }
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

// Bytes per store into rows of n elements at `out`: the alignment that every row has, up to 16.
inline int store_bytes(const void* out, int64_t n, hq_dtype dt) {
  const int64_t es = dt == HQ_F32 ? 4 : 2;
  int v = 16;
  while (n * es % v || reinterpret_cast<uintptr_t>(out) % v) v /= 2;
  return v;
}

// bf16 output [groups, rows, n], rows contiguous, in boxes of 32 rows x 64 elements, 128-byte swizzle.
inline bool encode_out(CUtensorMap* map, void* out, int64_t n, int64_t rows, int64_t groups) {
  const EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t size[3] = {static_cast<cuuint64_t>(n), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(groups)};
  const cuuint64_t stride[2] = {static_cast<cuuint64_t>(n * 2), static_cast<cuuint64_t>(n * rows * 2)};
  const cuuint32_t box[3] = {64, 32, 1}, step[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, out, size, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace hq
