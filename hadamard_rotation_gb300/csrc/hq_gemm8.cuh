// hq_gemm8.cuh -- device code of the product of INT8 codes (sm_103a).
#pragma once

#include <cuda_bf16.h>

#include "hq_kernels.cuh"

namespace hq {

struct Gemm8Params {
  const int8_t *x, *w;
  const float *xs, *ws;
  int M, N, K;
  void* out;
  int out_f32;
};

// 64 x 64 outputs per CTA, integer products on the integer units.
__global__ void __launch_bounds__(256) k_gemm8(const __grid_constant__ Gemm8Params p) {
  __shared__ int xs[64][17], ws[64][17];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  int acc[4][4] = {};
  for (int k0 = 0; k0 < p.K; k0 += 64) {
    const int row = threadIdx.x / 4, at = threadIdx.x % 4 * 16;
    int4 a = make_int4(0, 0, 0, 0), b = a;
    if (m0 + row < p.M && k0 + at < p.K) a = *reinterpret_cast<const int4*>(p.x + static_cast<int64_t>(m0 + row) * p.K + k0 + at);
    if (n0 + row < p.N && k0 + at < p.K) b = *reinterpret_cast<const int4*>(p.w + static_cast<int64_t>(n0 + row) * p.K + k0 + at);
    xs[row][at / 4] = a.x, xs[row][at / 4 + 1] = a.y, xs[row][at / 4 + 2] = a.z, xs[row][at / 4 + 3] = a.w;
    ws[row][at / 4] = b.x, ws[row][at / 4 + 1] = b.y, ws[row][at / 4 + 2] = b.z, ws[row][at / 4 + 3] = b.w;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(xs[ty + 16 * i][k], ws[tx + 16 * j][k], acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= p.M || n >= p.N) continue;
      const float v = __fmul_rn(__fmul_rn(static_cast<float>(acc[i][j]), __ldg(p.xs + m)), __ldg(p.ws + n));
      const int64_t to = static_cast<int64_t>(m) * p.N + n;
      if (p.out_f32) static_cast<float*>(p.out)[to] = v;
      else static_cast<__nv_bfloat16*>(p.out)[to] = __float2bfloat16_rn(v);
    }
}

}  // namespace hq
