// hq_gemm.cu -- C ABI of the FP4 products (include/hq.h) and their launch logic.  The kernel is
// in hq_gemm.cuh.
#include <cuda_runtime.h>

#include <cstdint>

#include "hq.h"
#include "hq_gemm.cuh"
#include "hq_internal.h"

namespace {

using hq::cuda_fail;
using hq::GemmKind;
using hq::GemmParams;

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// cuTensorMapEncodeTiled through the runtime's driver entry points (the library does not link
// the driver library).
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
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

// Codes [groups, rows, row_bytes] in boxes of box_rows rows x 128 bytes, 128-byte swizzle; what a
// box reaches past the rows of its group or past a row's end reads as code 0.
bool encode_codes(CUtensorMap* map, const uint8_t* q, int64_t row_bytes, int64_t rows, int64_t groups, int box_rows,
                  int dims) {
  const EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t size[3] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(groups)};
  const cuuint64_t stride[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(row_bytes * rows)};
  const cuuint32_t box[3] = {128, static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t step[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, static_cast<cuuint32_t>(dims), const_cast<uint8_t*>(q), size, stride,
            box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Bytes per store into rows of n elements at `out`: the alignment that every row has, up to 16.
int store_bytes(const void* out, int64_t n, hq_dtype dt) {
  const int64_t es = dt == HQ_F32 ? 4 : 2;
  int v = 16;
  while (n * es % v || !aligned(out, v)) v /= 2;
  return v;
}

// Multiprocessors of the current device, asked for once per device.
cudaError_t sm_count(int* sms) {
  static int known[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && known[dev]) {
    *sms = known[dev];
    return cudaSuccess;
  }
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && dev < 64) known[dev] = *sms;
  return e;
}

// One operand's codes as the launch needs them.
struct Codes {
  const uint8_t* q;
  int64_t row_bytes, rows, groups;
};

template <int KIND, bool MX, int T, bool LORA = false>
hq_status launch(GemmParams p, const Codes& a, const Codes& b, int64_t most_tiles, hq_stream stream) {
  using S = hq::GemmShape<KIND, MX, T, LORA>;
  auto kernel = hq::k_fp4_gemm<KIND, MX, T, LORA>;
  CUtensorMap ma, mb;
  if (!encode_codes(&ma, a.q, a.row_bytes, a.rows, a.groups, hq::kGemmLanes, 3) ||
      !encode_codes(&mb, b.q, b.row_bytes, b.rows, 1, S::kBox, 2))
    return cuda_fail(cudaErrorInvalidValue);
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e);
  const size_t smem = hq::gemm_smem_bytes(S::kSmemBytes, p.groups);
  if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem))) !=
      cudaSuccess)
    return cuda_fail(e);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(most_tiles < sms ? most_tiles : sms));
  cfg.blockDim = dim3(hq::kGemmThreads + (LORA ? hq::kLoraThreads : 0));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, ma, mb, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? HQ_OK : cuda_fail(e);
}

constexpr int64_t kMaxExtent = (int64_t{1} << 31) - 1024;  // sizes and row indexes are ints in the kernel

hq_status out_zero(void* out, int64_t n, hq_dtype dt, hq_stream stream) {
  const cudaError_t e = cudaMemsetAsync(out, 0, static_cast<size_t>(n) * (dt == HQ_F32 ? 4 : 2),
                                        static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HQ_OK : cuda_fail(e);
}

// What grouped_gemm and lora_gemm share: the operands of a product with ragged rows.
template <bool MX>
GemmParams rows_params(const uint8_t* xs, const float* x_sg, const uint8_t* ws, const float* w_sg, int64_t M, int64_t N,
                       int64_t K, int64_t groups, void* out, hq_dtype dt) {
  GemmParams p = {};
  p.k_tiles = static_cast<int>((K + (MX ? 127 : 63)) / (MX ? 128 : 64));
  p.tiles_a = static_cast<int>((N + 127) / 128);
  p.sfa = ws;
  p.sfa_group_bytes = static_cast<int64_t>(p.tiles_a) * p.k_tiles * 512;
  p.sfb = xs;
  p.sfb_row_bytes = static_cast<int>(K / (MX ? 32 : 16));
  p.sfb_mode = p.sfb_row_bytes % 16 == 0 && aligned(xs, 16) ? 16
               : p.sfb_row_bytes % 8 == 0 && aligned(xs, 8) ? 8
               : aligned(xs, 4)                             ? 4
                                                            : 1;
  p.sg_a = w_sg;
  p.sg_b = x_sg;
  p.groups = static_cast<int>(groups);
  p.extent = static_cast<int>(M);
  p.na = static_cast<int>(N);
  p.k = static_cast<int>(K);
  p.out = out;
  p.out_f32 = dt == HQ_F32;
  p.out_vec = store_bytes(out, N, dt);
  return p;
}

template <bool MX>
hq_status grouped_gemm(const uint8_t* xq, const uint8_t* xs, const float* x_sg, const uint8_t* wq, const uint8_t* ws,
                       const float* w_sg, const int32_t* offsets, int64_t M, int64_t N, int64_t K, int64_t E, void* out,
                       hq_dtype dt, hq_stream stream) {
  if (dt != HQ_F32 && dt != HQ_BF16) return HQ_ERR_DTYPE;
  if (M < 0 || N < 0 || K < 0 || E < 0 || K % 32 != 0) return HQ_ERR_SHAPE;
  if (M > kMaxExtent || N > kMaxExtent || K > kMaxExtent || E > hq::kGemmMaxGroups) return HQ_ERR_SHAPE;
  if (M == 0 || N == 0 || E == 0) return HQ_OK;
  if (!out || !offsets) return HQ_ERR_NULL;
  if (!aligned(out, dt == HQ_F32 ? 4 : 2) || !aligned(offsets, 4)) return HQ_ERR_ALIGN;
  const int64_t tiles_a = (N + 127) / 128;
  const bool narrow = M <= 64 * E;
  const int64_t tiles = ((M + (narrow ? 63 : 191)) / (narrow ? 64 : 192) + (E < M ? E : M)) * tiles_a;
  if (tiles > kMaxExtent) return HQ_ERR_SHAPE;
  if (K == 0) return out_zero(out, M * N, dt, stream);
  if (!xq || !xs || !wq || !ws || (!MX && (!x_sg || !w_sg))) return HQ_ERR_NULL;
  if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(ws, 32) || (!MX && (!aligned(x_sg, 4) || !aligned(w_sg, 4))))
    return HQ_ERR_ALIGN;
  GemmParams p = rows_params<MX>(xs, x_sg, ws, w_sg, M, N, K, E, out, dt);
  p.offsets = offsets;
  const Codes a = {wq, K / 2, N, E}, b = {xq, K / 2, M, 1};
  return narrow ? launch<hq::kGemmRows, MX, 64>(p, a, b, tiles, stream)
                : launch<hq::kGemmRows, MX, 192>(p, a, b, tiles, stream);
}

template <bool MX>
hq_status grouped_wgrad(const uint8_t* gq, const uint8_t* gs, const float* g_sg, const uint8_t* xq, const uint8_t* xs,
                        const float* x_sg, const int32_t* offsets, int64_t T, int64_t N, int64_t K, int64_t E,
                        void* out, hq_dtype dt, hq_stream stream) {
  if (dt != HQ_F32 && dt != HQ_BF16) return HQ_ERR_DTYPE;
  if (T < 0 || N < 0 || K < 0 || E < 0 || T % 128 != 0) return HQ_ERR_SHAPE;
  if (T > kMaxExtent || N > kMaxExtent || K > kMaxExtent || E > hq::kGemmMaxGroups) return HQ_ERR_SHAPE;
  if (N == 0 || K == 0 || E == 0) return HQ_OK;
  if (!out || !offsets) return HQ_ERR_NULL;
  if (!aligned(out, dt == HQ_F32 ? 4 : 2) || !aligned(offsets, 4)) return HQ_ERR_ALIGN;
  const int64_t tiles_a = (K + 127) / 128, tiles_b = (N + 191) / 192;
  if (tiles_a * tiles_b > kMaxExtent / E) return HQ_ERR_SHAPE;
  if (T == 0) return out_zero(out, E * N * K, dt, stream);
  if (!gq || !gs || !xq || !xs || (!MX && (!g_sg || !x_sg))) return HQ_ERR_NULL;
  if (!aligned(gq, 16) || !aligned(xq, 16) || !aligned(gs, 32) || !aligned(xs, 32) ||
      (!MX && (!aligned(g_sg, 4) || !aligned(x_sg, 4))))
    return HQ_ERR_ALIGN;
  GemmParams p = {};
  p.k_tiles = static_cast<int>(T / (MX ? 128 : 64));
  p.sfa = xs;
  p.sfb = gs;
  p.sg_a = x_sg;
  p.sg_b = g_sg;
  p.offsets = offsets;
  p.groups = static_cast<int>(E);
  p.extent = static_cast<int>(T);
  p.na = static_cast<int>(K);
  p.nb = static_cast<int>(N);
  p.tiles_a = static_cast<int>(tiles_a);
  p.tiles_b = static_cast<int>(tiles_b);
  p.out = out;
  p.out_f32 = dt == HQ_F32;
  p.out_vec = store_bytes(out, K, dt);
  const Codes a = {xq, T / 2, K, 1}, b = {gq, T / 2, N, 1};
  return launch<hq::kGemmContr, MX, 192>(p, a, b, E * tiles_a * tiles_b, stream);
}

template <int NB, int TG>
cudaError_t launch_shrink(hq::ShrinkParams p, int sms, cudaStream_t stream) {
  const int tiles = (p.rows + 32 * TG - 1) / (32 * TG), chunks = p.K / 32;
  // As many slices of k as keep every warp a chunk, up to a portable cluster; then, where few
  // rows leave multiprocessors idle, several CTAs share a tile's adapters.
  p.slices = 1;
  while (p.slices < 8 && p.slices * 2 * (8 / TG) <= chunks && tiles * p.slices < 2 * sms) p.slices *= 2;
  p.jobs = 1;
  while (p.jobs < 32 && tiles * p.slices * p.jobs < sms) p.jobs *= 2;
  auto kernel = hq::k_lora_shrink<NB, TG>;
  const size_t smem = sizeof(float) * (8 / TG) * (32 * TG) * (16 * NB);
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles) * p.slices * p.jobs);
  cfg.blockDim = dim3(hq::kShrinkThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.slices);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

template <int TG>
cudaError_t launch_shrink(const hq::ShrinkParams& p, int sms, cudaStream_t stream) {
  return p.rank <= 16   ? launch_shrink<1, TG>(p, sms, stream)
         : p.rank <= 32 ? launch_shrink<2, TG>(p, sms, stream)
                        : launch_shrink<4, TG>(p, sms, stream);
}

template <bool MX>
hq_status lora_gemm(const uint8_t* xq, const uint8_t* xs, const float* x_sg, const uint8_t* wq, const uint8_t* ws,
                    const float* w_sg, const void* x, int64_t ldx, const void* a, const void* b, const float* scaling,
                    const int32_t* ids, int64_t M, int64_t N, int64_t K, int64_t n, int64_t R, void* out, hq_dtype dt,
                    void* workspace, hq_stream stream) {
  if (dt != HQ_F32 && dt != HQ_BF16) return HQ_ERR_DTYPE;
  if (M < 0 || N < 0 || K <= 0 || n < 0 || K % 32 != 0 || R < 8 || R > 128 || R % 8 != 0 || ldx < K)
    return HQ_ERR_SHAPE;
  if (M > kMaxExtent || N > kMaxExtent || K > kMaxExtent || n > kMaxExtent || ldx > INT64_MAX / 2 / (M ? M : 1))
    return HQ_ERR_SHAPE;
  if (M == 0 || N == 0) return HQ_OK;
  if (!out || !xq || !xs || !wq || !ws || !x || !ids || !workspace || (n > 0 && (!a || !b || !scaling)) ||
      (!MX && (!x_sg || !w_sg)))
    return HQ_ERR_NULL;
  if (!aligned(out, dt == HQ_F32 ? 4 : 2) || !aligned(xq, 16) || !aligned(wq, 16) || !aligned(ws, 32) ||
      !aligned(x, 16) || (M > 1 && ldx % 8 != 0) || !aligned(a, 16) || !aligned(b, 16) || !aligned(scaling, 4) ||
      !aligned(ids, 4) || !aligned(workspace, 16) || !aligned(x_sg, 4) || !aligned(w_sg, 4))
    return HQ_ERR_ALIGN;
  const bool narrow = M <= 64;
  const int64_t tiles = (M + (narrow ? 63 : 191)) / (narrow ? 64 : 192) * ((N + 127) / 128);
  if (tiles > kMaxExtent) return HQ_ERR_SHAPE;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e);
  hq::ShrinkParams s = {};
  s.x = static_cast<const uint8_t*>(x);
  s.ldx = ldx * 2;
  s.a = static_cast<const uint8_t*>(a);
  s.scaling = scaling;
  s.sg_a = w_sg;
  s.sg_b = x_sg;
  s.ids = ids;
  s.t = static_cast<uint8_t*>(workspace);
  s.rows = static_cast<int>(M);
  s.K = static_cast<int>(K);
  s.adapters = static_cast<int>(n);
  s.rank = static_cast<int>(R);
  if (n > 0) {
    e = M <= 32 ? launch_shrink<1>(s, sms, static_cast<cudaStream_t>(stream))
                : launch_shrink<2>(s, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e);
  }
  GemmParams p = rows_params<MX>(xs, x_sg, ws, w_sg, M, N, K, 1, out, dt);
  p.lora_b = static_cast<const uint8_t*>(b);
  p.lora_t = s.t;
  p.lora_ids = ids;
  p.adapters = s.adapters;
  p.rank = s.rank;
  const Codes ca = {wq, K / 2, N, 1}, cb = {xq, K / 2, M, 1};
  return narrow ? launch<hq::kGemmRows, MX, 64, true>(p, ca, cb, tiles, stream)
                : launch<hq::kGemmRows, MX, 192, true>(p, ca, cb, tiles, stream);
}

// Row-major scale bytes [groups, rows, cols] -> the tile layout, a 16-byte row of a tile per thread.
__global__ void k_swizzle_scales(const uint8_t* __restrict__ s, int64_t rows, int64_t cols, int64_t row_tiles,
                                 int64_t col_tiles, int64_t n, uint4* __restrict__ out) {
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t tile = i / 32, r = i % 32;
    const int64_t ct = tile % col_tiles, rt = tile / col_tiles % row_tiles, g = tile / col_tiles / row_tiles;
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t row = rt * 128 + q * 32 + r;
      w[q] = 0;
      if (row < rows) {
        const uint8_t* src = s + (g * rows + row) * cols + ct * 4;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (ct * 4 + c < cols) w[q] |= static_cast<uint32_t>(src[c]) << (8 * c);
      }
    }
    out[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace

cudaError_t hq::gemm_fault_word(unsigned int* fault, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(fault, g_hq_fault, sizeof(unsigned int));
  if (e == cudaSuccess && clear && *fault) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_hq_fault, &zero, sizeof(unsigned int));
  }
  return e;
}

extern "C" {

hq_status hq_grouped_gemm_nvfp4(const uint8_t* xq, const uint8_t* xs, const float* x_sg, const uint8_t* wq,
                                const uint8_t* ws, const float* w_sg, const int32_t* offsets, int64_t M, int64_t N,
                                int64_t K, int64_t E, void* out, hq_dtype out_dtype, hq_stream stream) {
  return grouped_gemm<false>(xq, xs, x_sg, wq, ws, w_sg, offsets, M, N, K, E, out, out_dtype, stream);
}

hq_status hq_grouped_gemm_mxfp4(const uint8_t* xq, const uint8_t* xs, const uint8_t* wq, const uint8_t* ws,
                                const int32_t* offsets, int64_t M, int64_t N, int64_t K, int64_t E, void* out,
                                hq_dtype out_dtype, hq_stream stream) {
  return grouped_gemm<true>(xq, xs, nullptr, wq, ws, nullptr, offsets, M, N, K, E, out, out_dtype, stream);
}

hq_status hq_grouped_wgrad_nvfp4(const uint8_t* gq, const uint8_t* gs, const float* g_sg, const uint8_t* xq,
                                 const uint8_t* xs, const float* x_sg, const int32_t* offsets, int64_t T, int64_t N,
                                 int64_t K, int64_t E, void* out, hq_dtype out_dtype, hq_stream stream) {
  return grouped_wgrad<false>(gq, gs, g_sg, xq, xs, x_sg, offsets, T, N, K, E, out, out_dtype, stream);
}

hq_status hq_grouped_wgrad_mxfp4(const uint8_t* gq, const uint8_t* gs, const uint8_t* xq, const uint8_t* xs,
                                 const int32_t* offsets, int64_t T, int64_t N, int64_t K, int64_t E, void* out,
                                 hq_dtype out_dtype, hq_stream stream) {
  return grouped_wgrad<true>(gq, gs, nullptr, xq, xs, nullptr, offsets, T, N, K, E, out, out_dtype, stream);
}

int64_t hq_lora_gemm_workspace_bytes(int64_t M, int64_t R) {
  if (M < 0 || M > kMaxExtent || R < 8 || R > 128 || R % 8 != 0) return -1;
  return 4 * M * R;
}

hq_status hq_lora_gemm_nvfp4(const uint8_t* xq, const uint8_t* xs, const float* x_sg, const uint8_t* wq,
                             const uint8_t* ws, const float* w_sg, const void* x, int64_t ldx, const void* lora_a,
                             const void* lora_b, const float* scaling, const int32_t* row_adapter, int64_t M,
                             int64_t N, int64_t K, int64_t adapters, int64_t R, void* out, hq_dtype out_dtype,
                             void* workspace, hq_stream stream) {
  return lora_gemm<false>(xq, xs, x_sg, wq, ws, w_sg, x, ldx, lora_a, lora_b, scaling, row_adapter, M, N, K, adapters,
                          R, out, out_dtype, workspace, stream);
}

hq_status hq_lora_gemm_mxfp4(const uint8_t* xq, const uint8_t* xs, const uint8_t* wq, const uint8_t* ws, const void* x,
                             int64_t ldx, const void* lora_a, const void* lora_b, const float* scaling,
                             const int32_t* row_adapter, int64_t M, int64_t N, int64_t K, int64_t adapters, int64_t R,
                             void* out, hq_dtype out_dtype, void* workspace, hq_stream stream) {
  return lora_gemm<true>(xq, xs, nullptr, wq, ws, nullptr, x, ldx, lora_a, lora_b, scaling, row_adapter, M, N, K,
                         adapters, R, out, out_dtype, workspace, stream);
}

hq_status hq_swizzle_scales(const uint8_t* scales, int64_t groups, int64_t rows, int64_t cols, uint8_t* out,
                            hq_stream stream) {
  if (groups < 0 || rows < 0 || cols < 0 || rows > INT64_MAX - 127 || cols > INT64_MAX / 16) return HQ_ERR_SHAPE;
  const int64_t bytes = hq_swizzled_scales_bytes(rows, cols * 16);
  if (bytes < 0 || (groups > 0 && bytes > INT64_MAX / groups)) return HQ_ERR_SHAPE;
  if (bytes == 0 || groups == 0) return HQ_OK;
  if (!scales || !out) return HQ_ERR_NULL;
  if (!aligned(out, 32)) return HQ_ERR_ALIGN;
  const int64_t n = groups * bytes / 16;
  const int64_t want = (n + 255) / 256;
  k_swizzle_scales<<<static_cast<unsigned>(want < 4096 ? want : 4096), 256, 0, static_cast<cudaStream_t>(stream)>>>(
      scales, rows, cols, (rows + 127) / 128, (cols + 3) / 4, n, reinterpret_cast<uint4*>(out));
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? HQ_OK : cuda_fail(e);
}

}  // extern "C"
