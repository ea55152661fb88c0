// hq_gemm8.cu -- C ABI of the product of INT8 codes (include/hq.h) and its launch logic.  The kernel is in
// hq_gemm8.cuh.
#include <cuda_runtime.h>

#include <cstdint>

#include "hq.h"
#include "hq_gemm8.cuh"
#include "hq_internal.h"
#include "hq_tensor_map.h"

namespace {

using hq::cuda_fail;

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxExtent = (int64_t{1} << 31) - 1024;  // sizes and row indexes are ints in the kernel
constexpr int64_t kMaxK = int64_t{1} << 17;

// Codes [rows, K] in boxes of box_rows rows x `block` codes (64, 128), swizzle of as many bytes; past the last row or a row's end: 0.
bool encode_rows(CUtensorMap* map, const int8_t* q, int64_t K, int64_t rows, int box_rows, int block) {
  const hq::EncodeTiledFn fn = hq::encode_tiled();
  if (!fn) return false;
  const cuuint64_t size[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t stride[1] = {static_cast<cuuint64_t>(K)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(block), static_cast<cuuint32_t>(box_rows)}, step[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(q), size, stride, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, block == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a product is cut: wide tiles by pairs of CTAs or narrow ones, a narrow tile's channels, and how many CTAs share
// its sum.
struct Plan {
  bool wide;
  int splits;
  int tiles_a, tiles_b, lanes, width;
};

// The cheapest by this estimate, in cycles: 128 codes take a pair 1300 (two stages through its warps); a single CTA 330
// (likewise) or 5.5 per channel (an SM's share of the memory's rate, where all of them load).  A wide tile ends with an
// epilogue of 3500 that nothing hides, a split one with the cluster's sum.  Sums are split only where all clusters run at
// once: each one after the first would start anew.
// Measured, us, M x N x K:                  narrow   wide      wide tiles of fewer tokens take hardly less (512 x
//   64 x 4096 x 4096                          12.3   23.7      4096 x 4096 in 32 tiles of 256 tokens 26.9, in 64 of
//   777 x 1100 x 1056                          7.1   11.7      128 25.1): a stage's time is the channels' way through
//   8192 x 8192 x 8192                        1221    634      the widening warps
//   48 x 28672 x 8192    narrow tiles of 128 channels (224 on 152 SMs) 60, of 96 (299) 50
//   64 x 4096 x 4096     sums split 12.3, whole 15.1;   1 x 4096 x 4096 8.7 and 14.3
//   2000 x 600 x 8192    sums split in two rounds of clusters 54, whole 49
Plan plan_of(int64_t M, int64_t N, int64_t K, int sms, const int (&clusters)[9]) {
  const int64_t stages = (K + 127) / 128;
  Plan best = {};
  int64_t least = INT64_MAX;
  for (int wide = 0; wide < 2; ++wide) {
    const int64_t T = wide ? 256 : 64, unit = wide ? 32 : 16;
    const int64_t parts = (M + T - 1) / T, width = ((M + parts - 1) / parts + unit - 1) / unit * unit;
    for (int64_t lanes = 128; lanes >= (wide ? 128 : 64); lanes -= 16) {
      const int64_t tiles_a = (N + lanes * (1 + wide) - 1) / (lanes * (1 + wide)), tiles = tiles_a * parts;
      for (int64_t s = 1; s <= (wide ? 1 : hq::kGemm8MaxSplits); s *= 2) {
        if (s > 1 && (stages < 2 * s || tiles > clusters[s])) break;
        const int64_t places = wide ? sms / 2 : s > 1 ? clusters[s] : sms, waves = (tiles + places - 1) / places;
        const int64_t stage = wide ? 1300 : lanes * 11 / 2 > 330 ? lanes * 11 / 2 : 330;
        const int64_t cost = waves * ((stages + s - 1) / s * stage + (wide ? 3500 : s > 1 ? 2500 : 1200));
        if (cost < least) {
          least = cost;
          best = {wide != 0, static_cast<int>(s), static_cast<int>(tiles_a), static_cast<int>(parts), static_cast<int>(lanes),
                  static_cast<int>(width)};
        }
      }
    }
  }
  return best;
}

// How many clusters of 2, 4 and 8 CTAs that share a sum run at a time.
cudaError_t clusters_of(int sms, int (&n)[9]) {
  auto kernel = hq::k_gemm8<false, true>;
  const size_t smem = hq::Gemm8Shape<false>::kSmemBytes + 1024;
  cudaError_t e = hq::allow_smem(reinterpret_cast<const void*>(kernel), static_cast<int>(smem));
  for (int s = 2; s <= hq::kGemm8MaxSplits && e == cudaSuccess; s *= 2) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(sms / s * s));
    cfg.blockDim = dim3(hq::Gemm8Shape<false>::kThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(s);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = hq::clusters_at_a_time(reinterpret_cast<const void*>(kernel), cfg, s, &n[s]);
  }
  return e;
}

template <bool WIDE, bool SPLIT>
hq_status launch(hq::Gemm8Params p, const Plan& plan, const int8_t* x, const int8_t* w, int sms, cudaStream_t stream) {
  using S = hq::Gemm8Shape<WIDE>;
  auto kernel = hq::k_gemm8<WIDE, SPLIT>;
  const size_t smem = S::kSmemBytes + 1024;
  // (Before the tensor maps: encoding one fails in a thread that has made no CUDA call yet, and this makes the context
  // current there.)
  cudaError_t e = hq::allow_smem(reinterpret_cast<const void*>(kernel), static_cast<int>(smem));
  if (e != cudaSuccess) return cuda_fail(e);
  p.box_b = plan.width / S::kCtas;
  CUtensorMap mw, mx, mo = {};
  if (!encode_rows(&mw, w, p.K, p.N, p.lanes, S::kBlock) || !encode_rows(&mx, x, p.K, p.M, p.box_b, S::kBlock)) return cuda_fail(cudaErrorInvalidValue);
  p.out_tma = !p.out_f32 && p.out_vec == 16 && p.lanes == 128 && hq::encode_out(&mo, p.out, p.N, p.M, 1);
  cudaLaunchConfig_t cfg = {};
  const int64_t ctas = S::kCtas * plan.splits, tiles = static_cast<int64_t>(p.tiles_a) * p.tiles_b, places = sms / ctas;
  cfg.gridDim = dim3(static_cast<unsigned>((SPLIT || tiles < places ? tiles : places) * ctas));
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kernel, mw, mx, mo, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? HQ_OK : cuda_fail(e);
}

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
  if ((M + 63) / 64 * ((N + 127) / 128) > kMaxExtent) return HQ_ERR_SHAPE;  // tiles
  if (M == 0 || N == 0) return HQ_OK;
  if (!out || !x_scales || !w_scales || (K > 0 && (!xq || !wq))) return HQ_ERR_NULL;
  if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4) ||
      !aligned(out, out_dtype == HQ_F32 ? 4 : 2))
    return HQ_ERR_ALIGN;
  const int es = out_dtype == HQ_F32 ? 4 : 2;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (K == 0) {
    const cudaError_t e = cudaMemsetAsync(out, 0, static_cast<size_t>(M * N) * es, cs);
    return e == cudaSuccess ? HQ_OK : cuda_fail(e);
  }
  int sms = 0;
  cudaError_t e = hq::sm_count(&sms);
  int clusters[9] = {};
  if (e == cudaSuccess) e = clusters_of(sms, clusters);
  if (e != cudaSuccess) return cuda_fail(e);
  const Plan plan = plan_of(M, N, K, sms, clusters);
  hq::Gemm8Params p = {};
  p.xs = x_scales;
  p.ws = w_scales;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.tiles_a = plan.tiles_a;
  p.tiles_b = plan.tiles_b;
  p.lanes = plan.lanes;
  p.width = plan.width;
  p.out = out;
  p.out_f32 = out_dtype == HQ_F32;
  p.out_vec = hq::store_bytes(out, N, out_dtype);
  return plan.wide         ? launch<true, false>(p, plan, xq, wq, sms, cs)
         : plan.splits > 1 ? launch<false, true>(p, plan, xq, wq, sms, cs)
                           : launch<false, false>(p, plan, xq, wq, sms, cs);
}
