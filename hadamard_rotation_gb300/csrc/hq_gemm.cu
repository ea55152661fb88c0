// hq_gemm.cu -- C ABI of the FP4 products (include/hq.h) and their launch logic.  The kernel is
// in hq_gemm.cuh.
#include <cuda_runtime.h>

#include <cstdint>

#include "hq.h"
#include "hq_gemm.cuh"
#include "hq_internal.h"
#include "hq_tensor_map.h"

namespace {

using hq::cuda_fail;
using hq::encode_out;
using hq::encode_tiled;
using hq::EncodeTiledFn;
using hq::store_bytes;
using hq::GemmKind;
using hq::GemmParams;

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

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

// Scale tiles [row_tiles][k_tiles] of 512 bytes, as words: boxes of `box` tiles along k, `box_rows` of rows.
bool encode_scales(CUtensorMap* map, const uint8_t* s, int64_t k_tiles, int64_t row_tiles, int box, int box_rows) {
  const EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t size[3] = {128, static_cast<cuuint64_t>(k_tiles), static_cast<cuuint64_t>(row_tiles)};
  const cuuint64_t stride[2] = {512, static_cast<cuuint64_t>(k_tiles * 512)};
  const cuuint32_t dim[3] = {128, static_cast<cuuint32_t>(box), static_cast<cuuint32_t>(box_rows)}, step[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t*>(s), size, stride, dim, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One operand's codes as the launch needs them.
struct Codes {
  const uint8_t* q;
  int64_t row_bytes, rows, groups;
};

template <int KIND, bool MX, int T, bool LORA, bool SPLIT = false>
hq_status launch(GemmParams p, const Codes& a, const Codes& b, int64_t b_scale_row_tiles, int64_t most_tiles,
                 int splits, hq_stream stream) {
  using S = hq::GemmShape<KIND, MX, T, LORA>;
  auto kernel = hq::k_fp4_gemm<KIND, MX, T, LORA, SPLIT>;
  int sms = 0;
  cudaError_t e = hq::sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e);
  // (Before the tensor maps: encoding one fails in a thread that has made no CUDA call yet, and this makes the
  // context current there.)
  const size_t smem = hq::gemm_smem_bytes(S::kSmemBytes, p.groups);
  if ((e = hq::allow_smem(reinterpret_cast<const void*>(kernel), static_cast<int>(smem))) != cudaSuccess)
    return cuda_fail(e);
  CUtensorMap ma, mb, msa, msb = {}, mo = {};
  if (!encode_codes(&ma, a.q, a.row_bytes, a.rows, a.groups, hq::kGemmLanes, 3) ||
      !encode_codes(&mb, b.q, b.row_bytes, b.rows, 1, S::kBox, 2) ||
      !encode_scales(&msa, p.sfa, p.k_tiles, a.groups * p.a_row_tiles, S::kTilesPerBlock, 1) ||
      (S::kWide && !encode_scales(&msb, p.sfb, p.k_tiles, b_scale_row_tiles, S::kTilesPerBlock, S::kRowTilesB)))
    return cuda_fail(cudaErrorInvalidValue);
  p.out_tma = !p.out_f32 && p.out_vec == 16 &&
              encode_out(&mo, p.out, p.na, KIND == hq::kGemmRows ? p.extent : p.nb, KIND == hq::kGemmRows ? 1 : p.groups);
  cudaLaunchConfig_t cfg = {};
  const int ctas = S::kCtas * splits;
  const int64_t most = SPLIT ? most_tiles : sms / ctas;
  cfg.gridDim = dim3(static_cast<unsigned>((most_tiles < most ? most_tiles : most) * ctas));
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kernel, ma, mb, msa, msb, mo, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? HQ_OK : cuda_fail(e);
}

// The scales of ragged rows in the tile layout, each group's rows from a multiple of 64 on (units of 64
// rows: a tile of the wide kernel starts at one).  A CTA per 128 rows; padding rows are not written
// (the products of their columns are not stored).
__global__ void __launch_bounds__(256) k_group_scales(const uint8_t* __restrict__ s, const int32_t* offsets, int groups,
                                                      int rows, int row_bytes, int col_tiles, uint4* __restrict__ out) {
  __shared__ int first[2], count[2];  // of the CTA's two units: the first row of x, how many
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x < 2) count[threadIdx.x] = 0;
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int base = 0;
    for (int g0 = 0; g0 < groups && base < 2 * static_cast<int>(blockIdx.x) + 2; g0 += 32) {
      const int g = g0 + lane;
      int a = 0, b = 0;
      if (g < groups) {
        a = offsets ? offsets[g] : 0;
        b = offsets ? offsets[g + 1] : rows;
        a = max(0, min(a, rows));
        b = max(a, min(b, rows));
      }
      const int u = (b - a + 63) / 64, sum = hq::warp_scan(u, lane);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int at = 2 * static_cast<int>(blockIdx.x) + q - (base + sum - u);  // the unit within this group
        if (at >= 0 && at < u) {
          first[q] = a + 64 * at;
          count[q] = min(64, b - a - 64 * at);
        }
      }
      base += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
  }
  __syncthreads();
  if (count[0] + count[1] == 0) return;
  const int r = threadIdx.x & 31;
  for (int ct = threadIdx.x >> 5; ct < col_tiles; ct += 8) {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      w[q] = 0;
      const int at = (q & 1) * 32 + r;
      if (at >= count[q >> 1]) continue;
      const uint8_t* src = s + static_cast<int64_t>(first[q >> 1] + at) * row_bytes + 4 * ct;
      if (row_bytes % 4 == 0 && reinterpret_cast<uintptr_t>(s) % 4 == 0) {
        w[q] = __ldg(reinterpret_cast<const uint32_t*>(src));
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (4 * ct + c < row_bytes) w[q] |= static_cast<uint32_t>(__ldg(src + c)) << (8 * c);
      }
    }
    out[(static_cast<int64_t>(blockIdx.x) * col_tiles + ct) * 32 + r] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

constexpr int64_t kMaxExtent = (int64_t{1} << 31) - 1024;  // sizes and row indexes are ints in the kernel

hq_status out_zero(void* out, int64_t n, hq_dtype dt, hq_stream stream) {
  const cudaError_t e = cudaMemsetAsync(out, 0, static_cast<size_t>(n) * (dt == HQ_F32 ? 4 : 2),
                                        static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HQ_OK : cuda_fail(e);
}

// Tiles of narrow groups, at most: group sizes add up to M.
int64_t narrow_tiles(int64_t M, int64_t E, int64_t tiles_a) { return (M + 63 * (E < M ? E : M)) / 64 * tiles_a; }

// Tiles of 128 x 64 by single CTAs or of 256 x 192 by pairs.  The wide ones read each operand a half to
// a third as often, but need the tokens' scales laid out first (3 us) and fill 76 places, not 152.  Narrow
// where a group has a few rows, or where all its tiles take the 152 SMs some 36 stages each (4 for a tile's
// start and end).  Measured, us narrow / wide: 8 experts 2048 x 2048, 32 rows each 6.2 / 9.9, 192 rows
// 12.8 / 13.5, 512 rows 26.4 / 18.5; 12 of 1100 x 1056, 256 rows 12.4 / 15.1, 512 rows 18.6 / 18.6; 64 of
// 2048 x 4096, 32 rows 46 / 48, 64 rows 67 / 55; 32 of 512 x 512, 256 rows 8.8 / 9.6, 512 rows 13.4 / 11.8.
bool narrow_rows(int64_t M, int64_t N, int64_t K, int64_t E) {
  return M <= 32 * E ||
         narrow_tiles(M, E, (N + 127) / 128) <= 36 * 152 / ((K + hq::kGemmKBlock - 1) / hq::kGemmKBlock + 4);
}

// Tiles of the kernel that is taken, at most.
int64_t rows_tiles(int64_t M, int64_t N, int64_t K, int64_t E) {
  return narrow_rows(M, N, K, E) ? narrow_tiles(M, E, (N + 127) / 128) : (M + 191 * (E < M ? E : M)) / 192 * ((N + 255) / 256);
}

// The narrow kernel, its summed axis shared by a cluster where there are few tiles: as many CTAs as
// SMs, each with two pairs of stages at least (a shorter part is mostly start and end).
template <bool MX, bool LORA>
hq_status launch_narrow(const GemmParams& p, const Codes& a, const Codes& b, int64_t most_tiles, hq_stream stream) {
  int sms = 0;
  const cudaError_t e = hq::sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e);
  int splits = 1;
  while (splits < hq::kMaxSplits && most_tiles * splits * 2 <= sms && p.k >= splits * 2 * 4 * hq::kGemmKBlock) splits *= 2;
  return splits > 1 ? launch<hq::kGemmRows, MX, 64, LORA, true>(p, a, b, 0, most_tiles, splits, stream)
                    : launch<hq::kGemmRows, MX, 64, LORA>(p, a, b, 0, most_tiles, 1, stream);
}

// 128-row tiles of k_group_scales' output, and its bytes.
int64_t group_scale_tiles(int64_t M, int64_t groups) {
  return ((M + 63) / 64 + (groups < M ? groups : M) + 1) / 2;
}
int64_t group_scale_bytes(int64_t M, int64_t K, int64_t groups, bool mx) {
  return group_scale_tiles(M, groups) * ((K + (mx ? 127 : 63)) / (mx ? 128 : 64)) * 512;
}

// Lay the scales of ragged rows out for the wide kernel and point `p` at them.
hq_status tile_scales(GemmParams& p, uint8_t* work, hq_stream stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(group_scale_tiles(p.extent, p.groups)));
  cfg.blockDim = dim3(256);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, k_group_scales, p.sfb, p.offsets, p.groups, p.extent, p.sfb_row_bytes,
                                     p.k_tiles, reinterpret_cast<uint4*>(work));
  if (e == cudaSuccess) e = cudaGetLastError();
  p.sfb = work;
  return e == cudaSuccess ? HQ_OK : cuda_fail(e);
}

// What grouped_gemm and lora_gemm share: the operands of a product with ragged rows.
template <bool MX>
GemmParams rows_params(const uint8_t* xs, const float* x_sg, const uint8_t* ws, const float* w_sg, int64_t M, int64_t N,
                       int64_t K, int64_t groups, void* out, hq_dtype dt) {
  GemmParams p = {};
  p.k_tiles = static_cast<int>((K + (MX ? 127 : 63)) / (MX ? 128 : 64));
  p.a_row_tiles = static_cast<int>((N + 127) / 128);
  p.tiles_a = static_cast<int>(narrow_rows(M, N, K, groups) ? (N + 127) / 128 : (N + 255) / 256);
  p.sfa = ws;
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

// The sizes that the calls and their workspace functions refuse.
bool grouped_sizes(int64_t M, int64_t N, int64_t K, int64_t E) {
  if (M < 0 || N < 0 || K < 0 || E < 0 || K % 32 != 0) return false;
  if (M > kMaxExtent || N > kMaxExtent || K > kMaxExtent || E > hq::kGemmMaxGroups) return false;
  return M == 0 || N == 0 || E == 0 || rows_tiles(M, N, K, E) <= kMaxExtent;
}

bool lora_sizes(int64_t M, int64_t N, int64_t K, int64_t R) {
  if (M < 0 || N < 0 || K <= 0 || K % 32 != 0 || R < 8 || R > 128 || R % 8 != 0) return false;
  if (M > kMaxExtent || N > kMaxExtent || K > kMaxExtent) return false;
  return M == 0 || N == 0 || rows_tiles(M, N, K, 1) <= kMaxExtent;
}

template <bool MX>
hq_status grouped_gemm(const uint8_t* xq, const uint8_t* xs, const float* x_sg, const uint8_t* wq, const uint8_t* ws,
                       const float* w_sg, const int32_t* offsets, int64_t M, int64_t N, int64_t K, int64_t E, void* out,
                       hq_dtype dt, void* workspace, hq_stream stream) {
  if (dt != HQ_F32 && dt != HQ_BF16) return HQ_ERR_DTYPE;
  if (!grouped_sizes(M, N, K, E)) return HQ_ERR_SHAPE;
  if (M == 0 || N == 0 || E == 0) return HQ_OK;
  if (!out || !offsets) return HQ_ERR_NULL;
  if (!aligned(out, dt == HQ_F32 ? 4 : 2) || !aligned(offsets, 4)) return HQ_ERR_ALIGN;
  const bool narrow = narrow_rows(M, N, K, E);
  const int64_t tiles = rows_tiles(M, N, K, E);
  if (K == 0) return out_zero(out, M * N, dt, stream);
  if (!xq || !xs || !wq || !ws || (!MX && (!x_sg || !w_sg))) return HQ_ERR_NULL;
  if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(ws, 32) || (!MX && (!aligned(x_sg, 4) || !aligned(w_sg, 4))))
    return HQ_ERR_ALIGN;
  GemmParams p = rows_params<MX>(xs, x_sg, ws, w_sg, M, N, K, E, out, dt);
  p.offsets = offsets;
  const Codes a = {wq, K / 2, N, E}, b = {xq, K / 2, M, 1};
  if (!narrow) {
    if (!workspace) return HQ_ERR_NULL;
    if (!aligned(workspace, 32)) return HQ_ERR_ALIGN;
    const hq_status st = tile_scales(p, static_cast<uint8_t*>(workspace), stream);
    if (st != HQ_OK) return st;
  }
  return narrow ? launch_narrow<MX, false>(p, a, b, tiles, stream)
                : launch<hq::kGemmRows, MX, 192, false>(p, a, b, group_scale_tiles(M, E), tiles, 1, stream);
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
  const int64_t tiles_a = (K + 255) / 256, tiles_b = (N + 191) / 192;
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
  p.a_row_tiles = static_cast<int>((K + 127) / 128);
  p.tiles_a = static_cast<int>(tiles_a);
  p.tiles_b = static_cast<int>(tiles_b);
  p.out = out;
  p.out_f32 = dt == HQ_F32;
  p.out_vec = store_bytes(out, K, dt);
  const Codes a = {xq, T / 2, K, 1}, b = {gq, T / 2, N, 1};
  return launch<hq::kGemmContr, MX, 192, false>(p, a, b, (N + 127) / 128, E * tiles_a * tiles_b, 1, stream);
}

// bf16 [groups, rows, cols], rows `stride` bytes apart, in boxes of box_rows rows x 64 elements, 128-byte
// swizzle; past a group's rows or a row's end: 0.
bool encode_bf16(CUtensorMap* map, const void* x, int64_t cols, int64_t stride_bytes, int64_t rows, int64_t groups,
                 int box_rows, int dims) {
  const EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t size[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(groups)};
  const cuuint64_t stride[2] = {static_cast<cuuint64_t>(stride_bytes), static_cast<cuuint64_t>(stride_bytes * rows)};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1}, step[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(dims), const_cast<void*>(x), size, stride,
            box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

hq_status launch_shrink(hq::ShrinkParams p, const void* x, int64_t ldx, const void* a, hq_stream stream) {
  int sms = 0;
  cudaError_t e = hq::sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e);
  // As many slices of k as there are places for (two CTAs per SM), up to a portable cluster; then, where
  // few rows leave SMs idle, several CTAs share a tile's adapters.
  const int tiles = (p.rows + hq::kShrinkRows - 1) / hq::kShrinkRows, blocks = (p.K + 63) / 64;
  p.slices = 1;
  while (p.slices < 8 && p.slices * 2 <= blocks && tiles * p.slices * 2 <= 2 * sms) p.slices *= 2;
  const int most = p.rows < hq::kShrinkRows ? p.rows : hq::kShrinkRows;
  const int most_adapters = p.adapters < most ? p.adapters : most;
  p.jobs = 1;
  while (p.jobs < 32 && tiles * p.slices * p.jobs * 2 <= 2 * sms) p.jobs *= 2;
  if (p.jobs > most_adapters) p.jobs = most_adapters;
  // Stages no larger than the rows there are and the adapters a CTA can meet: beside a small CTA the
  // products' CTA fits on the SM and starts under it.
  const int padded = (p.rank + 15) / 16 * 16, adapters = (most_adapters + p.jobs - 1) / p.jobs;
  p.box_rows = (most + 7) / 8 * 8;
  p.cols = adapters * padded < hq::kShrinkCols ? adapters * padded : hq::kShrinkCols / padded * padded;
  const int columns = p.cols + (adapters * padded > p.cols ? padded : 0);
  p.tmem_cols = 32;
  while (p.tmem_cols < columns) p.tmem_cols *= 2;
  const int stage = (p.box_rows + p.cols) * 128;
  p.stages = stage <= 8 * 1024 ? hq::kShrinkMaxStages : 3;
  // (the instruction reads 128 rows of x from a stage's start; the sums lie over the ring)
  int bytes = p.stages * stage;
  if (bytes < (p.stages - 1) * stage + hq::kShrinkRows * 128) bytes = (p.stages - 1) * stage + hq::kShrinkRows * 128;
  if (bytes < hq::kShrinkRows * (padded + hq::kShrinkPad) * 4) bytes = hq::kShrinkRows * (padded + hq::kShrinkPad) * 4;
  bytes += 1024;
  // (before the tensor maps, as in `launch`)
  if ((e = hq::allow_smem(reinterpret_cast<const void*>(hq::k_lora_shrink), bytes)) != cudaSuccess) return cuda_fail(e);
  CUtensorMap mx, ma;
  if (!encode_bf16(&mx, x, p.K, ldx * 2, p.rows, 1, p.box_rows, 2) ||
      !encode_bf16(&ma, a, p.K, int64_t{2} * p.K, p.rank, p.adapters, padded, 3))
    return cuda_fail(cudaErrorInvalidValue);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles) * p.slices * p.jobs);
  cfg.blockDim = dim3(hq::kShrinkThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(bytes);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.slices);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.slices > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, hq::k_lora_shrink, mx, ma, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? HQ_OK : cuda_fail(e);
}

int64_t lora_t_bytes(int64_t M, int64_t R) { return (4 * M * R + 31) / 32 * 32; }

template <bool MX>
hq_status lora_gemm(const uint8_t* xq, const uint8_t* xs, const float* x_sg, const uint8_t* wq, const uint8_t* ws,
                    const float* w_sg, const void* x, int64_t ldx, const void* a, const void* b, const float* scaling,
                    const int32_t* ids, int64_t M, int64_t N, int64_t K, int64_t n, int64_t R, void* out, hq_dtype dt,
                    void* workspace, hq_stream stream) {
  if (dt != HQ_F32 && dt != HQ_BF16) return HQ_ERR_DTYPE;
  if (!lora_sizes(M, N, K, R) || n < 0 || n > kMaxExtent || ldx < K || ldx > INT64_MAX / 2 / (M ? M : 1))
    return HQ_ERR_SHAPE;
  if (M == 0 || N == 0) return HQ_OK;
  if (!out || !xq || !xs || !wq || !ws || !x || !ids || !workspace || (n > 0 && (!a || !b || !scaling)) ||
      (!MX && (!x_sg || !w_sg)))
    return HQ_ERR_NULL;
  if (!aligned(out, dt == HQ_F32 ? 4 : 2) || !aligned(xq, 16) || !aligned(wq, 16) || !aligned(ws, 32) ||
      !aligned(x, 16) || (M > 1 && ldx % 8 != 0) || !aligned(a, 16) || !aligned(b, 16) || !aligned(scaling, 4) ||
      !aligned(ids, 4) || !aligned(workspace, 32) || !aligned(x_sg, 4) || !aligned(w_sg, 4))
    return HQ_ERR_ALIGN;
  const bool narrow = narrow_rows(M, N, K, 1);
  const int64_t tiles = rows_tiles(M, N, K, 1);
  hq::ShrinkParams s = {};
  s.scaling = scaling;
  s.sg_a = w_sg;
  s.sg_b = x_sg;
  s.ids = ids;
  s.t = static_cast<__nv_bfloat16*>(workspace);
  s.rows = static_cast<int>(M);
  s.K = static_cast<int>(K);
  s.adapters = static_cast<int>(n);
  s.rank = static_cast<int>(R);
  GemmParams p = rows_params<MX>(xs, x_sg, ws, w_sg, M, N, K, 1, out, dt);
  uint8_t* const tiles_at = static_cast<uint8_t*>(workspace) + lora_t_bytes(M, R);
  if (n > 0) {
    if (!narrow) {
      s.scales = xs;
      s.tiles = reinterpret_cast<uint4*>(tiles_at);
      s.scale_row_bytes = p.sfb_row_bytes;
      s.scale_tiles = p.k_tiles;
      p.sfb = tiles_at;
    }
    const hq_status st = launch_shrink(s, x, M > 1 ? ldx : K, a, stream);
    if (st != HQ_OK) return st;
  }
  p.lora_b = static_cast<const uint8_t*>(b);
  p.lora_t = static_cast<const uint8_t*>(workspace);
  p.lora_ids = ids;
  p.adapters = s.adapters;
  p.rank = s.rank;
  p.after_shrink = n > 0;
  if (!narrow && n == 0) {
    const hq_status st = tile_scales(p, tiles_at, stream);
    if (st != HQ_OK) return st;
  }
  const Codes ca = {wq, K / 2, N, 1}, cb = {xq, K / 2, M, 1};
  return narrow ? launch_narrow<MX, true>(p, ca, cb, tiles, stream)
                : launch<hq::kGemmRows, MX, 192, true>(p, ca, cb, group_scale_tiles(M, 1), tiles, 1, stream);
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
                                int64_t K, int64_t E, void* out, hq_dtype out_dtype, void* workspace, hq_stream stream) {
  return grouped_gemm<false>(xq, xs, x_sg, wq, ws, w_sg, offsets, M, N, K, E, out, out_dtype, workspace, stream);
}

hq_status hq_grouped_gemm_mxfp4(const uint8_t* xq, const uint8_t* xs, const uint8_t* wq, const uint8_t* ws,
                                const int32_t* offsets, int64_t M, int64_t N, int64_t K, int64_t E, void* out,
                                hq_dtype out_dtype, void* workspace, hq_stream stream) {
  return grouped_gemm<true>(xq, xs, nullptr, wq, ws, nullptr, offsets, M, N, K, E, out, out_dtype, workspace, stream);
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

int64_t hq_grouped_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t E) {
  if (!grouped_sizes(M, N, K, E)) return -1;
  return M == 0 || E == 0 || narrow_rows(M, N, K, E) ? 0 : group_scale_bytes(M, K, E, false);
}

int64_t hq_lora_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t R) {
  if (!lora_sizes(M, N, K, R)) return -1;
  return lora_t_bytes(M, R) + (narrow_rows(M, N, K, 1) ? 0 : group_scale_bytes(M, K, 1, false));
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
