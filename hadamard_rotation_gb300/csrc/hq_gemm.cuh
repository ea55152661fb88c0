// hq_gemm.cuh -- device code of the FP4 products (sm_103a): matrix products that read the
// codes and block scales this library writes, on the 5th-generation tensor cores.
//
//   rows of a group (ROWS):         D_g[m, n] = a_g sum_k X[m, k] W_g[n, k],  off[g] <= m < off[g+1]
//   contraction of a group (CONTR): D_g[n, k] = a   sum_t G[n, t] X[k, t],    off[g] <= t < off[g+1]
//
// X, W, G are E2M1 codes with one scale per 16 (NVFP4, E4M3) or 32 values (MXFP4, E8M0) along
// the summed axis; a is the product of the operands' per-tensor scales (1 for MXFP4).
//
// The tensor core multiplies code x scale exactly and sums in fp32 (tcgen05.mma, kinds
// mxf4nvf4 and mxf4, one K = 64 step per instruction); the only rounding to fewer bits is the
// output's, after the multiplication by a in fp32.
//
// Which operand is which.  The M = 128 side of the instruction (the 128 lanes of tensor
// memory) takes the operand whose extent is long and regular: the weights' output channels
// (ROWS) or X's channels (CONTR).  The ragged side -- the tokens of an expert -- is the N side,
// whose width is chosen per tile in steps of 16 columns: an expert with 5 rows costs one
// 16-column instruction per step, not a 128-row tile.
//
// One CTA per SM takes tiles (128 lanes x up to T columns) from a static cyclic order; the
// group sizes are read on the device, so the call does not wait for the host to know them.
// Roles of a CTA:
//   warp 0        TMA: codes of both operands (128-byte swizzled boxes of 256 codes per row) and
//                 the scales that are stored in the tile layout (512 bytes = 128 rows x 4 scales,
//                 already the order that tensor memory wants)
//   warp 1        copies the scales to tensor memory (tcgen05.cp) and issues the products
//   warp 2        allocates tensor memory
//   warps 4..7    epilogue: tensor memory -> registers -> * a -> global
//   warps 8..11   (ROWS) the tokens' scales: row-major in global memory, since a group starts at
//                 any row; moved through registers into the tile layout
// Shared memory holds a ring of kStages stages (256 steps of the summed axis each); tensor
// memory holds two accumulators, so the epilogue of a tile runs under the products of the next.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "hq_kernels.cuh"

namespace hq {

constexpr int kGemmLanes = 128;      // rows of operand A per tile (lanes of tensor memory)
constexpr int kGemmKBlock = 256;     // summed elements per stage: 128 bytes of codes per row
constexpr int kGemmMaxGroups = 1024;

enum GemmKind { kGemmRows = 0, kGemmContr = 1 };

struct GemmParams {
  const uint8_t* sfa;       // scales of A in the tile layout
  int64_t sfa_group_bytes;  // bytes of one group's scales of A (ROWS)
  const uint8_t* sfb;       // scales of B: row-major (ROWS), tile layout (CONTR)
  const float* sg_a;        // per-tensor scales (ROWS: one per group; CONTR: one); NULL: 1
  const float* sg_b;
  const int32_t* offsets;   // groups + 1; NULL: one group of all `extent` rows
  int groups;
  int extent;               // bound of the offsets: rows of X (ROWS), summed elements (CONTR)
  int na;                   // rows of A (per group for ROWS)
  int nb;                   // CONTR: rows of B
  int k;                    // ROWS: summed elements
  int tiles_a;              // ceil(na / 128)
  int tiles_b;              // CONTR: ceil(nb / T)
  int k_tiles;              // 512-byte scale tiles per 128 rows
  int sfb_row_bytes;        // ROWS: bytes of one row of scales
  int sfb_vec;              // ROWS: bytes per load of them (rows aligned to it)
  void* out;                // ROWS: [extent, na]; CONTR: [groups, nb, na]
  int out_f32;
};

// ---------------------------------------------------------------------------
// Geometry of one kernel instance.  T: columns of a tile (tokens, or rows of G).
// ---------------------------------------------------------------------------
template <bool MX, int T>
struct GemmShape {
  static constexpr int kTilesPerBlock = MX ? 2 : 4;  // scale tiles along K per stage
  static constexpr int kRowTilesB = (T + 127) / 128;
  static constexpr int kBox = T >= 128 ? 64 : 16;    // rows of B per TMA box
  static constexpr int kBytesA = kGemmLanes * 128;
  static constexpr int kBytesB = T * 128;
  static constexpr int kBytesSfa = kTilesPerBlock * 512;
  static constexpr int kBytesSfb = kRowTilesB * kTilesPerBlock * 512;
  static constexpr int kStageBytes = kBytesA + kBytesB + kBytesSfa + kBytesSfb;
  static_assert(kStageBytes % 1024 == 0, "stages stay aligned to the swizzle atom");
  static constexpr int kStages = (200 * 1024) / kStageBytes < 8 ? (200 * 1024) / kStageBytes : 8;
  // tensor memory columns: two accumulators, then two sets of scales (stage parity)
  static constexpr int kColsSfa = kTilesPerBlock * 4;
  static constexpr int kColsSfb = kTilesPerBlock * kRowTilesB * 4;
  static constexpr int kColSf = 2 * T;
  static constexpr int kColsUsed = 2 * T + 2 * (kColsSfa + kColsSfb);
  static constexpr int kCols = kColsUsed <= 256 ? 256 : 512;
  static_assert(kColsUsed <= 512, "tensor memory has 512 columns");
};

struct GemmBars {
  uint64_t full[8], empty[8];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem;
  int failed;
  int tiles;
};

inline size_t gemm_smem_bytes(int stage_bytes, int stages, int groups) {
  return 1024 + static_cast<size_t>(stage_bytes) * stages + 12 * static_cast<size_t>(groups + 1);
}

// ---------------------------------------------------------------------------
// PTX.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tma_tile3(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_tile2(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// A bulk copy whose bytes have been announced on `bar` already.
__device__ __forceinline__ void tma_bulk(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Arrive on `bar` once every tensor-core operation this thread has issued is complete.
__device__ __forceinline__ void umma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}

// One 512-byte scale tile -> 4 columns of tensor memory, repeated for the 4 groups of 32 lanes.
__device__ __forceinline__ void umma_copy_scales(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

template <bool MX>
__device__ __forceinline__ void umma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
  if constexpr (MX) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  }
}

// Shared-memory matrix descriptors.  Codes: rows of 128 bytes, 128-byte swizzle, 8-row groups
// 1024 bytes apart.  Scale tiles: unswizzled, 8-row groups of 16-byte rows 128 bytes apart.
__device__ __forceinline__ uint64_t desc_codes(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (uint64_t{1} << 16) | (uint64_t{1024 >> 4} << 32) |
         (uint64_t{1} << 46) | (uint64_t{2} << 61);
}
__device__ __forceinline__ uint64_t desc_scales(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (uint64_t{1} << 16) | (uint64_t{128 >> 4} << 32) |
         (uint64_t{1} << 46);
}

// Instruction descriptor: E2M1 x E2M1, both operands along K, M = 128, N columns; which pair of
// a 4-byte scale word MXFP4 takes (0 or 2; NVFP4 takes all four).
template <bool MX>
__device__ __forceinline__ uint32_t umma_idesc(int n, int pair) {
  return (static_cast<uint32_t>(pair) << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         ((MX ? 1u : 0u) << 23) | (1u << 27) | (static_cast<uint32_t>(pair) << 29);
}

// Order tensor-memory operations across a barrier between threads.
__device__ __forceinline__ void umma_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void umma_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}

// ---------------------------------------------------------------------------
// Tiles.
// ---------------------------------------------------------------------------
struct GemmTile {
  int g;       // group
  int a0;      // first row of A
  int b0;      // first row of B (ROWS: a row of X)
  int valid;   // columns that exist
  int n;       // columns of the instruction (valid rounded up to 16)
  int k0, k;   // summed range
};

template <int KIND, int T>
__device__ __forceinline__ GemmTile gemm_tile(const GemmParams& p, const int* start, const int* lo, const int* hi,
                                              int tile) {
  int l = 0, r = p.groups;  // the last group that starts at or before `tile`
  while (r - l > 1) {
    const int m = (l + r) >> 1;
    if (start[m] <= tile) l = m;
    else r = m;
  }
  GemmTile t;
  t.g = l;
  const int local = tile - start[l];
  const int span = hi[l] - lo[l];
  if constexpr (KIND == kGemmRows) {
    // equal widths rather than one narrow last tile
    const int parts = (span + T - 1) / T;
    const int width = ((span + parts - 1) / parts + 15) & ~15;
    const int bt = local % parts;
    t.a0 = (local / parts) * kGemmLanes;
    t.b0 = lo[l] + bt * width;
    t.valid = min(width, hi[l] - t.b0);
    t.k0 = 0;
    t.k = p.k;
  } else {
    const int bt = local % p.tiles_b;
    t.a0 = (local / p.tiles_b) * kGemmLanes;
    t.b0 = bt * T;
    t.valid = min(T, p.nb - t.b0);
    t.k0 = lo[l];
    t.k = span;
  }
  t.n = (t.valid + 15) & ~15;
  return t;
}

// The ring position of a role: stage s, and the parity of its current pass.
struct GemmRing {
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) {
      s = 0;
      phase ^= 1;
    }
  }
};

// ---------------------------------------------------------------------------
// The scales of a row of X for one stage: `bytes` of them from `src`, zero past the row's end.
// ---------------------------------------------------------------------------
template <int BYTES>
__device__ __forceinline__ void load_scale_row(const uint8_t* src, int left, int vec, uint32_t (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = 0;
  if (vec == 16) {  // rows of whole stages' scales (NVFP4: K a multiple of 256)
    if (left >= 16) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(src));
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
  } else if (vec == 8) {
#pragma unroll
    for (int i = 0; i < BYTES / 8; ++i)
      if (left >= 8 * i + 8) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(src) + i);
        w[2 * i] = v.x, w[2 * i + 1] = v.y;
      }
  } else if (vec == 4) {
#pragma unroll
    for (int i = 0; i < BYTES / 4; ++i)
      if (left >= 4 * i + 4) w[i] = __ldg(reinterpret_cast<const uint32_t*>(src) + i);
  } else if (vec == 2) {
#pragma unroll
    for (int i = 0; i < BYTES / 2; ++i)
      if (left >= 2 * i + 2)
        w[i / 2] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(src) + i)) << (16 * (i % 2));
  } else {
#pragma unroll
    for (int i = 0; i < BYTES; ++i)
      if (left > i) w[i / 4] |= static_cast<uint32_t>(__ldg(src + i)) << (8 * (i % 4));
  }
}

// ---------------------------------------------------------------------------
// The kernel.
// ---------------------------------------------------------------------------
constexpr int kGemmThreads = 384;
constexpr int kScaleThreads = 128;

template <int KIND, bool MX, int T>
__global__ void __launch_bounds__(kGemmThreads, 1)
    k_fp4_gemm(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
               const __grid_constant__ GemmParams p) {
  using S = GemmShape<MX, T>;
  constexpr int kTpb = S::kTilesPerBlock;
  constexpr int kScaleK = MX ? 128 : 64;  // summed elements of one scale tile
  extern __shared__ uint8_t gemm_smem_raw[];
  __shared__ GemmBars bars;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(gemm_smem_raw) + 1023) & ~uintptr_t{1023});
  int* start = reinterpret_cast<int*>(smem + S::kStages * S::kStageBytes);
  int* lo = start + p.groups + 1;
  int* hi = lo + p.groups + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&bars.tmem)),
                 "r"(S::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 1 && lane == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(smem_addr(&bars.full[i]), KIND == kGemmRows ? 1 + kScaleThreads / 32 : 1);
      mbar_init(smem_addr(&bars.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&bars.acc_full[i]), 1);
      mbar_init(smem_addr(&bars.acc_empty[i]), 4);
    }
    mbar_init(smem_addr(&bars.drain), 1);
    bars.failed = 0;
    fence_mbar_init();
  }
  // The kernel before this one on the stream wrote the operands.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == 0) {  // where each group's tiles begin
    int base = 0;
    for (int g0 = 0; g0 < p.groups; g0 += 32) {
      const int g = g0 + lane;
      int a = 0, b = 0, n = 0;
      if (g < p.groups) {
        a = p.offsets ? p.offsets[g] : 0;
        b = p.offsets ? p.offsets[g + 1] : p.extent;
        a = max(0, min(a, p.extent));
        b = max(a, min(b, p.extent));
        if constexpr (KIND == kGemmContr) {  // whole scale tiles
          a &= ~127;
          b &= ~127;
          n = p.tiles_a * p.tiles_b;
        } else {
          n = p.tiles_a * ((b - a + T - 1) / T);
        }
      }
      int incl = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += o;
      }
      if (g < p.groups) {
        start[g] = base + incl - n;
        lo[g] = a;
        hi[g] = b;
      }
      base += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    if (lane == 0) bars.tiles = base;
  }
  umma_fence_before();
  __syncthreads();
  umma_fence_after();
  const uint32_t tmem = bars.tmem;
  const int tiles = bars.tiles;
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {
      GemmRing ring;
      long long fills = 0;
      for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
        const GemmTile t = gemm_tile<KIND, T>(p, start, lo, hi, tile);
        const int blocks = (t.k + kGemmKBlock - 1) / kGemmKBlock;
        const int boxes = (t.n + S::kBox - 1) / S::kBox;
        const int kt0 = t.k0 / kScaleK;
        const uint8_t* sfa = p.sfa + (KIND == kGemmRows ? t.g * p.sfa_group_bytes : 0) +
                             (static_cast<int64_t>(t.a0 / 128) * p.k_tiles + kt0) * 512;
        int row_tiles = 0;
        const uint8_t* sfb = nullptr;
        if constexpr (KIND == kGemmContr) {
          const int first = t.b0 / 128;
          row_tiles = min((t.b0 + t.valid + 127) / 128 - first, S::kRowTilesB);
          sfb = p.sfb + (static_cast<int64_t>(first) * p.k_tiles + kt0) * 512;
        }
        for (int kb = 0; kb < blocks; ++kb) {
          const uint32_t bar = smem_addr(&bars.full[ring.s]);
          if (!mbar_wait(smem_addr(&bars.empty[ring.s]), ring.phase ^ 1)) {
            ok = false;
            break;
          }
          const uint32_t st = smem_addr(smem + ring.s * S::kStageBytes);
          const uint32_t sa = st + S::kBytesA + S::kBytesB;
          const int sf_tiles = min(kTpb, p.k_tiles - kt0 - kb * kTpb);
          mbar_expect_tx(bar, S::kBytesA + boxes * S::kBox * 128 + sf_tiles * 512 * (1 + row_tiles));
          const int kx = (t.k0 + kb * kGemmKBlock) / 2;
          tma_tile3(st, &map_a, kx, t.a0, KIND == kGemmRows ? t.g : 0, bar);
          for (int i = 0; i < boxes; ++i)
            tma_tile2(st + S::kBytesA + i * S::kBox * 128, &map_b, kx, t.b0 + i * S::kBox, bar);
          tma_bulk(sa, sfa + static_cast<int64_t>(kb) * kTpb * 512, sf_tiles * 512, bar);
          for (int i = 0; i < row_tiles; ++i)
            tma_bulk(sa + S::kBytesSfa + i * kTpb * 512,
                     sfb + (static_cast<int64_t>(i) * p.k_tiles + kb * kTpb) * 512, sf_tiles * 512, bar);
          ++fills;
          ring.next(S::kStages);
        }
      }
      if (!ok) {  // let the copies in flight land (bounded) before the CTA may end
        for (long long f = fills > S::kStages ? fills - S::kStages : 0; f < fills; ++f)
          mbar_wait(smem_addr(&bars.full[f % S::kStages]), (f / S::kStages) & 1);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      GemmRing ring;
      int acc = 0;
      uint32_t acc_phase = 0;
      uint32_t parity = 0;
      for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
        const GemmTile t = gemm_tile<KIND, T>(p, start, lo, hi, tile);
        const int blocks = (t.k + kGemmKBlock - 1) / kGemmKBlock;
        if (!mbar_wait(smem_addr(&bars.acc_empty[acc]), acc_phase ^ 1)) {
          ok = false;
          break;
        }
        umma_fence_after();
        const uint32_t d = tmem + acc * T;
        const uint32_t shift = KIND == kGemmContr ? (t.b0 % 128) / 32 : 0;
        for (int kb = 0; kb < blocks; ++kb) {
          if (!mbar_wait(smem_addr(&bars.full[ring.s]), ring.phase)) {
            ok = false;
            break;
          }
          umma_fence_after();
          const uint32_t st = smem_addr(smem + ring.s * S::kStageBytes);
          const uint32_t sa = st + S::kBytesA + S::kBytesB, sb = sa + S::kBytesSfa;
          const uint32_t ca = tmem + S::kColSf + parity * (S::kColsSfa + S::kColsSfb), cb = ca + S::kColsSfa;
          const int steps = min(4, (t.k - kb * kGemmKBlock + 63) / 64);
          const int sf_tiles = (steps * 64 + kScaleK - 1) / kScaleK;
          const int row_tiles = (shift * 32 + t.n + 127) / 128;
          for (int j = 0; j < sf_tiles; ++j) {
            umma_copy_scales(ca + 4 * j, desc_scales(sa + 512 * j));
            for (int i = 0; i < row_tiles; ++i)
              umma_copy_scales(cb + (j * S::kRowTilesB + i) * 4, desc_scales(sb + (i * kTpb + j) * 512));
          }
          for (int j = 0; j < steps; ++j) {
            const int sj = MX ? j / 2 : j;
            umma_fp4<MX>(d, desc_codes(st + 32 * j), desc_codes(st + S::kBytesA + 32 * j),
                         umma_idesc<MX>(t.n, MX ? 2 * (j & 1) : 0), ca + 4 * sj,
                         cb + sj * S::kRowTilesB * 4 + shift, (kb | j) != 0);
          }
          umma_commit(smem_addr(&bars.empty[ring.s]));
          parity ^= 1;
          ring.next(S::kStages);
        }
        if (!ok) break;
        umma_commit(smem_addr(&bars.acc_full[acc]));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
      if (!ok) {  // let the products in flight finish (bounded) before tensor memory is freed
        umma_commit(smem_addr(&bars.drain));
        mbar_wait(smem_addr(&bars.drain), 0);
      }
    }
  } else if (warp >= 4 && warp < 8) {
    const int quarter = warp & 3;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
      const GemmTile t = gemm_tile<KIND, T>(p, start, lo, hi, tile);
      float a = 1.0f;
      if (!MX) a = __fmul_rn(__ldg(p.sg_a + (KIND == kGemmRows ? t.g : 0)), __ldg(p.sg_b));
      ok = mbar_wait(smem_addr(&bars.acc_full[acc]), acc_phase);
      if (!__all_sync(0xFFFFFFFFu, ok)) {
        ok = false;
        break;
      }
      umma_fence_after();
      const int n = t.a0 + quarter * 32 + lane;
      const int64_t row0 = KIND == kGemmRows ? t.b0 : static_cast<int64_t>(t.g) * p.nb + t.b0;
      const int64_t at = row0 * p.na + n;
      const bool live = n < p.na;
      const bool none = t.k == 0;  // an empty sum: no product wrote the accumulator
      for (int c0 = 0; c0 < t.valid; c0 += 16) {
        uint32_t v[16];
        tmem_ld16(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + acc * T + c0, v);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
        if (live) {
          if (p.out_f32) {
            float* o = static_cast<float*>(p.out) + at + static_cast<int64_t>(c0) * p.na;
#pragma unroll
            for (int c = 0; c < 16; ++c)
              if (c0 + c < t.valid)
                o[static_cast<int64_t>(c) * p.na] = none ? 0.0f : __fmul_rn(__uint_as_float(v[c]), a);
          } else {
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + at + static_cast<int64_t>(c0) * p.na;
#pragma unroll
            for (int c = 0; c < 16; ++c)
              if (c0 + c < t.valid)
                o[static_cast<int64_t>(c) * p.na] =
                    __float2bfloat16_rn(none ? 0.0f : __fmul_rn(__uint_as_float(v[c]), a));
          }
        }
      }
      umma_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&bars.acc_empty[acc]));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
  } else if (KIND == kGemmRows && warp >= 8) {
    constexpr int kRowsPerThread = (T + kScaleThreads - 1) / kScaleThreads;
    constexpr int kAhead = 4;  // stages whose scales are loaded together
    constexpr int kBlockBytes = MX ? 8 : 16;
    const int tid = threadIdx.x - 256;
    GemmRing ring;
    for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
      const GemmTile t = gemm_tile<KIND, T>(p, start, lo, hi, tile);
      const int blocks = (t.k + kGemmKBlock - 1) / kGemmKBlock;
      for (int kb0 = 0; kb0 < blocks && ok; kb0 += kAhead) {
        uint32_t w[kRowsPerThread][kAhead][4];
#pragma unroll
        for (int i = 0; i < kRowsPerThread; ++i) {
          const int r = tid + kScaleThreads * i;
          const uint8_t* src = p.sfb + static_cast<int64_t>(t.b0 + r) * p.sfb_row_bytes;
#pragma unroll
          for (int j = 0; j < kAhead; ++j) {
            const int at = (kb0 + j) * kBlockBytes;
            load_scale_row<kBlockBytes>(src + at, r < t.valid ? p.sfb_row_bytes - at : 0, p.sfb_vec, w[i][j]);
          }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (kb0 + j >= blocks || !ok) break;
          ok = mbar_wait(smem_addr(&bars.empty[ring.s]), ring.phase ^ 1);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          uint8_t* sb = smem + ring.s * S::kStageBytes + S::kBytesA + S::kBytesB + S::kBytesSfa;
#pragma unroll
          for (int i = 0; i < kRowsPerThread; ++i) {
            const int r = tid + kScaleThreads * i;
            if (r < t.n) {
              uint8_t* dst = sb + (r / 128) * kTpb * 512 + (r % 32) * 16 + ((r % 128) / 32) * 4;
#pragma unroll
              for (int q = 0; q < kTpb; ++q) *reinterpret_cast<uint32_t*>(dst + 512 * q) = w[i][j][q];
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&bars.full[ring.s]));
          ring.next(S::kStages);
        }
      }
    }
  }
  if (!ok) {
    bars.failed = 1;
    if (lane == 0) atomicOr(&g_hq_fault, kFaultWaitTimeout);
  }
  __syncwarp();
  umma_fence_before();
  __syncthreads();
  umma_fence_after();
  if (warp == 2)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kCols) : "memory");
}

}  // namespace hq
