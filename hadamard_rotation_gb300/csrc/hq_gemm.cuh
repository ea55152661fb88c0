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
// Small groups are taken by single CTAs in tiles of 128 lanes x up to 64 columns.  Large ones, and the
// CONTR form, by pairs of CTAs (cta_group::2) in tiles of 256 lanes x up to 192 columns: each CTA keeps its
// 128 lanes of A and half of B's rows, so a stage brings 34 KB into a CTA for what 46 KB would be
// needed alone.  An SM's shared memory moves 128 bytes a cycle; the FP4 products of 128 x 192 alone read
// 107 and their loads write 120.
//
// With fewer tiles than SMs (a few rows and one projection) the CTAs of a cluster share a tile's summed
// axis (SPLIT) and add their parts through distributed shared memory, always in the same order.
//
// One CTA per SM takes tiles from a static cyclic order; the
// group sizes are read on the device, so the call does not wait for the host to know them.
// Roles of a CTA:
//   warp 0        TMA: codes of both operands (128-byte swizzled boxes of 256 codes per row) and
//                 the scales that are stored in the tile layout (512 bytes = 128 rows x 4 scales,
//                 already the order that tensor memory wants)
//   warp 1        copies the scales to tensor memory (tcgen05.cp) and issues the products
//   warp 2        allocates tensor memory
//   warps 4..7    epilogue: tensor memory -> registers -> * a -> shared memory -> global (wide: 4..15,
//                 with adapters 4..11)
//   warps 8..11   (ROWS, narrow tiles) the tokens' scales: row-major in global memory, since a group
//                 starts at any row; moved through registers into the tile layout
//   then 4 warps  (adapters) the operands of the adapters' second product, below
// Shared memory holds a ring of kStages stages (256 steps of the summed axis each); tensor
// memory holds two accumulators, so the epilogue of a tile runs under the products of the next.
//
// Adapters (the shared projection of hq_lora_gemm): out += s_a (x A_a^T) B_a^T for the rows of adapter
// a.  The first, thin product is a kernel of its own (k_lora_shrink) that leaves t = s_a x A_a^T / a in
// two bf16 terms per value, t = hi + lo, so nothing is lost to the type (2^-17).  The second product
// is more steps of the same accumulator: 16 bf16 columns ("a slot") hold 16 ranks of one adapter, B_a on the
// lanes' side and t -- zero in the rows of other adapters -- on the columns' side, hi and lo in turn.
// Four slots make a chunk; a tile takes as many as its rows have distinct adapters, so a tile of
// one request pays for one adapter and a tile of 64 requests for those that occur.  Chunks are
// multiplied at fixed places of the main loop: the order of the sum does not depend on timing.
// A zero times an infinity is not zero, so an infinity or NaN in B_a goes into the product as 0, or it would reach the
// rows of other adapters.  What it gives the rows of its own is added to the output at the end (add_special), a walk over
// the rows and lanes that only a call with such a value pays for.
//
// What bounds it, measured.
//   A few rows per expert: the weights' bytes.  64 experts of 4096 x 2048 (MXFP4), 512 rows: 34 to 38 us, 5.4 to 6.1
//   TB/s of what has to move, 0.79 to 0.90 of a copy.  One token at 8 experts of 2048 x 4096: 9.1 to 9.7 us, of which 5.6
//   are bytes and the rest a launch's start and the sum over the cluster.
//   Large groups: 64 experts of 2048 x 4096 (NVFP4), 32768 rows: 134 us, 4.1 PFLOP/s.  Tensor pipe 51% busy, DRAM 50%, L2
//   58% (2.4 GB for 0.48 GB of DRAM traffic): none is full, and which wait it is has not been settled.  (Not the L2 alone:
//   the adapters' form takes a quarter less per second from it and keeps the pipe no busier.  The order in which warp 1
//   issues scale copies and products was not varied.)  A square-ish projection without groups ([4096, 4096] x
//   [8192, 4096]) 56 us, 4.9 PFLOP/s.  Wider tiles would read less, but tensor memory holds two accumulators of 192
//   columns beside the scales, and with one the epilogue (a third of a tile's time) stood alone.
//   Weight gradients: their output.  16 experts of 2048 x 4096 bf16 from 8192 tokens: 61 to 63 us for 0.30 GB, 0.72 of a
//   copy; an expert's sum is 2 stages long, so a tile is mostly its 98 KB of output.
//   Adapters: [4096, 4096] x [8192, 4096] with 8 adapters of rank 64 in runs of 200 rows: 80 to 89 us = 15 us of the thin
//   product (bound by reading x at 3.9 TB/s from its first copy to its last, then by its clusters' barriers) and 65 us;
//   32 rows of 24 adapters of rank 16 beside 4096 x 4096: 17.5 us, two kernels' latencies one after the other.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <limits.h>

#include "hq_kernels.cuh"

namespace hq {

constexpr int kGemmLanes = 128;      // rows of operand A per tile (lanes of tensor memory)
constexpr int kGemmKBlock = 256;     // summed elements per stage: 128 bytes of codes per row
constexpr int kGemmMaxGroups = 512;

enum GemmKind { kGemmRows = 0, kGemmContr = 1 };

struct GemmParams {
  const uint8_t* sfa;       // scales of A in the tile layout
  int a_row_tiles;          // its 128-row tiles per group (ROWS)
  const uint8_t* sfb;       // scales of B: row-major (narrow ROWS), or in the tile layout
  const float* sg_a;        // per-tensor scales (ROWS: one per group; CONTR: one); NULL: 1
  const float* sg_b;
  const int32_t* offsets;   // groups + 1; NULL: one group of all `extent` rows
  int groups;
  int extent;               // bound of the offsets: rows of X (ROWS), summed elements (CONTR)
  int na;                   // rows of A (per group for ROWS)
  int nb;                   // CONTR: rows of B
  int k;                    // ROWS: summed elements
  int tiles_a;              // tiles over na: of 128 lanes, or 256 (pairs)
  int tiles_b;              // CONTR: ceil(nb / T)
  int k_tiles;              // 512-byte scale tiles per 128 rows
  int sfb_row_bytes;        // bytes of one row of row-major scales
  int sfb_mode;             // how they are read (load_scales)
  void* out;                // ROWS: [extent, na]; CONTR: [groups, nb, na]
  int out_f32;
  int out_tma;              // bf16 rows aligned to 16 bytes: map_out is valid
  int out_vec;              // bytes per store: what the rows of out are aligned to, up to 16
  // adapters
  const uint8_t* lora_b;    // bf16 [adapters, na, rank]
  const uint8_t* lora_t;    // bf16 [extent][hi, lo][rank]
  const int32_t* lora_ids;  // [extent]
  int adapters, rank;
  int after_shrink;         // narrow: the kernel before this one is k_lora_shrink, and made only lora_t
};

// ---------------------------------------------------------------------------
// Geometry of one kernel instance.  T: columns of a tile (tokens, or rows of G).
// ---------------------------------------------------------------------------
template <int KIND, bool MX, int T, bool LORA>
struct GemmShape {
  static constexpr bool kWide = KIND == kGemmContr || T >= 128;  // pairs of CTAs; B's scales in the tile layout
  static constexpr int kCtas = kWide ? 2 : 1;
  static constexpr int kTileLanes = kCtas * kGemmLanes;
  static constexpr int kRowsB = T / kCtas;           // rows of B in a CTA's shared memory
  static constexpr int kTilesPerBlock = MX ? 2 : 4;  // scale tiles along K per stage
  static constexpr int kRowTilesB = (T + 127) / 128;
  static constexpr int kBox = kWide ? kRowsB : 16;   // rows of B per TMA box
  static constexpr int kBytesA = kGemmLanes * 128;
  static constexpr int kBytesB = kRowsB * 128;
  static constexpr int kBytesSfa = kTilesPerBlock * 512;
  static constexpr int kBytesSfb = kRowTilesB * kTilesPerBlock * 512;
  static constexpr int kStageBytes = kBytesA + kBytesB + kBytesSfa + kBytesSfb;
  static_assert(kStageBytes % 1024 == 0, "stages stay aligned to the swizzle atom");
  // adapters: chunks of 64 bf16 columns: B_a of 128 lanes, then t's hi and lo of kRowsB rows
  static constexpr int kChunkBytes = LORA ? kGemmLanes * 128 + 2 * kRowsB * 128 : 0;
  static constexpr int kChunks = kWide ? 1 : 2;
  static constexpr int kChunkGap = kWide ? 8 : 2;         // stages between two chunks of a tile
  // The first chunk's place.  Wide: a little later than it could be, so that a tile does not wait for it (1024 rows
  // 30.2 -> 29.4 us).
  static constexpr int kChunkPlace = kWide ? 5 : 1;
  static constexpr int kEpilogues = !kWide ? 1 : LORA ? 2 : 3;  // groups of 128 threads
  // 32-column blocks of the output per chunk.  CONTR: two, three groups then take a tile in one chunk each.
  static constexpr int kBlocks = KIND == kGemmContr ? 2 : 1;
  static constexpr int kOuts = kEpilogues * kBlocks * 8 * 1024;  // the groups' output buffers
  static constexpr int kLoraWarp = 4 + 4 * (kWide ? kEpilogues : 2);  // the adapters' first warp
  static constexpr int kThreads = 32 * (kLoraWarp + (LORA ? 4 : 0));
  static constexpr int kRingBytes = 216 * 1024 - kChunks * kChunkBytes - kOuts;
  static constexpr int kMostStages = LORA && !kWide ? 4 : 7;  // (4: the CTA fits beside one of the thin product)
  static constexpr int kStages = kRingBytes / kStageBytes < kMostStages ? kRingBytes / kStageBytes : kMostStages;
  static constexpr int kSmemBytes = kStages * kStageBytes + kChunks * kChunkBytes + kOuts;
  static_assert(kSmemBytes + 1024 + 16 * (LORA ? 2 : kGemmMaxGroups + 1) + 2048 <= 227 * 1024, "a CTA has 227 KB");
  // (its columns of tensor memory are held while it waits for the CTAs of its cluster)
  static_assert(2 * kSmemBytes > 228 * 1024, "no two CTAs of these kernels share an SM");
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
  uint64_t chunk_full[2], chunk_empty[2];
  int chunk_steps[2], chunk_last[2];  // 16-column steps of a chunk; whether the tile ends with it
  int32_t ids[192], distinct[192];     // a tile's adapters by row, and each once
  int n_distinct;
  int special;  // an infinity or NaN of the adapters' B was left out of a product
  uint32_t tmem;
  int tiles;
};

inline size_t gemm_smem_bytes(int bytes, int groups) { return 1024 + static_cast<size_t>(bytes) + 16 * static_cast<size_t>(groups + 1); }

// ---------------------------------------------------------------------------
// PTX.
// ---------------------------------------------------------------------------
// Tensor copies into this CTA's shared memory.  PAIR: `bar` is a cluster address, of either CTA of the pair.
template <bool PAIR>
__device__ __forceinline__ void tma_tile3(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void tma_tile2(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// The cluster address of a shared variable of CTA `rank`, and an arrival there.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The same without waiting for this thread's stores (2000 cycles with output rows in flight): for an
// arrival that hands over tensor memory, which the tcgen05 fence orders.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A wait of the whole warp: every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity));
}

// Tensor-core operations, of this CTA or (PAIR) of the pair, issued by its first CTA: operands and
// scales lie at the same addresses of both CTAs' shared and tensor memory.

// Arrive on `bar` (PAIR: of both CTAs) once every operation this thread has issued is complete.
template <bool PAIR>
__device__ __forceinline__ void umma_commit(uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// One 512-byte scale tile -> 4 columns of tensor memory, repeated for the 4 groups of 32 lanes.
template <bool PAIR>
__device__ __forceinline__ void umma_copy_scales(uint32_t tmem, uint64_t desc) {
  if constexpr (PAIR)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

template <bool PAIR, bool MX>
__device__ __forceinline__ void umma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
  if constexpr (PAIR && MX)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else if constexpr (MX)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void umma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
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

// Instruction descriptor: E2M1 x E2M1, both operands along K, M lanes, N columns; which pair of
// a 4-byte scale word MXFP4 takes (0 or 2; NVFP4 takes all four).
template <bool MX>
__device__ __forceinline__ uint32_t umma_idesc(int m, int n, int pair) {
  return (static_cast<uint32_t>(pair) << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         ((MX ? 1u : 0u) << 23) | (static_cast<uint32_t>(m >> 4) << 24) | (static_cast<uint32_t>(pair) << 29);
}

// The same for bf16 x bf16 into fp32.
__device__ __forceinline__ uint32_t umma_idesc_bf16(int m, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

// Order tensor-memory operations across a barrier between threads.
__device__ __forceinline__ void umma_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void umma_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Columns of the thread's lane into registers; the wait is part of the statement, so nothing reads
// the registers before it.
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
// Registers into columns of the thread's lane; complete when the statement is.
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// A warp's 32 lanes x 32 columns in the shape of matrix fragments: v[h] is lanes 16 h .. 16 h + 15.
__device__ __forceinline__ void tmem_load_fragments(uint32_t taddr, uint32_t (&v)[2][16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0][0]), "=r"(v[0][1]), "=r"(v[0][2]), "=r"(v[0][3]), "=r"(v[0][4]), "=r"(v[0][5]), "=r"(v[0][6]), "=r"(v[0][7]),
        "=r"(v[0][8]), "=r"(v[0][9]), "=r"(v[0][10]), "=r"(v[0][11]), "=r"(v[0][12]), "=r"(v[0][13]), "=r"(v[0][14]), "=r"(v[0][15]),
        "=r"(v[1][0]), "=r"(v[1][1]), "=r"(v[1][2]), "=r"(v[1][3]), "=r"(v[1][4]), "=r"(v[1][5]), "=r"(v[1][6]), "=r"(v[1][7]),
        "=r"(v[1][8]), "=r"(v[1][9]), "=r"(v[1][10]), "=r"(v[1][11]), "=r"(v[1][12]), "=r"(v[1][13]), "=r"(v[1][14]), "=r"(v[1][15])
      : "r"(taddr), "r"(taddr + (16u << 16))
      : "memory");
}

// ---------------------------------------------------------------------------
// Tiles.
// ---------------------------------------------------------------------------
struct GemmTile {
  int g;       // group
  int a0;      // first row of A (of the pair)
  int b0;      // first row of B (ROWS: a row of X)
  int valid;   // columns that exist
  int n;       // columns of the instruction (valid rounded up to 16, pairs: 32)
  int k0, k;   // summed range
  int s0;      // first row of B's scales in the tile layout, a multiple of 64
};

template <int KIND, int T>
__device__ __forceinline__ GemmTile gemm_tile(const GemmParams& p, const int* start, const int* lo, const int* hi,
                                              const int* units, int tile) {
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
    constexpr int kStep = T >= 128 ? 64 : 16;
    const int width = ((span + parts - 1) / parts + kStep - 1) & ~(kStep - 1);
    const int at = local / parts, bt = local - at * parts;
    t.a0 = at * (T >= 128 ? 2 * kGemmLanes : kGemmLanes);
    t.b0 = lo[l] + bt * width;
    t.valid = min(width, hi[l] - t.b0);
    t.s0 = T >= 128 ? units[l] * 64 + bt * width : 0;
    t.k0 = 0;
    t.k = p.k;
  } else {
    const int at = local / p.tiles_b, bt = local - at * p.tiles_b;
    t.a0 = at * 2 * kGemmLanes;
    t.b0 = t.s0 = bt * T;
    t.valid = min(T, p.nb - t.b0);
    t.k0 = lo[l];
    t.k = span;
  }
  t.n = T >= 128 ? (t.valid + 31) & ~31 : (t.valid + 15) & ~15;
  return t;
}

// Sums of v over the lanes up to this one.
__device__ __forceinline__ int warp_scan(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// The tiles of a CTA in their order, for one warp: 32 are worked out at a time, one per lane (the search and
// the divisions take 500 cycles), and handed out by shuffles.
template <int KIND, int T>
struct GemmTiles {
  const GemmParams& p;
  const int *start, *lo, *hi, *units;
  int tiles, step;
  int next;      // the next tile
  int splits, part;  // the part of the summed axis that is this CTA's
  int count = 0;  // handed out since the last 32 were worked out
  GemmTile mine;

  // The next tile into t; false: there is none.
  __device__ __forceinline__ bool get(GemmTile& t) {
    if (next >= tiles) return false;
    if ((count & 31) == 0) {
      const int tile = next + static_cast<int>(threadIdx.x & 31) * step;
      mine = gemm_tile<KIND, T>(p, start, lo, hi, units, tile < tiles ? tile : next);
      if (splits > 1) {  // parts of whole pairs of stages (16 bytes of the tokens' scales)
        constexpr int kUnit = 2 * kGemmKBlock;
        const int all = (mine.k + kUnit - 1) / kUnit;
        mine.k0 = all * part / splits * kUnit;
        mine.k = min(mine.k, all * (part + 1) / splits * kUnit) - mine.k0;
      }
    }
    const int from = count & 31;
    auto pick = [&](int v) { return __shfl_sync(0xFFFFFFFFu, v, from); };
    t = {pick(mine.g), pick(mine.a0), pick(mine.b0), pick(mine.valid), pick(mine.n), pick(mine.k0), pick(mine.k), pick(mine.s0)};
    ++count;
    next += step;
    return true;
  }
};

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
// The scales of a row of X for a batch of stages, as words in registers: W words, of which the thread
// takes what lies in its row when it writes them.  `mode`: 16, 8: rows aligned to that many bytes;
// 4: rows at any byte of a 4-byte aligned tensor, read as the aligned words around them (one more,
// shifted when they are written); 1: a tensor at any byte.  The loads are volatile so that they stay
// ahead of the batch written before them.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t ld_word(const uint8_t* p) {
  uint32_t v;
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

struct ScaleRow {
  int shift;  // bits to drop from the first word
  int left;   // bytes of the row from the batch's first one on; <= 0: nothing
};

template <int W>
__device__ __forceinline__ ScaleRow load_scales(const GemmParams& p, int64_t row, bool live, int at, uint32_t (&w)[W + 1]) {
  ScaleRow s{0, live ? p.sfb_row_bytes - at : 0};
  if (p.sfb_mode >= 8) {
    const int vec = p.sfb_mode;
    const uint8_t* src = p.sfb + (s.left > 0 ? row * p.sfb_row_bytes + at : 0);
#pragma unroll
    for (int i = 0; i < W; i += 4) {  // past the row's end: its first bytes again, dropped later
      const uint8_t* q = src + (4 * i < s.left ? 4 * i : 0);
      if (vec == 16) {
        asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                     : "l"(q));
      } else {
        const uint8_t* q2 = src + (4 * i + 8 < s.left ? 4 * i + 8 : 0);
        asm volatile("ld.global.nc.v2.b32 {%0, %1}, [%2];" : "=r"(w[i]), "=r"(w[i + 1]) : "l"(q));
        asm volatile("ld.global.nc.v2.b32 {%0, %1}, [%2];" : "=r"(w[i + 2]), "=r"(w[i + 3]) : "l"(q2));
      }
    }
    return s;
  }
  const int64_t first = row * p.sfb_row_bytes + at, end = static_cast<int64_t>(p.extent) * p.sfb_row_bytes;
  if (p.sfb_mode == 4 && (s.left <= 0 || first + s.left <= (end & ~int64_t{3}))) {
    // every word that holds a byte of the row lies inside the tensor; later words: the first again
    const int64_t base = s.left > 0 ? first & ~int64_t{3} : 0;
    s.shift = s.left > 0 ? static_cast<int>(first & 3) * 8 : 0;
    const int words = s.left > 0 ? (s.left + s.shift / 8 + 3) / 4 : (end >= 4 ? 1 : 0);
#pragma unroll
    for (int i = 0; i <= W; ++i) w[i] = words > 0 ? ld_word(p.sfb + base + (i < words ? 4 * i : 0)) : 0;
    return s;
  }
#pragma unroll
  for (int i = 0; i <= W; ++i) {  // the tensor's last bytes, or an unaligned tensor
    w[i] = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b)
      if (4 * i + b < s.left) w[i] |= static_cast<uint32_t>(__ldg(p.sfb + first + 4 * i + b)) << (8 * b);
  }
  return s;
}

// Word i of a loaded row, zero past its end.
template <int W>
__device__ __forceinline__ uint32_t scale_word(const uint32_t (&w)[W + 1], const ScaleRow& s, int i) {
  const uint32_t v = __funnelshift_r(w[i], w[i + 1], s.shift);
  const int left = s.left - 4 * i;
  return left >= 4 ? v : left <= 0 ? 0u : v & ((1u << (8 * left)) - 1);
}

// Barriers among 128 threads of a role (1: adapters, 2 to 4: epilogue); the second tells all of them
// whether `ok` held for all: a wait that ran out for one warp must not leave the others at a barrier.
template <int ID>
__device__ __forceinline__ void role_sync() {
  asm volatile("bar.sync %0, 128;" ::"n"(ID) : "memory");
}
template <int ID>
__device__ __forceinline__ bool role_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(ok)), "n"(ID)
      : "memory");
  return r;
}

// ---------------------------------------------------------------------------
// Epilogue: accumulator columns [0, valid) of 128 lanes, times a, to rows of `out`.
//
// In tensor memory a thread holds one lane, and lanes are consecutive elements of an output row: stored
// as they come, a warp writes 64 bytes of a row at a time (bf16), which took 12,000 cycles for 192
// columns, more than a tile's products.  So a chunk of columns goes through shared memory, as
// rows of the output, and from there
//   bf16   read from tensor memory in the matrix-fragment shape (16x256b), packed in pairs and stored
//          transposed by stmatrix, 4 stores per 32 columns in place of 32; a whole chunk leaves by TMA
//          (two boxes of 64 elements x 32 rows, 128-byte swizzle), a chunk that the group's rows end
//          in, and rows not aligned to 16 bytes, by plain stores;
//   fp32   one store per element and plain stores.
// ---------------------------------------------------------------------------
constexpr int kOutBytes = 8 * 1024;  // a block: 128 lanes x 32 columns of bf16 or 16 of fp32

// Byte `at` of row r of a block.  bf16: two halves of 32 rows x 128 bytes, 16-byte pieces swizzled by the
// row.  fp32: 16 rows x 512 bytes.
template <bool F32>
__device__ __forceinline__ int out_place(int r, int at) {
  if constexpr (F32) return r * 512 + at;
  return (at >> 7) * 4096 + r * 128 + ((((at >> 4) & 7) ^ (r & 7)) << 4) + (at & 15);
}

// The block's first `rows` rows, the first `bytes` of each, to global rows `stride` bytes apart: all
// reads before the writes.
template <typename V, bool F32>
__device__ __forceinline__ void store_rows(const uint8_t* buf, uint8_t* out, int64_t stride, int rows, int bytes,
                                           int tid) {
  constexpr int kPerRow = (F32 ? 512 : 256) / sizeof(V), kRows = F32 ? 16 : 32;
  if constexpr (kPerRow <= 128) {
    constexpr int kStep = 128 / kPerRow, kTimes = kRows / kStep, kBatch = kTimes < 8 ? kTimes : 8;
    const int at = tid % kPerRow * static_cast<int>(sizeof(V)), r0 = tid / kPerRow;
    if (at >= bytes) return;
#pragma unroll 1
    for (int i0 = 0; i0 < kTimes; i0 += kBatch) {
      V v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        v[i] = *reinterpret_cast<const V*>(buf + out_place<F32>(r0 + (i0 + i) * kStep, at));
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = r0 + (i0 + i) * kStep;
        if (r < rows) *reinterpret_cast<V*>(out + r * stride + at) = v[i];
      }
    }
  }
}

template <bool F32>
__device__ __forceinline__ void store_rows(int vec, const uint8_t* buf, uint8_t* out, int64_t stride, int rows,
                                           int bytes, int tid) {
  if (vec == 16) store_rows<uint4, F32>(buf, out, stride, rows, bytes, tid);
  else if (vec == 8) store_rows<uint2, F32>(buf, out, stride, rows, bytes, tid);
  else if (vec == 4) store_rows<uint32_t, F32>(buf, out, stride, rows, bytes, tid);
  else if constexpr (!F32) store_rows<uint16_t, F32>(buf, out, stride, rows, bytes, tid);
}

// A block of the accumulator's columns (32 of bf16, 16 of fp32), times a, into registers as they are
// stored (16 words), and from there into the buffer.  `from`: the address of the warp's 32 lanes and the
// first column.
__device__ __forceinline__ void fetch_f32(uint32_t from, float a, bool none, uint32_t (&w)[16]) {
  tmem_load(from, w);
#pragma unroll
  for (int c = 0; c < 16; ++c) w[c] = none ? 0u : __float_as_uint(__fmul_rn(__uint_as_float(w[c]), a));
}

__device__ __forceinline__ void put_f32(uint8_t* buf, const uint32_t (&w)[16], int tid) {
#pragma unroll
  for (int c = 0; c < 16; ++c) reinterpret_cast<uint32_t*>(buf)[c * 128 + tid] = w[c];
}

__device__ __forceinline__ void fetch_bf16(uint32_t from, float a, bool none, uint32_t (&w)[16]) {
  // v[h][4 i + 0..3]: lanes 16 h + lane / 4 and + 8, columns 8 i + 2 (lane % 4) and + 1
  uint32_t v[2][16];
  tmem_load_fragments(from, v);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const uint32_t* f = &v[m >> 1][4 * i + 2 * (m & 1)];
      const __nv_bfloat162 b = __floats2bfloat162_rn(__fmul_rn(__uint_as_float(f[0]), a), __fmul_rn(__uint_as_float(f[1]), a));
      w[4 * i + m] = none ? 0u : *reinterpret_cast<const uint32_t*>(&b);
    }
}

__device__ __forceinline__ void put_bf16(uint8_t* buf, const uint32_t (&w)[16], int quarter, int lane) {
  // matrix m = lane / 8 of a store is lanes 8 m .. 8 m + 7 of the warp; its row lane % 8 a column
  const uint32_t to = smem_addr(buf) + out_place<false>(lane & 7, quarter * 64 + (lane >> 3) * 16);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared::cta.b16 [%0], {%1, %2, %3, %4};" ::"r"(to + 1024 * i),
                 "r"(w[4 * i]), "r"(w[4 * i + 1]), "r"(w[4 * i + 2]), "r"(w[4 * i + 3])
                 : "memory");
}

__device__ __forceinline__ void tma_store3(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y), "r"(z)
               : "memory");
}

// ---------------------------------------------------------------------------
// The kernel.
// ---------------------------------------------------------------------------
constexpr int kScaleThreads = 128;

constexpr int kLoraThreads = 128;
constexpr int kMaxSplits = 8;

// Four floats of CTA `rank` of the cluster, at the address of shared variables of this one.
__device__ __forceinline__ float4 load_cluster4(const float* p, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(smem_addr(p)), "r"(rank)
      : "memory");
  return v;
}

// A pair of bf16, each half made 0 if it is infinite or NaN.
__device__ __forceinline__ uint32_t without_special(uint32_t w) {
  return w & ~((((w & 0x7F807F80u) + 0x00800080u) >> 15 & 0x00010001u) * 0xFFFFu);
}
// zero * w + sum: NaN once there was an infinity or NaN.
__device__ __forceinline__ __nv_bfloat162 add_zeros(uint32_t w, __nv_bfloat162 sum) {
  return __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w), __floats2bfloat162_rn(0.0f, 0.0f), sum);
}

// What the infinities and NaN of adapter id's B add to output channel n of row m (before the multiplication by a): the
// sum of t B over them, infinite or NaN; 0 where there are none.  Of the ranks whose slots are this CTA's: slot0 is
// the adapter's first.
__device__ __forceinline__ float special_sum(const GemmParams& p, int id, int64_t m, int n, int slot0, int splits,
                                             int part) {
  const __nv_bfloat16* const b =
      reinterpret_cast<const __nv_bfloat16*>(p.lora_b) + (static_cast<int64_t>(id) * p.na + n) * p.rank;
  const __nv_bfloat16* const t = reinterpret_cast<const __nv_bfloat16*>(p.lora_t) + m * 2 * p.rank;
  float sum = 0.0f;
  for (int r = 0; r < p.rank; ++r) {
    const float v = __bfloat162float(b[r]);
    if (isfinite(v) || (slot0 + r / 16) / 4 % splits != part) continue;
    // t = hi + lo has hi's sign, and is zero, infinite or NaN where hi is
    sum += __uint_as_float(static_cast<uint32_t>(__ldcg(reinterpret_cast<const uint16_t*>(t + r))) << 16) * v;
  }
  return sum;
}

// What the chunks of this CTA left out, added to the rows and lanes of its tiles, whose stores (the cluster's) are
// complete.  Infinities and NaN: the order in which CTAs of a cluster add theirs does not matter.
template <bool MX, int T>
__device__ __forceinline__ void add_special(const GemmParams& p, const GemmBars& bars, GemmTiles<kGemmRows, T> order, int rank,
                                            int splits, int part) {
  float a = 1.0f;
  if (!MX) a = __fmul_rn(__ldg(p.sg_a), __ldg(p.sg_b));
  GemmTile t;
  while (order.get(t)) {
    const int n = t.a0 + rank * kGemmLanes + static_cast<int>(threadIdx.x % kGemmLanes);
    if (n < p.na)
      for (int c = threadIdx.x / kGemmLanes; c < t.valid; c += blockDim.x / kGemmLanes) {
        const int64_t m = t.b0 + c;
        const int id = __ldg(p.lora_ids + m);
        if (id < 0 || id >= p.adapters) continue;
        int at = 0;  // (one part: it has every slot)
        if (splits > 1)
          while (at + 1 < bars.n_distinct && bars.distinct[at] != id) ++at;
        const float add = special_sum(p, id, m, n, at * ((p.rank + 15) / 16), splits, part);
        if (add == 0.0f) continue;
        if (p.out_f32) atomicAdd(static_cast<float*>(p.out) + m * p.na + n, add * a);
        else atomicAdd(static_cast<__nv_bfloat16*>(p.out) + m * p.na + n, __float2bfloat16_rn(add * a));
      }
    __syncwarp();
  }
}

template <int KIND, bool MX, int T, bool LORA, bool SPLIT>
__global__ void __launch_bounds__((GemmShape<KIND, MX, T, LORA>::kThreads), 1)
    k_fp4_gemm(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
               const __grid_constant__ CUtensorMap map_sfa, const __grid_constant__ CUtensorMap map_sfb,
               const __grid_constant__ CUtensorMap map_out, const __grid_constant__ GemmParams p) {
  using S = GemmShape<KIND, MX, T, LORA>;
  constexpr int kTpb = S::kTilesPerBlock;
  constexpr int kScaleK = MX ? 128 : 64;  // summed elements of one scale tile
  constexpr int kEpilogues = S::kEpilogues, kBlocks = S::kBlocks, kCtas = S::kCtas;
  constexpr bool kPair = S::kWide;
  extern __shared__ uint8_t gemm_smem_raw[];
  __shared__ GemmBars bars;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(gemm_smem_raw) + 1023) & ~uintptr_t{1023});
  uint8_t* const chunks = smem + S::kStages * S::kStageBytes;
  uint8_t* const outs = chunks + S::kChunks * S::kChunkBytes;
  int* start = reinterpret_cast<int*>(smem + S::kSmemBytes);
  int* lo = start + p.groups + 1;
  int* hi = lo + p.groups + 1;
  int* units = hi + p.groups + 1;  // (tiled scales of ragged rows) 64-row units of scales before a group's
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  static_assert(!(SPLIT && kPair), "pairs do not split the sum");
  const uint32_t rank = kPair ? cluster_rank() : 0;  // of the pair; CTA 0 issues the products
  const int splits = SPLIT ? static_cast<int>(cluster_size()) : 1, part_k = SPLIT ? static_cast<int>(cluster_rank()) : 0;

  if (warp == 2) {
    if constexpr (kPair) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&bars.tmem)),
                   "r"(S::kCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&bars.tmem)),
                   "r"(S::kCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // Only now, and by this warp: the kernel after this one takes tensor memory too before it waits for this
    // one, and must not find it free before this CTA has its own.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
  if (warp == 1 && lane == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(smem_addr(&bars.full[i]), S::kWide ? 1 : 1 + kScaleThreads / 32);
      mbar_init(smem_addr(&bars.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&bars.acc_full[i]), 1);
      mbar_init(smem_addr(&bars.acc_empty[i]), 4 * kEpilogues * kCtas);
      mbar_init(smem_addr(&bars.chunk_full[i]), kLoraThreads / 32 * kCtas);
      mbar_init(smem_addr(&bars.chunk_empty[i]), 1);
    }
    mbar_init(smem_addr(&bars.drain), 1);
    bars.special = 0;
    fence_mbar_init();
  }
  // The kernel before this one on the stream wrote the operands.  (Where it is the adapters' first product,
  // which lets this kernel start once it has itself waited for what was before it: only lora_t, and only the
  // adapters' warps wait for it.)
  if (!(LORA && !kPair && p.after_shrink)) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == 0) {  // where each group's tiles begin
    int base = 0, unit_base = 0;
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
      const int incl = warp_scan(n, lane);
      if (g < p.groups) {
        start[g] = base + incl - n;
        lo[g] = a;
        hi[g] = b;
      }
      base += __shfl_sync(0xFFFFFFFFu, incl, 31);
      if constexpr (KIND == kGemmRows && S::kWide) {
        const int u = (b - a + 63) / 64, sum = warp_scan(u, lane);
        if (g < p.groups) units[g] = unit_base + sum - u;
        unit_base += __shfl_sync(0xFFFFFFFFu, sum, 31);
      }
    }
    if (lane == 0) bars.tiles = base;
  }
  umma_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_sync();  // the peer's barriers are there
  umma_fence_after();
  const uint32_t tmem = bars.tmem;
  // (SPLIT: the launch has a cluster for every tile; each takes one)
  const int places = static_cast<int>(gridDim.x) / (kCtas * splits), place = static_cast<int>(blockIdx.x) / (kCtas * splits);
  const int tiles = SPLIT ? min(bars.tiles, places) : bars.tiles;
  GemmTiles<KIND, T> order{p, start, lo, hi, units, tiles, places, place, splits, part_k};
  bool ok = true;
  // Arrivals on a barrier of the CTA that issues the products.
  auto arrive_first = [&](uint32_t bar) {
    if (rank) mbar_arrive_cluster(cluster_addr(bar, 0));
    else mbar_arrive(bar);
  };
  auto release_acc = [&](uint32_t bar) {
    if (rank) mbar_arrive_cluster_relaxed(cluster_addr(bar, 0));
    else mbar_arrive(bar);
  };

  if (warp == 0) {
    GemmRing ring;
    long long fills = 0;
    GemmTile t;
    while (ok && order.get(t)) {
      const int blocks = (t.k + kGemmKBlock - 1) / kGemmKBlock;
      const int rows_b = t.n / kCtas, boxes = S::kWide ? 1 : (rows_b + S::kBox - 1) / S::kBox;
      const int a0 = t.a0 + static_cast<int>(rank) * kGemmLanes, b0 = t.b0 + static_cast<int>(rank) * rows_b;
      const int kt0 = t.k0 / kScaleK;
      // scale tiles of this CTA's lanes and of all the tile's columns
      const int ta = (KIND == kGemmRows ? t.g * p.a_row_tiles : 0) + a0 / 128, tb = S::kWide ? t.s0 / 128 : 0;
      const uint32_t bytes = kCtas * (S::kBytesA + boxes * S::kBox * 128 + S::kBytesSfa + (S::kWide ? S::kBytesSfb : 0));
      for (int kb = 0; kb < blocks; ++kb) {
        ok = warp_wait(smem_addr(&bars.empty[ring.s]), ring.phase ^ 1);
        if (!ok) break;
        const uint32_t full = smem_addr(&bars.full[ring.s]);
        const uint32_t bar = kPair ? cluster_addr(full, 0) : full;
        const uint32_t st = smem_addr(smem) + ring.s * S::kStageBytes;
        const uint32_t sa = st + S::kBytesA + S::kBytesB;
        const int kx = (t.k0 + kb * kGemmKBlock) / 2;
        const int kt = kt0 + kb * kTpb;
        if (elect_one()) {
          if (rank == 0)
            mbar_expect_tx(full, bytes);
          tma_tile3<kPair>(st, &map_a, kx, a0, KIND == kGemmRows ? t.g : 0, bar);
          tma_tile3<kPair>(sa, &map_sfa, 0, kt, ta, bar);
          for (int i = 0; i < boxes; ++i)
            tma_tile2<kPair>(st + S::kBytesA + i * S::kBox * 128, &map_b, kx, b0 + i * S::kBox, bar);
          if constexpr (S::kWide) tma_tile3<kPair>(sa + S::kBytesSfa, &map_sfb, 0, kt, tb, bar);
        }
        __syncwarp();
        ++fills;
        ring.next(S::kStages);
      }
    }
    if (!ok && rank == 0) {  // let the copies in flight land (bounded) before the CTA (the pair) may end
      for (long long f = fills > S::kStages ? fills - S::kStages : 0; f < fills; ++f)
        mbar_wait(smem_addr(&bars.full[f % S::kStages]), (f / S::kStages) & 1);
    }
  } else if (warp == 1 && rank == 0) {
    GemmRing ring;
    int acc = 0;
    uint32_t acc_phase = 0;
    uint32_t parity = 0;
    GemmRing chunk;
    const uint64_t codes0 = desc_codes(smem_addr(smem));
    const uint64_t scales0 = desc_scales(smem_addr(smem) + S::kBytesA + S::kBytesB);
    const uint64_t chunk0 = desc_codes(smem_addr(chunks));
    GemmTile t;
    while (ok && order.get(t)) {
      const int blocks = (t.k + kGemmKBlock - 1) / kGemmKBlock;
      ok = warp_wait(smem_addr(&bars.acc_empty[acc]), acc_phase ^ 1);
      if (!ok) break;
      umma_fence_after();
      const uint32_t d = tmem + acc * T;
      const uint32_t shift = S::kWide ? (t.s0 % 128) / 32 : 0;
      const int row_tiles = (shift * 32 + t.n + 127) / 128;
      const uint32_t idesc0 = umma_idesc<MX>(S::kTileLanes, t.n, 0);
      const uint32_t idesc1 = umma_idesc<MX>(S::kTileLanes, t.n, MX ? 2 : 0);
      bool chunks_left = LORA;
      auto take_chunk = [&]() {
        ok = warp_wait(smem_addr(&bars.chunk_full[chunk.s]), chunk.phase);
        if (!ok) return;
        umma_fence_after();
        const int steps = bars.chunk_steps[chunk.s];
        chunks_left = !bars.chunk_last[chunk.s];
        const uint64_t ch = chunk0 + chunk.s * (S::kChunkBytes >> 4);
        if (elect_one()) {
          for (int part = 0; part < 2; ++part)  // hi, lo
            for (int j = 0; j < steps; ++j)
              umma_bf16<kPair>(d, ch + 2 * j, ch + ((kGemmLanes * 128 + part * S::kRowsB * 128) >> 4) + 2 * j,
                               umma_idesc_bf16(S::kTileLanes, t.n), 1);
          umma_commit<kPair>(smem_addr(&bars.chunk_empty[chunk.s]));
        }
        __syncwarp();
        chunk.next(S::kChunks);
      };
      for (int kb = 0; kb < blocks; ++kb) {
        if (LORA && chunks_left && kb % S::kChunkGap == S::kChunkPlace) take_chunk();
        if (!ok) break;
        ok = warp_wait(smem_addr(&bars.full[ring.s]), ring.phase);
        if (!ok) break;
        umma_fence_after();
        const uint32_t at = ring.s * (S::kStageBytes >> 4);  // (descriptor addresses are in 16 bytes)
        const uint64_t st = codes0 + at, sa = scales0 + at;
        const uint32_t ca = tmem + S::kColSf + parity * (S::kColsSfa + S::kColsSfb), cb = ca + S::kColsSfa;
        const uint32_t more = kb != 0;
        auto copy_scales = [&](int j) {
          umma_copy_scales<kPair>(ca + 4 * j, sa + 32 * j);
          umma_copy_scales<kPair>(cb + j * S::kRowTilesB * 4, sa + (S::kBytesSfa >> 4) + 32 * j);
        };
        auto copy_scales2 = [&](int j) {  // the second 128 columns
          umma_copy_scales<kPair>(cb + (j * S::kRowTilesB + 1) * 4, sa + (S::kBytesSfa >> 4) + (kTpb + j) * 32);
        };
        auto multiply = [&](int j) {
          const int sj = MX ? j / 2 : j;
          umma_fp4<kPair, MX>(d, st + 2 * j, st + (S::kBytesA >> 4) + 2 * j, (j & 1) ? idesc1 : idesc0, ca + 4 * sj,
                              cb + sj * S::kRowTilesB * 4 + shift, j ? 1u : more);
        };
        const int left = t.k - kb * kGemmKBlock;
        if (elect_one()) {
          if (left >= kGemmKBlock - 63) {  // all four steps
#pragma unroll
            for (int j = 0; j < kTpb; ++j) copy_scales(j);
            if (S::kRowTilesB > 1 && row_tiles > 1) {
#pragma unroll
              for (int j = 0; j < kTpb; ++j) copy_scales2(j);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) multiply(j);
          } else {
            const int steps = (left + 63) / 64;
            for (int j = 0; j * kScaleK < left; ++j) {
              copy_scales(j);
              if (S::kRowTilesB > 1 && row_tiles > 1) copy_scales2(j);
            }
            for (int j = 0; j < steps; ++j) multiply(j);
          }
          umma_commit<kPair>(smem_addr(&bars.empty[ring.s]));
        }
        __syncwarp();
        parity ^= 1;
        ring.next(S::kStages);
      }
      while (LORA && chunks_left && ok) take_chunk();
      if (!ok) break;
      if (elect_one()) umma_commit<kPair>(smem_addr(&bars.acc_full[acc]));
      __syncwarp();
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
    if (!ok) {  // let the products in flight finish (bounded) before tensor memory is freed
      if (elect_one()) umma_commit<kPair>(smem_addr(&bars.drain));
      __syncwarp();
      mbar_wait(smem_addr(&bars.drain), 0);
    }
  } else if (warp >= 4 && warp < 4 + 4 * kEpilogues) {
    // Group `part` of 128 threads takes every kEpilogues-th chunk of kBlocks blocks.  (With short sums the
    // output is most of the work: a chunk takes 1000 cycles, mostly latencies.)
    const int part = (warp - 4) / 4, quarter = warp & 3, tid = threadIdx.x & 127;
    auto sync = [&]() {
      if (part == 0) role_sync<2>();
      else if (part == 1) role_sync<3>();
      else role_sync<4>();
    };
    int acc = 0;
    uint32_t acc_phase = 0;
    const int es = p.out_f32 ? 4 : 2, block = p.out_f32 ? 16 : 32, step = kBlocks * block;
    uint8_t* const buf = outs + part * kBlocks * kOutBytes;
    GemmTile t;
    while (order.get(t)) {
      float a = 1.0f;
      if (!MX) a = __fmul_rn(__ldg(p.sg_a + (KIND == kGemmRows ? t.g : 0)), __ldg(p.sg_b));
      const bool full = mbar_wait(smem_addr(&bars.acc_full[acc]), acc_phase);
      ok = part == 0 ? role_all<2>(full) : part == 1 ? role_all<3>(full) : role_all<4>(full);
      if (!ok) break;
      umma_fence_after();
      const int64_t row0 = KIND == kGemmRows ? t.b0 : static_cast<int64_t>(t.g) * p.nb + t.b0;
      const int64_t stride = static_cast<int64_t>(p.na) * es;
      const int a0 = t.a0 + static_cast<int>(rank) * kGemmLanes;
      uint8_t* const out = static_cast<uint8_t*>(p.out) + row0 * stride + static_cast<int64_t>(a0) * es;
      const int bytes = min(128, p.na - a0) * es;  // (not positive: the pair's second CTA has no lanes here)
      const bool none = t.k == 0;  // an empty sum: no product wrote the accumulator
      const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + acc * T;
      bool held = true;
      if constexpr (SPLIT) {  // the partial sums as they are, over the ring, whose stages have been multiplied
        float* const sums = reinterpret_cast<float*>(smem);
        for (int c0 = 0; c0 < t.valid; c0 += 16) {
          uint32_t v[16];
          tmem_load(from + c0, v);
#pragma unroll
          for (int c = 0; c < 16; ++c) sums[(c0 + c) * kGemmLanes + tid] = __uint_as_float(v[c]);
        }
        umma_fence_before();
      } else
      for (int c0 = part * step; c0 < t.valid; c0 += kEpilogues * step) {
        uint32_t w[kBlocks][16];
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {  // (past t.valid: columns of the accumulator that are not stored)
          if (p.out_f32) fetch_f32(from + c0 + i * block, a, none, w[i]);
          else fetch_bf16(from + c0 + i * block, a, none, w[i]);
        }
        if (c0 + kEpilogues * step >= t.valid) {  // the group's last chunk: its part has been read
          umma_fence_before();
          __syncwarp();
          if (lane == 0) release_acc(smem_addr(&bars.acc_empty[acc]));
          held = false;
        }
        // (The copies of a block's two halves are issued by two warps, by the same elected lane each time.)
        if (quarter < 2 * kBlocks) {
          if (elect_one()) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();
        }
        sync();  // the last chunk has left the buffer
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
          if (p.out_f32) put_f32(buf + i * kOutBytes, w[i], tid);
          else put_bf16(buf + i * kOutBytes, w[i], quarter, lane);
        }
        fence_proxy_async_smem();
        sync();
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
          const int c = c0 + i * block, rows = min(block, t.valid - c);
          if (rows <= 0) break;
          const uint8_t* const b = buf + i * kOutBytes;
          // (CONTR: rows past nb are past the tensor map's end and not written)
          if (p.out_tma && (KIND == kGemmContr || rows == 32)) {
            const int half = quarter - 2 * i, x = a0 + 64 * half;
            if (half >= 0 && half < 2 && x < p.na && elect_one()) {
              tma_store3(&map_out, smem_addr(b) + 4096 * half, x, t.b0 + c, KIND == kGemmRows ? 0 : t.g);
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
          } else if (p.out_f32) {
            store_rows<true>(p.out_vec, b, out + c * stride, stride, rows, bytes, tid);
          } else {
            store_rows<false>(p.out_vec, b, out + c * stride, stride, rows, bytes, tid);
          }
        }
        __syncwarp();
      }
      if (held) {  // no chunk for this group
        __syncwarp();
        if (lane == 0) release_acc(smem_addr(&bars.acc_empty[acc]));
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
    if (elect_one()) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  } else if (!S::kWide && warp >= 8 && warp < 12) {
    constexpr int kRowsPerThread = (T + kScaleThreads - 1) / kScaleThreads;
    constexpr int kAhead = 4;  // stages whose scales are loaded together: a batch
    constexpr int kBlockBytes = MX ? 8 : 16;
    const int tid = threadIdx.x - 256;
    GemmRing ring;
    struct Batch {
      bool live;  // there is one
      int kb, end, b0, valid, n;  // stages [kb, end) of the rows' scales
    };
    auto enter = [&](Batch& b) {  // the next tile's first batch
      GemmTile t;
      b.live = order.get(t);
      if (b.live) {
        b.kb = t.k0 / kGemmKBlock, b.end = b.kb + (t.k + kGemmKBlock - 1) / kGemmKBlock;
        b.b0 = t.b0, b.valid = t.valid, b.n = t.n;
      }
    };
    auto after = [&](const Batch& b) {
      Batch c = b;
      c.kb += kAhead;
      if (c.live && c.kb >= c.end) enter(c);
      return c;
    };
    constexpr int kWords = kAhead * kBlockBytes / 4;
    struct Loaded {
      uint32_t w[kRowsPerThread][kWords + 1];
      ScaleRow row[kRowsPerThread];
    };
    auto load = [&](const Batch& b, Loaded& l) {
      if (!b.live) return;
#pragma unroll
      for (int i = 0; i < kRowsPerThread; ++i) {
        const int r = tid + kScaleThreads * i;
        l.row[i] = load_scales<kWords>(p, b.b0 + r, r < b.valid, b.kb * kBlockBytes, l.w[i]);
      }
    };
    // The next batch is loaded after this one's first stage is written: its words have arrived by then
    // (waiting for them later would wait for the newer loads too), and there is the time of the
    // other stages for the new ones.
    auto write = [&](const Batch& b, const Loaded& l, const Batch& next, Loaded& into) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (b.kb + j >= b.end || !ok) break;
        ok = warp_wait(smem_addr(&bars.empty[ring.s]), ring.phase ^ 1);
        if (!ok) break;
        uint8_t* sb = smem + ring.s * S::kStageBytes + S::kBytesA + S::kBytesB + S::kBytesSfa;
#pragma unroll
        for (int i = 0; i < kRowsPerThread; ++i) {
          const int r = tid + kScaleThreads * i;
          if (r < b.n) {
            uint8_t* dst = sb + (r / 128) * kTpb * 512 + (r % 32) * 16 + ((r % 128) / 32) * 4;
#pragma unroll
            for (int q = 0; q < kTpb; ++q)
              *reinterpret_cast<uint32_t*>(dst + 512 * q) = scale_word<kWords>(l.w[i], l.row[i], j * kTpb + q);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&bars.full[ring.s]));
        ring.next(S::kStages);
        if (j == 0) load(next, into);
      }
    };
    Loaded w0, w1;
    Batch b0, b1;
    enter(b0);
    load(b0, w0);
    while (b0.live && ok) {
      b1 = after(b0);
      write(b0, w0, b1, w1);
      if (!b1.live || !ok) break;
      b0 = after(b1);
      write(b1, w1, b0, w0);
    }
  }
  if constexpr (LORA) {
    if (warp >= S::kLoraWarp) {
      const int tid = threadIdx.x - 32 * S::kLoraWarp;
      const int rank_steps = (p.rank + 15) / 16;
      GemmRing chunk;
      GemmTile t;
      bool waited = false;
      auto wait_for_t = [&]() {
        if (!kPair && !waited && p.after_shrink) asm volatile("griddepcontrol.wait;" ::: "memory");
        waited = true;
      };
      // Eight threads take the eight 16-byte pieces of a row (half a slot each), 16 rows at a time: a request of a
      // warp is then four whole rows where an adapter has 64 ranks.  (A thread per row took 5000 cycles for a
      // chunk's loads, and with two adapters per tile more than the tile's products.)
      const int piece = tid & 7, row_of = tid >> 3;
      constexpr int kRowsAtOnce = kLoraThreads / 8, kTimesB = kGemmLanes / kRowsAtOnce, kTimesT = S::kRowsB / kRowsAtOnce;
      int got[T / 32];
      auto load_ids = [&]() {
#pragma unroll
        for (int c = 0; c < T / 32; ++c)  // (all in flight together)
          got[c] = 32 * c + lane < t.valid ? __ldg(p.lora_ids + t.b0 + 32 * c + lane) : -1;
      };
      bool live = order.get(t);
      if (live && warp == S::kLoraWarp) load_ids();
      while (ok && live) {
        role_sync<1>();  // the last tile's lists have been read
        const GemmTile now = t;
        live = order.get(t);
        if (warp == S::kLoraWarp) {
          int n = 0;
#pragma unroll
          for (int c = 0; c < T / 32; ++c) {
            const int r = 32 * c + lane, id = got[c] >= 0 && got[c] < p.adapters ? got[c] : -1;
            const uint32_t same = __match_any_sync(0xFFFFFFFFu, id);
            bool fresh = id >= 0 && lane == __ffs(same) - 1;
            for (int k = 0; k < n; ++k) fresh = fresh && bars.distinct[k] != id;
            const uint32_t firsts = __ballot_sync(0xFFFFFFFFu, fresh);
            if (fresh) bars.distinct[n + __popc(firsts & ((1u << lane) - 1))] = id;
            bars.ids[r] = id;
            n += __popc(firsts);
            __syncwarp();
          }
          if (lane == 0) bars.n_distinct = n;
          if (live) load_ids();  // the next tile's
        }
        role_sync<1>();
        // Slot q holds ranks 16 (q % rank_steps) .. of the tile's adapter q / rank_steps.  (SPLIT: the parts take
        // the chunks in turn.)
        const int slots = bars.n_distinct * rank_steps;
        const int rows_b = now.n / kCtas, r0 = static_cast<int>(rank) * rows_b;
        const int n0 = now.a0 + static_cast<int>(rank) * kGemmLanes + row_of;  // this thread's first lane
        int first = 4 * part_k;
        bool more = true;
        do {
          more = first + 4 * splits < slots;
          const int steps = max(0, min(4, slots - first)), slot = first + (piece >> 1);
          first += 4 * splits;
          const int r = slot % rank_steps * 16 + (piece & 1) * 8;
          const int a = slot < slots && r < p.rank ? bars.distinct[slot / rank_steps] : -1;
          const uint4 zero = make_uint4(0, 0, 0, 0);
          uint4 b[kTimesB];  // B_a
          const uint8_t* const src_b = p.lora_b + ((static_cast<int64_t>(a) * p.na + n0) * p.rank + r) * 2;
#pragma unroll
          for (int k = 0; k < kTimesB; ++k) {
            b[k] = zero;
            if (a >= 0 && n0 + kRowsAtOnce * k < p.na)
              b[k] = __ldg(reinterpret_cast<const uint4*>(src_b + static_cast<int64_t>(k) * kRowsAtOnce * p.rank * 2));
          }
          wait_for_t();
          uint4 v[kTimesT][2];  // t's hi and lo: zero in the rows of other adapters
          const uint8_t* const src_t = p.lora_t + ((static_cast<int64_t>(now.b0) + r0 + row_of) * 2 * p.rank + r) * 2;
#pragma unroll
          for (int k = 0; k < kTimesT; ++k) {
            const int row = row_of + kRowsAtOnce * k;
            v[k][0] = v[k][1] = zero;
            if (a < 0 || row >= rows_b || bars.ids[r0 + row] != a) continue;
            const uint8_t* src = src_t + static_cast<int64_t>(k) * kRowsAtOnce * p.rank * 4;
            v[k][0] = __ldcg(reinterpret_cast<const uint4*>(src));
            v[k][1] = __ldcg(reinterpret_cast<const uint4*>(src + p.rank * 2));
          }
          // all four warps go on, or none: they meet at barriers
          ok = role_all<1>(mbar_wait(smem_addr(&bars.chunk_empty[chunk.s]), chunk.phase ^ 1));
          if (!ok) break;
          // Infinities and NaN among B's values?  (Looked for here, where all loads are behind.)
          __nv_bfloat162 zeros = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
          for (int k = 0; k < kTimesB; ++k)
            zeros = add_zeros(b[k].x, add_zeros(b[k].y, add_zeros(b[k].z, add_zeros(b[k].w, zeros))));
          if (!__hbeq2(zeros, zeros)) {
            bars.special = 1;
#pragma unroll
            for (int k = 0; k < kTimesB; ++k)
              b[k] = make_uint4(without_special(b[k].x), without_special(b[k].y), without_special(b[k].z), without_special(b[k].w));
          }
          // (rows 16 apart have the same place in the swizzle)
          uint8_t* const dst = chunks + chunk.s * S::kChunkBytes + row_of * 128 + ((piece ^ (row_of & 7)) << 4);
#pragma unroll
          for (int k = 0; k < kTimesB; ++k) *reinterpret_cast<uint4*>(dst + k * kRowsAtOnce * 128) = b[k];
#pragma unroll
          for (int k = 0; k < kTimesT; ++k)
#pragma unroll
            for (int part = 0; part < 2; ++part)
              *reinterpret_cast<uint4*>(dst + (kGemmLanes + part * S::kRowsB + k * kRowsAtOnce) * 128) = v[k][part];
          if (tid == 0) {
            bars.chunk_steps[chunk.s] = steps;
            bars.chunk_last[chunk.s] = !more;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) arrive_first(smem_addr(&bars.chunk_full[chunk.s]));
          chunk.next(S::kChunks);
        } while (more);
      }
      wait_for_t();  // (a CTA without a tile too: this kernel ends after the one before)
    }
  }
  if (!ok) {
    if (lane == 0) atomicOr(&g_hq_fault, kFaultWaitTimeout);
  }
  __syncwarp();
  if constexpr (SPLIT) {  // each CTA of the cluster finishes its share of the columns, adding the parts in order
    cluster_sync();
    GemmTile t;
    GemmTiles<KIND, T> again{p, start, lo, hi, units, tiles, places, place, 1, 0};
    if (again.get(t)) {
      float a = 1.0f;
      if (!MX) a = __fmul_rn(__ldg(p.sg_a + t.g), __ldg(p.sg_b));
      // Four lanes of a column per thread.
      const float* const sums = reinterpret_cast<const float*>(smem) + (threadIdx.x & 31) * 4;
      const int n = t.a0 + static_cast<int>(threadIdx.x & 31) * 4, es = p.out_f32 ? 4 : 2;
      if (n < p.na)
        for (int c = part_k + splits * static_cast<int>(threadIdx.x >> 5); c < t.valid;
             c += splits * static_cast<int>(blockDim.x >> 5)) {
          float4 v[kMaxSplits];
#pragma unroll
          for (int k = 0; k < kMaxSplits; ++k)  // without a condition: all in flight before the first is added
            v[k] = load_cluster4(sums + c * kGemmLanes, min(k, splits - 1));
          float sum[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
          for (int k = 1; k < kMaxSplits; ++k) {
            if (k >= splits) continue;
            sum[0] += v[k].x, sum[1] += v[k].y, sum[2] += v[k].z, sum[3] += v[k].w;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) sum[k] = __fmul_rn(sum[k], a);
          uint8_t* const out = static_cast<uint8_t*>(p.out) + (static_cast<int64_t>(t.b0 + c) * p.na + n) * es;
          const __nv_bfloat162 half[2] = {__floats2bfloat162_rn(sum[0], sum[1]), __floats2bfloat162_rn(sum[2], sum[3])};
          if (p.out_vec >= 4 * es && n + 3 < p.na) {
            if (p.out_f32) *reinterpret_cast<float4*>(out) = make_float4(sum[0], sum[1], sum[2], sum[3]);
            else *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(half);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (n + k >= p.na) continue;
              if (p.out_f32) reinterpret_cast<float*>(out)[k] = sum[k];
              else reinterpret_cast<__nv_bfloat16*>(out)[k] = reinterpret_cast<const __nv_bfloat16*>(half)[k];
            }
          }
        }
    }
    cluster_sync();  // the peers have read this CTA's sums
  }
  umma_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_sync();  // nothing of the pair reads or signals this CTA any more
  umma_fence_after();
  if (warp == 2) {
    if constexpr (kPair)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kCols) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kCols) : "memory");
  }
  if constexpr (LORA) {
    if (bars.special)
      add_special<MX, T>(p, bars, GemmTiles<kGemmRows, T>{p, start, lo, hi, units, tiles, places, place, 1, 0},
                         static_cast<int>(rank), splits, part_k);
  }
}

// Row r (of 32) of scale tile `ct` of `rows` rows from row0 on: 4 scales each of the rows r, r + 32, r + 64,
// r + 96; zeros past the rows and past a row's end.
__device__ __forceinline__ uint4 scale_tile_row(const uint8_t* s, int64_t row0, int rows, int row_bytes, int ct, int r) {
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    w[q] = 0;
    if (q * 32 + r >= rows) continue;
    const uint8_t* src = s + (row0 + q * 32 + r) * row_bytes + 4 * ct;
    if (row_bytes % 4 == 0 && reinterpret_cast<uintptr_t>(s) % 4 == 0) {
      w[q] = __ldg(reinterpret_cast<const uint32_t*>(src));
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (4 * ct + c < row_bytes) w[q] |= static_cast<uint32_t>(__ldg(src + c)) << (8 * c);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---------------------------------------------------------------------------
// The adapters' first product: t[m, r] = scaling[a] / (x_sg w_sg) sum_k x[m, k] A_a[r, k] for row m of
// adapter a, in two bf16 terms.  (The division undoes what the epilogue multiplies the whole
// accumulator by.)
//
// A CTA takes a tile of 128 rows (the lanes of tensor memory) and a slice of k.  The columns of one
// instruction are the ranks of several of the tile's distinct adapters side by side, up to 128: x is
// read once for all of them, and a row keeps the columns of its own adapter.  More adapters than
// fit take further passes; with few row tiles, several CTAs per slice share the adapters (`jobs`).  The
// slices of a tile are a cluster, which adds their sums in distributed shared memory in a fixed order.
//
// Tensor memory is taken after the wait for the kernel before and freed before the cluster's barriers: CTAs of
// several launches share an SM's 512 columns in whatever order they come, and one that held columns while it waited
// for a peer, which waits for columns elsewhere, could wait for ever.  So the sums of several passes, a row's own
// columns of each, are gathered beside the accumulator (`own`) until the last pass is done, and exchanged once.
// Bound by reading x and each distinct adapter of every tile once ([4096, 4096], 8 adapters of rank 64: 15 us for
// 38 MB; 32 rows of 24 adapters: 7 us, latencies); two CTAs per SM keep 192 KB of loads in flight.  Warps 0..3: the tile's lanes; warp 4: TMA; warp 5: the products.
// ---------------------------------------------------------------------------
constexpr int kShrinkThreads = 192;
constexpr int kShrinkRows = 128;
constexpr int kShrinkCols = 128;                    // columns of a pass, at most
constexpr int kShrinkMaxStages = 4;
constexpr int kShrinkPad = 4;                       // floats between rows of sums

struct ShrinkParams {
  const float* scaling;    // [adapters]
  const float* sg_a;       // NULL: 1
  const float* sg_b;
  const int32_t* ids;
  __nv_bfloat16* t;        // [rows][hi, lo][rank]
  // x's scales, row-major, and where they go in the tile layout for the wide products (NULL: nowhere)
  const uint8_t* scales;
  uint4* tiles;
  int scale_row_bytes, scale_tiles;
  int rows, K, adapters, rank, slices, jobs;
  // rows of x in a stage (fewer than the 128 lanes where there are not so many: the others' columns are
  // not read), columns of a pass, stages
  int box_rows, cols, stages;
  // columns of tensor memory: those of a pass and, where there may be several, of a row's sums behind them; no more
  // than needed, or the SM's next CTAs wait for them
  int tmem_cols;
};

__global__ void __launch_bounds__(kShrinkThreads)
    k_lora_shrink(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_a,
                  const __grid_constant__ ShrinkParams p) {
  extern __shared__ uint8_t shrink_smem_raw[];
  __shared__ struct {
    uint64_t full[kShrinkMaxStages], empty[kShrinkMaxStages], done;
    uint32_t tmem;
    int n;                        // adapters of this CTA
    int16_t slot[kShrinkRows];    // a row's place among them, or -1
    int adapter[kShrinkRows];     // the tile's distinct adapters, in the order of their first row
  } sh;
  uint8_t* const ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(shrink_smem_raw) + 1023) & ~uintptr_t{1023});
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int slice = blockIdx.x % p.slices, job = blockIdx.x / p.slices % p.jobs;
  const int row0 = blockIdx.x / p.slices / p.jobs * kShrinkRows;
  const int padded = (p.rank + 15) & ~15;

  if (threadIdx.x == 128) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(smem_addr(&sh.full[i]), 1);
      mbar_init(smem_addr(&sh.empty[i]), 1);
    }
    mbar_init(smem_addr(&sh.done), 1);
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)),
                 "r"(p.tmem_cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    // After the wait, since the products may start under this kernel and read what it waited for; and with the
    // columns in hand, since the products take theirs when they start.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
  if (warp == 0) {  // the distinct adapters; every jobs-th of them is this CTA's
    int ids[kShrinkRows / 32], n = 0;
#pragma unroll
    for (int c = 0; c < kShrinkRows / 32; ++c) {
      const int r = row0 + 32 * c + lane;
      ids[c] = r < p.rows ? __ldg(p.ids + r) : -1;
    }
#pragma unroll
    for (int c = 0; c < kShrinkRows / 32; ++c) {
      const int id = ids[c] >= 0 && ids[c] < p.adapters ? ids[c] : -1;
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, id);
      int at = -1;
      for (int j = 0; j < n; ++j)
        if (sh.adapter[j] == id) at = j;
      const bool first = id >= 0 && at < 0 && lane == __ffs(same) - 1;
      const uint32_t firsts = __ballot_sync(0xFFFFFFFFu, first);
      if (id >= 0 && at < 0) at = n + __popc(firsts & ((1u << (__ffs(same) - 1)) - 1));
      if (first) sh.adapter[at] = id;
      sh.slot[32 * c + lane] = static_cast<int16_t>(at >= 0 && at % p.jobs == job ? at / p.jobs : -1);
      n += __popc(firsts);
      __syncwarp();
    }
    if (lane == 0) sh.n = n > job ? (n - job + p.jobs - 1) / p.jobs : 0;
  }
  umma_fence_before();
  __syncthreads();
  umma_fence_after();
  const uint32_t tmem = sh.tmem;
  const int n = sh.n, per_pass = p.cols / padded, passes = (n + per_pass - 1) / per_pass;
  const int stage_bytes = (p.box_rows + p.cols) * 128;
  const int blocks = (p.K + 63) / 64, per = (blocks + p.slices - 1) / p.slices;
  const int kb0 = slice * per, kb1 = min(blocks, kb0 + per);
  bool ok = true;
  float inv = 1.0f;
  if (p.sg_a) inv = __fdiv_rn(1.0f, __fmul_rn(__ldg(p.sg_a), __ldg(p.sg_b)));
  // The sums [row][rank], in 16-byte pieces: with this pitch lanes (rows) write them without bank conflicts; a row
  // is read from other CTAs along its ranks (32 rows at once are 32 requests each: 20 us for 4096 rows).
  float* const sums = reinterpret_cast<float*>(ring);
  const int pitch = padded + kShrinkPad;
  const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);  // (warps 0..3)
  auto put_sums = [&](int r, const uint32_t (&v)[16]) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *reinterpret_cast<uint4*>(sums + (warp * 32 + lane) * pitch + r + 4 * k) =
          kb1 > kb0 ? make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]) : make_uint4(0, 0, 0, 0);
  };
  GemmRing at;
  const uint64_t ring0 = desc_codes(smem_addr(ring));
  long long fills = 0;

  if (warp < 4 && p.tiles && job == 0)  // under the products: this slice's part of the rows' scales
    for (int ct = slice * 4 + warp; ct < p.scale_tiles; ct += 4 * p.slices)
      p.tiles[(static_cast<int64_t>(row0 / 128) * p.scale_tiles + ct) * 32 + lane] =
          scale_tile_row(p.scales, row0, min(128, p.rows - row0), p.scale_row_bytes, ct, lane);

  for (int pass = 0; pass < passes; ++pass) {  // (as many in every CTA of the cluster)
    const int slots = min(per_pass, n - pass * per_pass);
    if (warp == 4) {
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = ok && warp_wait(smem_addr(&sh.empty[at.s]), at.phase ^ 1);
        const uint32_t bar = smem_addr(&sh.full[at.s]), st = smem_addr(ring) + at.s * stage_bytes;
        if (!ok) break;
        ++fills;
        if (elect_one()) {
          mbar_expect_tx(bar, (p.box_rows + slots * padded) * 128);
          tma_tile2<false>(st, &map_x, kb * 64, row0, bar);
          for (int i = 0; i < slots; ++i)
            tma_tile3<false>(st + (p.box_rows + i * padded) * 128, &map_a, kb * 64, 0,
                             sh.adapter[job + (pass * per_pass + i) * p.jobs], bar);
        }
        __syncwarp();
        at.next(p.stages);
      }
    } else if (warp == 5) {
      const uint32_t idesc = umma_idesc_bf16(kShrinkRows, slots * padded);
      for (int kb = kb0; kb < kb1 && ok; ++kb) {
        ok = warp_wait(smem_addr(&sh.full[at.s]), at.phase);
        umma_fence_after();
        const uint64_t st = ring0 + at.s * (stage_bytes >> 4);
        if (ok && elect_one()) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            umma_bf16<false>(tmem, st + 2 * j, st + (p.box_rows * 128 >> 4) + 2 * j, idesc, kb > kb0 || j > 0);
          umma_commit<false>(smem_addr(&sh.empty[at.s]));
        }
        __syncwarp();
        at.next(p.stages);
      }
      if (elect_one()) umma_commit<false>(smem_addr(&sh.done));
      __syncwarp();
    }
    // Every copy has been read and every product is complete (a failed wait: bounded here too).
    ok = mbar_wait(smem_addr(&sh.done), pass & 1) && ok;
    umma_fence_after();
    __syncthreads();
    if (warp < 4) {  // each row's own columns
      const int mine = sh.slot[warp * 32 + lane] - pass * per_pass;
      for (int i = 0; i < slots; ++i) {
        if (!__any_sync(0xFFFFFFFFu, mine == i)) continue;
        for (int r = 0; r < padded; r += 16) {
          uint32_t v[16];
          tmem_load(lanes + i * padded + r, v);
          if (passes == 1) {
            if (mine == i) put_sums(r, v);
          } else {
            uint32_t own[16];
            tmem_load(lanes + p.cols + r, own);
#pragma unroll
            for (int k = 0; k < 16; ++k) own[k] = mine == i ? v[k] : own[k];
            tmem_store(lanes + p.cols + r, own);
          }
        }
      }
    }
    umma_fence_before();
    __syncthreads();  // the accumulator has been read
    umma_fence_after();
  }
  if (passes > 1 && warp < 4) {
    for (int r = 0; r < padded; r += 16) {
      uint32_t v[16];
      tmem_load(lanes + p.cols + r, v);
      if (sh.slot[warp * 32 + lane] >= 0) put_sums(r, v);
    }
    umma_fence_before();
  }
  if (passes > 1) __syncthreads();
  umma_fence_after();
  if (warp == 5)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.tmem_cols) : "memory");
  __syncwarp();
  cluster_sync();
  // Each CTA of the cluster finishes every slices-th row, 4 ranks per thread.
  const int quads = p.rank / 4, items = kShrinkRows / p.slices * quads;
  for (int item = threadIdx.x; item < items; item += kShrinkThreads) {
    const int row = slice + item / quads * p.slices, r = item % quads * 4, slot = sh.slot[row];
    if (slot < 0) continue;
    const float scale = __ldg(p.scaling + sh.adapter[job + slot * p.jobs]) * inv;
    float4 part[kMaxSplits];
#pragma unroll
    for (int k = 0; k < kMaxSplits; ++k)  // without a condition: all in flight before the first is added
      part[k] = load_cluster4(sums + row * pitch + r, min(k, p.slices - 1));
    float v[4] = {part[0].x, part[0].y, part[0].z, part[0].w};
#pragma unroll
    for (int k = 1; k < kMaxSplits; ++k) {
      if (k >= p.slices) continue;
      v[0] += part[k].x, v[1] += part[k].y, v[2] += part[k].z, v[3] += part[k].w;
    }
    __nv_bfloat162 hi[2], lo[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float x = v[2 * k] * scale, y = v[2 * k + 1] * scale;
      hi[k] = __floats2bfloat162_rn(x, y);
      // (of an infinity nothing is left: inf - inf would make the sum NaN)
      const float hx = __low2float(hi[k]), hy = __high2float(hi[k]);
      lo[k] = __floats2bfloat162_rn(isinf(hx) ? 0.0f : x - hx, isinf(hy) ? 0.0f : y - hy);
    }
    __nv_bfloat16* const t = p.t + static_cast<int64_t>(row0 + row) * 2 * p.rank + r;
    *reinterpret_cast<uint2*>(t) = *reinterpret_cast<const uint2*>(hi);
    *reinterpret_cast<uint2*>(t + p.rank) = *reinterpret_cast<const uint2*>(lo);
  }
  if (!ok && warp == 4)  // let the copies in flight land (bounded)
    for (long long f = fills > p.stages ? fills - p.stages : 0; f < fills; ++f)
      mbar_wait(smem_addr(&sh.full[f % p.stages]), (f / p.stages) & 1);
  if (!ok && lane == 0) atomicOr(&g_hq_fault, kFaultWaitTimeout);
  __syncwarp();
  cluster_sync();  // the peers have read this CTA's sums
}

}  // namespace hq
