// hq_tcgen05.cuh -- what the products on the 5th-generation tensor cores share (sm_103a): copies, matrix products and
// tensor memory in inline PTX, and the way of an accumulator's columns to rows of the output.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "hq_kernels.cuh"

namespace hq {

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

// d += A (tensor memory) B (shared memory), both f16.
template <bool PAIR>
__device__ __forceinline__ void umma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

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
// The same in two steps.
__device__ __forceinline__ void tmem_store_nowait(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
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

}  // namespace hq
