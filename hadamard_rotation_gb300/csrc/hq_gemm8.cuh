// hq_gemm8.cuh -- device code of the product of INT8 codes (sm_103a).
//
//   out[m, n] = (sum_k X[m, k] W[n, k]) xs[m] ws[n]
//
// This chip multiplies 8-bit integers at a small part of its 16-bit rate, so the codes are widened to f16 on the way to
// the tensor cores (tcgen05.mma, kind f16).  A code has 8 bits and f16 holds 11, so the operands and their products
// are exact, and so is the fp32 sum while it stays below 2^24.
//
// The weights' channels are the M side of the instruction and lie in tensor memory; the tokens are its N side and lie in
// shared memory.  Both come from global memory as they are (TMA, 64 or 128 codes of a row, swizzled), are read
// a row per thread, widened, and written: channels by tcgen05.st, tokens by 16-byte stores in the swizzle that the
// instruction reads.  Widening: a code with its sign bit flipped, as the low byte of f16 0x64.., is 1024 + 128 +
// code; one subtraction of pairs gives code.
//
// Large products are taken by pairs of CTAs (WIDE, cta_group::2) in tiles of 256 channels x up to 256 tokens: each CTA
// widens 128 rows of each side, and its shared memory moves 64 KB in the 512 cycles of a stage, of 66 KB that it can.
// With the channels in shared memory too it would be 96.
// Few tokens: single CTAs, up to 128 channels x up to 64 tokens (fewer channels where that evens out what the SMs get; the
// instruction's other lanes hold whatever lies there and are not stored); with fewer tiles than SMs the CTAs of a cluster
// share the summed axis (SPLIT) and add their parts through distributed shared memory in a fixed order.
//
// Roles of a CTA:
//   warp 0         TMA
//   warp 1         issues the products
//   warp 2         allocates tensor memory
//   sets of 8      four warps widen the channels (a quarter of the lanes each), four the tokens; the sets take stages in
//                  turn, for a stage's way through one warp is mostly latency
//   the last       epilogue, groups of four warps: tensor memory -> registers -> scales -> shared memory -> global
#pragma once

#include <cuda_fp16.h>

#include "hq_tcgen05.cuh"

namespace hq {

struct Gemm8Params {
  const float *xs, *ws;
  int M, N, K;
  int tiles_a, tiles_b;  // over the channels, over the tokens
  int lanes;             // channels of a tile (of the pair's CTA: 128)
  int width;             // tokens of a tile
  int box_b;             // rows of a copy of tokens
  void* out;
  int out_f32;
  int out_tma;  // bf16 rows aligned to 16 bytes: map_out is valid
  int out_vec;  // bytes per store: what the rows of out are aligned to, up to 16
};

constexpr int kGemm8MaxSplits = 8;

template <bool WIDE>
struct Gemm8Shape {
  static constexpr int kCtas = WIDE ? 2 : 1;
  static constexpr int T = WIDE ? 256 : 64;     // tokens of a tile, at most
  static constexpr int kBlock = WIDE ? 64 : 128;  // summed codes per stage
  static constexpr int kRowsB = T / kCtas;      // in a CTA
  static constexpr int kTileLanes = 128 * kCtas;
  static constexpr int kRawA = 128 * kBlock, kRawB = kRowsB * kBlock, kRawBytes = kRawA + kRawB;
  static constexpr int kRaw = 6;                // stages of codes
  static constexpr int kWideBytes = kRowsB * kBlock * 2;
  static constexpr int kWides = WIDE ? 6 : 4;   // stages of widened operands
  static constexpr int kAccs = WIDE ? 1 : 2;
  static constexpr int kColA = kAccs * T;       // the channels' columns of tensor memory: kBlock / 2 per stage
  static_assert(kColA + kBlock / 2 * kWides <= 512, "tensor memory has 512 columns");
  static constexpr int kEpilogues = WIDE ? 2 : 1;
  // Sets of eight warps (four for the channels, four for the tokens) that widen stages in turn.
  static constexpr int kSets = 2;
  // A place is used by the same set each time.  Otherwise a set could come to a place two uses ahead of the copy that
  // another set still waits for, where the parity says that its own has landed.
  static_assert(kRaw % kSets == 0 && kWides % kSets == 0, "a place belongs to one set");
  static constexpr int kEpilogueWarp = 4 + 8 * kSets;
  static constexpr int kThreads = 32 * (kEpilogueWarp + 4 * kEpilogues);
  static constexpr int kWideAt = kRaw * kRawBytes, kOutAt = kWideAt + kWides * kWideBytes;
  static constexpr int kSmemBytes = kOutAt + kEpilogues * kOutBytes;
  static_assert(kSmemBytes + 1024 + 4096 <= 227 * 1024, "a CTA has 227 KB");
  static_assert(2 * kSmemBytes > 228 * 1024, "no two CTAs of these kernels share an SM");
  static_assert(WIDE || kWides * kWideBytes >= T * 128 * 4, "a part's sums lie over the widened tokens");
};

struct Gemm8Bars {
  uint64_t raw_full[12], raw_empty[12];
  uint64_t wide_full[12], wide_empty[12];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  float xs[2][256];  // a tile's token scales, by epilogue group
  uint32_t tmem;
};

// f16 x f16 into fp32, both operands along K.
__device__ __forceinline__ uint32_t umma_idesc_f16(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// Four codes into two pairs of f16.
__device__ __forceinline__ uint2 widen8(uint32_t w) {
  w ^= 0x80808080u;
  const uint32_t lo = __byte_perm(w, 0x64646464u, 0x4140), hi = __byte_perm(w, 0x64646464u, 0x4342);
  const __half2 bias = __floats2half2_rn(-1152.0f, -1152.0f);
  const __half2 a = __hadd2(*reinterpret_cast<const __half2*>(&lo), bias), b = __hadd2(*reinterpret_cast<const __half2*>(&hi), bias);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// Sixteen codes, 16-byte piece `j` of row r of a stage: rows of BLOCK bytes, swizzled by the copy.
template <int BLOCK>
__device__ __forceinline__ void widen_piece(const uint8_t* rows, int r, int j, uint32_t (&v)[8]) {
  const int at = BLOCK == 128 ? j ^ (r & 7) : j ^ ((r >> 1) & 3);
  const uint4 w = *reinterpret_cast<const uint4*>(rows + r * BLOCK + (at << 4));
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint2 p = widen8(u[i]);
    v[2 * i] = p.x;
    v[2 * i + 1] = p.y;
  }
}

// An arrival on a barrier of the pair's first CTA that releases what this CTA's threads wrote to their own shared and
// tensor memory: there the tensor core reads it, and the fences in front have made it visible to it.  (Released to the whole
// cluster, an arrival waits for 1000 cycles and more: [8192, 8192] x 8192 1093 us in place of 666.)
__device__ __forceinline__ void mbar_arrive_cta(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

struct Gemm8Tile {
  int a0, b0;    // first channel and token (of the pair)
  int valid, n;  // tokens that exist, columns of the instruction
};

template <bool WIDE>
__device__ __forceinline__ Gemm8Tile gemm8_tile(const Gemm8Params& p, int tile) {
  const int at = tile / p.tiles_b, bt = tile - at * p.tiles_b;
  Gemm8Tile t;
  t.a0 = at * (WIDE ? 256 : p.lanes);
  t.b0 = bt * p.width;
  t.valid = min(p.width, p.M - t.b0);
  t.n = WIDE ? (t.valid + 31) & ~31 : (t.valid + 15) & ~15;
  return t;
}

// 32 columns (bf16) or 16 (fp32) of the accumulator, times both scales, as they are stored.  xs: of the columns.
__device__ __forceinline__ void fetch8_bf16(uint32_t from, const float* xs, const float (&ws)[4], int lane, uint32_t (&w)[16]) {
  uint32_t v[2][16];
  tmem_load_fragments(from, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = *reinterpret_cast<const float2*>(xs + 8 * i + 2 * (lane & 3));
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const uint32_t* f = &v[m >> 1][4 * i + 2 * (m & 1)];
      const __nv_bfloat162 b = __floats2bfloat162_rn(__fmul_rn(__fmul_rn(__uint_as_float(f[0]), x.x), ws[m]),
                                                     __fmul_rn(__fmul_rn(__uint_as_float(f[1]), x.y), ws[m]));
      w[4 * i + m] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
}
__device__ __forceinline__ void fetch8_f32(uint32_t from, const float* xs, float ws, uint32_t (&w)[16]) {
  tmem_load(from, w);
#pragma unroll
  for (int c = 0; c < 16; ++c) w[c] = __float_as_uint(__fmul_rn(__fmul_rn(__uint_as_float(w[c]), xs[c]), ws));
}

template <bool WIDE, bool SPLIT>
__global__ void __launch_bounds__((Gemm8Shape<WIDE>::kThreads), 1)
    k_gemm8(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
            const __grid_constant__ CUtensorMap map_out, const __grid_constant__ Gemm8Params p) {
  using S = Gemm8Shape<WIDE>;
  static_assert(!(WIDE && SPLIT), "pairs do not split the sum");
  constexpr int kCtas = S::kCtas, kEpilogues = S::kEpilogues;
  extern __shared__ uint8_t gemm8_smem_raw[];
  __shared__ Gemm8Bars bars;
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(gemm8_smem_raw) + 1023) & ~uintptr_t{1023});
  uint8_t* const wide = smem + S::kWideAt;
  uint8_t* const outs = smem + S::kOutAt;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = WIDE ? cluster_rank() : 0;  // of the pair; CTA 0 issues the products
  const int splits = SPLIT ? static_cast<int>(cluster_size()) : 1, part_k = SPLIT ? static_cast<int>(cluster_rank()) : 0;

  if (warp == 2) {
    if constexpr (WIDE) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&bars.tmem)) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&bars.tmem)) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // Only now, and by this warp: the kernel after this one may take tensor memory before it waits for this one,
    // and must not find it free before this CTA has its own.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
  if (warp == 1 && lane == 0) {
    for (int i = 0; i < S::kRaw; ++i) {
      mbar_init(smem_addr(&bars.raw_full[i]), 1);
      mbar_init(smem_addr(&bars.raw_empty[i]), 8);
    }
    for (int i = 0; i < S::kWides; ++i) {
      mbar_init(smem_addr(&bars.wide_full[i]), 8 * kCtas);
      mbar_init(smem_addr(&bars.wide_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&bars.acc_full[i]), 1);
      mbar_init(smem_addr(&bars.acc_empty[i]), 4 * kEpilogues * kCtas);
    }
    mbar_init(smem_addr(&bars.drain), 1);
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the kernel before this one wrote the operands
  umma_fence_before();
  __syncthreads();
  if constexpr (WIDE) cluster_sync();  // the peer's barriers are there
  umma_fence_after();
  const uint32_t tmem = bars.tmem;
  const int group = kCtas * splits, step = static_cast<int>(gridDim.x) / group, first = static_cast<int>(blockIdx.x) / group;
  const int tiles = p.tiles_a * p.tiles_b;
  // this CTA's part of the summed axis, in stages
  const int all = (p.K + S::kBlock - 1) / S::kBlock;
  const int kb0 = all * part_k / splits, kb1 = all * (part_k + 1) / splits;
  bool ok = true;

  if (warp == 0) {
    GemmRing ring;
    long long fills = 0;
    for (int tile = first; ok && tile < tiles; tile += step) {
      const Gemm8Tile t = gemm8_tile<WIDE>(p, tile);
      const int a0 = t.a0 + static_cast<int>(rank) * 128, b0 = t.b0 + static_cast<int>(rank) * (t.n / 2);
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = warp_wait(smem_addr(&bars.raw_empty[ring.s]), ring.phase ^ 1);
        if (!ok) break;
        const uint32_t full = smem_addr(&bars.raw_full[ring.s]), st = smem_addr(smem) + ring.s * S::kRawBytes;
        if (elect_one()) {
          mbar_expect_tx(full, (p.lanes + p.box_b) * S::kBlock);
          tma_tile2<false>(st, &map_w, kb * S::kBlock, a0, full);
          tma_tile2<false>(st + S::kRawA, &map_x, kb * S::kBlock, b0, full);
        }
        __syncwarp();
        ++fills;
        ring.next(S::kRaw);
      }
    }
    if (!ok)  // let the copies in flight land (bounded) before the CTA may end
      for (long long f = fills > S::kRaw ? fills - S::kRaw : 0; f < fills; ++f)
        mbar_wait(smem_addr(&bars.raw_full[f % S::kRaw]), (f / S::kRaw) & 1);
  } else if (warp == 1 && rank == 0) {
    GemmRing ring;
    int acc = 0;
    uint32_t acc_phase = 0;
    const uint64_t b_desc = desc_codes(smem_addr(wide));
    for (int tile = first; ok && tile < tiles; tile += step) {
      const Gemm8Tile t = gemm8_tile<WIDE>(p, tile);
      ok = warp_wait(smem_addr(&bars.acc_empty[acc]), acc_phase ^ 1);
      if (!ok) break;
      umma_fence_after();
      const uint32_t d = tmem + acc * S::T, idesc = umma_idesc_f16(S::kTileLanes, t.n);
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = warp_wait(smem_addr(&bars.wide_full[ring.s]), ring.phase);
        if (!ok) break;
        umma_fence_after();
        if (elect_one()) {
          const uint32_t a = tmem + S::kColA + S::kBlock / 2 * ring.s;
          const uint64_t b = b_desc + ring.s * (S::kWideBytes >> 4);
#pragma unroll
          for (int j = 0; j < S::kBlock / 16; ++j)  // 16 codes each; four in a row of the swizzle
            umma_f16_ts<WIDE>(d, a + 8 * j, b + (j / 4) * (S::kRowsB * 128 >> 4) + 2 * (j % 4), idesc, kb > kb0 || j > 0);
          umma_commit<WIDE>(smem_addr(&bars.wide_empty[ring.s]));
        }
        __syncwarp();
        ring.next(S::kWides);
      }
      if (!ok) break;
      if (elect_one()) umma_commit<WIDE>(smem_addr(&bars.acc_full[acc]));
      __syncwarp();
      if (++acc == S::kAccs) {
        acc = 0;
        acc_phase ^= 1;
      }
    }
    if (!ok) {  // let the products in flight finish (bounded) before tensor memory is freed
      if (elect_one()) umma_commit<WIDE>(smem_addr(&bars.drain));
      __syncwarp();
      mbar_wait(smem_addr(&bars.drain), 0);
    }
  } else if (warp >= 4 && warp < S::kEpilogueWarp) {
    const int set = (warp - 4) / 8;
    const bool channels = ((warp - 4) & 4) == 0;
    // (64 tokens at most: two threads a row, each half of a stage's codes)
    const int r = (channels || WIDE ? warp & 3 : warp & 1) * 32 + lane;
    constexpr int kPieces = S::kBlock / 16, kPiecesB = WIDE ? kPieces : kPieces / 2;
    const int half0 = !WIDE && (warp & 2) ? kPiecesB : 0;
    GemmRing raw, ring;
    int turn = 0;
    for (int tile = first; ok && tile < tiles; tile += step) {
      const Gemm8Tile t = gemm8_tile<WIDE>(p, tile);
      const int rows_b = t.n / kCtas;
      const bool mine = channels || r < rows_b;
      for (int kb = kb0; kb < kb1; ++kb, raw.next(S::kRaw), ring.next(S::kWides)) {
        const bool another = turn != set;
        if (++turn == S::kSets) turn = 0;
        if (another) continue;
        ok = warp_wait(smem_addr(&bars.wide_empty[ring.s]), ring.phase ^ 1) && warp_wait(smem_addr(&bars.raw_full[raw.s]), raw.phase);
        if (!ok) break;
        const uint8_t* const rows = smem + raw.s * S::kRawBytes + (channels ? 0 : S::kRawA);
        if (channels) {
          umma_fence_after();
          const uint32_t to = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + S::kColA + S::kBlock / 2 * ring.s;
#pragma unroll
          for (int j = 0; j < kPieces; j += 2) {
            uint32_t v[16];
            widen_piece<S::kBlock>(rows, r, j, *reinterpret_cast<uint32_t(*)[8]>(v));
            widen_piece<S::kBlock>(rows, r, j + 1, *reinterpret_cast<uint32_t(*)[8]>(v + 8));
            tmem_store_nowait(to + 8 * j, v);
          }
          tmem_store_wait();
          umma_fence_before();
        } else if (mine) {
          uint8_t* const to = wide + ring.s * S::kWideBytes + r * 128;
#pragma unroll
          for (int i = 0; i < kPiecesB; ++i) {
            const int j = half0 + i, at = 2 * (j % 4);
            uint32_t v[8];
            widen_piece<S::kBlock>(rows, r, j, v);
            uint8_t* const half = to + (j / 4) * (S::kRowsB * 128);
            *reinterpret_cast<uint4*>(half + ((at ^ (r & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<uint4*>(half + (((at + 1) ^ (r & 7)) << 4)) = make_uint4(v[4], v[5], v[6], v[7]);
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_addr(&bars.raw_empty[raw.s]));
          if (rank) mbar_arrive_cta(cluster_addr(smem_addr(&bars.wide_full[ring.s]), 0));
          else mbar_arrive(smem_addr(&bars.wide_full[ring.s]));
        }
      }
    }
  } else if (warp >= S::kEpilogueWarp) {
    const int part = (warp - S::kEpilogueWarp) / 4, quarter = warp & 3, tid = threadIdx.x & 127;
    auto sync = [&]() {
      if (part == 0) role_sync<2>();
      else role_sync<3>();
    };
    int acc = 0;
    uint32_t acc_phase = 0;
    const int es = p.out_f32 ? 4 : 2, block = p.out_f32 ? 16 : 32;
    uint8_t* const buf = outs + part * kOutBytes;
    float* const xs = bars.xs[part];
    for (int tile = first; tile < tiles; tile += step) {
      const Gemm8Tile t = gemm8_tile<WIDE>(p, tile);
      const int a0 = t.a0 + static_cast<int>(rank) * 128;
      float ws[4];  // of the lanes of a fragment, or (fp32) of the thread's lane
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int n = a0 + quarter * 32 + (p.out_f32 ? lane : 8 * m + lane / 4);
        ws[m] = n < p.N ? __ldg(p.ws + n) : 0.0f;
      }
      sync();  // the last tile's scales have been read
      for (int c = tid; c < S::T; c += 128) xs[c] = c < t.valid ? __ldg(p.xs + t.b0 + c) : 0.0f;
      const bool full = mbar_wait(smem_addr(&bars.acc_full[acc]), acc_phase);
      ok = part == 0 ? role_all<2>(full) : role_all<3>(full);
      if (!ok) break;
      umma_fence_after();
      const int64_t stride = static_cast<int64_t>(p.N) * es;
      uint8_t* const out = static_cast<uint8_t*>(p.out) + t.b0 * stride + static_cast<int64_t>(a0) * es;
      const int bytes = min(p.lanes, p.N - a0) * es;  // (not positive: the pair's second CTA has no channels here)
      const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + acc * S::T;
      bool held = true;
      if constexpr (SPLIT) {  // the partial sums as they are, over the widened tokens, which have been multiplied
        float* const sums = reinterpret_cast<float*>(wide);
        for (int c0 = 0; c0 < t.valid; c0 += 16) {
          uint32_t v[16];
          tmem_load(from + c0, v);
#pragma unroll
          for (int c = 0; c < 16; ++c) sums[(c0 + c) * 128 + tid] = kb1 > kb0 ? __uint_as_float(v[c]) : 0.0f;
        }
        umma_fence_before();
      } else
      for (int c0 = part * block; c0 < t.valid; c0 += kEpilogues * block) {
        uint32_t w[16];
        if (p.out_f32) fetch8_f32(from + c0, xs + c0, ws[0], w);
        else fetch8_bf16(from + c0, xs + c0, ws, lane, w);
        if (c0 + kEpilogues * block >= t.valid) {  // the group's last chunk: its part has been read
          umma_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (rank) mbar_arrive_cluster_relaxed(cluster_addr(smem_addr(&bars.acc_empty[acc]), 0));
            else mbar_arrive(smem_addr(&bars.acc_empty[acc]));
          }
          held = false;
        }
        // (The copies of a block's two halves are issued by two warps, by the same elected lane each time.)
        if (quarter < 2) {
          if (elect_one()) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();
        }
        sync();  // the last chunk has left the buffer
        if (p.out_f32) put_f32(buf, w, tid);
        else put_bf16(buf, w, quarter, lane);
        fence_proxy_async_smem();
        sync();
        const int rows = min(block, t.valid - c0);
        if (p.out_tma && rows == 32) {
          const int x = a0 + 64 * quarter;
          if (quarter < 2 && x < p.N && elect_one()) {
            tma_store3(&map_out, smem_addr(buf) + 4096 * quarter, x, t.b0 + c0, 0);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        } else if (p.out_f32) {
          store_rows<true>(p.out_vec, buf, out + c0 * stride, stride, rows, bytes, tid);
        } else {
          store_rows<false>(p.out_vec, buf, out + c0 * stride, stride, rows, bytes, tid);
        }
        __syncwarp();
      }
      if (held) {  // no chunk for this group
        __syncwarp();
        if (lane == 0) {
          if (rank) mbar_arrive_cluster_relaxed(cluster_addr(smem_addr(&bars.acc_empty[acc]), 0));
          else mbar_arrive(smem_addr(&bars.acc_empty[acc]));
        }
      }
      if (++acc == S::kAccs) {
        acc = 0;
        acc_phase ^= 1;
      }
    }
    if (elect_one()) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  if (!ok && lane == 0) atomicOr(&g_hq_fault, kFaultWaitTimeout);
  __syncwarp();
  if constexpr (SPLIT) {  // each CTA of the cluster finishes its share of the columns, adding the parts in order
    cluster_sync();
    if (first < tiles) {
      const Gemm8Tile t = gemm8_tile<WIDE>(p, first);
      const float* const sums = reinterpret_cast<const float*>(wide) + lane * 4;  // four lanes of a column per thread
      const int n = t.a0 + lane * 4, es = p.out_f32 ? 4 : 2;
      float ws[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) ws[k] = n + k < p.N ? __ldg(p.ws + n + k) : 0.0f;
      if (n < p.N && lane * 4 < p.lanes)
        for (int c = part_k + splits * warp; c < t.valid; c += splits * static_cast<int>(blockDim.x >> 5)) {
          float4 v[kGemm8MaxSplits];
          const float x = __ldg(p.xs + t.b0 + c);
#pragma unroll
          for (int k = 0; k < kGemm8MaxSplits; ++k)  // without a condition: all in flight before the first is added
            v[k] = load_cluster4(sums + c * 128, min(k, splits - 1));
          float sum[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
          for (int k = 1; k < kGemm8MaxSplits; ++k) {
            if (k >= splits) continue;
            sum[0] += v[k].x, sum[1] += v[k].y, sum[2] += v[k].z, sum[3] += v[k].w;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) sum[k] = __fmul_rn(__fmul_rn(sum[k], x), ws[k]);
          uint8_t* const out = static_cast<uint8_t*>(p.out) + (static_cast<int64_t>(t.b0 + c) * p.N + n) * es;
          const __nv_bfloat162 half[2] = {__floats2bfloat162_rn(sum[0], sum[1]), __floats2bfloat162_rn(sum[2], sum[3])};
          if (p.out_vec >= 4 * es && n + 3 < p.N) {
            if (p.out_f32) *reinterpret_cast<float4*>(out) = make_float4(sum[0], sum[1], sum[2], sum[3]);
            else *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(half);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (n + k >= p.N) continue;
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
  if constexpr (WIDE) cluster_sync();  // nothing of the pair reads or signals this CTA any more
  umma_fence_after();
  if (warp == 2) {
    if constexpr (WIDE) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

}  // namespace hq
