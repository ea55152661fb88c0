// hq_kv.cuh -- device code of the paged NVFP4 cache of keys and values (sm_103a): appending to it, reading it back,
// and attention over it for few queries per sequence (hq_kv_prompt.cuh: for many).
//
// The cache is made of records: 16 tokens of one head, 18 D bytes in one piece,
//   K codes [16, D / 2] | V codes [16, D / 2] | K scales [16, D / 16] | V scales [16, D / 16],
// so that everything a step of the attention reads of 16 tokens is one contiguous copy, whatever the page size (a
// multiple of 16) is.  A page is [kv_heads][page_size / 16] records.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <limits.h>

#include "hq_kernels.cuh"

namespace hq {

constexpr int kKvUnit = 16;  // tokens of a record

template <int D>
struct KvRecord {
  static constexpr int kCodes = 16 * D / 2;   // K's (V's) code bytes
  static constexpr int kScales = 16 * D / 16;
  static constexpr int kV = kCodes, kKs = 2 * kCodes, kVs = 2 * kCodes + kScales;
  static constexpr int kBytes = 2 * kCodes + 2 * kScales;
  static_assert(kBytes == 18 * D, "a record");
};

// s_global of amax, as the quantizer has it.
__device__ __forceinline__ float kv_global_scale(float amax) {
  const float s = __fdiv_rn(amax, 2688.0f);
  return s == 0.0f ? 1.0f : s;
}

// ---------------------------------------------------------------------------
// Appending.
//
// A thread takes 16 channels of a (token, head): position rotation (two products and a sum, each rounded, as the
// definition in hq.h has them), butterfly in pairs of channels, then for K and V the block scale and codes exactly as
// hq_rotate_quant_nvfp4, with the quantizer's corrected quotients.  PAIRED (all of a head turned, halves against each
// other): a thread loads and turns 8 channels of either half, so that each table entry and each channel is loaded once,
// and swaps one of them with its neighbour.
// Instructions and the latency of positions and tables bound it, not memory: 8192 tokens of 32 + 2 * 8 heads of 128 in
// bf16 take 45 us (52 without pairs of halves; 60 with a butterfly of single channels and divisions besides), 36 without
// the position rotation; the bytes alone 26.  CTAs per SM: five (48 registers) where that does not spill, 47 us with
// four; the form without pairs spills at 48 (36 us without rotation become 41).  Fewer, longer threads lost: one that
// went over the heads of its token with cosines in registers needed 91 registers and took 60 us; the next row's
// position read one row ahead cost 4 us.
// ---------------------------------------------------------------------------
struct KvAppendParams {
  const uint8_t* in[3];  // q, k, v
  int64_t ld[3];         // bytes between tokens
  int heads[3];
  int64_t T;
  const float *cos_t, *sin_t;
  int64_t rows;          // of the tables
  int rotary, interleaved;
  const int32_t* positions;
  const int64_t* slots;
  const float* kv_amax;
  __nv_bfloat16* q_out;
  uint8_t* cache;
  int64_t n_slots;       // pages * page_size
  int page_units;        // records of a page and head
  int kv_heads;
};

template <bool BF16>
__device__ __forceinline__ void kv_load8(const uint8_t* p, float (&f)[8]) {
  if constexpr (BF16) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  } else {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
}

// The rotation's butterfly over 16 channels of a thread, and (G = 256) over 16 lanes.
template <int G>
__device__ __forceinline__ void kv_rotate(float (&x)[16]) {
  if constexpr (G != 0) {
#pragma unroll
    for (int h = 1; h < 16; h <<= 1)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if ((i & h) == 0) {
          const float a = x[i], b = x[i + h];
          x[i] = __fadd_rn(a, b);
          x[i + h] = __fsub_rn(a, b);
        }
    if constexpr (G == 256) {
      const int lane = threadIdx.x & 31;
#pragma unroll
      for (int m = 1; m < 16; m <<= 1)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float o = __shfl_xor_sync(0xFFFFFFFFu, x[i], m);
          x[i] = (lane & m) ? __fsub_rn(o, x[i]) : __fadd_rn(x[i], o);
        }
    }
    constexpr float c = inv_sqrt_g<G>();
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(x[i], c);
  }
}

// The same for pairs v[i] = (x[i], x[i + 8]): two channels an instruction.  Each sum and product is rounded alike.
template <int G, bool PAIRED>
__device__ __forceinline__ void kv_rotate(float2 (&v)[8]) {
  if constexpr (G != 0) {
#pragma unroll
    for (int h = 1; h < 8; h <<= 1)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if ((i & h) == 0) {
          const float2 a = v[i], b = v[i + h];
          v[i] = add2(a, b);
          v[i + h] = sub2(a, b);
        }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = make_float2(__fadd_rn(v[i].x, v[i].y), __fsub_rn(v[i].x, v[i].y));
    if constexpr (G == 256) {
      const int lane = threadIdx.x & 31;
#pragma unroll
      for (int k = 1; k < 16; k <<= 1) {  // blocks k apart; the lanes that hold them
        const int m = !PAIRED ? k : k < 8 ? 2 * k : 1;
        const float sign = (lane & m) ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 o = make_float2(__shfl_xor_sync(0xFFFFFFFFu, v[i].x, m), __shfl_xor_sync(0xFFFFFFFFu, v[i].y, m));
          v[i] = fma2(v[i], make_float2(sign, sign), o);  // (exact product)
        }
      }
    }
    constexpr float c = inv_sqrt_g<G>();
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = mul2(v[i], make_float2(c, c));
  }
}

// The record that holds slot `slot`, and the token's place in it.
template <int D>
__device__ __forceinline__ int64_t kv_record(int64_t slot, int head, int kv_heads, int page_units, int& at) {
  const int64_t unit = slot / kKvUnit, page = unit < INT_MAX ? static_cast<int>(unit) / page_units : unit / page_units;
  at = static_cast<int>(slot % kKvUnit);
  return ((page * kv_heads + head) * page_units + (unit - page * page_units)) * KvRecord<D>::kBytes;
}

template <int D, int G, bool BF16, bool PAIRED>
__global__ void __launch_bounds__(256, !BF16 ? 3 : PAIRED ? 5 : 4) k_kv_append(const __grid_constant__ KvAppendParams p) {
  using R = KvRecord<D>;
  constexpr int kBlocks = D / 16, es = BF16 ? 2 : 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t heads = p.heads[0] + 2 * p.kv_heads, rows = static_cast<uint32_t>(p.T) * heads;  // (below 2^31)
  const int at_b = threadIdx.x % kBlocks, b = PAIRED ? at_b / 2 + at_b % 2 * (kBlocks / 2) : at_b;  // the thread's block of 16 channels
  const float r6 = __frcp_rn(6.0f);
  const float sg[2] = {kv_global_scale(__ldg(p.kv_amax)), kv_global_scale(__ldg(p.kv_amax + 1))};
  // (every lane of a warp goes on while one does: the lanes exchange values)
  for (uint32_t r0 = blockIdx.x * (256 / kBlocks); r0 < rows; r0 += gridDim.x * (256 / kBlocks)) {
    const uint32_t r = r0 + threadIdx.x / kBlocks;
    const bool live = r < rows;
    const uint32_t t32 = live ? r / heads : 0;
    const int64_t t = t32;
    int head = live ? static_cast<int>(r - t32 * heads) : 0, which = 0;
    if (head >= p.heads[0]) {
      head -= p.heads[0];
      which = head < p.kv_heads ? 1 : 2;
      head -= (which - 1) * p.kv_heads;
    }
    const int64_t slot = which ? __ldg(p.slots + t) : 0;
    const bool store = live && slot >= 0 && (which == 0 || slot < p.n_slots);
    const uint8_t* const src = p.in[which] + t * p.ld[which] + static_cast<int64_t>(head) * (D * es);
    float2 x[8];  // channels k and k + 8
    if constexpr (PAIRED) {  // 8 channels of either half turned together; then neighbours swap, for 16 in one piece each
      float lo[8], hi[8];
      kv_load8<BF16>(src + 8 * at_b * es, lo);
      kv_load8<BF16>(src + (D / 2 + 8 * at_b) * es, hi);
      if (which < 2) {
        int64_t pos = __ldg(p.positions + t);
        pos = pos < 0 ? 0 : pos >= p.rows ? p.rows - 1 : pos;
        float c[8], s[8];
        kv_load8<false>(reinterpret_cast<const uint8_t*>(p.cos_t + pos * (D / 2) + 8 * at_b), c);
        kv_load8<false>(reinterpret_cast<const uint8_t*>(p.sin_t + pos * (D / 2) + 8 * at_b), s);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x1 = lo[i], x2 = hi[i];
          lo[i] = __fsub_rn(__fmul_rn(x1, c[i]), __fmul_rn(x2, s[i]));
          hi[i] = __fadd_rn(__fmul_rn(x2, c[i]), __fmul_rn(x1, s[i]));
        }
      }
      const bool odd = at_b & 1;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? lo[i] : hi[i], 1);
        x[i] = odd ? make_float2(got, hi[i]) : make_float2(lo[i], got);
      }
    } else {
      float lo[8], hi[8];
      kv_load8<BF16>(src + 16 * b * es, lo);
      kv_load8<BF16>(src + (16 * b + 8) * es, hi);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = make_float2(lo[i], hi[i]);
    }
    if (!PAIRED && which < 2 && 16 * b < p.rotary) {
      int64_t pos = __ldg(p.positions + t);
      pos = pos < 0 ? 0 : pos >= p.rows ? p.rows - 1 : pos;
      const int half = p.rotary / 2;
      const float *ct = p.cos_t + pos * half, *st = p.sin_t + pos * half;
      if (p.interleaved) {
        float c[8], s[8];
        kv_load8<false>(reinterpret_cast<const uint8_t*>(ct + 8 * b), c);
        kv_load8<false>(reinterpret_cast<const uint8_t*>(st + 8 * b), s);
#pragma unroll
        for (int k = 0; k < 8; ++k) {  // pair k: channels 2 k and 2 k + 1
          float& x1 = k < 4 ? x[2 * k].x : x[2 * k - 8].y;
          float& x2 = k < 4 ? x[2 * k + 1].x : x[2 * k - 7].y;
          const float a = x1, o = x2;
          x1 = __fsub_rn(__fmul_rn(a, c[k]), __fmul_rn(o, s[k]));
          x2 = __fadd_rn(__fmul_rn(o, c[k]), __fmul_rn(a, s[k]));
        }
      } else {
#pragma unroll
        for (int q = 0; q < 2; ++q) {  // 8 channels: in the first half of the pairs, in the second, or behind them
          const int c0 = 16 * b + 8 * q;
          if (c0 < p.rotary) {
            const bool second = c0 >= half;
            const int at = second ? c0 - half : c0;
            float c[8], s[8], o[8];
            kv_load8<false>(reinterpret_cast<const uint8_t*>(ct + at), c);
            kv_load8<false>(reinterpret_cast<const uint8_t*>(st + at), s);
            kv_load8<BF16>(src + (second ? at : c0 + half) * es, o);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float& mine = q ? x[i].y : x[i].x;
              // (a - b is a + -b, and -(o s) is o (-s), rounded alike)
              mine = __fadd_rn(__fmul_rn(mine, c[i]), __fmul_rn(o[i], second ? s[i] : -s[i]));
            }
          }
        }
      }
    }
    kv_rotate<G, PAIRED>(x);
    if (!store) continue;
    if (which == 0) {
      uint32_t w[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(x[2 * k].x, x[2 * k + 1].x), hi = __floats2bfloat162_rn(x[2 * k].y, x[2 * k + 1].y);
        w[k] = *reinterpret_cast<const uint32_t*>(&lo);
        w[4 + k] = *reinterpret_cast<const uint32_t*>(&hi);
      }
      uint4* const dst = reinterpret_cast<uint4*>(p.q_out + ((t * p.heads[0] + head) * D + 16 * b));
      dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
      dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
      continue;
    }
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max3_nan(top, fabsf(x[k].x), fabsf(x[k].y));
    // Block scale and codes: correctly rounded quotients, by the quantizer's corrected products where its conditions hold
    // (top and both scales far from the ends of fp32's range), else divided.
    const float g = sg[which - 1];
    const bool fast = top <= 0x1p60f && g >= 0x1p-60f && g <= 0x1p60f;
    const float v = fast ? div_markstein(div_markstein(top, 6.0f, r6), g, __frcp_rn(g)) : __fdiv_rn(__fdiv_rn(top, 6.0f), g);
    const uint32_t sb = e4m3x2(v, 0.0f) & 0xFFu;
    const float sf = __fmul_rn(e4m3x2_to_f32(sb).x, g);
    uint2 codes = make_uint2(0, 0);
    if (sf != 0.0f) {
      float2 n[8];
      uint32_t flip = 0;
      if (fast) {  // -q, with the sign of zero; the codes' signs are turned back
        const float nr = -__frcp_rn(sf);
        flip = 0x88888888u;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 q0 = mul2(x[k], make_float2(nr, nr));
          n[k] = fma2(fma2(q0, make_float2(sf, sf), x[k]), make_float2(nr, nr), q0);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) n[k] = make_float2(__fdiv_rn(x[k].x, sf), __fdiv_rn(x[k].y, sf));
      }
      codes = make_uint2(e2m1x8(n[0].x, n[1].x, n[2].x, n[3].x, n[4].x, n[5].x, n[6].x, n[7].x) ^ flip,
                         e2m1x8(n[0].y, n[1].y, n[2].y, n[3].y, n[4].y, n[5].y, n[6].y, n[7].y) ^ flip);
    }
    int at;
    uint8_t* const rec = p.cache + kv_record<D>(slot, head, p.kv_heads, p.page_units, at);
    *reinterpret_cast<uint2*>(rec + (which == 1 ? 0 : R::kV) + at * (D / 2) + 8 * b) = codes;
    rec[(which == 1 ? R::kKs : R::kVs) + at * kBlocks + b] = static_cast<uint8_t>(sb);
  }
}

// ---------------------------------------------------------------------------
// Reading back: the values of the tokens at `slots`, zeros where a slot is none.
// ---------------------------------------------------------------------------
struct KvReadParams {
  const uint8_t* cache;
  const int64_t* slots;
  const float* kv_amax;
  int64_t T, n_slots;
  int page_units, kv_heads;
  void *k, *v;  // [T, kv_heads, D]
};

template <int D, int G, bool BF16>
__global__ void __launch_bounds__(256) k_kv_read(const __grid_constant__ KvReadParams p) {
  using R = KvRecord<D>;
  constexpr int kBlocks = D / 16;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t rows = static_cast<uint32_t>(p.T) * p.kv_heads;
  const int b = threadIdx.x % kBlocks;
  const float sg[2] = {kv_global_scale(__ldg(p.kv_amax)), kv_global_scale(__ldg(p.kv_amax + 1))};
  for (uint32_t r0 = blockIdx.x * (256 / kBlocks); r0 < rows; r0 += gridDim.x * (256 / kBlocks)) {
    const uint32_t r = r0 + threadIdx.x / kBlocks;
    const bool live = r < rows;
    const uint32_t t = live ? r / p.kv_heads : 0;
    const int head = live ? static_cast<int>(r - t * p.kv_heads) : 0;
    const int64_t slot = __ldg(p.slots + t);
    const bool there = slot >= 0 && slot < p.n_slots;
    int at;
    const uint8_t* const rec = p.cache + kv_record<D>(there ? slot : 0, head, p.kv_heads, p.page_units, at);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float x[16];
      uint2 w = make_uint2(0, 0);
      uint32_t sb = 0;
      if (there) {
        w = *reinterpret_cast<const uint2*>(rec + (which ? R::kV : 0) + at * (D / 2) + 8 * b);
        sb = rec[(which ? R::kVs : R::kKs) + at * kBlocks + b];
      }
      const float sf = __fmul_rn(e4m3x2_to_f32(sb).x, sg[which]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 c = e2m1x2_to_f32((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
        x[2 * i] = __fmul_rn(c.x, sf);
        x[2 * i + 1] = __fmul_rn(c.y, sf);
      }
      kv_rotate<G>(x);
      if (!live) continue;
      void* const dst = which ? p.v : p.k;
      const int64_t to = static_cast<int64_t>(r) * D + 16 * b;
      if constexpr (BF16) {
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
          o[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        uint4* const d = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(dst) + to);
        d[0] = make_uint4(o[0], o[1], o[2], o[3]);
        d[1] = make_uint4(o[4], o[5], o[6], o[7]);
      } else {
        float4* const d = reinterpret_cast<float4*>(static_cast<float*>(dst) + to);
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
      }
    }
  }
}

}  // namespace hq
