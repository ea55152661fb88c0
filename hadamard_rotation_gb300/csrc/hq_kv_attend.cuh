// hq_kv_attend.cuh -- attention of few queries per sequence over the paged NVFP4 cache (decoding, drafts).
//
//   o = sum_t p_t V_t / sum_t p_t,   p_t = 2^(scale log2(e) q . K_t - m),   m a running reference per row.
//
// One pass over the records.  The rows of a product's N side are the queries that share a key head: up to 8 (or 16)
// of (query token, head of the group); its M side are the 16 tokens of a record.  So
//   S^T [16 tokens, rows] = K [16, D] Q^T,   O^T [D, rows] += V^T [D, 16] P^T
// and a group of up to 8 heads wastes nothing.  The products are mma.sync: a step of 16 tokens has 16 products for
// 2304 bytes (D = 128), far below what the tensor cores of either kind can do; what it costs are the instructions
// that widen the codes.  Those are exact in f16: a code has 2 significant bits, an E4M3 scale 4, their product lies
// in [2^-10, 2688].  The per-tensor scales are applied in fp32.  q is scaled by a power of two per row (to below
// 2^9), so its 8 bits are exact too, and scores are rounded only by the fp32 sums.
//
// p is carried in f16 (2^-11 of each p; sums of p and of p V in fp32).  The reference m moves only when a score
// exceeds it by 2^8, which saves the maximum across lanes at each step; p is scaled by 2^7, so p stays below 2^15
// (where a step of fp32 at the score is 8, m - 7 is m - 8, and without the scores at 2^8 itself p would be 2^16) and what is
// flushed is below 2^-31 of the reference's.
//
// Channels and tokens are permuted within a record so that every thread reads whole words: thread (g, c) = (lane / 4,
// lane % 4) takes channels [D c / 4, D (c + 1) / 4) of two tokens of K, and [D g / 8, D (g + 1) / 8) of four tokens of
// V, whose nibbles it pairs by token before they are widened.  Sums do not mind the order.
//
// The work of all sequences, heads and rows is laid end to end in records and cut into equal parts, one per CTA; an
// item (sequence, rows, head) that a cut goes through is finished by k_kv_combine from parts in the workspace, in the
// order of the parts.  Lengths are read on the device.  In a CTA a producer warp copies records into a ring
// (cp.async.bulk, one per record), and the other warps take them in turn.
#pragma once

#include <float.h>
#include <limits.h>

#include <type_traits>

#include "hq_kv.cuh"

namespace hq {

struct KvAttendParams {
  const __nv_bfloat16* q;
  int64_t ld_q;  // elements between tokens
  const uint8_t* cache;
  int64_t pages;
  int page_units;
  const int32_t* table;
  int64_t ld_table;
  int most;  // tokens that a row of the table can name
  const int32_t *kv_len, *q_start;
  int S, T, heads, kv_heads, share;  // share: query heads per key head
  const float* kv_amax;
  float scale;
  int window;  // 0: none
  int group;   // of the rotation to undo
  __nv_bfloat16* out;
  float* lse;
  float* part;  // parts of items that were cut: 2 per CTA
};

constexpr int kKvMaxCtas = 160;
constexpr int kKvMinUnits = 60;  // work per CTA at least where items have as many: fewer CTAs rather than emptier ones
// What an item costs beside its records (Q, the joining of the warps' sums), as work of this many before its first.
// (Without, CTAs with many short items ended last: 37 sequences of 12 heads and some 60 records each 42 us, with it 24.)
constexpr int kKvItemUnits = 28;
constexpr float kKvNone = -FLT_MAX;  // the reference before a row's first score, below or equal to any
constexpr float kKvSlack = 8.0f, kKvShift = 7.0f;

template <int D, int NT>
struct KvAttendShape {
  static constexpr int kRows = 8 * NT;
  static constexpr int kWarps = D == 256 ? (NT == 1 ? 11 : 7) : NT == 1 ? 15 : D == 64 ? 15 : 11;  // that multiply
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kUnit = KvRecord<D>::kBytes;
  static constexpr int kPitch = D + 4;  // floats of a row of the warps' sums
  static constexpr int kMergeBytes = kWarps * kRows * kPitch * 4;
  // Places of the ring; each belongs to one warp.  (Else a warp could come to a place whose copy before its own has not
  // landed for another warp, where the parity says that its own has.)
  static constexpr int kFit = (222 * 1024 - kMergeBytes) / kUnit, kSlots = (kFit < 96 ? kFit : 96) / kWarps * kWarps;
  static_assert(kSlots >= 2 * kWarps, "copies ahead of every warp");
  static constexpr int kSmemBytes = kSlots * kUnit + kMergeBytes;
  static constexpr int kPartFloats = kRows * (D + 2);
};

// Bytes of the workspace: parts of items that were cut, 2 per CTA, and a record per CTA of the item it begins and does not
// end, behind the parts of 16 rows.
inline int64_t kv_part_bytes(int D) { return int64_t{2} * kKvMaxCtas * 16 * (D + 2) * 4 + kKvMaxCtas * 32; }

struct KvCut {
  int s, tile, head, last;  // the item; the CTA that has its end (-1: none)
  int pad[4];
};
template <int D>
__device__ __forceinline__ KvCut* kv_cuts(float* part) {
  return reinterpret_cast<KvCut*>(part + static_cast<int64_t>(2) * kKvMaxCtas * 16 * (D + 2));
}

// ---------------------------------------------------------------------------
// The work, as every warp of a launch sees it.
// ---------------------------------------------------------------------------
struct KvSeq {
  int q0, nq, n;  // first query, queries, keys
};

__device__ __forceinline__ KvSeq kv_seq(const KvAttendParams& p, int s) {
  int a = __ldg(p.q_start + s), b = __ldg(p.q_start + s + 1), n = __ldg(p.kv_len + s);
  a = max(0, min(a, p.T));
  b = max(a, min(b, p.T));
  return {a, b - a, max(0, min(n, p.most))};
}

// The same for a whole warp that goes through the sequences in order: 32 are fetched at a time.
struct KvSeqs {
  int base = INT_MIN;
  KvSeq mine;
  __device__ __forceinline__ KvSeq get(const KvAttendParams& p, int s) {
    if (s < base || s >= base + 32) {
      base = s;
      const int lane = threadIdx.x & 31;
      mine = s + lane < p.S ? kv_seq(p, s + lane) : KvSeq{0, 0, 0};
    }
    const int l = s - base;
    return {__shfl_sync(0xFFFFFFFFu, mine.q0, l), __shfl_sync(0xFFFFFFFFu, mine.nq, l), __shfl_sync(0xFFFFFFFFu, mine.n, l)};
  }
};

// Items of a sequence per head; records per item (the same for all of its rows, at least 1 so that every row is
// written) and the first of them.
template <int ROWS>
struct KvSpan {
  int tiles, units, first;
  int64_t cost;  // of an item
  __device__ __forceinline__ KvSpan(const KvAttendParams& p, const KvSeq& s) {
    tiles = (s.nq * p.share + ROWS - 1) / ROWS;
    const int lo = p.window ? max(0, s.n - s.nq - p.window + 1) : 0;
    first = lo / kKvUnit;
    units = max(1, (s.n + kKvUnit - 1) / kKvUnit - first);
    cost = units + kKvItemUnits;
  }
  __device__ __forceinline__ int64_t work(const KvAttendParams& p) const { return tiles * cost * p.kv_heads; }
};

// All work and its items; and the sequence at `at` of it, with the work before that sequence.  For a whole warp.
struct KvTotal {
  int64_t work, items;
};
template <int ROWS>
__device__ __forceinline__ KvTotal kv_total(const KvAttendParams& p) {
  const int lane = threadIdx.x & 31;
  KvTotal t = {0, 0};
  for (int s = lane; s < p.S; s += 32) {
    const KvSpan<ROWS> span(p, kv_seq(p, s));
    t.work += span.work(p);
    t.items += static_cast<int64_t>(span.tiles) * p.kv_heads;
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) {
    t.work += __shfl_xor_sync(0xFFFFFFFFu, t.work, m);
    t.items += __shfl_xor_sync(0xFFFFFFFFu, t.items, m);
  }
  return t;
}

template <int ROWS>
__device__ __forceinline__ int kv_find(const KvAttendParams& p, int64_t at, int64_t& before) {
  const int lane = threadIdx.x & 31;
  before = 0;
  for (int s0 = 0; s0 < p.S; s0 += 32) {
    const int64_t mine = s0 + lane < p.S ? KvSpan<ROWS>(p, kv_seq(p, s0 + lane)).work(p) : 0;
    int64_t sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= d) sum += o;
    }
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, before + sum > at);
    if (past) {
      const int l = __ffs(past) - 1;
      before += __shfl_sync(0xFFFFFFFFu, sum - mine, l);
      return s0 + l;
    }
    before += __shfl_sync(0xFFFFFFFFu, sum, 31);
  }
  return p.S;
}

// The CTA's share [w0, w1) of the work, `per` records each.
struct KvShare {
  int64_t total, per, w0, w1;
};
template <int ROWS>
__device__ __forceinline__ KvShare kv_share(const KvAttendParams& p, int ctas, int cta) {
  KvShare s;
  const KvTotal t = kv_total<ROWS>(p);
  s.total = t.work;
  // As many shares as CTAs, but none much shorter than an item or, where items are long, than kKvMinUnits.
  const int64_t item = t.items ? (t.work + t.items - 1) / t.items : 1, least = item < kKvMinUnits ? item : kKvMinUnits;
  s.per = (s.total + ctas - 1) / ctas;
  if (s.per < least) s.per = least;
  s.w0 = s.per * cta < s.total ? s.per * cta : s.total;
  s.w1 = s.w0 + s.per < s.total ? s.w0 + s.per : s.total;
  return s;
}

// A walk over the segments of a share: an item each, or the part of one that lies in the share.
template <int ROWS>
struct KvWalk {
  const KvAttendParams& p;
  int64_t at, end;   // the next segment's start, the share's end
  int s, tile, head; // the item at `at`
  int64_t item;      // its start
  KvSeqs seqs;
  KvSeq seq;
  KvSpan<ROWS> span;

  // The segment: records [u0, u1) of the sequence (none where u0 >= u1); does it hold the item's first record and
  // its last; what its rows see.
  struct Segment {
    int s, tile, head, u0, u1;
    bool starts, ends;
    KvSeq seq;
    int i0, i1;    // first and last query token of the rows
    int64_t stop;  // the work up to the item's end
  };

  __device__ __forceinline__ KvWalk(const KvAttendParams& p, int64_t w0, int64_t w1)
      : p(p), at(w0), end(w1), s(0), tile(0), head(0), item(0), seq{0, 0, 0}, span(p, seq) {
    if (at >= end) return;
    s = kv_find<ROWS>(p, at, item);
    seq = seqs.get(p, s);
    span = KvSpan<ROWS>(p, seq);
    const int64_t local = (at - item) / span.cost;
    tile = static_cast<int>(local / p.kv_heads);
    head = static_cast<int>(local - static_cast<int64_t>(tile) * p.kv_heads);
    item += local * span.cost;
  }

  __device__ __forceinline__ bool next(Segment& g) {
    if (at >= end) return false;
    const int64_t stop = item + span.cost;
    g.s = s, g.tile = tile, g.head = head, g.seq = seq;
    g.starts = at == item;
    g.ends = stop <= end;
    g.stop = stop;
    const int from = span.first + max(0, static_cast<int>(at - item) - kKvItemUnits);
    const int to = span.first + max(0, static_cast<int>((g.ends ? stop : end) - item) - kKvItemUnits);
    g.i0 = tile * ROWS / p.share;
    g.i1 = min(seq.nq - 1, (tile * ROWS + ROWS - 1) / p.share);
    const int hi = max(0, min(seq.n, seq.n - seq.nq + g.i1 + 1));
    const int lo = p.window ? max(0, seq.n - seq.nq + g.i0 + 1 - p.window) : 0;
    g.u0 = max(from, lo / kKvUnit);
    g.u1 = lo < hi ? min(to, (hi + kKvUnit - 1) / kKvUnit) : 0;
    at = stop;
    item = stop;
    if (at < end && ++head == p.kv_heads) {
      head = 0;
      if (++tile == span.tiles) {
        tile = 0;
        do {
          seq = seqs.get(p, ++s);
          span = KvSpan<ROWS>(p, seq);
        } while (span.tiles == 0 && s < p.S);  // (there is work left, so a sequence with rows)
      }
    }
    return true;
  }
};

// ---------------------------------------------------------------------------
// Widening and products.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void kv_widen(uint32_t w, __half2 (&h)[4]) {
  uint32_t r[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = *reinterpret_cast<const __half2*>(&r[i]);
}
__device__ __forceinline__ __half2 kv_scales(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return *reinterpret_cast<const __half2*>(&r);
}
// A bit for each of four E4M3 scales that is a NaN.
__device__ __forceinline__ uint32_t kv_nan_scales(uint32_t four) { return ((four & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t bits_of(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The power of two that brings a row of largest magnitude `top` to [2^8, 2^9), and its inverse.  (bf16 below 2^-118 and
// above 2^127 keep a factor that is a normal number.)
__device__ __forceinline__ float2 kv_row_factor(float top) {
  const int e = max(9, static_cast<int>((__float_as_uint(top) >> 23) & 255));
  return make_float2(__uint_as_float(static_cast<uint32_t>(262 - e) << 23), __uint_as_float(static_cast<uint32_t>(e - 8) << 23));
}

// The end of a row: eight channels of the sum of p V per thread, D / 8 neighbouring lanes a row.
template <int D>
__device__ __forceinline__ void kv_finish(const KvAttendParams& p, float (&o)[8], float top, float sum, float v_sg, int64_t row,
                                          int head, int e, bool store) {
  const float f = sum > 0.0f || sum != sum ? __fdiv_rn(v_sg, sum) : 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] *= f;
  if (p.group) {
#pragma unroll
    for (int h = 1; h < 8; h <<= 1)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if ((i & h) == 0) {
          const float a = o[i], b = o[i + h];
          o[i] = a + b;
          o[i + h] = a - b;
        }
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      if (8 * m >= p.group) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float other = __shfl_xor_sync(0xFFFFFFFFu, o[i], m);
        o[i] = (lane & m) ? other - o[i] : o[i] + other;
      }
    }
    const float c = p.group == 16 ? 0.25f : 0.0625f;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] *= c;
  }
  if (!store) return;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p.out + (row * p.heads + head) * D + 8 * e) = make_uint4(w[0], w[1], w[2], w[3]);
  if (p.lse && e == 0)
    p.lse[row * p.heads + head] = sum > 0.0f || sum != sum ? (top - kKvShift + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

// Is the phase of `bar` with parity `parity` complete?
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok;
}

template <int D, int NT>
__global__ void __launch_bounds__((KvAttendShape<D, NT>::kThreads), 1) k_kv_attend(const __grid_constant__ KvAttendParams p) {
  using S = KvAttendShape<D, NT>;
  using R = KvRecord<D>;
  constexpr int kRows = S::kRows, kWarps = S::kWarps, kSlots = S::kSlots;
  constexpr int kSteps = D / 16;             // products per record and 8 rows, of either kind
  constexpr int kPiece = D == 64 ? 8 : 16;   // bytes of K that a thread reads together
  constexpr int kWordsK = D / 32, kWordsV = D / 64;
  using Walk = KvWalk<kRows>;
  extern __shared__ __align__(128) uint8_t kv_smem[];
  __shared__ uint64_t full[kSlots], empty[kSlots];
  // Segments, from the producer to the other warps: kept here, not in every warp's registers.
  constexpr int kRing = 8;
  __shared__ uint64_t task_full[kRing], task_empty[kRing], met[2];
  __shared__ typename KvWalk<kRows>::Segment tasks[kRing];
  __shared__ float merge_m[kWarps][kRows], merge_l[kWarps][kRows];
  float* const merge = reinterpret_cast<float*>(kv_smem + kSlots * S::kUnit);
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_addr(&full[i]), 1);
      mbar_init(smem_addr(&empty[i]), 1);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(smem_addr(&task_full[i]), 1);
      mbar_init(smem_addr(&task_empty[i]), kWarps);
    }
    for (int i = 0; i < 2; ++i) mbar_init(smem_addr(&met[i]), kWarps);
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();
  bool ok = true;

  if (warp == kWarps) {  // the producer: lane l copies every 32nd record
    uint32_t k = 0, last = 0;  // records so far, and of a batch that a wait gave up in
    const uint64_t policy = l2_stream_policy();
    const KvShare share = kv_share<kRows>(p, static_cast<int>(gridDim.x), static_cast<int>(blockIdx.x));
    Walk walk(p, share.w0, share.w1);
    // Batches of 32 records.  The pages of the next one are looked up before this one's copies are issued, unless its
    // segment has to wait for a place of the ring: that place may be held by the segment of the batch in hand, which ends only
    // once its records are there, and segments without records take places too.
    enum Next { kNone, kBatch, kLater };
    typename Walk::Segment g;
    int turn = 0, u0 = 0, id = 0;
    bool more = true, told = true;  // there is a segment in `g`; the other warps know of it
    KvCut cut{0, 0, 0, -1, {}};
    g.u0 = g.u1 = 0;
    auto advance = [&](bool wait) {  // to the next batch; kLater: its segment, `g`, would have to wait
      if (told) u0 += 32;
      while (!told || u0 >= g.u1) {
        if (told) {
          more = walk.next(g);
          if (!more) g.s = -1, g.u0 = g.u1 = 0;
          else if (g.starts && !g.ends) cut = KvCut{g.s, g.tile, g.head, static_cast<int>((g.stop - 1) / share.per), {}};
          told = false;
        }
        const uint32_t place = smem_addr(&task_empty[turn % kRing]), parity = turn / kRing & 1 ^ 1;
        if (!wait && !__all_sync(0xFFFFFFFFu, mbar_test(place, parity))) return kLater;
        ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(place, parity));
        if (!ok) return kNone;
        if (lane == 0) {
          tasks[turn % kRing] = g;
          asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(&task_full[turn % kRing])) : "memory");
        }
        ++turn;
        told = true;
        if (!more) return kNone;
        u0 = g.u0;
      }
      if (u0 + lane < g.u1)
        asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(id) : "l"(p.table + g.s * p.ld_table + (u0 + lane) / p.page_units));
      return kBatch;
    };
    for (Next next = kLater; next != kNone;) {
      const int u = u0 + lane, n = next == kBatch ? min(32, g.u1 - u0) : 0, head = g.head, page = id;
      next = advance(n == 0);
      if (n == 0) continue;
      const int64_t at = min(static_cast<int64_t>(max(page, 0)), p.pages - 1);
      const uint8_t* const src = p.cache + ((at * p.kv_heads + head) * p.page_units + u % p.page_units) * R::kBytes;
      const uint32_t slot = (k + lane) % kSlots, pass = (k + lane) / kSlots & 1;
      bool issued = false;
      for (int part = 0; part < 4; ++part) {  // eight at a time: the first are on their way before the last have a slot
        if (lane < n && lane / 8 == part && ok) {
          ok = mbar_wait(smem_addr(&empty[slot]), pass ^ 1);
          if (ok) tma_load(smem_addr(kv_smem) + slot * S::kUnit, src, R::kBytes, smem_addr(&full[slot]), policy);
          issued = ok;
        }
        __syncwarp();
      }
      if (!__all_sync(0xFFFFFFFFu, ok)) {  // a wait gave up: the last copy into each of these places lands (bounded)
        if (issued) mbar_wait(smem_addr(&full[slot]), pass);
        else if (lane < n && lane < kSlots && k + lane >= kSlots) mbar_wait(smem_addr(&full[slot]), pass ^ 1);
        ok = false;
        last = n;
        break;
      }
      k += n;
    }
    if (lane == 0) kv_cuts<D>(p.part)[blockIdx.x] = cut;
    // What else is on its way lands (bounded) before the CTA may end, whoever has given up: the last copies into the other
    // places.
    for (uint32_t i = lane; i + last < kSlots && i < k; i += 32) {
      const uint32_t seq = k - 1 - i;
      const bool landed = mbar_wait(smem_addr(&full[seq % kSlots]), seq / kSlots & 1);
      ok = ok && landed;
    }
  } else {
    const int gq = lane >> 2, c = lane & 3;
    auto token = [](int t) { return t ^ ((t >> 1) & 1); };  // (two rows of V of a phase in other halves of the banks)
    const int t_k = token(gq), t_a = token(2 * c), t_b = token(2 * c + 1);
    const float k_sg = kv_global_scale(__ldg(p.kv_amax)), v_sg = kv_global_scale(__ldg(p.kv_amax + 1));
    const float to_log2 = p.scale * 1.4426950408889634f * k_sg;
    uint32_t k0 = 0;  // records of the segments before
    int slot = warp;  // of this warp's next record, and its pass
    uint32_t pass = 0;
    // Segment `round`; false: there is none.
    const typename Walk::Segment* task = tasks;
    auto find = [&](int round) {
      ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(smem_addr(&task_full[round % kRing]), round / kRing & 1));
      task = tasks + round % kRing;
      return ok && task->s >= 0;
    };
    // All multiplying warps; a wait that runs out for one of them must not leave the others waiting for ever.
    auto meet = [&](int which, int round) {
      __syncwarp();
      if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(&met[which])) : "memory");
      ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(smem_addr(&met[which]), round & 1));
      return ok;
    };
    for (int round = 0; find(round); ++round) {
      const typename Walk::Segment& g = *task;
      // Their fragments.
      uint32_t qf[NT][kSteps][2];
      float mult[NT][2];
      int lo[NT][2], hi[NT][2];
      const int live = g.seq.nq * p.share - g.tile * kRows;  // rows of the tile that exist
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = 8 * nt + gq, at = g.tile * kRows + r;
        const int64_t i = g.seq.q0 + at / p.share;
        const __nv_bfloat16* const src = r < live ? p.q + i * p.ld_q + (static_cast<int64_t>(g.head) * p.share + at % p.share) * D : nullptr;
        uint32_t w[kSteps * 2];
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < kSteps; j += 2) {  // 8 channels, as K's
          constexpr int kPer = kPiece / 2;     // steps of a piece
          const int ch = j / kPer * (8 * kPiece) + c * (2 * kPiece) + (j % kPer) * 4;
          const uint4 v = src ? __ldg(reinterpret_cast<const uint4*>(src + ch)) : make_uint4(0, 0, 0, 0);
          w[2 * j] = v.x, w[2 * j + 1] = v.y, w[2 * j + 2] = v.z, w[2 * j + 3] = v.w;
        }
#pragma unroll
        for (int j = 0; j < 2 * kSteps; ++j)
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xFFFF0000u))));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const float2 f = kv_row_factor(top);
#pragma unroll
        for (int j = 0; j < 2 * kSteps; ++j)
          qf[nt][j / 2][j & 1] = bits_of(__floats2half2_rn(__uint_as_float(w[j] << 16) * f.x, __uint_as_float(w[j] & 0xFFFF0000u) * f.x));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mult[nt][h] = __shfl_sync(0xFFFFFFFFu, f.y, 4 * (2 * c + h)) * to_log2;
          const int row = 8 * nt + 2 * c + h;
          const int end = row < live ? g.seq.n - g.seq.nq + (g.tile * kRows + row) / p.share + 1 : 0;
          hi[nt][h] = end;
          lo[nt][h] = p.window ? end - p.window : 0;
        }
      }
      // What all rows see, and what needs no mask.
      const int first_end = g.seq.n - g.seq.nq + g.i0 + 1, last_start = p.window ? g.seq.n - g.seq.nq + g.i1 + 1 - p.window : 0;
      float o[NT][kSteps][4];
      float m[NT][2], l[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < kSteps; ++j) o[nt][j][0] = o[nt][j][1] = o[nt][j][2] = o[nt][j][3] = 0.0f;
        m[nt][0] = m[nt][1] = kKvNone;
        l[nt][0] = l[nt][1] = 0.0f;
      }
      const int skip = (warp + kWarps - static_cast<int>(k0 % kWarps)) % kWarps;
      // U records at once, kWarps apart: what comes with a step is shared by them, and their chains run side by side.
      auto take = [&](int u, auto count) {
        constexpr int U = decltype(count)::value;
        const uint8_t* rec[U];
        uint32_t done[U];
#pragma unroll
        for (int x = 0; x < U; ++x) {
          ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(smem_addr(&full[slot]), pass));
          rec[x] = kv_smem + slot * S::kUnit;
          done[x] = smem_addr(&empty[slot]);
          if ((slot += kWarps) >= kSlots) {
            slot -= kSlots;
            pass ^= 1;
          }
        }
        if (!ok) return;
        float s[U][NT][4];  // S^T
#pragma unroll
        for (int x = 0; x < U; ++x) {
          uint32_t kw[2][kWordsK];
          uint32_t sb[2][(kWordsK + 1) / 2];  // scale bytes, by two
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint8_t* const row = rec[x] + (t_k + 8 * h) * (D / 2);
            const uint8_t* const sc = rec[x] + R::kKs + (t_k + 8 * h) * (D / 16);
            if constexpr (D == 64) {
              const uint2 v = *reinterpret_cast<const uint2*>(row + 8 * c);
              kw[h][0] = v.x, kw[h][1] = v.y;
              sb[h][0] = sc[c];
            } else {
#pragma unroll
              for (int i = 0; i < kWordsK / 4; ++i) {
                const uint4 v = *reinterpret_cast<const uint4*>(row + 64 * i + 16 * c);
                kw[h][4 * i] = v.x, kw[h][4 * i + 1] = v.y, kw[h][4 * i + 2] = v.z, kw[h][4 * i + 3] = v.w;
                sb[h][i] = *reinterpret_cast<const uint16_t*>(sc + 8 * i + 2 * c);
              }
            }
          }
          float acc[NT][2][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[nt][0][i] = acc[nt][1][i] = 0.0f;
#pragma unroll
          for (int w = 0; w < kWordsK; ++w) {  // 8 channels: two products
            __half2 a[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              kv_widen(kw[h][w], a[h]);
              const __half2 two = kv_scales(sb[h][w / 4]);
              const __half2 sc = (w / 2) & 1 ? __high2half2(two) : __low2half2(two);
#pragma unroll
              for (int i = 0; i < 4; ++i) a[h][i] = __hmul2(a[h][i], sc);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                mma_f16(acc[nt][i], bits_of(a[0][2 * i]), bits_of(a[1][2 * i]), bits_of(a[0][2 * i + 1]), bits_of(a[1][2 * i + 1]),
                        qf[nt][2 * w + i][0], qf[nt][2 * w + i][1]);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[x][nt][i] = (acc[nt][0][i] + acc[nt][1][i]) * mult[nt][i & 1];
        }
        const int key = u * kKvUnit, last = (u + (U - 1) * kWarps) * kKvUnit;
        if (key < last_start || last + kKvUnit > first_end) {
#pragma unroll
          for (int x = 0; x < U; ++x)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int t = key + x * (kWarps * kKvUnit) + t_k + 8 * (i >> 1);
                if (t < lo[nt][i & 1] || t >= hi[nt][i & 1]) s[x][nt][i] = -INFINITY;
              }
        }
        bool above = false;
#pragma unroll
        for (int x = 0; x < U; ++x)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) above |= s[x][nt][i] >= m[nt][i & 1] + kKvSlack;
        if (__any_sync(0xFFFFFFFFu, above)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float top = m[nt][h];
#pragma unroll
              for (int x = 0; x < U; ++x) top = fmaxf(top, fmaxf(s[x][nt][h], s[x][nt][h + 2]));
#pragma unroll
              for (int y = 4; y < 32; y <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, y));
              const float f = exp2_fast(m[nt][h] - top);
              m[nt][h] = top;
              l[nt][h] *= f;
#pragma unroll
              for (int j = 0; j < kSteps; ++j) {
                o[nt][j][h] *= f;
                o[nt][j][h + 2] *= f;
              }
            }
        }
        uint32_t pb[U][NT][2];
#pragma unroll
        for (int x = 0; x < U; ++x)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] = exp2_fast(s[x][nt][i] - (m[nt][i & 1] - kKvShift));
            l[nt][0] += e[0] + e[2];
            l[nt][1] += e[1] + e[3];
            pb[x][nt][0] = transposed8(bits_of(__floats2half2_rn(e[0], e[1])));
            pb[x][nt][1] = transposed8(bits_of(__floats2half2_rn(e[2], e[3])));
          }
#pragma unroll
        for (int x = 0; x < U; ++x) {  // O^T
          uint32_t even[2][kWordsV], odd[2][kWordsV];
          uint32_t sv[2][D == 256 ? 2 : 1];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t wa[kWordsV], wb[kWordsV];
            const uint8_t *const ra = rec[x] + R::kV + (t_a + 8 * h) * (D / 2) + gq * (D / 16), *const rb = ra + (t_b - t_a) * (D / 2);
            if constexpr (kWordsV == 1) {
              wa[0] = *reinterpret_cast<const uint32_t*>(ra);
              wb[0] = *reinterpret_cast<const uint32_t*>(rb);
            } else if constexpr (kWordsV == 2) {
              const uint2 a = *reinterpret_cast<const uint2*>(ra), b = *reinterpret_cast<const uint2*>(rb);
              wa[0] = a.x, wa[1] = a.y, wb[0] = b.x, wb[1] = b.y;
            } else {
              const uint4 a = *reinterpret_cast<const uint4*>(ra), b = *reinterpret_cast<const uint4*>(rb);
              wa[0] = a.x, wa[1] = a.y, wa[2] = a.z, wa[3] = a.w, wb[0] = b.x, wb[1] = b.y, wb[2] = b.z, wb[3] = b.w;
            }
#pragma unroll
            for (int w = 0; w < kWordsV; ++w) {
              even[h][w] = (wa[w] & 0x0F0F0F0Fu) | ((wb[w] & 0x0F0F0F0Fu) << 4);
              odd[h][w] = ((wa[w] >> 4) & 0x0F0F0F0Fu) | (wb[w] & 0xF0F0F0F0u);
            }
            const uint8_t *const va = rec[x] + R::kVs + (t_a + 8 * h) * (D / 16), *const vb = rec[x] + R::kVs + (t_b + 8 * h) * (D / 16);
#pragma unroll
            for (int i = 0; i < (D == 256 ? 2 : 1); ++i) {
              const int block = D == 64 ? gq / 2 : D == 128 ? gq : 2 * gq + i;
              sv[h][i] = va[block] | static_cast<uint32_t>(vb[block]) << 8;
            }
          }
          const int left = g.seq.n - key - x * (kWarps * kKvUnit);
          if (left < kKvUnit) {  // (scales behind the sequence's end may be NaN)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = 0; i < (D == 256 ? 2 : 1); ++i)
                sv[h][i] &= (t_a + 8 * h < left ? 0xFFu : 0u) | (t_b + 8 * h < left ? 0xFF00u : 0u);
          }
          uint32_t nan = 0;
#pragma unroll
          for (int i = 0; i < (D == 256 ? 2 : 1); ++i) nan |= kv_nan_scales(sv[0][i] | sv[1][i] << 16);
          if (__any_sync(0xFFFFFFFFu, nan != 0)) {  // for the rows that see them only: the product would give them to all
#pragma unroll
            for (int i = 0; i < (D == 256 ? 2 : 1); ++i) {
              uint32_t where = 0;  // tokens of the record with a NaN in the thread's channels
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int y = 0; y < 2; ++y)
                  if ((sv[h][i] >> (8 * y) & 0x7Fu) == 0x7Fu) {
                    where |= 1u << ((y ? t_b : t_a) + 8 * h);
                    sv[h][i] &= y ? 0x00FFu : 0xFF00u;
                  }
              where |= __shfl_xor_sync(0xFFFFFFFFu, where, 1);
              where |= __shfl_xor_sync(0xFFFFFFFFu, where, 2);
              const int first = key + x * (kWarps * kKvUnit);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const int a = max(0, lo[nt][h] - first), b = min(kKvUnit, hi[nt][h] - first);
                  if (a < b && (where & ((1u << b) - (1u << a))) != 0)
#pragma unroll
                    for (int j = (D == 256 ? 8 * i : 0); j < (D == 256 ? 8 * i + 8 : kSteps); ++j)
                      o[nt][j][h] = o[nt][j][h + 2] = __int_as_float(0x7FC00000);
                }
            }
          }
          __half2 sc[2][D == 256 ? 2 : 1];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < (D == 256 ? 2 : 1); ++i) sc[h][i] = kv_scales(sv[h][i]);
#pragma unroll
          for (int w = 0; w < kWordsV; ++w) {  // 8 channels per thread: four products
            __half2 a[2][2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              kv_widen(even[h][w], a[h][0]);
              kv_widen(odd[h][w], a[h][1]);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                a[h][0][i] = __hmul2(a[h][0][i], sc[h][D == 256 ? w / 2 : 0]);
                a[h][1][i] = __hmul2(a[h][1][i], sc[h][D == 256 ? w / 2 : 0]);
              }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                mma_f16(o[nt][4 * w + i], bits_of(a[0][0][i]), bits_of(a[0][1][i]), bits_of(a[1][0][i]), bits_of(a[1][1][i]),
                        pb[x][nt][0], pb[x][nt][1]);
          }
        }
        __syncwarp();
        if (lane == 0) {
#pragma unroll
          for (int x = 0; x < U; ++x) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(done[x]) : "memory");
        }
      };
      int u = g.u0 + skip;
      if constexpr (D * NT <= 128)  // (more would not fit the registers)
        for (; ok && u + kWarps < g.u1; u += 2 * kWarps) take(u, std::integral_constant<int, 2>());
      for (; ok && u < g.u1; u += kWarps) take(u, std::integral_constant<int, 1>());
      // The warps' sums, one after another, once those of the segment before have been read.
      if (!meet(0, round)) break;
      float* const mine = merge + warp * kRows * S::kPitch;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float sum = l[nt][h];
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
          const int row = 8 * nt + 2 * c + h;
          if (gq == 0) {
            merge_m[warp][row] = m[nt][h];
            merge_l[warp][row] = sum;
          }
#pragma unroll
          for (int j = 0; j < kSteps; ++j)
            *reinterpret_cast<float2*>(mine + row * S::kPitch + gq * (D / 8) + 2 * j) = make_float2(o[nt][j][h], o[nt][j][h + 2]);
        }
      k0 += max(0, g.u1 - g.u0);
      if (!meet(1, round)) break;
      // Each time by other warps: the rest are in the next segment.
      constexpr int kLanes = D / 8, kParts = kRows * kLanes / 32;  // threads of a row; warps' worth of rows
      for (int part = (warp + kWarps - round * kParts % kWarps) % kWarps; part < kParts; part += kWarps) {
        const int task = part * 32 + lane, row = task / kLanes, e = task % kLanes;
        float top = kKvNone;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, merge_m[w][row]);
        float sum = 0.0f, v[8] = {};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float by = exp2_fast(merge_m[w][row] - top);
          sum += merge_l[w][row] * by;
          const float4* const src = reinterpret_cast<const float4*>(merge + (w * kRows + row) * S::kPitch + 8 * e);
          const float4 a = src[0], b = src[1];
          v[0] += a.x * by, v[1] += a.y * by, v[2] += a.z * by, v[3] += a.w * by;
          v[4] += b.x * by, v[5] += b.y * by, v[6] += b.z * by, v[7] += b.w * by;
        }
        const int at = g.tile * kRows + row;
        if (g.starts && g.ends) {
          kv_finish<D>(p, v, top, sum, v_sg, g.seq.q0 + at / p.share, g.head * p.share + at % p.share, e, at < g.seq.nq * p.share);
        } else {  // (an item that began before is the share's first segment, one that goes on its last)
          float* const to = p.part + (static_cast<int64_t>(blockIdx.x) * 2 + g.starts) * S::kPartFloats;
          float4* const dst = reinterpret_cast<float4*>(to + row * D + 8 * e);
          dst[0] = make_float4(v[0], v[1], v[2], v[3]);
          dst[1] = make_float4(v[4], v[5], v[6], v[7]);
          if (e == 0) {
            to[kRows * D + row] = top;
            to[kRows * D + kRows + row] = sum;
          }
        }
      }
      __syncwarp();
      if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(&task_empty[round % kRing])) : "memory");
    }
  }
  if (!__all_sync(0xFFFFFFFFu, ok) && lane == 0) atomicOr(&g_hq_fault, kFaultWaitTimeout);
}

// Items that were cut: blockIdx.x the CTA that an item begins in, blockIdx.y its row.  The parts are taken by groups of
// threads, all at once: with one thread for all parts of its channels 19 parts took 10 us.
template <int D, int NT>
__global__ void __launch_bounds__(256) k_kv_combine(const __grid_constant__ KvAttendParams p) {
  using S = KvAttendShape<D, NT>;
  constexpr int kRows = S::kRows, kLanes = D / 8, kGroups = 256 / kLanes;
  __shared__ float tops[kGroups], totals[kGroups], sums[kGroups][D + 4];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int cta = static_cast<int>(blockIdx.x), row = static_cast<int>(blockIdx.y);
  const int4 cut = __ldcg(reinterpret_cast<const int4*>(kv_cuts<D>(p.part) + cta));
  const int last = cut.w;
  if (last < 0) return;
  const KvSeq seq = kv_seq(p, cut.x);
  const int at = cut.y * kRows + row, e = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  if (at >= seq.nq * p.share) return;
  float top = kKvNone, sum = 0.0f, v[8] = {};
#pragma unroll 2
  for (int k = cta + group; k <= last; k += kGroups) {
    const float* const from = p.part + (static_cast<int64_t>(k) * 2 + (k == cta)) * S::kPartFloats;
    const float m = __ldcg(from + kRows * D + row), l = __ldcg(from + kRows * D + kRows + row);
    const float4 a = __ldcg(reinterpret_cast<const float4*>(from + row * D + 8 * e)), b = __ldcg(reinterpret_cast<const float4*>(from + row * D + 8 * e) + 1);
    const float both = fmaxf(top, m), f = exp2_fast(top - both), g = exp2_fast(m - both);
    top = both;
    sum = sum * f + l * g;
    v[0] = v[0] * f + a.x * g, v[1] = v[1] * f + a.y * g, v[2] = v[2] * f + a.z * g, v[3] = v[3] * f + a.w * g;
    v[4] = v[4] * f + b.x * g, v[5] = v[5] * f + b.y * g, v[6] = v[6] * f + b.z * g, v[7] = v[7] * f + b.w * g;
  }
  if (e == 0) tops[group] = top, totals[group] = sum;
  *reinterpret_cast<float4*>(&sums[group][8 * e]) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(&sums[group][8 * e + 4]) = make_float4(v[4], v[5], v[6], v[7]);
  __syncthreads();
  if (threadIdx.x >= 32) return;  // (a whole warp for the lanes' exchange)
  top = kKvNone;
#pragma unroll
  for (int k = 0; k < kGroups; ++k) top = fmaxf(top, tops[k]);
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.0f;
#pragma unroll 4
  for (int k = 0; k < kGroups; ++k) {
    const float f = exp2_fast(tops[k] - top);
    sum += totals[k] * f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += sums[k][8 * e + i] * f;
  }
  kv_finish<D>(p, v, top, sum, kv_global_scale(__ldg(p.kv_amax + 1)), seq.q0 + at / p.share, cut.z * p.share + at % p.share, e,
               threadIdx.x < kLanes);
}

}  // namespace hq
