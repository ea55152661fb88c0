// hq_kv_prompt.cuh -- attention of many queries per sequence over the paged NVFP4 cache (prompts, chunks of prompts), on
// the 5th-generation tensor cores.
//
// The mathematics and the number formats are those of hq_kv_attend.cuh: codes widened exactly to f16, q scaled by a power of
// two per row, p in f16 scaled by 2^7 against a reference that moves only when a score exceeds it by 2^8 (and then by a power of two).
//
// A CTA takes 128 rows (query token, head of the group that shares a key head) per tile of the tensor core.  Where there are
// more, and up to D = 128, it takes two such tiles at once (SUB = 2), so that the scores of one are multiplied while the
// other's are exponentiated; with one, the next scores go into columns of their own.  Keys come in tiles of 128 (64 for
// D = 256), widened once for both:
//   S = Q K^T   Q and K in shared memory along the channels, S in tensor memory
//   O += P V    P in tensor memory (two tiles, D = 128: over S's columns), V in shared memory as it comes (the instruction takes it across)
// Roles of a CTA:
//   warp 0        issues the products
//   warp 1        allocates tensor memory
//   warp 2        the segments of the CTA's share, one after another, for the other roles
//   warps 4..11   widen keys (4..7) and values: a token per thread, from global memory through registers (the next
//                 tile's bytes are on their way meanwhile) into the swizzle that the products read
//   warps 12..    softmax, a row per thread, four warps per tile; they also load and scale Q, correct O when a reference
//                 moves, and finish the rows
// Products into different columns need not end in the order of their issue, so what a product writes is never what an
// earlier one may still read; but a commit covers all products before it: with two tiles of rows, when S of a tile is
// complete, so is the O that the correction changes.
//
// The work, in key tiles, is laid end to end (sequence, head, rows) and cut into equal parts, one per CTA; what a cut
// goes through is finished by k_kv_prompt_combine from parts in the workspace, in the order of the parts.
#pragma once

#include "hq_kv_attend.cuh"
#include "hq_tcgen05.cuh"

namespace hq {

template <int D, int SUB>
struct KvPromptShape {
  static constexpr int kSub = SUB;                    // tiles of 128 rows
  static constexpr int kRows = 128 * kSub;
  static constexpr int kKeys = D == 256 ? 64 : 128;   // of a tile
  static constexpr int kQBytes = 128 * D * 2;         // of a tile of rows
  static constexpr int kKvBytes = kKeys * D * 2;      // of a tile of keys or values
  static constexpr int kAtomQ = 128 * 128, kAtomK = kKeys * 128;  // 64 channels
  static constexpr int kQAt = 0, kKAt = kSub * kQBytes, kVAt = kKAt + 2 * kKvBytes;
  static constexpr int kUsed = kVAt + 2 * kKvBytes;
  static constexpr int kSmemBytes = kUsed < 116 * 1024 ? 116 * 1024 : kUsed;  // (a CTA takes all of tensor memory)
  static constexpr int kThreads = 32 * (12 + 4 * kSub);
  // Tensor memory: two of S, O of each tile, two of P; for two tiles and D = 128 there is no room for P but in S's first
  // columns.
  static constexpr bool kOver = D == 128 && kSub == 2;
  static constexpr int kColO = 2 * kKeys, kColP = kOver ? 0 : kColO + kSub * D;
  static constexpr int kStepP = kOver ? kKeys : kKeys / 2;  // columns from one P to the other
  static_assert(kColO + kSub * D <= 512 && kColP + 2 * (kKeys / 2) <= 512, "tensor memory has 512 columns");
  static_assert(kSmemBytes + 1024 + 8192 <= 227 * 1024 && 2 * (kSmemBytes + 1024) > 228 * 1024, "one CTA per SM");
  // Registers of a thread: at the launch, and by role.
  static constexpr int kRegsLaunch = kSub == 1 ? 128 : 96, kRegsControl = kSub == 1 ? 80 : 64, kRegsWiden = kSub == 1 ? 80 : 64;
  static constexpr int kRegsSoftmax = kSub == 1 ? 184 : 144;
  static_assert(128 * kRegsControl + 256 * kRegsWiden + 128 * kSub * kRegsSoftmax <= kThreads * kRegsLaunch, "what the launch has");
  static constexpr int kPerToken = 128 / kKeys;       // threads that widen a token
  static constexpr int kWords = D / 8 / kPerToken;    // words of codes of a thread, and a quarter as many pairs of scales
  static constexpr int kPartFloats = kRows * (D + 2);
};

// Bytes of the workspace: parts of items that were cut, 2 per CTA, and a record per CTA of the item it begins and
// does not end.
inline int64_t kv_prompt_bytes(int D) {
  return int64_t{2} * kKvMaxCtas * (D == 256 ? 128 : 256) * (D + 2) * 4 + kKvMaxCtas * 32;
}

constexpr int64_t kKvMinTiles = 6;  // of work per CTA at least
// What an item costs beside its key tiles (Q, the first scores, the rows' end), as work of this many tiles before its first.
constexpr int kKvItemTiles = 3;

// Key tiles of the rows `tile` of a sequence: [first, first + n) of `keys` keys.
struct KvReach {
  int first, n;
};
template <int ROWS, int KEYS>
__device__ __forceinline__ KvReach kv_reach(const KvAttendParams& p, const KvSeq& s, int tile) {
  const int i0 = tile * ROWS / p.share, i1 = min(s.nq - 1, (tile * ROWS + ROWS - 1) / p.share);
  const int hi = max(0, min(s.n, s.n - s.nq + i1 + 1));
  const int lo = p.window ? max(0, s.n - s.nq + i0 + 1 - p.window) : 0;
  return lo < hi ? KvReach{lo / KEYS, (hi + KEYS - 1) / KEYS - lo / KEYS} : KvReach{0, 0};
}
template <int ROWS>
__device__ __forceinline__ int kv_row_tiles(const KvAttendParams& p, const KvSeq& s) {
  return (s.nq * p.share + ROWS - 1) / ROWS;
}

// Where a CTA's share begins.
struct KvStart {
  int64_t at, end;  // of the work
  int64_t per;
  int s, head, tile;
  int64_t item;     // the work before the item
};

// The plan of a launch, by all threads of a CTA: sums of the sequences by the warps in turn, the start by each thread.
template <int ROWS, int KEYS>
__device__ __forceinline__ KvStart kv_plan(const KvAttendParams& p, int64_t (&sums)[512], int ctas, int cta) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = static_cast<int>(blockDim.x >> 5);
  auto fill = [&](int s0) {  // per head
    for (int s = s0 + warp; s < p.S && s < s0 + 512; s += warps) {
      const KvSeq q = kv_seq(p, s);
      const int tiles = kv_row_tiles<ROWS>(p, q);
      int64_t sum = 0;
      for (int t = lane; t < tiles; t += 32) sum += kv_reach<ROWS, KEYS>(p, q, t).n + kKvItemTiles;
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, m);
      if (lane == 0) sums[s - s0] = sum;
    }
    __syncthreads();
  };
  int64_t total = 0;
  for (int s0 = 0; s0 < p.S; s0 += 512) {
    if (s0) __syncthreads();
    fill(s0);
    int64_t sum = 0;
    for (int s = s0 + lane; s < p.S && s < s0 + 512; s += 32) sum += sums[s - s0];
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, m);
    total += sum * p.kv_heads;
  }
  KvStart r = {};
  int64_t use = (total + kKvMinTiles - 1) / kKvMinTiles;
  use = use < 1 ? 1 : use > ctas ? ctas : use;
  r.per = (total + use - 1) / use;
  r.at = r.per * cta < total ? r.per * cta : total;
  r.end = r.at + r.per < total ? r.at + r.per : total;
  // the sequence
  int64_t before = 0, mine = 0;
  bool found = r.at >= r.end;
  for (int s0 = 0; s0 < p.S; s0 += 512) {  // (to the end in any case: the threads meet in `fill`)
    if (p.S > 512) {
      __syncthreads();
      fill(s0);
    }
    for (int b = s0; b < p.S && b < s0 + 512 && !found; b += 32) {
      const int64_t v = b + lane < p.S && b + lane < s0 + 512 ? sums[b + lane - s0] : 0;
      int64_t sum = v * p.kv_heads;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
        if (lane >= d) sum += o;
      }
      const uint32_t past = __ballot_sync(0xFFFFFFFFu, before + sum > r.at);
      if (past) {
        const int l = __ffs(past) - 1;
        found = true;
        r.s = b + l;
        mine = __shfl_sync(0xFFFFFFFFu, v, l);
        before += __shfl_sync(0xFFFFFFFFu, sum - v * p.kv_heads, l);
      } else {
        before += __shfl_sync(0xFFFFFFFFu, sum, 31);
      }
    }
  }
  if (r.at >= r.end) return r;
  // its head and rows
  r.head = static_cast<int>((r.at - before) / mine);
  r.item = before + r.head * mine;
  const KvSeq q = kv_seq(p, r.s);
  for (int t0 = 0;; t0 += 32) {  // (ends: the rows' work adds up to `mine`)
    const int v = t0 + lane < kv_row_tiles<ROWS>(p, q) ? kv_reach<ROWS, KEYS>(p, q, t0 + lane).n + kKvItemTiles : 0;
    int64_t sum = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= d) sum += o;
    }
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, r.item + sum > r.at);
    if (past) {
      const int l = __ffs(past) - 1;
      r.tile = t0 + l;
      r.item += __shfl_sync(0xFFFFFFFFu, sum - v, l);
      return r;
    }
    r.item += __shfl_sync(0xFFFFFFFFu, sum, 31);
    if (t0 > kv_row_tiles<ROWS>(p, q)) return r;
  }
}

// The segments of a share: an item each, or the part of one that lies in the share.  For a whole warp.
template <int ROWS, int KEYS>
struct KvPromptWalk {
  const KvAttendParams& p;
  int64_t at, end, item;
  int s, head, tile;
  KvSeq seq;
  KvReach reach;

  struct Segment {
    int s, head, tile;
    KvSeq seq;
    int j0, j1;  // key tiles
    bool starts, ends;
    int64_t stop;  // the work up to the item's end
  };

  __device__ __forceinline__ KvPromptWalk(const KvAttendParams& p, const KvStart& b)
      : p(p), at(b.at), end(b.end), item(b.item), s(b.s), head(b.head), tile(b.tile), seq{0, 0, 0}, reach{0, 0} {
    if (at >= end) return;
    seq = kv_seq(p, s);
    reach = kv_reach<ROWS, KEYS>(p, seq, tile);
  }

  __device__ __forceinline__ bool next(Segment& g) {
    if (at >= end) return false;
    const int64_t stop = item + reach.n + kKvItemTiles;
    g.s = s, g.head = head, g.tile = tile, g.seq = seq;
    g.starts = at == item;
    g.ends = stop <= end;
    g.stop = stop;
    g.j0 = reach.first + max(0, static_cast<int>(at - item) - kKvItemTiles);
    g.j1 = reach.first + max(0, static_cast<int>((g.ends ? stop : end) - item) - kKvItemTiles);
    at = item = stop;
    if (at < end) {
      if (++tile == kv_row_tiles<ROWS>(p, seq)) {
        tile = 0;
        if (++head == p.kv_heads) {
          head = 0;
          // The next sequence with rows (there is work left), 32 at a time: the other roles wait for it.
          const int lane = threadIdx.x & 31;
          for (++s; s < p.S; s += 32) {
            const uint32_t rows = __ballot_sync(0xFFFFFFFFu, s + lane < p.S && kv_seq(p, s + lane).nq > 0);
            if (!rows) continue;
            s += __ffs(rows) - 1;
            seq = kv_seq(p, s);
            break;
          }
        }
      }
      reach = kv_reach<ROWS, KEYS>(p, seq, tile);
    }
    return true;
  }
};

// The key tiles that rows [128 sub, 128 sub + 128) of a segment's rows see of it, and what of them needs no mask.
struct KvSub {
  int j0, j1;
  int first_end, last_start;  // keys below the one and from the other on are seen by all rows that exist
  int live;                   // rows that exist
};
template <int ROWS, int KEYS, typename Segment>
__device__ __forceinline__ KvSub kv_sub(const KvAttendParams& p, const Segment& g, int sub) {
  KvSub r;
  const int row0 = g.tile * ROWS + 128 * sub;
  r.live = max(0, min(128, g.seq.nq * p.share - row0));
  const int i0 = row0 / p.share, i1 = (row0 + max(1, r.live) - 1) / p.share, base = g.seq.n - g.seq.nq + 1;
  const int hi = max(0, min(g.seq.n, base + i1)), lo = p.window ? max(0, base + i0 - p.window) : 0;
  r.first_end = base + i0;
  r.last_start = p.window ? base + i1 - p.window : 0;
  r.j0 = r.j1 = g.j0;
  if (r.live > 0 && lo < hi) {
    r.j0 = max(g.j0, lo / KEYS);
    r.j1 = max(r.j0, min(g.j1, (hi + KEYS - 1) / KEYS));
  }
  return r;
}

// A segment as the roles see it, handed to them through a ring in shared memory: worked out once, by a warp of its own,
// instead of in every role's registers and code.
struct KvTask {
  const int32_t* table;  // the sequence's pages; NULL: there are no more segments
  KvSeq seq;
  int head, tile;
  int j0, j1;            // key tiles
  int starts, ends;
  KvSub sub[2];
};
constexpr int kKvTasks = 3;

struct KvPromptBars {
  uint64_t task_full[kKvTasks], task_empty[kKvTasks];
  KvTask tasks[kKvTasks];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
  uint64_t drain;
  uint32_t tmem;
  uint32_t v_nan;  // a NaN among the values that this CTA has widened
};

// Columns of the thread's row, on their way until tmem_load_wait.
__device__ __forceinline__ void tmem_load32(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]),
        "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]),
        "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}

template <int N>
__device__ __forceinline__ void tmem_load_wait(float (&v)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));  // (not used before the wait)
}

// f16 x f16 into fp32; `across`: B has its columns, not the summed axis, along its rows.
__device__ __forceinline__ uint32_t kv_idesc(int n, bool across) {
  return (1u << 4) | (static_cast<uint32_t>(across) << 16) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ void umma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  umma_bf16<false>(d, a, b, idesc, accumulate);  // (the kind is the same, the types are the descriptor's)
}
// Values: rows of 64 channels (128 bytes, swizzled), 8-token groups 1024 bytes apart, the next 64 channels `atom` bytes on.
__device__ __forceinline__ uint64_t desc_across(uint32_t addr, int atom) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (static_cast<uint64_t>(atom >> 4) << 16) | (uint64_t{1024 >> 4} << 32) |
         (uint64_t{1} << 46) | (uint64_t{2} << 61);
}

// Sixteen columns of the thread's row through the rotation's butterfly (not yet divided by 4).
__device__ __forceinline__ void kv_butterfly(uint32_t (&w)[16]) {
  float2 x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = __uint_as_float(w[2 * i]), b = __uint_as_float(w[2 * i + 1]);
    x[i] = make_float2(a + b, a - b);
  }
#pragma unroll
  for (int h = 1; h < 8; h <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((i & h) == 0) {
        const float2 a = x[i], b = x[i + h];
        x[i] = add2(a, b);
        x[i + h] = sub2(a, b);
      }
#pragma unroll
  for (int i = 0; i < 8; ++i) w[2 * i] = __float_as_uint(x[i].x), w[2 * i + 1] = __float_as_uint(x[i].y);
}

// Blocks of 16 channels (a bit each) in which one of the keys [max(k0, begin), min(k1, end)) of a sequence has a NaN for a
// value: of each lane's `begin` and `end`, by a warp; k0 a multiple of 16.  512 keys at a time, a record's scales per lane, and single
// tokens only where a row's keys begin or end: the other roles wait for it, and 2^25 keys are looked through well before they
// give up (0.1 s; a token per lane took 0.8 to 1.4).
template <int D>
__device__ __noinline__ uint32_t kv_nan_blocks(const KvAttendParams& p, const int32_t* table, int head, int k0, int k1, int begin,
                                               int end) {
  using R = KvRecord<D>;
  constexpr int kWords = D / 64;  // of a token's scales
  const int lane = threadIdx.x & 31;
  begin = max(begin, k0);
  end = min(end, k1);
  uint32_t mine = 0;
  for (int base = k0; base < k1; base += 32 * kKvUnit) {
    const int unit = base / kKvUnit + lane;
    const uint8_t* scales = nullptr;
    uint32_t w[kWords] = {};  // the top bit of a block's byte: a NaN of any of the record's tokens
    if (unit * kKvUnit < k1) {
      const int at = unit / p.page_units;
      const int64_t page = min(static_cast<int64_t>(max(__ldg(table + at), 0)), p.pages - 1);
      scales = p.cache + ((page * p.kv_heads + head) * p.page_units + (unit - at * p.page_units)) * R::kBytes + R::kVs;
#pragma unroll
      for (int i = 0; i < R::kScales / 16; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(scales) + i);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c % kWords] |= kv_nan_scales(u[c]);
      }
    }
    auto blocks = [](const uint32_t (&w)[kWords]) {
      uint32_t bits = 0;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) bits |= (w[i / 4] >> (8 * (i % 4) + 7) & 1u) << i;
      return bits;
    };
    const uint32_t bad = blocks(w), all = __reduce_or_sync(0xFFFFFFFFu, bad);
    if (all == 0) continue;
    const bool whole = base >= begin && base + 32 * kKvUnit <= end;
    if (whole) mine |= all;
    if (!__any_sync(0xFFFFFFFFu, !whole && base < end && base + 32 * kKvUnit > begin)) continue;
    for (uint32_t records = __ballot_sync(0xFFFFFFFFu, bad != 0); records; records &= records - 1) {
      const int r = __ffs(records) - 1;
      const uint8_t* const from = reinterpret_cast<const uint8_t*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<uint64_t>(scales), r));
      uint32_t one[kWords] = {};
      if (lane < kKvUnit)
#pragma unroll
        for (int i = 0; i < kWords; ++i) one[i] = kv_nan_scales(__ldg(reinterpret_cast<const uint32_t*>(from) + lane * kWords + i));
      const uint32_t token = blocks(one);
      for (uint32_t left = __ballot_sync(0xFFFFFFFFu, token != 0); left; left &= left - 1) {
        const int t = __ffs(left) - 1, key = base + r * kKvUnit + t;
        const uint32_t of = __shfl_sync(0xFFFFFFFFu, token, t);
        if (key >= begin && key < end) mine |= of;
      }
    }
  }
  return mine;
}

template <int D, int SUB>
__global__ void __launch_bounds__((KvPromptShape<D, SUB>::kThreads), 1) k_kv_prompt(const __grid_constant__ KvAttendParams p) {
  using S = KvPromptShape<D, SUB>;
  using R = KvRecord<D>;
  constexpr int kSub = S::kSub, kRows = S::kRows, kKeys = S::kKeys;
  using Walk = KvPromptWalk<kRows, kKeys>;
  using Segment = typename Walk::Segment;
  extern __shared__ uint8_t kv_prompt_raw[];
  __shared__ KvPromptBars bars;
  __shared__ int64_t sums[512];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(kv_prompt_raw) + 1023) & ~uintptr_t{1023});
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&bars.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&bars.k_full[i]), 4);
      mbar_init(smem_addr(&bars.k_empty[i]), 1);
      mbar_init(smem_addr(&bars.v_full[i]), 4);
      mbar_init(smem_addr(&bars.v_empty[i]), 1);
      mbar_init(smem_addr(&bars.q_full[i]), 4);
      mbar_init(smem_addr(&bars.s_full[i]), 1);
      mbar_init(smem_addr(&bars.p_full[i]), 4);
      mbar_init(smem_addr(&bars.o_full[i]), 1);
    }
    for (int i = 0; i < kKvTasks; ++i) {
      mbar_init(smem_addr(&bars.task_full[i]), 1);
      mbar_init(smem_addr(&bars.task_empty[i]), 9 + 4 * kSub);  // (the warps of the roles)
    }
    mbar_init(smem_addr(&bars.drain), 1);
    bars.v_nan = 0;
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // (by the warp that has taken tensor memory: the kernel after this one may take some before it waits for this one)
  if (warp == 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  umma_fence_before();
  __syncthreads();
  umma_fence_after();
  const uint32_t tmem = bars.tmem;
  const KvStart start = kv_plan<kRows, kKeys>(p, sums, static_cast<int>(gridDim.x), static_cast<int>(blockIdx.x));
  GemmRing turn;  // of the tasks
  bool ok = true;
  // The next segment, for a warp of a role; it is copied, and its place free, before the role goes on.
  auto next = [&](KvTask& g) {
    ok = ok && warp_wait(smem_addr(&bars.task_full[turn.s]), turn.phase);
    if (!ok) return false;
    g = bars.tasks[turn.s];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&bars.task_empty[turn.s]));
    turn.next(kKvTasks);
    return g.table != nullptr;
  };

  // Registers where they are used: a thread of the softmax holds half a row of a key tile.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kRegsControl));
  if (warp == 0) {
    GemmRing kv;  // the place of key tile j + 1's keys; values follow one tile behind
    uint32_t q_phase = 0, p_phase = 0, o_phase = 0;  // a bit per barrier (rows that see nothing of a segment take no part in it)
    const uint64_t q_desc = desc_codes(smem_addr(smem)), k_desc = desc_codes(smem_addr(smem) + S::kKAt);
    const uint64_t v_desc = desc_across(smem_addr(smem) + S::kVAt, S::kAtomK);
    KvTask g;
    while (ok && next(g)) {
      GemmRing vr = kv;
      // S = Q K^T; `over`: into columns whose P the last product into O may still read.  (In two halves, of which only the
      // one over P waits, the products of 64 columns take as long as those of 128: 778 us for four prompts at a time when one piece took 682.)
      auto scores = [&](int t, int buffer, bool over) {
        if (S::kOver && over) {
          ok = warp_wait(smem_addr(&bars.o_full[t]), o_phase >> t & 1 ^ 1);
          if (!ok) return;
        }
        umma_fence_after();
        const uint64_t q = q_desc + t * (S::kQBytes >> 4), k = k_desc + kv.s * (S::kKvBytes >> 4);
        if (elect_one()) {
#pragma unroll 1
          for (int i = 0; i < D / 64; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              umma_f16_ss(tmem + buffer * kKeys, q + i * (S::kAtomQ >> 4) + 2 * c, k + i * (S::kAtomK >> 4) + 2 * c,
                          kv_idesc(kKeys, false), i > 0 || c > 0);
          umma_commit<false>(smem_addr(&bars.s_full[buffer]));
        }
        __syncwarp();
      };
      auto values = [&](int t, int buffer, bool more) {  // O += P V
        umma_fence_after();
        const uint64_t v = v_desc + vr.s * (S::kKvBytes >> 4);
        if (elect_one()) {
#pragma unroll 4
          for (int i = 0; i < kKeys / 16; ++i)
            umma_f16_ts<false>(tmem + S::kColO + t * D, tmem + S::kColP + buffer * S::kStepP + 8 * i, v + i * (2048 >> 4),
                               kv_idesc(D, true), more || i > 0);
          umma_commit<false>(smem_addr(&bars.o_full[t]));
        }
        __syncwarp();
        o_phase ^= 1u << t;
      };
      auto wait_bit = [&](uint64_t* bar, int t, uint32_t& phases) {
        ok = ok && warp_wait(smem_addr(bar + t), phases >> t & 1);
        phases ^= 1u << t;
        return ok;
      };
      if constexpr (kSub == 1) {
        // One tile of rows: two of S in turn, so the next scores are multiplied while these are exponentiated.
        for (int j = g.j0 - 1; ok && j < g.j1; ++j) {
          if (j + 1 < g.j1) {
            if (j < g.j0 && !wait_bit(bars.q_full, 0, q_phase)) break;
            ok = warp_wait(smem_addr(&bars.k_full[kv.s]), kv.phase);
            if (!ok) break;
            scores(0, (j + 1) & 1, false);
            if (elect_one()) umma_commit<false>(smem_addr(&bars.k_empty[kv.s]));
            __syncwarp();
            kv.next(2);
          }
          if (j >= g.j0) {
            ok = warp_wait(smem_addr(&bars.v_full[vr.s]), vr.phase);
            if (!wait_bit(bars.p_full, j & 1, p_phase)) break;
            values(0, j & 1, j > g.j0);
            if (elect_one()) umma_commit<false>(smem_addr(&bars.v_empty[vr.s]));
            __syncwarp();
            vr.next(2);
          }
        }
      } else {
        for (int j = g.j0 - 1; ok && j < g.j1; ++j) {
          if (j >= g.j0) ok = warp_wait(smem_addr(&bars.v_full[vr.s]), vr.phase);
          if (j + 1 < g.j1) ok = ok && warp_wait(smem_addr(&bars.k_full[kv.s]), kv.phase);
#pragma unroll 1  // (short code: the roles share the instruction cache)
          for (int t = 0; t < kSub && ok; ++t) {
            const int t0 = t ? g.sub[1].j0 : g.sub[0].j0, t1 = t ? g.sub[1].j1 : g.sub[0].j1;
            if (j >= t0 && j < t1) {
              if (!wait_bit(bars.p_full, t, p_phase)) break;
              values(t, t, j > t0);
            }
            if (j + 1 >= t0 && j + 1 < t1) {
              if (j + 1 == t0 && !wait_bit(bars.q_full, t, q_phase)) break;
              scores(t, t, j >= t0);
              if (!ok) break;
            }
          }
          if (!ok) break;
          if (elect_one()) {
            if (j >= g.j0) umma_commit<false>(smem_addr(&bars.v_empty[vr.s]));
            if (j + 1 < g.j1) umma_commit<false>(smem_addr(&bars.k_empty[kv.s]));
          }
          __syncwarp();
          if (j >= g.j0) vr.next(2);
          if (j + 1 < g.j1) kv.next(2);
        }
      }
    }
    if (!ok) {  // let the products in flight finish (bounded) before tensor memory is freed
      if (elect_one()) umma_commit<false>(smem_addr(&bars.drain));
      __syncwarp();
      mbar_wait(smem_addr(&bars.drain), 0);
    }
  } else if (warp == 2) {  // the segments; and of the items that this CTA begins the one that it does not end
    Walk walk(p, start);
    Segment g;
    KvCut cut{0, 0, 0, -1, {}};
    for (bool more = true; more;) {
      more = walk.next(g);
      if (more && g.starts && !g.ends) cut = KvCut{g.s, g.tile, g.head, static_cast<int>((g.stop - 1) / start.per), {}};
      ok = warp_wait(smem_addr(&bars.task_empty[turn.s]), turn.phase ^ 1);
      if (!ok) break;
      KvTask& to = bars.tasks[turn.s];
      if (lane == 0) {
        to.table = more ? p.table + g.s * p.ld_table : nullptr;
        if (more) {
          to.seq = g.seq;
          to.head = g.head, to.tile = g.tile;
          to.j0 = g.j0, to.j1 = g.j1;
          to.starts = g.starts, to.ends = g.ends;
        }
      } else if (more && lane <= kSub) {
        to.sub[lane - 1] = kv_sub<kRows, kKeys>(p, g, lane - 1);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&bars.task_full[turn.s]));
      turn.next(kKvTasks);
      if (more && g.j0 < g.j1)  // its rows of Q into the L2: they are read once, with nothing else to do
        for (int r = g.tile * kRows + lane; r < min((g.tile + 1) * kRows, g.seq.nq * p.share); r += 32) {
          const __nv_bfloat16* const row = p.q + (g.seq.q0 + r / p.share) * p.ld_q + (static_cast<int64_t>(g.head) * p.share + r % p.share) * D;
#pragma unroll
          for (int c = 0; c < D; c += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + c));
        }
    }
    KvCut* const cuts = reinterpret_cast<KvCut*>(p.part + static_cast<int64_t>(2) * kKvMaxCtas * S::kPartFloats);
    if (lane == 0) cuts[blockIdx.x] = cut;
  }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kRegsWiden));
    constexpr int kWords = S::kWords;
    const int which = warp >= 8;  // K or V
    const int tid = threadIdx.x & 127, t = tid % kKeys, half = tid / kKeys;  // (half of the channels, for D = 256)
    uint64_t *const full = which ? bars.v_full : bars.k_full, *const empty = which ? bars.v_empty : bars.k_empty;
    uint8_t* const tiles = smem + (which ? S::kVAt : S::kKAt);
    GemmRing ring;
    KvTask g = {};
    // (The loads are volatile so that they stay a tile ahead of what waits for them.)
    struct Place {
      int page;  // of the table's row
      int unit;  // record in the page
      int id;    // the page, as the table has it
      bool live; // nothing past the sequence's end is read
    };
    auto look = [&](Place& at, int j) {  // the token of key tile j
      const int key = j * kKeys + t;
      at.live = j < g.j1 && key < g.seq.n;
      if (at.live) asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(at.id) : "l"(g.table + at.page));
    };
    auto step = [&](Place& at) {
      at.unit += kKeys / kKvUnit;
      while (at.unit >= p.page_units) at.unit -= p.page_units, ++at.page;
    };
    auto load16 = [](uint32_t* to, const uint8_t* from) {
      asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(to[0]), "=r"(to[1]), "=r"(to[2]), "=r"(to[3]) : "l"(from));
    };
    // The codes of the thread and their scales (8; 4 for D = 64).
    auto load = [&](const Place& at, uint32_t (&w)[kWords], uint2& scales) {
      scales = make_uint2(0, 0);  // (widened to zeros)
      if (!at.live) return;
      const int64_t page = min(static_cast<int64_t>(max(at.id, 0)), p.pages - 1);
      const uint8_t* const rec = p.cache + ((page * p.kv_heads + g.head) * p.page_units + at.unit) * R::kBytes;
      const uint8_t* const codes = rec + which * R::kV + t % kKvUnit * (D / 2) + half * (4 * kWords);
#pragma unroll
      for (int i = 0; i < kWords; i += 4) load16(w + i, codes + 4 * i);
      const uint8_t* const sc = rec + R::kKs + which * R::kScales + t % kKvUnit * (D / 16) + half * 8;
      if constexpr (D == 64) asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(scales.x) : "l"(sc));
      else asm volatile("ld.global.nc.v2.b32 {%0, %1}, [%2];" : "=r"(scales.x), "=r"(scales.y) : "l"(sc));
    };
    auto widen = [&](uint8_t* to, const uint32_t (&w)[kWords], uint2 scales) {
      // A value's NaN is for the rows that see it only, but the product would give it to all: the rows' end puts it in.
      if (which && (kv_nan_scales(scales.x) | kv_nan_scales(scales.y)) != 0) {
        *const_cast<volatile uint32_t*>(&bars.v_nan) = 1;
        scales.x &= ~((kv_nan_scales(scales.x) >> 7) * 0xFFu);
        scales.y &= ~((kv_nan_scales(scales.y) >> 7) * 0xFFu);
      }
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        __half2 h[4];
        kv_widen(w[i], h);
        const __half2 two = kv_scales((i < 8 ? scales.x : scales.y) >> (16 * ((i / 4) & 1)));
        const __half2 sc = (i / 2) & 1 ? __high2half2(two) : __low2half2(two);
        const uint4 o = make_uint4(bits_of(__hmul2(h[0], sc)), bits_of(__hmul2(h[1], sc)), bits_of(__hmul2(h[2], sc)), bits_of(__hmul2(h[3], sc)));
        const int c = half * kWords + i;  // 8 channels
        *reinterpret_cast<uint4*>(to + (c / 8) * S::kAtomK + t * 128 + (((c % 8) ^ (t & 7)) << 4)) = o;
      }
      fence_proxy_async_smem();
      __syncwarp();
    };
    while (ok && next(g)) {
      if (g.j0 >= g.j1) continue;
      uint32_t codes[kWords] = {};
      uint2 scales;
      Place now, ahead;
      const int unit = (g.j0 * kKeys + t) / kKvUnit;
      now.page = unit / p.page_units;
      now.unit = unit - now.page * p.page_units;
      now.id = ahead.id = 0;
      look(now, g.j0);
      load(now, codes, scales);
      ahead = now;
      step(ahead);
      look(ahead, g.j0 + 1);
      for (int j = g.j0; j < g.j1; ++j) {
        ok = warp_wait(smem_addr(empty + ring.s), ring.phase ^ 1);
        if (!ok) break;
        widen(tiles + ring.s * S::kKvBytes, codes, scales);
        if (lane == 0) mbar_arrive(smem_addr(full + ring.s));
        ring.next(2);
        // The next tile's place has landed with this tile's bytes.  (Used right after newer loads it would wait for those.)
        now = ahead;
        step(ahead);
        look(ahead, j + 2);
        load(now, codes, scales);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kRegsSoftmax));
    const int t = (warp - 12) / 4, quarter = warp & 3, r = quarter * 32 + lane;  // the thread's row of its tile
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t to = tmem + lanes + S::kColO + t * D;
    const float k_sg = kv_global_scale(__ldg(p.kv_amax)), v_sg = kv_global_scale(__ldg(p.kv_amax + 1));
    const float to_log2 = fabsf(p.scale) * 1.4426950408889634f * k_sg;
    uint32_t s_phase = 0, o_phase = 0;
    constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
    // 16 bytes of a row of the warp in the tile's Q; later the same of its output.
    auto piece = [&](int row, int c) {
      return smem + t * S::kQBytes + (c / 8) * S::kAtomQ + (quarter * 32 + row) * 128 + (((c % 8) ^ (row & 7)) << 4);
    };
    KvTask g;
    while (ok && next(g)) {
      const KvSub sub = t ? g.sub[1] : g.sub[0];
      const bool live = r < sub.live;
      const int at = g.tile * kRows + 128 * t + r, i = at / p.share;
      const int64_t token = g.seq.q0 + i;
      const int head = g.head * p.share + (at - i * p.share);
      const bool some = sub.j0 < sub.j1;
      const int end = live ? g.seq.n - g.seq.nq + i + 1 : 0, begin = p.window ? end - p.window : 0;
      // Q: the warp's rows along their channels, kLanes lanes a row.
      float mult = 0.0f;
      if (some) {
        const int64_t mine = token * p.ld_q + static_cast<int64_t>(head) * D;
        const int left = sub.live - quarter * 32;  // of the warp's rows
#pragma unroll 1
        for (int b = 0; b < kLanes; b += 8) {
          uint4 v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int row = (b + k) * kAtOnce + lane / kLanes;
            const int64_t from = __shfl_sync(0xFFFFFFFFu, mine, row);
            v[k] = row < left ? __ldg(reinterpret_cast<const uint4*>(p.q + from) + lane % kLanes) : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int row = (b + k) * kAtOnce + lane / kLanes;
            const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
            float top = 0.0f;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[c] << 16)), fabsf(__uint_as_float(u[c] & 0xFFFF0000u))));
#pragma unroll
            for (int x = 1; x < kLanes; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
            const float2 f = kv_row_factor(top);
            const float back = __shfl_sync(0xFFFFFFFFu, f.y, lane % kAtOnce * kLanes);
            if (lane / kAtOnce == b + k) mult = back;
            const float factor = p.scale < 0.0f ? -f.x : f.x;
            uint32_t o[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
              o[c] = bits_of(__floats2half2_rn(__uint_as_float(u[c] << 16) * factor, __uint_as_float(u[c] & 0xFFFF0000u) * factor));
            *reinterpret_cast<uint4*>(piece(row, lane % kLanes)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        mult *= to_log2;
        // (not 0: a masked score is -inf times it; a NaN is for the rows that see a key)
        if (mult < 1e-37f || end <= 0) mult = 1e-37f;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&bars.q_full[t]));
      }
      // A sum over D channels of q and K as they are multiplied is below 2^29, so with a factor up to 2^-7 scores stay below
      // 2^22, and the reference, which is the rounding of a product, within 2^-3 of it.  Larger ones are rounded themselves first:
      // what the reference's rounding alone left of a score could be more than f16 holds as a power of two.
      const bool large = __any_sync(0xFFFFFFFFu, mult > 0x1p-7f);
      const float by = large ? 1.0f : mult;
      float m = kKvNone, l = 0.0f;
      for (int j = sub.j0; j < sub.j1; ++j) {
        const int buffer = kSub == 1 ? j & 1 : t;
        const uint32_t ts = tmem + lanes + buffer * kKeys, tp = tmem + lanes + S::kColP + buffer * S::kStepP;
        ok = warp_wait(smem_addr(&bars.s_full[buffer]), s_phase >> buffer & 1);
        if (!ok) break;
        s_phase ^= 1u << buffer;
        umma_fence_after();
        const int key = j * kKeys;
        const bool masked = key < sub.last_start || key + kKeys > sub.first_end;
        const int lo = begin - key, hi = end - key;  // columns [lo, hi) are seen
        if (masked) {  // (seldom, so apart from the rest and short)
#pragma unroll 1
          for (int c0 = 0; c0 < kKeys; c0 += 16) {
            uint32_t w[16];
            tmem_load(ts + c0, w);
#pragma unroll
            for (int c = 0; c < 16; ++c) w[c] = c0 + c >= lo && c0 + c < hi ? w[c] : 0xFF800000u;  // -inf
            tmem_store(ts + c0, w);
          }
        }
        if (kSub == 1 && j > sub.j0) {  // (these scores did not wait for the product into O before this tile's)
          ok = warp_wait(smem_addr(&bars.o_full[0]), o_phase ^ 1);
          if (!ok) break;
          umma_fence_after();
        }
        // 64 columns at a time, in one pass: where a score leaves the reference's reach, what has been summed against it is
        // scaled by a power of two, which is exact.
#pragma unroll 1  // (short code: the roles share the instruction cache)
        for (int c0 = 0; c0 < kKeys; c0 += 64) {
          float v[64];
          tmem_load32(ts + c0, v);
          tmem_load32(ts + c0 + 32, v + 32);
          tmem_load_wait(v);
          if (large) {
#pragma unroll
            for (int c = 0; c < 64; ++c) v[c] *= mult;
          }
          float tops[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
          for (int c = 4; c < 64; c += 4)
#pragma unroll
            for (int k = 0; k < 4; ++k) tops[k] = fmaxf(tops[k], v[c + k]);
          float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
          top = top == -INFINITY ? top : top * by;  // (-inf: no score)
          const bool above = top >= m + kKvSlack;
          if (__any_sync(0xFFFFFFFFu, above)) {
            // (from 2^21 on, also at the row's first score, m + ceil(top - m) is not near top)
            const float moved = !above ? m : fmaxf(fabsf(m), fabsf(top)) > 0x1p21f ? top : m + ceilf(top - m);
            const float f = exp2_fast(m - moved);
            m = moved;
            l *= f;
            auto scale = [&](uint32_t at, int columns, auto by) {
#pragma unroll 1
              for (int c = 0; c < columns; c += 16) {
                uint32_t w[16];
                tmem_load(at + c, w);
#pragma unroll
                for (int k = 0; k < 16; ++k) w[k] = by(w[k]);
                tmem_store(at + c, w);
              }
            };
            if (j > sub.j0) scale(to, D, [&](uint32_t w) { return __float_as_uint(__uint_as_float(w) * f); });
            if (c0 > 0) {
              tmem_store_wait();  // (the first columns' weights are there before they are loaded again)
              scale(tp, c0 / 2, [&](uint32_t w) {
                const float2 e = __half22float2(*reinterpret_cast<const __half2*>(&w));
                return bits_of(__floats2half2_rn(e.x * f, e.y * f));
              });
            }
          }
          const float off = kKvShift - m;
          float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t w[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const int at = 32 * half + 2 * c;
              float2 e = fma2(make_float2(v[at], v[at + 1]), make_float2(by, by), make_float2(off, off));
              e = make_float2(exp2_fast(e.x), exp2_fast(e.y));
              sum[c & 1] = add2(sum[c & 1], e);
              w[c] = bits_of(__floats2half2_rn(e.x, e.y));
            }
            tmem_store_nowait(tp + c0 / 2 + 16 * half, w);  // (kOver: over columns of S that have been read)
          }
          l += sum[0].x + sum[0].y + (sum[1].x + sum[1].y);
        }
        tmem_store_wait();
        umma_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&bars.p_full[buffer]));
        o_phase ^= 1;
      }
      if (!ok) break;
      if (some) {
        ok = warp_wait(smem_addr(&bars.o_full[t]), o_phase ^ 1);
        if (!ok) break;
        umma_fence_after();
        if (__any_sync(0xFFFFFFFFu, *const_cast<volatile uint32_t*>(&bars.v_nan) != 0)) {
          const uint32_t bad = kv_nan_blocks<D>(p, g.table, g.head, sub.j0 * kKeys, min(sub.j1 * kKeys, g.seq.n), begin, end);
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            if (!__any_sync(0xFFFFFFFFu, bad >> c & 1)) continue;
            uint32_t w[16];
            tmem_load(to + 16 * c, w);
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = bad >> c & 1 ? 0x7FC00000u : w[k];
            tmem_store(to + 16 * c, w);
          }
        }
      }
      if (g.starts && g.ends) {
        const float f = l > 0.0f || l != l ? __fdiv_rn(v_sg, l) * (p.group == 256 ? 0.0625f : p.group ? 0.25f : 1.0f) : 0.0f;
        if (D == 256 && p.group == 256 && some) {  // the butterfly across the blocks of 16, in place
#pragma unroll 1
          for (int c = 0; c < 16; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 16; ++k)
              asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(w[k]) : "r"(to + (16 * k + c) % D) : "memory");
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
            for (int k = 0; k < 16; ++k) asm volatile("" : "+r"(w[k]));  // (not used before the wait)
            kv_butterfly(w);
#pragma unroll
            for (int k = 0; k < 16; ++k)
              asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(to + (16 * k + c) % D), "r"(w[k]) : "memory");
            tmem_store_wait();
          }
        }
#pragma unroll 2
        for (int c0 = 0; c0 < D; c0 += 16) {
          uint32_t w[16] = {};
          if (some) tmem_load(to + c0, w);
          if (p.group) kv_butterfly(w);
          uint32_t o[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(w[2 * c]) * f, __uint_as_float(w[2 * c + 1]) * f);
            o[c] = l == 0.0f ? 0u : *reinterpret_cast<const uint32_t*>(&h);
          }
          *reinterpret_cast<uint4*>(piece(lane, c0 / 8)) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(piece(lane, c0 / 8 + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
        }
        __syncwarp();
        const int64_t mine = (token * p.heads + head) * D;  // rows leave along their channels
#pragma unroll 4
        for (int b = 0; b < kLanes; ++b) {
          const int row = b * kAtOnce + lane / kLanes;
          const int64_t to_row = __shfl_sync(0xFFFFFFFFu, mine, row);
          if (row < sub.live - quarter * 32)
            reinterpret_cast<uint4*>(p.out + to_row)[lane % kLanes] = *reinterpret_cast<const uint4*>(piece(row, lane % kLanes));
        }
        __syncwarp();
        if (p.lse && live)
          p.lse[token * p.heads + head] = l > 0.0f || l != l ? (m - kKvShift + log2f(l)) * 0.6931471805599453f : -INFINITY;
      } else {  // (an item that began before is the share's first segment, one that goes on its last)
        float* const part = p.part + (static_cast<int64_t>(blockIdx.x) * 2 + g.starts) * S::kPartFloats;
        const int row = 128 * t + r;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 16) {
          uint32_t w[16] = {};
          if (some) tmem_load(to + c0, w);
#pragma unroll
          for (int c = 0; c < 16; c += 4)
            *reinterpret_cast<uint4*>(part + static_cast<int64_t>(row) * D + c0 + c) = make_uint4(w[c], w[c + 1], w[c + 2], w[c + 3]);
        }
        part[kRows * D + row] = m;
        part[kRows * D + kRows + row] = l;
      }
      umma_fence_before();  // (the tile's next product into O follows this warp's next arrival)
    }
  }
  if (!ok && lane == 0) atomicOr(&g_hq_fault, kFaultWaitTimeout);
  __syncwarp();
  umma_fence_before();
  __syncthreads();
  umma_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Items that were cut: blockIdx.x the CTA that an item begins in, blockIdx.y a slice of its rows.
template <int D, int SUB>
__global__ void __launch_bounds__(256) k_kv_prompt_combine(const __grid_constant__ KvAttendParams p) {
  using S = KvPromptShape<D, SUB>;
  constexpr int kRows = S::kRows, kLanes = D / 8;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int cta = static_cast<int>(blockIdx.x);
  const KvCut* const cuts = reinterpret_cast<const KvCut*>(p.part + static_cast<int64_t>(2) * kKvMaxCtas * S::kPartFloats);
  const int4 cut = __ldcg(reinterpret_cast<const int4*>(cuts + cta));
  const int last = cut.w;
  if (last < 0) return;
  const KvSeq seq = kv_seq(p, cut.x);
  const float v_sg = kv_global_scale(__ldg(p.kv_amax + 1));
  auto part = [&](int k) { return p.part + (static_cast<int64_t>(k) * 2 + (k == cta)) * S::kPartFloats; };
  for (int task = blockIdx.y * 256 + threadIdx.x; task < kRows * kLanes; task += 256 * gridDim.y) {
    const int row = task / kLanes, e = task % kLanes;
    float top = kKvNone;
    for (int k = cta; k <= last; ++k) top = fmaxf(top, __ldcg(part(k) + kRows * D + row));
    float sum = 0.0f, v[8] = {};
#pragma unroll 4
    for (int k = cta; k <= last; ++k) {
      const float* const from = part(k);
      const float f = exp2_fast(__ldcg(from + kRows * D + row) - top);
      sum += __ldcg(from + kRows * D + kRows + row) * f;
      const float4* const src = reinterpret_cast<const float4*>(from + row * D + 8 * e);
      const float4 a = __ldcg(src), b = __ldcg(src + 1);
      v[0] += a.x * f, v[1] += a.y * f, v[2] += a.z * f, v[3] += a.w * f;
      v[4] += b.x * f, v[5] += b.y * f, v[6] += b.z * f, v[7] += b.w * f;
    }
    const int at = cut.y * kRows + row;
    kv_finish<D>(p, v, top, sum, v_sg, seq.q0 + at / p.share, cut.z * p.share + at % p.share, e, at < seq.nq * p.share);
  }
}

}  // namespace hq
