// hq_norm.cuh -- device code of the norms before and after a block (sm_103a), forward and backward.
//
//   u  = y r_post w_post            r_post = 1 / sqrt(mean y^2 + eps)   (u = y without the post norm)
//   h' = alpha h + gate u           gate: per channel, per token, per element, or none
//   n  = h' r_pre w_pre             r_pre = 1 / sqrt(mean h'^2 + eps)
//
// One pass over h and y writes h' and n; n is computed from h' in fp32, before its rounding.
// Optionally the pass also takes max |rotated n|, the amax that the quantizer's pass 1 would read n
// again for: the rotation runs on the rounded n in the quantizer's own butterfly order, so the
// result is that pass's bit for bit.
//
// Backward, with gn = dn w_pre:
//   d  = dh' + r_pre (gn - h' k), k = r_pre^2 / D sum(gn h')       the whole gradient at h'
//   dh = alpha d,  dgate = d u,  du = d gate
//   dy = r_post du w_post - (y r_post) c r_post,  c = r_post / D sum(du w_post y)
//   dw_pre = sum_rows dn h' r_pre,  dw_post = sum_rows du y r_post
// The second row sum contains d, which needs the first; since d is linear in k, three sums over the
// inputs alone -- sum(gn h'), sum((dh' + r_pre gn) q), sum(h' q), q = gate w_post y -- give both, so a row
// has one reduction.  dw_post and a per-channel dgate are the same column sum A = sum_rows d y r_post
// times gate and times w_post, so two column sums are kept, not three.
//
// Bound by memory: 8 bytes per element forward, 12 backward (bf16).  A CTA keeps its columns for all
// its rows, so the column sums and the parameters stay in registers; rows arrive through a ring of
// bulk copies (cp.async.bulk).  A row's phases are spread over the steps of the loop -- forward: the sum
// over y; h' and the sum over it; n -- so that a step works on three rows (backward: two) and has one
// barrier, behind which the sums of all of them travel: with one row at a time a CTA waited for its
// reductions half of the time (bf16 [16384, 8192] forward 313 us; 169 now, 6.4 TB/s, 0.94 of a copy).  Rows of more columns than a CTA
// holds are split over a cluster, whose warps write their sums into every CTA's shared memory;
// narrow rows are taken several at a time.  Column sums end as one partial row per cluster, added in
// a fixed order by k_norm_columns: no atomics, the same bits each time.  Backward bf16 [8192, 8192] takes 140 us,
// 5.75 TB/s, 0.85 of a copy: 16 warps of 128 registers fill the register file, and with no more of them what a step
// costs beside its bytes is not all hidden.  fp32 [1021, 1360] takes 16.8 us for 33 MB: its first rows arrive 4 us
// after the start, five steps take some 1.8 us each, and the column sums have a second kernel.
#pragma once

#include <cuda_bf16.h>

#include "hq_kernels.cuh"

namespace hq {

constexpr int kNormThreads = 512;    // most threads of a CTA
constexpr int kNormMaxStages = 8;
constexpr int kNormMaxCluster = 8;
constexpr int kNormMaxPartials = 192;  // clusters of the backward kernel, at most

enum NormGate { kGateNone = 0, kGateChannel = 1, kGateToken = 2, kGateFull = 3 };

struct NormParams {
  const uint8_t* in[4];   // forward: h, y.  backward: h', dn, dh', y.  NULL: absent
  int64_t ld[4];          // their row strides in bytes
  const void* w_post;     // [D] of the parameter type, or NULL (ones)
  const void* w_pre;
  const void* gate;       // [D], [M] (parameter type) or [M, D] (data type)
  int64_t ld_gate;        // bytes (full gate)
  int params_bf16;
  int gate_kind;
  int post, pre, has_y;
  int64_t M;
  int D, cols, tpr, rows, stages;  // cols: columns per CTA; tpr: threads per row; rows: rows per step
  float alpha, eps;
  // forward
  void* h_out;
  void* n;
  float* r_post;
  float* r_pre;
  int group;              // rotation of the amax (0, 16, 256), or -1: no amax
  unsigned* amax;
  // backward
  const float* r_post_in;
  const float* r_pre_in;
  void* dh;
  void* dy;
  void* dgate;            // [M] fp32 (token) or [M, D] of the data type (full)
  float* partial;         // [2][clusters][D]: sums of dn h' r_pre, and A
};

// ---------------------------------------------------------------------------
// A unit is 8 consecutive elements of a row.
// ---------------------------------------------------------------------------
template <bool BF16>
struct Unit {
  uint4 w[BF16 ? 1 : 2];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (auto& x : w) x = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void load(const uint8_t* p) {
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  // From a row in shared memory, where neighbouring lanes read neighbouring units.  fp32: half of the lanes read
  // the second 16 bytes first, or lanes 4 apart would meet in the same banks.
  __device__ __forceinline__ void load_row(const uint8_t* p) {
    if constexpr (BF16) {
      load(p);
    } else {
      const bool second = threadIdx.x & 4;
      const uint4 a = reinterpret_cast<const uint4*>(p)[second], b = reinterpret_cast<const uint4*>(p)[!second];
      w[0] = second ? b : a;
      w[1] = second ? a : b;
    }
  }
  __device__ __forceinline__ void store(uint8_t* p) const {
    if constexpr (!BF16) {
      if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {  // whole sectors
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0].x), "r"(w[0].y),
                     "r"(w[0].z), "r"(w[0].w), "r"(w[1].x), "r"(w[1].y), "r"(w[1].z), "r"(w[1].w)
                     : "memory");
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
  }
  // values 2 i and 2 i + 1 in f[i]
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
    if constexpr (BF16) {
      const uint32_t x[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xFFFF0000u));
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f[2 * i] = make_float2(__uint_as_float(w[i].x), __uint_as_float(w[i].y));
        f[2 * i + 1] = make_float2(__uint_as_float(w[i].z), __uint_as_float(w[i].w));
      }
    }
  }
  // rounds to the data type (to nearest even)
  __device__ __forceinline__ void set(const float2 (&f)[4]) {
    if constexpr (BF16) {
      uint32_t x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        __nv_bfloat162 b = __floats2bfloat162_rn(f[i].x, f[i].y);
        x[i] = *reinterpret_cast<uint32_t*>(&b);
      }
      w[0] = make_uint4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        w[i] = make_uint4(__float_as_uint(f[2 * i].x), __float_as_uint(f[2 * i].y), __float_as_uint(f[2 * i + 1].x),
                          __float_as_uint(f[2 * i + 1].y));
    }
  }
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

__device__ __forceinline__ float norm_param(const void* w, int64_t i, int bf16) {
  if (!w) return 1.0f;
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]) : static_cast<const float*>(w)[i];
}

// A unit of a parameter vector (ones where it is absent; zeros outside the row).
__device__ __forceinline__ void param_unit(const void* w, int64_t col, int bf16, bool in, float2 (&f)[4]) {
  if (in && w && (reinterpret_cast<uintptr_t>(w) & 15) == 0) {  // the usual case: two loads at most
    if (bf16) {
      Unit<true> u;
      u.load(static_cast<const uint8_t*>(w) + col * 2);
      u.get(f);
    } else {
      Unit<false> u;
      u.load(static_cast<const uint8_t*>(w) + col * 4);
      u.get(f);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    f[e] = in ? make_float2(norm_param(w, col + 2 * e, bf16), norm_param(w, col + 2 * e + 1, bf16)) : both(0.0f);
}

// The row sums of four steps.  In a cluster every warp sends its sums to every CTA by asynchronous stores that
// count on the step's mbarrier there: no barrier of the cluster, whose release would also wait for the output
// rows' stores (bf16 [2000, 12288] forward 67 -> 51 us, 3.9 TB/s).  Four steps' slots are enough: a warp sends
// for step j after it has all sums of step j - 2, every warp sent those after it had read the sums of step j - 4.
constexpr int kNormSlots = 4;

struct NormShared {
  uint64_t full[kNormMaxStages];
  uint64_t sums[kNormSlots];
  float part[kNormSlots][3][kNormMaxCluster * 16];  // [.][.][rank * 16 + warp]
  float most[kNormThreads / 32];
};

// A float into the same shared variable of CTA `rank` of the cluster, counted on that CTA's barrier.
__device__ __forceinline__ void send_cluster(const float* p, const uint64_t* bar, uint32_t rank, float v) {
  asm volatile(
      "{\n\t.reg .b32 a, b;\n\tmapa.shared::cluster.u32 a, %0, %2;\n\tmapa.shared::cluster.u32 b, %1, %2;\n\t"
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [a], %3, [b];\n\t}" ::"r"(smem_addr(p)),
      "r"(smem_addr(bar)), "r"(rank), "r"(__float_as_uint(v))
      : "memory");
}

// Waits for a step's sums, up to the limit of mbar_wait.
__device__ __forceinline__ bool wait_sums(const NormShared& sh, int step) {
  const uint32_t bar = smem_addr(&sh.sums[step & (kNormSlots - 1)]), parity = step / kNormSlots & 1;
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((i & 15u) == 0) {
      const uint64_t now = global_timer_ns();
      if (i == 0)
        t0 = now;
      else if (now - t0 > kWaitLimitNs)
        return false;
    }
  }
}

// This warp's sums of two or three values, for every CTA of the cluster.  The lanes halve the values among them
// while they halve each other: 5 or 6 shuffles, where a value at a time takes 5 each (they are a third of the
// instructions that the step waits for); sum q ends in lanes 8 q .. 8 q + 7.
template <int NS>
__device__ __forceinline__ void put_sums(NormShared& sh, int step, uint32_t ranks, uint32_t rank, const float (&s)[NS]) {
  static_assert(NS == 2 || NS == 3, "halved twice");
  const int lane = threadIdx.x & 31;
  const bool hi = lane & 16, odd = lane & 8;
  float a = hi ? (NS == 3 ? s[2] : 0.0f) : s[0], b = hi ? 0.0f : s[1];
  a += __shfl_xor_sync(0xFFFFFFFFu, hi ? s[0] : (NS == 3 ? s[2] : 0.0f), 16);
  b += __shfl_xor_sync(0xFFFFFFFFu, hi ? s[1] : 0.0f, 16);
  float v = odd ? b : a;
  v += __shfl_xor_sync(0xFFFFFFFFu, odd ? a : b, 8);
#pragma unroll
  for (int m = 4; m >= 1; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  const int q = lane >> 3, at = static_cast<int>(rank) * 16 + (threadIdx.x >> 5), slot = step & (kNormSlots - 1);
  if (q >= NS) return;
  if (ranks == 1) {
    if ((lane & 7) == 0) sh.part[slot][q][at] = v;
  } else if ((lane & 7) < static_cast<int>(ranks)) {
    send_cluster(&sh.part[slot][q][at], &sh.sums[slot], lane & 7, v);
  }
}

// The sums of a row of an earlier step, over its warps and the cluster, in a fixed order: eight lanes add one.
template <int NS>
__device__ __forceinline__ void get_sums(const NormShared& sh, int step, int warps, int row, uint32_t ranks,
                                         float (&s)[NS]) {
  const int lane = threadIdx.x & 31, q = lane >> 3, j = lane & 7;
  const float* const part = sh.part[step & (kNormSlots - 1)][q < NS ? q : 0] + row * warps;
  float v = 0.0f;
  for (uint32_t r = 0; r < ranks; ++r) {
    if (j < warps) v += part[r * 16 + j];
    if (j + 8 < warps) v += part[r * 16 + j + 8];
  }
#pragma unroll
  for (int m = 4; m >= 1; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
#pragma unroll
  for (int i = 0; i < NS; ++i) s[i] = __shfl_sync(0xFFFFFFFFu, v, 8 * i);
}

// max |x . H_G / sqrt(G)| over one unit per lane (G = 16: two lanes; G = 256: the warp), in the
// butterfly order of the quantizer: stages h = 1, 2, 4, ... G / 2, then the scale.
__device__ __forceinline__ float rotated_absmax(const float2 (&v)[4], int group, int lane) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = v[i].x, f[2 * i + 1] = v[i].y;
  if (group) {
#pragma unroll
    for (int h = 1; h < 8; h <<= 1)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!(i & h)) {
          const float a = f[i], b = f[i + h];
          f[i] = __fadd_rn(a, b);
          f[i + h] = __fsub_rn(a, b);
        }
    for (int h = 8; h < group; h <<= 1) {
      const bool low = !(lane & (h >> 3));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float o = __shfl_xor_sync(0xFFFFFFFFu, f[i], h >> 3);
        f[i] = low ? __fadd_rn(f[i], o) : __fsub_rn(o, f[i]);
      }
    }
  }
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(f[i]));
  return __fmul_rn(m, group == 16 ? 0.25f : group == 256 ? 0.0625f : 1.0f);
}

// ---------------------------------------------------------------------------
// The ring of rows.  Stage layout: tensor t, row r of the step at (t * rows + r) * cols * es.  Positions
// are kept as stage numbers that are stepped along: a division per row and thread would cost as much as
// the row.
// ---------------------------------------------------------------------------
template <bool BF16, int NT>
struct RowRing {
  static constexpr int kEs = BF16 ? 2 : 4;
  const NormParams& p;
  uint8_t* base;
  NormShared& sh;
  int64_t first, stride;  // this cluster's first step, and the step between its steps (in steps)
  int steps;
  int col0, bytes;        // bytes of a row's part

  __device__ __forceinline__ int tensor_bytes() const { return p.rows * p.cols * kEs; }
  __device__ __forceinline__ int next(int s) const { return s + 1 == p.stages ? 0 : s + 1; }

  // One warp: the copies of this cluster's step i into stage s; rows that follow one another in one copy.
  __device__ __forceinline__ void fetch(int i, int s) const {
    if (i >= steps) return;
    const uint32_t bar = smem_addr(&sh.full[s]);
    const int64_t row0 = (first + i * stride) * p.rows;
    const int n = static_cast<int>(p.M - row0 < p.rows ? p.M - row0 : p.rows);
    int tensors = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t) tensors += p.in[t] != nullptr;
    if (elect_one()) {
      mbar_expect_tx(bar, static_cast<uint32_t>(tensors * n * bytes));
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (!p.in[t]) continue;
        const uint8_t* src = p.in[t] + row0 * p.ld[t] + static_cast<int64_t>(col0) * kEs;
        uint32_t dst = smem_addr(base) + (s * NT + t) * tensor_bytes();
        const bool whole = p.ld[t] == bytes;
        const int copies = whole ? 1 : n;
        const uint32_t size = static_cast<uint32_t>(whole ? n * bytes : bytes);
        for (int r = 0; r < copies; ++r) {
          asm volatile(
              "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
              "l"(src), "r"(size), "r"(bar)
              : "memory");
          src += p.ld[t];
          dst += p.cols * kEs;
        }
      }
    }
    __syncwarp();
  }
  __device__ __forceinline__ bool wait(int s, uint32_t phase) const { return mbar_wait(smem_addr(&sh.full[s]), phase); }
};

// What both kernels set up: the ring, the thread's place, its units of the parameters.
// w_pre[j], w_post[j]: the j-th unit's parameters, the latter times a per-channel gate.
#define HQ_NORM_SETUP(NT)                                                                             \
  constexpr int kEs = BF16 ? 2 : 4;                                                                   \
  extern __shared__ __align__(128) uint8_t norm_smem[];                                               \
  __shared__ NormShared sh;                                                                           \
  const uint32_t ranks = cluster_size(), rank = cluster_rank();                                       \
  const int col0 = static_cast<int>(rank) * p.cols;                                                   \
  const int my_cols = min(p.cols, p.D - col0);                                                        \
  const int my_units = my_cols / 8;                                                                   \
  const int64_t all_steps = (p.M + p.rows - 1) / p.rows;                                              \
  const int64_t cluster = blockIdx.x / ranks, clusters = gridDim.x / ranks;                           \
  RowRing<BF16, NT> ring{p, norm_smem, sh, cluster, clusters,                                         \
                         static_cast<int>((all_steps - cluster + clusters - 1) / clusters), col0,     \
                         my_cols * kEs};                                                        \
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");                                     \
  /* the last warp fetches the rows */                                                                \
  const bool fetches = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0) == (blockDim.x >> 5) - 1;        \
  if (threadIdx.x == blockDim.x - 32) {                                                               \
    for (int i = 0; i < p.stages; ++i) mbar_init(smem_addr(&sh.full[i]), 1);                          \
    for (int i = 0; i < kNormSlots; ++i) mbar_init(smem_addr(&sh.sums[i]), 1);                        \
    fence_mbar_init();                                                                                \
  }                                                                                                   \
  asm volatile("griddepcontrol.wait;" ::: "memory");                                                  \
  if (fetches) {                                                                                      \
    __syncwarp();                                                                                     \
    for (int i = 0; i < p.stages; ++i) ring.fetch(i, i);                                              \
  }                                                                                                   \
  const int row = threadIdx.x / p.tpr, lane_u = threadIdx.x - row * p.tpr, warps = p.tpr >> 5;        \
  float2 w_pre[V][4], w_post[V][4];                                                                   \
  bool in[V];                                                                                         \
  _Pragma("unroll") for (int j = 0; j < V; ++j) {                                                     \
    const int u = j * p.tpr + lane_u;                                                                 \
    in[j] = u < my_units;                                                                             \
    param_unit(p.w_pre, col0 + u * 8, p.params_bf16, in[j], w_pre[j]);                                \
    param_unit(p.post ? p.w_post : nullptr, col0 + u * 8, p.params_bf16, in[j], w_post[j]);           \
    if (p.gate_kind == kGateChannel) {                                                                \
      float2 g[4];                                                                                    \
      param_unit(p.gate, col0 + u * 8, p.params_bf16, in[j], g);                                      \
      _Pragma("unroll") for (int e = 0; e < 4; ++e) w_post[j][e] = mul2(w_post[j][e], g[e]);          \
    }                                                                                                 \
  }                                                                                                   \
  const bool post = PLAIN || p.post, pre = PLAIN || p.pre, has_y = PLAIN || p.has_y;                  \
  const bool by_token = !PLAIN && p.gate_kind == kGateToken, full = !PLAIN && p.gate_kind == kGateFull; \
  const float inv_d = __fdiv_rn(1.0f, static_cast<float>(p.D));                                       \
  /* of a row in the ring: this thread's first unit of tensor 0 in stage 0; from there on, bytes */   \
  const uint8_t* const units0 = ring.base + row * p.cols * kEs + lane_u * 8 * kEs;                    \
  const int tensor = ring.tensor_bytes(), unit = p.tpr * 8 * kEs;                                     \
  /* of the row of a step in an [M, D] tensor: bytes from one step to the next */                     \
  const int64_t row_step = ring.stride * p.rows * p.D * kEs;                                          \
  int s0 = 0, s1 = 0; /* the stages of this step's row and of the one before */                       \
  uint32_t phase = 0;                                                                                 \
  bool ok = true;                                                                                     \
  __syncthreads();                                                                                    \
  if (ranks > 1) cluster_sync() /* the peers' shared memory is there */

// In a cluster: thread 0 says how many sums per warp a step will bring.
__device__ __forceinline__ void expect_sums(const NormShared& sh, int step, int sums, uint32_t ranks, bool ok) {
  if (ranks > 1 && threadIdx.x == 0 && ok)
    mbar_expect_tx(smem_addr(&sh.sums[step & (kNormSlots - 1)]), sums * ranks * (blockDim.x >> 5) * 4);
}

// After the last step: report a wait that ran out, with the copies in flight given time to land.
#define HQ_NORM_FINISH()                                                                              \
  if (!ok) {                                                                                          \
    if (fetches)                                                                                      \
      for (int i = ring.steps > p.stages ? ring.steps - p.stages : 0; i < ring.steps; ++i)            \
        ring.wait(i % p.stages, (i / p.stages) & 1);                                                  \
    if ((threadIdx.x & 31) == 0) atomicOr(&g_hq_fault, kFaultWaitTimeout);                            \
  }                                                                                                   \
  if (ranks > 1) {                                                                                    \
    cluster_sync();                                                                                   \
    if (!ok) __nanosleep(1000000); /* sums that were not waited for land in this CTA's memory */      \
  }                                                                                                   \
  static_assert(true, "")

// PLAIN: both norms, y, no gate or one per channel, no amax -- known to the compiler, which then has no
// branch in the loop (bf16 [16384, 8192] forward 169 us; 235 without when this was chosen).  With the amax the same
// call takes 214 us without a rotation, 240 with 16 and 312 with 256 points: the branches, then the exchange.
template <bool BF16, int V, bool PLAIN>
__global__ void __launch_bounds__(kNormThreads, 1) k_block_norm(const __grid_constant__ NormParams p) {
  HQ_NORM_SETUP(2);
  float most = 0.0f;
  float2 t[V][4];  // h' of the row before
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) t[j][e] = both(0.0f);
  const int64_t stride = ring.stride * p.rows;
  int64_t m0 = ring.first * p.rows + row;  // row of step i
  // this thread's first unit of the output rows of steps i - 1 and i - 2
  int64_t at1 = ((m0 - stride) * p.D + col0 + lane_u * 8) * kEs;
  // Step i: the sum over y of its i-th row; h' of row i - 1; n of row i - 2.
  for (int i = 0; i < ring.steps + 2; ++i) {
    const int64_t m1 = m0 - stride, m2 = m1 - stride;
    if (i <= ring.steps) expect_sums(sh, i, 2, ranks, ok);
    const bool live1 = i >= 1 && i <= ring.steps && m1 < p.M, live2 = i >= 2 && m2 < p.M;
    float gate = 1.0f;
    if (by_token && live1) gate = norm_param(p.gate, m1, p.params_bf16);
    float put[2] = {0.0f, 0.0f};  // the sum over y of this step's row; over h' of the one before
    if (i < ring.steps) {
      ok = ok && ring.wait(s0, phase);
      if (post) {
        float2 sq = both(0.0f);
        const uint8_t* src = units0 + (s0 * 2 + 1) * tensor;
        if (m0 < p.M)
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (in[j]) {
              Unit<BF16> yu;
              float2 y[4];
              yu.load_row(src + j * unit);
              yu.get(y);
#pragma unroll
              for (int e = 0; e < 4; ++e) sq = fma2(y[e], y[e], sq);
            }
        put[0] = sq.x + sq.y;
      }
    }
    float got[2] = {0.0f, 0.0f};  // of the step before
    if (i >= 1) {
      if (ranks > 1) ok = ok && wait_sums(sh, i - 1);
      get_sums<2>(sh, i - 1, warps, row, ranks, got);
    }
    if (pre && i >= 2) {  // n of row i - 2, from t
      const float r_pre = rsqrtf(fmaf(got[1], inv_d, p.eps));
      if (live2 && lane_u == 0 && rank == 0) p.r_pre[m2] = r_pre;
      uint8_t* const dst = static_cast<uint8_t*>(p.n) + (at1 - row_step);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float2 f[4];
        Unit<BF16> o;
        // (What is not there is 0 in the amax, also times a reciprocal norm that is infinite where eps is 0.)
        const float r = PLAIN || (live2 && in[j]) ? r_pre : 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = mul2(mul2(t[j][e], both(r)), w_pre[j][e]);
        o.set(f);
        if (live2 && in[j]) o.store(dst + j * unit);
        if (!PLAIN && p.group >= 0) {  // (the same for the grid: every lane takes part in the exchange)
          o.get(f);
          most = max_nan(most, rotated_absmax(f, p.group, threadIdx.x & 31));
        }
      }
    }
    if (i >= 1 && i <= ring.steps) {  // h' of row i - 1
      float r_post = 1.0f;
      if (post) {
        r_post = rsqrtf(fmaf(got[0], inv_d, p.eps));
        if (live1 && lane_u == 0 && rank == 0) p.r_post[m1] = r_post;
      }
      r_post *= gate;
      float2 sq = both(0.0f);
      const uint8_t* src = units0 + s1 * 2 * tensor;
      uint8_t* const dst = static_cast<uint8_t*>(p.h_out) + at1;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (!live1 || !in[j]) {
#pragma unroll
          for (int e = 0; e < 4; ++e) t[j][e] = both(0.0f);
          continue;
        }
        Unit<BF16> x;
        x.load_row(src + j * unit);
        x.get(t[j]);
        if (has_y) {
          float2 y[4], g[4];
          x.load_row(src + tensor + j * unit);
          x.get(y);
          if (full) {
            x.load(static_cast<const uint8_t*>(p.gate) + m1 * p.ld_gate + (col0 + lane_u * 8) * kEs + j * unit);
            x.get(g);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = mul2(y[e], g[e]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            t[j][e] = fma2(mul2(y[e], both(r_post)), w_post[j][e], mul2(both(p.alpha), t[j][e]));
          x.set(t[j]);
          x.store(dst + j * unit);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) sq = fma2(t[j][e], t[j][e], sq);
      }
      put[1] = sq.x + sq.y;
    }
    if (i <= ring.steps) put_sums<2>(sh, i, ranks, rank, put);  // (every sum that is sent is waited for)
    __syncthreads();  // one CTA's sums put before it can be got after it; and the stage is free
    if (fetches && i >= 1) {  // row i - 1 has left its stage
      fence_proxy_async_smem();
      ring.fetch(i - 1 + p.stages, s1);
    }
    m0 += stride;
    at1 += row_step;
    s1 = s0;
    s0 = ring.next(s0);
    if (s0 == 0) phase ^= 1;
  }
  if (!PLAIN && p.group >= 0) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) most = max_nan(most, __shfl_xor_sync(0xFFFFFFFFu, most, m));
    if ((threadIdx.x & 31) == 0) sh.most[threadIdx.x >> 5] = most;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (unsigned w = 1; w < blockDim.x / 32; ++w) most = max_nan(most, sh.most[w]);
      atomicMax(p.amax, __float_as_uint(most));
    }
  }
  HQ_NORM_FINISH();
}

// PLAIN: both norms, y, dh', no gate or one per channel.
template <bool BF16, int V, bool PLAIN>
__global__ void __launch_bounds__(kNormThreads, 1) k_block_norm_bwd(const __grid_constant__ NormParams p) {
  HQ_NORM_SETUP(4);
  float2 sum_w[V][4], sum_a[V][4];
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) sum_w[j][e] = sum_a[j][e] = both(0.0f);
  struct RowScalars {
    float r_pre, r_post, tok;
  };
  auto scalars = [&](int i, int64_t m) {
    const bool live = i < ring.steps && m < p.M;
    return RowScalars{pre && live ? __ldg(p.r_pre_in + m) : 0.0f, post && live ? __ldg(p.r_post_in + m) : 1.0f,
                      by_token && live ? norm_param(p.gate, m, p.params_bf16) : 1.0f};
  };
  const int64_t stride = ring.stride * p.rows;
  int64_t m0 = ring.first * p.rows + row;  // row of step i
  int64_t at1 = ((m0 - stride) * p.D + col0 + lane_u * 8) * kEs;  // this thread's first unit of row i - 1
  RowScalars next = scalars(0, m0), now = next, before = next;
  // Step i: the sums of its i-th row; the gradients of row i - 1.
  for (int i = 0; i < ring.steps + 1; ++i) {
    const int64_t m1 = m0 - stride;
    if (i < ring.steps) expect_sums(sh, i, 3, ranks, ok);
    before = now;
    now = next;
    next = scalars(i + 1, m0 + stride);
    if (i < ring.steps) {
      ok = ok && ring.wait(s0, phase);
      float2 c[3] = {both(0.0f), both(0.0f), both(0.0f)};
      const uint8_t* src = units0 + s0 * 4 * tensor;
      if (m0 < p.M)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (!in[j]) continue;
          Unit<BF16> x;
          float2 h[4], n[4];
          x.zero();
          if (pre) x.load_row(src + j * unit);
          x.get(h);
          if (pre) x.load_row(src + tensor + j * unit);
          x.get(n);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sum_w[j][e] = fma2(mul2(n[e], both(now.r_pre)), h[e], sum_w[j][e]);
            n[e] = mul2(n[e], w_pre[j][e]);
            c[0] = fma2(n[e], h[e], c[0]);
          }
          if (!has_y) continue;
          float2 d[4], y[4];
          x.zero();
          if (PLAIN || p.in[2]) x.load_row(src + 2 * tensor + j * unit);
          x.get(d);
          x.load_row(src + 3 * tensor + j * unit);
          x.get(y);
          if (full) {
            float2 g[4];
            x.load(static_cast<const uint8_t*>(p.gate) + m0 * p.ld_gate + (col0 + lane_u * 8) * kEs + j * unit);
            x.get(g);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = mul2(y[e], g[e]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 q = mul2(w_post[j][e], y[e]);
            c[1] = fma2(fma2(both(now.r_pre), n[e], d[e]), q, c[1]);
            c[2] = fma2(h[e], q, c[2]);
          }
        }
      float s[3] = {c[0].x + c[0].y, c[1].x + c[1].y, c[2].x + c[2].y};
      put_sums<3>(sh, i, ranks, rank, s);
    }
    if (i >= 1) {
      if (ranks > 1) ok = ok && wait_sums(sh, i - 1);
      float s[3];
      get_sums<3>(sh, i - 1, warps, row, ranks, s);
      const float r_pre = before.r_pre, r_post = before.r_post, tok = before.tok;
      // (The third powers of the reciprocal norms, which leave fp32 for rows of 1e13 and more, do not occur: one more
      // product per pair of elements, bf16 [8192, 8192] 139 -> 140 us.)
      const float k = r_pre * (r_pre * s[0] * inv_d);
      const float dot = fmaf(-r_pre, k * s[2], s[1]);  // sum d q (a per-token gate left out)
      const float c_post = r_post * (tok * dot * r_post * inv_d);
      if (by_token && m1 < p.M && lane_u == 0 && rank == 0)
        static_cast<float*>(p.dgate)[m1] = dot * r_post;
      const uint8_t* src = units0 + s1 * 4 * tensor;
      if (m1 < p.M)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (!in[j]) continue;
          Unit<BF16> x;
          float2 d[4], v[4], o[4];
          x.zero();
          if (PLAIN || p.in[2]) x.load_row(src + 2 * tensor + j * unit);
          x.get(d);
          if (pre) {
            x.load_row(src + tensor + j * unit);
            x.get(o);
            x.load_row(src + j * unit);
            x.get(v);
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] = fma2(both(r_pre), fma2(v[e], both(-k), mul2(o[e], w_pre[j][e])), d[e]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = mul2(both(p.alpha), d[e]);
          x.set(o);
          x.store(static_cast<uint8_t*>(p.dh) + at1 + j * unit);
          if (!has_y) continue;
          x.load_row(src + 3 * tensor + j * unit);
          x.get(v);
          if (full) {
            float2 g[4];
            x.load(static_cast<const uint8_t*>(p.gate) + m1 * p.ld_gate + (col0 + lane_u * 8) * kEs + j * unit);
            x.get(g);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[e] = mul2(d[e], mul2(mul2(w_post[j][e], v[e]), both(r_post)));
              d[e] = mul2(d[e], g[e]);
            }
            x.set(o);
            x.store(static_cast<uint8_t*>(p.dgate) + at1 + j * unit);
          }
          const float dr = tok * r_post;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            d[e] = mul2(d[e], both(dr));
            sum_a[j][e] = fma2(d[e], v[e], sum_a[j][e]);
            o[e] = mul2(d[e], w_post[j][e]);
            if (post) o[e] = fma2(mul2(v[e], both(r_post)), both(-c_post), o[e]);
          }
          x.set(o);
          x.store(static_cast<uint8_t*>(p.dy) + at1 + j * unit);
        }
    }
    __syncthreads();  // one CTA's sums put before it can be got after it; and the stage is free
    if (fetches && i >= 1) {  // row i - 1 has left its stage
      fence_proxy_async_smem();
      ring.fetch(i - 1 + p.stages, s1);
    }
    m0 += stride;
    at1 += row_step;
    s1 = s0;
    s0 = ring.next(s0);
    if (s0 == 0) phase ^= 1;
  }
  HQ_NORM_FINISH();
  if (p.rows == 1) {  // as they are
    float* const to = p.partial + cluster * p.D + col0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (!in[j]) continue;
      float4* const w4 = reinterpret_cast<float4*>(to + (j * p.tpr + lane_u) * 8);
      float4* const a4 = reinterpret_cast<float4*>(to + clusters * p.D + (j * p.tpr + lane_u) * 8);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        w4[k] = make_float4(sum_w[j][2 * k].x, sum_w[j][2 * k].y, sum_w[j][2 * k + 1].x, sum_w[j][2 * k + 1].y);
        a4[k] = make_float4(sum_a[j][2 * k].x, sum_a[j][2 * k].y, sum_a[j][2 * k + 1].x, sum_a[j][2 * k + 1].y);
      }
    }
    return;
  }
  // The step's rows leave their column sums side by side over the ring, which is free now (8 bytes per
  // row and column, of at least 24), and are added in their order.
  float* const s_sum = reinterpret_cast<float*>(ring.base);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (!in[j]) continue;
    float2* const at = reinterpret_cast<float2*>(s_sum + row * 2 * p.cols) + (j * p.tpr + lane_u) * 4;
#pragma unroll
    for (int e = 0; e < 4; ++e) at[e] = sum_w[j][e], at[p.cols / 2 + e] = sum_a[j][e];
  }
  __syncthreads();
  for (int c = threadIdx.x * 4; c < 2 * p.cols; c += blockDim.x * 4) {
    const int second = c >= p.cols, col = c - second * p.cols;
    if (col >= my_cols) continue;
    float4 v = *reinterpret_cast<const float4*>(s_sum + c);
    for (int r = 1; r < p.rows; ++r) {
      const float4 o = *reinterpret_cast<const float4*>(s_sum + r * 2 * p.cols + c);
      v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
    }
    *reinterpret_cast<float4*>(p.partial + (second * clusters + cluster) * p.D + col0 + col) = v;
  }
}

// The clusters' partial column sums, added in a fixed order; dw_post = gate A, dgate = w_post A.
// 32 columns x 16 slices of the clusters per CTA: a thread's dozen loads are in flight together.
__global__ void __launch_bounds__(512) k_norm_columns(const float* __restrict__ partial, int clusters, int D,
                                                      const void* w_post, const void* gate, int params_bf16,
                                                      float* dw_pre, float* dw_post, float* dgate) {
  constexpr int kSlices = 16, kMost = (kNormMaxPartials + kSlices - 1) / kSlices;
  __shared__ float s[2][kSlices][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float x[kMost], v = 0.0f;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      const int at = slice + i * kSlices;
      x[i] = c < D && at < clusters ? partial[(static_cast<int64_t>(k) * clusters + at) * D + c] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kMost; ++i) v += x[i];
    s[k][slice][threadIdx.x & 31] = v;
  }
  __syncthreads();
  if (slice < 2 && c < D) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kSlices; ++i) v += s[slice][i][threadIdx.x & 31];
    if (slice == 0) {
      if (dw_pre) dw_pre[c] = v;
    } else {
      if (dw_post) dw_post[c] = v * norm_param(gate, c, params_bf16);
      if (dgate) dgate[c] = v * norm_param(w_post, c, params_bf16);
    }
  }
}

}  // namespace hq
