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
//   d  = dh' + r_pre gn - h' k,   k = r_pre^3 / D sum(gn h')       the whole gradient at h'
//   dh = alpha d,  dgate = d u,  du = d gate
//   dy = r_post du w_post - y r_post^3 / D sum(du w_post y)
//   dw_pre = sum_rows dn h' r_pre,  dw_post = sum_rows du y r_post
// The second row sum contains d, which needs the first; since d is linear in k, three sums over the
// inputs alone -- sum(gn h'), sum((dh' + r_pre gn) q), sum(h' q), q = gate w_post y -- give both, so a row
// has one reduction.  dw_post and a per-channel dgate are the same column sum A = sum_rows d y r_post
// times gate and times w_post, so two column sums are kept, not three.
//
// Bound by memory: 8 bytes per element forward, 12 backward (bf16).  A CTA keeps its columns for all
// its rows, so the column sums stay in registers and the parameters in shared memory; rows arrive
// through a ring of bulk copies (cp.async.bulk), so the loads of the next rows run under a row's
// reduction.  Rows of more columns than a CTA holds are split over a cluster, which adds its row sums
// in distributed shared memory; narrow rows are taken several at a time.  Column sums end as one
// partial row per cluster, added in a fixed order by k_norm_columns: no atomics, the same bits each time.
#pragma once

#include <cuda_bf16.h>

#include "hq_kernels.cuh"

namespace hq {

constexpr int kNormThreads = 512;    // most threads of a CTA
constexpr int kNormMaxStages = 4;
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
  __device__ __forceinline__ void store(uint8_t* p) const {
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (BF16) {
      const uint32_t x[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(x[i] << 16);
        f[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(w[i].x), f[4 * i + 1] = __uint_as_float(w[i].y);
        f[4 * i + 2] = __uint_as_float(w[i].z), f[4 * i + 3] = __uint_as_float(w[i].w);
      }
    }
  }
  // rounds to the data type (to nearest even); f becomes the rounded values
  __device__ __forceinline__ void set(float (&f)[8]) {
    if constexpr (BF16) {
      uint32_t x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        x[i] = *reinterpret_cast<uint32_t*>(&b);
      }
      w[0] = make_uint4(x[0], x[1], x[2], x[3]);
      get(f);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        w[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                          __float_as_uint(f[4 * i + 3]));
    }
  }
};

__device__ __forceinline__ float norm_param(const void* w, int64_t i, int bf16) {
  if (!w) return 1.0f;
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]) : static_cast<const float*>(w)[i];
}

// A CTA's columns of a parameter in shared memory: the first halves of all units, then the second
// halves (16-byte reads of neighbouring threads then meet no bank twice).
__device__ __forceinline__ void read_param(const float* s, int units, int u, float (&f)[8]) {
  const float4 a = reinterpret_cast<const float4*>(s)[u], b = reinterpret_cast<const float4*>(s)[units + u];
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ int param_slot(int units, int col) {
  return ((col & 4) ? 4 * units : 0) + (col >> 3) * 4 + (col & 3);
}

// A float into the same shared variable of CTA `rank` of the cluster.
__device__ __forceinline__ void store_cluster(const float* p, uint32_t rank, float v) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.f32 [a], %2;\n\t}" ::"r"(smem_addr(p)),
      "r"(rank), "f"(v)
      : "memory");
}

struct NormShared {
  uint64_t full[kNormMaxStages];
  float part[2][kNormThreads / 32][3];       // a warp's sums, by parity of the reduction
  float cluster[2][kNormMaxCluster][3];
  float most[kNormThreads / 32];
};

// The row sums of NS values over the threads of a row (tpr of them) and over the cluster; every
// thread of the CTA calls it.  Sums are added in a fixed order.
template <int NS>
__device__ __forceinline__ void row_sums(NormShared& sh, int& parity, const NormParams& p, int row, uint32_t ranks,
                                         uint32_t rank, float (&s)[NS]) {
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) s[i] += __shfl_xor_sync(0xFFFFFFFFu, s[i], m);
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < NS; ++i) sh.part[parity][threadIdx.x >> 5][i] = s[i];
  __syncthreads();
  const int warps = p.tpr >> 5;
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    s[i] = 0.0f;
    for (int w = 0; w < warps; ++w) s[i] += sh.part[parity][row * warps + w][i];
  }
  if (ranks > 1) {  // (one row per step)
    if (threadIdx.x < ranks)
#pragma unroll
      for (int i = 0; i < NS; ++i) store_cluster(&sh.cluster[parity][rank][i], threadIdx.x, s[i]);
    cluster_sync();
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      s[i] = 0.0f;
      for (uint32_t r = 0; r < ranks; ++r) s[i] += sh.cluster[parity][r][i];
    }
  }
  parity ^= 1;
}

// max |x . H_G / sqrt(G)| over one unit per lane (G = 16: two lanes; G = 256: the warp), in the
// butterfly order of the quantizer: stages h = 1, 2, 4, ... G / 2, then the scale.
__device__ __forceinline__ float rotated_absmax(float (&f)[8], int group, int lane) {
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
// The ring of rows.  Stage layout: tensor t, row r of the step at (t * rows + r) * cols * es.
// ---------------------------------------------------------------------------
template <bool BF16, int NT>
struct RowRing {
  static constexpr int kEs = BF16 ? 2 : 4;
  const NormParams& p;
  uint8_t* base;
  NormShared& sh;
  int64_t first, stride;  // this cluster's first step, and the step between its steps (in steps)
  int64_t steps;
  int col0, bytes;        // bytes of a row's part

  __device__ __forceinline__ int stage_bytes() const { return NT * p.rows * p.cols * kEs; }

  // Thread 0: the copies of this cluster's step i.
  __device__ __forceinline__ void fetch(int64_t i) const {
    if (i >= steps) return;
    const int s = static_cast<int>(i % p.stages);
    const uint32_t bar = smem_addr(&sh.full[s]);
    const int64_t row0 = (first + i * stride) * p.rows;
    const int n = static_cast<int>(p.M - row0 < p.rows ? p.M - row0 : p.rows);
    int tensors = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t) tensors += p.in[t] != nullptr;
    mbar_expect_tx(bar, static_cast<uint32_t>(tensors * n * bytes));
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (!p.in[t]) continue;
      for (int r = 0; r < n; ++r) {
        const uint8_t* src = p.in[t] + (row0 + r) * p.ld[t] + static_cast<int64_t>(col0) * kEs;
        const uint32_t dst = smem_addr(base + s * stage_bytes() + (t * p.rows + r) * p.cols * kEs);
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
            "l"(src), "r"(static_cast<uint32_t>(bytes)), "r"(bar)
            : "memory");
      }
    }
  }
  __device__ __forceinline__ bool wait(int64_t i) const {
    return mbar_wait(smem_addr(&sh.full[i % p.stages]), static_cast<uint32_t>((i / p.stages) & 1));
  }
  __device__ __forceinline__ const uint8_t* at(int64_t i, int t, int r) const {
    return base + (i % p.stages) * stage_bytes() + (t * p.rows + r) * p.cols * kEs;
  }
};

// What both kernels set up: the ring, the parameters' columns in shared memory, the thread's place.
// params[0]: w_pre; params[1]: w_post, times a per-channel gate.
#define HQ_NORM_SETUP(NT)                                                                             \
  constexpr int kEs = BF16 ? 2 : 4;                                                                   \
  extern __shared__ __align__(128) uint8_t norm_smem[];                                               \
  __shared__ NormShared sh;                                                                           \
  const uint32_t ranks = cluster_size(), rank = cluster_rank();                                       \
  const int units = p.cols / 8;                                                                       \
  float* const s_pre = reinterpret_cast<float*>(norm_smem);                                           \
  float* const s_post = s_pre + p.cols;                                                               \
  const int col0 = static_cast<int>(rank) * p.cols;                                                   \
  const int my_cols = min(p.cols, p.D - col0);                                                        \
  const int my_units = my_cols / 8;                                                                   \
  const int64_t all_steps = (p.M + p.rows - 1) / p.rows;                                              \
  const int64_t cluster = blockIdx.x / ranks, clusters = gridDim.x / ranks;                           \
  RowRing<BF16, NT> ring{p, norm_smem + 8 * static_cast<size_t>(p.cols), sh, cluster, clusters,       \
                         cluster < all_steps ? (all_steps - cluster + clusters - 1) / clusters : 0,   \
                         col0, my_cols * kEs};                                                        \
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");                                     \
  if (threadIdx.x == 0) {                                                                             \
    for (int i = 0; i < p.stages; ++i) mbar_init(smem_addr(&sh.full[i]), 1);                          \
    fence_mbar_init();                                                                                \
    asm volatile("griddepcontrol.wait;" ::: "memory");                                                \
    for (int i = 0; i < p.stages; ++i) ring.fetch(i);                                                 \
  }                                                                                                   \
  asm volatile("griddepcontrol.wait;" ::: "memory");                                                  \
  for (int c = threadIdx.x; c < my_cols; c += blockDim.x) {                                           \
    const int slot = param_slot(units, c);                                                            \
    s_pre[slot] = norm_param(p.w_pre, col0 + c, p.params_bf16);                                       \
    float w = norm_param(p.post ? p.w_post : nullptr, col0 + c, p.params_bf16);                       \
    if (p.gate_kind == kGateChannel) w = __fmul_rn(w, norm_param(p.gate, col0 + c, p.params_bf16));   \
    s_post[slot] = w;                                                                                 \
  }                                                                                                   \
  const int row = threadIdx.x / p.tpr, lane_u = threadIdx.x - row * p.tpr;                            \
  int parity = 0;                                                                                     \
  bool ok = true;                                                                                     \
  __syncthreads();                                                                                    \
  if (ranks > 1) cluster_sync() /* the peers' shared memory is there */

// After the last step: report a wait that ran out, with the copies in flight given time to land.
#define HQ_NORM_FINISH()                                                                              \
  if (!ok) {                                                                                          \
    if (threadIdx.x == 0)                                                                             \
      for (int64_t i = ring.steps > p.stages ? ring.steps - p.stages : 0; i < ring.steps; ++i)        \
        ring.wait(i);                                                                                 \
    if ((threadIdx.x & 31) == 0) atomicOr(&g_hq_fault, kFaultWaitTimeout);                            \
  }

template <bool BF16, int V>
__global__ void __launch_bounds__(kNormThreads, 1) k_block_norm(const __grid_constant__ NormParams p) {
  HQ_NORM_SETUP(2);
  float most = 0.0f;
  for (int64_t i = 0; i < ring.steps; ++i) {
    const int64_t m = (ring.first + i * ring.stride) * p.rows + row;
    const bool live = m < p.M;
    ok = ok && ring.wait(i);
    Unit<BF16> hu[V], yu[V];
    float ss[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int u = j * p.tpr + lane_u;
      hu[j].zero(), yu[j].zero();
      if (live && u < my_units) {
        hu[j].load(ring.at(i, 0, row) + u * 8 * kEs);
        if (p.has_y) yu[j].load(ring.at(i, 1, row) + u * 8 * kEs);
      }
      if (p.post) {
        float y[8];
        yu[j].get(y);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss[0] = fmaf(y[e], y[e], ss[0]);
      }
    }
    float r_post = 1.0f;
    if (p.post) {
      row_sums<1>(sh, parity, p, row, ranks, rank, ss);
      r_post = __frsqrt_rn(__fadd_rn(__fdiv_rn(ss[0], static_cast<float>(p.D)), p.eps));
    } else {
      __syncthreads();
    }
    if (threadIdx.x == 0) {  // every thread has its part of the stage in registers
      fence_proxy_async_smem();
      ring.fetch(i + p.stages);
    }
    if (p.post && live && lane_u == 0 && rank == 0) p.r_post[m] = r_post;
    if (p.gate_kind == kGateToken && live) r_post *= norm_param(p.gate, m, p.params_bf16);
    float t[V][8];
    ss[0] = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int u = j * p.tpr + lane_u;
      const bool in = live && u < my_units;
      hu[j].get(t[j]);
      if (p.has_y) {
        float y[8], w[8];
        yu[j].get(y);
        if (in) read_param(s_post, units, u, w);
        else
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = 0.0f;
        if (p.gate_kind == kGateFull && in) {
          Unit<BF16> gu;
          float g[8];
          gu.load(static_cast<const uint8_t*>(p.gate) + m * p.ld_gate + static_cast<int64_t>(col0 + u * 8) * kEs);
          gu.get(g);
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] *= g[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) t[j][e] = fmaf(y[e] * r_post, w[e], p.alpha * t[j][e]);
        if (in) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = t[j][e];
          Unit<BF16> o;
          o.set(f);
          o.store(static_cast<uint8_t*>(p.h_out) + (m * p.D + col0 + u * 8) * kEs);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) ss[0] = fmaf(t[j][e], t[j][e], ss[0]);
    }
    if (!p.pre) continue;
    row_sums<1>(sh, parity, p, row, ranks, rank, ss);
    const float r_pre = __frsqrt_rn(__fadd_rn(__fdiv_rn(ss[0], static_cast<float>(p.D)), p.eps));
    if (live && lane_u == 0 && rank == 0) p.r_pre[m] = r_pre;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int u = j * p.tpr + lane_u;
      const bool in = live && u < my_units;
      float f[8];
      if (in) {
        read_param(s_pre, units, u, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= t[j][e] * r_pre;
        Unit<BF16> o;
        o.set(f);
        o.store(static_cast<uint8_t*>(p.n) + (m * p.D + col0 + u * 8) * kEs);
      }
      if (p.group >= 0) {  // (uniform over the grid: every lane takes part in the exchange)
        if (!in)
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = 0.0f;
        most = max_nan(most, rotated_absmax(f, p.group, threadIdx.x & 31));
      }
    }
  }
  if (p.group >= 0) {
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
  if (ranks > 1) cluster_sync();
}

template <bool BF16, int V>
__global__ void __launch_bounds__(kNormThreads, 1) k_block_norm_bwd(const __grid_constant__ NormParams p) {
  HQ_NORM_SETUP(4);
  float sum_w[V][8], sum_a[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum_w[j][e] = sum_a[j][e] = 0.0f;
  const float inv_d = __fdiv_rn(1.0f, static_cast<float>(p.D));
  for (int64_t i = 0; i < ring.steps; ++i) {
    const int64_t m = (ring.first + i * ring.stride) * p.rows + row;
    const bool live = m < p.M;
    ok = ok && ring.wait(i);
    const float r_pre = p.pre && live ? __ldg(p.r_pre_in + m) : 0.0f;
    const float r_post = p.post && live ? __ldg(p.r_post_in + m) : 1.0f;
    const float tok = p.gate_kind == kGateToken && live ? norm_param(p.gate, m, p.params_bf16) : 1.0f;
    // hu: h'; nu: dn; du: dh'; yu: y
    Unit<BF16> hu[V], nu[V], du[V], yu[V], gu[V];
    float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int u = j * p.tpr + lane_u;
      hu[j].zero(), nu[j].zero(), du[j].zero(), yu[j].zero();
      if (live && u < my_units) {
        if (p.pre) hu[j].load(ring.at(i, 0, row) + u * 8 * kEs), nu[j].load(ring.at(i, 1, row) + u * 8 * kEs);
        if (p.in[2]) du[j].load(ring.at(i, 2, row) + u * 8 * kEs);
        float h[8], n[8], w[8];
        hu[j].get(h), nu[j].get(n);
        read_param(s_pre, units, u, w);
        if (p.has_y) {
          yu[j].load(ring.at(i, 3, row) + u * 8 * kEs);
          float d[8], y[8], q[8];
          du[j].get(d), yu[j].get(y);
          read_param(s_post, units, u, q);
          if (p.gate_kind == kGateFull) {
            gu[j].load(static_cast<const uint8_t*>(p.gate) + m * p.ld_gate + static_cast<int64_t>(col0 + u * 8) * kEs);
            float g[8];
            gu[j].get(g);
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] *= g[e];
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float gn = n[e] * w[e], qy = q[e] * y[e];
            s[0] = fmaf(gn, h[e], s[0]);
            s[1] = fmaf(fmaf(r_pre, gn, d[e]), qy, s[1]);
            s[2] = fmaf(h[e], qy, s[2]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) s[0] = fmaf(n[e] * w[e], h[e], s[0]);
        }
      }
    }
    row_sums<3>(sh, parity, p, row, ranks, rank, s);
    if (threadIdx.x == 0) {  // every thread has its part of the stage in registers
      fence_proxy_async_smem();
      ring.fetch(i + p.stages);
    }
    const float k1 = r_pre * r_pre * r_pre * (s[0] * inv_d);
    const float dot = fmaf(-k1, s[2], s[1]);  // sum d q (a per-token gate left out)
    const float k2 = r_post * r_post * r_post * (tok * dot * inv_d);
    if (p.gate_kind == kGateToken && live && lane_u == 0 && rank == 0) static_cast<float*>(p.dgate)[m] = dot * r_post;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int u = j * p.tpr + lane_u;
      if (!live || u >= my_units) continue;
      const int64_t at = (m * p.D + col0 + u * 8) * kEs;
      float h[8], n[8], d[8], w[8], o[8];
      hu[j].get(h), nu[j].get(n), du[j].get(d);
      read_param(s_pre, units, u, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum_w[j][e] = fmaf(n[e] * r_pre, h[e], sum_w[j][e]);
        d[e] = fmaf(-h[e], k1, fmaf(r_pre, n[e] * w[e], d[e]));
        o[e] = p.alpha * d[e];
      }
      Unit<BF16> out;
      out.set(o);
      out.store(static_cast<uint8_t*>(p.dh) + at);
      if (!p.has_y) continue;
      float y[8];
      yu[j].get(y);
      read_param(s_post, units, u, w);
      if (p.gate_kind == kGateFull) {
        float g[8];
        gu[j].get(g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          o[e] = d[e] * (w[e] * y[e] * r_post);
          d[e] *= g[e];
        }
        out.set(o);
        out.store(static_cast<uint8_t*>(p.dgate) + at);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[e] *= tok;
        sum_a[j][e] = fmaf(d[e] * r_post, y[e], sum_a[j][e]);
        o[e] = d[e] * w[e];
        if (p.post) o[e] = fmaf(r_post, o[e], -y[e] * k2);
      }
      out.set(o);
      out.store(static_cast<uint8_t*>(p.dy) + at);
    }
  }
  HQ_NORM_FINISH();
  // The rows of a step add their column sums one after another; the ring is free now.
  float* const s_sum = reinterpret_cast<float*>(ring.base);
  for (int r = 0; r < p.rows; ++r) {
    __syncthreads();
    if (r != row) continue;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int u = j * p.tpr + lane_u;
      if (u >= my_units) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int slot = param_slot(units, u * 8 + e);
        s_sum[slot] = (r ? s_sum[slot] : 0.0f) + sum_w[j][e];
        s_sum[p.cols + slot] = (r ? s_sum[p.cols + slot] : 0.0f) + sum_a[j][e];
      }
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < my_cols; c += blockDim.x) {
    const int slot = param_slot(units, c);
    p.partial[cluster * p.D + col0 + c] = s_sum[slot];
    p.partial[(clusters + cluster) * p.D + col0 + c] = s_sum[p.cols + slot];
  }
  if (ranks > 1) cluster_sync();
}

// The clusters' partial column sums, added in a fixed order; dw_post = gate A, dgate = w_post A.
// 32 columns x 8 slices of the clusters per CTA.
__global__ void __launch_bounds__(256) k_norm_columns(const float* __restrict__ partial, int clusters, int D,
                                                      const void* w_post, const void* gate, int params_bf16,
                                                      float* dw_pre, float* dw_post, float* dgate) {
  __shared__ float s[2][8][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float v = 0.0f;
    if (c < D)
#pragma unroll 8
      for (int i = slice; i < clusters; i += 8) v += partial[(static_cast<int64_t>(k) * clusters + i) * D + c];
    s[k][slice][threadIdx.x & 31] = v;
  }
  __syncthreads();
  if (slice < 2 && c < D) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += s[slice][i][threadIdx.x & 31];
    if (slice == 0) {
      if (dw_pre) dw_pre[c] = v;
    } else {
      if (dw_post) dw_post[c] = v * norm_param(gate, c, params_bf16);
      if (dgate) dgate[c] = v * norm_param(w_post, c, params_bf16);
    }
  }
}

}  // namespace hq
