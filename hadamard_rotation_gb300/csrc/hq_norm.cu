// hq_norm.cu -- C ABI of the norms before and after a block (include/hq.h) and their launch logic.
// The kernels are in hq_norm.cuh.
#include <cuda_runtime.h>

#include <cstdint>

#include "hq.h"
#include "hq_internal.h"
#include "hq_norm.cuh"

namespace {

using hq::cuda_fail;
using hq::NormParams;

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxD = 32768;
constexpr int kSmemBytes = 216 * 1024;  // the ring, of the 227 KB a CTA may have
constexpr int kMinStages = 3;           // a step holds two rows' stages while the third is loaded

// Columns per CTA: two units per thread, and no more than leave room for three stages.
struct Shape {
  int ranks, cols, tpr, units, rows, stages;
  size_t smem;
};

Shape shape_of(int64_t M, int D, int es, int tensors, int sms) {
  Shape s;
  const int most = tensors == 4 && es == 4 ? 4096 : 8192;  // (fp32 backward: one unit per thread)
  s.ranks = (D + most - 1) / most;
  s.cols = ((D + s.ranks - 1) / s.ranks + 255) / 256 * 256;  // whole rotation groups
  if (s.ranks == 1) s.cols = D;
  const int u = (s.cols + 7) / 8;
  // Two units per thread where there are rows enough for all SMs all the same: what a step costs a thread
  // beside its elements (the sums' way through shuffles and shared memory) is then shared by 16 of them.
  // (One against two when this was chosen: bf16 [8192, 2048] forward 40.0 / 30.1 us, backward 60.5 / 50.9; now 28.6
  // and 47.0.  Not backward in fp32, whose stages leave room for half the threads then: [4096, 4096] 111 / 186 us.)
  const bool fp32_bwd = tensors == 4 && es == 4;
  s.units = u > hq::kNormThreads || (u >= 64 && M >= 4 * sms && !fp32_bwd) ? 2 : 1;
  s.tpr = ((u + s.units - 1) / s.units + 31) / 32 * 32;
  // narrow rows: several per step, while every SM still gets a step
  int64_t rows = s.ranks > 1 ? 1 : hq::kNormThreads / s.tpr;
  if (rows > (M + sms - 1) / sms) rows = (M + sms - 1) / sms;
  const int64_t row_bytes = static_cast<int64_t>(tensors) * s.cols * es;
  if (rows > kSmemBytes / kMinStages / row_bytes) rows = kSmemBytes / kMinStages / row_bytes;  // (1 at least)
  s.rows = static_cast<int>(rows);
  const size_t stage = static_cast<size_t>(row_bytes * s.rows), n = kSmemBytes / stage;
  s.stages = static_cast<int>(n > hq::kNormMaxStages ? hq::kNormMaxStages : n);
  s.smem = s.stages * stage;
  return s;
}

// Launches as many clusters as there are steps and as run at a time (clusters of 4: 36 of them on 144 of the 152
// SMs; two more would run after all others), and says how many.
template <typename Kernel>
cudaError_t launch(Kernel kernel, const NormParams& p, const Shape& s, int sms, int* clusters, cudaStream_t stream) {
  cudaError_t e = hq::allow_smem(reinterpret_cast<const void*>(kernel), static_cast<int>(s.smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sms / s.ranks * s.ranks));
  cfg.blockDim = dim3(static_cast<unsigned>(s.tpr * s.rows));
  cfg.dynamicSmemBytes = s.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(s.ranks);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  int at_a_time = sms;
  if (s.ranks > 1) {
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = hq::clusters_at_a_time(reinterpret_cast<const void*>(kernel), cfg, s.ranks, &at_a_time)) != cudaSuccess)
      return e;
  }
  const int64_t steps = (p.M + s.rows - 1) / s.rows;
  int64_t n = at_a_time < hq::kNormMaxPartials ? at_a_time : hq::kNormMaxPartials;
  if (n > steps) n = steps;
  *clusters = static_cast<int>(n);
  cfg.gridDim = dim3(static_cast<unsigned>(n * s.ranks));
  cfg.attrs = s.ranks > 1 ? attr : attr + 1;
  cfg.numAttrs = s.ranks > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

hq_status check_sizes(hq_dtype dt, hq_dtype params, int64_t M, int64_t D, hq_gate_kind kind, const void* gate,
                      bool has_y) {
  if ((dt != HQ_F32 && dt != HQ_BF16) || (params != HQ_F32 && params != HQ_BF16)) return HQ_ERR_DTYPE;
  if (M < 0 || D <= 0 || D > kMaxD || D % 16 != 0 || M > INT64_MAX / (D * 4)) return HQ_ERR_SHAPE;
  if (kind < HQ_GATE_NONE || kind > HQ_GATE_FULL) return HQ_ERR_SHAPE;
  if (kind != HQ_GATE_NONE && !has_y) return HQ_ERR_NULL;
  if (kind != HQ_GATE_NONE && !gate && M > 0) return HQ_ERR_NULL;
  return HQ_OK;
}

// A tensor [M, D] with row stride ld (elements).
hq_status check_rows(const void* x, int64_t M, int64_t D, int64_t ld, int es) {
  if (ld < D || ld > INT64_MAX / es || (M > 1 && ld > INT64_MAX / es / M)) return HQ_ERR_SHAPE;
  if (!aligned(x, 16) || (M > 1 && ld * es % 16 != 0)) return HQ_ERR_ALIGN;
  return HQ_OK;
}

hq_status check_params(hq_gate_kind kind, const void* gate, int64_t M, int64_t D, int64_t ld_gate, int es,
                       const void* w_post, const void* w_pre, int ps) {
  if (!aligned(w_post, ps) || !aligned(w_pre, ps)) return HQ_ERR_ALIGN;
  if (kind == HQ_GATE_FULL) return check_rows(gate, M, D, ld_gate, es);
  return kind != HQ_GATE_NONE && !aligned(gate, ps) ? HQ_ERR_ALIGN : HQ_OK;
}

}  // namespace

cudaError_t hq::norm_fault_word(unsigned int* fault, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(fault, g_hq_fault, sizeof(unsigned int));
  if (e == cudaSuccess && clear && *fault) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_hq_fault, &zero, sizeof(unsigned int));
  }
  return e;
}

extern "C" {

hq_status hq_block_norm(const void* h, int64_t ld_h, const void* y, int64_t ld_y, hq_dtype dtype, int64_t M, int64_t D,
                        const void* w_post, const void* w_pre, hq_dtype param_dtype, hq_gate_kind gate_kind,
                        const void* gate, int64_t ld_gate, int norms, float alpha, float eps, void* h_out, void* n,
                        float* r_post, float* r_pre, int group, float* amax, hq_stream stream) {
  const bool post = norms & HQ_NORM_POST, pre = norms & HQ_NORM_PRE;
  hq_status st = check_sizes(dtype, param_dtype, M, D, gate_kind, gate, y != nullptr || M == 0);
  if (st != HQ_OK) return st;
  if (norms & ~(HQ_NORM_POST | HQ_NORM_PRE)) return HQ_ERR_SHAPE;
  if (amax && group != 0 && group != 16 && group != 256) return HQ_ERR_GROUP;
  if (amax && D % (group ? group : 16) != 0) return HQ_ERR_SHAPE;
  if (amax && (!pre || !aligned(amax, 4))) return pre ? HQ_ERR_ALIGN : HQ_ERR_NULL;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (M == 0) {
    const cudaError_t e = amax ? cudaMemsetAsync(amax, 0, 4, cs) : cudaSuccess;
    return e == cudaSuccess ? HQ_OK : cuda_fail(e);
  }
  if (!h || (post && !y) || (!y && !pre) || (y && !h_out) || (post && !r_post) || (pre && (!n || !r_pre)))
    return HQ_ERR_NULL;
  const int es = dtype == HQ_BF16 ? 2 : 4, ps = param_dtype == HQ_BF16 ? 2 : 4;
  if ((st = check_rows(h, M, D, ld_h, es)) != HQ_OK) return st;
  if (y && (st = check_rows(y, M, D, ld_y, es)) != HQ_OK) return st;
  if ((st = check_params(gate_kind, gate, M, D, ld_gate, es, w_post, w_pre, ps)) != HQ_OK) return st;
  if (!aligned(h_out, 16) || !aligned(n, 16) || !aligned(r_post, 4) || !aligned(r_pre, 4)) return HQ_ERR_ALIGN;

  NormParams p = {};
  p.in[0] = static_cast<const uint8_t*>(h);
  p.in[1] = static_cast<const uint8_t*>(y);
  p.ld[0] = ld_h * es;
  p.ld[1] = ld_y * es;
  p.w_post = w_post;
  p.w_pre = w_pre;
  p.gate = gate;
  p.ld_gate = ld_gate * es;
  p.params_bf16 = param_dtype == HQ_BF16;
  p.gate_kind = gate_kind;
  p.post = post;
  p.pre = pre;
  p.has_y = y != nullptr;
  p.M = M;
  p.D = static_cast<int>(D);
  p.alpha = alpha;
  p.eps = eps;
  p.h_out = h_out;
  p.n = n;
  p.r_post = r_post;
  p.r_pre = r_pre;
  p.group = amax ? group : -1;
  p.amax = reinterpret_cast<unsigned*>(amax);
  int sms = 0;
  cudaError_t e = hq::sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e);
  const Shape s = shape_of(M, p.D, es, 2, sms);
  p.cols = s.cols;
  p.tpr = s.tpr;
  p.rows = s.rows;
  p.stages = s.stages;
  if (amax && (e = cudaMemsetAsync(amax, 0, 4, cs)) != cudaSuccess) return cuda_fail(e);
  int n_cl = 0;
  const bool plain = post && pre && y && !amax && (gate_kind == HQ_GATE_NONE || gate_kind == HQ_GATE_CHANNEL);
  if (dtype == HQ_BF16)
    e = plain ? (s.units == 1 ? launch(hq::k_block_norm<true, 1, true>, p, s, sms, &n_cl, cs)
                              : launch(hq::k_block_norm<true, 2, true>, p, s, sms, &n_cl, cs))
              : (s.units == 1 ? launch(hq::k_block_norm<true, 1, false>, p, s, sms, &n_cl, cs)
                              : launch(hq::k_block_norm<true, 2, false>, p, s, sms, &n_cl, cs));
  else
    e = plain ? (s.units == 1 ? launch(hq::k_block_norm<false, 1, true>, p, s, sms, &n_cl, cs)
                              : launch(hq::k_block_norm<false, 2, true>, p, s, sms, &n_cl, cs))
              : (s.units == 1 ? launch(hq::k_block_norm<false, 1, false>, p, s, sms, &n_cl, cs)
                              : launch(hq::k_block_norm<false, 2, false>, p, s, sms, &n_cl, cs));
  return e == cudaSuccess ? HQ_OK : cuda_fail(e);
}

int64_t hq_block_norm_bwd_workspace_bytes(int64_t M, int64_t D) {
  if (M < 0 || D <= 0 || D > kMaxD || D % 16 != 0) return -1;
  return 8 * D * (M < hq::kNormMaxPartials ? M : hq::kNormMaxPartials);
}

hq_status hq_block_norm_bwd(const void* dh_out, int64_t ld_dh, const void* dn, int64_t ld_dn, const void* h_out,
                            int64_t ld_h, const void* y, int64_t ld_y, hq_dtype dtype, int64_t M, int64_t D,
                            const void* w_post, const void* w_pre, hq_dtype param_dtype, hq_gate_kind gate_kind,
                            const void* gate, int64_t ld_gate, int norms, const float* r_post, const float* r_pre,
                            float alpha, void* dh, void* dy, float* dw_post, void* dgate, float* dw_pre,
                            void* workspace, hq_stream stream) {
  const bool post = norms & HQ_NORM_POST, pre = norms & HQ_NORM_PRE;
  hq_status st = check_sizes(dtype, param_dtype, M, D, gate_kind, gate, y != nullptr || M == 0);
  if (st != HQ_OK) return st;
  if (norms & ~(HQ_NORM_POST | HQ_NORM_PRE)) return HQ_ERR_SHAPE;
  const bool channel = gate_kind == HQ_GATE_CHANNEL;
  if (!aligned(dw_post, 4) || !aligned(dw_pre, 4) || !aligned(dgate, gate_kind == HQ_GATE_FULL ? 16 : 4)) return HQ_ERR_ALIGN;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (M == 0) {  // empty sums
    if (dw_post) e = cudaMemsetAsync(dw_post, 0, D * 4, cs);
    if (e == cudaSuccess && dw_pre) e = cudaMemsetAsync(dw_pre, 0, D * 4, cs);
    if (e == cudaSuccess && dgate && channel) e = cudaMemsetAsync(dgate, 0, D * 4, cs);
    return e == cudaSuccess ? HQ_OK : cuda_fail(e);
  }
  if ((!dh_out && !pre) || (pre && (!dn || !h_out || !r_pre)) || (post && (!y || !r_post)) || !dh || (y && !dy) ||
      (gate_kind != HQ_GATE_NONE && !dgate) || !workspace)
    return HQ_ERR_NULL;
  const int es = dtype == HQ_BF16 ? 2 : 4, ps = param_dtype == HQ_BF16 ? 2 : 4;
  if (dh_out && (st = check_rows(dh_out, M, D, ld_dh, es)) != HQ_OK) return st;
  if (pre && (st = check_rows(dn, M, D, ld_dn, es)) != HQ_OK) return st;
  if (pre && (st = check_rows(h_out, M, D, ld_h, es)) != HQ_OK) return st;
  if (y && (st = check_rows(y, M, D, ld_y, es)) != HQ_OK) return st;
  if ((st = check_params(gate_kind, gate, M, D, ld_gate, es, w_post, w_pre, ps)) != HQ_OK) return st;
  if (!aligned(dh, 16) || !aligned(dy, 16) || !aligned(workspace, 16) || !aligned(r_post, 4) || !aligned(r_pre, 4))
    return HQ_ERR_ALIGN;

  NormParams p = {};
  p.in[0] = pre ? static_cast<const uint8_t*>(h_out) : nullptr;
  p.in[1] = pre ? static_cast<const uint8_t*>(dn) : nullptr;
  p.in[2] = static_cast<const uint8_t*>(dh_out);
  p.in[3] = static_cast<const uint8_t*>(y);
  p.ld[0] = ld_h * es;
  p.ld[1] = ld_dn * es;
  p.ld[2] = ld_dh * es;
  p.ld[3] = ld_y * es;
  p.w_post = w_post;
  p.w_pre = w_pre;
  p.gate = gate;
  p.ld_gate = ld_gate * es;
  p.params_bf16 = param_dtype == HQ_BF16;
  p.gate_kind = gate_kind;
  p.post = post;
  p.pre = pre;
  p.has_y = y != nullptr;
  p.M = M;
  p.D = static_cast<int>(D);
  p.alpha = y ? alpha : 1.0f;
  p.r_post_in = r_post;
  p.r_pre_in = r_pre;
  p.dh = dh;
  p.dy = dy;
  p.dgate = dgate;
  p.partial = static_cast<float*>(workspace);
  int sms = 0;
  if ((e = hq::sm_count(&sms)) != cudaSuccess) return cuda_fail(e);
  const Shape s = shape_of(M, p.D, es, 4, sms);
  p.cols = s.cols;
  p.tpr = s.tpr;
  p.rows = s.rows;
  p.stages = s.stages;
  int n_cl = 0;
  const bool plain = post && pre && dh_out && (gate_kind == HQ_GATE_NONE || gate_kind == HQ_GATE_CHANNEL);
  if (dtype == HQ_BF16)
    e = plain ? (s.units == 1 ? launch(hq::k_block_norm_bwd<true, 1, true>, p, s, sms, &n_cl, cs)
                              : launch(hq::k_block_norm_bwd<true, 2, true>, p, s, sms, &n_cl, cs))
              : (s.units == 1 ? launch(hq::k_block_norm_bwd<true, 1, false>, p, s, sms, &n_cl, cs)
                              : launch(hq::k_block_norm_bwd<true, 2, false>, p, s, sms, &n_cl, cs));
  else
    e = plain ? launch(hq::k_block_norm_bwd<false, 1, true>, p, s, sms, &n_cl, cs)
              : launch(hq::k_block_norm_bwd<false, 1, false>, p, s, sms, &n_cl, cs);
  if (e != cudaSuccess) return cuda_fail(e);
  float* const to_pre = pre ? dw_pre : nullptr;
  float* const to_post = post ? dw_post : nullptr;
  float* const to_gate = channel ? static_cast<float*>(dgate) : nullptr;
  if (!to_pre && !to_post && !to_gate) return HQ_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((D + 31) / 32));
  cfg.blockDim = dim3(512);
  cfg.stream = cs;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, hq::k_norm_columns, const_cast<const float*>(p.partial), n_cl, p.D,
                         post ? w_post : static_cast<const void*>(nullptr),
                         channel ? gate : static_cast<const void*>(nullptr), p.params_bf16, to_pre, to_post, to_gate);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? HQ_OK : cuda_fail(e);
}

}  // extern "C"
