// hq_kv.cu -- C ABI of the paged NVFP4 cache of keys and values (include/hq.h) and its launch logic.  The kernels are
// in hq_kv.cuh, hq_kv_attend.cuh and hq_kv_prompt.cuh.
#include <cuda_runtime.h>

#include <cstdint>

#include "hq.h"
#include "hq_internal.h"
#include "hq_kv.cuh"
#include "hq_kv_attend.cuh"
#include "hq_kv_prompt.cuh"

namespace {

using hq::cuda_fail;

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxTokens = (int64_t{1} << 31) - 1024;  // counts of tokens and of rows (token, head)
constexpr int64_t kMaxHeads = 4096;
constexpr int64_t kMaxSequences = int64_t{1} << 20;  // a warp's way over idle ones ends long before a wait gives up
constexpr int64_t kMaxKeys = int64_t{1} << 25;  // of a sequence: its rows' way over them ends before a wait gives up

// Heads, head size, rotation group, pages.
hq_status check_cache(int64_t kv_heads, int64_t D, int group, int64_t pages, int64_t page_size) {
  if (kv_heads < 1 || kv_heads > kMaxHeads || (D != 64 && D != 128 && D != 256)) return HQ_ERR_SHAPE;
  if (group != 0 && group != 16 && group != 256) return HQ_ERR_GROUP;
  if (group == 256 && D != 256) return HQ_ERR_SHAPE;
  if (page_size < 16 || page_size % 16 != 0 || page_size > kMaxTokens || pages < 0) return HQ_ERR_SHAPE;
  if (pages > INT64_MAX / (18 * D) / kv_heads / page_size) return HQ_ERR_SHAPE;
  return HQ_OK;
}

template <typename Kernel, typename... Args>
cudaError_t launch(Kernel kernel, dim3 grid, int block, size_t smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(block));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

// Calls f with the head size, the rotation group and the element type as constants.
template <int D, typename F>
cudaError_t with_group(int group, bool bf16, F f) {
  using std::integral_constant;
  integral_constant<int, D> d;
  integral_constant<bool, true> yes;
  integral_constant<bool, false> no;
  if constexpr (D == 256)
    if (group == 256) return bf16 ? f(d, integral_constant<int, 256>(), yes) : f(d, integral_constant<int, 256>(), no);
  if (group == 16) return bf16 ? f(d, integral_constant<int, 16>(), yes) : f(d, integral_constant<int, 16>(), no);
  return bf16 ? f(d, integral_constant<int, 0>(), yes) : f(d, integral_constant<int, 0>(), no);
}
template <typename F>
cudaError_t with_sizes(int64_t D, int group, bool bf16, F f) {
  return D == 64 ? with_group<64>(group, bf16, f) : D == 128 ? with_group<128>(group, bf16, f) : with_group<256>(group, bf16, f);
}

// CTAs for rows of D channels, 16 per thread: as many as there are, up to what fills the SMs.
dim3 row_grid(int64_t rows, int64_t D, int sms) {
  const int64_t per = 256 / (D / 16), most = int64_t{16} * sms;
  return dim3(static_cast<unsigned>((rows + per - 1) / per < most ? (rows + per - 1) / per : most));
}

template <int D, int NT>
cudaError_t launch_attend(const hq::KvAttendParams& p, int sms, cudaStream_t stream) {
  using S = hq::KvAttendShape<D, NT>;
  auto kernel = hq::k_kv_attend<D, NT>;
  cudaError_t e = hq::allow_smem(reinterpret_cast<const void*>(kernel), S::kSmemBytes);
  if (e != cudaSuccess) return e;
  const int ctas = sms < hq::kKvMaxCtas ? sms : hq::kKvMaxCtas;
  if ((e = launch(kernel, dim3(ctas), S::kThreads, S::kSmemBytes, stream, p)) != cudaSuccess) return e;
  return launch(hq::k_kv_combine<D, NT>, dim3(ctas, S::kRows), 256, 0, stream, p);
}

template <int D, int SUB>
cudaError_t launch_prompt(const hq::KvAttendParams& p, int sms, cudaStream_t stream) {
  using S = hq::KvPromptShape<D, SUB>;
  auto kernel = hq::k_kv_prompt<D, SUB>;
  const size_t smem = S::kSmemBytes + 1024;
  cudaError_t e = hq::allow_smem(reinterpret_cast<const void*>(kernel), static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int ctas = sms < hq::kKvMaxCtas ? sms : hq::kKvMaxCtas;
  if ((e = launch(kernel, dim3(ctas), S::kThreads, smem, stream, p)) != cudaSuccess) return e;
  return launch(hq::k_kv_prompt_combine<D, SUB>, dim3(ctas, 8), 256, 0, stream, p);
}

// The kernel for few rows (query tokens x heads that share a key head) of a sequence, or the ones for many.  The one reads
// the keys again for every 16 rows (or takes 8 at a time: 31 us for 8 rows, D = 128, where the form of 16 takes 35); the
// others take 128 or 256 and little less time for fewer.  Those of 128, one tile, multiply the next scores while these are
// exponentiated; two tiles take turns, with the keys widened once for both.  Measured, us, few / one tile / two, of 32 query
// heads over 8 key heads:
//   rows                                      16                 32                48             128            400
//   16 sequences of 4096 keys, D = 64      34 / 44 / 54      51 / 44 / 54      67 / 44 / 54       44 / 54
//                              D = 128     38 / 57 / 90      61 / 57 / 91      84 / 57 / 92       58 / 93
//                              D = 256     62 / 112         106 / 113         151 / 114
//   64 sequences of 300 keys, D = 128      39 / 44 / 56      56 / 45 / 57      77 / 44 / 57       46 / 60
//   1 sequence of 65536 keys, D = 128      34 / 56 / 86      52 / 56 / 84      71 / 56 / 86       56 / 85
//   4 sequences of 4000 keys, D = 128                                                                            55 / 55
// and of 4 sequences of 1000 tokens behind 4000 (4000 rows) one tile 346, two 264.  One answer for all sequences of a call: 63
// single tokens of some 8192 keys take 153 by themselves and a prompt of 2048 tokens 65, both in one call 546.
bool few_rows(int64_t T, int64_t max_q, int64_t share, int64_t D) {
  return (max_q < T ? max_q : T) <= (D == 256 ? 32 : 16) / share;
}
bool one_tile(int64_t T, int64_t max_q, int64_t share, int64_t D) {
  return D == 256 || (max_q < T ? max_q : T) <= 128 / share;
}

}  // namespace

cudaError_t hq::kv_fault_word(unsigned int* fault, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(fault, g_hq_fault, sizeof(unsigned int));
  if (e == cudaSuccess && clear && *fault) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_hq_fault, &zero, sizeof(unsigned int));
  }
  return e;
}

extern "C" {

int64_t hq_kv_page_bytes(int64_t page_size, int64_t kv_heads, int64_t D) {
  return check_cache(kv_heads, D, 0, 1, page_size) == HQ_OK ? 18 * D / 16 * page_size * kv_heads : -1;
}

hq_status hq_kv_append_nvfp4(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v, int64_t ld_v,
                             hq_dtype dtype, int64_t T, int64_t q_heads, int64_t kv_heads, int64_t D, const float* cos,
                             const float* sin, int64_t table_rows, int64_t rotary, int interleaved,
                             const int32_t* positions, const int64_t* slots, int group, const float* kv_amax, void* q_out,
                             uint8_t* cache, int64_t pages, int64_t page_size, hq_stream stream) {
  if (dtype != HQ_F32 && dtype != HQ_BF16) return HQ_ERR_DTYPE;
  const hq_status st = check_cache(kv_heads, D, group, pages, page_size);
  if (st != HQ_OK) return st;
  if (T < 0 || T > kMaxTokens || q_heads < 0 || q_heads > kMaxHeads) return HQ_ERR_SHAPE;
  if (T * (q_heads + 2 * kv_heads) > kMaxTokens) return HQ_ERR_SHAPE;
  if (rotary < 0 || rotary > D || rotary % 16 != 0 || (rotary > 0 && table_rows < 1)) return HQ_ERR_SHAPE;
  if (T == 0) return HQ_OK;
  const int es = dtype == HQ_BF16 ? 2 : 4;
  const void* in[3] = {q, k, v};
  const int64_t ld[3] = {ld_q, ld_k, ld_v};
  for (int i = 0; i < 3; ++i) {
    const int64_t heads = i == 0 ? q_heads : kv_heads;
    if (heads == 0) continue;
    if (ld[i] < heads * D || ld[i] > INT64_MAX / es / T) return HQ_ERR_SHAPE;
  }
  if ((q_heads > 0 && (!q || !q_out)) || !k || !v || !slots || !kv_amax || (pages > 0 && !cache) ||
      (rotary > 0 && (!cos || !sin || !positions)))
    return HQ_ERR_NULL;
  for (int i = 0; i < 3; ++i)
    if ((i > 0 || q_heads > 0) && (!aligned(in[i], 16) || (T > 1 && ld[i] * es % 16 != 0))) return HQ_ERR_ALIGN;
  if (!aligned(q_out, 16) || !aligned(cache, 16) || !aligned(slots, 8) || !aligned(kv_amax, 4)) return HQ_ERR_ALIGN;
  if (rotary > 0 && (!aligned(cos, 16) || !aligned(sin, 16) || !aligned(positions, 4))) return HQ_ERR_ALIGN;
  hq::KvAppendParams p = {};
  for (int i = 0; i < 3; ++i) {
    p.in[i] = static_cast<const uint8_t*>(in[i]);
    p.ld[i] = ld[i] * es;
    p.heads[i] = static_cast<int>(i == 0 ? q_heads : kv_heads);
  }
  p.T = T;
  p.cos_t = cos;
  p.sin_t = sin;
  p.rows = table_rows;
  p.rotary = static_cast<int>(rotary);
  p.interleaved = interleaved != 0;
  p.positions = positions;
  p.slots = slots;
  p.kv_amax = kv_amax;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.cache = cache;
  p.n_slots = pages * page_size;
  p.page_units = static_cast<int>(page_size / 16);
  p.kv_heads = static_cast<int>(kv_heads);
  int sms = 0;
  cudaError_t e = hq::sm_count(&sms);
  if (e == cudaSuccess)
    e = with_sizes(D, group, dtype == HQ_BF16, [&](auto d, auto g, auto b) {
      auto kernel = rotary == D && !interleaved ? hq::k_kv_append<d, g, b, true> : hq::k_kv_append<d, g, b, false>;
      return launch(kernel, row_grid(T * (q_heads + 2 * kv_heads), D, sms), 256, 0,
                    static_cast<cudaStream_t>(stream), p);
    });
  return e == cudaSuccess ? HQ_OK : cuda_fail(e);
}

hq_status hq_kv_read_nvfp4(const uint8_t* cache, int64_t pages, int64_t page_size, int64_t kv_heads, int64_t D,
                           const int64_t* slots, int64_t T, const float* kv_amax, int group, void* k, void* v,
                           hq_dtype out_dtype, hq_stream stream) {
  if (out_dtype != HQ_F32 && out_dtype != HQ_BF16) return HQ_ERR_DTYPE;
  const hq_status st = check_cache(kv_heads, D, group, pages, page_size);
  if (st != HQ_OK) return st;
  if (T < 0 || T > kMaxTokens || T * kv_heads > kMaxTokens) return HQ_ERR_SHAPE;
  if (T == 0) return HQ_OK;
  if (!slots || !kv_amax || !k || !v || (pages > 0 && !cache)) return HQ_ERR_NULL;
  if (!aligned(cache, 16) || !aligned(slots, 8) || !aligned(kv_amax, 4) || !aligned(k, 16) || !aligned(v, 16)) return HQ_ERR_ALIGN;
  hq::KvReadParams p = {};
  p.cache = cache;
  p.slots = slots;
  p.kv_amax = kv_amax;
  p.T = T;
  p.n_slots = pages * page_size;
  p.page_units = static_cast<int>(page_size / 16);
  p.kv_heads = static_cast<int>(kv_heads);
  p.k = k;
  p.v = v;
  int sms = 0;
  cudaError_t e = hq::sm_count(&sms);
  if (e == cudaSuccess)
    e = with_sizes(D, group, out_dtype == HQ_BF16, [&](auto d, auto g, auto b) {
      return launch(hq::k_kv_read<d, g, b>, row_grid(T * kv_heads, D, sms), 256, 0, static_cast<cudaStream_t>(stream), p);
    });
  return e == cudaSuccess ? HQ_OK : cuda_fail(e);
}

int64_t hq_kv_attention_workspace_bytes(int64_t q_heads, int64_t kv_heads, int64_t D, int64_t T, int64_t max_q) {
  if (check_cache(kv_heads, D, 0, 0, 16) != HQ_OK || q_heads < 1 || q_heads > kMaxHeads || q_heads % kv_heads != 0) return -1;
  if (T < 0 || T * (q_heads / kv_heads) > kMaxTokens || T > kMaxTokens || max_q < 0) return -1;
  return few_rows(T, max_q, q_heads / kv_heads, D) ? hq::kv_part_bytes(static_cast<int>(D)) : hq::kv_prompt_bytes(static_cast<int>(D));
}

hq_status hq_kv_attention_nvfp4(const void* q, int64_t ld_q, int64_t T, int64_t q_heads, const uint8_t* cache, int64_t pages,
                                int64_t page_size, int64_t kv_heads, int64_t D, const int32_t* page_table, int64_t ld_table,
                                int64_t table_pages, const int32_t* kv_len, const int32_t* q_start, int64_t S, int64_t max_q,
                                const float* kv_amax, float scale, int64_t window, int group, void* out, float* lse,
                                void* workspace, hq_stream stream) {
  const hq_status st = check_cache(kv_heads, D, group, pages, page_size);
  if (st != HQ_OK) return st;
  if (T < 0 || T > kMaxTokens || S < 0 || S > kMaxSequences || q_heads < 1 || q_heads > kMaxHeads || q_heads % kv_heads != 0)
    return HQ_ERR_SHAPE;
  if (T * (q_heads / kv_heads) > kMaxTokens || max_q < 0 || window < 0) return HQ_ERR_SHAPE;
  if (table_pages < 0 || ld_table < table_pages || table_pages > kMaxKeys / page_size || (table_pages > 0 && pages == 0))
    return HQ_ERR_SHAPE;
  if (T == 0 || S == 0) return HQ_OK;
  if (ld_q < q_heads * D || ld_q > INT64_MAX / 2 / T || ld_table > INT64_MAX / 4 / S) return HQ_ERR_SHAPE;
  if (!q || !out || !kv_len || !q_start || !kv_amax || !workspace || (table_pages > 0 && (!page_table || !cache))) return HQ_ERR_NULL;
  if (!aligned(q, 16) || (T > 1 && ld_q * 2 % 16 != 0) || !aligned(cache, 16) || !aligned(page_table, 4) || !aligned(kv_len, 4) ||
      !aligned(q_start, 4) || !aligned(kv_amax, 4) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 16))
    return HQ_ERR_ALIGN;
  hq::KvAttendParams p = {};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.ld_q = ld_q;
  p.cache = cache;
  p.pages = pages;
  p.page_units = static_cast<int>(page_size / 16);
  p.table = page_table;
  p.ld_table = ld_table;
  p.most = static_cast<int>(table_pages * page_size);
  p.kv_len = kv_len;
  p.q_start = q_start;
  p.S = static_cast<int>(S);
  p.T = static_cast<int>(T);
  p.heads = static_cast<int>(q_heads);
  p.kv_heads = static_cast<int>(kv_heads);
  p.share = static_cast<int>(q_heads / kv_heads);
  p.kv_amax = kv_amax;
  p.scale = scale;
  // (A window that no key leaves is none; others are below 2^25, far from where differences with them would leave 32 bits.)
  p.window = static_cast<int>(window < p.most ? window : 0);
  p.group = group;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.part = static_cast<float*>(workspace);
  int sms = 0;
  cudaError_t e = hq::sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (!few_rows(T, max_q, p.share, D))
    e = !one_tile(T, max_q, p.share, D) ? (D == 64 ? launch_prompt<64, 2>(p, sms, cs) : launch_prompt<128, 2>(p, sms, cs))
        : D == 64 ? launch_prompt<64, 1>(p, sms, cs) : D == 128 ? launch_prompt<128, 1>(p, sms, cs) : launch_prompt<256, 1>(p, sms, cs);
  else if ((max_q < T ? max_q : T) * p.share <= 8)
    e = D == 64 ? launch_attend<64, 1>(p, sms, cs) : D == 128 ? launch_attend<128, 1>(p, sms, cs) : launch_attend<256, 1>(p, sms, cs);
  else
    e = D == 64 ? launch_attend<64, 2>(p, sms, cs) : D == 128 ? launch_attend<128, 2>(p, sms, cs) : launch_attend<256, 2>(p, sms, cs);
  return e == cudaSuccess ? HQ_OK : cuda_fail(e);
}

}  // extern "C"
