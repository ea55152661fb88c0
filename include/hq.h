/*
 * hq.h -- C ABI of libhq: fused Hadamard rotation + NVFP4 quantization on GB300 (sm_103a).
 *
 * What is computed ("A Fused Hadamard + NVFP4 Quantization Kernel in Triton", §1 "The format,
 * precisely" and §2 "The kernel"; storage layout from "NVFP4 Quantization" (Atlas docs),
 * "The numeric format"):
 *
 *   x       : M x K activations, row-major, row stride ldx elements (ldx >= K).
 *   rotation: every run of G consecutive elements of a row is multiplied by the
 *             Sylvester-Hadamard matrix H_G scaled by 1/sqrt(G):  y = x . H_G / sqrt(G).
 *             G = 16, G = 256 (= H16 (x) H16, scaled by 1/16), or G = 0 (rotation off: y = x).
 *             Computed as a fixed-order fp32 butterfly: stages h = 1, 2, 4, ..., G/2, each
 *             (a, b) -> (a + b, a - b), then one multiply by 1/sqrt(G).
 *   amax    : max |y| over the whole tensor (exact).
 *   s_global: amax / (448 * 6) in one fp32 division; 1.0 if that quotient is 0.
 *   blocks  : every 16 consecutive elements of a row of y form one NVFP4 block.
 *   s_block : E4M3 (float8 e4m3fn) value nearest to (block_amax / 6) / s_global, ties to even,
 *             saturating at 448.  Stored as its 8-bit pattern.
 *   codes   : s_f = s_block * s_global; if s_f == 0 every code of the block is 0, otherwise
 *             code = E2M1 value nearest to y / s_f (IEEE fp32 division), grid
 *             {0, .5, 1, 1.5, 2, 3, 4, 6}, ties to the even code, saturating at 6; bit 3 copies
 *             the sign bit of the quotient (so -0.0 encodes as 0x8).
 *   packing : q[r][j] = code[r][2j] | (code[r][2j+1] << 4)   (even element in the low nibble).
 *
 * Layouts (all row-major, contiguous, owned by the caller):
 *   q       : uint8 [M, K/2]
 *   scales  : uint8 [M, K/16]  (E4M3 bit patterns)
 *
 * Conventions shared by every entry point:
 *   - Every pointer is a DEVICE pointer owned by the caller.  The library allocates no memory,
 *     creates no stream and never synchronises the host; all work is enqueued on `stream`
 *     (a cudaStream_t / CUstream of the current device; NULL = the legacy default stream).
 *   - Argument errors are detected on the host before anything is enqueued and are returned
 *     synchronously; nothing is launched in that case.
 *   - A failed launch returns HQ_ERR_CUDA; hq_last_cuda_error() then gives the cudaError_t.
 *   - An empty tensor (M == 0 or K == 0, with valid sizes) is a no-op that returns HQ_OK; its
 *     data pointers may be NULL.  hq_rot_amax still writes 0 to `amax`, which must be valid.
 *   - Non-finite input is outside the contract.  hq_rot_amax reports it: a NaN anywhere gives
 *     a NaN amax and an infinity gives +inf, which the caller can read back.  Codes and scales
 *     for such tensors are unspecified.  Nothing traps or waits on the device.
 *   - Sizes are 64-bit element counts.
 */
#ifndef HQ_H_
#define HQ_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define HQ_API __attribute__((visibility("default")))
#else
#define HQ_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  HQ_OK = 0,
  HQ_ERR_NULL = 1,  /* a required pointer is NULL */
  HQ_ERR_SHAPE = 2, /* M < 0, K < 0, ldx < K, K not a multiple of max(16, G), M * K beyond
                       int64, or, in the calls that read x, K >= 2^36 (a row of 2^32 or
                       more 16-element blocks) */
  HQ_ERR_ALIGN = 3, /* a pointer or the row stride breaks the alignment rules below */
  HQ_ERR_DTYPE = 4, /* unknown element type */
  HQ_ERR_GROUP = 5, /* rotation group not in {0, 16, 256} */
  HQ_ERR_CUDA = 6,  /* the CUDA runtime refused a launch or an enqueue */
  HQ_ERR_TOO_LARGE = 7, /* the tensor does not fit the fixed scratch of
                           hq_quantize_nvfp4_host_noalloc */
  HQ_ERR_ALIAS = 8      /* two buffers that must be distinct are the same */
} hq_status;

typedef enum {
  HQ_F32 = 0, /* IEEE binary32 */
  HQ_BF16 = 1 /* bfloat16; widened to fp32 exactly */
} hq_dtype;

/* A cudaStream_t (CUstream) passed as a plain pointer. */
typedef void* hq_stream;

/*
 * hq_rot_amax -- pass 1: rotate and reduce the global amax.
 *   ("A Fused Hadamard + NVFP4 Quantization Kernel in Triton", §2, "The global scale is the one
 *    thing not fused": the amax of the whole rotated tensor is needed before any block scale.)
 *
 *   x      : [M, K] of `dtype`, row stride ldx elements.  16-byte aligned; ldx * sizeof(dtype)
 *            a multiple of 16 bytes.
 *   group  : 0, 16 or 256.  K must be a multiple of max(16, group).
 *   amax   : 1 float, overwritten with max |y| (this call zeroes it first, on `stream`).
 *            4-byte aligned.
 *   y      : optional fp32 [M, K] (row stride K), 16-byte aligned, receives the rotated tensor;
 *            NULL to skip (the normal case: the rotation is never stored).
 */
HQ_API hq_status hq_rot_amax(const void* x, hq_dtype dtype, int64_t M, int64_t K, int64_t ldx,
                      int group, float* amax, float* y, hq_stream stream);

/*
 * hq_rotate_quant_nvfp4 -- pass 2: one read of x, one write of the codes and block scales.
 *   ("A Fused Hadamard + NVFP4 Quantization Kernel in Triton", §1 table and §2 kernel: rotate,
 *    block amax, E4M3 scale, E2M1 codes, two codes per byte.)
 *
 *   x, dtype, M, K, ldx, group : as for hq_rot_amax.
 *   amax     : 1 float on the device, the global amax of the rotated tensor (normally written by
 *              hq_rot_amax on the same stream; any non-negative finite value is accepted, e.g.
 *              an amax kept from an earlier step).
 *   q        : uint8 [M, K/2], 16-byte aligned.
 *   scales   : uint8 [M, K/16], 4-byte aligned.
 *   s_global : optional 1 float, receives s_global (the per-tensor fp32 scale); NULL to skip.
 */
HQ_API hq_status hq_rotate_quant_nvfp4(const void* x, hq_dtype dtype, int64_t M, int64_t K,
                                int64_t ldx, int group, const float* amax, uint8_t* q,
                                uint8_t* scales, float* s_global, hq_stream stream);

/* Size of the workspace of hq_quantize_nvfp4 and the _ws entry points (hq_rotate_quant_nvfp4_ws,
 * hq_rotate_quant_nvfp4_swizzled_ws, hq_rotate_quant_nvfp4_delayed_ws, hq_rotate_quant_mxfp4_ws),
 * in 32-bit words
 * (control words and the counters of the run-time tile schedule, each on its own 128-byte
 * line). */
#define HQ_QUANTIZE_WORKSPACE_WORDS 288

/*
 * hq_quantize_nvfp4 -- both passes in one call: *amax, then codes, scales and s_global exactly as
 *   hq_rot_amax followed by hq_rotate_quant_nvfp4 on the same stream.
 *   ("A Fused Hadamard + NVFP4 Quantization Kernel in Triton", §2: the global scale needs the
 *    amax of the whole rotated tensor before any block is quantized, hence two passes over x.)
 *
 *   Two launches, pass 1 then pass 2.  With `workspace`, pass 1 reduces the amax into the
 *   workspace and its last CTA writes *amax (no memset before it); pass 2 is
 *   hq_rotate_quant_nvfp4_ws (tiles handed out at run time) and fetches its first tiles of x
 *   while pass 1 ends; both launches are programmatic dependents of the kernel before them on
 *   the stream (each waits for that kernel to complete before it reads what the kernel
 *   wrote).  Without, pass 1 is hq_rot_amax and pass 2 hq_rotate_quant_nvfp4.
 *
 *   x, dtype, M, K, ldx, group : as for hq_rot_amax.
 *   amax      : 1 float on the device (written; 0 for an empty tensor).
 *   q, scales, s_global : as for hq_rotate_quant_nvfp4.
 *   workspace : NULL (hq_rot_amax then hq_rotate_quant_nvfp4), or HQ_QUANTIZE_WORKSPACE_WORDS
 *               uint32 on the device, 4-byte aligned, all 0 before its first use (e.g.
 *               cudaMemset).  Each call that records no fault leaves it 0 again.  Calls that may
 *               run at the same time (different streams) need different workspaces.
 */
HQ_API hq_status hq_quantize_nvfp4(const void* x, hq_dtype dtype, int64_t M, int64_t K,
                                   int64_t ldx, int group, float* amax, uint8_t* q,
                                   uint8_t* scales, float* s_global, uint32_t* workspace,
                                   hq_stream stream);

/*
 * hq_rotate_quant_nvfp4_ws -- pass 2 exactly as hq_rotate_quant_nvfp4 (same arguments, same
 *   outputs), with the tiles of x handed to the warps at run time instead of by a fixed split.
 *   (Not a step of the pages' method: a schedule.  With a fixed split the warps of an SM
 *   advance at different speeds, and the last ones still run while the others have left,
 *   with the memory system part idle.  Here each warp takes its next tile from a counter in
 *   `workspace`, so all warps run out of work at about the same time.)
 *
 *   workspace : HQ_QUANTIZE_WORKSPACE_WORDS uint32 on the device, 4-byte aligned, all 0 before
 *               its first use (e.g. cudaMemset); each call that records no fault leaves it 0
 *               again.  Calls that may run at the same time (different streams) need different
 *               workspaces; hq_quantize_nvfp4's may be shared with it on one stream.
 *               NULL: the fixed split of hq_rotate_quant_nvfp4.
 */
HQ_API hq_status hq_rotate_quant_nvfp4_ws(const void* x, hq_dtype dtype, int64_t M, int64_t K,
                                          int64_t ldx, int group, const float* amax, uint8_t* q,
                                          uint8_t* scales, float* s_global, uint32_t* workspace,
                                          hq_stream stream);

/*
 * hq_rotate_quant_nvfp4_swizzled -- pass 2 exactly as hq_rotate_quant_nvfp4, with the E4M3 block
 * scales written straight into the tiled layout that block-scaled NVFP4 GEMMs read.
 *   ("A Fused Hadamard + NVFP4 Quantization Kernel in Triton", §6 "From interpreter to
 *    hardware", Layout: cuBLASLt and CUTLASS take the block scales in a swizzled tiled layout,
 *    and a production kernel writes it directly; the page does not spell the layout out.  The
 *    layout here is cuBLASLt's for 16-element block scales; the GPU tests check it by feeding
 *    the output to cuBLASLt's NVFP4 GEMM.)
 *
 *   scales : hq_swizzled_scales_bytes(M, K) bytes, 32-byte aligned.  The [M, K/16] scale
 *            matrix is padded to R = round_up(M, 128) rows and C = round_up(K/16, 4) columns
 *            and cut into tiles of 128 rows x 4 columns; tile (i, j) is the 512 bytes at
 *            (i * C/4 + j) * 512, and inside it row r, column c (r < 128, c < 4) is the byte
 *            (r % 32) * 16 + (r / 32) * 4 + c.  Every byte is written, padding entries as 0
 *            (a GEMM reads them).
 *   Everything else (x, amax, q, s_global, group, errors) as hq_rotate_quant_nvfp4.
 */
HQ_API hq_status hq_rotate_quant_nvfp4_swizzled(const void* x, hq_dtype dtype, int64_t M,
                                                int64_t K, int64_t ldx, int group,
                                                const float* amax, uint8_t* q, uint8_t* scales,
                                                float* s_global, hq_stream stream);

/*
 * hq_rotate_quant_nvfp4_swizzled_ws -- hq_rotate_quant_nvfp4_swizzled exactly (same arguments,
 *   same outputs), with its units of work (8 rows x 128 blocks) handed to the warps at run time
 *   as in hq_rotate_quant_nvfp4_ws (a schedule, not a step of the method).
 *   workspace : as for hq_rotate_quant_nvfp4_ws.  NULL: hq_rotate_quant_nvfp4_swizzled.
 */
HQ_API hq_status hq_rotate_quant_nvfp4_swizzled_ws(const void* x, hq_dtype dtype, int64_t M,
                                                   int64_t K, int64_t ldx, int group,
                                                   const float* amax, uint8_t* q,
                                                   uint8_t* scales, float* s_global,
                                                   uint32_t* workspace, hq_stream stream);

/* Size in bytes of the swizzled scale buffer for an [M, K] tensor (-1 if M < 0, K < 0,
 * K % 16 != 0, or the size does not fit int64). */
HQ_API int64_t hq_swizzled_scales_bytes(int64_t M, int64_t K);

/*
 * hq_rotate_quant_nvfp4_delayed -- single-pass mode: quantize with an amax kept from an earlier
 *   step while reducing this tensor's amax for the next one.
 *   ("A Fused Hadamard + NVFP4 Quantization Kernel in Triton", §2, on the global scale:
 *    production stacks run a small amax reduction ahead of the kernel *or reuse an amax from a
 *    previous step*, so that the per-block work stays a single pass.)
 *
 *   Reads x once.  Codes, scales and s_global are exactly those of hq_rotate_quant_nvfp4 with
 *   amax = *amax_prev; *amax_next receives max |y| of this tensor, exactly as hq_rot_amax would
 *   (this call zeroes it first, on `stream`).  When *amax_prev is smaller than this tensor's
 *   amax, blocks whose scale would exceed 448 saturate (scale 448, codes clipped at 6): the
 *   price of a stale global scale.
 *
 *   x, dtype, M, K, ldx, group, q, scales, s_global : as for hq_rotate_quant_nvfp4.
 *   amax_prev : 1 float on the device (read).      amax_next : 1 float on the device (written).
 *   The two must be different floats; passing the same pointer returns HQ_ERR_ALIAS.
 */
HQ_API hq_status hq_rotate_quant_nvfp4_delayed(const void* x, hq_dtype dtype, int64_t M,
                                               int64_t K, int64_t ldx, int group,
                                               const float* amax_prev, float* amax_next,
                                               uint8_t* q, uint8_t* scales, float* s_global,
                                               hq_stream stream);

/*
 * hq_rotate_quant_nvfp4_delayed_ws -- hq_rotate_quant_nvfp4_delayed exactly (same arguments, same
 *   outputs), with a workspace: the tiles of x are handed to the warps at run time as in
 *   hq_rotate_quant_nvfp4_ws, and *amax_next is reduced in the workspace and written by the
 *   kernel's last CTA, so no memset runs before it (one launch per call).
 *   workspace : as for hq_rotate_quant_nvfp4_ws.  NULL: hq_rotate_quant_nvfp4_delayed.
 */
HQ_API hq_status hq_rotate_quant_nvfp4_delayed_ws(const void* x, hq_dtype dtype, int64_t M,
                                                  int64_t K, int64_t ldx, int group,
                                                  const float* amax_prev, float* amax_next,
                                                  uint8_t* q, uint8_t* scales, float* s_global,
                                                  uint32_t* workspace, hq_stream stream);

/*
 * hq_rotate_quant_mxfp4 -- MXFP4 variant: E2M1 codes with one power-of-two (E8M0) scale per 32
 *   consecutive elements of a row and no per-tensor scale, so a single pass over x.
 *   ("A Fused Hadamard + NVFP4 Quantization Kernel in Triton", §1: MXFP4 has 32-element blocks and
 *    power-of-two E8M0 scales; "Try this": the error study with MXFP4 semantics.)
 *   The pages give no rule for the scale; this library uses the usual MX rule:
 *   X = 2^(floor(log2 amax_32) - 2), so amax_32 / X lies in [4, 8) (2 is the exponent of E2M1's
 *   largest value, 6); the stored byte is the exponent + 127, clamped to [0, 254] (0 for an
 *   all-zero block); codes = E2M1(y / X) as for NVFP4 (ties to even, saturating at 6, sign bit
 *   copied).  The rotation is as for NVFP4 (group 0, 16 or 256).
 *
 *   x, dtype, M, K, ldx, group : as for hq_rotate_quant_nvfp4, with K a multiple of 32 as well.
 *   q      : uint8 [M, K/2], 16-byte aligned (same packing as NVFP4).
 *   scales : uint8 [M, K/32] E8M0 bytes.
 */
HQ_API hq_status hq_rotate_quant_mxfp4(const void* x, hq_dtype dtype, int64_t M, int64_t K,
                                       int64_t ldx, int group, uint8_t* q, uint8_t* scales,
                                       hq_stream stream);

/*
 * hq_rotate_quant_mxfp4_ws -- hq_rotate_quant_mxfp4 exactly (same arguments, same outputs), with
 *   the tiles of x handed to the warps at run time as in hq_rotate_quant_nvfp4_ws (a schedule,
 *   not a step of the method).
 *   workspace : as for hq_rotate_quant_nvfp4_ws (HQ_QUANTIZE_WORKSPACE_WORDS uint32, all 0
 *               before its first use and left 0 by each call that records no fault; one per
 *               stream that may run at the same time).  NULL: hq_rotate_quant_mxfp4.
 */
HQ_API hq_status hq_rotate_quant_mxfp4_ws(const void* x, hq_dtype dtype, int64_t M, int64_t K,
                                          int64_t ldx, int group, uint8_t* q, uint8_t* scales,
                                          uint32_t* workspace, hq_stream stream);

/* hq_dequant_mxfp4 -- value = (+-grid[code & 7]) * 2^(byte - 127), then the rotation again when
 * `unrotate` (group 16 or 256).  out: fp32 [M, K], 16-byte aligned; q 8-byte aligned. */
HQ_API hq_status hq_dequant_mxfp4(const uint8_t* q, const uint8_t* scales, int64_t M, int64_t K,
                                  int group, int unrotate, float* out, hq_stream stream);

/*
 * hq_rotate_quant_int8 -- INT8 per-token rotate-quant with the regular Hadamard.
 *   ("hyperflow_h3_flash_int8.py", HyperFlow: regular_hadamard, rotate_quant_kernel; the
 *    activation side of a W8A8 linear whose weight was rotated offline.)
 *
 *   y      = x . R_G on every run of G consecutive channels of a row, R_G = kron(H4/2, ...)
 *            (log4 G factors), H4 = [[1,1,1,-1],[1,1,-1,1],[1,-1,1,1],[-1,1,1,1]] (orthonormal,
 *            symmetric, rows summing to one).  Fixed fp32 order: the base-4 digits of the
 *            channel index from the least significant, each 4-point step out_k = RN(S/2 -
 *            v_(3-k)), S = (v0 + v1) + (v2 + v3).  (The page's group of 1024 is computed from
 *            its 16 x 64 factors; the Kronecker power is the same matrix, and the digit order
 *            fixes the rounding.)
 *   scales : fp32 [M], scale = max(amax_row |y|, 1e-12) / 127.
 *   q      : int8 [M, K] row-major, q = clamp(rint(y * (1/scale)), -127, 127) (half to even).
 *   For K <= 120832, x is read once and the rotated row stays on chip until its amax is known
 *   (tensor memory up to 32768 channels, tensor and shared memory beyond); a longer row is read
 *   twice, first for its amax and then to quantize it (the second read mostly from L2).
 *
 *   group  : 4, 16, 64, 256 or 1024; K a multiple of the group and of 16 (the kernels move
 *            whole 16-channel blocks), K / 2048 below 2^30.
 *   x      : [M, K] of dtype, row stride ldx (16-byte aligned; ldx * sizeof(dtype) % 16 == 0).
 *   q      : 16-byte aligned.   scales : 4-byte aligned.
 */
HQ_API hq_status hq_rotate_quant_int8(const void* x, hq_dtype dtype, int64_t M, int64_t K,
                                      int64_t ldx, int group, int8_t* q, float* scales,
                                      hq_stream stream);

/*
 * hq_dequant_nvfp4 -- round trip for checks (not part of the quantization hot path).
 *   ("A Fused Hadamard + NVFP4 Quantization Kernel in Triton", §2 dequantize:
 *    value = (+-grid[code & 7]) * (s_block * s_global), then the rotation applied again when the
 *    data was rotated; H_G / sqrt(G) is symmetric and orthonormal, so it is its own inverse.)
 *
 *   q, scales : as written by hq_rotate_quant_nvfp4 (q 8-byte aligned).
 *   s_global  : 1 float on the device.
 *   group     : 0, 16 or 256; the rotation to undo when `unrotate` is non-zero (then 16 or 256,
 *               and K a multiple of it); otherwise only checked.
 *   out       : fp32 [M, K] (row stride K), 16-byte aligned.
 *   The two products are rounded in that order (s_f first), then the butterfly as above.
 */
HQ_API hq_status hq_dequant_nvfp4(const uint8_t* q, const uint8_t* scales, const float* s_global,
                           int64_t M, int64_t K, int group, int unrotate, float* out,
                           hq_stream stream);

/*
 * Products of the codes.
 *
 * The calls below multiply matrices of E2M1 codes with block scales, as the quantizing calls
 * above write them, on the tensor cores: exact products of codes and scales, fp32 sums, the
 * product of the per-tensor scales applied in fp32, one rounding to the output's type.  A
 * rotation of both operands by the same orthonormal symmetric H along the summed axis cancels
 * ((x H)(w H)^T = x w^T), so operands are rotated alike or not at all.
 *
 * No gradient passes through the codes.  A training step's three products are three calls:
 * y = hq_grouped_gemm(x, w); dx = hq_grouped_gemm(dy quantized along N, w^T quantized along N);
 * dw = hq_grouped_wgrad(dy^T, x^T, both quantized along the tokens).
 *
 * Shared by them:
 *   - Codes: two per byte, even element in the low nibble, rows contiguous, 16-byte aligned.
 *   - Scales "in the tile layout" are those of hq_rotate_quant_nvfp4_swizzled, or of
 *     hq_swizzle_scales for either format: padding entries must be 0.  32-byte aligned.
 *   - offsets: int32 [E + 1] on the device, non-decreasing from 0: group e is the half-open range
 *     offsets[e] .. offsets[e + 1].  Values outside the tensor are clamped to it; the host never
 *     reads them.  E <= 512.
 *   - out_dtype: HQ_BF16 or HQ_F32; out is row-major and contiguous, aligned to its element.
 *   - Sizes beyond 2^31 - 1024 return HQ_ERR_SHAPE.
 *   - A launch may start while the kernel before it on the stream ends; it waits for that kernel
 *     before it reads.
 */

/*
 * hq_grouped_gemm_nvfp4 -- products grouped by expert, ragged rows (NVFP4 operands):
 *   out[m, n] = x_sg * w_sg[e] * sum_k x[m, k] w[e, n, k]    for the rows m of group e.
 *   Rows that belong to no group are not written.  An empty group costs nothing.
 *
 *   xq [M, K/2], xs [M, K/16] row-major (hq_quantize_nvfp4, hq_rotate_quant_nvfp4), x_sg 1 float;
 *   wq [E, N, K/2], ws E buffers of hq_swizzled_scales_bytes(N, K) in the tile layout, w_sg E
 *   floats; out [M, N].  K a multiple of 32; K == 0 zeroes out.
 *   workspace : hq_grouped_gemm_workspace_bytes(M, N, K, E) bytes, 32-byte aligned; contents need no
 *               preparation (large groups: x's scales in the tile layout).  Calls that may run at the
 *               same time need different ones.
 */
HQ_API hq_status hq_grouped_gemm_nvfp4(const uint8_t* xq, const uint8_t* xs, const float* x_sg,
                                       const uint8_t* wq, const uint8_t* ws, const float* w_sg,
                                       const int32_t* offsets, int64_t M, int64_t N, int64_t K,
                                       int64_t E, void* out, hq_dtype out_dtype, void* workspace,
                                       hq_stream stream);

/* Bytes of hq_grouped_gemm's workspace: 0 for a few rows per expert (workspace may then be NULL), -1
 * for sizes it refuses. */
HQ_API int64_t hq_grouped_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t E);

/* hq_grouped_gemm_mxfp4 -- the same for MXFP4 operands: xs [M, K/32], ws E buffers of
 * hq_swizzled_scales_bytes(N, K/2) (hq_swizzle_scales of [E, N, K/32]), no per-tensor scales. */
HQ_API hq_status hq_grouped_gemm_mxfp4(const uint8_t* xq, const uint8_t* xs, const uint8_t* wq,
                                       const uint8_t* ws, const int32_t* offsets, int64_t M,
                                       int64_t N, int64_t K, int64_t E, void* out,
                                       hq_dtype out_dtype, void* workspace, hq_stream stream);

/*
 * hq_grouped_wgrad_nvfp4 -- the weights' gradients of the products above: the summed axis is the
 * ragged one.
 *   out[e, n, k] = g_sg * x_sg * sum_{t in group e} g[n, t] x[k, t];   0 for an empty group.
 *
 *   gq [N, T/2] and xq [K, T/2]: dy and x transposed, quantized (and rotated) along the tokens;
 *   gs, xs: hq_swizzled_scales_bytes(N, T) and (K, T) in the tile layout; out [E, N, K].  Each
 *   expert's tokens are padded with zeros to a multiple of 128, so T and the offsets are multiples
 *   of 128 (other offsets are rounded down).
 */
HQ_API hq_status hq_grouped_wgrad_nvfp4(const uint8_t* gq, const uint8_t* gs, const float* g_sg,
                                        const uint8_t* xq, const uint8_t* xs, const float* x_sg,
                                        const int32_t* offsets, int64_t T, int64_t N, int64_t K,
                                        int64_t E, void* out, hq_dtype out_dtype, hq_stream stream);

/* hq_grouped_wgrad_mxfp4 -- the same for MXFP4 operands (scales hq_swizzled_scales_bytes(N, T/2) and
 * (K, T/2)). */
HQ_API hq_status hq_grouped_wgrad_mxfp4(const uint8_t* gq, const uint8_t* gs, const uint8_t* xq,
                                        const uint8_t* xs, const int32_t* offsets, int64_t T,
                                        int64_t N, int64_t K, int64_t E, void* out,
                                        hq_dtype out_dtype, hq_stream stream);

/*
 * hq_lora_gemm_nvfp4 -- a shared projection with the low-rank adapters of many requests (NVFP4
 * projection, bf16 adapters):
 *   out[m, n] = x_sg * w_sg * sum_k xq[m, k] wq[n, k] + scaling[a] * sum_r (sum_k x[m, k] A_a[r, k]) B_a[n, r]
 *   with a = row_adapter[m]; no second term where a is negative or not below `adapters`.
 *   Both terms are added in fp32 before the one rounding to out_dtype; the inner sums of the second
 *   are carried in two bf16 terms (to 2^-17).  x_sg * w_sg must be a normal fp32 number.
 *   An infinity or NaN in x, lora_a or lora_b reaches the rows that use it and no other.
 *
 *   xq [M, K/2], xs [M, K/16] row-major, x_sg 1 float: x as quantized (rotated along K like the
 *   weights); x bf16 [M, K], row stride ldx: x itself, which the adapters read; wq [N, K/2], ws
 *   hq_swizzled_scales_bytes(N, K) in the tile layout, w_sg 1 float; lora_a bf16 [adapters, R, K],
 *   lora_b bf16 [adapters, N, R], scaling float [adapters]; row_adapter int32 [M] on the device, rows in
 *   any order (rows of one request next to one another cost least).  R a multiple of 8 up to 128
 *   (adapters of a smaller rank padded with zeros), K a multiple of 32.  x, lora_a, lora_b and x's rows
 *   16-byte aligned.
 *   workspace : hq_lora_gemm_workspace_bytes(M, N, K, R) bytes, 32-byte aligned; contents need no
 *               preparation.  Calls that may run at the same time need different ones.
 */
HQ_API hq_status hq_lora_gemm_nvfp4(const uint8_t* xq, const uint8_t* xs, const float* x_sg,
                                    const uint8_t* wq, const uint8_t* ws, const float* w_sg,
                                    const void* x, int64_t ldx, const void* lora_a,
                                    const void* lora_b, const float* scaling,
                                    const int32_t* row_adapter, int64_t M, int64_t N, int64_t K,
                                    int64_t adapters, int64_t R, void* out, hq_dtype out_dtype,
                                    void* workspace, hq_stream stream);

/* hq_lora_gemm_mxfp4 -- the same beside an MXFP4 projection (no per-tensor scales). */
HQ_API hq_status hq_lora_gemm_mxfp4(const uint8_t* xq, const uint8_t* xs, const uint8_t* wq,
                                    const uint8_t* ws, const void* x, int64_t ldx,
                                    const void* lora_a, const void* lora_b, const float* scaling,
                                    const int32_t* row_adapter, int64_t M, int64_t N, int64_t K,
                                    int64_t adapters, int64_t R, void* out, hq_dtype out_dtype,
                                    void* workspace, hq_stream stream);

/* Bytes of hq_lora_gemm's workspace (-1 for sizes it refuses). */
HQ_API int64_t hq_lora_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t R);

/*
 * hq_swizzle_scales -- row-major block scales into the tile layout of
 * hq_rotate_quant_nvfp4_swizzled (for weights' scales, laid out once, and for MXFP4).
 *   scales: uint8 [groups, rows, cols], any alignment; out: groups buffers of
 *   hq_swizzled_scales_bytes(rows, 16 * cols) bytes, every byte written, padding as 0.
 */
HQ_API hq_status hq_swizzle_scales(const uint8_t* scales, int64_t groups, int64_t rows,
                                   int64_t cols, uint8_t* out, hq_stream stream);

/*
 * hq_block_norm -- the norms after a block and before the next one, with the block's gate and the
 * residual scale: what makes the tensor that is quantized next, in one pass.
 *   u = y * r_post * w_post,  r_post = 1 / sqrt(mean(y^2) + eps)   (HQ_NORM_POST; u = y without)
 *   h_out = alpha * h + gate * u
 *   n = h_out * r_pre * w_pre,  r_pre = 1 / sqrt(mean(h_out^2) + eps)   (HQ_NORM_PRE)
 *   In fp32 throughout; h_out and n are each rounded once, n from the h_out before its rounding.
 *
 *   h, y    : [M, D] of dtype, row strides ld_h, ld_y elements; 16-byte aligned rows.  y NULL: h_out
 *             is h and is not written (a first block's norm); then norms is HQ_NORM_PRE.
 *   D       : a multiple of 16, at most 32768.
 *   w_post, w_pre : [D] of param_dtype, or NULL for ones.
 *   gate    : by gate_kind NULL, [D] or [M] of param_dtype, or [M, D] of dtype (row stride ld_gate).
 *   h_out, n: [M, D] of dtype, contiguous, 16-byte aligned; may not overlap the inputs, except that
 *             h_out may be h itself (ld_h == D).
 *   r_post, r_pre : float [M], the rows' reciprocal norms for hq_block_norm_bwd.
 *   amax    : NULL, or 1 float that receives max |n . H_group / sqrt(group)| exactly as hq_rot_amax(n)
 *             would, so that n is quantized with one pass (hq_rotate_quant_nvfp4).  Needs HQ_NORM_PRE;
 *             D a multiple of group.
 */
typedef enum {
  HQ_GATE_NONE = 0,
  HQ_GATE_CHANNEL = 1, /* gate [D] */
  HQ_GATE_TOKEN = 2,   /* gate [M] */
  HQ_GATE_FULL = 3     /* gate [M, D] */
} hq_gate_kind;
#define HQ_NORM_POST 1
#define HQ_NORM_PRE 2

HQ_API hq_status hq_block_norm(const void* h, int64_t ld_h, const void* y, int64_t ld_y,
                               hq_dtype dtype, int64_t M, int64_t D, const void* w_post,
                               const void* w_pre, hq_dtype param_dtype, hq_gate_kind gate_kind,
                               const void* gate, int64_t ld_gate, int norms, float alpha, float eps,
                               void* h_out, void* n, float* r_post, float* r_pre, int group,
                               float* amax, hq_stream stream);

/*
 * hq_block_norm_bwd -- the gradients of hq_block_norm.
 *   dh_out, dn : gradients at h_out and n, [M, D] of dtype (dh_out NULL: zeros; dn is read with
 *                HQ_NORM_PRE).  h_out, r_post, r_pre: what the forward call wrote (h where y is NULL).
 *   dh, dy     : [M, D] of dtype, contiguous, 16-byte aligned (dy where y is given).
 *   dw_post, dw_pre : float [D], or NULL to skip.  Sums over the rows in fp32 in a fixed order.
 *   dgate      : float [D] (HQ_GATE_CHANNEL), float [M] (HQ_GATE_TOKEN), [M, D] of dtype (HQ_GATE_FULL).
 *   workspace  : hq_block_norm_bwd_workspace_bytes(M, D) bytes, 16-byte aligned; contents need no
 *                preparation.  Calls that may run at the same time need different ones.
 */
HQ_API hq_status hq_block_norm_bwd(const void* dh_out, int64_t ld_dh, const void* dn, int64_t ld_dn,
                                   const void* h_out, int64_t ld_h, const void* y, int64_t ld_y,
                                   hq_dtype dtype, int64_t M, int64_t D, const void* w_post,
                                   const void* w_pre, hq_dtype param_dtype, hq_gate_kind gate_kind,
                                   const void* gate, int64_t ld_gate, int norms, const float* r_post,
                                   const float* r_pre, float alpha, void* dh, void* dy,
                                   float* dw_post, void* dgate, float* dw_pre, void* workspace,
                                   hq_stream stream);

/* Bytes of hq_block_norm_bwd's workspace (-1 for sizes it refuses). */
HQ_API int64_t hq_block_norm_bwd_workspace_bytes(int64_t M, int64_t D);

/*
 * hq_gemm_int8 -- the product that reads what hq_rotate_quant_int8 writes: INT8 codes with a scale per token and per
 * channel.
 *   out[m, n] = (sum_k xq[m, k] wq[n, k]) * x_scales[m] * w_scales[n]
 *   The sum is exact while its partial sums stay below 2^24 in magnitude (fp32 sums of exact products beyond); then
 *   two fp32 products in this order and one rounding to out_dtype.
 *
 *   xq int8 [M, K], x_scales float [M]: activations; wq int8 [N, K], w_scales float [N]: weights, rotated like them.
 *   Rows contiguous, xq and wq 16-byte aligned.  K a multiple of 16 below 2^17; K == 0 gives zeros.
 *   out [M, N] of out_dtype, contiguous, aligned to its element.
 */
HQ_API hq_status hq_gemm_int8(const int8_t* xq, const float* x_scales, const int8_t* wq,
                              const float* w_scales, int64_t M, int64_t N, int64_t K, void* out,
                              hq_dtype out_dtype, hq_stream stream);

/*
 * A paged NVFP4 cache of keys and values.
 *
 *   cache : uint8 [pages][kv_heads][page_size / 16][18 D], 16-byte aligned, owned by the caller.  A record of 18 D bytes
 *           holds 16 tokens of a head: K codes [16, D/2], V codes [16, D/2], K scales [16, D/16], V scales [16, D/16],
 *           codes and E4M3 scales as hq_rotate_quant_nvfp4 writes them.  D is 64, 128 or 256; page_size a multiple
 *           of 16.  Any contents are allowed where no token has been stored.
 *   slot  : int64, page * page_size + place in the page.
 *   kv_amax : 2 floats on the device, the amax of K and of V that stand behind s_global (amax / 2688, as in
 *           hq_rotate_quant_nvfp4).  They are kept with the cache: every call on it takes the same two.  Blocks larger than
 *           they allow saturate.
 *   group : rotation of each head's channels, as in hq_rotate_quant_nvfp4; 256 needs D == 256.  q and K are rotated alike,
 *           so scores do not change; V is rotated and the attention's output rotated back.
 *   Each launch may start while the kernel before it on the stream ends; it waits for that kernel before it reads.
 */

/* Bytes of a page: kv_heads * page_size / 16 * 18 D (-1 for sizes that the calls refuse). */
HQ_API int64_t hq_kv_page_bytes(int64_t page_size, int64_t kv_heads, int64_t D);

/*
 * hq_kv_append_nvfp4 -- the way of T tokens into the cache, with the position rotation on it.
 *   q, k : pairs of channels (a, b) -> (a cos - b sin, b cos + a sin), each product and sum rounded to fp32; pair i is
 *          channels i and i + rotary/2, or 2i and 2i + 1 (interleaved); channels from `rotary` on stay.
 *   then q, k, v: y = x . H_group / sqrt(group) (fp32 butterfly); q_out = y rounded to bf16; k and v quantized as
 *          hq_rotate_quant_nvfp4 with amax = kv_amax[0], kv_amax[1], and stored at the token's slot.
 *
 *   q [T, q_heads, D], k, v [T, kv_heads, D] of dtype: heads contiguous, ld_* elements between tokens, 16-byte aligned
 *          tokens (parts of one fused projection qualify).  q_heads == 0: no queries.
 *   cos, sin : float [table_rows, rotary/2], 16-byte aligned.  rotary: a multiple of 16 up to D, 0 for none.
 *   positions : int32 [T] on the device, rows of the tables (others are clamped to them).
 *   slots : int64 [T] on the device; a token whose slot is negative or behind the last page is not stored.  Two
 *          tokens with one slot leave it with parts of either.
 *   q_out : bf16 [T, q_heads, D], contiguous, 16-byte aligned; may not overlap the inputs.
 *   T * (q_heads + 2 kv_heads) below 2^31 - 1024.
 */
HQ_API hq_status hq_kv_append_nvfp4(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v,
                                    int64_t ld_v, hq_dtype dtype, int64_t T, int64_t q_heads,
                                    int64_t kv_heads, int64_t D, const float* cos, const float* sin,
                                    int64_t table_rows, int64_t rotary, int interleaved,
                                    const int32_t* positions, const int64_t* slots, int group,
                                    const float* kv_amax, void* q_out, uint8_t* cache, int64_t pages,
                                    int64_t page_size, hq_stream stream);

/*
 * hq_kv_read_nvfp4 -- the values of cached tokens (to hand a prefix on, or to check): k, v [T, kv_heads, D] of
 * out_dtype, contiguous, 16-byte aligned; code * (scale * s_global) in fp32, then the rotation by `group` again (0:
 * as stored), one rounding.  Tokens without a slot (negative, behind the last page) are zeros.  T * kv_heads below
 * 2^31 - 1024.
 */
HQ_API hq_status hq_kv_read_nvfp4(const uint8_t* cache, int64_t pages, int64_t page_size, int64_t kv_heads,
                                  int64_t D, const int64_t* slots, int64_t T, const float* kv_amax,
                                  int group, void* k, void* v, hq_dtype out_dtype, hq_stream stream);

/*
 * hq_kv_attention_nvfp4 -- causal attention of S sequences over the cache.
 *   Sequence s has the queries q_start[s] .. q_start[s + 1] - 1, the last of its kv_len[s] tokens: its i-th of n
 *   queries sees the keys j <= p = kv_len[s] - n + i, with a window only the `window` last of them (j > p - window).
 *   out = (softmax(scale q K^T) V) . H_group / sqrt(group);  query head h reads key head h / (q_heads / kv_heads).
 *   lse = the natural logarithm of the sum of exp(scale q K^T).  A query without keys gets out = 0, lse = -inf.
 *   A NaN among the stored values reaches the rows that see its token and no others.
 *   Scores are exact up to their fp32 sums; weights are carried in 11 bits into sums in fp32; one rounding to bf16.
 *
 *   q, out : bf16 [T, q_heads, D]; q as hq_kv_append_nvfp4 leaves it, ld_q elements between tokens, 16-byte aligned
 *          tokens; out contiguous, 16-byte aligned, apart from q.  Rows of no sequence are not written.  q_heads a multiple of
 *          kv_heads.
 *   page_table : int32 [S, table_pages] on the device, rows ld_table apart: page of the tokens page_size * i .. of the
 *          sequence (others than 0 .. pages - 1 are clamped).  Entries behind a sequence's last page are not read.
 *          table_pages * page_size is at most 2^25.
 *   kv_len int32 [S], q_start int32 [S + 1] on the device, clamped to table_pages * page_size and to 0 .. T.  S is at most 2^20.
 *   max_q : the most queries of a sequence, as far as the host knows (T is always right).  It chooses the kernel, one for all
 *          sequences of the call; the result is defined for any value.  Single tokens in the kernel that prompts take cost
 *          three times as much: a step of single tokens names its max_q of 1, and single tokens beside a prompt are better off in a
 *          call of their own.
 *   window : 0 for none.    lse : float [T, q_heads], or NULL.
 *   workspace : hq_kv_attention_workspace_bytes(q_heads, kv_heads, D, T, max_q) bytes, 16-byte aligned; contents need
 *          no preparation.  Calls that may run at the same time need different ones.
 */
HQ_API hq_status hq_kv_attention_nvfp4(const void* q, int64_t ld_q, int64_t T, int64_t q_heads,
                                       const uint8_t* cache, int64_t pages, int64_t page_size,
                                       int64_t kv_heads, int64_t D, const int32_t* page_table,
                                       int64_t ld_table, int64_t table_pages, const int32_t* kv_len,
                                       const int32_t* q_start, int64_t S, int64_t max_q,
                                       const float* kv_amax, float scale, int64_t window, int group,
                                       void* out, float* lse, void* workspace, hq_stream stream);

/* Bytes of hq_kv_attention_nvfp4's workspace (-1 for sizes it refuses). */
HQ_API int64_t hq_kv_attention_workspace_bytes(int64_t q_heads, int64_t kv_heads, int64_t D, int64_t T,
                                               int64_t max_q);

/* Human-readable name of a status code (static storage). */
HQ_API const char* hq_status_string(hq_status status);

/* The cudaError_t behind the last HQ_ERR_CUDA returned on the calling host thread (0 if none). */
HQ_API int hq_last_cuda_error(void);

/*
 * hq_read_fault -- the library's device fault word on the current device (synchronous: waits
 * for all work on the device first).  0 means no kernel recorded a fault.  Bit 0 (value 1):
 * a kernel's wait for one of its own copies into shared memory, or for its own tensor-core products or other warps or
 * CTAs, exceeded about one second; what waited stopped early, so the outputs of the affected call are incomplete.  With
 * `clear` non-zero the word is reset to 0 after reading.
 */
HQ_API hq_status hq_read_fault(unsigned int* fault, int clear);

/*
 * hq_selftest_bounded_wait -- a test of the failure detection above, not part of the
 * quantization path (the pages have no counterpart).  Launches one warp on `stream` that waits,
 * through the same bounded mbarrier wait as the kernels' tile pipelines, on a barrier that nothing
 * ever completes.  After about one second the wait gives up, the kernel sets bit 0 of the fault
 * word and returns; no memory is touched and the context stays usable.  Returns once the launch
 * is enqueued (read the result with hq_read_fault).
 *   unit : 0 runs the wait in the translation unit of the NVFP4 / MXFP4 kernels, 1 in that of
 *          the INT8 kernel (each has its own copy of the fault word; hq_read_fault reads both).
 *          Anything else: HQ_ERR_SHAPE.
 */
HQ_API hq_status hq_selftest_bounded_wait(int unit, hq_stream stream);

/*
 * Host pipeline -- quantize tensors that live in (pinned) host memory.
 *   Not a step of the method itself: the transport around it.  One submission copies x to the
 *   device, runs hq_rot_amax and hq_rotate_quant_nvfp4 there, and moves the codes, the scales
 *   and s_global back.  Consecutive submissions overlap: the pipeline alternates between two
 *   buffer sets in the caller's device workspace and runs input copies, kernels and output
 *   transfers on three streams of its own, ordered by events, so the input copy of one
 *   submission runs while the previous one computes and sends its results back.  The outputs
 *   are written into the host buffers by a small kernel when the device can address them
 *   (pinned or registered memory, or any host memory on a device that reaches pageable memory
 *   through the host page tables), and copied otherwise.
 *
 *   The pipeline object is host memory owned by the library (freed by _destroy); it also owns
 *   three CUDA streams and six events on the device that is current at _create.  It allocates
 *   no device memory: `d_work` (at least hq_host_pipeline_workspace_bytes(M, K, dtype) bytes,
 *   256-byte aligned, owned by the caller) holds both buffer sets.  Host buffers should be pinned
 *   (cudaHostAlloc / cudaHostRegister) for the copies to be asynchronous; every host buffer of a
 *   submission must stay valid and untouched until hq_host_pipeline_wait() returns.
 */
typedef struct hq_host_pipeline hq_host_pipeline;

/* Device workspace bytes for M x K tensors of `dtype`.  0 if the sizes are invalid: M or K not
 * positive, K not a multiple of 16, K >= 2^36, or more than 2^58 elements. */
HQ_API size_t hq_host_pipeline_workspace_bytes(int64_t M, int64_t K, hq_dtype dtype);

/* Create a pipeline for M x K row-major tensors (contiguous rows) and rotation `group`. */
HQ_API hq_status hq_host_pipeline_create(int64_t M, int64_t K, hq_dtype dtype, int group,
                                         void* d_work, size_t work_bytes,
                                         hq_host_pipeline** out);

/* Enqueue one quantization and return at once.  x_host: [M, K] of dtype; q_host: [M, K/2] bytes;
 * scales_host: [M, K/16] bytes; s_global_host: 1 float.  Results are complete after
 * hq_host_pipeline_wait().
 * If a step fails after part of the submission was enqueued (HQ_ERR_CUDA), the buffer set's
 * ordering events may not cover the work in flight, so the pipeline refuses every later
 * submission with HQ_ERR_CUDA (hq_last_cuda_error() gives the first failure); wait for it and
 * destroy it.  A submission refused before anything was enqueued (HQ_ERR_NULL) leaves it usable. */
HQ_API hq_status hq_host_pipeline_submit(hq_host_pipeline* p, const void* x_host, uint8_t* q_host,
                                         uint8_t* scales_host, float* s_global_host);

/* Block the calling thread until every submitted quantization has finished. */
HQ_API hq_status hq_host_pipeline_wait(hq_host_pipeline* p);

/* Wait for outstanding work, then release the streams, events and the object (NULL is a no-op). */
HQ_API hq_status hq_host_pipeline_destroy(hq_host_pipeline* p);

/* hq_host_pipeline_inject_failure -- a test of the failure handling above, not part of the
 * quantization path (the pages have no counterpart).  The next submission to `p` behaves as if
 * the CUDA runtime refused its step `step` (0 the input copy, 1 pass 1, 2 pass 2, 3 the output
 * transfer): that step and the ones after it are not enqueued, the submission returns
 * HQ_ERR_CUDA with cudaErrorNotPermitted recorded, and the steps before it stay enqueued.
 * Nothing on the device fails.  step < 0 cancels a pending injection; step > 3: HQ_ERR_SHAPE. */
HQ_API hq_status hq_host_pipeline_inject_failure(hq_host_pipeline* p, int step);

/*
 * hq_quantize_nvfp4_host_noalloc -- the quantization of one host tensor with no device
 * allocation at all.  The pages have no counterpart: this entry point is for callers that cannot
 * obtain device memory themselves.  Examples: a plug-in loaded into a host program that owns the
 * whole device memory pool and hands its extensions no allocator; a serving loop that fixed its
 * memory footprint at start-up and must not allocate on the request path (an allocation there
 * can fail, or stall on the allocator).  Those callers can neither provide the workspace of the
 * host pipeline nor let the library allocate one.
 *
 * It does what one submission of the host pipeline does, in order on `stream`: copy x_host to the
 * device, hq_rot_amax, hq_rotate_quant_nvfp4, copy the codes, scales and s_global back.  Results
 * are complete when `stream` reaches that point (synchronize it, or record an event).  Its
 * device staging is one fixed array of HQ_NOALLOC_SCRATCH_BYTES inside the library, reserved on
 * every device where the library is loaded and held until the process exits.
 *
 *   Limit: the tensor must fit that array: with n = M*K and e = 2 (bf16) or 4 (fp32) bytes,
 *   r(b) = b rounded up to a multiple of 256, it needs r(n e) + r(n/2) + r(n/16) + 512 bytes
 *   (about 13.1 million bf16 or 7.35 million fp32 elements).  Larger tensors return
 *   HQ_ERR_TOO_LARGE before anything is enqueued.
 *   Set-up: the first call on a device looks up the array's device address (once per device,
 *   with that device current), so make that first call before any stream capture.  The address
 *   belongs to the device's context: after cudaDeviceReset the next call looks it up again (and
 *   is then a first call again).
 *   Sharing: every call on a device uses the same array and leaves its contents there; calls
 *   whose work overlaps on the GPU (other streams, other host threads) race on it, so order
 *   them (one stream, or events).  The call clears what must start at zero (the amax).
 *   Host buffers should be pinned for the copies to be asynchronous.  x_host: [M, K] of dtype,
 *   contiguous rows; q_host: [M, K/2]; scales_host: [M, K/16]; s_global_host: 1 float.
 */
#define HQ_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)
HQ_API hq_status hq_quantize_nvfp4_host_noalloc(const void* x_host, hq_dtype dtype, int64_t M,
                                                int64_t K, int group, uint8_t* q_host,
                                                uint8_t* scales_host, float* s_global_host,
                                                hq_stream stream);

/* Library version: major * 10000 + minor * 100 + patch. */
HQ_API int hq_version(void);

#ifdef __cplusplus
}
#endif

#endif /* HQ_H_ */
