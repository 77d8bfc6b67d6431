/*
 * fp4q.h - C ABI of the GB300 (sm_103a) fused residual-add + RMSNorm +
 * block-scaled FP4 quantization library (libfp4q.so).
 *
 * The operation is the one on the FlashInfer page `add_rmsnorm_fp4quant.py`
 * (module docstring; `AddRMSNormFP4QuantKernel.kernel` phases 1-3;
 * `add_rmsnorm_fp4quant` Parameters / Returns / Notes).  Per row m of an
 * M x H batch, with b = 16 (NVFP4) or 32 (MXFP4), nb = H / b:
 *
 *   h        = round_dtype(float(input) + float(residual))   -> residual (in place)
 *   rstd     = 1 / sqrt(sum(h^2) / H + eps)                   (fp32, each op rounded)
 *   y        = (h * weight) * rstd                            (fp32: h * weight is exact,
 *                                                              so y is rounded once)
 *   per block of b elements (amax = max |y| over the block):
 *     NVFP4: scale = E4M3 nearest-even of min(amax / 6, 448)
 *     MXFP4: scale = UE8M0, the power of two at or above amax / 6
 *     code  = E2M1 nearest-even of y * rn(1 / scale) on {0,.5,1,1.5,2,3,4,6},
 *             saturating, sign in bit 3 (the page's kernel scales by the
 *             reciprocal of the decoded scale); a zero scale gives zero codes
 *   out_packed[m, j] = code[2j] | code[2j+1] << 4
 *
 * Scale layouts (same page, `is_sf_swizzled_layout`, `output_both_sf_layouts`):
 *   row-major : sf[m * nb + k]
 *   tiled     : sf[(m/128)*nkt*512 + (k/4)*512 + (m%32)*16 + ((m%128)/32)*4 + k%4],
 *               nkt = ceil(nb / 4), buffer = ceil(M/128) * nkt * 512 bytes, every
 *               padding byte (rows >= M, k >= nb) written 0.  This is the scale
 *               layout the FlashRT `fp4-gemm` README (Tensor Contract) names as
 *               the CUTLASS SFA input of its NVFP4 GEMM.
 *
 * Conventions shared by every entry point:
 *   - All tensor pointers are DEVICE pointers owned by the caller; the library
 *     allocates nothing and keeps no state between calls.
 *   - Tensors are dense row-major (row stride = H elements / H/2 bytes).
 *   - Calls are asynchronous on `stream` (NULL = legacy default stream);
 *     argument errors are detected on the host before anything is launched.
 *   - Status codes, never exceptions or aborts.
 */
#ifndef FP4Q_H_
#define FP4Q_H_

#include <stdint.h>

/* Only the entry points below are exported from libfp4q.so (built with hidden
 * visibility). */
#if defined(__GNUC__)
#define FP4Q_API __attribute__((visibility("default")))
#else
#define FP4Q_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same handle type as cudaStream_t / CUstream. */
typedef struct CUstream_st* fp4q_stream_t;

/* FP4_DT_FP32 is a type of logits alone (fp4_beam_select). */
typedef enum { FP4_DT_BF16 = 0, FP4_DT_FP16 = 1, FP4_DT_FP32 = 2 } fp4_dtype_t;

/* NVFP4: 16-element blocks, E4M3 scale bytes.  MXFP4: 32-element blocks,
 * UE8M0 scale bytes.  E4M3_B32: 32-element blocks with E4M3 scale bytes
 * (FlashInfer page, `block_size` / `scale_format`: "e4m3" on the block-32
 * branch).  A global scale applies to the two E4M3 formats only. */
typedef enum { FP4_NVFP4 = 0, FP4_MXFP4 = 1, FP4_E4M3_B32 = 2 } fp4_format_t;

typedef enum {
  FP4_SF_ROWMAJOR = 0, /* (M, nb) bytes                                  */
  FP4_SF_SWIZZLED = 1, /* 128x4 tiled, padded to whole tiles             */
  FP4_SF_BOTH = 2      /* tiled into out_sf AND row-major into out_sf_rowmajor */
} fp4_sf_layout_t;

typedef enum {
  FP4_OK = 0,
  FP4_ERR_INVALID_ARG = 1,       /* null pointer, bad enum, negative size, overlap */
  FP4_ERR_UNSUPPORTED_SHAPE = 2, /* H % b != 0, H < 64, or H above the maximum     */
  FP4_ERR_MISALIGNED = 3,        /* a pointer breaks the alignment rule below       */
  FP4_ERR_CUDA = 4,              /* the CUDA runtime reported an error on launch    */
  FP4_ERR_TIMEOUT = 5,           /* a kernel gave up on a bounded wait (device status word) */
  FP4_ERR_NO_PAGES = 6           /* a sequence found no free page, or no room in its table (device status word) */
} fp4_status_t;

/*
 * Device status word.  The kernels that wait on asynchronous copies (the
 * wide-row fused kernel, which streams rows through a shared-memory ring
 * filled by the copy engine, and every GEMM schedule) bound each wait at about
 * one second of clock cycles.  A CTA whose wait runs out does not hang or
 * trap: it stops, marks what it could not compute and returns, and the
 * context stays usable.  The calls that take an optional `status` (a DEVICE
 * pointer to one int32_t owned by the caller) then store FP4_ERR_TIMEOUT
 * there.  The library never clears it (and writes nothing else to it, but
 * FP4_ERR_NO_PAGES in fp4_kv_fork_nvfp4):
 * zero it before the call, synchronise, and read it (fp4_read_device_status
 * does the last two).  What a timed-out call leaves behind:
 *   fused op: every scale byte of the rows the CTA did not finish is 0xFF
 *             (NaN in E4M3 and in UE8M0); their codes, residual rows and y
 *             rows are unspecified (the residual row may be the old value);
 *   GEMM:     the output tiles of the CTA are NaN (bf16 out), or their scale
 *             bytes 0xFF (NVFP4 out).
 * The host-side return value of the call itself only reports what is known
 * at launch (FP4_OK once the launch succeeded).
 */

/* Largest supported H: one CTA holds up to 32768 elements of a row in
 * registers and a thread-block cluster of up to 8 CTAs shares one row.  Above
 * 32768, H / 16 must split evenly over the cluster (over chunk pairs for MXFP4). */
#define FP4Q_MAX_H 262144

/*
 * fp4_add_rmsnorm_quant - the fused op (FlashInfer page, `add_rmsnorm_fp4quant`).
 *
 *   input           [M, H] dtype, read only.                      32-byte aligned.
 *   residual        [M, H] dtype, read then overwritten with h.   32-byte aligned.
 *   weight          [H]    dtype, read only.                      32-byte aligned.
 *   eps             added to the mean of squares (fp32).
 *   M               rows, >= 0 (M == 0: nothing is launched, FP4_OK).
 *   H               hidden size: multiple of the block size, 64 <= H <= FP4Q_MAX_H.
 *   out_packed      [M, H/2] bytes, two E2M1 codes per byte.       8-byte aligned.
 *   out_sf          row-major scales (FP4_SF_ROWMAJOR) or the tiled buffer
 *                   (FP4_SF_SWIZZLED / FP4_SF_BOTH, 4-byte aligned); size from
 *                   fp4_sf_size_bytes.
 *   out_sf_rowmajor row-major scales for FP4_SF_BOTH, else ignored (may be NULL).
 *
 * input must not overlap residual; outputs must not overlap inputs or each
 * other.  Global scale is 1 (the page's default when none is given).
 */
FP4Q_API fp4_status_t fp4_add_rmsnorm_quant(const void* input, void* residual, const void* weight,
                                            float eps, int64_t M, int64_t H, fp4_dtype_t dtype,
                                            fp4_format_t format, fp4_sf_layout_t sf_layout,
                                            uint8_t* out_packed, uint8_t* out_sf,
                                            uint8_t* out_sf_rowmajor, fp4q_stream_t stream);

/*
 * fp4_add_rmsnorm_quant_gs - fp4_add_rmsnorm_quant with a device-resident
 * global scale (FlashInfer page, `global_scale`; read on the device, so a
 * captured CUDA graph picks up a new value).  global_scale: DEVICE pointer to
 * one positive finite fp32, or NULL for 1.  For the E4M3 formats each block
 * scale becomes E4M3(min(gs * amax / 6, 448)) and codes round from
 * y * rn(rn(1 / scale) * gs) (so dequantised values are y * gs: a consumer divides by gs,
 * e.g. gs = 448 * 6 / max|y| fills the E4M3 range); UE8M0 scales ignore it.
 * All other arguments as fp4_add_rmsnorm_quant.
 */
FP4Q_API fp4_status_t fp4_add_rmsnorm_quant_gs(const void* input, void* residual, const void* weight,
                                               const float* global_scale, float eps, int64_t M,
                                               int64_t H, fp4_dtype_t dtype, fp4_format_t format,
                                               fp4_sf_layout_t sf_layout, uint8_t* out_packed,
                                               uint8_t* out_sf, uint8_t* out_sf_rowmajor,
                                               fp4q_stream_t stream);

/*
 * fp4_add_rmsnorm_quant_ex - the general form of the fused op: strided rows,
 * an optional y output, a device status word and programmatic dependent
 * launch (API variants of the FlashInfer page's `add_rmsnorm_fp4quant`,
 * which views 3-D input as 2-D rows).
 *
 *   input_row_stride, residual_row_stride  elements between consecutive rows
 *                  (0 = H); >= H and a multiple of 16 (rows start 32-byte
 *                  aligned).  Outputs stay dense.
 *   out_y          [M, H] dtype, dense, 32-byte aligned, or NULL: receives y =
 *                  (h * w) * rstd rounded to the storage dtype (the value the
 *                  codes quantize), for consumers that want it unquantized.
 *   global_scale   as in fp4_add_rmsnorm_quant_gs (NULL = 1).
 *   status         DEVICE int32_t, 4-byte aligned, or NULL: receives
 *                  FP4_ERR_TIMEOUT if a bounded wait ran out (see "Device
 *                  status word" above); left untouched otherwise.
 *   pdl            nonzero: launched as a programmatic dependent of the kernel
 *                  before it on `stream` (e.g. the GEMM that produced `input`),
 *                  so the launch overlaps that kernel's tail; the kernel waits
 *                  for its results before reading anything.  Every kernel of
 *                  this library lets its own dependents launch once its CTAs
 *                  have issued their loads.
 * Everything else as fp4_add_rmsnorm_quant; the outputs, y and status must
 * not overlap the inputs or each other.
 */
FP4Q_API fp4_status_t fp4_add_rmsnorm_quant_ex(const void* input, int64_t input_row_stride,
                                               void* residual, int64_t residual_row_stride,
                                               const void* weight, const float* global_scale, float eps,
                                               int64_t M, int64_t H, fp4_dtype_t dtype,
                                               fp4_format_t format, fp4_sf_layout_t sf_layout,
                                               uint8_t* out_packed, uint8_t* out_sf,
                                               uint8_t* out_sf_rowmajor, void* out_y,
                                               int32_t* status, int pdl, fp4q_stream_t stream);

/*
 * fp4_quantize - block quantization of `input` [M, H] itself, without the
 * residual add and the normalisation: the standalone producer of packed E2M1
 * plus scales (FlashRT `fp4-gemm` README, `quantize_fp4_sfa_bf16` /
 * `quantize_fp4_sfa_fp16`).  The same layouts serve as the GEMM's A-operand
 * scales (rows = M) or B-operand scales (rows = N).  input 32-byte aligned,
 * H a multiple of the block size (>= 16); global_scale as in
 * fp4_add_rmsnorm_quant_gs; outputs as fp4_add_rmsnorm_quant; pdl as in
 * fp4_add_rmsnorm_quant_ex (launched as a programmatic dependent of the
 * kernel before it on `stream`, e.g. the kernel that produced `input`).
 */
FP4Q_API fp4_status_t fp4_quantize(const void* input, const float* global_scale, int64_t M, int64_t H,
                                   fp4_dtype_t dtype, fp4_format_t format, fp4_sf_layout_t sf_layout,
                                   uint8_t* out_packed, uint8_t* out_sf, uint8_t* out_sf_rowmajor,
                                   int pdl, fp4q_stream_t stream);

/*
 * fp4_dequant - validation helper: out[m, i] = E2M1 value of code (m, i) times
 * its block scale, fp32 (exact).  Mirrors the dequantise-and-compare method of
 * the FlashRT `fp4-gemm` README (Validation; `dequantize_fp4_sfa_fp16`).
 *
 *   packed    [M, H/2] bytes.                      8-byte aligned.
 *   sf        scales in `sf_layout` (FP4_SF_ROWMAJOR or FP4_SF_SWIZZLED).
 *   out       [M, H] fp32.                         16-byte aligned.
 * H must be a multiple of the block size (>= 16); M >= 0.
 */
FP4Q_API fp4_status_t fp4_dequant(const uint8_t* packed, const uint8_t* sf, int64_t M, int64_t H,
                                  fp4_format_t format, fp4_sf_layout_t sf_layout, float* out,
                                  fp4q_stream_t stream);

/*
 * fp4_sf_size_bytes - bytes of ONE scale buffer in `layout` (FlashInfer page,
 * output allocation; FlashRT README `sfa_size_bytes`): row-major M * (H/b);
 * tiled ceil(M/128) * ceil((H/b)/4) * 512.  FP4_SF_BOTH returns the tiled size
 * (the size of out_sf).  Returns -1 on bad arguments.  Host only; no GPU needed.
 */
FP4Q_API int64_t fp4_sf_size_bytes(int64_t M, int64_t H, fp4_format_t format, fp4_sf_layout_t layout);

/*
 * fp4_launch_shape - the launch the library would make for fp4_add_rmsnorm_quant
 * with these sizes on the current device (diagnostics; launches nothing).
 * Fills out[8] = {kernel (0 = persistent TMA-ring kernel, 1 = register-resident
 * kernel), chunks per thread, threads per row slice, row slices per CTA,
 * CTAs per cluster, shared-memory ring stages, threads per CTA, CTAs}.
 * Returns FP4_OK, or the status fp4_add_rmsnorm_quant would return for the sizes.
 */
FP4Q_API fp4_status_t fp4_launch_shape(int64_t M, int64_t H, fp4_dtype_t dtype, fp4_format_t format,
                                       fp4_sf_layout_t sf_layout, int64_t out[8]);

/*
 * fp4_gemm_variant - the schedule (the `variant` numbers of
 * fp4_gemm_nvfp4_bf16 below) the GEMM entry points would run for an
 * M x N x K product of `format` operands (FP4_NVFP4 or FP4_MXFP4); fp4_out
 * nonzero for fp4_gemm_nvfp4_gelu_nvfp4.  `variant` -1 asks for the
 * automatic choice; any other accepted value is returned as given.  Returns
 * -1 for sizes or a variant the GEMM would reject.  Host only (diagnostics;
 * launches nothing): the choice depends on the current device's SM count,
 * taken as 152 when no device is visible.
 */
FP4Q_API int fp4_gemm_variant(int64_t M, int64_t N, int64_t K, fp4_format_t format, int fp4_out,
                              int variant);

/*
 * fp4_gemm_nvfp4_bf16 - the consumer of the packed codes and tiled scales:
 * out = bf16(alpha * deq(A) @ deq(B)^T (+ bias) (+ residual)) on the tensor
 * cores (FlashRT `fp4-gemm` README: Tensor Contract; `nvfp4_gemm_bf16`,
 * `nvfp4_gemm_bias_bf16`, `nvfp4_gemm_residual_bf16`,
 * `nvfp4_gemm_bias_residual_bf16`), deq = E2M1 value times its E4M3 block
 * scale (16 elements per block), accumulation in fp32.
 *
 *   a_packed  [M, K/2] bytes: rows of A, two E2M1 codes per byte (element 2j in
 *             the low nibble), e.g. out_packed of the fused op or fp4_quantize.
 *   b_packed  [N, K/2] bytes: rows of B (the weight, one row per output column).
 *   sfa, sfb  NVFP4 scales of A (M rows) and of B (N rows) in the 128x4 tiled
 *             layout (FP4_SF_SWIZZLED), fp4_sf_size_bytes(M or N, K, ...) bytes.
 *   alpha     fp32 multiplier of the product (e.g. 1 / (gs_a * gs_b) for
 *             operands quantized with global scales).
 *   bias      [N] bf16 or NULL, added after alpha.
 *   residual  [M, N] bf16 or NULL, added last; may be `out` itself.
 *   out       [M, N] bf16, row-major.
 *   variant   tile schedule (the README's `variant`; fp4_gemm_variant reports
 *             the automatic choice): -1 automatic; one CTA per output tile with
 *             0 = 128 x 128 tiles (two CTAs per SM) or 1 = 128 x 256 tiles;
 *             persistent CTAs walking the tiles, one accumulator each, loading
 *             the next tile while the epilogue drains the last, with
 *             2 = 128 x 128 (two CTAs per SM) or 3 = 128 x 256 (one per SM;
 *             automatic when the output has more 128 x 128 tiles than twice
 *             the SMs); 4 = 128 x 128 tiles with the K loop of each tile split
 *             over a thread-block cluster of up to 16 CTAs (partial tiles
 *             summed in rank order through distributed shared memory;
 *             automatic when the output has at most half as many 128 x 128
 *             tiles as SMs and K > 1536, e.g. the M = 41 decode product with
 *             K = 6144).
 *   pdl       1: launched as a programmatic dependent of the previous kernel
 *             on `stream`, so its prologue overlaps that kernel's tail (it
 *             waits for that kernel's results before reading anything).
 *             2: the same, and the caller states that the previous kernel
 *             writes neither b_packed nor sfb (weights, as in a decode step
 *             after the fused op): the one-CTA-per-tile and split-K schedules
 *             then start B's first ring of copies before the wait.  0: none.
 *             Other values: FP4_ERR_INVALID_ARG.
 * K must be a multiple of 32 (a packed row a whole number of 16-byte units;
 * the FlashRT contract's K % 16 otherwise) and N of 8; every pointer 16-byte
 * aligned; out must not overlap the inputs (except residual == out).  When K
 * is not a multiple of 64, the last K = 64 step reads the k-padding scales of
 * the tiled layout against zero codes: they must be finite (this library's
 * producers write them as 0).  A tile whose inputs never arrive (a bounded
 * wait runs out) is written as NaN.
 */
FP4Q_API fp4_status_t fp4_gemm_nvfp4_bf16(const uint8_t* a_packed, const uint8_t* b_packed,
                                          const uint8_t* sfa, const uint8_t* sfb, float alpha,
                                          const void* bias, const void* residual, int64_t M, int64_t N,
                                          int64_t K, void* out, int variant, int pdl,
                                          fp4q_stream_t stream);

/*
 * fp4_gemm_mxfp4_bf16 - the same product for MXFP4 operands: E2M1 codes with
 * one UE8M0 scale per 32 elements (the fused op's and fp4_quantize's MXFP4
 * output, tiled layout, fp4_sf_size_bytes(M or N, K, FP4_MXFP4, ...) bytes).
 * Not on the FlashRT page (its GEMM is NVFP4 only): the consumer of this
 * library's own MXFP4 producer.  Arguments, checks and variants as
 * fp4_gemm_nvfp4_bf16 (every variant).
 */
FP4Q_API fp4_status_t fp4_gemm_mxfp4_bf16(const uint8_t* a_packed, const uint8_t* b_packed,
                                          const uint8_t* sfa, const uint8_t* sfb, float alpha,
                                          const void* bias, const void* residual, int64_t M,
                                          int64_t N, int64_t K, void* out, int variant, int pdl,
                                          fp4q_stream_t stream);

/*
 * fp4_gemm_nvfp4_gelu_bf16 - out = bf16(GELU(alpha * deq(A) @ deq(B)^T + bias))
 * (FlashRT `fp4-gemm` README, `nvfp4_gemm_bias_gelu_bf16`; GELU is the exact
 * x * Phi(x), computed with erff; bias may be NULL).  Arguments as
 * fp4_gemm_nvfp4_bf16 without the residual.
 */
FP4Q_API fp4_status_t fp4_gemm_nvfp4_gelu_bf16(const uint8_t* a_packed, const uint8_t* b_packed,
                                               const uint8_t* sfa, const uint8_t* sfb,
                                               float alpha, const void* bias, int64_t M,
                                               int64_t N, int64_t K, void* out, int variant,
                                               int pdl, fp4q_stream_t stream);

/*
 * fp4_gemm_nvfp4_gelu_nvfp4 - the same GELU values, rounded to fp32 and
 * quantized in the epilogue to NVFP4 for the next GEMM (README,
 * `nvfp4_gemm_bias_gelu_nvfp4`: "packed FP4 plus CUTLASS SFA"): the
 * producer's rules (E4M3 scale of amax / 6 per 16 values, codes of
 * v * rn(1/s), no global scale).
 *   out_packed  [M, N/2] bytes, 16-byte aligned.
 *   out_sf      tiled scales of the M x N output (fp4_sf_size_bytes(M, N,
 *               FP4_NVFP4, FP4_SF_SWIZZLED) bytes), padding rows and k padding
 *               written 0.
 * N must be a multiple of 16; variant 4 (split K) is not available
 * (FP4_ERR_INVALID_ARG); outputs must not overlap the inputs or each other.
 */
FP4Q_API fp4_status_t fp4_gemm_nvfp4_gelu_nvfp4(const uint8_t* a_packed,
                                                const uint8_t* b_packed, const uint8_t* sfa,
                                                const uint8_t* sfb, float alpha,
                                                const void* bias, int64_t M, int64_t N,
                                                int64_t K, uint8_t* out_packed,
                                                uint8_t* out_sf, int variant, int pdl,
                                                fp4q_stream_t stream);

/* Output of the general GEMM entry point fp4_gemm_ex. */
typedef enum {
  FP4_EPI_BF16 = 0,        /* alpha * product (+ bias) (+ residual) -> bf16 out   */
  FP4_EPI_GELU_BF16 = 1,   /* GELU(alpha * product (+ bias)) -> bf16 out          */
  FP4_EPI_GELU_NVFP4 = 2   /* GELU(...) -> NVFP4 codes + tiled scales (out_packed, out_sf) */
} fp4_epilogue_t;

/*
 * fp4_gemm_ex - the general form of the four GEMM entry points above: operand
 * `format` (FP4_NVFP4 or FP4_MXFP4; FP4_EPI_GELU_NVFP4 takes NVFP4 only), the
 * `epilogue`, and a device `status` word (DEVICE int32_t, 4-byte aligned, or
 * NULL) that receives FP4_ERR_TIMEOUT when a CTA's bounded wait ran out (its
 * tiles are then NaN, or 0xFF scale bytes for NVFP4 output; see "Device status
 * word").  `residual` is used by FP4_EPI_BF16 only; `out` by the bf16
 * epilogues, `out_packed` / `out_sf` by FP4_EPI_GELU_NVFP4.  Every other
 * argument, check and variant as fp4_gemm_nvfp4_bf16 /
 * fp4_gemm_nvfp4_gelu_nvfp4; the four named entry points are this call with
 * status = NULL.
 */
FP4Q_API fp4_status_t fp4_gemm_ex(const uint8_t* a_packed, const uint8_t* b_packed,
                                  const uint8_t* sfa, const uint8_t* sfb, fp4_format_t format,
                                  fp4_epilogue_t epilogue, float alpha, const void* bias,
                                  const void* residual, int64_t M, int64_t N, int64_t K, void* out,
                                  uint8_t* out_packed, uint8_t* out_sf, int variant, int pdl,
                                  int32_t* status, fp4q_stream_t stream);

/*
 * The NVFP4 key/value cache: attention's keys and values held in this
 * library's own 4-bit blocks (E2M1 codes, one E4M3 scale per 16 channels of a
 * head of a token), in pages.  Per page and key/value head:
 *
 *   k_packed, v_packed  [num_pages, num_kv_heads, page_size, head_dim/2] bytes, channel 2j in
 *                       the low nibble of byte j;
 *   k_sf                [num_pages, num_kv_heads, page_size, head_dim/16] bytes;
 *   v_sf                [num_pages, num_kv_heads, head_dim/16, page_size] bytes: the scales of
 *                       consecutive tokens lie side by side, because the product with V runs
 *                       over tokens.
 *
 * Slot number = page * page_size + place in the page.  Every buffer is dense
 * and 16-byte aligned; page_size is a multiple of 16, head_dim 64 or 128.
 * k_global_scale, v_global_scale: DEVICE pointers to one positive finite fp32
 * each, or NULL for 1, with the meaning of fp4_quantize's global_scale (blocks
 * hold value * scale; the readers divide by it).
 * A slot that was never written may hold any bytes as long as no sequence
 * counts it; a counted slot holds what fp4_kv_append_nvfp4 writes (scale
 * bytes that are finite).
 */
typedef struct {
  uint8_t* k_packed;
  uint8_t* k_sf;
  uint8_t* v_packed;
  uint8_t* v_sf;
  const float* k_global_scale;
  const float* v_global_scale;
  int64_t num_pages;
  int64_t page_size;
  int64_t num_kv_heads;
  int64_t head_dim;
} fp4_kv_cache_t;

/*
 * fp4_kv_append_nvfp4 - rotates the queries and keys of T tokens by their
 * positions, quantizes keys and values and stores them in the tokens' slots.
 *
 *   q, q_stride        [T, Hq, head_dim] dtype, q_stride elements between tokens (0: dense);
 *                      NULL with Hq = 0 when there is nothing to rotate but the keys.
 *   out_q, out_q_stride  the rotated queries, rounded once to dtype; may be q itself (same
 *                      stride).  NULL exactly when q is NULL.
 *   k, k_stride, v, v_stride  [T, num_kv_heads, head_dim] dtype, e.g. column slices of one
 *                      fused projection's output.
 *   positions          [T] int64, each token's row of cos_sin.  A token whose position is
 *                      outside [0, max_position) is left out altogether: no out_q row, nothing
 *                      appended.
 *   cos_sin            [max_position, rot_dim] fp32: rot_dim/2 cosines, then rot_dim/2 sines.
 *   rot_dim            channels of each head that are rotated, a multiple of 32, at most
 *                      head_dim; 0: no rotation (positions, cos_sin NULL; q is then copied).
 *                      Channels x1, x2 of a pair become rn(rn(x1 cos) - rn(x2 sin)) and
 *                      rn(rn(x2 cos) + rn(x1 sin)) in fp32; keys are quantized from these.
 *   interleaved        0: pair i is channels i and i + rot_dim/2; 1: channels 2i and 2i + 1.
 *   slots              [T] int64.  A slot outside [0, num_pages * page_size) appends nothing
 *                      (padding tokens: -1).  The slots of one call have to differ: what a
 *                      slot that two tokens name holds afterwards is not specified.
 *   pdl                as in fp4_add_rmsnorm_quant_ex.
 * Codes and scales are those of fp4_quantize (NVFP4) on the rotated keys and on
 * the values.  q, k, v and out_q rows start on 32-byte boundaries (strides
 * multiples of 16); positions and slots are 8-byte aligned.  Nothing that is
 * written may overlap anything else the call reads or writes, out_q = q excepted.
 */
FP4Q_API fp4_status_t fp4_kv_append_nvfp4(const void* q, int64_t q_stride, void* out_q,
                                          int64_t out_q_stride, const void* k, int64_t k_stride,
                                          const void* v, int64_t v_stride,
                                          const int64_t* positions, const float* cos_sin,
                                          int64_t max_position, int64_t rot_dim, int interleaved,
                                          const int64_t* slots, int64_t T, int64_t Hq,
                                          fp4_dtype_t dtype, const fp4_kv_cache_t* cache, int pdl,
                                          fp4q_stream_t stream);

/*
 * fp4_kv_gather_nvfp4 - reads the tokens of T slots back: out_k, out_v
 * [T, num_kv_heads, head_dim] dtype, dense, 32-byte aligned (either may be
 * NULL), code * scale / global scale in fp32, rounded once to dtype (exact
 * without a global scale).  A slot outside the cache leaves its rows as they
 * were.  Slots may repeat.
 */
FP4Q_API fp4_status_t fp4_kv_gather_nvfp4(const fp4_kv_cache_t* cache, const int64_t* slots,
                                          int64_t T, fp4_dtype_t dtype, void* out_k, void* out_v,
                                          int pdl, fp4q_stream_t stream);

/*
 * fp4_attention_nvfp4 - attention over the cached sequences of a batch:
 *
 *   out = softmax(sm_scale * q k^T) v,   lse = log(sum(exp(sm_scale * q k^T)))
 *
 * per query row and head, keys and values taken from the cache as code * scale
 * / global scale.  Query head h reads key/value head h / (Hq / num_kv_heads).
 *
 *   q, q_stride     [T, Hq, head_dim] dtype (rotated, e.g. out_q above), rows 32-byte aligned.
 *   block_tables    [B, max_pages] int32: the pages of each sequence in order.  Keys of a page
 *                   whose number is outside [0, num_pages) are masked.
 *   seq_lens        [B] int32: cached tokens of each sequence, this call's own among them
 *                   (taken as clamped to [0, max_pages * page_size]).
 *   cu_seqlens_q    [B + 1] int32, ascending: sequence b's query rows are cu[b] .. cu[b+1]-1.
 *                   NULL: one row per sequence (T == B).  Rows outside [cu[0], cu[B]) are
 *                   left as they were.
 *   causal          nonzero: row i of a sequence's n_q rows sees its first len - n_q + i + 1
 *                   keys; zero: all of them (cross attention to an encoder's states).
 *   sm_scale        > 0, finite; a logit times log2(e) has to stay within fp32's numbers.
 *   out             [T, Hq, head_dim] dtype, dense, 32-byte aligned.  A row that sees no key is
 *                   0, with lse -inf.
 *   lse             [T, Hq] fp32 (natural logarithm), or NULL.
 *   workspace       at least fp4_attention_workspace_bytes(...) bytes (or _bound's, of the
 *                   largest sizes), 16-byte aligned, any contents; two calls that may run at
 *                   the same time need one each.
 *   status, pdl     as in fp4_add_rmsnorm_quant_ex.
 * Lengths and tables are read on the device, so a captured call follows them.
 * Rows that a kernel gave up on (a bounded wait ran out: status) are NaN, lse too.
 * Logits, references, sums and accumulators are fp32.  Two things are rounded to 16
 * bits on the way: each weight exp(..) to fp16's 11 bits (relative 2^-11; one that is 2^20 times
 * smaller than the row's largest to 2^-31 of that) before it is
 * multiplied with v, while the sum takes it unrounded; and each query element, scaled
 * by a power of two, by at most 2^-39 of its row's largest (most elements by nothing).
 * Keys and values are exact.  One kernel serves a call, chosen by the average number of
 * rows per sequence and the table's width: prompts and single rows are faster in two
 * calls (each over its rows of q and out), and so are short sequences in a table cut
 * to their pages.  Nothing that is written may overlap anything else the call reads or
 * writes.
 */
FP4Q_API fp4_status_t fp4_attention_nvfp4(const void* q, int64_t q_stride,
                                          const fp4_kv_cache_t* cache, const int32_t* block_tables,
                                          int64_t max_pages, const int32_t* seq_lens,
                                          const int32_t* cu_seqlens_q, int64_t B, int64_t T,
                                          int64_t Hq, fp4_dtype_t dtype, float sm_scale, int causal,
                                          void* out, float* lse, void* workspace,
                                          int64_t workspace_bytes, int32_t* status, int pdl,
                                          fp4q_stream_t stream);

/*
 * fp4_attention_nvfp4_ex - the same with capped logits, a bias that grows with distance,
 * a window and a prefix.  With a sequence's rows at places pos = len - n_q + i of its keys
 * (i = 0 .. n_q - 1), the logit of row pos, query head h and key j is
 *
 *   x = sm_scale * q k^T                             (softcap = 0)
 *   x = softcap * tanh(sm_scale * q k^T / softcap)    (softcap > 0)
 *   x - alibi_slopes[h] * |pos - j|                   (alibi_slopes not NULL)
 *
 * and the row sees the keys j with
 *
 *   j <= pos, or j < prefix_lens[b]        (causal; prefix_lens NULL: the first alone)
 *   j > pos - window                       (window > 0)
 *
 *   softcap        >= 0, at most 2^20.
 *   alibi_slopes   [Hq] fp32 or NULL.
 *   window         >= 0; 0: none.  With causal only.  Pages that hold nothing but keys before the
 *                  first row's window are not read (fp4_kv_trim_nvfp4 gives them up).
 *   prefix_lens    [B] int32 or NULL (taken as clamped to [0, len]).  With causal only.  Of a prefix
 *                  before a row's window the row sees nothing.
 *   workspace      fp4_attention_workspace_bytes for max_keys, with a window for
 *                  min(max_keys, window + ceil(T / B) + 63) (or _bound's).
 * Logits are fp32, rounded once after each of the steps above; the cap's is off by a few 2^-24
 * of softcap, or, with a softcap above 256, by 2^-19 of itself at most (prompts then take up to three
 * times as long).  What is rounded to 16 bits is as above, but that calls of many rows with a cap or a
 * bias round a weight that is 2^14 times smaller than the row's largest to 2^-25 of that.
 * Other arguments as above.
 */
FP4Q_API fp4_status_t fp4_attention_nvfp4_ex(const void* q, int64_t q_stride,
                                             const fp4_kv_cache_t* cache,
                                             const int32_t* block_tables, int64_t max_pages,
                                             const int32_t* seq_lens, const int32_t* cu_seqlens_q,
                                             int64_t B, int64_t T, int64_t Hq, fp4_dtype_t dtype,
                                             float sm_scale, int causal, float softcap,
                                             const float* alibi_slopes, int64_t window,
                                             const int32_t* prefix_lens, void* out, float* lse,
                                             void* workspace, int64_t workspace_bytes,
                                             int32_t* status, int pdl, fp4q_stream_t stream);

/* Bytes of workspace fp4_attention_nvfp4 needs for exactly these sizes on the current
 * device (152 SMs taken when none is visible); max_keys = max_pages * page_size of its
 * call.  0 or more (0: none, workspace may be NULL), -1 on bad arguments.  A call with
 * fewer rows, sequences or keys may need more: one that fills the device by itself needs
 * none, one that has to cut its keys into ranges does. */
FP4Q_API int64_t fp4_attention_workspace_bytes(int64_t B, int64_t T, int64_t Hq, int64_t num_kv_heads,
                                               int64_t head_dim, int64_t max_keys);

/* Bytes that are enough for every call of at most B sequences, T query rows and
 * max_keys keys with these heads on the current device: what a program allocates once.
 * Grows with each size up to 4096 * SMs * (head_dim + 2) bytes (81 MB with 152 SMs and 128
 * channels), or to 8 bytes per sequence and per 8 rows of every key/value head where that
 * is more.  -1 on bad arguments. */
FP4Q_API int64_t fp4_attention_workspace_bound(int64_t B, int64_t T, int64_t Hq, int64_t num_kv_heads,
                                               int64_t head_dim, int64_t max_keys);

/*
 * fp4_attention_launch_shape - the kernel fp4_attention_nvfp4 would run for these
 * sizes on the current device (diagnostics; launches nothing; arguments as above).
 * Fills out[2] = {kernel (0 = the one for few rows or short sequences, 1 = the one in
 * 256-row items), parts}: of kernel 0 the CTAs that share an item (1 to 8; 0 = the keys
 * of all items are split evenly over the device and joined by a second kernel), of
 * kernel 1 the ranges that an item's keys are cut into (joined likewise if more than one).
 * FP4_OK, or FP4_ERR_INVALID_ARG.
 */
FP4Q_API fp4_status_t fp4_attention_launch_shape(int64_t B, int64_t T, int64_t Hq,
                                                 int64_t num_kv_heads, int64_t head_dim,
                                                 int64_t max_keys, int64_t out[2]);

/*
 * Pages of the cache between two tokens.  A sequence's pages are the first
 * ceil(len / page_size) entries of its row of block_tables; refs counts for every page
 * how many entries hold it, those of tables that are not in the call and those of any other
 * keeper (a store of prompts) included.  A page with refs <= 0 is free.  Entries outside
 * [0, num_pages) hold no page (pages given up behind a window: -1).
 * The three calls below read tables, lengths and counts and write new ones: the old ones
 * stay as they are, so a call can be repeated, and a loop goes back and forth between two
 * sets of buffers.  What they choose goes by the lowest number and does not change from call
 * to call.  All arrays are on the device and read there, so that a captured call follows
 * them; nothing that is written may overlap anything else the call reads or writes.
 *
 * fp4_kv_fork_nvfp4 - sequences are continued by their children (the next step of a beam
 * search, samples of one prompt, one more token of every sequence), and end.
 *
 *   refs           [num_pages] int32.
 *   tables, max_pages, seq_lens  [B, max_pages] and [B] int32: the old sequences.  All of them end
 *                  with the call; one goes on as itself by being a child's parent.
 *   parents        [N] int32: the old sequence that child i continues; outside [0, B) (beams that have
 *                  no candidate: -1): the child is empty.  NULL: child i continues sequence i (N == B, or
 *                  N == 0: all of them end).
 *   new_lens, new_tokens  [N] int32, or NULL: tokens that child i is about to append, at most (NULL:
 *                  exactly) new_tokens; 0 for an empty child.
 *   out_tables, out_seq_lens  [N, max_pages] and [N] int32: the children, with room for their new
 *                  tokens, which out_seq_lens counts (as fp4_attention_nvfp4 does); -1 behind a row's end.
 *   out_refs       [num_pages] int32, never negative.
 *   out_slots      [N, new_tokens] int64: where the new tokens go, as fp4_kv_append_nvfp4 takes them; -1
 *                  behind a child's last and where there is no page.  NULL with new_tokens 0.
 *   workspace      at least fp4_kv_pages_workspace_bytes(num_pages, N) bytes, 16-byte aligned, any
 *                  contents; two calls that may run at the same time need one each.
 *   status         as in fp4_add_rmsnorm_quant_ex; receives FP4_ERR_NO_PAGES where free pages or a
 *                  table's entries run out: the children behind (in order) then lack pages (entries
 *                  and slots -1), and a length stops at max_pages * page_size.
 * Children share their parents' full pages.  A last page that is not full and is about to be
 * written stays with its first child if nobody else holds it; every other child gets a
 * copy, of its tokens up to the next multiple of 16.  Pages are taken in the children's order, each the
 * lowest free one, those that the old sequences have left among them.
 */
FP4Q_API fp4_status_t fp4_kv_fork_nvfp4(const fp4_kv_cache_t* cache, const int32_t* refs,
                                        const int32_t* tables, int64_t max_pages,
                                        const int32_t* seq_lens, int64_t B, const int32_t* parents,
                                        const int32_t* new_lens, int64_t N, int64_t new_tokens,
                                        int32_t* out_tables, int32_t* out_seq_lens,
                                        int32_t* out_refs, int64_t* out_slots, void* workspace,
                                        int64_t workspace_bytes, int32_t* status, int pdl,
                                        fp4q_stream_t stream);

/*
 * fp4_kv_trim_nvfp4 - sequences give up tokens: those that end, drafted tokens that were not
 * taken, what lies behind a window.
 *
 *   first, end     [B] int32, or NULL (0; the length): tokens first .. end - 1 stay.  Pages that end
 *                  before place `first` and pages that begin at place `end` or behind it are given up:
 *                  out_tables has -1 there and everywhere behind the sequence's pages (and for an
 *                  entry that holds no page).  A page that both places lie in stays, and so it does
 *                  where no token does (first >= end): the next token goes there.
 *   out_seq_lens   [B] int32: min(end, length), not changed by first.
 *   out_refs       [num_pages] int32.
 * Other arguments as above.  Only the sizes of `cache` count; no page is read or written.
 */
FP4Q_API fp4_status_t fp4_kv_trim_nvfp4(const fp4_kv_cache_t* cache, const int32_t* refs,
                                        const int32_t* tables, int64_t max_pages,
                                        const int32_t* seq_lens, int64_t B, const int32_t* first,
                                        const int32_t* end, int32_t* out_tables,
                                        int32_t* out_seq_lens, int32_t* out_refs, int pdl,
                                        fp4q_stream_t stream);

/*
 * fp4_kv_compact_nvfp4 - the n pages with refs > 0 become pages 0 .. n - 1: those from n on
 * move to the free ones before n, both in ascending order, the others stay.
 *
 *   out_tables     [B, max_pages] int32: tables with the new numbers, -1 behind a sequence's pages and
 *                  for an entry that holds no page.
 *   out_refs       [num_pages] int32: the counts by the new numbers, 0 from n on.
 *   out_map        [num_pages] int32: every page's new number, -1 for a free one (for tables that
 *                  are not in the call).
 *   out_live       one int32: n.
 *   workspace      at least fp4_kv_pages_workspace_bytes(num_pages, 0) bytes, as above.
 * Pages from n on keep their bytes.
 */
FP4Q_API fp4_status_t fp4_kv_compact_nvfp4(const fp4_kv_cache_t* cache, const int32_t* refs,
                                           const int32_t* tables, int64_t max_pages,
                                           const int32_t* seq_lens, int64_t B, int32_t* out_tables,
                                           int32_t* out_refs, int32_t* out_map, int32_t* out_live,
                                           void* workspace, int64_t workspace_bytes, int pdl,
                                           fp4q_stream_t stream);

/* fp4_read_device_status and fp4_status_string under the names that cache programs use. */
FP4Q_API fp4_status_t fp4_kv_read_status(const int32_t* status, fp4q_stream_t stream);
FP4Q_API const char* fp4_kv_status_string(fp4_status_t status);

/* Bytes of workspace of a fork into N children (of a compaction: N = 0); grows with both.
 * -1 on bad arguments. */
FP4Q_API int64_t fp4_kv_pages_workspace_bytes(int64_t num_pages, int64_t N);

/*
 * fp4_beam_select - the best continuations of every beam search of a batch:
 * of batch entry b the n candidates (beam k, token v) with the largest
 *
 *   scores[b, k] + logits[b, k, v] - log(sum_v exp(logits[b, k, v]))
 *
 * in descending order.  Candidates of one beam are ordered by their logits,
 * equal ones by token, lowest first; of different beams by their scores (48 bits, and none
 * below a 64-bit number's steps), equal ones by beam.
 *
 *   logits, row_stride  [B * K, V] dtype (bf16, fp16 or fp32), row_stride elements between rows
 *                  (0: V); row b * K + k is beam k of entry b.  Any alignment that the type has.
 *   scores         [B, K] fp32.  A beam whose score is not finite has no candidates (dead beams, and
 *                  all but one at the start: -infinity), nor has one with a logit that is NaN or
 *                  above 2^125.  A logit of at most -2^125 (a mask of -infinity or of the type's lowest
 *                  value) is no candidate and adds nothing to the sum.  Between these they may lie
 *                  anywhere: tokens filled with -1e10 or -1e30, rows that are all as far from 0.
 *   finished       [B, K] bytes or NULL: a beam with a nonzero byte has ended; its one candidate
 *                  is end_token with its score as it is, whatever its logits are.
 *   end_token      in [0, V).
 *   K, V, n        beams (at most 256), vocabulary (at most 2^24), candidates to take (at most 64).
 *   out_scores     [B, n] fp32: the scores, rounded once; -infinity behind the last candidate.
 *   out_parents    [B, n] int32: row b * K + k of logits; -1 behind the last candidate.
 *   out_tokens     [B, n] int32: v; -1 behind the last candidate.
 *   out_finished   [B, n] bytes, NULL exactly when finished is: 1 where the parent has ended or the
 *                  token is end_token.
 *   workspace      at least fp4_beam_select_workspace_bytes(...) bytes, 16-byte aligned, any
 *                  contents; two calls that may run at the same time need one each.
 *   pdl            as in fp4_add_rmsnorm_quant_ex.
 * The exponentials are summed in fp32, the sums of a row's parts and the scores in pairs of fp32
 * (48 bits).  Results do not change from call to call.  Nothing that is written may overlap anything else the call
 * reads or writes.  out_parents is what fp4_kv_fork_nvfp4 takes as parents.
 */
FP4Q_API fp4_status_t fp4_beam_select(const void* logits, int64_t row_stride, fp4_dtype_t dtype,
                                      const float* scores, const uint8_t* finished,
                                      int64_t end_token, int64_t B, int64_t K, int64_t V, int64_t n,
                                      float* out_scores, int32_t* out_parents, int32_t* out_tokens,
                                      uint8_t* out_finished, void* workspace,
                                      int64_t workspace_bytes, int pdl, fp4q_stream_t stream);

/* Bytes of workspace of fp4_beam_select; grows with each size.  -1 on bad arguments. */
FP4Q_API int64_t fp4_beam_select_workspace_bytes(int64_t B, int64_t K, int64_t V, int64_t n,
                                                 fp4_dtype_t dtype);

/*
 * fp4_read_device_status - synchronises `stream`, then copies the device
 * status word back and returns it as a status: FP4_OK (0), FP4_ERR_TIMEOUT or
 * FP4_ERR_NO_PAGES; FP4_ERR_INVALID_ARG for a NULL or misaligned pointer or a value that is no
 * status; FP4_ERR_CUDA if the synchronisation or the copy failed.  Blocks the
 * calling thread; not for use inside stream capture.
 */
FP4Q_API fp4_status_t fp4_read_device_status(const int32_t* status, fp4q_stream_t stream);

/*
 * Debug build.  `python -m rmsnorm_fp4_quant_gb300.build --debug` also builds
 * libfp4q_debug.so: the same entry points compiled with checks of every
 * global address a kernel computes against the extent of its buffer (an
 * access outside it is counted and skipped, never made), and with a fault
 * injector for the bounded waits.  The default libfp4q.so carries neither.
 *
 * fp4_debug_build - 1 in the debug build, 0 in the default one.
 *
 * fp4_debug_configure - process-wide knobs of the debug build, applied to
 * every later launch (FP4_ERR_INVALID_ARG in the default build):
 *   wait_limit_cycles  clock cycles each bounded wait allows (> 0; about one
 *                      second, 2e9, unless changed);
 *   shrink_bytes       bytes taken off every buffer extent the checks use
 *                      (>= 0; 0 for the real extents), so a test can see the
 *                      checks catch the accesses near the end of a buffer;
 *   drop_kernel        0 none, 1 the wide-row fused kernel, 2 the GEMM: CTA
 *                      `drop_cta` arrives on a stage's barrier expecting the
 *                      bytes of a copy it then never issues, at ring iteration
 *                      (fused) or K-block count (GEMM) `drop_iter`, so that
 *                      the wait on that stage runs out with nothing in flight
 *                      for it and the kernel's timeout path runs;
 *   violations         DEVICE uint32_t counter (4-byte aligned) that the
 *                      checks increment, or NULL (not counted).
 * These knobs are for tests; no default build reads them.
 */
FP4Q_API int fp4_debug_build(void);
FP4Q_API fp4_status_t fp4_debug_configure(int64_t wait_limit_cycles, int64_t shrink_bytes,
                                          int drop_kernel, int drop_cta, int drop_iter,
                                          uint32_t* violations);

/* Static, NUL-terminated description of a status code. */
FP4Q_API const char* fp4_status_string(fp4_status_t status);

/* cudaError_t value behind the last FP4_ERR_CUDA returned on this thread (0 if none). */
FP4Q_API int fp4_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* FP4Q_H_ */
