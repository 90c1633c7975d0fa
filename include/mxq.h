/*
 * mxq.h -- C ABI of the MI355X (gfx950) block-scaled weight-quantization library.
 *
 * Five entry points make up the path:
 *   mxq_fake_quantize_mxfp4     per-1x32 MXFP4 projection, output in the input dtype
 *   mxq_mxfp4_to_mxfp8_row      direct MXFP8 rowwise lift (E4M3 payload + E8M0 codes)
 *   mxq_mxfp4_to_fp8_block128   direct 128x128 blockwise FP8 (E4M3 payload + tile codes)
 *   mxq_export_mxfp8            unpadded (*shape[:-1], ceil(K/32)) E8M0 scale export
 *   mxq_dequantize              FP8 payload + E8M0 codes -> bf16 / fp32
 * variants of them:
 *   mxq_fake_quantize_mxfp4_with_mxfp8_row    projection + row lift in one pass
 *   mxq_mxfp4_to_mxfp8_row_guarded,
 *   mxq_mxfp4_to_fp8_block128_guarded         the direct conversions behind a device no-op flag
 *   mxq_mxfp4_to_mxfp8_row_grouped, mxq_fake_quantize_mxfp4_grouped,
 *   mxq_mxfp4_to_fp8_block128_grouped,
 *   mxq_dequantize_grouped                    the row lift / projection / fold / decode of a list
 *                                             of weights in few launches
 * the packed MXFP4 deployment format:
 *   mxq_quantize_mxfp4, mxq_dequantize_mxfp4,
 *   mxq_mxfp4_packed_to_mxfp8_row, mxq_mxfp4_packed_to_fp8_block128,
 *   mxq_quantize_mxfp4_grouped (the encode of a list of weights in few launches)
 * and MXFP8 columnwise (32x1) from the decomposition:
 *   mxq_mxfp4_to_mxfp8_col, mxq_mxfp4_to_mxfp8_row_col (row and column in one pass),
 *   and their no-op-flag-gated forms mxq_mxfp4_to_mxfp8_col_guarded,
 *   mxq_mxfp4_to_mxfp8_row_col_guarded
 * and the products of a layer whose weights are 128x128 blockwise FP8, with the
 * routing of a layer of experts around them:
 *   mxq_quantize_fp8_group128, mxq_quantize_fp8_group128_col,
 *   mxq_quantize_fp8_group128_row_col       activations and gradients in FP8, groups of 128
 *   mxq_matmul_fp8_block128                 y = x w^T
 *   mxq_matmul_fp8_block128_dgrad           dx = dy w
 *   mxq_matmul_fp8_group128_wgrad           dw = dy^T x
 *   mxq_sort_experts, mxq_sort_experts_workspace, mxq_dispatch_rows,
 *   mxq_combine_rows, mxq_combine_rows_backward
 * and what stands between those products, each with its backward pass:
 *   mxq_rms_norm, mxq_rms_norm_fp8_group128, mxq_rms_norm_fp8_group128_row_col,
 *   mxq_rms_norm_backward           the norm before them, with the residual's addition
 *   mxq_activate_fp8_group128, mxq_activate_fp8_group128_row_col,
 *   mxq_activate_fp8_group128_backward      the (gated) activation between two of them
 *   mxq_route_experts, mxq_route_experts_backward   tokens to experts, and their weights
 *
 * Sources, by page title and section:
 *   [QAT] "[PyTorch] MXFP4 weight QAT on MXFP8 and FP8 block-scaling recipes"
 *         (TransformerEngine pull request 3264): Description, Test results (B200),
 *         Known limitations.
 *   [EXP] "MXFP8TensorStorage.export_components()" (TransformerEngine pull request
 *         3790): Description.
 *
 * Conventions for every entry point:
 *   - A matrix is [rows, K]: leading dimensions are flattened into rows and the
 *     last dimension K is contiguous.  Every ld / scale_ld / tile_ld is a row
 *     stride counted in elements of that buffer.
 *   - All pointers are device pointers.  The caller owns every buffer; the
 *     library never allocates, frees or keeps a pointer, holds no state and is
 *     safe to call from several host threads.
 *   - Work is enqueued on `stream` (0 = the null stream) and is asynchronous.
 *     Argument errors are detected on the host and returned before anything is
 *     enqueued; no kernel asserts on the device.
 *   - rows == 0 or K == 0 returns MXQ_OK and enqueues nothing.
 *   - Results of the quantizers are bit-exact (the products and the rows'
 *     weighted sums round as stated at their entry points) and do not depend
 *     on the build's floating-point flags: the scale exponents are integer arithmetic on bit patterns, and the
 *     kernels set the wave's denormal mode before using the gfx950 scaled
 *     conversions.
 */
#ifndef MXQ_H
#define MXQ_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of a high-precision buffer.  fp16 exists only to be rejected:
 * the MXFP4 grid exceeds its range ([QAT] Description, STE paragraph, and
 * Known limitations). */
typedef enum { MXQ_BF16 = 0, MXQ_FP32 = 1, MXQ_FP16 = 2 } mxq_dtype;

/* FP8 payload format: OCP E4M3 "FN" (bias 7, max 448, NaN = S.1111.111, no Inf)
 * or E5M2 (bias 15, IEEE Inf/NaN) -- the torch.float8_e4m3fn / float8_e5m2 views
 * of [EXP] Description. */
typedef enum { MXQ_E4M3 = 0, MXQ_E5M2 = 1 } mxq_fp8;

/* Where a payload element's E8M0 code lives: one per 1x32 block of a row
 * (scale[r*scale_ld + c/32]), one per 128x128 tile anchored at (0,0)
 * (scale[(r/128)*scale_ld + c/128]), or one per 32x1 block of a column
 * anchored at row 0 (scale[(r/32)*scale_ld + c]). */
typedef enum { MXQ_SCALE_ROW_1X32 = 0, MXQ_SCALE_TILE_128X128 = 1, MXQ_SCALE_COL_32X1 = 2 } mxq_scale_layout;

/* Status codes. */
enum {
  MXQ_OK = 0,
  MXQ_ERR_NULL = 1,             /* a required pointer is NULL (non-empty shape) */
  MXQ_ERR_SHAPE = 2,            /* negative dims, ld < K, scale_ld / tile_ld too small, too many steps
                                   for one launch, or a matrix spanning 2^56 bytes or more (or past the
                                   end of the address space) */
  MXQ_ERR_DTYPE = 3,            /* fp16 or an unknown dtype / format / layout */
  MXQ_ERR_NO_ROWWISE_DATA = 4,  /* export without payload or scale storage ([EXP]: ValueError) */
  MXQ_ERR_ALIAS = 5,            /* an output overlaps an input (other than the allowed exact in-place) */
  MXQ_ERR_HIP = 6               /* the HIP runtime refused a launch: hipGetLastError() was not
                                   hipSuccess right after it.  That includes an error left pending by
                                   an earlier HIP call on the calling thread, which the call then
                                   consumes, as hipGetLastError() does. */
};

/* Human-readable text of a status code (static storage; never NULL). */
const char* mxq_status_string(int status);

/*
 * MXFP4 projection (fake quantization), [QAT] Description, conversion mode 1.
 * For each 1x32 block of a row (the last block of a row may be shorter and
 * keeps its own scale, [EXP] Description): amax = max |x|; scale exponent
 * e = clamp(ceil(log2(amax/6)), -126, 125), taken from amax's bit pattern;
 * y = RTNE_E2M1(x / 2^e) * 2^e, i.e. x rounded to the nearest of
 * {0, .5, 1, 1.5, 2, 3, 4, 6} * 2^e with ties to the even E2M1 code, sign kept
 * (including -0), saturating at 6 * 2^e ([QAT] Known limitations: amax above
 * 6*2^125 saturates at the cap).  A block holding any Inf or NaN becomes all
 * canonical quiet NaN (0x7FC0 / 0x7FC00000) ([QAT] Test results: non-finite
 * block poisoning).  amax = 0 uses e = -126.
 *   x    [rows, K] bf16 or fp32, row stride ld_x >= K
 *   y    [rows, K] same dtype, row stride ld_y >= K.  y == x with ld_y == ld_x
 *        (in place) is allowed; any other overlap is MXQ_ERR_ALIAS.
 *   dt   MXQ_BF16 or MXQ_FP32 (MXQ_FP16 -> MXQ_ERR_DTYPE)
 */
int mxq_fake_quantize_mxfp4(const void* x, int64_t ld_x, void* y, int64_t ld_y,
                            int64_t rows, int64_t K, mxq_dtype dt, hipStream_t stream);

/*
 * Direct MXFP8 rowwise lift, [QAT] Description, conversion mode 2: a lift by a
 * fixed shift of 6 whose scale stops at UE8M0 code 0, the payload taking up the
 * rest of the shift exactly.
 * From each block's MXFP4 decomposition x ~ p * 2^e of the master weight (the
 * same e and p as mxq_fake_quantize_mxfp4): scale code = max(e + 121, 0), i.e.
 * scale 2^(e-6) clamped at 2^-127, and payload = E4M3(p * 2^min(6, e+127)),
 * which is always exact.  Decoding payload * 2^(code-127) gives back the
 * projection bit for bit.  A poisoned block gets code 255 and payload 0x7F.
 *   x         [rows, K] bf16 or fp32, row stride ld_x >= K
 *   data      [rows, K] uint8 E4M3 payload, contiguous (row stride K)
 *   scale     [rows, scale_ld] uint8 E8M0 codes, scale_ld >= ceil(K/32); columns
 *             j >= ceil(K/32) (padding) are not written
 *   data and scale must not overlap x or each other (MXQ_ERR_ALIAS).
 */
int mxq_mxfp4_to_mxfp8_row(const void* x, int64_t ld_x, int64_t rows, int64_t K, mxq_dtype dt,
                           uint8_t* data, uint8_t* scale, int64_t scale_ld, hipStream_t stream);

/*
 * Direct 128x128 blockwise FP8, [QAT] Description, conversion mode 2: the block
 * exponents are folded into one scale per tile, 2^(largest FP4 exponent - 6)
 * with 2^-127 as its floor, and the payload is rounded to nearest-even onto
 * E4M3, subnormals included.  Tiles are anchored at (0,0) and truncated at the
 * edges.  Per tile: M = max e over its finite 1x32 blocks (-126 if none);
 * S = max(M - 6, -127); tile code = S + 127; payload = RTNE_E4M3(p * 2^(e - S))
 * with E4M3 subnormals and ties to even.  Exact while the tile's exponent
 * spread M - e is at most 14 ([QAT] Test results).  Poisoned blocks are left out
 * of M and get payload 0x7F.
 *   x          [rows, K] bf16 or fp32, row stride ld_x >= K
 *   data       [rows, K] uint8 E4M3 payload, contiguous (row stride K)
 *   tile_code  [ceil(rows/128), tile_ld] uint8 E8M0 codes, tile_ld >= ceil(K/128)
 *   data and tile_code must not overlap x or each other (MXQ_ERR_ALIAS).
 */
int mxq_mxfp4_to_fp8_block128(const void* x, int64_t ld_x, int64_t rows, int64_t K, mxq_dtype dt,
                              uint8_t* data, uint8_t* tile_code, int64_t tile_ld, hipStream_t stream);

/*
 * Projection and direct MXFP8 row lift in one pass over the weight: writes the
 * outputs of mxq_fake_quantize_mxfp4 (y) and of mxq_mxfp4_to_mxfp8_row (data,
 * scale) from a single read of x.  [QAT] Known limitations names a fused
 * projection + quantize kernel as future work; the results are bit-identical to
 * the two separate calls.  Arguments and rules as for those two calls (y == x
 * with ld_y == ld_x is allowed; every other overlap is MXQ_ERR_ALIAS).
 */
int mxq_fake_quantize_mxfp4_with_mxfp8_row(const void* x, int64_t ld_x, void* y, int64_t ld_y, int64_t rows,
                                           int64_t K, mxq_dtype dt, uint8_t* data, uint8_t* scale,
                                           int64_t scale_ld, hipStream_t stream);

/*
 * mxq_mxfp4_to_mxfp8_row / mxq_mxfp4_to_fp8_block128 gated by a device-side
 * no-op flag: when *noop != 0 at the time the work runs on the stream, every
 * output is left untouched.  For cached-weight updates inside a captured HIP
 * graph, where a replay must be able to keep the existing workspace ([QAT]
 * review: the CUDA-graph skip-update flag must gate the cached update).
 *   noop   device pointer to one int32, read by the kernels; required (NULL ->
 *          MXQ_ERR_NULL).  Other arguments as for the ungated calls.  The
 *          input is read either way (the kernels issue their input loads
 *          before they read the flag), so x must be valid in both cases.
 */
int mxq_mxfp4_to_mxfp8_row_guarded(const void* x, int64_t ld_x, int64_t rows, int64_t K, mxq_dtype dt,
                                   uint8_t* data, uint8_t* scale, int64_t scale_ld, const int32_t* noop,
                                   hipStream_t stream);
int mxq_mxfp4_to_fp8_block128_guarded(const void* x, int64_t ld_x, int64_t rows, int64_t K, mxq_dtype dt,
                                      uint8_t* data, uint8_t* tile_code, int64_t tile_ld, const int32_t* noop,
                                      hipStream_t stream);

/*
 * One weight of a grouped row lift: the arguments of mxq_mxfp4_to_mxfp8_row for
 * that weight (x, data and scale are device pointers).
 */
typedef struct {
  const void* x;      /* [rows, K], row stride ld_x >= K */
  int64_t ld_x;
  int64_t rows;
  int64_t K;
  uint8_t* data;      /* [rows, K] E4M3 payload, contiguous */
  uint8_t* scale;     /* [rows, scale_ld] E8M0 codes, scale_ld >= ceil(K/32); padding not written */
  int64_t scale_ld;
} mxq_row_group;

/*
 * The direct MXFP8 row lift of mxq_mxfp4_to_mxfp8_row applied to a list of
 * weights of one dtype (the experts of a grouped linear layer, [QAT] Test
 * results, end-to-end cases), in as few launches as possible: every launch
 * carries a fixed cost of a few microseconds, which dominates for small weights.
 * Results are bit-identical to one mxq_mxfp4_to_mxfp8_row call per weight.
 *   groups    HOST array of n_groups descriptors, read during the call only
 *   n_groups  >= 0; groups with rows == 0 or K == 0 are skipped
 *   Every group is checked as mxq_mxfp4_to_mxfp8_row checks its arguments (the
 *   first failing group's status is returned and nothing is enqueued).  In
 *   addition no group's data or scale may overlap any group's x, data or scale
 *   (MXQ_ERR_ALIAS); inputs may overlap each other.
 */
int mxq_mxfp4_to_mxfp8_row_grouped(const mxq_row_group* groups, int64_t n_groups, mxq_dtype dt,
                                   hipStream_t stream);

/*
 * One weight of a grouped projection: the arguments of mxq_fake_quantize_mxfp4
 * for that weight (x and y are device pointers).
 */
typedef struct {
  const void* x;      /* [rows, K], row stride ld_x >= K */
  int64_t ld_x;
  void* y;            /* [rows, K] same dtype, row stride ld_y >= K; y == x with ld_y == ld_x is in place */
  int64_t ld_y;
  int64_t rows;
  int64_t K;
} mxq_proj_group;

/*
 * The MXFP4 projection of mxq_fake_quantize_mxfp4 ([QAT] Description, conversion
 * mode 1, the default mode) applied to a list of weights of one dtype, in as
 * few launches as possible.  Results are bit-identical to one
 * mxq_fake_quantize_mxfp4 call per weight.
 *   groups    HOST array of n_groups descriptors, read during the call only
 *   n_groups  >= 0; groups with rows == 0 or K == 0 are skipped
 *   Every group is checked as mxq_fake_quantize_mxfp4 checks its arguments
 *   (the first failing group's status is returned and nothing is enqueued).
 *   In addition no group's y may overlap any other group's x or y
 *   (MXQ_ERR_ALIAS); inputs may overlap each other, and a group may be in place.
 */
int mxq_fake_quantize_mxfp4_grouped(const mxq_proj_group* groups, int64_t n_groups, mxq_dtype dt,
                                    hipStream_t stream);

/*
 * One weight of a grouped 128x128 fold: the arguments of
 * mxq_mxfp4_to_fp8_block128 for that weight (x, data and tile_code are device
 * pointers).
 */
typedef struct {
  const void* x;      /* [rows, K], row stride ld_x >= K */
  int64_t ld_x;
  int64_t rows;
  int64_t K;
  uint8_t* data;      /* [rows, K] E4M3 payload, contiguous */
  uint8_t* tile_code; /* [ceil(rows/128), tile_ld] E8M0 tile codes, tile_ld >= ceil(K/128) */
  int64_t tile_ld;
} mxq_block128_group;

/*
 * The direct 128x128 blockwise FP8 fold of mxq_mxfp4_to_fp8_block128 ([QAT]
 * Description, conversion mode 2) applied to a list of weights of one dtype,
 * in as few launches as possible.  Results are bit-identical to one
 * mxq_mxfp4_to_fp8_block128 call per weight.
 *   groups    HOST array of n_groups descriptors, read during the call only
 *   n_groups  >= 0; groups with rows == 0 or K == 0 are skipped
 *   Every group is checked as mxq_mxfp4_to_fp8_block128 checks its arguments
 *   (the first failing group's status is returned and nothing is enqueued).
 *   In addition no group's data or tile_code may overlap any group's x, data
 *   or tile_code (MXQ_ERR_ALIAS); inputs may overlap each other.
 */
int mxq_mxfp4_to_fp8_block128_grouped(const mxq_block128_group* groups, int64_t n_groups, mxq_dtype dt,
                                      hipStream_t stream);

/*
 * MXFP8 columnwise from the MXFP4 decomposition ([QAT] Description, conversion
 * mode 2, and its MXFP8 weight dataflow without a backward override, where the
 * dgrad operand is built from the same decomposition): a fresh MXFP8
 * quantization of the projected weight y = p * 2^e over 32x1 blocks, i.e. 32
 * consecutive rows of one column, anchored at row 0 (the last block may be
 * short).  The pages require these bytes to equal the host quantizer's bytes for
 * the projected weight and name its amax rule without writing it out; the rule
 * taken is the OCP MX one: S = floor(log2 amax) - 8 (8 = E4M3's largest
 * exponent), raised to -127 if lower; code = S + 127; payload =
 * RTNE_E4M3(y / 2^S) with subnormals.  On projected weights amax has at most two
 * significant bits, so S also equals ceil(log2(amax / 448)) and nothing
 * saturates.  amax is over the block's finite values: elements of poisoned row
 * blocks (NaN in the projection) get payload 0x7F; a block with no nonzero
 * finite value gets code 0.  Unlike the row lift this re-rounds: decode gives
 * back the projection wherever y / 2^S is a multiple of 2^-9.
 *   x      [rows, K] bf16 or fp32, row stride ld_x >= K
 *   data   [rows, K] uint8 E4M3 payload in x's (untransposed) layout, contiguous
 *   scale  [ceil(rows/32), scale_ld] uint8 E8M0 codes, scale_ld >= K; columns
 *          j >= K of each scale row are left untouched
 *   data and scale must not overlap x or each other (MXQ_ERR_ALIAS).
 */
int mxq_mxfp4_to_mxfp8_col(const void* x, int64_t ld_x, int64_t rows, int64_t K, mxq_dtype dt, uint8_t* data,
                           uint8_t* scale, int64_t scale_ld, hipStream_t stream);

/*
 * The MXFP8 rowwise lift (mxq_mxfp4_to_mxfp8_row) and the columnwise conversion
 * (mxq_mxfp4_to_mxfp8_col) from one read of x: the pair the MXFP8 weight
 * dataflow without a backward override keeps for the forward and backward GEMMs
 * ([QAT] Description, weight dataflows).  Outputs are bit-identical to the two
 * separate calls; arguments as for them.  No output may overlap x or another
 * output (MXQ_ERR_ALIAS).
 */
int mxq_mxfp4_to_mxfp8_row_col(const void* x, int64_t ld_x, int64_t rows, int64_t K, mxq_dtype dt,
                               uint8_t* row_data, uint8_t* row_scale, int64_t row_scale_ld, uint8_t* col_data,
                               uint8_t* col_scale, int64_t col_scale_ld, hipStream_t stream);

/*
 * mxq_mxfp4_to_mxfp8_col / mxq_mxfp4_to_mxfp8_row_col gated by a device-side
 * no-op flag, as mxq_mxfp4_to_mxfp8_row_guarded: when *noop != 0 at the time
 * the work runs on the stream, every output is left untouched.  [QAT]'s
 * flowchart has the skip-update flag gate every conversion into the cached
 * workspace, the columnwise one included.
 *   noop   device pointer to one int32; required (NULL -> MXQ_ERR_NULL).
 *          Other arguments as for the ungated calls.
 */
int mxq_mxfp4_to_mxfp8_col_guarded(const void* x, int64_t ld_x, int64_t rows, int64_t K, mxq_dtype dt,
                                   uint8_t* data, uint8_t* scale, int64_t scale_ld, const int32_t* noop,
                                   hipStream_t stream);
int mxq_mxfp4_to_mxfp8_row_col_guarded(const void* x, int64_t ld_x, int64_t rows, int64_t K, mxq_dtype dt,
                                       uint8_t* row_data, uint8_t* row_scale, int64_t row_scale_ld,
                                       uint8_t* col_data, uint8_t* col_scale, int64_t col_scale_ld,
                                       const int32_t* noop, hipStream_t stream);

/*
 * Unpadded export of MXFP8 rowwise scales, [EXP] Description: scale_inv holds
 * E8M0 codes with shape (*shape[:-1], ceil(K/32)), without padding; a partial
 * last block keeps its own scale.  Copies the first ceil(K/32) columns of each
 * row of the padded storage into a compact [rows, ceil(K/32)] array.  The
 * payload needs no copy: it is `data` viewed with the tensor's shape.
 *   data           the payload (only checked for presence)
 *   scale_storage  [rows, scale_ld] uint8, scale_ld >= ceil(K/32)
 *   scale_out      [rows, ceil(K/32)] uint8, contiguous
 * data == NULL or scale_storage == NULL -> MXQ_ERR_NO_ROWWISE_DATA ([EXP]: a
 * tensor without row-scaled data raises ValueError).  scale_out == scale_storage
 * with scale_ld == ceil(K/32) is the view case and returns MXQ_OK without work;
 * any other overlap is MXQ_ERR_ALIAS.
 */
int mxq_export_mxfp8(const uint8_t* data, const uint8_t* scale_storage, int64_t rows, int64_t K,
                     int64_t scale_ld, uint8_t* scale_out, hipStream_t stream);

/*
 * Decode FP8 payload with E8M0 codes: out = RNE_out(FP8(q) * 2^(code - 127)).
 * Code 0 is 2^-127 and code 255 is NaN ([QAT] Description: decode UE8M0 code 0
 * as 2^-127 and code 255 as NaN; Test results: planted extreme codes).  A NaN
 * payload or code 255 gives canonical quiet NaN; an E5M2 infinity stays
 * infinite; values beyond the output range round to Inf.
 *   data     [rows, K] uint8 payload, contiguous (row stride K)
 *   scale    E8M0 codes: [rows, scale_ld] for MXQ_SCALE_ROW_1X32 (scale_ld >=
 *            ceil(K/32)), [ceil(rows/128), scale_ld] for MXQ_SCALE_TILE_128X128
 *            (scale_ld >= ceil(K/128)) or [ceil(rows/32), scale_ld] for
 *            MXQ_SCALE_COL_32X1 (scale_ld >= K)
 *   out      [rows, K] bf16 or fp32, row stride ld_out >= K; must not overlap
 *            data or scale
 */
int mxq_dequantize(const uint8_t* data, const uint8_t* scale, int64_t scale_ld, int64_t rows, int64_t K,
                   mxq_fp8 fmt, mxq_scale_layout layout, void* out, int64_t ld_out, mxq_dtype out_dt,
                   hipStream_t stream);

/*
 * One weight of a grouped decode: the arguments of mxq_dequantize for that
 * weight (data, scale and out are device pointers).
 */
typedef struct {
  const uint8_t* data;   /* [rows, K] uint8 payload, contiguous */
  const uint8_t* scale;  /* E8M0 codes in the call's layout, row stride scale_ld */
  int64_t scale_ld;
  int64_t rows;
  int64_t K;
  void* out;             /* [rows, K] in the call's output dtype, row stride ld_out >= K */
  int64_t ld_out;
} mxq_dequant_group;

/*
 * The decode of mxq_dequantize (code 0 is 2^-127 and code 255 NaN, [QAT]
 * Description; the same NaN and overflow rules) applied to a list of weights
 * with one payload format, scale layout and output dtype (the experts of a
 * grouped linear layer, [QAT] Test results, end-to-end cases), in as few
 * launches as possible.  Results are bit-identical to one mxq_dequantize call
 * per weight.
 *   groups    HOST array of n_groups descriptors, read during the call only
 *   n_groups  >= 0; groups with rows == 0 or K == 0 are skipped
 *   Every group is checked as mxq_dequantize checks its arguments (the first
 *   failing group's status is returned and nothing is enqueued).  In addition
 *   no group's out may overlap any group's data, scale or out (MXQ_ERR_ALIAS);
 *   inputs may overlap each other.
 */
int mxq_dequantize_grouped(const mxq_dequant_group* groups, int64_t n_groups, mxq_fp8 fmt,
                           mxq_scale_layout layout, mxq_dtype out_dt, hipStream_t stream);

/*
 * Packed MXFP4, the deployment format: E2M1 payloads with 1x32 power-of-two
 * E8M0 scales ([QAT] Description: the weight seen in training is the deployed
 * one; the export issue's workflow 2, quantizing weights for inference).
 * Layout: packed [rows, ceil(K/2)] uint8, contiguous, element 2i in the low
 * nibble of byte i and 2i+1 in the high nibble (0 when K is odd); each nibble
 * is S.EE.M (sign, then the 3-bit E2M1 code of {0, .5, 1, 1.5, 2, 3, 4, 6}).
 * scale [rows, scale_ld] uint8 E8M0 codes, scale_ld >= ceil(K/32).
 *
 * mxq_quantize_mxfp4: the projection's decomposition (same blocks, same RTNE),
 * except that above the cap the scale moves to 2^126 ([QAT] Known limitations):
 * e = clamp(ceil(log2(amax/6)), -126, 126), code = e + 127.  Below the cap the
 * decoded packed weight equals mxq_fake_quantize_mxfp4's output bit for bit.
 * A block holding Inf or NaN gets code 255 and zero nibbles.
 */
int mxq_quantize_mxfp4(const void* x, int64_t ld_x, int64_t rows, int64_t K, mxq_dtype dt, uint8_t* packed,
                       uint8_t* scale, int64_t scale_ld, hipStream_t stream);

/*
 * One weight of a grouped packed MXFP4 encode: the arguments of
 * mxq_quantize_mxfp4 for that weight (x, packed and scale are device pointers).
 */
typedef struct {
  const void* x;      /* [rows, K], row stride ld_x >= K */
  int64_t ld_x;
  int64_t rows;
  int64_t K;
  uint8_t* packed;    /* [rows, ceil(K/2)] nibble pairs, contiguous */
  uint8_t* scale;     /* [rows, scale_ld] E8M0 codes, scale_ld >= ceil(K/32); padding not written */
  int64_t scale_ld;
} mxq_mxfp4_group;

/*
 * The packed MXFP4 encode of mxq_quantize_mxfp4 (the deployment format, [QAT]
 * Description and Known limitations) applied to a list of weights of one
 * dtype (the experts of a grouped linear layer), in as few launches as
 * possible.  Results are bit-identical to one mxq_quantize_mxfp4 call per
 * weight.
 *   groups    HOST array of n_groups descriptors, read during the call only
 *   n_groups  >= 0; groups with rows == 0 or K == 0 are skipped
 *   Every group is checked as mxq_quantize_mxfp4 checks its arguments (the
 *   first failing group's status is returned and nothing is enqueued).  In
 *   addition no group's packed or scale may overlap any group's x, packed or
 *   scale (MXQ_ERR_ALIAS); inputs may overlap each other.
 */
int mxq_quantize_mxfp4_grouped(const mxq_mxfp4_group* groups, int64_t n_groups, mxq_dtype dt,
                               hipStream_t stream);

/* Decode packed MXFP4: out = RNE_out(E2M1 * 2^(code-127)); code 255 -> canonical
 * NaN; values beyond the output range (codes 253, 254) -> Inf.  out [rows, K]
 * bf16 / fp32 with row stride ld_out >= K; must not overlap the inputs. */
int mxq_dequantize_mxfp4(const uint8_t* packed, const uint8_t* scale, int64_t scale_ld, int64_t rows, int64_t K,
                         void* out, int64_t ld_out, mxq_dtype out_dt, hipStream_t stream);

/* Direct MXFP8 row lift from packed MXFP4 (no bf16 re-encode): the fixed-shift-6
 * lift of mxq_mxfp4_to_mxfp8_row with (p, e = code - 127) read from the packed
 * weight: scale_out code max(code - 6, 0), payload E4M3(p * 2^min(6, code)),
 * exact; code 255 -> code 255 and payload 0x7F.  data [rows, K] contiguous;
 * scale_out [rows, scale_out_ld], padding columns untouched. */
int mxq_mxfp4_packed_to_mxfp8_row(const uint8_t* packed, const uint8_t* scale, int64_t scale_ld, int64_t rows,
                                  int64_t K, uint8_t* data, uint8_t* scale_out, int64_t scale_out_ld,
                                  hipStream_t stream);

/* Direct 128x128 blockwise FP8 from packed MXFP4: the tile fold of
 * mxq_mxfp4_to_fp8_block128 with each block's (p, e) read from the packed
 * weight; blocks with code 255 are the poisoned ones. */
int mxq_mxfp4_packed_to_fp8_block128(const uint8_t* packed, const uint8_t* scale, int64_t scale_ld, int64_t rows,
                                     int64_t K, uint8_t* data, uint8_t* tile_code, int64_t tile_ld,
                                     hipStream_t stream);

/*
 * FP8 quantization of activations and gradients: the operands that meet a
 * 128x128 blockwise FP8 weight (mxq_mxfp4_to_fp8_block128) in a product.  One
 * E8M0 code for each group of 128: amax = max |x| over the group, S =
 * max(ceil(log2(amax / 448)), -127), code = S + 127, payload = RTNE_E4M3(x / 2^S)
 * with subnormals (nothing saturates).  amax = 0 gets code 0.  A group holding
 * an Inf or NaN gets code 255 and payload 0x7F.  The last group of an axis may
 * be short and keeps its own code.
 *   x        [x_rows, K] bf16 or fp32, row stride ld_x >= K
 *   rows     rows of the result.  slots == NULL: row r is x's row r (rows <=
 *            x_rows).  Else slots is a device array of `rows` int32 and row r is
 *            x's row slots[r] / top_k, the token of that slot as
 *            mxq_sort_experts numbers them; a negative slot or one whose row is
 *            not below x_rows gives a row of zeros.
 * mxq_quantize_fp8_group128: groups along the row.
 *   data     [rows, K] E4M3 payload, row stride ld_data >= K
 *   scale    [rows, scale_ld] E8M0 codes, scale_ld >= ceil(K/128)
 * mxq_quantize_fp8_group128_col: groups of 128 rows of one column, the operand of
 * a weight gradient (payload in x's layout, not transposed).
 *   offsets  NULL: groups are anchored at row 0 and scale is [ceil(rows/128),
 *            scale_ld].  Else a device array of n_experts + 1 int32 (1 <=
 *            n_experts <= 512): expert e owns rows [offsets[e], offsets[e+1]),
 *            its groups begin at its first row, and scale is [rows/128 (rounded
 *            down) + n_experts, scale_ld], the experts' groups in order; code
 *            rows that no group needs are 0 (also in a call on no rows), and rows of no expert (from
 *            offsets[n_experts] on, or before offsets[0]) have payload 0.  Offsets are taken as
 *            clamped to [0, rows] and to a rising order.
 *   data     [rows, K], row stride ld_data >= K;  scale_ld >= K
 * mxq_quantize_fp8_group128_row_col: both from one read of x (the row groups of
 * rows of no expert are quantized like any others).
 * Any overlap of an output with an input or another output is MXQ_ERR_ALIAS.
 * Dimensions above 2^30 are MXQ_ERR_SHAPE, here and below.
 */
int mxq_quantize_fp8_group128(const void* x, int64_t ld_x, int64_t x_rows, int64_t rows, int64_t K, mxq_dtype dt,
                              const int32_t* slots, int64_t top_k, uint8_t* data, int64_t ld_data, uint8_t* scale,
                              int64_t scale_ld, hipStream_t stream);
int mxq_quantize_fp8_group128_col(const void* x, int64_t ld_x, int64_t x_rows, int64_t rows, int64_t K, mxq_dtype dt,
                                  const int32_t* slots, int64_t top_k, const int32_t* offsets, int64_t n_experts,
                                  uint8_t* data, int64_t ld_data, uint8_t* scale, int64_t scale_ld,
                                  hipStream_t stream);
int mxq_quantize_fp8_group128_row_col(const void* x, int64_t ld_x, int64_t x_rows, int64_t rows, int64_t K,
                                      mxq_dtype dt, const int32_t* slots, int64_t top_k, const int32_t* offsets,
                                      int64_t n_experts, uint8_t* row_data, int64_t ld_row, uint8_t* row_scale,
                                      int64_t row_scale_ld, uint8_t* col_data, int64_t ld_col, uint8_t* col_scale,
                                      int64_t col_scale_ld, hipStream_t stream);

/*
 * Products with 128x128 blockwise FP8 weights, on the matrix cores.  Operands are
 * E4M3 payloads with E8M0 codes as above; the sum over the reduction is held in
 * fp32 and rounded once to the output's type (fast_accum below).  Its order is fixed by
 * the sizes and alignment of the call: the same call gives the same bits, but a
 * row's last places may differ between calls with other numbers of rows.
 *   mxq_matmul_fp8_block128        y[M, N]  = x[M, K] w[N, K]^T,  x's groups along K
 *   mxq_matmul_fp8_block128_dgrad  dx[M, K] = dy[M, N] w[N, K],   dy's groups along N
 *   mxq_matmul_fp8_group128_wgrad  dw[N, K] = dy[M, N]^T x[M, K], both in groups of
 *                                  128 rows (mxq_quantize_fp8_group128_col)
 *   w          [N, K] payload, row stride ld_w >= K; tile_code [ceil(N/128), tile_ld]
 *   offsets    NULL: one weight.  Else n_experts of them and the rows sorted by
 *              expert (a device array of n_experts + 1 int32, as for the
 *              quantizer): expert e's rows meet the weight at w + e * w_stride
 *              with codes at tile_code + e * tile_stride; rows of no expert give
 *              rows of zeros; dw is [n_experts, N, K], dw_stride elements apart,
 *              zeros for an expert without rows.
 *   out_dt     MXQ_BF16 or MXQ_FP32
 *   fast_accum 0: products are summed in fp32.  Otherwise the matrix cores' FP8
 *              instructions sum them, at about twice the rate: they line up each
 *              8 products to the largest of them and drop what falls below 2^-13
 *              of it, so a result may be off by 2^-10 of the sum of its products'
 *              magnitudes, payloads below 2^-6 counted as 2^-6 (a bf16 result is
 *              rounded by 2^-9 of itself).  Sums of blocks of 128 are added in
 *              fp32 either way.  Weight gradients are always summed in fp32.
 * A code 255 or payload 0x7F (or 0xFF) makes what it meets NaN.  A reduction of
 * length 0 gives zeros.  Outputs must not overlap any input (MXQ_ERR_ALIAS).
 */
int mxq_matmul_fp8_block128(const uint8_t* x, int64_t ld_x, const uint8_t* x_scale, int64_t x_scale_ld,
                            const uint8_t* w, int64_t ld_w, int64_t w_stride, const uint8_t* tile_code,
                            int64_t tile_ld, int64_t tile_stride, int64_t M, int64_t N, int64_t K,
                            const int32_t* offsets, int64_t n_experts, void* y, int64_t ld_y, mxq_dtype out_dt,
                            int fast_accum, hipStream_t stream);
int mxq_matmul_fp8_block128_dgrad(const uint8_t* dy, int64_t ld_dy, const uint8_t* dy_scale, int64_t dy_scale_ld,
                                  const uint8_t* w, int64_t ld_w, int64_t w_stride, const uint8_t* tile_code,
                                  int64_t tile_ld, int64_t tile_stride, int64_t M, int64_t N, int64_t K,
                                  const int32_t* offsets, int64_t n_experts, void* dx, int64_t ld_dx,
                                  mxq_dtype out_dt, int fast_accum, hipStream_t stream);
int mxq_matmul_fp8_group128_wgrad(const uint8_t* dy, int64_t ld_dy, const uint8_t* dy_scale, int64_t dy_scale_ld,
                                  const uint8_t* x, int64_t ld_x, const uint8_t* x_scale, int64_t x_scale_ld,
                                  int64_t M, int64_t N, int64_t K, const int32_t* offsets, int64_t n_experts,
                                  void* dw, int64_t ld_dw, int64_t dw_stride, mxq_dtype out_dt, hipStream_t stream);

/*
 * Token slots sorted by expert.  A slot is one (token, choice) pair, numbered
 * token * top_k + choice; the sort is stable.
 *   ids        [n_tokens, top_k] int32 expert of each slot, row stride ld_ids >=
 *              top_k.  An id outside [0, n_experts) drops the slot.
 *   offsets    [n_experts + 1] int32: expert e owns sorted rows [offsets[e],
 *              offsets[e+1]); offsets[n_experts] counts the slots that are kept
 *   slots      [n_tokens * top_k] int32: the slot of each sorted row; dropped
 *              slots come last, each as its complement ~slot (negative)
 *   position   [n_tokens * top_k] int32: the sorted row of each slot; that of a
 *              dropped slot as its complement
 *   workspace  at least mxq_sort_experts_workspace(n_tokens, top_k, n_experts)
 *              bytes, 4-byte aligned (NULL where that is 0), free again when the
 *              work is done
 * 1 <= n_experts <= 512.  With no tokens the offsets are still written.
 */
int64_t mxq_sort_experts_workspace(int64_t n_tokens, int64_t top_k, int64_t n_experts);
int mxq_sort_experts(const int32_t* ids, int64_t ld_ids, int64_t n_tokens, int64_t top_k, int64_t n_experts,
                     int32_t* offsets, int32_t* slots, int32_t* position, void* workspace, int64_t workspace_bytes,
                     hipStream_t stream);

/*
 * Rows into sorted order: out[r] = x[slots[r] / top_k], zeros for a dropped slot
 * or one whose row is not below x_rows.  Its gradient is mxq_combine_rows without
 * weights.
 *   x [x_rows, H], out [rows, H], both of type dt
 */
int mxq_dispatch_rows(const void* x, int64_t ld_x, int64_t x_rows, const int32_t* slots, int64_t rows, int64_t top_k,
                      int64_t H, mxq_dtype dt, void* out, int64_t ld_out, hipStream_t stream);

/*
 * Rows back to their tokens: y[t] = sum over j of weights[t, j] *
 * rows[position[t, j]], summed in fp32 in the order of j and rounded once; slots
 * that are dropped (negative) or not below n_rows add nothing and are not read.
 *   weights  [n_tokens, top_k] fp32, contiguous; NULL: all 1
 *   position [n_tokens, top_k] int32, contiguous
 * mxq_combine_rows_backward: drows[position[t, j]] = weights[t, j] * dy[t], zeros
 * for the row of a dropped slot; dweights[t, j] = sum over h of dy[t, h] *
 * rows[position[t, j], h] in fp32 (NULL: not wanted), 0 for a dropped slot.  Two
 * slots must not share a position; rows that no slot names are left untouched.
 */
int mxq_combine_rows(const void* rows, int64_t ld_rows, int64_t n_rows, const int32_t* position, const float* weights,
                     int64_t n_tokens, int64_t top_k, int64_t H, mxq_dtype dt, void* y, int64_t ld_y,
                     hipStream_t stream);
int mxq_combine_rows_backward(const void* dy, int64_t ld_dy, const void* rows, int64_t ld_rows, int64_t n_rows,
                              const int32_t* position, const float* weights, int64_t n_tokens, int64_t top_k,
                              int64_t H, mxq_dtype dt, void* drows, int64_t ld_drows, float* dweights,
                              hipStream_t stream);

/*
 * Root-mean-square norm of rows, with the residual's addition before it.
 *   s = x + residual in fp32, rounded once to the residual's type (s = x without a
 *   residual); y = s / sqrt(mean(s^2) + eps) * weight in fp32, rounded once to each output.
 * The norm is that of s as it is stored, so that the backward pass, or the norm run
 * again from a stored s, sees the same values.  A row's sum is in fp32 and its squares do not
 * overflow.  A row that holds an Inf or NaN follows the formula: with a NaN all of it is NaN, with an
 * Inf its finite elements are 0 and the others NaN.
 *   x         [rows, K] of type dt, row stride ld_x >= K
 *   residual  [rows, K] of type residual_dt; NULL: none, and residual_dt is not looked at
 *   weight    [K] of type weight_dt, contiguous; NULL: all 1
 *   eps       finite and at least 2^-126 (MXQ_ERR_SHAPE otherwise)
 *   sum       [rows, K] of type residual_dt: s.  NULL: not wanted; MXQ_ERR_NULL where it is
 *             wanted without a residual.  sum == residual with the same row stride (in place) is
 *             allowed.
 *   y         [rows, K] of type dt; NULL: not wanted (the FP8 forms only)
 *   data, scale   y in FP8, groups of 128 along the row, as mxq_quantize_fp8_group128 lays
 *             them out; quantized from y in fp32
 * mxq_rms_norm_fp8_group128_row_col also writes groups of 128 rows of a column (as
 * mxq_quantize_fp8_group128_col without experts).
 *   workspace at least mxq_rms_norm_fp8_group128_row_col_workspace(rows) bytes, 8-byte
 *             aligned, free again when the work is done
 */
int mxq_rms_norm(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual, mxq_dtype residual_dt,
                 const void* weight, mxq_dtype weight_dt, float eps, int64_t rows, int64_t K, mxq_dtype dt, void* sum,
                 int64_t ld_sum, void* y, int64_t ld_y, hipStream_t stream);
int mxq_rms_norm_fp8_group128(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual,
                              mxq_dtype residual_dt, const void* weight, mxq_dtype weight_dt, float eps, int64_t rows,
                              int64_t K, mxq_dtype dt, void* sum, int64_t ld_sum, void* y, int64_t ld_y, uint8_t* data,
                              int64_t ld_data, uint8_t* scale, int64_t scale_ld, hipStream_t stream);
int64_t mxq_rms_norm_fp8_group128_row_col_workspace(int64_t rows);
int mxq_rms_norm_fp8_group128_row_col(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual,
                                      mxq_dtype residual_dt, const void* weight, mxq_dtype weight_dt, float eps,
                                      int64_t rows, int64_t K, mxq_dtype dt, void* sum, int64_t ld_sum, void* y,
                                      int64_t ld_y, uint8_t* row_data, int64_t ld_row, uint8_t* row_scale,
                                      int64_t row_scale_ld, uint8_t* col_data, int64_t ld_col, uint8_t* col_scale,
                                      int64_t col_scale_ld, void* workspace, int64_t workspace_bytes,
                                      hipStream_t stream);

/*
 * Gradients of the norm: with r = 1 / sqrt(mean(s^2) + eps), u = s r and g = dy w,
 *   dx = r (g - u mean(g u)) + dresidual, the gradient of x and of the residual alike
 *   dweight = sum over the rows of dy u, in fp32 and in an order that the sizes fix
 *   dy         [rows, K] of type dt
 *   x          [rows, K] of type x_dt: s, what was normalized (sum, or x without a residual)
 *   dresidual  [rows, K] of type x_dt, the gradient that reaches s past the norm; NULL: none
 *   dx         [rows, K] of type x_dt
 *   dweight    [K] fp32; NULL: not wanted.  With no rows it is set to 0.
 *   workspace  at least mxq_rms_norm_backward_workspace(rows, K) bytes, 16-byte aligned
 */
int64_t mxq_rms_norm_backward_workspace(int64_t rows, int64_t K);
int mxq_rms_norm_backward(const void* dy, int64_t ld_dy, mxq_dtype dt, const void* x, int64_t ld_x, mxq_dtype x_dt,
                          const void* weight, mxq_dtype weight_dt, float eps, const void* dresidual,
                          int64_t ld_dresidual, int64_t rows, int64_t K, void* dx, int64_t ld_dx, float* dweight,
                          void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* The activations: silu(g) = g / (1 + exp(-g)); gelu in its tanh form, g (1 + tanh(sqrt(2/pi)
 * (g + 0.044715 g^3))) / 2; the squared relu, max(g, 0)^2. */
typedef enum { MXQ_SILU = 0, MXQ_GELU_TANH = 1, MXQ_RELU2 = 2 } mxq_activation;

/*
 * The activation between the two products of a feed-forward layer, in FP8:
 * a = act(gate) * up, or act(gate) where up is NULL; computed in fp32 and rounded once, to E4M3 in
 * groups of 128 (codes and payloads as mxq_quantize_fp8_group128 gives them for a).
 *   gate, up  [rows, F] bf16 or fp32, row strides ld_gate, ld_up >= F: the halves of an up
 *             projection's result lie in one matrix of row stride 2 F
 *   data      [rows, F], scale [rows, scale_ld >= ceil(F/128)]
 * mxq_activate_fp8_group128_row_col: groups along the columns as well, begun anew with
 * each expert's rows where offsets is given (see mxq_quantize_fp8_group128_col for the layout).
 * mxq_activate_fp8_group128_backward: the gradients of both halves for da [rows, F],
 *   dgate = da up act'(gate), dup = da act(gate), as one matrix [rows, 2 F] (dgate in its first F
 *   columns; [rows, F] where up is NULL) in groups along rows and columns: the operands of the up
 *   projection's own gradients.
 * F is at most 2^29.
 */
int mxq_activate_fp8_group128(const void* gate, int64_t ld_gate, const void* up, int64_t ld_up, int64_t rows, int64_t F,
                              mxq_dtype dt, mxq_activation act, uint8_t* data, int64_t ld_data, uint8_t* scale,
                              int64_t scale_ld, hipStream_t stream);
int mxq_activate_fp8_group128_row_col(const void* gate, int64_t ld_gate, const void* up, int64_t ld_up, int64_t rows,
                                      int64_t F, mxq_dtype dt, mxq_activation act, const int32_t* offsets,
                                      int64_t n_experts, uint8_t* row_data, int64_t ld_row, uint8_t* row_scale,
                                      int64_t row_scale_ld, uint8_t* col_data, int64_t ld_col, uint8_t* col_scale,
                                      int64_t col_scale_ld, hipStream_t stream);
int mxq_activate_fp8_group128_backward(const void* da, int64_t ld_da, const void* gate, int64_t ld_gate, const void* up,
                                       int64_t ld_up, int64_t rows, int64_t F, mxq_dtype dt, mxq_activation act,
                                       const int32_t* offsets, int64_t n_experts, uint8_t* row_data, int64_t ld_row,
                                       uint8_t* row_scale, int64_t row_scale_ld, uint8_t* col_data, int64_t ld_col,
                                       uint8_t* col_scale, int64_t col_scale_ld, hipStream_t stream);

/* How a router's logits become scores: softmax over the experts, or 1 / (1 + exp(-logit)) of each. */
typedef enum { MXQ_SOFTMAX = 0, MXQ_SIGMOID = 1 } mxq_score;

/*
 * Each token's experts and their weights.  An expert's key is its logit, or with a bias
 * score + bias, compared as 64 bits give it.  The top_k experts with the largest keys are chosen, in
 * falling order; of equal keys the lower index comes first.
 *   logits      [n_tokens, n_experts] bf16 or fp32, row stride ld_logits >= n_experts.  An expert
 *               whose logit is -inf has score 0 and is closed to that token: never chosen.
 *   bias        [n_experts] fp32, added to the scores for the choice alone (-inf closes an expert);
 *               NULL: none
 *   mask        [n_tokens] bytes; a token whose byte is 0 gets no experts.  NULL: all take part
 *   n_groups, top_groups, group_top   the experts form n_groups groups of neighbours, as many in
 *               each; only those of the top_groups best groups take part.  A group ranks by its largest
 *               key (group_top 1) or by the sum of the scores, biased if there is a bias, of its two
 *               experts with the largest keys (2; of one where no other is open); of equal groups
 *               the lower index goes first.  n_groups 1: no such choice
 *   ids         [n_tokens, top_k] int32, contiguous; -1 where no expert is left (such a slot is
 *               dropped by mxq_sort_experts)
 *   weights     [n_tokens, top_k] fp32: scale * score, or with renormalize scale * score / the sum
 *               of the chosen scores; 0 for an id of -1
 * Weights and gradients are computed in fp32 at least.
 * A NaN key counts as the smallest of those that are open; weights of such a token may be NaN.
 * 1 <= top_k <= top_groups * (n_experts / n_groups), n_experts <= 512, scale finite.
 * mxq_route_experts_backward: the gradient of the logits for dweights [n_tokens, top_k], the
 * choice held fixed (the bias has no gradient); slots whose id is not an expert's count nothing, and a
 * token without any other has gradient 0, whatever its logits are.
 *   dlogits     [n_tokens, n_experts] of the logits' type, row stride ld_dlogits >= n_experts
 */
int mxq_route_experts(const void* logits, int64_t ld_logits, int64_t n_tokens, int64_t n_experts, mxq_dtype dt,
                      const float* bias, const uint8_t* mask, mxq_score score, int renormalize, float scale,
                      int64_t n_groups, int64_t top_groups, int64_t group_top, int64_t top_k, int32_t* ids,
                      float* weights, hipStream_t stream);
int mxq_route_experts_backward(const float* dweights, const void* logits, int64_t ld_logits, const int32_t* ids,
                               int64_t n_tokens, int64_t n_experts, int64_t top_k, mxq_dtype dt, mxq_score score,
                               int renormalize, float scale, void* dlogits, int64_t ld_dlogits, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_H */
