/*
 * librazer.h -- C ABI of librazer, the RaZeR-NVFP4 W4A16 layer for AMD MI355X
 * (CDNA4, gfx950).
 *
 * Sources cited below (page title, then section):
 *   [notes]   "RaZeR: Pushing the Limits of NVFP4 Quantization with Redundant
 *             Zero Remapping" (papernotes.org notes)
 *   [summary] "Technical Summary: RaZeR - Pushing the Limits of NVFP4
 *             Quantization with Redundant Zero Remapping" (gist.science)
 *
 * THE FORMAT ([notes] Background, Overall framework, Key design 1-3;
 * [summary] §2.1-2.2).  A tensor X[rows, cols] (row-major, cols % 16 == 0) is
 * cut into 16-element blocks along each row.  It carries one FP32 tensor
 * scale st and, per block, one scale byte and 16 four-bit element codes:
 *
 *   st       = amax(|X|) / (6 * S_MAX)                       (fp32)
 *   sb_code  = round_nearest_even(S_MAX * amax_block / amax(|X|))
 *              onto E3M3 (weights: 3 exp bits, bias 3, max 30) or
 *              E4M3 (activations: OCP E4M3FN, max 448)
 *   y_j      = x_j * (1 / (sb * st))                         (fp32)
 *   code_j   = FP4-E2M1 of y_j: sign bit 3, magnitude index 0..7 of
 *              {0, 0.5, 1, 1.5, 2, 3, 4, 6}, nearest-even, saturating at 6;
 *              zero is always written as +0 (0b0000)
 *   The redundant -0 code 0b1000 is remapped to a per-block special value
 *   SV = sign * (6 + off/2).  Each block keeps the candidate with the lowest
 *   block squared error ([notes] Key design 2, block MSE equation), ties to
 *   the lowest candidate index; an element takes SV only if SV is strictly
 *   nearer than its FP4 rounding.
 *     weights:     4 candidates +M0, -M0, +M1, -M1 (two +/- pairs),
 *                  scale byte = sign << 7 | pair << 6 | E3M3 code (6 bits)
 *     activations: 2 candidates +M0, -M0,
 *                  scale byte = sign << 7 | E4M3 code (7 bits)
 *   with M_i = 6 + sv_off_half[i] / 2 ([notes] Key design 3: 4-bit offset
 *   registers holding [-3.5, 3.5] in steps of 0.5).
 *
 * MEMORY LAYOUT of a packed tensor (all device memory, caller-owned):
 *   codes[r * cols/2 + i]   = code(r, 2i) | code(r, 2i+1) << 4   (u8)
 *   scales[r * cols/16 + b] = scale byte of block b of row r     (u8)
 *   tensor_scale[0]         = st                                 (fp32)
 * A weight W[N, K] is stored like a PyTorch Linear weight (row n holds the K
 * inputs of output n); products compute y[M, N] = x[M, K] * W^T.
 *
 * CONVENTIONS for every call:
 *   - Pointers marked "device" point to GPU memory on the current HIP device.
 *     The caller allocates and frees every buffer, including workspaces; the
 *     library never allocates, frees or synchronises, and keeps no mutable
 *     global state, except the 4 KiB per-device scratch array of
 *     razer_quantize_act_noalloc.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).  All
 *     work is enqueued on it, asynchronously, in stream order.
 *   - Host-side argument checks are synchronous: on RAZER_E_INVALID or
 *     RAZER_E_UNSUPPORTED nothing is enqueued and nothing is written.
 *     RAZER_E_HIP reports a failed kernel launch.
 *   - Data errors are reported through data, not status: a non-finite input
 *     element makes the encoder write tensor_scale = NaN and all codes and
 *     scale bytes 0; a product whose weight has a NaN tensor scale outputs NaN.
 *   - Device pointers must be 16-byte aligned (x, w, y, codes) and 4-byte
 *     aligned (scales, tensor_scale, workspace).
 *   - Calls on different streams may run concurrently if they write disjoint
 *     buffers (including workspaces).
 */
#ifndef LIBRAZER_H
#define LIBRAZER_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The two enums below carry range markers so that every 32-bit value a C
 * caller may pass is a valid value of the type (the library rejects the ones
 * that are not a listed constant). */
typedef enum razer_status {
  RAZER_OK = 0,
  RAZER_E_INVALID = 1,     /* bad argument: null pointer, shape, alignment, offsets, workspace */
  RAZER_E_UNSUPPORTED = 2, /* valid but not implemented (dtype/kind/shape combination) */
  RAZER_E_HIP = 3,         /* the HIP runtime refused a launch */
  RAZER_STATUS_RANGE_MIN_ = -0x7FFFFFFF - 1,
  RAZER_STATUS_RANGE_MAX_ = 0x7FFFFFFF
} razer_status;

typedef enum razer_dtype {
  RAZER_F32 = 0,
  RAZER_F16 = 1,
  RAZER_BF16 = 2,
  RAZER_DTYPE_RANGE_MIN_ = -0x7FFFFFFF - 1,
  RAZER_DTYPE_RANGE_MAX_ = 0x7FFFFFFF
} razer_dtype;

/* Which scale format and candidate set a packed tensor uses ([notes] Key
 * design 1: weights free 2 scale bits, activations 1). */
typedef enum razer_kind { RAZER_WEIGHT = 0, RAZER_ACT = 1 } razer_kind;

/* flags of razer_packed */
enum {
  /* Encode as plain NVFP4 (no special value; sel = 0 everywhere) with the same
   * scale format: the comparator of the pages' main table, used to measure
   * what the special-value search costs ([notes] Key design 2 states the
   * activation search adds under 2% to quantizer time). */
  RAZER_FLAG_NO_REMAP = 1u,
  /* Encode with the Four Over Six baseline (page "Four Over Six: More Accurate
   * NVFP4 Quantization with Adaptive Block Scaling", technical framework and
   * key innovation): plain FP4 (no special value), and each block takes the
   * block scale whose code is nearest to S_MAX * amax_block / amax_tensor
   * (max -> 6) or to 1.5 times that (max -> 4, saturating at the format
   * maximum), whichever gives the smaller squared error against the input in
   * real units (summed in fp64 in element order; a tie keeps max -> 6).  The
   * tensor scale and the packed layout are unchanged, so every decoding call
   * reads such a tensor as plain NVFP4.  Takes precedence over NO_REMAP.
   * The quantize calls reject any other flag bit than these three with
   * RAZER_E_INVALID. */
  RAZER_FLAG_FOUR_OVER_SIX = 2u,
  /* Read by the product calls only (the encoders reject it): launch the
   * product with the untrimmed plan -- the K range split over the most waves
   * or workgroups the kernel allows and the fewest rows per wave, so every CU
   * gets work however small the matrix -- instead of the launch plan sized
   * per shape.  For measuring what the launch sizing gains: the counterpart
   * of the pages' adaptive trimming of SM launches for small matrices ([notes]
   * Key design 3).  Outputs agree within the product tolerance (the
   * summation order changes).  razer_gemm then needs
   * razer_workspace_bytes(RAZER_OP_GEMM_UNTRIMMED, ...). */
  RAZER_FLAG_UNTRIMMED_PLAN = 4u,
  /* Encode with rescaled large special values (a reading of [notes] Training
   * strategy, whose best weight pairs include +/-7, +/-8 and +/-9, values a
   * block scaled so that its maximum maps to 6 almost never reaches): every
   * candidate special value v is tried on its own -- one with |v| > 6 at the
   * block scale whose code is nearest to S_MAX * amax_block / amax_tensor *
   * 6 / |v| (fp32: (sb_real * 6) / |v|), so the block maximum maps to |v|, the
   * others at the usual scale -- and the block keeps the encoding with the
   * smallest squared error against the input in real units (fp64, element
   * order; ties to the lowest candidate index).  Decoding is unchanged (the
   * scale byte holds the chosen scale and the metadata the chosen value).
   * 16-element blocks with byte scales only (other layouts:
   * RAZER_E_UNSUPPORTED); NO_REMAP and FOUR_OVER_SIX take precedence. */
  RAZER_FLAG_RESCALE_LARGE_SV = 8u
};

/* Block-scale storage of a packed tensor (razer_packed.scale_fmt). */
enum {
  /* One byte per block: E3M3 (weights) / E4M3 (activations) scale code with
   * the metadata in bits 7-6 ([notes] Key design 1).  The default. */
  RAZER_SCALE_BYTE = 0,
  /* Weights only: one 16-bit FP16 scale per block whose sign bit and top
   * exponent bit hold the metadata (bit 15 = sign of the special value, bit
   * 14 = pair) and whose other 14 bits are the scale, an FP16 number with
   * exponent field 0..15, at most 2 - 2^-10 ([notes] Key design 3: the
   * layout of the pages' Blackwell kernels, there with 128-element blocks).
   * The tensor scale is amax / (6 * (2 - 2^-10)). */
  RAZER_SCALE_F16 = 1
};

typedef struct razer_packed {
  int32_t kind;          /* razer_kind */
  uint32_t flags;        /* RAZER_FLAG_* (encoder flags; RAZER_FLAG_UNTRIMMED_PLAN for products) */
  int64_t rows;          /* >= 0 */
  int64_t cols;          /* >= 0, multiple of the block size */
  int8_t sv_off_half[2]; /* special-value offsets in units of 0.5, each in [-7, 7];
                            weights use both, activations use [0] only */
  uint8_t block_log2;    /* elements per block = 2^block_log2, 4..7 (16..128, [notes]
                            Key findings: block sizes 32, 64, 128); 0 reads as 4 */
  uint8_t scale_fmt;     /* RAZER_SCALE_BYTE or RAZER_SCALE_F16 */
  int8_t reserved[4];
  uint8_t* codes;        /* device, rows*cols/2 bytes */
  uint8_t* scales;       /* device, rows*cols/block entries of 1 (byte) or 2 (F16) bytes */
  float* tensor_scale;   /* device, 1 float */
} razer_packed;
/* The encoders and razer_dequant take every layout.  The product calls take
 * 16-element blocks with byte scales; razer_gemv, razer_gemv_group (all
 * members in one layout) and razer_gemm (any m) also take the pages' kernel
 * layout, 128-element blocks (block_log2 7) with RAZER_SCALE_F16.  Other
 * layouts, and any layout but the default for razer_gemm_w4a4, return
 * RAZER_E_UNSUPPORTED. */

/* Operation ids for razer_workspace_bytes. */
enum {
  RAZER_OP_QUANTIZE_WEIGHT = 0,
  RAZER_OP_QUANTIZE_ACT = 1,
  RAZER_OP_GEMV = 2,
  RAZER_OP_GEMM = 3,
  RAZER_OP_OFFSET_SEARCH = 4, /* n = rows, k = cols of the weight */
  RAZER_OP_GEMM_W4A4 = 5,     /* m = rows of x, n = rows of w, k = cols */
  RAZER_OP_GEMM_UNTRIMMED = 6 /* razer_gemm of a weight with RAZER_FLAG_UNTRIMMED_PLAN */
};

/* Offline weight encoder: 4-candidate block-MSE search ([notes] Key design 2:
 * weights are searched offline over two +/- pairs; [summary] §2.2).
 * w: device [out->rows, out->cols] in w_dt (F32, F16 or BF16).  out: describes
 * the destination; kind must be RAZER_WEIGHT; codes/scales/tensor_scale are
 * written.  ws: device workspace of at least
 * razer_workspace_bytes(RAZER_OP_QUANTIZE_WEIGHT, rows, 0, cols) bytes. */
razer_status razer_quantize_weight(const void* w, razer_dtype w_dt, const razer_packed* out,
                                   void* ws, size_t ws_bytes, void* stream);

/* Online activation encoder: 2 candidates +/-M0 with the E4M3 block scale
 * ([notes] Key design 1 and 2; [summary] §2.2).  x: device [rows, cols] in
 * F16 or BF16 (F32 also accepted).  out->kind must be RAZER_ACT. */
razer_status razer_quantize_act(const void* x, razer_dtype x_dt, const razer_packed* out,
                                void* ws, size_t ws_bytes, void* stream);

/* razer_quantize_act without a workspace, for callers that cannot allocate
 * device memory: code under HIP graph capture, tight serving loops, harnesses
 * that forbid allocation.  Same arguments (minus ws / ws_bytes), checks and
 * output bytes as razer_quantize_act.  The amax partials live in a 4 KiB
 * static device array that the library holds on each device it runs on until
 * the process ends; the first call on a device resolves that array's address
 * (hipGetSymbolAddress), so make it outside stream capture.  Every call on one
 * device shares the array: calls that overlap on one device (different
 * streams, concurrent graph launches) race and must be ordered by the caller.
 * The array is large enough for every input size (the partials never exceed
 * it); RAZER_E_UNSUPPORTED would report a build where they did.  Allocates
 * nothing, frees nothing, synchronises nothing. */
razer_status razer_quantize_act_noalloc(const void* x, razer_dtype x_dt, const razer_packed* out,
                                        void* stream);

/* Decode a packed tensor ([notes] Key design 3 decoder): out[r, c] =
 * value(code) * sb * st, with value(0b1000) = (bit7 ? -1 : 1) * (6 + off/2).
 * F32 output is fl32(fl32(value * sb) * st); F16/BF16 output is that fp32
 * value rounded to nearest even.  out: device [rows, cols] in out_dt. */
razer_status razer_dequant(const razer_packed* t, void* out, razer_dtype out_dt, void* stream);

/* Batch-1 W4A16 product y[1, N] = x[1, K] * W^T with W decoded in registers
 * ([notes] Key design 3: weight-only GEMV kernels; [summary] §2.3).
 * x: device [K] in F16 or BF16.  w: packed tensor [N, K] of either kind
 * (weights, or an activation encoding used as the right operand).  y: device [N] in
 * F32, F16 or BF16.  Accumulation is fp32.  ws: at least
 * razer_workspace_bytes(RAZER_OP_GEMV, 1, N, K) bytes (may be 0 -> ws NULL). */
razer_status razer_gemv(const void* x, razer_dtype x_dt, const razer_packed* w, void* y,
                        razer_dtype y_dt, void* ws, size_t ws_bytes, void* stream);

/* Largest count accepted by razer_gemv_group. */
#define RAZER_GEMV_GROUP_MAX 4

/* Several batch-1 products that share one input vector, y_g[1, N_g] = x[1, K] *
 * W_g^T for g < count, in one launch where the GEMV kernel serves them (the
 * product of razer_gemv for each weight, [notes] Key design 3; sharing the
 * launch is the counterpart of the pages' launch sizing for small matrices:
 * two weights of one input, such as an MLP's gate and up projections, cost
 * one launch and one ramp instead of two).  x: device [K] in F16 or BF16.
 * w: host array of count packed-tensor descriptors (either kind, each with its
 * own tensor scale and offsets) with equal cols K.  y: host array of count
 * device outputs [N_g] in y_dt (16-byte aligned; may be NULL where N_g == 0).
 * 1 <= count <= RAZER_GEMV_GROUP_MAX.  Each y_g is bitwise what razer_gemv
 * writes for W_g.  No workspace.  Errors: RAZER_E_INVALID for a bad count,
 * unequal K or any argument razer_gemv would reject; RAZER_E_UNSUPPORTED as
 * for razer_gemv. */
razer_status razer_gemv_group(const void* x, razer_dtype x_dt, const razer_packed* const* w,
                              void* const* y, int count, razer_dtype y_dt, void* stream);

/* Batched W4A16 product y[M, N] = x[M, K] * W^T ([notes] Key design 3;
 * [summary] §2.3: weight-only GEMM kernels for small and large batches).
 * x: device [m, K] row-major in F16 or BF16.  w: packed tensor [N, K] of either
 * kind, default layout or 128-element blocks with FP16 scales.  y: device
 * [m, N] in F32, F16 or BF16.  m >= 1; m == 1 runs the GEMV path.  ws: at least
 * razer_workspace_bytes(RAZER_OP_GEMM, m, N, K) bytes (enough for either
 * layout).  For m >= 256 (the 256x256-tile kernel) the workspace is optional:
 * NULL, smaller or not 16-byte aligned, the product runs without it; with it,
 * when the tile count leaves a last round of tiles on at most half of the
 * compute units, those tiles are computed as two K halves (fp32 partial tiles
 * in ws, then added in one more launch). */
razer_status razer_gemm(const void* x, razer_dtype x_dt, int64_t m, const razer_packed* w, void* y,
                        razer_dtype y_dt, void* ws, size_t ws_bytes, void* stream);

/* W4A4 product y[M, N] = dequant(x)[M, K] * dequant(w)^T of two packed
 * tensors ([notes] Overall framework, Key designs 1-2: activations encoded
 * online with 2 candidates, weights offline with 4).  On matrix units without
 * an FP4 path it runs in two passes: x's codes are decoded to value * sb in
 * fp16 (exact), the W4A16 product runs on them in fp32, and the result is
 * multiplied by x's tensor scale and rounded once to y_dt.  x: packed [M, K]
 * (normally RAZER_ACT, either kind accepted); w: packed [N, K] of either kind;
 * y: device [M, N] in F32, F16 or BF16.  K == 0 is RAZER_E_UNSUPPORTED.
 * ws: at least razer_workspace_bytes(RAZER_OP_GEMM_W4A4, M, N, K) bytes,
 * 256-byte aligned.  The accuracy bound is the W4A16 product's plus one fp32
 * rounding. */
razer_status razer_gemm_w4a4(const razer_packed* x, const razer_packed* w, void* y, razer_dtype y_dt,
                             void* ws, size_t ws_bytes, void* stream);

/* Second-pair offset search for the offline weight encoder ([notes] Loss
 * function / training strategy: the extra weight pair is picked offline by a
 * grid search).  For each offset o = -7..7 of the second pair, the weight is
 * encoded exactly as razer_quantize_weight would with offsets (off0_half, o),
 * and sse[o + 7] receives sum((w - value * sb * st)^2) over the tensor,
 * accumulated in fp64 (value * sb * st is exact in fp64).  The caller picks
 * the offset (e.g. the lowest sse, ties to the lowest offset) and passes it to
 * razer_quantize_weight.  w: device [rows, cols] in w_dt (F32, F16, BF16),
 * cols % 16 == 0.  sse: device, 15 doubles, 8-byte aligned.  A non-finite
 * weight gives NaN in all 15; an all-zero or empty weight gives 0.  ws: at
 * least razer_workspace_bytes(RAZER_OP_OFFSET_SEARCH, 0, rows, cols) bytes,
 * 8-byte aligned.  Summation order is fixed, so results repeat bit for bit. */
razer_status razer_weight_offset_sse(const void* w, razer_dtype w_dt, int64_t rows, int64_t cols,
                                     int off0_half, double* sse, void* ws, size_t ws_bytes,
                                     void* stream);

/* Workspace bytes an operation needs for the given sizes (m rows of x, n
 * weight rows / output features, k reduction length).  0 means none.  For
 * RAZER_OP_GEMM with m >= 256 the figure is what the prefill kernel's tail
 * split uses (it depends on the current device's compute-unit count); that
 * workspace is optional there. */
size_t razer_workspace_bytes(int op, int64_t m, int64_t n, int64_t k);

/* ---- microscaled 4-bit tensors (MXFP4) ----------------------------------------
 *
 * THE FORMAT (Open Compute Project, "Microscaling Formats (MX) Specification
 * v1.0", MXFP4).  X[rows, cols], row-major, cols % 32 == 0, is cut into
 * 32-element blocks along each row, each with one E8M0 scale byte:
 *
 *   byte   = floor(log2(amax_block)) - 2 + 127, at least 0 (a zero block: 0);
 *            its value is 2^(byte - 127)
 *   code_j = FP4-E2M1 of x_j / 2^(byte - 127): sign bit 3 (a zero keeps its
 *            sign), magnitude index 0..7 of {0, 0.5, 1, 1.5, 2, 3, 4, 6},
 *            nearest-even, saturating at 6
 *
 * A block with an infinity or NaN gets byte 255 (NaN) and codes 0: all its
 * values, and every product they enter, are NaN.  Unlike the RaZeR formats there
 * is no tensor scale and no special value: the matrix units read codes and
 * scales as they are stored, and both operands of a product are in 4 bits. */
typedef struct razer_mx {
  int64_t rows;    /* >= 0 */
  int64_t cols;    /* >= 0, multiple of 32 */
  uint8_t* codes;  /* device, rows*cols/2 bytes, 16-byte aligned, even column in the low half */
  uint8_t* scales; /* device, rows*cols/32 bytes, row-major */
} razer_mx;

/* Encode x[out->rows, out->cols] (F32, F16 or BF16; x_stride elements from row
 * to row, a multiple of 16 bytes).  No workspace.  At most 2^34 elements
 * (RAZER_E_UNSUPPORTED above). */
razer_status razer_mx_quantize(const void* x, razer_dtype x_dt, int64_t x_stride, const razer_mx* out,
                               void* stream);

/* Encode silu(g) * u = g * u / (1 + exp(-g)), the input of an MLP's down
 * projection: gu is [out->rows, 2 * out->cols], g its first out->cols columns
 * and u the others (the output of one product with the gate and up weights
 * stacked).  The fp32 product is packed directly. */
razer_status razer_mx_quantize_gated(const void* gu, razer_dtype gu_dt, int64_t gu_stride, const razer_mx* out,
                                     void* stream);

/* Decode to out[rows, cols]: value(code) * 2^(byte - 127), exact in fp32 (infinity
 * above its range, which no encoded block reaches); F16 and BF16 round it to
 * nearest even. */
razer_status razer_mx_dequant(const razer_mx* t, void* out, razer_dtype out_dt, void* stream);

/* y[M, N] = x[M, K] * w[N, K]^T of two MXFP4 tensors, M from one token up; fp32
 * accumulation in an order that is the same from call to call, one rounding to
 * y_dt (F16 above its range: infinity).  K == 0, K > 2^23 and M or N > 2^30 are
 * RAZER_E_UNSUPPORTED.  y: 16-byte aligned, and not in memory that x or w hold.
 * ws: at least razer_mx_workspace_bytes(M, N, K, 0) bytes, 16-byte aligned (may
 * be 0 -> NULL). */
razer_status razer_mx_gemm(const razer_mx* x, const razer_mx* w, void* y, razer_dtype y_dt, void* ws,
                           size_t ws_bytes, void* stream);

/* Largest expert count of razer_mx_gemm_grouped. */
#define RAZER_MX_MAX_EXPERTS 4096

/* The products of a mixture of experts: w stacks `experts` weights [N, K], N =
 * w->rows / experts, and y[M, N] takes rows offsets[e] .. offsets[e + 1] - 1
 * through weight e:
 *
 *   y[r] = x[x_rows[r]] * w_e^T        (x[r] where x_rows is NULL: M = x->rows)
 *
 * offsets: device, experts + 1 ascending row numbers; x_rows: device, M row
 * numbers of x.  Neither is read on the host, so a router's output can be used
 * without waiting for it and the call can be captured.  Runs of no rows are
 * allowed; rows of y outside every run are left as they were; a row number
 * outside x (such as -1, padding) makes its row of y zero.  Offsets outside
 * [0, M] are clamped.  Limits as of razer_mx_gemm; with x_rows the codes of x
 * are less than 4 GiB (RAZER_E_UNSUPPORTED).  ws: razer_mx_workspace_bytes(M, N,
 * K, experts) bytes, 16-byte aligned. */
razer_status razer_mx_gemm_grouped(const razer_mx* x, const razer_mx* w, const int32_t* offsets,
                                   int64_t experts, const int32_t* x_rows, int64_t m, void* y,
                                   razer_dtype y_dt, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes of a product (experts = 0) or of a grouped one (n: columns of
 * one expert).  Depends on the current device's compute-unit count. */
size_t razer_mx_workspace_bytes(int64_t m, int64_t n, int64_t k, int64_t experts);

/* The step between two blocks of a transformer, in one pass:
 *
 *   h_out = h + residual_scale * gate . N(y; post_weight)
 *   x_out = N(h_out; pre_weight)            N(v; w) = w * v / sqrt(mean(v^2) + eps)
 *
 * with fp32 arithmetic; h_out, x_out and the packed x are each rounded once from
 * fp32 (x from the unrounded h_out).  Optional parts are NULL, others 16-byte
 * aligned. */
enum { RAZER_NORM_POST = 1u /* y is normalised; without it h_out = h + residual_scale * gate . post_weight . y */ };
typedef struct razer_norm {
  int64_t rows;           /* rows times 64 (cols <= 1024), 256 (cols <= 8192) or 1024 threads are one launch: at
                             most 2^26 - 4, 2^24 - 1 or 2^22 - 1 rows (RAZER_E_UNSUPPORTED above) */
  int64_t cols;           /* multiple of 32, at most 32768 */
  int32_t dtype;          /* razer_dtype of y, h, the weights, gate, h_out and x_out */
  uint32_t flags;         /* RAZER_NORM_POST */
  const void* y;          /* device [rows, cols], the block's output; NULL: h_out = h */
  const void* h;          /* device [rows, cols], the residual stream */
  int64_t y_stride;       /* elements from row to row, a multiple of 16 bytes */
  int64_t h_stride;
  const void* post_weight; /* device [cols]; NULL: ones */
  const void* pre_weight;  /* device [cols]; NULL: ones */
  const void* gate;        /* device [gate_rows, cols]; NULL: ones.  Row r takes gate row
                              r / (rows / gate_rows): one gate for all, one a sequence, one a row */
  int64_t gate_rows;       /* divides rows */
  float residual_scale;
  float eps;
  void* h_out;             /* device [rows, cols]; may be NULL, may be h (if its rows are contiguous) */
  void* x_out;             /* device [rows, cols]; may be NULL */
  const razer_mx* packed;  /* x as MXFP4; may be NULL */
} razer_norm;
razer_status razer_block_norm(const razer_norm* a, void* stream);

/* ---- 8-bit integer tensors -------------------------------------------------------
 *
 * THE FORMAT.  X[rows, cols], row-major, cols % 16 == 0, is held as whole numbers
 * with one fp32 scale a row: a scale for each token of an activation, for each
 * output channel of a weight.
 *
 *   scale_r = amax_r / 127                     amax_r = max |x_rc|
 *   code_rc = x_rc * (127 / amax_r), rounded to nearest even (from -127 to 127)
 *
 * in fp32, one rounding an operation (rows with amax_r < 2^-64 are scaled by 2^64
 * on the way, which keeps the quotient finite).  A row of zeros has scale 0 and
 * codes 0; a row with an infinity or NaN has scale NaN and codes 0: all its values,
 * and every product they enter, are NaN. */
typedef struct razer_i8 {
  int64_t rows;  /* >= 0 */
  int64_t cols;  /* >= 0, multiple of 16 */
  int8_t* codes; /* device, rows*cols bytes, 16-byte aligned */
  float* scales; /* device, rows */
} razer_i8;

/* Encode x[out->rows, out->cols] (F32, F16 or BF16; x_stride elements from row to
 * row, a multiple of 16 bytes).  No workspace.  At most 2^34 elements
 * (RAZER_E_UNSUPPORTED above). */
razer_status razer_i8_quantize(const void* x, razer_dtype x_dt, int64_t x_stride, const razer_i8* out,
                               void* stream);

/* Encode silu(g) * u = g * u / (1 + exp(-g)) as razer_mx_quantize_gated does: gu is
 * [out->rows, 2 * out->cols] = [g | u]; the fp32 product is encoded directly. */
razer_status razer_i8_quantize_gated(const void* gu, razer_dtype gu_dt, int64_t gu_stride, const razer_i8* out,
                                     void* stream);

/* Decode to out[rows, cols] = code * scale: one rounding in fp32, and one more to
 * F16 or BF16.  out: 16-byte aligned. */
razer_status razer_i8_dequant(const razer_i8* t, void* out, razer_dtype out_dt, void* stream);

/* y[m, n] = sx[m] * sw[n] * sum_k x[m, k] * w[n, k], M from one token up.  The sum is
 * exact (32-bit integers), is rounded to fp32 and multiplied by sx, then sw; y_dt
 * takes one more rounding.  K == 0, K > RAZER_I8_MAX_K (codes of -128, which the
 * encoder does not write, are summed exactly too) and M or N > 2^30 are
 * RAZER_E_UNSUPPORTED.  y: 16-byte aligned, not in memory that x or w hold.  ws: at
 * least razer_i8_workspace_bytes(M, N, K, 0) bytes, 16-byte aligned (may be 0 -> NULL);
 * launches that can overlap need one each. */
#define RAZER_I8_MAX_K 131056
razer_status razer_i8_gemm(const razer_i8* x, const razer_i8* w, void* y, razer_dtype y_dt, void* ws,
                           size_t ws_bytes, void* stream);

/* The products of a mixture of experts, as razer_mx_gemm_grouped takes them: w stacks
 * `experts` (at most RAZER_MX_MAX_EXPERTS) weights [N, K]; rows offsets[e] ..
 * offsets[e + 1] - 1 of y[M, N] are x[x_rows[r]] * w_e^T (x[r] where x_rows is NULL:
 * M = x->rows).  offsets (experts + 1 ascending row numbers) and x_rows (M) stay on
 * the device.  Rows of y outside every run are left as they were; a row number outside
 * x makes its row zero; offsets outside [0, M] are clamped.  With x_rows the codes of x
 * are less than 4 GiB (RAZER_E_UNSUPPORTED).  ws: razer_i8_workspace_bytes(M, N, K,
 * experts) bytes, 16-byte aligned. */
razer_status razer_i8_gemm_grouped(const razer_i8* x, const razer_i8* w, const int32_t* offsets, int64_t experts,
                                   const int32_t* x_rows, int64_t m, void* y, razer_dtype y_dt, void* ws,
                                   size_t ws_bytes, void* stream);

/* Workspace bytes of a product (experts = 0) or of a grouped one (n: columns of
 * one expert).  Depends on the current device's compute-unit count. */
size_t razer_i8_workspace_bytes(int64_t m, int64_t n, int64_t k, int64_t experts);

/* ---- mixture of experts: from router logits to the products, and back ------------
 *
 * For each token the `top` experts with the best scores, their weights, and the order
 * of rows that razer_i8_gemm_grouped and razer_mx_gemm_grouped take:
 *
 *   s = softmax(logits) or sigmoid(logits)          c = s + bias
 *   groups > 1: the experts are `groups` equal runs; a group's score is the sum of its
 *               group_best largest c; the groups_kept best groups stay
 *   chosen: the `top` largest c of what stays, the best first
 *   weights = scale * s (RAZER_ROUTE_RENORM: s / sum of the chosen s, 0 where that is 0)
 *
 * Equal values go to the lowest index, of groups too.  Scores and choices are worked
 * out in fp64 (experts' scores lie close together: fp32 would now and then choose
 * another), weights are rounded to fp32 once.
 *
 * Logits of -inf, and experts with a bias of -inf or NaN, are never chosen.  Where
 * fewer than `top` experts can be, the rest of a token's places are expert -1, weight
 * 0, slot -1 (a padding token has all its logits -inf).  A token with a NaN or +inf
 * logit has experts -1 and weights NaN.
 *
 * offsets, rows and slots (all given, or all NULL) order the pairs (token, place) by
 * expert, then token: expert e has rows offsets[e] .. offsets[e + 1] - 1 of the grouped
 * products, rows[r] is the token of row r (-1 behind the last one), and slots[t, j] the
 * row of token t's place j.  The order is the same from call to call. */
#define RAZER_MOE_MAX_EXPERTS 1024
#define RAZER_MOE_MAX_TOP 32
#define RAZER_MOE_MAX_GROUPS 64
enum { RAZER_SCORE_SOFTMAX = 0, RAZER_SCORE_SIGMOID = 1 };
enum { RAZER_ROUTE_RENORM = 1u };
typedef struct razer_route {
  int64_t tokens;      /* >= 0; tokens * top < 2^30, tokens <= 2^26, with an order 2^20 (RAZER_E_UNSUPPORTED above:
                          longer batches are routed in parts; an order's time grows with the square of the tokens) */
  int64_t stride;      /* elements from row to row of logits, >= experts */
  int32_t experts;     /* 1 .. RAZER_MOE_MAX_EXPERTS (RAZER_E_UNSUPPORTED above) */
  int32_t top;         /* 1 .. RAZER_MOE_MAX_TOP, at most the experts of the groups kept */
  int32_t groups;      /* 1 .. RAZER_MOE_MAX_GROUPS, divides experts */
  int32_t groups_kept; /* 1 .. groups */
  int32_t group_best;  /* 1 or 2 */
  int32_t score;       /* RAZER_SCORE_* */
  int32_t dtype;       /* razer_dtype of logits */
  uint32_t flags;      /* RAZER_ROUTE_RENORM */
  float scale;
  const void* logits;  /* device [tokens, experts] */
  const float* bias;   /* device [experts]; NULL: none */
  int32_t* chosen;     /* device [tokens, top] */
  float* weights;      /* device [tokens, top] */
  int32_t* offsets;    /* device [experts + 1] */
  int32_t* rows;       /* device [tokens * top] */
  int32_t* slots;      /* device [tokens, top] */
} razer_route;
/* ws: razer_moe_workspace_bytes(tokens, experts, top) bytes, 16-byte aligned (0 without
 * offsets, rows and slots); launches that can overlap need one each. */
razer_status razer_moe_route(const razer_route* a, void* ws, size_t ws_bytes, void* stream);
size_t razer_moe_workspace_bytes(int64_t tokens, int64_t experts, int64_t top);

/* The experts' rows, joined again: out[t] = add[t] + sum_j weights[t, j] * y[slots[t, j]],
 * in fp32 in the order of j, rounded once.  A slot outside [0, y_rows) stands for a row
 * of zeros. */
typedef struct razer_combine {
  int64_t tokens, top, cols; /* top: 1 .. RAZER_MOE_MAX_TOP */
  int64_t y_rows;
  int64_t y_stride;          /* elements from row to row */
  int64_t add_stride;
  int32_t dtype;             /* razer_dtype of y, add and out */
  const void* y;             /* device [y_rows, cols] */
  const int32_t* slots;      /* device [tokens, top] */
  const float* weights;      /* device [tokens, top] */
  const void* add;           /* device [tokens, cols], such as the residual or a shared expert's output; NULL: zeros */
  void* out;                 /* device [tokens, cols]; may be add (if its rows are contiguous), not in memory that y holds */
} razer_combine;
razer_status razer_moe_combine(const razer_combine* a, void* stream);

/* Static, human-readable name of a status code. */
const char* razer_status_string(razer_status s);

#ifdef __cplusplus
}
#endif
#endif /* LIBRAZER_H */
