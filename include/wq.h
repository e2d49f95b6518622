/*
 * wq.h -- C ABI of the group-wise low-bit weight-quantized linear layer
 * library for AMD Instinct MI355X (gfx950).
 *
 * Pages the operations follow (titles translated):
 *   [P1] "LLM quantization selection: five mainstream schemes compared"
 *        (www.0539edu.com/news/5934728)
 *   [P2] the quantization-concepts article "many people's understanding of
 *        quantization stops at making the model smaller"
 *        (aicoding.csdn.net/6a6874d110ee7a33f2936327.html)
 *   [P3] "LLM quantization hands-on manual" (devpress.csdn.net/awstech/...)
 *   [P5] "Inference & deployment 05: quantized deployment compared (GPTQ,
 *        AWQ, GGUF, FP8)" (devpress.csdn.net/amd/6a55d4ea662f9a54cb8f2c4c.html)
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - W is [n][k] row-major: n output features, k input features.  x is
 *    [m][k] row-major, y is [m][n] row-major, y = x . w_hat^T.
 *  - Every data pointer is a DEVICE pointer owned by the caller, except
 *    the wq_weight descriptor itself and wq_nf4_codebook's output, which
 *    are host memory read/written during the call.  The library allocates
 *    nothing on the device and frees nothing; scratch space, where an
 *    operation needs it, is the caller's `workspace`, sized by the matching
 *    *_workspace() query.
 *  - `stream` is a hipStream_t passed as an opaque pointer (NULL = the
 *    null stream).  Calls only enqueue work on `stream` and never
 *    synchronize; outputs are valid once `stream` reaches them.  Calls on
 *    different streams that write distinct buffers may overlap.
 *  - Argument checks happen before any HIP call, so a call that returns an
 *    error other than WQ_ERR_HIP has enqueued nothing.  WQ_ERR_HIP reports
 *    a failed kernel launch.  NaN/Inf inputs are not checked and give
 *    unspecified (but memory-safe) results.
 *  - Sizes: every dimension (m, n, k) is below 2^23 and every matrix
 *    (n x k weights, m x k activations, m x n outputs) holds at most 2^34
 *    elements; larger sizes return WQ_ERR_SHAPE.
 *  - Rounding: every "round" is round-half-to-even; every division is an
 *    IEEE fp32 division; 16-bit conversions round to nearest even.
 *  - The library's only mutable global state is the per-kernel LDS limit it
 *    raises once (atomically) on first use and, per GPU, the address of the
 *    no-allocation scratch array (looked up once, under a lock); calls are
 *    thread-safe, except that wq_linear_int8_decomp_noalloc calls sharing a
 *    GPU's scratch must not overlap.
 */
#ifndef WQ_H
#define WQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  WQ_OK = 0,
  WQ_ERR_NULL = 1,        /* a required pointer is NULL                       */
  WQ_ERR_SHAPE = 2,       /* sizes are negative, zero where not allowed, or   */
                          /* not multiples of what the format needs           */
  WQ_ERR_ALIGN = 3,       /* a pointer misses its documented alignment        */
  WQ_ERR_UNSUPPORTED = 4, /* a valid but unimplemented combination            */
  WQ_ERR_WORKSPACE = 5,   /* workspace NULL or smaller than the query says    */
  WQ_ERR_HIP = 6          /* a kernel launch failed                           */
} wq_status;

typedef enum { WQ_F16 = 0, WQ_BF16 = 1, WQ_F32 = 2, WQ_E4M3 = 3 /* caches only */ } wq_dtype;

typedef enum {
  WQ_FMT_INT4_ASYM = 0,   /* wq_quantize_groupwise(bits=4, symmetric=0)       */
  WQ_FMT_NF4 = 1,         /* wq_pack_nf4                                      */
  WQ_FMT_INT8_SYM_ROW = 2,/* wq_quantize_groupwise(bits=8, symmetric=1, k)    */
  WQ_FMT_FP4 = 3,         /* wq_pack_fp4                                      */
  WQ_FMT_FP8_BLOCK = 4    /* wq_quantize_fp8_block                            */
} wq_format;

/*
 * A quantized weight matrix, as produced by the quantize/pack calls.
 *
 *  fmt = WQ_FMT_INT4_ASYM:
 *    codes   uint32 [n][k/8]; element (r, c) in bits 4*(c%8)..+3 of word
 *            (r, c/8).  16-byte aligned.
 *    scales  fp16 [n][G], G = k/group.  2-byte aligned.
 *    zeros   uint8 [n][ceil(G/2)]; zero point of group g in byte g/2, low
 *            nibble when g is even.
 *    group   the group size along k (128 is the workload value).
 *  fmt = WQ_FMT_NF4:
 *    codes   uint8 [n*k/2]; element 2j is the low nibble of byte j (the
 *            same order as INT4 inside a little-endian word).  16-byte
 *            aligned.
 *    scales  int8 [n*k/group] double-quantized absmax when scales2 != NULL,
 *            else fp32 [n*k/group] absmax.
 *    scales2 fp32 [ceil(n*k/group / group2)] second-level scales, or NULL.
 *    group   NF4 block size (64); group2 the double-quant block (256).
 *  fmt = WQ_FMT_FP4: the NF4 layout with E2M1 codes (see wq_pack_fp4).
 *  perm (INT4 only, optional): act-order.  The input channels were
 *    quantized in the order perm[0], perm[1], ... ([P1] 3.2, [P4] 3.2), so
 *    the groups run along that order: codes, scales and zeros hold the
 *    columns in that order (column j is input channel perm[j]; quantize
 *    W[:, perm], made by wq_permute_columns).  wq_linear_w4a16 then gathers
 *    x[:, perm] into its workspace before the multiply.  NULL: plain order.
 *  fmt = WQ_FMT_INT8_SYM_ROW:
 *    codes   int8 [n][k], 16-byte aligned; scales fp32 [n]; group = k.
 *  fmt = WQ_FMT_FP8_BLOCK:
 *    codes   E4M3 (OCP: largest 448, no infinities) [n][k], one byte each,
 *            16-byte aligned, k % 16 == 0.
 *    scales  fp32 [ceil(n/128)][ceil(k/128)], one per block of 128 rows x 128
 *            columns (blocks at the ends may be smaller); group = 128.
 */
typedef struct {
  int32_t fmt;            /* wq_format                                        */
  int32_t group;
  int64_t n, k;
  const void* codes;
  const void* scales;
  const uint8_t* zeros;   /* INT4 only, else NULL                             */
  const float* scales2;   /* NF4 double quantization only, else NULL          */
  int32_t group2;
  int32_t reserved;
  const int32_t* perm;    /* INT4 act-order: device int32 [k], else NULL      */
} wq_weight;

/*
 * Group-wise weight quantization (one launch).
 *
 * bits = 4, symmetric = 0 (asymmetric INT4, [P5] section 2.3 with b = 4;
 * per-group granularity [P5] 2.2, group 128 [P1] 3.2):
 *   for each row r and group g of `group` consecutive k:
 *     lo = min(min w, 0), hi = max(max w, 0)     (the range holds float 0,
 *                                                 which the zero point encodes)
 *     s  = fp16((hi - lo) / 15)   (1.0 if that rounds to 0)
 *     z  = clamp(round(-lo / s), 0, 15)
 *     q  = clamp(round(w / s) + z, 0, 15)
 *   outputs: codes uint32 [n][k/8], scales fp16 [n][k/group],
 *   zeros uint8 [n][ceil((k/group)/2)] (layout as in wq_weight).
 *   group in {32, 64, 128}; k % group == 0.
 *
 * bits = 8, symmetric = 1, group = k (vector-wise INT8, one scale per output
 * feature, [P1] 2.1; symmetric formula [P5] 2.3):
 *     s = max|w[r,:]| / 127 (1.0 for an all-zero row),
 *     q = clamp(round(w / s), -127, 127)
 *   outputs: codes int8 [n][k], scales fp32 [n]; zeros must be NULL.
 *
 * w: fp16 or bf16 [n][k] (wdt), 16-byte aligned, k % 8 == 0.
 * Other (bits, symmetric, group) combinations return WQ_ERR_UNSUPPORTED.
 */
wq_status wq_quantize_groupwise(const void* w, int32_t wdt, int64_t n, int64_t k,
                                int32_t bits, int32_t group, int32_t symmetric,
                                void* codes, void* scales, uint8_t* zeros,
                                void* stream);

/*
 * NF4 blockwise quantization ([P1] sections 6.1-6.3, [P5] 6.1-6.2).
 *
 *   Blocks of `block` (64) consecutive elements of the row-major W:
 *     a = max|w| (fp32); code = number of the 15 level midpoints that w/a
 *     exceeds (nearest NF4 level, ties to the lower); a == 0 gives code 7.
 *   double_quant != 0: blocks of `block2` (256) consecutive absmax values,
 *     c2 = max(a)/127 (1.0 if 0), q8 = clamp(round(a/c2), 0, 127);
 *     absmax receives int8 q8 [nblocks], absmax_scale fp32 c2
 *     [ceil(nblocks/block2)].
 *   double_quant == 0: absmax receives fp32 a [nblocks]; absmax_scale must
 *     be NULL.
 *   codes: uint8 [n*k/2], two codes per byte, element 2j low nibble.
 *
 * w: fp16 or bf16, 16-byte aligned; n*k % block == 0; block == 64;
 * block2 == 256 when double_quant.
 */
wq_status wq_pack_nf4(const void* w, int32_t wdt, int64_t n, int64_t k,
                      int32_t block, int32_t double_quant, int32_t block2,
                      uint8_t* codes, void* absmax, float* absmax_scale,
                      void* stream);

/*
 * FP4 blockwise quantization, the FP4 variant of the NF4 path ([P1] 6.3
 * names bitsandbytes' NF4 and FP4 formats; the E2M1 layout, sign bit,
 * 2-bit exponent, 1-bit mantissa, is [P5] 7.2).  Arguments, blocks, absmax
 * and double quantization exactly as wq_pack_nf4; only the codes differ:
 *   code bit 3 = (w/a < 0); bits 0-2 = number of the 7 midpoints between
 *   adjacent E2M1 magnitudes {0, 1/2, 1, 3/2, 2, 3, 4, 6}/6 that |w/a|
 *   exceeds (nearest magnitude, ties to the lower); a == 0 gives code 0.
 * Code c decodes to wq_fp4_codebook()[c] * absmax (code 8 is -0).
 */
wq_status wq_pack_fp4(const void* w, int32_t wdt, int64_t n, int64_t k,
                      int32_t block, int32_t double_quant, int32_t block2,
                      uint8_t* codes, void* absmax, float* absmax_scale,
                      void* stream);

/*
 * The FP4 codebook (host call, no GPU): out[c] = E2M1 value of code c / 6
 * in fp32, exponent bias 1 (out[7] = 1, out[15] = -1, out[8] = -0).
 */
wq_status wq_fp4_codebook(float* out);

/*
 * The NF4 codebook the library uses (host call, no GPU): 16 fp32 levels,
 * ascending, out[0] = -1, out[7] = 0, out[15] = 1.  Level i > 7 is
 * PhiInv(p_i)/PhiInv(31/32) for p_i = 1/2 + (31/32 - 1/2) (i-7)/8, level
 * i < 7 is -PhiInv(q_i)/PhiInv(31/32) for q_i = 1/2 + (31/32 - 1/2)(7-i)/7
 * (quantiles at evenly spaced probabilities, [P1] 6.1).  `out` is host
 * memory of 16 floats.
 */
wq_status wq_nf4_codebook(float* out);

/*
 * Scratch bytes wq_linear_w4a16 needs for this (m, weight) pair: an
 * act-order weight needs m * k * 2 bytes (rounded up to 256) for the
 * gathered activations; every other weight needs none (0).  Returns 0 for
 * invalid arguments as well (the call itself then reports the error).
 */
size_t wq_linear_w4a16_workspace(int64_t m, const wq_weight* w);

/*
 * Fused dequantize-and-multiply (W4A16: 4-bit weights, 16-bit activations;
 * the weights are dequantized back to 16 bits and multiplied in 16-bit
 * with fp32 accumulation, [P1] section 5 opening, [P1] 6.2, [P2] 十一).
 *
 *   y[i][j] = sum_c x[i][c] * w_hat[j][c]
 *     INT4: w_hat = (q - z) * s, NF4 and FP4: w_hat = L[code] * a_hat
 *     (L the format's codebook), with fp32 accumulation.
 *
 * Decode-shaped calls (m <= 16) run a bandwidth-bound dequant-GEMV; larger
 * m runs an MFMA dequant-GEMM (the GEMV / GEMM kernel versions of [P1] 4.3).
 *
 * x: xdt in {WQ_F16, WQ_BF16}, [m][k], 16-byte aligned.  w: fmt INT4_ASYM
 * (group 128, 64 or 32: the group-size knob of [P5] 2.2 and [P1] 3.2), NF4
 * or FP4 (block 64).  y: ydt in {F16, BF16, F32}, [m][n].
 * workspace: at least wq_linear_w4a16_workspace(m, w) bytes, 256-byte
 * aligned (may be NULL when that is 0).  m >= 1; k % 128 == 0.  With
 * w->perm set (INT4 act-order) the activations are gathered into the
 * workspace first; NF4/FP4 with perm give WQ_ERR_UNSUPPORTED.
 */
wq_status wq_linear_w4a16(const void* x, int32_t xdt, int64_t m,
                          const wq_weight* w, void* y, int32_t ydt,
                          void* workspace, size_t ws_bytes, void* stream);

/*
 * The gate and up projections of a gated MLP block ([P3] step 4 lists the
 * gate, up and down projections of each block) as one call sharing x:
 *
 *   act = 0:  y_gate = x * W_gate_hat^T,  y_up = x * W_up_hat^T
 *             (each exactly what wq_linear_w4a16 computes for it);
 *   act = 1:  y_gate = silu(g) * u with silu(v) = v / (1 + exp(-v)), for
 *             m <= 16 with g, u those two products in fp32 (y_up is not
 *             written and may be NULL); for m > 16 with g, u the two GEMM
 *             outputs as stored in ydt (y_up is required: it receives u).
 *
 * For m <= 16 one pass streams both matrices with the activations staged
 * once; larger m runs the two GEMMs.
 *
 * x: xdt in {WQ_F16, WQ_BF16}, [m][k], 16-byte aligned.  w_gate, w_up: one
 * format for both -- INT4_ASYM (group 128, 64 or 32), NF4 or FP4 (block 64,
 * both with or both without double quantization) -- with equal n and k.
 * y_gate, y_up: ydt in {F16, BF16, F32}, [m][n] each (y_up may be NULL when
 * act = 1 and m <= 16).
 * Errors: WQ_ERR_SHAPE when n, k or the group size differ; WQ_ERR_NULL when
 * y_up is NULL for act = 0 or for act = 1 with m > 16; WQ_ERR_UNSUPPORTED
 * for mixed formats, INT8 weights, NF4/FP4 with double quantization on one
 * matrix only, act-order weights or act outside {0, 1}.  No workspace.
 */
wq_status wq_linear_w4a16_gate_up(const void* x, int32_t xdt, int64_t m,
                                  const wq_weight* w_gate, const wq_weight* w_up,
                                  int32_t act, void* y_gate, void* y_up, int32_t ydt,
                                  void* stream);

/*
 * LLM.int8() activation side ([P1] 2.1; threshold 6.0 in [P5] 6.1):
 *   outlier columns O = { c : |x[i][c]| > threshold for some row i }
 *     (strict); mask[c] = 1 for c in O else 0; idx = ascending list of O,
 *     *count = |O| (device int32).
 *   per row i: sx[i] = max_{c not in O} |x[i][c]| / 127 (1.0 if 0),
 *     qx[i][c] = clamp(round(x[i][c] / sx[i]), -127, 127), 0 for c in O.
 * x: fp16 [m][k], 16-byte aligned, k % 16 == 0.  mask uint8 [k] (16-byte
 * aligned), idx int32 [k], count int32 [1], qx int8 [m][k] (16-byte
 * aligned), sx fp32 [m].  threshold >= 0 (use +inf for no outliers).
 */
wq_status wq_int8_prepare_activations(const void* x, int64_t m, int64_t k,
                                      float threshold, uint8_t* mask,
                                      int32_t* idx, int32_t* count, int8_t* qx,
                                      float* sx, void* stream);

/* Scratch bytes of wq_linear_int8_decomp (mask, idx, count, qx, sx). */
size_t wq_linear_int8_decomp_workspace(int64_t m, int64_t k);

/*
 * LLM.int8() mixed-precision decomposition ([P1] 2.1):
 *   y = acc * sx[i] * sw[j] + sum_{c in O} x[i][c] * w16[j][c]
 *   acc[i][j] = sum_c qx[i][c] * qw[j][c]   (exact int32)
 *   w16 = fp16(fp32(qw) * sw)               (the int8 weights dequantized;
 *                                            no fp16 copy of W is kept)
 * x: fp16 [m][k], 16-byte aligned; w: fmt INT8_SYM_ROW with k % 128 == 0 and
 * k <= 133,143 (so that 127 * 127 * k, the largest possible |acc|, fits in
 * int32; larger k returns WQ_ERR_SHAPE); y: ydt in {F16, BF16, F32}
 * (acc * sx * sw plus the outlier sum in fp32, rounded once to ydt).
 * workspace: at least
 * wq_linear_int8_decomp_workspace(m, k) bytes, 256-byte aligned.
 * outlier_count (device int32, nullable) receives |O|; acc_out (device int32
 * [m][n], nullable) receives acc.
 */
wq_status wq_linear_int8_decomp(const void* x, int64_t m, const wq_weight* w,
                                float threshold, void* y, int32_t ydt,
                                void* workspace, size_t ws_bytes,
                                int32_t* outlier_count, int32_t* acc_out,
                                void* stream);

/*
 * wq_linear_int8_decomp for callers that cannot allocate device memory
 * (code under HIP graph capture, serving loops and harnesses that forbid
 * allocation): the same computation and kernels, with no workspace
 * argument.  The scratch (outlier mask and list, count, int8 activations,
 * row scales) is a device array of WQ_INT8_NOALLOC_SCRATCH_BYTES inside the
 * library, one per GPU, held until the process ends; the call allocates and
 * frees nothing.  Arguments, results and errors as wq_linear_int8_decomp;
 * calls whose wq_linear_int8_decomp_workspace(m, k) exceeds the array return
 * WQ_ERR_WORKSPACE, and WQ_ERR_HIP also reports a failure to find the
 * array on the current device.  Every call on one GPU uses that GPU's
 * array and leaves its contents behind (no byte of it needs to start at
 * zero): calls that overlap on one GPU -- on different streams or from
 * different host threads -- race, and the caller must order them.
 */
#define WQ_INT8_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)
wq_status wq_linear_int8_decomp_noalloc(const void* x, int64_t m, const wq_weight* w,
                                        float threshold, void* y, int32_t ydt,
                                        int32_t* outlier_count, int32_t* acc_out,
                                        void* stream);

/*
 * Column gather (act-order reordering, [P1] 3.2, [P4] 3.2):
 *   dst[r][j] = src[r][perm[j]],  r < rows, j < k.
 * src, dst: dt in {F16, BF16} [rows][k], distinct buffers, dst 16-byte
 * aligned; perm: device int32 [k], a permutation of 0..k-1 (entries outside
 * [0, k) are clamped: wrong values, no out-of-bounds access); k % 8 == 0.
 */
wq_status wq_permute_columns(const void* src, int32_t dt, int64_t rows, int64_t k,
                             const int32_t* perm, void* dst, void* stream);

/*
 * Column scaling for SmoothQuant-style W8A8 ([P1] section 5: the
 * activation range is moved into the weights by a per-channel s, folded
 * offline; then the INT8 product runs with no outlier columns, i.e.
 * wq_linear_int8_decomp with threshold = +inf):
 *   dst[r][c] = round16(src[r][c] * scale[c])  (fp32 product, one rounding)
 * Use scale = s on the weights before wq_quantize_groupwise(bits = 8) and
 * scale = 1/s on the activations.  src, dst: dt in {F16, BF16} [rows][k],
 * 16-byte aligned, may be the same buffer; scale: device fp32 [k];
 * k % 8 == 0.
 */
wq_status wq_scale_columns(const void* src, int32_t dt, int64_t rows, int64_t k,
                           const float* scale, void* dst, void* stream);

/*
 * Residual addition and root-mean-square norm, with 16-bit and / or FP8
 * outputs.  Per row of k values:
 *   h = x + residual  (x alone when residual is NULL), in fp32
 *   residual_out = round16(h)
 *   v = h * rsqrt(sum(h^2) / k + eps) * gain, in fp32, of the unrounded h
 *   y = round16(v)
 *   per block b of 128 consecutive values (the last may be shorter):
 *     s = max|v| / 448 (1.0 if 0; at least 2^-126),
 *     q = E4M3(v / s), the fp32 quotient rounded to nearest, scales[b][row] = s
 *
 * x, residual, residual_out, gain, y: dt in {WQ_F16, WQ_BF16}; x [m] rows of
 * k, ldx elements apart; residual and residual_out [m] rows ldr apart; gain
 * [k]; y [m][k]; q E4M3 [m][k]; scales fp32 [ceil(k/128)][m] (the scales of
 * one block over all rows are contiguous).  residual and residual_out are
 * both given or both NULL; residual_out may be the residual, or x with
 * ldx == ldr (in place); no other output may overlap an input.  y may be
 * NULL when q is given; q and scales are both given or both NULL.
 * k % 8 == 0; ldx and ldr at least k and multiples of 8; m, k and the strides
 * below 2^23; every 16-bit pointer 16-byte, q 8-byte, scales 4-byte aligned;
 * eps >= 0.  Infinities and NaN follow the formula, within their row: a NaN
 * makes all of v NaN; an infinity, or a sum of squares past the fp32 range
 * (bf16 values above 1e18), makes v 0, and NaN where h is infinite.  A block
 * of v with a NaN has a NaN scale.
 */
wq_status wq_add_rmsnorm(const void* x, int32_t dt, int64_t m, int64_t k, int64_t ldx,
                         const void* residual, void* residual_out, int64_t ldr,
                         const void* gain, float eps, void* y, void* q, float* scales,
                         void* stream);

/*
 * Quantize activation rows to E4M3 with a scale per 128 values:
 *   v = x, or silu(x) * up when up is given (silu(t) = t / (1 + exp(-t)), fp32),
 *   s, q as in wq_add_rmsnorm.
 * x, up: dt in {WQ_F16, WQ_BF16} [m][k], 16-byte aligned; q E4M3 [m][k], 8-byte
 * aligned; scales fp32 [ceil(k/128)][m]; k % 8 == 0.  A block with a NaN has a
 * NaN scale, one with an infinity an infinite scale, and what q * s gives is not
 * finite where the value was not.
 */
wq_status wq_quantize_fp8_rows(const void* x, const void* up, int32_t dt, int64_t m, int64_t k,
                               void* q, float* scales, void* stream);

/*
 * Quantize a weight to WQ_FMT_FP8_BLOCK: per block of 128 x 128
 *   s = max|w| / 448 (1.0 if 0; at least 2^-126), q = E4M3(w / s).
 * w: wdt in {WQ_F16, WQ_BF16} [n][k], 16-byte aligned, k % 16 == 0; codes E4M3
 * [n][k], 16-byte aligned; scales fp32 [ceil(n/128)][ceil(k/128)].
 */
wq_status wq_quantize_fp8_block(const void* w, int32_t wdt, int64_t n, int64_t k, void* codes,
                                float* scales, void* stream);

/*
 * Scratch bytes of wq_linear_fp8 for this (m, weight) pair and any ydt, at most
 * 64 MiB: fp32 totals of the parts k is split into where the output tiles alone do
 * not fill the GPU, 0 elsewhere (and for invalid arguments).
 */
size_t wq_linear_fp8_workspace(int64_t m, const wq_weight* w);

/*
 * FP8 linear with block scales:
 *   y[i][j] = sum_b sx[b][i] * sw[j/128][b] * sum_{c in block b} q[i][c] * codes[j][c]
 * For a 16-bit y a sum over a block of 128 is formed by the FP8 matrix
 * instructions, which cut every product towards zero at 2^-17 of the largest
 * power of two among the block's products (a code below 2^-6 counted as 2^-6):
 * off by at most 2^-10 of the largest product, by 1.5e-5 of the sum for codes
 * spread normally.  For an fp32 y it is formed from exact products in fp32; the scaled sums are added in fp32, in an order fixed
 * by the sizes (results are deterministic), and rounded once to ydt.
 * q: E4M3 [m][k], 16-byte aligned; scales fp32 [ceil(k/128)][m] (as
 * wq_add_rmsnorm and wq_quantize_fp8_rows write them); w: fmt FP8_BLOCK, any n;
 * y: ydt in {F16, BF16, F32} [m][n], 16-byte aligned.  workspace: at least
 * wq_linear_fp8_workspace(m, w) bytes, 256-byte aligned (may be NULL when that
 * is 0).  m >= 1.  NaN codes give NaN in the rows or columns that hold them.
 */
wq_status wq_linear_fp8(const void* q, const float* scales, int64_t m, const wq_weight* w,
                        void* y, int32_t ydt, void* workspace, size_t ws_bytes, void* stream);

/*
 * Mixture-of-experts layer for a few tokens (m <= 64):
 *   l = x . router^T (fp32), or the caller's `logits`
 *   p = softmax(l); the top_k experts of the largest l, ties to the lowest
 *   index; renormalize != 0: their p divided by their sum
 *   a = round16(silu(x . gate_e^T) * (x . up_e^T))
 *   y = sum_j p_j * (a . down_e^T)
 * with fp32 sums; a is rounded to xdt (as any 16-bit model keeps it: in fp16 it
 * is infinite from 65520 on), y to ydt.
 * The order of every sum is fixed by the sizes and the routing: results are
 * deterministic.  INT4 weights enter as (q - z) * s, unrounded.
 *
 * x: xdt in {F16, BF16} [m][h], 16-byte aligned.  router: xdt [experts][h],
 * 16-byte aligned, or NULL with logits: fp32 [m][experts] (exactly one of the
 * two).  gate, up: the experts' matrices stacked, n = experts * i, k = h; down:
 * n = experts * h, k = i; all three in one format: INT4_ASYM without perm
 * (equal groups) or FP8_BLOCK.  y: ydt in {F16, BF16, F32} [m][h].
 * ids: int32 [m][top_k] and probs: fp32 [m][top_k], NULL or written, in the
 * order of decreasing l.  workspace: at least wq_moe_workspace(m, top_k, gate,
 * experts) bytes, 256-byte aligned (0 for arguments that wq_moe refuses).
 * h and i multiples of 128; INT4 scales 8-byte and zeros 2-byte aligned;
 * experts <= 512; top_k <= min(experts, 16).
 *
 * A logit of -inf masks its expert: its p is 0 and it is chosen only after all
 * others; a token whose experts are all masked gets p = 0 and y = 0.  A choice
 * with p = 0 is not computed.  A NaN or +inf logit gives NaN in that token's
 * probs and y, and in no other token's.
 * Errors: WQ_ERR_UNSUPPORTED for m, experts or top_k past their limits, mixed
 * or other formats.
 */
size_t wq_moe_workspace(int64_t m, int32_t top_k, const wq_weight* gate, int64_t experts);
wq_status wq_moe(const void* x, int32_t xdt, int64_t m, const void* router, const float* logits,
                 int64_t experts, int32_t top_k, int32_t renormalize, const wq_weight* gate,
                 const wq_weight* up, const wq_weight* down, void* y, int32_t ydt, int32_t* ids,
                 float* probs, void* workspace, size_t ws_bytes, void* stream);

/*
 * A paged cache of the keys and values of one layer, written by wq_append_kv and
 * read by the attention calls below.  It has `pages` pages of page_size tokens;
 * token t of a page p, head h and component c of k and of v are element
 *   p * page_stride + h * head_stride + t * token_stride + c
 * (strides in elements, the same for k and v), so a page may hold its heads or its
 * tokens outermost.  A slot is page * page_size + place of the token in the page.
 *  dt          WQ_F16, WQ_BF16, or WQ_E4M3: codes with one fp32 scale per token and
 *              head, k_scales and v_scales fp32 [pages][kv_heads][page_size]
 *              (NULL for the 16-bit types)
 *  head_dim    64 or 128
 *  page_size   a power of two, at most 65536; pages * page_size below 2^31
 *  strides     multiples of 16 bytes, such that no two places overlap; k and v span
 *              at most 2^34 elements each
 * k and v 16-byte, scales 4-byte aligned.
 */
typedef struct {
  int32_t dt;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t page_size;
  int64_t pages;
  int64_t page_stride, head_stride, token_stride;
  void* k;
  void* v;
  float* k_scales;
  float* v_scales;
} wq_kv_cache;

/*
 * Rotary rotation of queries and keys, and append of keys and values to the cache.
 *   (c, s) = cos_sin[positions[row]][i], [rot/2 + i];  for every pair i < rot/2 of a
 *   head, (a, b) = elements (i, i + rot/2), or (2i, 2i + 1) when interleaved != 0:
 *     a' = a c - b s,  b' = b c + a s         (fp32; the head's other elements stay)
 *   q_out = round(q'),  k of the slot = k', v of the slot = v: rounded to 16 bits, or
 *   for WQ_E4M3  scale = max|.| / 448 over the head (1 if 0; at least 2^-126),
 *   code = E4M3(. / scale) of the unrounded values (as wq_add_rmsnorm's q).
 * q [m][heads][head_dim], k and v [m][kv_heads][head_dim] in dt in {F16, BF16}, rows
 * ldq, ldk, ldv elements apart (so they may be parts of one projection's output);
 * q_out in dt, rows ldo apart, may be q with ldo == ldq (in place), and overlaps no
 * other input otherwise; q and q_out are both given or both NULL.  cos_sin fp32
 * [max_pos][rot], positions int32 [m]; both NULL when rot == 0; a position outside
 * [0, max_pos) is taken as the nearest one inside.  slots int32 [m]: a row whose
 * slot is negative or past the cache is not stored (its q_out is written); slots
 * that occur twice in one call hold a mix of their rows.
 * A 16-bit cache has dt; rot a multiple of 16, at most head_dim; ldq, ldk, ldv, ldo
 * multiples of 8, at least a row's elements; kv_heads and heads at most 1024; q, k,
 * v, q_out, cos_sin 16-byte, positions and slots 4-byte aligned.  NaN and infinities
 * stay in their head, and follow wq_quantize_fp8_rows in an E4M3 cache.
 */
wq_status wq_append_kv(const void* q, const void* k, const void* v, int32_t dt, int64_t m,
                       int64_t heads, int64_t ldq, int64_t ldk, int64_t ldv,
                       const int32_t* positions, const float* cos_sin, int64_t max_pos,
                       int64_t rot, int32_t interleaved, void* q_out, int64_t ldo,
                       const int32_t* slots, const wq_kv_cache* cache, void* stream);

/*
 * Attention of one new token for each of m sequences over the cache.  Query head h
 * reads kv head h / (heads / kv_heads).  For row i with n = lens[i] tokens, the new
 * one (at n - 1, already in the cache) among them:
 *   visible: j < n and (window == 0 or n - 1 - j < window or j < sinks)
 *   z_j = scale * q . k_j,  y = sum_j exp(z_j) v_j / sum_j exp(z_j),
 *   lse = log sum_j exp(z_j)                  (sums over the visible j)
 * A row that sees nothing (n <= 0) gets y = 0 and lse = -inf.  z and all sums are
 * fp32 and the order of every sum is fixed by the sizes and lens: results are
 * deterministic.  The weights of v are kept to 16 significant bits; those of an F16
 * cache no finer than 2^-32 of the row's largest weight.
 *
 * q [m][heads][head_dim] in dt in {F16, BF16}, rows ldq elements apart; a 16-bit
 * cache has dt.  pages int32 [m] rows of max_pages, ldp apart: token j of row i is
 * in page pages[i][j / page_size] at j % page_size.  Entries behind a row's last
 * token are not used; an entry outside the cache is taken as the nearest page
 * inside, lens past max_pages * page_size (at most 2^30) as that.  Places that no row
 * sees are not used, whatever they hold.  y dt [m][heads][head_dim]; lse fp32
 * [m][heads] or NULL; neither overlaps an input, the other or the workspace.
 * A query, key or scale that is not finite makes what it enters not finite or, where
 * its z is -inf, leaves it out; a value (or its scale) that is not finite makes the
 * components that it enters not finite (with a weight of 0, as z is -inf or the
 * exponential underflows, it may or may not).  No other row is touched by it.  Values past 2^118 over the number of tokens may overflow the
 * fp32 sums, whose weights go up to 2^8.
 * heads a multiple of kv_heads, at most 1024; ldq a multiple of 8; window and sinks
 * >= 0; scale > 0, finite; q and y 16-byte, pages, lens, lse 4-byte aligned.
 * workspace: at least wq_attention_decode_workspace(m, heads, cache) bytes, 256-byte
 * aligned; the query gives 0 for arguments that the call refuses.
 */
size_t wq_attention_decode_workspace(int64_t m, int64_t heads, const wq_kv_cache* cache);
wq_status wq_attention_decode(const void* q, int32_t dt, int64_t m, int64_t heads, int64_t ldq,
                              const wq_kv_cache* cache, const int32_t* pages, int64_t max_pages,
                              int64_t ldp, const int32_t* lens, float scale, int64_t window,
                              int64_t sinks, void* y, float* lse, void* workspace,
                              size_t ws_bytes, void* stream);

/*
 * Causal attention of several new tokens for each of `batch` sequences: sequence b
 * has the rows starts[b] .. starts[b+1] - 1 of q, the last of its lens[b] tokens
 * (all of them in the cache), so row r of it is at lens[b] - starts[b+1] + r.
 * Formula, arguments and limits as wq_attention_decode, with a row's own position in
 * the place of n - 1: it sees j at or before its position.  A row at a negative
 * position sees nothing (y = 0, lse = -inf).  Rows of q before starts[0] or from
 * starts[batch] on are not read, and y and lse not written there.
 * starts int32 [batch + 1], ascending, within [0, m]; lens int32 [batch]; pages
 * int32 [batch] rows of max_pages; batch * kv_heads below 2^21.  The weights of v are
 * rounded to dt (bf16 for WQ_E4M3; two bf16 parts, 16 bits, when dt is F16), those of an
 * F16 cache no finer than 2^-32 of the row's largest weight; the sum of weights is not
 * rounded.
 * workspace: at least wq_attention_prompt_workspace(m, heads, batch, cache) bytes,
 * 256-byte aligned (may be NULL when that is 0).  The query grows with m to at most 17
 * MB and does not depend on batch: what suffices for m rows does for fewer, in any
 * number of sequences.
 */
size_t wq_attention_prompt_workspace(int64_t m, int64_t heads, int64_t batch,
                                     const wq_kv_cache* cache);
wq_status wq_attention_prompt(const void* q, int32_t dt, int64_t m, int64_t heads, int64_t ldq,
                              const int32_t* starts, int64_t batch, const wq_kv_cache* cache,
                              const int32_t* pages, int64_t max_pages, int64_t ldp,
                              const int32_t* lens, float scale, int64_t window, int64_t sinks,
                              void* y, float* lse, void* workspace, size_t ws_bytes,
                              void* stream);

/*
 * Dequantize a whole weight into 16-bit values (a test and debugging hook;
 * an act-order weight comes out in its stored column order):
 * INT4: fp(q - z) * s rounded to odt; NF4, FP4: L[code] * a_hat rounded to odt;
 * INT8 and FP8: fp32(q) * s rounded to odt.  out: odt in {F16, BF16} [n][k].
 */
wq_status wq_dequantize(const wq_weight* w, void* out, int32_t odt, void* stream);

/* Static, human-readable name of a status code. */
const char* wq_status_string(int32_t status);

#ifdef __cplusplus
}
#endif

#endif /* WQ_H */
