/*
 * mx.h -- C ABI of the MI355X (gfx950) microscaling block-quantization library
 * (libmx.so).
 *
 * The method.  A tensor is cut into small blocks; each block's largest
 * magnitude fixes one shared scale, every element is divided by it and rounded
 * onto a 4- or 6-bit grid, and codes and scales are stored packed.  Sources,
 * cited by page title and section:
 *   [U]  "Unveiling the Potential of Quantization with MXFP4: Strategies for
 *        Quantization Error Reduction" (walkthrough of the paper's Sec. 2-5):
 *        MXFP4 = 32 E2M1 elements + one E8M0 scale; NVFP4 = 16 E2M1 elements +
 *        one E4M3 scale + a per-tensor scale (Sec. 2, FP4 quantization);
 *        QSNR eq. (1) and (2), the 12x range of E2M1 and 4.25 / 4.5 bits per
 *        element (Sec. 3); Overflow-Aware Scaling and Macro Block Scaling, and
 *        the A.B^T product with block scales (Sec. 4, Fig. 5); the dot-product
 *        unit that resolves per-block scales and adds block partial sums
 *        (Sec. 3, Fig. 4).
 *   [F]  "Is Finer Better? The Limits of Microscaling Formats in LLMs"
 *        (technical summary): UE4M3 scales (smallest 2^-9) need a per-tensor
 *        scale on narrow tensors; UE5M3 (smallest 2^-17) does not.
 *   [B]  "Bridging the Gap Between Promise and Performance for Microscaling FP4
 *        Quantization" (technical summary, Sec. 2.2): block-wise Hadamard
 *        rotation fused into activation quantization.
 *   [A]  ARITH 2025 report on MX quantization for LLM training (research flow
 *        step 3 and main results 3): element types E2M1 / INT4 / E3M0, RTNE,
 *        stochastic and ceil rounding, symmetric or asymmetric scaling, block
 *        size, row / column / 2D block organisation.
 *
 * Conventions for every entry point:
 *  - Every tensor pointer is a DEVICE pointer (memory of the current HIP
 *    device) unless the argument says "host".  The caller allocates and owns
 *    every buffer; the library allocates nothing and keeps no state between
 *    calls, so calls from several host threads on different streams are safe
 *    (the one exception, mx_quantize_noalloc, keeps a static scratch array
 *    per GPU; see there).
 *  - `stream` is a hipStream_t passed as void* (NULL = the null stream).  Work
 *    is enqueued and the call returns at once, except mx_qsnr, which waits.
 *  - Return value: MX_OK, or an MX_ERR_* code.  Every argument is checked
 *    before anything is launched; on error nothing is launched and no output
 *    is touched.  MX_ERR_HIP reports a failed launch.
 *  - 16-byte alignment is required of every tensor pointer (MX_ERR_ALIGN).
 */
#ifndef MX_H
#define MX_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------ */
#define MX_OK 0
#define MX_ERR_ARG 1          /* bad value, shape or null pointer            */
#define MX_ERR_UNSUPPORTED 2  /* valid format that this library does not run */
#define MX_ERR_ALIGN 3        /* pointer or leading dimension not aligned    */
#define MX_ERR_WORKSPACE 4    /* workspace missing or smaller than required  */
#define MX_ERR_HIP 5          /* a HIP launch failed                         */
#define MX_ERR_TOO_LARGE 6    /* mx_quantize_noalloc: the call needs more    *
                               * scratch than its static array holds         */

/* ---- element types [A], [U] --------------------------------------------
 * Codes are sign-magnitude unless noted; no format has Inf or NaN and every
 * element saturates at its largest magnitude.
 *  E2M1   4 bits, magnitudes {0, .5, 1, 1.5, 2, 3, 4, 6}, code = s<<3 | index
 *  INT4   4 bits; symmetric: -7..7 as a two's-complement nibble;
 *         asymmetric: 0..15 steps above the block offset
 *  FP6    6 bits, E2M3 (bias 1, max 7.5) or E3M2 (bias 3, max 28)
 *  E3M0   4 bits, magnitudes {0, 1/4, 1/2, 1, 2, 4, 8, 16} (exponent only)
 *  FP8    8 bits, E4M3 (bias 7, max 448) or E5M2 (bias 15, max 57344): the
 *         MX family's 8-bit elements ([U], current state: MX formats of 8, 6
 *         and 4 bits); their Inf/NaN codes are never produced               */
enum { MX_ELEM_E2M1 = 0, MX_ELEM_INT4 = 1, MX_ELEM_FP6_E2M3 = 2, MX_ELEM_FP6_E3M2 = 3,
       MX_ELEM_E3M0 = 4, MX_ELEM_FP8_E4M3 = 5, MX_ELEM_FP8_E5M2 = 6 };

/* ---- block-scale types [U], [F], [A] ------------------------------------
 *  E8M0   one byte, the power of two 2^(code-127); 0xFF marks a block that
 *         held a NaN or Inf
 *  UE4M3  unsigned E4M3 (bias 7, max 448, smallest 2^-9), RNE of amax/Qmax;
 *         0x7F marks a non-finite block
 *  NVFP4  UE4M3 block scale times an fp32 per-tensor scale g = amax_t/(Qmax*448)
 *  UE5M3  unsigned E5M3 (bias 15, smallest 2^-17, max 1.75*2^16), RNE of
 *         amax/Qmax, no per-tensor scale; 0xFF marks a non-finite block
 *  E3M0   three exponent bits read as a step-down c in 0..7 below a per-tensor
 *         exponent e_ref: scale = 2^(e_ref - c); 0xFF marks a non-finite block */
enum { MX_SCALE_E8M0 = 0, MX_SCALE_UE4M3 = 1, MX_SCALE_NVFP4 = 2, MX_SCALE_UE5M3 = 3,
       MX_SCALE_E3M0 = 4 };

/* ---- E8M0 exponent rule [U] Sec. 4 ---------------------------------------
 *  FLOOR  e = floor(log2 amax) - emax(element)        (the OCP MX rule)
 *  CEIL   smallest e with Qmax * 2^e >= amax           (amax maps onto Qmax)
 *  OAS    smallest e with tau * 2^e >= amax, Qmax <= tau < 2 Qmax: the block
 *         maximum may overflow Qmax (and saturate) so that fewer small values
 *         flush to zero.  E3M0 scales always use the CEIL rule.           */
enum { MX_RULE_FLOOR = 0, MX_RULE_CEIL = 1, MX_RULE_OAS = 2 };

/* ---- element rounding [A] ----------------------------------------------
 *  RTNE  nearest grid value, ties to the even code
 *  SR    stochastic: between neighbours lo <= |v| < hi go up iff r < f * 2^16,
 *        f = (|v| - lo) / (hi - lo), r = 16 bits of Philox4x32-10 with counter
 *        (idx/8, rng_offset), key seed, word (idx/2)%4, half idx%2, where idx =
 *        row*cols + col of the element in the tensor
 *  CEIL  the smallest grid value >= v (a negative value's magnitude rounds down) */
enum { MX_ROUND_RTNE = 0, MX_ROUND_SR = 1, MX_ROUND_CEIL = 2 };

enum { MX_DTYPE_F32 = 0, MX_DTYPE_BF16 = 1 };

/* A quantization format.  Block shapes: 1 x b (row), b x 1 (column) or b x b
 * (2D).  asymmetric: INT4 min/max scaling or E2M1 with a mid-range offset
 * (E8M0 scales only).  hadamard: 0, or h in {16, 32, 64, 128}: every
 * contiguous run of h values in a row is rotated by H_h / sqrt(h) before it is
 * quantized ([B]); codes, dequantized values and statistics are then in the
 * rotated domain.  macro_cols: 0, or 128 for Macro Block Scaling ([U] Sec. 4):
 * each 1x128 macro block gets a UE4M3 scale s_M in [1, 2] (the mantissa of
 * amax/Qmax), elements are divided by s_M, and 1 x block_cols sub-blocks get
 * E8M0 scales.  oas_tau: the OAS threshold.  seed, rng_offset: the SR key. */
typedef struct mx_format {
    int32_t elem, scale, rule, round;
    int32_t block_rows, block_cols;
    int32_t asymmetric;
    int32_t hadamard;
    int32_t macro_cols;
    float oas_tau;
    uint64_t seed, rng_offset;
} mx_format;

/* A quantized tensor (the struct is host memory; its pointers are device
 * memory; unused pointers may be NULL).  Layout, all row-major:
 *  codes         rows x (cols/2) bytes for 4-bit elements, element 2i in the
 *                low nibble of byte i; rows x (3*cols/4) bytes for FP6, a
 *                least-significant-bit-first stream of 6-bit codes per row;
 *                rows x cols bytes for FP8, one code per byte
 *  scales        (rows/block_rows) x (cols/block_cols) bytes
 *  offsets       same grid, bf16 (asymmetric only)
 *  macro_scales  rows x (cols/128) bytes of UE4M3 (Macro Block Scaling only)
 *  tensor_scale  one fp32 (NVFP4 only)
 *  ref_exp       one int32 (E3M0 scales only)                              */
typedef struct mx_qtensor {
    void *codes;
    void *scales;
    void *offsets;
    void *macro_scales;
    float *tensor_scale;
    int32_t *ref_exp;
    int64_t rows, cols;
} mx_qtensor;

/* Fidelity statistics [U] Sec. 3: sig2 = sum x^2 and err2 = sum (x - xq)^2
 * (float64), n elements, nonzero = #{x != 0}, flushed = #{x != 0 and xq = 0},
 * zero_blocks = #{blocks whose dequantized values are all zero}.
 * QSNR eq. (1) = 10 log10(sig2 / err2); MSE = err2 / n.                     */
typedef struct mx_stats {
    double sig2, err2;
    int64_t n, nonzero, flushed, zero_blocks;
} mx_stats;

/* Byte sizes of every output of mx_quantize for this format and shape, and of
 * the device workspace it needs (zero when it needs none).  `out` is host.
 * The storage is the format's bit budget: codes at the element width plus one
 * scale byte per block, 4 + 8/32 = 4.25 bits per element for 1 x 32 blocks
 * and 4.5 for 1 x 16 ([U] Sec. 3); plus the bf16 offsets, the macro scales
 * (one byte per 1 x 128), the fp32 tensor scale or the int32 reference
 * exponent where the format has them.  Returns MX_ERR_ARG / MX_ERR_UNSUPPORTED
 * for a format or shape mx_quantize would reject; `out` is then untouched.  */
typedef struct mx_sizes {
    size_t codes, scales, offsets, macro_scales, tensor_scale, ref_exp, workspace;
} mx_sizes;

int mx_query_sizes(const mx_format *f, int64_t rows, int64_t cols, mx_sizes *out);

/* Quantize x (rows x cols, row stride ld elements, dtype in_dtype) into `out`.
 * dequant (nullable): the dequantized tensor, rows x cols dense, dtype dq_dtype
 * (fake quantization).  stats (nullable, device): the statistics of x against
 * its dequantized values, written when the stream reaches them.  workspace:
 * device scratch of at least mx_query_sizes().workspace bytes (no initial
 * contents needed); calls that share one workspace must not overlap.
 * Shapes this library runs: rows % block_rows == 0 and cols % block_cols == 0;
 * row blocks b in {8, 16, 32, 64, 128, 256} with cols % 8 == 0; column and 2D
 * blocks b in {8, 16, 32}; ld a multiple of 16 bytes.                       */
int mx_quantize(const mx_format *f, int in_dtype, const void *x, int64_t rows,
                int64_t cols, int64_t ld, const mx_qtensor *out, void *dequant,
                int dq_dtype, mx_stats *stats, void *workspace, size_t ws_bytes,
                void *stream);

/* mx_quantize without a workspace argument, for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation.  It runs the same kernels as mx_quantize;
 * what they need beyond the caller's inputs and outputs (the statistics
 * partials and the NVFP4 / E3M0 pre-pass maxima) goes into a static device
 * array of MX_NOALLOC_SCRATCH_BYTES that the library holds on each GPU it runs
 * on until the process ends.  The call itself allocates nothing (no hipMalloc,
 * no allocating library routine).  Its first call on a device looks up that
 * device's address of the array.
 *  - Limit: a call whose mx_query_sizes().workspace exceeds
 *    MX_NOALLOC_SCRATCH_BYTES returns MX_ERR_TOO_LARGE before any launch
 *    (4 MiB holds the statistics of about 350 M elements of row blocks).
 *    Calls that need no workspace (no statistics, no pre-pass) have no limit.
 *  - Every call on one GPU shares that GPU's array: calls that overlap in
 *    time on one GPU (two streams, two host threads) race and give wrong
 *    statistics or tensor scales.  Serialise them.  No initial contents are
 *    needed: every call writes what it reads.
 * Other arguments, errors and outputs: as mx_quantize.                      */
#define MX_NOALLOC_SCRATCH_BYTES (4u << 20)
int mx_quantize_noalloc(const mx_format *f, int in_dtype, const void *x, int64_t rows,
                        int64_t cols, int64_t ld, const mx_qtensor *out, void *dequant,
                        int dq_dtype, mx_stats *stats, void *stream);

/* One tensor of an mx_quantize_many call: mx_quantize's arguments for it,
 * without a dequantized output.  The struct and `out` are host memory; x,
 * out's buffers, stats and workspace are device memory.  workspace: at least
 * mx_query_sizes(f, rows, cols).workspace bytes when the job has statistics
 * or the format a pre-pass (NULL and 0 otherwise). */
typedef struct mx_qjob {
    const void *x;
    int64_t rows, cols, ld;
    const mx_qtensor *out;
    mx_stats *stats;
    void *workspace;
    size_t ws_bytes;
} mx_qjob;

/* Quantize several tensors of one format and input dtype, such as both
 * operands of a layer's A.B^T ([U] Sec. 4, Fig. 5): job i's codes, scales and
 * statistics are those mx_quantize(f, in_dtype, jobs[i].x, jobs[i].rows, ...)
 * writes.  jobs: host array of `count` entries (count >= 0; jobs may be NULL
 * when count is 0).
 *  - Dense MXFP4-style row jobs share launches: E2M1 elements, E8M0 scales
 *    (any rule), round to nearest, symmetric, no rotation, no macro scales,
 *    1 x b blocks, ld == cols.  Up to eight such jobs run in one quantization launch,
 *    their workgroups split in proportion to their sizes, and the statistics
 *    of all of them in one finalize launch, where calling mx_quantize for
 *    each would launch two kernels per tensor.  Every other job runs as
 *    mx_quantize runs it, one after another.
 *  - Every job is checked before the first launch, as mx_quantize checks its
 *    arguments (first failing job's status); MX_ERR_ARG also when two jobs that
 *    need a workspace name overlapping workspace bytes.
 *  - Jobs must not write overlapping memory; the order in which they run is
 *    unspecified.  Calls that share a workspace must not overlap. */
int mx_quantize_many(const mx_format *f, int in_dtype, const mx_qjob *jobs, int count, void *stream);

/* Dequantize q into y (rows x cols, row stride ld elements, dtype out_dtype
 * MX_DTYPE_F32 or MX_DTYPE_BF16, rounded to nearest even): each element is its
 * code's value times its block's scale (plus the block's offset when
 * asymmetric, times the macro scale under MBS, times the tensor scale for
 * NVFP4), the value mx_quantize's dequant output and statistics use.  This is
 * the fake (simulated) quantization with which [A] (research flow step 1)
 * studies MX formats on hardware that does not run them.  A block whose scale
 * code is NaN dequantizes to NaN.  q's buffers as mx_quantize wrote them;
 * ld >= cols with ld * element size a multiple of 16 (MX_ERR_ALIGN).        */
int mx_dequantize(const mx_format *f, const mx_qtensor *q, int out_dtype, void *y,
                  int64_t ld, void *stream);

/* QSNR eq. (1)/(2) of [U] Sec. 3 between two tensors of n elements: `ref` is
 * the reference A (or the product A.B), `approx` its quantized counterpart.
 * host_stats (host, nullable) receives the statistics (zero_blocks = 0) and
 * qsnr_db (host) the QSNR in dB (+inf when the two are equal).  Waits for the
 * stream.  Returns MX_ERR_ARG if ||ref|| = 0.  workspace: device scratch of at
 * least mx_qsnr_workspace_size(n) bytes.                                   */
size_t mx_qsnr_workspace_size(int64_t n);
int mx_qsnr(int dtype, const void *ref, const void *approx, int64_t n,
            mx_stats *host_stats, double *qsnr_db, void *workspace, size_t ws_bytes,
            void *stream);

/* Block-scaled GEMM ([U] Sec. 3 Fig. 4, Sec. 4 Fig. 5): C = deq(A) . deq(B)^T
 * with A an M x K and B an N x K quantized tensor in row blocks along K; fp32
 * accumulation, C (M x N, row stride ldc elements) in bf16 (rounded to nearest
 * even) or fp32.  Formats, per operand:
 *  - E8M0 scales on 1 x 32 blocks (any rule) with E2M1 (MXFP4), FP6 E2M3 /
 *    E3M2 (MXFP6) or FP8 E4M3 / E5M2 (MXFP8) elements, chosen independently
 *    for A and B (the mixed 4-/6-bit products of [A], main results; MX also
 *    has 8-bit formats, [U] current state): the gfx950 block-scaled
 *    FP8/FP6/FP4 matrix instruction.  MXFP4 operands may carry macro-block
 *    scales (macro_cols 128, [U] Sec. 4 MBS and Fig. 5: each 128-wide K step's
 *    partial product is multiplied by the two rows' UE4M3 macro scales).
 *  - E2M1 elements under UE4M3, NVFP4 (UE4M3 + fp32 tensor scale), UE5M3 or
 *    E8M0 scales on 1 x b blocks, b a multiple of 8 (when the other operand
 *    is not of the kind above): the codes times their block scales are
 *    decoded exactly, to fp16 when both operands have UE4M3 scales and to
 *    bf16 otherwise, and the fp16 / bf16 matrix instruction multiplies.
 *    Macro-block scales over E8M0 sub-blocks of other widths (the 1 x 128
 *    macro over 1 x 16 blocks, [U] Sec. 4 MBS) take this route too, with E8M0
 *    block scales on both operands: each block's scale is 2^e times its macro
 *    block's UE4M3 scale (exact in fp32) and the decode applies it.
 * Anything else (INT4 / E3M0 elements, asymmetric, rotated, column or 2D
 * blocks, macro scales on FP6 / FP8 or against fp8 block scales):
 * MX_ERR_UNSUPPORTED.  Shapes: K % 32 == 0 and
 * whole blocks (MX_ERR_ARG otherwise); any M, N.  E8M0 products with K a
 * multiple of 128 run on LDS-staged kernels (MXFP4 x MXFP4 without macro
 * scales and K a multiple of 1024 on the most tuned one), other K on a
 * register-only kernel; the decoded formats with 1 x 16 or 1 x 32 blocks and
 * K a multiple of 128 on an LDS-staged kernel, the rest register-only.  A
 * block whose scale code is NaN (E8M0 0xFF, UE4M3 0x7F, UE5M3 0xFF) makes its
 * row of C (column, for B) NaN.  macro_scales must be set when
 * the format has macro_cols, tensor_scale for NVFP4 (MX_ERR_ARG).          */
int mx_gemm(const mx_format *fa, const mx_qtensor *a, const mx_format *fb,
            const mx_qtensor *b, void *c, int64_t ldc, int c_dtype, void *stream);

/* ---- one decode step with quantized weights and a quantized cache ----------
 * The entry points below serve new tokens with weights and a key-value cache
 * in this library's formats: the product of a few unquantized tokens with a
 * 4-bit weight, the norm and rotation of query and key heads (with its
 * gradient, for training), the write of new keys and values to a paged cache,
 * and the attention of one new token per sequence over that cache.  Index
 * vectors (positions, slots, lengths, page numbers) and lse need the alignment
 * of their elements alone, so slices of them serve.  A call whose launch would
 * hold 2^32 threads or more is refused (MX_ERR_ARG, nothing launched): none is
 * with up to 2^28 - 32 weight rows, 2^26 - 256 head vectors of mx_qk_rope,
 * 2^27 - 8 of mx_cache_write, and fewer than 2^23 pairs of a sequence and a
 * query head of mx_attend; larger calls are where their lanes do more each.  */

/* y = x . deq(W)^T + bias for a few tokens: x is tokens x w->cols (row stride
 * ldx elements, dtype x_dtype), W a quantized tensor of w->rows x w->cols, y
 * tokens x w->rows (row stride ldy, y_dtype, rounded to nearest even from the
 * fp32 sum), bias (nullable) w->rows values of x_dtype.
 *  - Formats: E2M1 or INT4 elements in row blocks 1 x b of 8 .. 256 elements
 *    under E8M0 (any rule), UE4M3, NVFP4 or UE5M3 scales, macro-block scales
 *    included, symmetric or asymmetric.  How the codes were rounded does not
 *    matter.  Anything else (other elements, E3M0 scales, rotation, column or
 *    2D blocks): MX_ERR_UNSUPPORTED.
 *  - W's values enter exactly (decoded to bf16, which holds every code times
 *    its scale as multiples of 2^-133; INT4 as multiples of 2^-129, which only
 *    macro scales can need more of; an E2M1 value past fp32's range makes its
 *    row's outputs non-finite), an fp32 x as the exact sum of three bf16
 *    parts (multiples of 2^-133); products are summed in fp32 in a fixed order.
 *    An offset or the INT4 bias enters as offset times the block's sum of x
 *    (multiples of 2^-129 beside INT4 offsets).  Symmetric INT4 is (u - 8) s
 *    with u = 0 .. 15, summed as u s x and -8 s x: its sums round by |u s x| and
 *    |8 s x|.
 *  - A NaN scale code makes its row's outputs NaN, a NaN or Inf in a token
 *    makes that token's outputs non-finite, other tokens are untouched.
 *  - Any number of tokens runs; the kernel is made for up to 16 (more read the
 *    weight once per 16).  0 < w->cols < 2^24, tokens <= 1048560, w->rows < 2^31
 *    and no more than a launch holds (above).
 *  - x, W's buffers, bias and y 16-byte aligned, ldx a multiple of 16 bytes
 *    (MX_ERR_ALIGN).  y must not overlap an input.                           */
int mx_matvec(const mx_format *fw, const mx_qtensor *w, int x_dtype, const void *x, int64_t tokens,
              int64_t ldx, const void *bias, void *y, int64_t ldy, int y_dtype, void *stream);

/* A set of heads: tokens x heads vectors of one dimension (given with it),
 * the vector contiguous, strides in elements.  Strides times the element size
 * are multiples of 16 bytes, and so is x (MX_ERR_ALIGN).  Outputs must not
 * hold one address twice.                                                    */
typedef struct mx_heads {
    void *x;
    int64_t token_stride, head_stride;
    int32_t heads, dtype;
} mx_heads;

/* What mx_qk_rope does to each head vector x of `dim` values (a multiple of
 * 8, at most 1024): with a weight w, n = x (mean(x^2) + eps)^-1/2 and u = w n;
 * without one (NULL) u = x.  Then the first rot_dim values (even, 0 .. dim)
 * are rotated in pairs by the angles of the token's position p:
 *   y_a = u_a cos - u_b sin,  y_b = u_b cos + u_a sin
 * with (a, b) = (i, i + rot_dim/2), or (2i, 2i + 1) when `interleaved`, and
 * cos, sin at [p][i] of two tables of table_rows x rot_dim/2 fp32 values.  A
 * position outside the table makes that token's rotated values NaN (all of
 * its gradients through a norm).  tokens x heads < 2^31, and no more than a
 * launch holds (above).  Everything
 * between load and store is fp32.  q_weight and k_weight have w_dtype.       */
typedef struct mx_rope {
    int64_t tokens;
    int32_t dim, rot_dim, interleaved, w_dtype;
    const void *q_weight, *k_weight;
    const float *cos, *sin;
    int64_t table_rows;
    const int32_t *positions;
    float eps;
} mx_rope;

/* Norm and rotation of query and key heads, one pass over both: q_out and
 * k_out have the inputs' heads and dtype and may be the inputs themselves
 * (same strides), else must not overlap them.  k and k_out may be NULL
 * (queries only).                                                            */
int mx_qk_rope(const mx_rope *r, const mx_heads *q, const mx_heads *k, const mx_heads *q_out,
               const mx_heads *k_out, void *stream);

/* Its gradient.  dy_q, dy_k: the gradients of its outputs; q, k: its inputs;
 * dq, dk: the gradients of its inputs (may be dy_q, dy_k themselves, same
 * strides); dq_weight, dk_weight: fp32, dim values each, required where the
 * weight is set (NULL otherwise), overwritten.  With g the dy rotated back,
 * dw = sum g n over tokens and heads, and dx = rstd (w g - n mean(n w g)).
 * The weight sums are formed in fp32 in a fixed order.  workspace: at least
 * mx_qk_rope_workspace_size(r) bytes where a weight is set; no initial
 * contents needed; calls that share one must not overlap.  k, dy_k and dk may
 * be NULL together.  All heads have one dtype.                               */
size_t mx_qk_rope_workspace_size(const mx_rope *r);
int mx_qk_rope_backward(const mx_rope *r, const mx_heads *dy_q, const mx_heads *dy_k, const mx_heads *q,
                        const mx_heads *k, const mx_heads *dq, const mx_heads *dk, float *dq_weight,
                        float *dk_weight, void *workspace, size_t ws_bytes, void *stream);

/* A paged cache of keys and values: `pages` pages of page_size tokens for
 * `heads` heads of `dim` values (64, 96, 128, 192 or 256).  k and v:
 * [page][head][token][dim] values in bf16 (format NULL), or codes as
 * mx_quantize lays out rows of dim elements (MXFP8 E4M3: dim bytes, MXFP4:
 * dim / 2) with k_scales and v_scales [page][head][token][dim / 32] E8M0
 * bytes.  format: E4M3 or E2M1 elements, E8M0 scales (any rule) on 1 x 32
 * blocks, to nearest, symmetric, not rotated (MX_ERR_UNSUPPORTED otherwise).
 * The struct is host memory.  page_size 1 .. 65536, pages * page_size < 2^40. */
typedef struct mx_kv_cache {
    const mx_format *format;
    void *k, *v, *k_scales, *v_scales;
    int64_t pages;
    int32_t page_size, heads, dim;
} mx_kv_cache;

/* Writes the keys and values of `tokens` new tokens to the cache.  k and v:
 * cache->heads heads of cache->dim values each, one dtype (fp32 inputs are
 * rounded to nearest even for a bf16 cache).  slots (device): token i goes to
 * page slots[i] / page_size at slots[i] % page_size; a slot outside the cache
 * (negative, or past its end) skips the token.  Codes and scales are those
 * mx_quantize writes for the same values.  Two tokens of one slot in one call
 * leave either's values.  tokens x heads < 2^30, and no more than a launch
 * holds (above).                                                             */
int mx_cache_write(const mx_kv_cache *cache, const mx_heads *k, const mx_heads *v, int64_t tokens,
                   const int64_t *slots, void *stream);

/* Attention of one new token per sequence: for sequence b and query head h
 *   out[b][h] = sum_t p_t v_t,  p = softmax over t < lengths[b] of
 *   scale * (q[b][h] . k_t),  lse[b][h] = log sum_t exp(scale q.k_t)
 * over the tokens that page_table[b][t / page_size] and t % page_size name in
 * the cache, of key-value head h / (q->heads / cache->heads).  q and out:
 * `batch` tokens of q->heads heads (a multiple of cache->heads), one dtype;
 * lse nullable, fp32, batch x q->heads dense.  page_table: batch rows of
 * table_cols int32 pages, row stride table_stride; lengths: int32.
 *  - lengths[b] <= 0 leaves an empty row: out 0, lse -inf.  A length past the
 *    table (table_cols * page_size) counts as that.  What lies in the cache
 *    at and past a length is not used, whatever it holds.  A page number
 *    outside the cache makes its sequence's outputs NaN.
 *  - Scores, softmax statistics and sums are fp32.  A bf16 q multiplies the
 *    cache's exact values; fp32 q enters as the exact sum of three bf16 parts
 *    (multiples of 2^-133).
 *    Probabilities enter the second product as two bf16 parts (16 bits; three
 *    parts for fp32), their sum in fp32.
 *  - The length is split over workgroups, their parts joined in a fixed order;
 *    the same inputs give the same bits.  workspace: at least
 *    mx_attend_workspace_size bytes; no initial contents needed; calls that
 *    share one must not overlap.  That size serves every call of at most this
 *    batch and these table_cols over a cache of the same format, page size,
 *    heads and dim, with the same query heads: a server allocates it once for
 *    its largest.  table_cols * page_size < 2^30.                            */
size_t mx_attend_workspace_size(const mx_kv_cache *cache, int64_t batch, int32_t q_heads, int64_t table_cols);
int mx_attend(const mx_kv_cache *cache, const mx_heads *q, int64_t batch, const int32_t *page_table,
              int64_t table_cols, int64_t table_stride, const int32_t *lengths, float scale,
              const mx_heads *out, float *lse, void *workspace, size_t ws_bytes, void *stream);

/* Reads cached keys and values back: token i's, which lie where mx_cache_write
 * puts slot slots[i], as cache->heads heads of cache->dim values in k and v
 * (one dtype; no two places the same).  A code counts its value times its
 * block's scale (NaN under scale code 255), rounded to nearest even for bf16
 * outputs; a bf16 cache's values as they are.  A slot outside the cache reads
 * as zeros.  One slot may come up any number of times.  Limits as
 * mx_cache_write's.                                                          */
int mx_cache_read(const mx_kv_cache *cache, const int64_t *slots, int64_t tokens, const mx_heads *k,
                  const mx_heads *v, void *stream);

/* ---- many requests on one base model ----------------------------------------
 * A batch whose requests share the quantized model and a prompt.  Index vectors
 * (prefix and page tables, lengths, ids, targets, top_ids) and vectors of fp32
 * per token or adapter (lse, logprob, entropy and their gradients,
 * top_logprobs, scales) need the alignment of their elements alone.  A call
 * whose launch would hold 2^32 threads or more is refused (MX_ERR_ARG).      */

/* mx_attend for sequences that share their first tokens: sequence b and query
 * head h attend over the prefix's tokens, t < *prefix_length at
 * prefix_table[t / page_size], and then over the sequence's own, t <
 * lengths[b] by page_table and lengths as in mx_attend.  The result is
 * mx_attend's for the prefix's and the own tokens as one sequence; the prefix
 * is read once for all sequences (for up to 256 pairs of a sequence and a query
 * head of one key-value head, 128 with fp32 queries or more than 128 values a
 * head, and once more for each further as many).
 *  - prefix_table, prefix_length (one number): int32 on the device.
 *    *prefix_length <= 0 is no prefix, one past the table counts as the table.
 *    lengths[b] <= 0: the prefix alone.  Neither: out 0, lse -inf.  A page
 *    outside the cache among the prefix's makes every sequence's outputs NaN.
 *  - Everything else, rounding and order included, as mx_attend; the two agree
 *    up to the order of sums in fp32, and but for tokens of the prefix of less
 *    than 2^-122 of the likeliest's probability (mx_attend: 2^-126), which
 *    count as 0.  workspace: at least
 *    mx_attend_shared_workspace_size bytes for this batch and these columns,
 *    which serves every smaller call over a cache of the same form.          */
size_t mx_attend_shared_workspace_size(const mx_kv_cache *cache, int64_t batch, int32_t q_heads,
                                       int64_t prefix_cols, int64_t table_cols);
int mx_attend_shared(const mx_kv_cache *cache, const mx_heads *q, int64_t batch, const int32_t *prefix_table,
                     int64_t prefix_cols, const int32_t *prefix_length, const int32_t *page_table,
                     int64_t table_cols, int64_t table_stride, const int32_t *lengths, float scale,
                     const mx_heads *out, float *lse, void *workspace, size_t ws_bytes, void *stream);

/* Low-rank adapters of one projection (n outputs, k inputs; the struct is host
 * memory).  a: count x rank x k and b: count x n x rank, dense, of `dtype`
 * (fp32 or bf16); scales (nullable: all 1): count fp32.  rank: a multiple of 8
 * up to 256 (pad with zeros); k: a multiple of 8 (MX_ERR_UNSUPPORTED
 * otherwise), below 2^24; n < 2^31.                                          */
typedef struct mx_adapters {
    const void *a, *b;
    const float *scales;
    int64_t k, n;
    int32_t count, rank, dtype;
} mx_adapters;

/* y[t] = base[t] + scales[i] b_i (a_i x[t]) with i = ids[t]: what each token's
 * request adds to a shared projection, such as mx_matvec's or mx_gemm's.  x:
 * tokens x k of the adapters' dtype (row stride ldx, a multiple of 16 bytes);
 * ids: int32 on the device; base (nullable: zero): tokens x n of base_dtype,
 * row stride ld_base; y: tokens x n of y_dtype, row stride ldy, rounded once,
 * to nearest even.  y may be base itself (same dtype and stride), else must
 * not overlap an input.
 *  - An id outside 0 .. count - 1 names no adapter: y[t] = base[t].  Tokens
 *    may come in any order; the adapters are read once for each 16 tokens in
 *    a row that name them, so tokens of one adapter are best side by side.
 *  - Products and sums are fp32 (a x too: bf16 operands enter exactly, and the
 *    rank values enter the second product as exact sums of three bf16 parts,
 *    multiples of 2^-133).  A NaN or Inf in a token's x reaches its y alone,
 *    one in an adapter the tokens that name it; an Inf in a bf16 b may leave
 *    NaN there, as it multiplies parts that are 0.
 *  - workspace: at least mx_lora_workspace_size(a, tokens) bytes, which serves
 *    fewer tokens and smaller ranks too; no initial contents needed; calls that
 *    share one must not overlap.  tokens <= 2^24.                             */
size_t mx_lora_workspace_size(const mx_adapters *a, int64_t tokens);
int mx_lora(const mx_adapters *a, const void *x, int64_t tokens, int64_t ldx, const int32_t *ids, int base_dtype,
            const void *base, int64_t ld_base, int y_dtype, void *y, int64_t ldy, void *workspace, size_t ws_bytes,
            void *stream);

/* What a step's logits say of given tokens: for each row z of logits (tokens x
 * vocab, row stride ld >= vocab, any; fp32 or bf16)
 *   lse = log sum_j exp(z_j),  logprob = z[target] - lse,
 *   entropy = -sum_j p_j log p_j  with p_j = exp(z_j - lse),
 * and, where top > 0, the `top` (at most 64 and vocab) likeliest: top_ids and
 * top_logprobs (tokens x top, dense), likeliest first, equal logits by the lower
 * id.  targets: int64; one outside 0 .. vocab - 1 has logprob 0 (padding).
 *  - Logits of -Inf (masked tokens) have probability 0 and count nothing.  A row
 *    of them alone: lse, logprob and top_logprobs -Inf, entropy 0.  A row with
 *    a NaN or +Inf: everything NaN (a padding target's logprob stays 0), the
 *    top_ids some ids of the vocabulary.
 *  - fp32 throughout, sums in an order fixed by the sizes and by where rows
 *    start against 16 bytes.  workspace: at least mx_logprobs_workspace_size
 *    bytes, which serves every smaller call; may be NULL where the row count
 *    alone fills the chip (1024 tokens or more).                             */
size_t mx_logprobs_workspace_size(int64_t tokens, int64_t vocab, int32_t top);
int mx_logprobs(int dtype, const void *logits, int64_t tokens, int64_t vocab, int64_t ld, const int64_t *targets,
                float *logprob, float *lse, float *entropy, int32_t top, float *top_logprobs, int64_t *top_ids,
                void *workspace, size_t ws_bytes, void *stream);

/* The gradient of logprob and entropy: with g = d_logprob[t] and e =
 * d_entropy[t] (either NULL: zero),
 *   d_logits[j] = g (1[j = target] - p_j) - e p_j (log p_j + entropy)
 * of the logits' dtype, row stride ld_d, rounded once; d_logits may be the
 * logits themselves (same stride).  lse and entropy: as mx_logprobs gave them
 * (entropy only where d_entropy is set).  A target outside the vocabulary has
 * no gradient of its logprob; a row without a possible token, none at all.    */
int mx_logprobs_backward(int dtype, const float *d_logprob, const float *d_entropy, const void *logits,
                         int64_t tokens, int64_t vocab, int64_t ld, const int64_t *targets, const float *lse,
                         const float *entropy, void *d_logits, int64_t ld_d, void *stream);

/* Text for a status code (static storage). */
const char *mx_status_string(int status);

#ifdef __cplusplus
}
#endif
#endif /* MX_H */
