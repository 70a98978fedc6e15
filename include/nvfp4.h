/*
 * nvfp4.h -- C ABI of the MI355X (gfx950) NVFP4 linear-layer library.
 *
 * The library implements the 4-bit linear-layer path of NVIDIA's NVFP4
 * pretraining recipe as described on these pages:
 *   [P1] hyper.ai, "NVIDIA revolutioniert KI-Praetrainingsgeschwindigkeit mit
 *        4-Bit-Genauigkeit" (body: 4-bit pretraining with dynamic scaling on
 *        accelerated GEMMs).
 *   [P3] aibuzzwire.news, Thinking Machines "End-to-End 4-Bit Training"
 *        article; sections "Warum weniger Bits ein schnelleres Training
 *        bedeuten" (rounding to the nearest representable value) and
 *        "Unterschiedliche Phasen, unterschiedliche Regeln" (backward passes
 *        are sensitive to rounding bias).
 *   [P4] aisight.pl, "Koniec marnowania mocy. NVIDIA udowadnia, ze 4 bity
 *        wystarcza do trenowania gigantow"; sections "Architektura NVFP4
 *        kontra ograniczenia mikroskalowania" (16-element blocks, E4M3 block
 *        scale, extra FP32 per-tensor scale) and "Technologie stabilizujace
 *        proces treningowy" (random Hadamard transforms on weight gradients,
 *        stochastic rounding).
 *
 * Conventions shared by every entry point
 *  - Pointers named x, y, c and every pointer inside nvfp4_tensor are DEVICE
 *    pointers owned by the caller; the library never allocates, frees or
 *    retains them.  nvfp4_tensor structs themselves are HOST memory.
 *  - hip_stream is a hipStream_t (NULL = the default stream).  All work is
 *    enqueued on it; calls return without synchronising.
 *  - Argument errors are reported synchronously, before anything is
 *    launched.  NVFP4_ERR_HIP reports a failed launch.
 *  - Sizes are int64_t and may be 0 (empty tensors are valid, see below).
 *    Limits of the launch geometry (NVFP4_ERR_SHAPE beyond them):
 *    quantization down the columns (axis 0, and the dual call) takes
 *    rows <= 4 194 240 (MXFP4: 16 776 960, MXFP8: 8 388 480); the NVFP4
 *    GEMMs take K <= 2^25 - 16 (MXFP8: K <= 2^24 - 128)
 *    and ceil(M/256) * ceil(N/128) <= INT32_MAX; every element count
 *    (rows * cols, outer * k, M * ldc) is at most 2^60.
 *  - Element types: NVFP4_F32 (binary32) or NVFP4_BF16 (bfloat16).
 *  - Thread safety: stateless; concurrent calls on different outputs are
 *    fine.  The calls keep no scratch memory between launches (the one
 *    workspace, of nvfp4_gemm_ws, belongs to the caller).
 */
#ifndef NVFP4_H
#define NVFP4_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    NVFP4_OK = 0,
    NVFP4_ERR_NULL = -1,   /* a required pointer is NULL                      */
    NVFP4_ERR_SHAPE = -2,  /* negative size, K % 16 != 0, mismatched shapes,
                              size beyond a documented limit                */
    NVFP4_ERR_ENUM = -3,   /* unknown dtype / rounding / axis value           */
    NVFP4_ERR_HIP = -4,    /* a HIP launch failed                             */
    NVFP4_ERR_ALIGN = -5,  /* a pointer or leading dimension is misaligned    */
    NVFP4_ERR_VALUE = -6   /* a scalar (eps, temperature) is out of range     */
} nvfp4_status;

typedef enum { NVFP4_F32 = 0, NVFP4_BF16 = 1 } nvfp4_dtype;
typedef enum { NVFP4_RNE = 0, NVFP4_SR = 1 } nvfp4_rounding;

/*
 * An NVFP4 tensor in its quantized layout [outer][k], k being the GEMM
 * reduction length ([P4] "Architektura NVFP4 ..."):
 *  codes  : u8 [outer][k/2]; element 2j of a row in the low nibble of byte j,
 *           element 2j+1 in the high nibble.  A nibble is an E2M1 code:
 *           bit 3 sign, bits 0-2 the magnitude 0, .5, 1, 1.5, 2, 3, 4, 6.
 *           8-byte aligned.
 *  scales : u8 [outer][k/16]; the OCP E4M3FN block scale of each 16-element
 *           block along k (never NaN, at most 448).  4-byte aligned when k %
 *           64 == 0 and the tensor is a GEMM operand (whole scale dwords move
 *           by DMA then); any alignment otherwise.
 *  meta   : f32 [2]; meta[0] = amax (the tensor maximum magnitude after the
 *           optional transform), meta[1] = g = amax / 2688, the FP32 decode
 *           scale.  4-byte aligned.
 *  outer, k : k % 16 == 0.
 * The value of element (o, kk) is e2m1(code) * e4m3(scale) * g.
 */
typedef struct {
    uint8_t *codes;
    uint8_t *scales;
    float *meta;
    int64_t outer;
    int64_t k;
} nvfp4_tensor;

/*
 * nvfp4_quantize -- quantize a row-major [rows][cols] matrix x to NVFP4
 * ([P4] "Architektura NVFP4 ..." for the format; [P3] "Warum weniger Bits
 * ..." for nearest rounding; [P4] "Technologie stabilizujace ..." for
 * stochastic rounding).
 *
 *  x        : device, x_dtype elements, row-major [rows][cols], 16-byte aligned.
 *  axis     : 1 -> outer = rows, k = cols (blocks run along rows of x);
 *             0 -> outer = cols, k = rows (blocks run down the columns of x;
 *             the output is the transpose, as needed for the K-major operand
 *             of a GEMM whose reduction runs over the rows of x).
 *  rounding : NVFP4_RNE (nearest, ties to the even code, saturate at 6) or
 *             NVFP4_SR (stochastic: with frac the position of |v| between
 *             its two neighbouring grid values, round up iff
 *             frac + (r16 + 1/2) / 2^16 >= 1, r16 being the 16 bits
 *             Philox4x32-10 assigns to the element; saturate at 6).
 *  seed, offset : Philox key = (lo32(seed), hi32(seed)); for the element with
 *             output index i = o*k + kk the counter is (lo32(i/8), hi32(i/8),
 *             lo32(offset), hi32(offset)) and r16 is half (i%2, low first) of
 *             output word (i%8)/2.  Ignored for NVFP4_RNE.
 *  out      : host struct; out->codes/scales/meta must point to buffers of
 *             the sizes above and out->outer, out->k must equal the view's.
 * Steps: amax over the whole tensor; s_enc = 2688/amax, per block
 * S = E4M3_rne_sat(blockmax * (448/amax)); element code of x * (s_enc / S).
 * amax == 0 gives all-zero scales and codes of +-0.  Non-finite input: meta[0]
 * becomes Inf/NaN and the codes and scales are unspecified.  An empty tensor
 * (outer == 0) writes meta = {0, 0} only.  Enqueues three kernels.
 */
int nvfp4_quantize(const void *x, int x_dtype, int64_t rows, int64_t cols, int axis,
                   int rounding, uint64_t seed, uint64_t offset, nvfp4_tensor *out,
                   void *hip_stream);

/*
 * nvfp4_rht_quantize -- as nvfp4_quantize, but each 16-element chunk along k
 * is first replaced by (1/4) H16 diag(s) chunk, the 16-point random Hadamard
 * transform ([P4] "Technologie stabilizujace ...": it spreads the outliers
 * of the weight gradients).  H16 is the Sylvester Hadamard matrix
 * H[i][j] = (-1)^popcount(i & j) and s_j = -1 where bit j of sign_mask is
 * set.  The butterfly runs in binary32 with stages 1, 2, 4, 8 (lower index
 * a+b, upper a-b).  amax and block maxima are those of the transformed
 * values.  Both operands of a weight-gradient GEMM must use the same
 * sign_mask along their shared reduction dimension; the transform then
 * cancels in the product.
 */
int nvfp4_rht_quantize(const void *x, int x_dtype, int64_t rows, int64_t cols, int axis,
                       int rounding, uint64_t seed, uint64_t offset, uint16_t sign_mask,
                       nvfp4_tensor *out, void *hip_stream);

/*
 * nvfp4_amax -- the first pass of a quantization alone: *amax = the tensor
 * amax of x viewed on `axis` (after the 16-point transform along k when
 * rht == 1, with sign_mask as in nvfp4_rht_quantize), the maximum of |value|
 * taken on IEEE bit patterns (exact; NaN > Inf > finite).  0 for an empty
 * tensor.  amax: device, one f32, 4-byte aligned.  Enqueues two kernels.
 *
 * nvfp4_quantize_amax -- the second pass alone: as nvfp4_quantize (rht == 0)
 * or nvfp4_rht_quantize (rht == 1) with the tensor amax read from device
 * memory instead of computed, which saves the first read of x when the
 * producer of x already knows its maximum ([P4] "Architektura NVFP4 ...":
 * the FP32 tensor-level scale).  out->meta becomes {*amax, *amax / 2688}.
 * *amax must be finite and >= 0 (not checked): with the true maximum the
 * result equals nvfp4_quantize's bit for bit; a smaller value saturates
 * (block scales at 448, codes at 6), so the decoded values are clipped to
 * +-*amax.  Non-finite input values leave the codes and scales unspecified,
 * as in nvfp4_quantize.  Enqueues two kernels.
 */
int nvfp4_amax(const void *x, int x_dtype, int64_t rows, int64_t cols, int axis, int rht,
               uint16_t sign_mask, float *amax, void *hip_stream);
int nvfp4_quantize_amax(const void *x, int x_dtype, int64_t rows, int64_t cols, int axis,
                        int rounding, uint64_t seed, uint64_t offset, int rht,
                        uint16_t sign_mask, const float *amax, nvfp4_tensor *out,
                        void *hip_stream);

/*
 * nvfp4_quantize_dual -- both layouts of one input with one amax read.  A
 * training step needs each of its tensors quantized along both of its
 * dimensions: dY along its columns for the data gradient and along its rows
 * for the weight gradient ([P4] "Technologie stabilizujace ...": stochastic
 * rounding of the gradients, the Hadamard transform for the weight
 * gradients).  Equivalent, bit for bit, to
 *   nvfp4_quantize(x, x_dtype, rows, cols, 1, rounding1, seed1, offset1, out1)
 * followed by nvfp4_quantize (rht0 == 0) or nvfp4_rht_quantize (rht0 == 1)
 * of x with axis 0, rounding0, seed0, offset0, sign_mask0 into out0, but
 * each of the two passes reads x once for both layouts: the amax pass takes
 * both maxima (the plain one, and the one after the column transform), the
 * encode pass writes both outputs from one tile of x staged in LDS.
 *  rows % 16 == 0 and cols % 16 == 0 (both layouts need whole blocks);
 *  out1: outer = rows, k = cols; out0: outer = cols, k = rows; the two meta
 *  pairs (8 bytes each) must not overlap (NVFP4_ERR_SHAPE otherwise) and the
 *  outputs must not overlap each other or x.  Enqueues three kernels.
 */
int nvfp4_quantize_dual(const void *x, int x_dtype, int64_t rows, int64_t cols,
                        int rounding1, uint64_t seed1, uint64_t offset1, nvfp4_tensor *out1,
                        int rht0, uint16_t sign_mask0, int rounding0, uint64_t seed0,
                        uint64_t offset0, nvfp4_tensor *out0, void *hip_stream);

/*
 * nvfp4_dequantize -- y[o][kk] = (e2m1(code) * e4m3(scale)) * g in binary32
 * (the first product is exact, the second rounds once); bf16 output is the
 * nearest-even rounding of that value.  y: device [q->outer][q->k] row-major
 * in the QUANTIZED layout (an axis-0 tensor comes back transposed), 16-byte
 * aligned.  Defines the values the GEMM multiplies ([P3] "Warum weniger Bits
 * ..." measures quantization error against these decoded values).
 */
int nvfp4_dequantize(const nvfp4_tensor *q, void *y, int y_dtype, void *hip_stream);

/*
 * nvfp4_gemm -- the block-scaled NVFP4 GEMM with FP32 accumulation
 * ([P1] body: accelerated 4-bit GEMMs; [P4] "Architektura NVFP4 ...").
 *
 *   C[m][n] = g_A * g_B * sum_k (qA*SA)[m][k] * (qB*SB)[n][k]
 *
 *  a : M x K NVFP4 tensor (a->outer = M), b : N x K (b->outer = N), a->k ==
 *      b->k.  Both operands are K-contiguous ("TN"): fprop Y = X W^T takes
 *      a = X (axis 1), b = W (axis 1); dgrad dX = dY W takes a = dY (axis 1),
 *      b = W quantized on axis 0; wgrad dW = X^T dY takes a = X (axis 0) and
 *      b = dY (axis 0).
 *  c : device, row-major [M][ldc], c_dtype NVFP4_F32 or NVFP4_BF16 (nearest
 *      even of the f32 result), ldc >= N, 4-byte aligned (f32) / 2-byte (bf16).
 * Accuracy: every decoded element q*S is exact in f16 and every product of
 * two is exact in f32.  Each MFMA adds one K step of 16 products -- 8 from
 * each of two different 16-blocks, with different block scales -- into the
 * f32 accumulator, so an output element goes through at least K/16 binary32
 * roundings and the worst-case error is of order
 * (K/16) * 2^-24 * g_A g_B sum_k |(qA SA)(qB SB)|: that guarantees the
 * 1e-5 * sum|ab| tolerance only up to K of about 2700.  Beyond, the
 * tolerance rests on successive rounding errors having independent signs
 * (error ~ sqrt(K/16) * 2^-24 * sum|ab|).  Measured worst |err| / sum|ab|:
 * zero-mean operands at the layer shapes (K = 5120 .. 20480) below 1e-6;
 * non-negative operands (the case where every partial sum grows) 2.5e-6 at
 * K = 20480, 6.9e-6 at K = 131072, and above the tolerance from K = 262144
 * (1.04e-5; 1.9e-4 at K = 2^25 - 256).  So for same-sign operands this call
 * meets 1e-5 for K <= 131072; nvfp4_gemm_ws splits long reductions of small
 * outputs (3.5e-7 at K = 2^25 - 256).
 * Deterministic: one kernel, no atomics, fixed summation order.  M == 0 or
 * N == 0: nothing is written; K == 0: C is set to zero.
 */
int nvfp4_gemm(const nvfp4_tensor *a, const nvfp4_tensor *b, void *c, int c_dtype,
               int64_t ldc, void *hip_stream);

/*
 * nvfp4_gemm_ws -- nvfp4_gemm with a caller-owned workspace, which lets it
 * balance the last, partly filled round of the CUs by splitting tiles along
 * K.  The data-parallel grid runs whole 256 x 256 output tiles, so when the
 * tile count is not a multiple of the CU count the last round leaves CUs
 * idle.  Two schedules use the workspace:
 *  - stream-K tail (at least one round of tiles, not a whole number of
 *    rounds, at least 4096 K positions per tile): all whole rounds but the
 *    last run data-parallel; the remaining tiles' K groups are dealt out in
 *    equal contiguous ranges to one round of workgroups, eight chunks (one
 *    per XCD) of whole tiles.  A tile is then the sum of at most two
 *    ranges: the workgroup holding its end adds the f32 partial of the one
 *    holding its start (kept in the workspace).
 *  - split tail (fewer tiles than one round): whole rounds run as before and
 *    each remaining tile is cut into up to CUs / tiles-left-over K ranges;
 *    the workgroup of the last range adds the others' partials.  Taken when
 *    fewer than half the CUs would get a tile or the ranges stay long (at
 *    least 4096 K positions).
 * Otherwise the call runs nvfp4_gemm's grid.  Partials add in a fixed order
 * -- deterministic for a given device, no atomics on the data.  Same
 * operands, output and accuracy contract as nvfp4_gemm; a split shortens
 * each f32 accumulation chain (the partials then add in binary32), which
 * keeps same-sign operands inside the tolerance at any K when the output
 * has few tiles.
 *  workspace       : device, at least nvfp4_gemm_workspace_bytes() bytes,
 *                    256-byte aligned, zero-filled before its FIRST use (the
 *                    kernel leaves it zero-filled again when it completes,
 *                    so it can be reused without clearing).  Calls that use
 *                    one workspace must not overlap in time (same stream,
 *                    or ordered by events).
 *  workspace_bytes : its size (NVFP4_ERR_SHAPE if smaller).
 * Errors as nvfp4_gemm, plus NVFP4_ERR_NULL for a NULL workspace and
 * NVFP4_ERR_ALIGN for a misaligned one.  Enqueues one kernel.
 */
int nvfp4_gemm_ws(const nvfp4_tensor *a, const nvfp4_tensor *b, void *c, int c_dtype,
                  int64_t ldc, void *workspace, int64_t workspace_bytes, void *hip_stream);

/*
 * nvfp4_gemm_noalloc -- nvfp4_gemm_ws with the library's own workspace, for
 * callers that cannot allocate device memory: code under HIP graph capture,
 * tight serving loops, harnesses that forbid allocation.  It allocates
 * nothing: the workspace is a file-scope device array of
 * nvfp4_gemm_workspace_bytes() bytes (64 MiB + 64 KiB), one per GPU the
 * library runs on, held until the process ends; its address is looked up
 * and its flags cleared (by a kernel on hip_stream) on the first call on
 * each device.  Same arguments, results and errors as nvfp4_gemm_ws without
 * the workspace; the output is bit-identical to nvfp4_gemm_ws's.  Every
 * call on one GPU shares that array, so calls that overlap in time on one
 * GPU race (use one stream, or order them); it keeps the last call's
 * partials.  Enqueues one kernel (two on the first call on a device).
 */
int nvfp4_gemm_noalloc(const nvfp4_tensor *a, const nvfp4_tensor *b, void *c, int c_dtype,
                       int64_t ldc, void *hip_stream);

/* Workspace bytes nvfp4_gemm_ws needs (the same for every shape: 64 KiB of
 * flags plus one 256 KiB partial per persistent workgroup, at most 256). */
int64_t nvfp4_gemm_workspace_bytes(void);

/*
 * MXFP4 -- the microscaling format the pages set NVFP4 against ([P4]
 * "Architektura NVFP4 kontra ograniczenia mikroskalowania": 32-element
 * blocks sharing a power-of-two scale; no tensor-level scale).
 *  codes  : u8 [outer][k/2], E2M1 codes two per byte (element 2j low
 *           nibble), 16-byte aligned.
 *  scales : u8 [outer][k/32], E8M0 exponents: the block scale is
 *           2^(code - 127).  4-byte aligned for a GEMM operand.
 *  outer, k : k % 32 == 0.
 * The value of element (o, kk) is e2m1(code) * 2^(scale - 127).
 */
typedef struct {
    uint8_t *codes;
    uint8_t *scales;
    int64_t outer;
    int64_t k;
} mxfp4_tensor;

/*
 * mxfp4_quantize -- x (row-major [rows][cols], x_dtype, 16-byte aligned)
 * viewed on `axis` as in nvfp4_quantize.  Per 32-block along k: the scale is
 * the smallest power of two 2^e with blockmax / 2^e <= 6 (e clamped to
 * [-127, 127]; an all-zero block takes e = -127), so the block maximum is
 * never clipped; each element is the nearest-even E2M1 code of x / 2^e.
 * Enqueues one kernel.
 */
int mxfp4_quantize(const void *x, int x_dtype, int64_t rows, int64_t cols, int axis,
                   mxfp4_tensor *out, void *hip_stream);

/*
 * mxfp4_gemm -- C[m][n] = sum_k (qA * 2^eA)[m][k] * (qB * 2^eB)[n][k] with
 * FP32 accumulation on gfx950's block-scaled FP4 MFMA (the codes are not
 * decoded).  a: M x K, b: N x K, both K-contiguous; K % 256 == 0
 * (NVFP4_ERR_SHAPE otherwise).  c: row-major [M][ldc], f32 or bf16 (nearest
 * even).  Accuracy as nvfp4_gemm: within 1e-5 * sum_k |a b|.  Deterministic.
 */
int mxfp4_gemm(const mxfp4_tensor *a, const mxfp4_tensor *b, void *c, int c_dtype,
               int64_t ldc, void *hip_stream);

/*
 * MXFP8 -- the 8-bit microscaling format, one of the three number formats
 * of a training run in [P3] "Drei Formate, ein Trainingslauf" (the one
 * quoted at about 5 PFLOPS on GB300), with the 32-element power-of-two
 * blocks of [P4] "Architektura NVFP4 kontra ograniczenia mikroskalowania".
 *  codes  : u8 [outer][k], OCP E4M3FN bytes (bias 7, max 448), 16-byte
 *           aligned.
 *  scales : u8 [outer][k/32], E8M0 exponents: the block scale is
 *           2^(code - 127).  4-byte aligned for a GEMM operand.
 *  outer, k : k % 32 == 0.
 * The value of element (o, kk) is e4m3(code) * 2^(scale - 127).
 */
typedef struct {
    uint8_t *codes;
    uint8_t *scales;
    int64_t outer;
    int64_t k;
} mxfp8_tensor;

/*
 * mxfp8_quantize -- x (row-major [rows][cols], x_dtype, 16-byte aligned)
 * viewed on `axis` as in nvfp4_quantize.  Per 32-block along k: the scale is
 * the smallest power of two 2^e with blockmax / 2^e <= 448 (e clamped to
 * [-127, 127]; an all-zero block takes e = -127), so the block maximum is
 * never clipped; each element is the nearest-even E4M3 code of x / 2^e with
 * the sign of x (-0.0 gives 0x80).  Axis 0 takes rows <= 8 388 480.
 * Enqueues one kernel.
 */
int mxfp8_quantize(const void *x, int x_dtype, int64_t rows, int64_t cols, int axis,
                   mxfp8_tensor *out, void *hip_stream);

/*
 * mxfp8_gemm -- C[m][n] = sum_k (qA * 2^eA)[m][k] * (qB * 2^eB)[n][k] with
 * FP32 accumulation on gfx950's block-scaled FP8 MFMA (the codes are not
 * decoded).  a: M x K, b: N x K, both K-contiguous; K % 128 == 0 and
 * K <= 2^24 - 128 (NVFP4_ERR_SHAPE otherwise).  c: row-major [M][ldc], f32
 * or bf16 (nearest even).  Accuracy: the instruction sums its 64 products
 * per step in groups of 8 consecutive K positions and truncates each
 * product toward zero to 13 bits below the group's largest exponent sum
 * (measured on MI355X), so an element can lose up to
 * sum over groups of sum_k min(|a_k b_k|, 2^(E_group - 13)) on top of the
 * binary32 accumulation of about K/64 steps; every element lies within
 * that bound plus 1e-5 * sum_k |a b| of the exact value.  Deterministic.
 */
int mxfp8_gemm(const mxfp8_tensor *a, const mxfp8_tensor *b, void *c, int c_dtype,
               int64_t ldc, void *hip_stream);

/*
 * nvfp4_layer_norm -- layer norm of every row of x, the norm in front of a
 * 4-bit linear layer:
 *   m = sum x / cols,  v = sum (x - m)^2 / cols,  r = 1 / sqrt(v + eps)
 *   y = (x - m) r weight + bias
 *  x         : device, row-major [rows][ldx], x_dtype, ldx >= cols >= 1 (at
 *              most 2^31 columns), aligned to its element only.
 *  weight,
 *  bias      : device, w_dtype [cols]; NULL = 1 and 0.
 *  eps       : >= 0 and finite (NVFP4_ERR_VALUE otherwise).
 *  y         : device, row-major [rows][ldy], y_dtype (bf16 = nearest even of
 *              the binary32 value, rounded once).
 *  mean,rstd : device, f32 [rows], m and r for the backward pass.
 *  amax      : device, f32 [1], or NULL.  The maximum |y| as stored (on IEEE
 *              bit patterns: NaN > Inf > finite; 0 when rows == 0), so that
 *              nvfp4_quantize_amax of y on axis 1 with it equals
 *              nvfp4_quantize bit for bit without the first read of y.
 *  workspace : device, with amax at least nvfp4_layer_norm_workspace_bytes
 *              (rows, cols) bytes (0 for a few rows), 4-byte aligned,
 *              contents ignored and overwritten; calls that share one must
 *              not overlap in time.  Unused (may be NULL) without amax.
 * All sums are binary32, the variance a sum of squared differences from the
 * mean.  A row's non-finite values reach that row only.  Outputs must not
 * overlap inputs (NVFP4_ERR_SHAPE for x and y; rows of both may lie side by
 * side in one buffer).  Deterministic.  Enqueues one kernel, two with amax (one for
 * a few rows).  The workspace size is NVFP4_ERR_SHAPE for sizes that the
 * call itself refuses.
 */
int nvfp4_layer_norm(const void *x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, const void *weight,
                     const void *bias, int w_dtype, float eps, void *y, int y_dtype, int64_t ldy, float *mean,
                     float *rstd, float *amax, void *workspace, int64_t workspace_bytes, void *hip_stream);
int64_t nvfp4_layer_norm_workspace_bytes(int64_t rows, int64_t cols);

/*
 * nvfp4_layer_norm_backward -- the gradients of nvfp4_layer_norm: with
 * a = dy weight and h = (x - mean) rstd,
 *   dx = rstd (a - sum(a) / cols - h sum(a h) / cols)     (x_dtype, [rows][lddx])
 *   dweight = sum over rows of dy h,  dbias = sum over rows of dy   (g_dtype, [cols])
 *  dx        : must not overlap dy or x (NVFP4_ERR_SHAPE).
 *  dweight,
 *  dbias     : either may be NULL; zeros when rows == 0.
 *  workspace : device, at least nvfp4_layer_norm_backward_workspace_bytes
 *              (rows, cols) bytes (0 for a few rows, NULL then allowed),
 *              16-byte aligned, contents ignored and overwritten; calls that share one must not overlap in time.
 * The sums over rows are binary32 partial sums of fixed sets of rows, added
 * in a fixed order: deterministic on one device.  The workspace size is
 * NVFP4_ERR_SHAPE for sizes that the call itself refuses.
 */
int nvfp4_layer_norm_backward(const void *dy, int dy_dtype, int64_t lddy, const void *x, int x_dtype, int64_t rows,
                              int64_t cols, int64_t ldx, const float *mean, const float *rstd, const void *weight,
                              int w_dtype, void *dx, int64_t lddx, void *dweight, void *dbias, int g_dtype,
                              void *workspace, int64_t workspace_bytes, void *hip_stream);
int64_t nvfp4_layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols);

/*
 * nvfp4_rms_norm -- root-mean-square norm of every row, after the addition of
 * the residual stream where there is one:
 *   h = x + residual,  r = 1 / sqrt(sum h^2 / cols + eps),  y = h weight r
 *  x         : device, row-major [rows][ldx], x_dtype, ldx >= cols >= 1 (at
 *              most 2^31 columns), aligned to its element only.
 *  residual  : device, row-major [rows][ldr], r_dtype, or NULL (h is x then).
 *  h         : device, row-major [rows][ldh], r_dtype: the sum, rounded to
 *              nearest even; what is normed is h as stored.  May be `residual`
 *              itself (same pointer and leading dimension).  Not used
 *              without a residual.
 *  weight    : device, w_dtype [cols]; NULL = 1.
 *  eps       : >= 0 and finite (NVFP4_ERR_VALUE otherwise).
 *  y         : device, row-major [rows][ldy], y_dtype (bf16 = nearest even of
 *              the binary32 value, rounded once).
 *  rstd      : device, f32 [rows], r for the backward pass.
 * Sums are binary32 (a row whose squares pass its range has r = 0).  A row's
 * non-finite values reach that row only.  Outputs must not overlap inputs or
 * each other (NVFP4_ERR_SHAPE; rows of two may lie side by side in one
 * buffer), but for h in the residual's place.  Deterministic.  Enqueues one
 * kernel.
 *
 * mxfp8_rms_norm -- the same with y in MXFP8: the codes and scales that
 * mxfp8_quantize forms, on axis 1, from the binary32 values (h weight) r where
 * these are finite; the operand of mxfp8_gemm.  cols % 32 == 0;
 * out->outer == rows, out->k == cols.
 */
int nvfp4_rms_norm(const void *x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, const void *residual,
                   int r_dtype, int64_t ldr, void *h, int64_t ldh, const void *weight, int w_dtype, float eps, void *y,
                   int y_dtype, int64_t ldy, float *rstd, void *hip_stream);
int mxfp8_rms_norm(const void *x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, const void *residual,
                   int r_dtype, int64_t ldr, void *h, int64_t ldh, const void *weight, int w_dtype, float eps,
                   mxfp8_tensor *out, float *rstd, void *hip_stream);

/*
 * nvfp4_rms_norm_backward -- the gradients of nvfp4_rms_norm: with
 * a = dy weight and n = h rstd,
 *   dx = rstd (a - n sum(a n) / cols) + dh                  (h_dtype, [rows][lddx])
 *   dweight = sum over rows of dy n                         (g_dtype, [cols])
 *  h         : what was normed, h_dtype.  dx is the gradient of x and of the
 *              residual alike.
 *  dh        : the gradient that reaches h from the residual stream, h_dtype,
 *              row-major [rows][lddh], or NULL (0).
 *  dx, dweight : must not overlap inputs or each other (NVFP4_ERR_SHAPE; rows
 *              of dx may lie in the gaps of dy, h or dh).  dweight may be
 *              NULL; zeros when rows == 0.
 *  workspace : device, at least nvfp4_rms_norm_backward_workspace_bytes
 *              (rows, cols) bytes (0 for a few rows, NULL then allowed),
 *              16-byte aligned, contents ignored and overwritten; calls that
 *              share one must not overlap in time.
 * The sums over rows are binary32 partial sums of fixed sets of rows, added
 * in a fixed order: deterministic on one device.  The workspace size is
 * NVFP4_ERR_SHAPE for sizes that the call itself refuses.
 */
int nvfp4_rms_norm_backward(const void *dy, int dy_dtype, int64_t lddy, const void *h, int h_dtype, int64_t rows,
                            int64_t cols, int64_t ldh, const float *rstd, const void *weight, int w_dtype,
                            const void *dh, int64_t lddh, void *dx, int64_t lddx, void *dweight, int g_dtype,
                            void *workspace, int64_t workspace_bytes, void *hip_stream);
int64_t nvfp4_rms_norm_backward_workspace_bytes(int64_t rows, int64_t cols);

/*
 * nvfp4_matvec, mxfp4_matvec -- a few rows of unquantized activations times
 * a 4-bit weight matrix, the single-token form of the linear layer:
 *   y[t][n] = g sum_k x[t][k] e2m1(code[n][k]) e4m3(scale[n][k/16])       (NVFP4)
 *   y[t][n] =   sum_k x[t][k] e2m1(code[n][k]) 2^(scale[n][k/32] - 127)   (MXFP4)
 *  w      : the weights [outer = N][k], quantized on axis 1 (W [out, in]).
 *  x      : device, row-major [tokens][ldx], x_dtype, ldx >= k, aligned to
 *           its element only.
 *  y      : device, row-major [tokens][ldy], y_dtype, ldy >= N; must not
 *           overlap x (NVFP4_ERR_SHAPE; their rows may lie side by side).
 *  tokens : made for 1 to 16 (the weights are read once for every 16);
 *           at most 1 048 560.  N <= 16 * INT32_MAX, k <= 2^25 - 16.
 *  workspace : device, at least nvfp4_matvec_workspace_bytes(N, k, tokens,
 *           x_dtype) bytes (for both formats), 16-byte aligned, contents
 *           ignored and overwritten; often 0, and NULL will do then.  Calls
 *           that share one must not overlap in time.
 * An MXFP4 scale of 255 is E8M0's NaN and makes its row NaN.
 * Weights and bf16 x enter the product exactly; a float32 x to within
 * 2^-133 of its value.  Sums are binary32.  k == 0 gives zeros.
 * Deterministic on one device.  Enqueues one kernel, or two where there is a
 * workspace.  The workspace size is NVFP4_ERR_SHAPE / NVFP4_ERR_ENUM for
 * arguments that the calls refuse.
 */
int nvfp4_matvec(const nvfp4_tensor *w, const void *x, int x_dtype, int64_t tokens, int64_t ldx, void *y, int y_dtype,
                 int64_t ldy, void *workspace, int64_t workspace_bytes, void *hip_stream);
int mxfp4_matvec(const mxfp4_tensor *w, const void *x, int x_dtype, int64_t tokens, int64_t ldx, void *y, int y_dtype,
                 int64_t ldy, void *workspace, int64_t workspace_bytes, void *hip_stream);
int64_t nvfp4_matvec_workspace_bytes(int64_t n, int64_t k, int64_t tokens, int x_dtype);

/*
 * nvfp4_grouped_matmul, mxfp4_grouped_matmul -- matrix products grouped by
 * expert: rows of unquantized activations in ragged groups, each with its own
 * 4-bit weights (as nvfp4_matvec's), the layers of a mixture of experts:
 *   y[t][n] = sum_k x[t][k] W_e[n][k]   for offsets[e] <= t < offsets[e + 1]
 *  w       : the stack of all experts' weights, one tensor: with transposed
 *            == 0 [outer = experts * N][k = K], expert after expert; with
 *            transposed == 1 [outer = N][k = experts * K], expert e's columns
 *            from e * K on, as the quantizers write the stack [experts * K][N]
 *            on axis 0 -- the form for the data gradient dx = dy W.
 *            K % 16 == 0 (MXFP4: 32).
 *  x       : device, row-major [rows][ldx], x_dtype, ldx >= K, aligned to its
 *            element only.
 *  offsets : device, int32 or int64 (index_bits 32 or 64), [experts + 1],
 *            not decreasing, 0 <= offsets[0] and offsets[experts] <= rows.
 *            Not checked; values outside are taken as the nearest inside, and
 *            where they decrease the result is unspecified (nothing outside
 *            x and y is touched).  experts: 1 .. 2^20.
 *  y       : device, row-major [rows][ldy], y_dtype, ldy >= N; must not
 *            overlap x (NVFP4_ERR_SHAPE; their rows may lie side by side).
 *  zero_rest : 0: rows of y that belong to no group are left as they are;
 *            1: they become zeros.
 *  workspace : device, at least nvfp4_grouped_matmul_workspace_bytes(experts,
 *            N, K, rows, x_dtype) bytes (for both formats), 16-byte aligned,
 *            contents ignored and overwritten; may be 0, and NULL will do then.
 *            Calls that share one must not overlap in time.
 *  ceil(N / 128) * (rows / 32 + min(experts, rows)) <= 2^24 - 8, K <= 2^25 - 16,
 *  w's k <= 2^28 - 32.
 * A group without rows costs nothing, and its weights are not read.  Weights
 * and bf16 x enter the product exactly; a float32 x to within 2^-133 of its
 * value.  Sums are binary32.  K == 0 gives zeros.  An MXFP4 scale of 255 is
 * NaN.  Deterministic on one device.  Enqueues one kernel, or two where there
 * is a workspace.
 *
 * nvfp4_grouped_wgrad -- the gradient of the experts' weights,
 *   dw[e][n][k] = sum over offsets[e] <= t < offsets[e + 1] of dy[t][n] x[t][k]
 *  dw        : device, dw_dtype [experts][n][k], written whole (zeros for a
 *              group without rows); must not overlap dy or x.
 *  workspace : device, at least nvfp4_grouped_wgrad_workspace_bytes(experts, n,
 *              k, rows, dy_dtype, x_dtype) bytes, 16-byte aligned, contents
 *              ignored and overwritten.  Calls that share one must not overlap
 *              in time.
 *  n, k <= 2^25 - 16, experts * (ceil(n / 128) * ceil(k / 128) + 7) <= 2^24 - 8.
 * bf16 products are exact; with a float32 operand products are off by at most
 * 2^-23 of their magnitude, and those with an infinity are infinite or NaN.
 * Sums are binary32, in a fixed order: deterministic on one device.  Enqueues
 * one kernel, one more for the operands that are float32 and one for bf16 ones
 * not of whole words (an odd number of columns, rows at odd places), and one
 * where few tiles share long groups.
 */
int nvfp4_grouped_matmul(const nvfp4_tensor *w, int transposed, const void *x, int x_dtype, int64_t rows, int64_t ldx,
                         const void *offsets, int index_bits, int64_t experts, void *y, int y_dtype, int64_t ldy,
                         int zero_rest, void *workspace, int64_t workspace_bytes, void *hip_stream);
int mxfp4_grouped_matmul(const mxfp4_tensor *w, int transposed, const void *x, int x_dtype, int64_t rows, int64_t ldx,
                         const void *offsets, int index_bits, int64_t experts, void *y, int y_dtype, int64_t ldy,
                         int zero_rest, void *workspace, int64_t workspace_bytes, void *hip_stream);
int64_t nvfp4_grouped_matmul_workspace_bytes(int64_t experts, int64_t n, int64_t k, int64_t rows, int x_dtype);
int nvfp4_grouped_wgrad(const void *dy, int dy_dtype, int64_t lddy, const void *x, int x_dtype, int64_t ldx,
                        int64_t rows, int64_t n, int64_t k, const void *offsets, int index_bits, int64_t experts,
                        void *dw, int dw_dtype, void *workspace, int64_t workspace_bytes, void *hip_stream);
int64_t nvfp4_grouped_wgrad_workspace_bytes(int64_t experts, int64_t n, int64_t k, int64_t rows, int dy_dtype,
                                            int x_dtype);

/*
 * nvfp4_adapters -- low-rank adapters of many requests at once, beside a
 * projection that they share (its weights 4-bit and frozen, say, its result
 * from nvfp4_matvec or nvfp4_gemm):
 *   u[t] = A_a x[t],   y[t] = base[t] + scale_a B_a u[t]
 * for the rows offsets[i] <= t < offsets[i + 1] of segment i (a request) and
 * its adapter a = index[i].
 *  x       : device, row-major [rows][ldx], x_dtype, ldx >= k, aligned to its
 *            element only.
 *  a, b    : device, w_dtype, contiguous: a [adapters][rank][k],
 *            b [adapters][n][rank].  1 <= rank <= 128, 1 <= adapters <= 65535.
 *            Adapters of a smaller rank are filled up with zeros.
 *  scale   : device, f32 [adapters]; NULL = 1.
 *  offsets : device, [segments + 1] of int32 or int64 (index_bits 32 or 64),
 *            not decreasing, 0 <= offsets[0] and offsets[segments] <= rows.
 *            Not checked; values outside are taken as the nearest inside, and
 *            where they decrease the result is unspecified (nothing outside
 *            the outputs is written).  1 <= segments <= 2^20.
 *  index   : device, [segments], of the same type.  A segment whose index lies
 *            outside [0, adapters) (-1, say) has no adapter.
 *  base    : device, row-major [rows][ldb], base_dtype, or NULL (zeros).
 *  y       : device, row-major [rows][ldy], y_dtype, written whole: rows
 *            without an adapter (those of no segment too) are base.  May be
 *            `base` itself (same pointer, type and leading dimension).
 *  u       : device, f32 [rows][rank], written whole (zeros without an
 *            adapter), for the backward pass.
 *  ceil(max(n, k) / 256) * (rows / 16 + min(segments + 2, rows)) <= 2^24 - 8.
 * Outputs must not overlap inputs or each other (NVFP4_ERR_SHAPE), but for y
 * in base's place.
 * bf16 operands enter the products exactly; a product of two float32 values
 * is off by at most 2^-23 of its magnitude, and one with an infinity infinite
 * or NaN.  Sums are binary32.  Deterministic.  Enqueues two kernels.
 *
 * nvfp4_adapters_backward -- with g[t] = scale_a B_a^T dy[t]:
 *   dx[t] = base[t] + A_a^T g[t]                             (dx_dtype)
 *   da[a] = sum of g[t] x[t]^T, db[a] = scale_a sum of dy[t] u[t]^T
 * over the rows of all segments of adapter a (g_dtype, zeros for an adapter
 * that no segment has).  base is what the shared projection gives, dx written
 * whole as y is above.  u: the forward call's.
 *  workspace : device, at least nvfp4_adapters_backward_workspace_bytes(rows,
 *            n, k, rank, adapters, segments, w_dtype) bytes, 16-byte aligned,
 *            contents ignored and overwritten; calls that share one must not
 *            overlap in time.
 * Outputs must not overlap inputs or each other (NVFP4_ERR_SHAPE), but for dx
 * in base's place.  Sums over rows are binary32, in a fixed order:
 * deterministic on one device.
 */
int nvfp4_adapters(const void *x, int x_dtype, int64_t rows, int64_t k, int64_t ldx, const void *a, const void *b,
                   int w_dtype, int64_t adapters, int64_t rank, int64_t n, const float *scale, const void *offsets,
                   const void *index, int index_bits, int64_t segments, const void *base, int base_dtype, int64_t ldb,
                   void *y, int y_dtype, int64_t ldy, float *u, void *hip_stream);
int nvfp4_adapters_backward(const void *dy, int dy_dtype, int64_t lddy, const void *x, int x_dtype, int64_t rows,
                            int64_t k, int64_t ldx, const float *u, const void *a, const void *b, int w_dtype,
                            int64_t adapters, int64_t rank, int64_t n, const float *scale, const void *offsets,
                            const void *index, int index_bits, int64_t segments, const void *base, int base_dtype,
                            int64_t ldb, void *dx, int dx_dtype, int64_t lddx, void *da, void *db, int g_dtype,
                            void *workspace, int64_t workspace_bytes, void *hip_stream);
int64_t nvfp4_adapters_backward_workspace_bytes(int64_t rows, int64_t n, int64_t k, int64_t rank, int64_t adapters,
                                                int64_t segments, int w_dtype);

/*
 * nvfp4_distill_topk -- the distillation loss of a student's logits against
 * a teacher's best logits, by which a model brought to 4 bits is trained:
 *   p    = softmax(teacher / temperature) over the row's valid entries
 *   lse  = log sum_v exp(logits_v / temperature)
 *   loss = temperature^2 sum_k p_k (log p_k - (logits_{i_k} / temperature - lse))
 *  logits  : device, row-major [tokens][ldz], z_dtype, ldz >= vocab,
 *            1 <= vocab <= INT32_MAX, aligned to its element only.
 *  indices : device, [tokens][top] of int32 or int64 (index_bits 32 or 64):
 *            vocabulary indices i_k.  An entry is valid when its index lies
 *            in [0, vocab) and its teacher logit is above -infinity; shorter
 *            lists are filled up with -1.  0 <= top <= 1024.
 *  teacher : device, t_dtype [tokens][top].
 *  temperature : at least 2^-126 and finite (NVFP4_ERR_VALUE otherwise).
 *  loss, lse   : device, f32 [tokens].
 *  workspace   : device, nvfp4_distill_topk_workspace_bytes(tokens, vocab)
 *                bytes, 16-byte aligned, contents ignored and overwritten;
 *                0 for short rows, and NULL will do then.  Calls that share
 *                one must not overlap in time.
 * A row without a valid entry has loss 0 and gradient 0 whatever its logits.
 * An index listed twice counts twice.  Logits of -infinity or of the type's
 * lowest value are ordinary (a vocabulary mask); lse of a row of nothing but
 * -infinity is -infinity.
 *
 * nvfp4_distill_topk_backward -- the gradient of sum_t dloss_t loss_t, from
 * the lse of the forward call:
 *   dlogits_v = dloss temperature (exp(logits_v / temperature - lse) - sum_{k: i_k = v} p_k)
 *  dlogits : device, z_dtype, row-major [tokens][lddz]; must not overlap
 *            logits (NVFP4_ERR_SHAPE).
 *  Rows with dloss == 0 get zeros.  lse in binary32 leaves the shares a
 *  relative error of |lse| 2^-23; from |lse| = 4096 on (a row that lies as a
 *  whole at a mask's value) the call reads such a row once more and forms its
 *  log-sum-exp anew, also where lse has overflowed.
 *
 * nvfp4_distill_topk_step -- both in one call, for a program that knows its
 * rows' weights beforehand: loss and lse as above and dlogits with
 * dloss = weight.
 * Deterministic.  Sums are binary32.
 */
int nvfp4_distill_topk(const void *logits, int z_dtype, int64_t tokens, int64_t vocab, int64_t ldz,
                       const void *indices, int index_bits, const void *teacher, int t_dtype, int64_t top,
                       float temperature, float *loss, float *lse, void *workspace, int64_t workspace_bytes,
                       void *hip_stream);
int nvfp4_distill_topk_backward(const void *logits, int z_dtype, int64_t tokens, int64_t vocab, int64_t ldz,
                                const void *indices, int index_bits, const void *teacher, int t_dtype, int64_t top,
                                float temperature, const float *lse, const float *dloss, void *dlogits, int64_t lddz,
                                void *hip_stream);
int nvfp4_distill_topk_step(const void *logits, int z_dtype, int64_t tokens, int64_t vocab, int64_t ldz,
                            const void *indices, int index_bits, const void *teacher, int t_dtype, int64_t top,
                            float temperature, const float *weight, float *loss, float *lse, void *dlogits,
                            int64_t lddz, void *workspace, int64_t workspace_bytes, void *hip_stream);
int64_t nvfp4_distill_topk_workspace_bytes(int64_t tokens, int64_t vocab);

/*
 * nvfp4_probe_mfma -- measurement helper, not part of the method: launches
 * 1024 workgroups of 256 threads that run `iters` x 32 v_mfma_f32_32x32x16_f16
 * per wave (one wave per SIMD, sixteen accumulators) on operands with the
 * values the NVFP4 GEMM multiplies (E2M1 codes times E4M3 block scales), with
 * no memory traffic, giving the ceiling of that MFMA on that data.  Work:
 * 1024 * 4 * iters * 32 * 32768 flop.  out: device, 1024 * 256 floats (the
 * per-thread sums, which keep the work live).
 */
int nvfp4_probe_mfma(int64_t iters, float *out, void *hip_stream);

/*
 * nvfp4_probe_philox -- measurement helper, not part of the method: runs the
 * stochastic-rounding random generator alone (Philox4x32-10, the same
 * routine the encodes use, counters 0 .. calls-1, one call per 8 elements)
 * with no memory traffic, over 4096 workgroups of 256 threads, giving the
 * floor the RNG contract puts under a stochastic-rounding encode of
 * 8 * calls elements.  out: device, 4096 * 256 words (per-thread XOR of the
 * outputs, which keeps the work live).
 */
int nvfp4_probe_philox(int64_t calls, uint32_t *out, void *hip_stream);

/* Human-readable name of a status code (static string). */
const char *nvfp4_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_H */
