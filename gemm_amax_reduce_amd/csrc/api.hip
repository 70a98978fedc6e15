// api.hip -- the extern "C" boundary declared in include/nvfp4.h: argument
// validation (synchronous, before any launch) and kernel launches on the
// caller's stream.  Nothing here allocates or synchronises.
#include "nvfp4.h"
#include "nvfp4_kernels.h"

#include <float.h>
#include <stdint.h>

namespace {

// Size limits of the launch geometry (each documented in nvfp4.h).
// Quantization down the columns (axis 0) puts 16-row blocks on the grid's
// y dimension (at most 65535): 4 blocks per y step for NVFP4, 8 x 32 rows
// for MXFP4.
constexpr int64_t kMaxRowsAxis0 = 65535LL * 4 * 16;       // 4 194 240
constexpr int64_t kMaxRowsAxis0Mx = 65535LL * 8 * 32;     // 16 776 960
constexpr int64_t kMaxRowsAxis0Mx8 = 65535LL * 4 * 32;    // 8 388 480
// The MXFP8 GEMM addresses 128 operand rows of K code bytes with 32-bit
// buffer offsets below 2^31.
constexpr int64_t kMaxGemmKMx8 = (1LL << 24) - 128;
// The GEMMs address 128 operand rows of K/2 code bytes with 32-bit buffer
// offsets below 2^31, and launch at most INT32_MAX workgroups (tiles of
// 256 x 128 or larger).
constexpr int64_t kMaxGemmK = (1LL << 25) - 16;
// Element counts (rows x cols, outer x k, M x ldc) stay at or below 2^60, so
// every byte offset the kernels form fits in int64.
constexpr int64_t kMaxCount = 1LL << 60;

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline bool count_ok(int64_t a, int64_t b) { return a <= 0 || b <= kMaxCount / a; }

inline bool gemm_shape_ok(int64_t M, int64_t N, int64_t K) {
  if (K > kMaxGemmK) return false;
  // ceil(M/256) * ceil(N/128) <= INT32_MAX, without overflow
  const int64_t tm = M / 256 + (M % 256 != 0), tn = N / 128 + (N % 128 != 0);
  return tn == 0 || tm <= INT32_MAX / tn;
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP; }

int check_tensor(const nvfp4_tensor *t) {
  if (!t || !t->meta) return NVFP4_ERR_NULL;
  if (t->outer < 0 || t->k < 0 || t->k % 16 != 0 || !count_ok(t->outer, t->k)) return NVFP4_ERR_SHAPE;
  if (t->outer > 0 && t->k > 0 && (!t->codes || !t->scales)) return NVFP4_ERR_NULL;
  if (!aligned(t->codes, 8) || !aligned(t->meta, 4)) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

// Operands and output of an NVFP4 GEMM (shared by its entry points).
int check_gemm_args(const nvfp4_tensor *a, const nvfp4_tensor *b, const void *c, int c_dtype, int64_t ldc) {
  int st = check_tensor(a);
  if (st != NVFP4_OK) return st;
  st = check_tensor(b);
  if (st != NVFP4_OK) return st;
  if (c_dtype != NVFP4_F32 && c_dtype != NVFP4_BF16) return NVFP4_ERR_ENUM;
  if (a->k != b->k) return NVFP4_ERR_SHAPE;
  const int64_t M = a->outer, N = b->outer;
  if (ldc < N || !count_ok(M, ldc) || !gemm_shape_ok(M, N, a->k)) return NVFP4_ERR_SHAPE;
  if (M > 0 && N > 0 && !c) return NVFP4_ERR_NULL;
  if (!aligned(c, c_dtype == NVFP4_F32 ? 4 : 2)) return NVFP4_ERR_ALIGN;
  // with K % 64 == 0 the kernels move the scale rows by DMA in whole dwords
  if (a->k % 64 == 0 && (!aligned(a->scales, 4) || !aligned(b->scales, 4))) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

int quantize_common(const void *x, int x_dtype, int64_t rows, int64_t cols, int axis, int rounding,
                    uint64_t seed, uint64_t offset, bool rht, uint32_t sign_mask, nvfp4_tensor *out,
                    void *hip_stream) {
  if (!out) return NVFP4_ERR_NULL;
  if (x_dtype != NVFP4_F32 && x_dtype != NVFP4_BF16) return NVFP4_ERR_ENUM;
  if (rounding != NVFP4_RNE && rounding != NVFP4_SR) return NVFP4_ERR_ENUM;
  if (axis != 0 && axis != 1) return NVFP4_ERR_ENUM;
  if (rows < 0 || cols < 0 || !count_ok(rows, cols)) return NVFP4_ERR_SHAPE;
  const int64_t outer = axis ? rows : cols;
  const int64_t k = axis ? cols : rows;
  if (k % 16 != 0) return NVFP4_ERR_SHAPE;
  if (out->outer != outer || out->k != k) return NVFP4_ERR_SHAPE;
  if (axis == 0 && rows > kMaxRowsAxis0) return NVFP4_ERR_SHAPE;
  if (rows > 0 && cols > 0 && !x) return NVFP4_ERR_NULL;
  int st = check_tensor(out);
  if (st != NVFP4_OK) return st;
  if (!aligned(x, 16)) return NVFP4_ERR_ALIGN;
  hipError_t e = nvfp4::launch_quantize(x, x_dtype, rows, cols, axis, rounding, seed, offset, rht, sign_mask,
                                        out->codes, out->scales, out->meta, (hipStream_t)hip_stream);
  return hip_status(e);
}

inline bool dtype_ok(int d) { return d == NVFP4_F32 || d == NVFP4_BF16; }
inline uintptr_t dtype_size(int d) { return d == NVFP4_F32 ? 4 : 2; }

// A row-major [rows][ld] matrix of `cols` used columns: size and leading
// dimension.
inline bool matrix_ok(int64_t rows, int64_t cols, int64_t ld) {
  return rows >= 0 && cols >= 0 && ld >= cols && count_ok(rows, ld);
}

// Do the used bytes of two matrices of `rows` rows meet?  pitch: bytes from
// row to row, used: those of a row that are its own.  (Matrices of one pitch
// may lie side by side, each in the other's gaps; of two pitches that meet
// as a whole no two are told apart.)
inline bool overlap(const void *a, int64_t pitch_a, int64_t used_a, const void *b, int64_t pitch_b, int64_t used_b,
                    int64_t rows) {
  if (rows <= 0 || used_a <= 0 || used_b <= 0) return false;
  const uintptr_t a0 = (uintptr_t)a, a1 = a0 + (uintptr_t)((rows - 1) * pitch_a + used_a);
  const uintptr_t b0 = (uintptr_t)b, b1 = b0 + (uintptr_t)((rows - 1) * pitch_b + used_b);
  if (a0 >= b1 || b0 >= a1) return false;
  if (rows == 1 || pitch_a != pitch_b) return true;
  const int64_t d = ((int64_t)(b0 - a0) % pitch_a + pitch_a) % pitch_a;      // b's rows start there in a's
  return d < used_a || d + used_b > pitch_a;
}

// The widest row layer norm takes (grids over its columns stay far inside 2^31
// workgroups, and are launched in parts where their threads would pass 2^32).
constexpr int64_t kMaxNormCols = 1LL << 31;
// The matvec puts at least 16 weight rows on the grid's x dimension and 16
// tokens on its y dimension; its offsets inside 64 weight rows are 32-bit,
// as in the GEMMs (kMaxGemmK).
constexpr int64_t kMaxMatvecRows = (int64_t)INT32_MAX * 16;
constexpr int64_t kMaxMatvecTokens = 65535LL * 16;
// The distillation kernels keep vocabulary indices in 32 bits.
constexpr int64_t kMaxVocab = INT32_MAX;

int matvec_common(bool mx, const uint8_t *codes, const uint8_t *scales, const float *meta, int64_t N, int64_t K,
                  const void *x, int x_dtype, int64_t tokens, int64_t ldx, void *y, int y_dtype, int64_t ldy,
                  void *workspace, int64_t workspace_bytes, void *hip_stream) {
  if (!dtype_ok(x_dtype) || !dtype_ok(y_dtype)) return NVFP4_ERR_ENUM;
  if (!matrix_ok(tokens, K, ldx) || !matrix_ok(tokens, N, ldy)) return NVFP4_ERR_SHAPE;
  if (N > kMaxMatvecRows || tokens > kMaxMatvecTokens || K > kMaxGemmK) return NVFP4_ERR_SHAPE;
  if (tokens > 0 && N > 0 && (!y || (K > 0 && !x))) return NVFP4_ERR_NULL;
  const int64_t need = nvfp4::matvec_workspace_bytes(N, K, tokens, x_dtype == NVFP4_F32);
  if (workspace_bytes < need) return NVFP4_ERR_SHAPE;
  if (need > 0 && !workspace) return NVFP4_ERR_NULL;
  if (!aligned(x, dtype_size(x_dtype)) || !aligned(y, dtype_size(y_dtype)) || !aligned(workspace, 16))
    return NVFP4_ERR_ALIGN;
  const int64_t xs = dtype_size(x_dtype), ys = dtype_size(y_dtype);
  if (overlap(x, ldx * xs, K * xs, y, ldy * ys, N * ys, tokens)) return NVFP4_ERR_SHAPE;
  return hip_status(nvfp4::launch_matvec(mx, codes, scales, meta, N, K, x, x_dtype, tokens, ldx, y, y_dtype, ldy,
                                         workspace, (hipStream_t)hip_stream));
}

// The arguments that the three distillation calls share.
int check_distill(const void *z, int z_dtype, int64_t tokens, int64_t vocab, int64_t ldz, const void *indices,
                  int index_bits, const void *teacher, int t_dtype, int64_t top, float tau, const float *lse) {
  if (!dtype_ok(z_dtype) || !dtype_ok(t_dtype) || (index_bits != 32 && index_bits != 64)) return NVFP4_ERR_ENUM;
  if (vocab < 1 || vocab > kMaxVocab || !matrix_ok(tokens, vocab, ldz)) return NVFP4_ERR_SHAPE;
  if (top < 0 || top > nvfp4::distill_max_top() || !count_ok(tokens, top)) return NVFP4_ERR_SHAPE;
  if (!(tau >= FLT_MIN) || tau > 3.0e38f) return NVFP4_ERR_VALUE;      // (log2(e) / tau stays finite)
  if (tokens > 0 && (!z || !lse || (top > 0 && (!indices || !teacher)))) return NVFP4_ERR_NULL;
  if (!aligned(z, dtype_size(z_dtype)) || !aligned(teacher, dtype_size(t_dtype)) || !aligned(lse, 4) ||
      !aligned(indices, index_bits / 8))
    return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

}  // namespace

extern "C" {

int nvfp4_quantize(const void *x, int x_dtype, int64_t rows, int64_t cols, int axis, int rounding, uint64_t seed,
                   uint64_t offset, nvfp4_tensor *out, void *hip_stream) {
  return quantize_common(x, x_dtype, rows, cols, axis, rounding, seed, offset, false, 0u, out, hip_stream);
}

int nvfp4_rht_quantize(const void *x, int x_dtype, int64_t rows, int64_t cols, int axis, int rounding,
                       uint64_t seed, uint64_t offset, uint16_t sign_mask, nvfp4_tensor *out, void *hip_stream) {
  return quantize_common(x, x_dtype, rows, cols, axis, rounding, seed, offset, true, sign_mask, out, hip_stream);
}

int nvfp4_amax(const void *x, int x_dtype, int64_t rows, int64_t cols, int axis, int rht, uint16_t sign_mask,
               float *amax, void *hip_stream) {
  if (!amax) return NVFP4_ERR_NULL;
  if (x_dtype != NVFP4_F32 && x_dtype != NVFP4_BF16) return NVFP4_ERR_ENUM;
  if (axis != 0 && axis != 1) return NVFP4_ERR_ENUM;
  if (rht != 0 && rht != 1) return NVFP4_ERR_ENUM;
  if (rows < 0 || cols < 0 || !count_ok(rows, cols)) return NVFP4_ERR_SHAPE;
  if ((axis ? cols : rows) % 16 != 0) return NVFP4_ERR_SHAPE;
  if (axis == 0 && rows > kMaxRowsAxis0) return NVFP4_ERR_SHAPE;
  if (rows > 0 && cols > 0 && !x) return NVFP4_ERR_NULL;
  if (!aligned(x, 16) || !aligned(amax, 4)) return NVFP4_ERR_ALIGN;
  return hip_status(nvfp4::launch_amax(x, x_dtype, rows, cols, axis, rht != 0, sign_mask, amax,
                                       (hipStream_t)hip_stream));
}

int nvfp4_quantize_amax(const void *x, int x_dtype, int64_t rows, int64_t cols, int axis, int rounding,
                        uint64_t seed, uint64_t offset, int rht, uint16_t sign_mask, const float *amax,
                        nvfp4_tensor *out, void *hip_stream) {
  if (!out || !amax) return NVFP4_ERR_NULL;
  if (x_dtype != NVFP4_F32 && x_dtype != NVFP4_BF16) return NVFP4_ERR_ENUM;
  if (rounding != NVFP4_RNE && rounding != NVFP4_SR) return NVFP4_ERR_ENUM;
  if (axis != 0 && axis != 1) return NVFP4_ERR_ENUM;
  if (rht != 0 && rht != 1) return NVFP4_ERR_ENUM;
  if (rows < 0 || cols < 0 || !count_ok(rows, cols)) return NVFP4_ERR_SHAPE;
  const int64_t outer = axis ? rows : cols;
  const int64_t k = axis ? cols : rows;
  if (k % 16 != 0) return NVFP4_ERR_SHAPE;
  if (out->outer != outer || out->k != k) return NVFP4_ERR_SHAPE;
  if (axis == 0 && rows > kMaxRowsAxis0) return NVFP4_ERR_SHAPE;
  if (rows > 0 && cols > 0 && !x) return NVFP4_ERR_NULL;
  int st = check_tensor(out);
  if (st != NVFP4_OK) return st;
  if (!aligned(x, 16) || !aligned(amax, 4)) return NVFP4_ERR_ALIGN;
  return hip_status(nvfp4::launch_quantize_amax(x, x_dtype, rows, cols, axis, rounding, seed, offset, rht != 0,
                                                sign_mask, amax, out->codes, out->scales, out->meta,
                                                (hipStream_t)hip_stream));
}

int nvfp4_quantize_dual(const void *x, int x_dtype, int64_t rows, int64_t cols, int rounding1, uint64_t seed1,
                        uint64_t offset1, nvfp4_tensor *out1, int rht0, uint16_t sign_mask0, int rounding0,
                        uint64_t seed0, uint64_t offset0, nvfp4_tensor *out0, void *hip_stream) {
  if (!out1 || !out0) return NVFP4_ERR_NULL;
  if (x_dtype != NVFP4_F32 && x_dtype != NVFP4_BF16) return NVFP4_ERR_ENUM;
  if ((rounding1 != NVFP4_RNE && rounding1 != NVFP4_SR) || (rounding0 != NVFP4_RNE && rounding0 != NVFP4_SR))
    return NVFP4_ERR_ENUM;
  if (rht0 != 0 && rht0 != 1) return NVFP4_ERR_ENUM;
  if (rows < 0 || cols < 0 || rows % 16 != 0 || cols % 16 != 0 || !count_ok(rows, cols)) return NVFP4_ERR_SHAPE;
  if (out1->outer != rows || out1->k != cols || out0->outer != cols || out0->k != rows) return NVFP4_ERR_SHAPE;
  if (rows > kMaxRowsAxis0) return NVFP4_ERR_SHAPE;
  if (rows > 0 && cols > 0 && !x) return NVFP4_ERR_NULL;
  int st = check_tensor(out1);
  if (st != NVFP4_OK) return st;
  st = check_tensor(out0);
  if (st != NVFP4_OK) return st;
  // each meta is two floats that the kernels write while other workgroups
  // read them: the two 8-byte ranges must not overlap
  if (out1->meta + 2 > out0->meta && out0->meta + 2 > out1->meta) return NVFP4_ERR_SHAPE;
  if (!aligned(x, 16)) return NVFP4_ERR_ALIGN;
  return hip_status(nvfp4::launch_quantize_dual(x, x_dtype, rows, cols, rounding1, seed1, offset1, out1->codes,
                                                out1->scales, out1->meta, rht0 != 0, sign_mask0, rounding0, seed0,
                                                offset0, out0->codes, out0->scales, out0->meta,
                                                (hipStream_t)hip_stream));
}

int mxfp4_quantize(const void *x, int x_dtype, int64_t rows, int64_t cols, int axis, mxfp4_tensor *out,
                   void *hip_stream) {
  if (!out) return NVFP4_ERR_NULL;
  if (x_dtype != NVFP4_F32 && x_dtype != NVFP4_BF16) return NVFP4_ERR_ENUM;
  if (axis != 0 && axis != 1) return NVFP4_ERR_ENUM;
  if (rows < 0 || cols < 0 || !count_ok(rows, cols)) return NVFP4_ERR_SHAPE;
  const int64_t outer = axis ? rows : cols, k = axis ? cols : rows;
  if (k % 32 != 0 || out->outer != outer || out->k != k) return NVFP4_ERR_SHAPE;
  if (axis == 0 && rows > kMaxRowsAxis0Mx) return NVFP4_ERR_SHAPE;
  if (rows > 0 && cols > 0 && (!x || !out->codes || !out->scales)) return NVFP4_ERR_NULL;
  if (!aligned(x, 16) || !aligned(out->codes, 16)) return NVFP4_ERR_ALIGN;
  return hip_status(nvfp4::launch_mx_quantize(x, x_dtype, rows, cols, axis, out->codes, out->scales,
                                              (hipStream_t)hip_stream));
}

int mxfp4_gemm(const mxfp4_tensor *a, const mxfp4_tensor *b, void *c, int c_dtype, int64_t ldc, void *hip_stream) {
  if (!a || !b) return NVFP4_ERR_NULL;
  if (a->outer < 0 || b->outer < 0 || a->k < 0 || a->k != b->k || a->k % 256 != 0) return NVFP4_ERR_SHAPE;
  if (!count_ok(a->outer, a->k) || !count_ok(b->outer, b->k)) return NVFP4_ERR_SHAPE;
  if (c_dtype != NVFP4_F32 && c_dtype != NVFP4_BF16) return NVFP4_ERR_ENUM;
  const int64_t M = a->outer, N = b->outer;
  if (ldc < N || !count_ok(M, ldc) || !gemm_shape_ok(M, N, a->k)) return NVFP4_ERR_SHAPE;
  if (M > 0 && N > 0 && (!c || (a->k > 0 && (!a->codes || !a->scales || !b->codes || !b->scales))))
    return NVFP4_ERR_NULL;
  if (!aligned(c, c_dtype == NVFP4_F32 ? 4 : 2)) return NVFP4_ERR_ALIGN;
  // the kernel moves codes in 16-byte and scales in 4-byte pieces by DMA
  if (!aligned(a->codes, 16) || !aligned(b->codes, 16) || !aligned(a->scales, 4) || !aligned(b->scales, 4))
    return NVFP4_ERR_ALIGN;
  return hip_status(nvfp4::launch_mx_gemm(a->codes, a->scales, b->codes, b->scales, M, N, a->k, c, c_dtype, ldc,
                                          (hipStream_t)hip_stream));
}

int mxfp8_quantize(const void *x, int x_dtype, int64_t rows, int64_t cols, int axis, mxfp8_tensor *out,
                   void *hip_stream) {
  if (!out) return NVFP4_ERR_NULL;
  if (x_dtype != NVFP4_F32 && x_dtype != NVFP4_BF16) return NVFP4_ERR_ENUM;
  if (axis != 0 && axis != 1) return NVFP4_ERR_ENUM;
  if (rows < 0 || cols < 0 || !count_ok(rows, cols)) return NVFP4_ERR_SHAPE;
  const int64_t outer = axis ? rows : cols, k = axis ? cols : rows;
  if (k % 32 != 0 || out->outer != outer || out->k != k) return NVFP4_ERR_SHAPE;
  if (axis == 0 && rows > kMaxRowsAxis0Mx8) return NVFP4_ERR_SHAPE;
  if (rows > 0 && cols > 0 && (!x || !out->codes || !out->scales)) return NVFP4_ERR_NULL;
  if (!aligned(x, 16) || !aligned(out->codes, 16)) return NVFP4_ERR_ALIGN;
  return hip_status(nvfp4::launch_mx8_quantize(x, x_dtype, rows, cols, axis, out->codes, out->scales,
                                               (hipStream_t)hip_stream));
}

int mxfp8_gemm(const mxfp8_tensor *a, const mxfp8_tensor *b, void *c, int c_dtype, int64_t ldc, void *hip_stream) {
  if (!a || !b) return NVFP4_ERR_NULL;
  if (a->outer < 0 || b->outer < 0 || a->k < 0 || a->k != b->k || a->k % 128 != 0) return NVFP4_ERR_SHAPE;
  if (a->k > kMaxGemmKMx8 || !count_ok(a->outer, a->k) || !count_ok(b->outer, b->k)) return NVFP4_ERR_SHAPE;
  if (c_dtype != NVFP4_F32 && c_dtype != NVFP4_BF16) return NVFP4_ERR_ENUM;
  const int64_t M = a->outer, N = b->outer;
  if (ldc < N || !count_ok(M, ldc) || !gemm_shape_ok(M, N, 0)) return NVFP4_ERR_SHAPE;
  if (M > 0 && N > 0 && (!c || (a->k > 0 && (!a->codes || !a->scales || !b->codes || !b->scales))))
    return NVFP4_ERR_NULL;
  if (!aligned(c, c_dtype == NVFP4_F32 ? 4 : 2)) return NVFP4_ERR_ALIGN;
  // the kernel moves codes in 16-byte and scales in 4-byte pieces by DMA
  if (!aligned(a->codes, 16) || !aligned(b->codes, 16) || !aligned(a->scales, 4) || !aligned(b->scales, 4))
    return NVFP4_ERR_ALIGN;
  return hip_status(nvfp4::launch_mx8_gemm(a->codes, a->scales, b->codes, b->scales, M, N, a->k, c, c_dtype, ldc,
                                           (hipStream_t)hip_stream));
}

int nvfp4_dequantize(const nvfp4_tensor *q, void *y, int y_dtype, void *hip_stream) {
  int st = check_tensor(q);
  if (st != NVFP4_OK) return st;
  if (y_dtype != NVFP4_F32 && y_dtype != NVFP4_BF16) return NVFP4_ERR_ENUM;
  if (q->outer > 0 && q->k > 0 && !y) return NVFP4_ERR_NULL;
  if (!aligned(y, 16)) return NVFP4_ERR_ALIGN;
  return hip_status(nvfp4::launch_dequantize(q->codes, q->scales, q->meta, q->outer, q->k, y, y_dtype,
                                              (hipStream_t)hip_stream));
}

int nvfp4_gemm(const nvfp4_tensor *a, const nvfp4_tensor *b, void *c, int c_dtype, int64_t ldc, void *hip_stream) {
  int st = check_gemm_args(a, b, c, c_dtype, ldc);
  if (st != NVFP4_OK) return st;
  return hip_status(nvfp4::launch_gemm(a->codes, a->scales, a->meta, b->codes, b->scales, b->meta, a->outer, b->outer, a->k, c,
                                       c_dtype, ldc, (hipStream_t)hip_stream));
}

int nvfp4_gemm_ws(const nvfp4_tensor *a, const nvfp4_tensor *b, void *c, int c_dtype, int64_t ldc, void *workspace,
                  int64_t workspace_bytes, void *hip_stream) {
  int st = check_gemm_args(a, b, c, c_dtype, ldc);
  if (st != NVFP4_OK) return st;
  if (!workspace) return NVFP4_ERR_NULL;
  if (workspace_bytes < nvfp4::gemm_split_workspace_bytes()) return NVFP4_ERR_SHAPE;
  if (!aligned(workspace, 256)) return NVFP4_ERR_ALIGN;
  return hip_status(nvfp4::launch_gemm_split(a->codes, a->scales, a->meta, b->codes, b->scales, b->meta, a->outer,
                                          b->outer, a->k, c, c_dtype, ldc, workspace, (hipStream_t)hip_stream));
}

int64_t nvfp4_gemm_workspace_bytes(void) { return nvfp4::gemm_split_workspace_bytes(); }

int nvfp4_gemm_noalloc(const nvfp4_tensor *a, const nvfp4_tensor *b, void *c, int c_dtype, int64_t ldc,
                       void *hip_stream) {
  int st = check_gemm_args(a, b, c, c_dtype, ldc);
  if (st != NVFP4_OK) return st;
  // the split launcher needs at most gemm_split_workspace_bytes() for any
  // shape; beyond the library's array the call is refused
  if (nvfp4::gemm_split_workspace_bytes() > nvfp4::gemm_scratch_bytes()) return NVFP4_ERR_SHAPE;
  void *ws = nullptr;
  hipError_t e = nvfp4::gemm_scratch((hipStream_t)hip_stream, &ws);
  if (e != hipSuccess) return NVFP4_ERR_HIP;
  return hip_status(nvfp4::launch_gemm_split(a->codes, a->scales, a->meta, b->codes, b->scales, b->meta, a->outer,
                                             b->outer, a->k, c, c_dtype, ldc, ws, (hipStream_t)hip_stream));
}

int64_t nvfp4_layer_norm_workspace_bytes(int64_t rows, int64_t cols) {
  if (cols < 1 || cols > kMaxNormCols || !matrix_ok(rows, cols, cols)) return NVFP4_ERR_SHAPE;
  return nvfp4::layer_norm_workspace_bytes(rows, cols);
}

int nvfp4_layer_norm(const void *x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, const void *weight,
                     const void *bias, int w_dtype, float eps, void *y, int y_dtype, int64_t ldy, float *mean,
                     float *rstd, float *amax, void *workspace, int64_t workspace_bytes, void *hip_stream) {
  if (!dtype_ok(x_dtype) || !dtype_ok(w_dtype) || !dtype_ok(y_dtype)) return NVFP4_ERR_ENUM;
  if (cols < 1 || cols > kMaxNormCols || !matrix_ok(rows, cols, ldx) || !matrix_ok(rows, cols, ldy))
    return NVFP4_ERR_SHAPE;
  if (!(eps >= 0.0f) || eps > 3.0e38f) return NVFP4_ERR_VALUE;
  const int64_t need = amax ? nvfp4::layer_norm_workspace_bytes(rows, cols) : 0;
  if (workspace_bytes < need) return NVFP4_ERR_SHAPE;
  if (rows > 0 && (!x || !y || !mean || !rstd)) return NVFP4_ERR_NULL;
  if (need > 0 && !workspace) return NVFP4_ERR_NULL;
  if (!aligned(x, dtype_size(x_dtype)) || !aligned(y, dtype_size(y_dtype)) || !aligned(weight, dtype_size(w_dtype)) ||
      !aligned(bias, dtype_size(w_dtype)) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(amax, 4) || !aligned(workspace, 4))
    return NVFP4_ERR_ALIGN;
  const int64_t xs = dtype_size(x_dtype), ys = dtype_size(y_dtype);
  if (overlap(x, ldx * xs, cols * xs, y, ldy * ys, cols * ys, rows)) return NVFP4_ERR_SHAPE;
  return hip_status(nvfp4::launch_layer_norm(x, x_dtype, rows, cols, ldx, weight, bias, w_dtype, eps, y, y_dtype, ldy,
                                             mean, rstd, amax, workspace, (hipStream_t)hip_stream));
}

int64_t nvfp4_layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  if (cols < 1 || cols > kMaxNormCols || !matrix_ok(rows, cols, cols)) return NVFP4_ERR_SHAPE;
  return nvfp4::layer_norm_backward_workspace_bytes(rows, cols);
}

int nvfp4_layer_norm_backward(const void *dy, int dy_dtype, int64_t lddy, const void *x, int x_dtype, int64_t rows,
                              int64_t cols, int64_t ldx, const float *mean, const float *rstd, const void *weight,
                              int w_dtype, void *dx, int64_t lddx, void *dweight, void *dbias, int g_dtype,
                              void *workspace, int64_t workspace_bytes, void *hip_stream) {
  if (!dtype_ok(dy_dtype) || !dtype_ok(x_dtype) || !dtype_ok(w_dtype) || !dtype_ok(g_dtype)) return NVFP4_ERR_ENUM;
  if (cols < 1 || cols > kMaxNormCols || !matrix_ok(rows, cols, ldx) || !matrix_ok(rows, cols, lddy) ||
      !matrix_ok(rows, cols, lddx))
    return NVFP4_ERR_SHAPE;
  const int64_t need = nvfp4::layer_norm_backward_workspace_bytes(rows, cols);
  if (workspace_bytes < need) return NVFP4_ERR_SHAPE;
  if (rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return NVFP4_ERR_NULL;
  if (need > 0 && !workspace) return NVFP4_ERR_NULL;
  if (!aligned(dy, dtype_size(dy_dtype)) || !aligned(x, dtype_size(x_dtype)) || !aligned(dx, dtype_size(x_dtype)) ||
      !aligned(weight, dtype_size(w_dtype)) || !aligned(dweight, dtype_size(g_dtype)) ||
      !aligned(dbias, dtype_size(g_dtype)) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(workspace, 16))
    return NVFP4_ERR_ALIGN;
  const int64_t xs = dtype_size(x_dtype), ds = dtype_size(dy_dtype);
  if (overlap(dy, lddy * ds, cols * ds, dx, lddx * xs, cols * xs, rows) ||
      overlap(x, ldx * xs, cols * xs, dx, lddx * xs, cols * xs, rows))
    return NVFP4_ERR_SHAPE;
  return hip_status(nvfp4::launch_layer_norm_backward(dy, dy_dtype, lddy, x, x_dtype, ldx, mean, rstd, weight, w_dtype,
                                                      dx, lddx, dweight, dbias, g_dtype, workspace, rows, cols,
                                                      (hipStream_t)hip_stream));
}

int64_t nvfp4_matvec_workspace_bytes(int64_t n, int64_t k, int64_t tokens, int x_dtype) {
  if (!dtype_ok(x_dtype)) return NVFP4_ERR_ENUM;
  if (n < 0 || k < 0 || k % 16 != 0 || !matrix_ok(tokens, k, k) || !matrix_ok(tokens, n, n) || !count_ok(n, k) ||
      n > kMaxMatvecRows || tokens > kMaxMatvecTokens || k > kMaxGemmK)
    return NVFP4_ERR_SHAPE;
  return nvfp4::matvec_workspace_bytes(n, k, tokens, x_dtype == NVFP4_F32);
}

int nvfp4_matvec(const nvfp4_tensor *w, const void *x, int x_dtype, int64_t tokens, int64_t ldx, void *y, int y_dtype,
                 int64_t ldy, void *workspace, int64_t workspace_bytes, void *hip_stream) {
  const int st = check_tensor(w);
  if (st != NVFP4_OK) return st;
  return matvec_common(false, w->codes, w->scales, w->meta, w->outer, w->k, x, x_dtype, tokens, ldx, y, y_dtype, ldy,
                       workspace, workspace_bytes, hip_stream);
}

int mxfp4_matvec(const mxfp4_tensor *w, const void *x, int x_dtype, int64_t tokens, int64_t ldx, void *y, int y_dtype,
                 int64_t ldy, void *workspace, int64_t workspace_bytes, void *hip_stream) {
  if (!w) return NVFP4_ERR_NULL;
  if (w->outer < 0 || w->k < 0 || w->k % 32 != 0 || !count_ok(w->outer, w->k)) return NVFP4_ERR_SHAPE;
  if (w->outer > 0 && w->k > 0 && (!w->codes || !w->scales)) return NVFP4_ERR_NULL;
  if (!aligned(w->codes, 16)) return NVFP4_ERR_ALIGN;
  return matvec_common(true, w->codes, w->scales, nullptr, w->outer, w->k, x, x_dtype, tokens, ldx, y, y_dtype, ldy,
                       workspace, workspace_bytes, hip_stream);
}

int64_t nvfp4_distill_topk_workspace_bytes(int64_t tokens, int64_t vocab) {
  if (vocab < 1 || vocab > kMaxVocab || !matrix_ok(tokens, vocab, vocab)) return NVFP4_ERR_SHAPE;
  return nvfp4::distill_workspace_bytes(tokens, vocab);
}

int nvfp4_distill_topk(const void *logits, int z_dtype, int64_t tokens, int64_t vocab, int64_t ldz,
                       const void *indices, int index_bits, const void *teacher, int t_dtype, int64_t top,
                       float temperature, float *loss, float *lse, void *workspace, int64_t workspace_bytes,
                       void *hip_stream) {
  const int st = check_distill(logits, z_dtype, tokens, vocab, ldz, indices, index_bits, teacher, t_dtype, top,
                               temperature, lse);
  if (st != NVFP4_OK) return st;
  const int64_t need = nvfp4::distill_workspace_bytes(tokens, vocab);
  if (workspace_bytes < need) return NVFP4_ERR_SHAPE;
  if ((tokens > 0 && !loss) || (need > 0 && !workspace)) return NVFP4_ERR_NULL;
  if (!aligned(loss, 4) || !aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
  return hip_status(nvfp4::launch_distill(logits, z_dtype, tokens, vocab, ldz, indices, index_bits == 64, teacher,
                                          t_dtype, (int)top, temperature, nullptr, loss, lse, nullptr, 0, workspace,
                                          true, (hipStream_t)hip_stream));
}

int nvfp4_distill_topk_backward(const void *logits, int z_dtype, int64_t tokens, int64_t vocab, int64_t ldz,
                                const void *indices, int index_bits, const void *teacher, int t_dtype, int64_t top,
                                float temperature, const float *lse, const float *dloss, void *dlogits, int64_t lddz,
                                void *hip_stream) {
  const int st = check_distill(logits, z_dtype, tokens, vocab, ldz, indices, index_bits, teacher, t_dtype, top,
                               temperature, lse);
  if (st != NVFP4_OK) return st;
  if (!matrix_ok(tokens, vocab, lddz)) return NVFP4_ERR_SHAPE;
  if (tokens > 0 && (!dloss || !dlogits)) return NVFP4_ERR_NULL;
  if (!aligned(dloss, 4) || !aligned(dlogits, dtype_size(z_dtype))) return NVFP4_ERR_ALIGN;
  const int64_t e = dtype_size(z_dtype);
  if (overlap(logits, ldz * e, vocab * e, dlogits, lddz * e, vocab * e, tokens)) return NVFP4_ERR_SHAPE;
  return hip_status(nvfp4::launch_distill(logits, z_dtype, tokens, vocab, ldz, indices, index_bits == 64, teacher,
                                          t_dtype, (int)top, temperature, dloss, nullptr, const_cast<float *>(lse),
                                          dlogits, lddz, nullptr, false, (hipStream_t)hip_stream));
}

int nvfp4_distill_topk_step(const void *logits, int z_dtype, int64_t tokens, int64_t vocab, int64_t ldz,
                            const void *indices, int index_bits, const void *teacher, int t_dtype, int64_t top,
                            float temperature, const float *weight, float *loss, float *lse, void *dlogits,
                            int64_t lddz, void *workspace, int64_t workspace_bytes, void *hip_stream) {
  const int st = check_distill(logits, z_dtype, tokens, vocab, ldz, indices, index_bits, teacher, t_dtype, top,
                               temperature, lse);
  if (st != NVFP4_OK) return st;
  if (!matrix_ok(tokens, vocab, lddz)) return NVFP4_ERR_SHAPE;
  const int64_t need = nvfp4::distill_workspace_bytes(tokens, vocab);
  if (workspace_bytes < need) return NVFP4_ERR_SHAPE;
  if ((tokens > 0 && (!weight || !loss || !dlogits)) || (need > 0 && !workspace)) return NVFP4_ERR_NULL;
  if (!aligned(weight, 4) || !aligned(loss, 4) || !aligned(dlogits, dtype_size(z_dtype)) || !aligned(workspace, 16))
    return NVFP4_ERR_ALIGN;
  const int64_t e = dtype_size(z_dtype);
  if (overlap(logits, ldz * e, vocab * e, dlogits, lddz * e, vocab * e, tokens)) return NVFP4_ERR_SHAPE;
  return hip_status(nvfp4::launch_distill(logits, z_dtype, tokens, vocab, ldz, indices, index_bits == 64, teacher,
                                          t_dtype, (int)top, temperature, weight, loss, lse, dlogits, lddz, workspace,
                                          true, (hipStream_t)hip_stream));
}

const char *nvfp4_status_string(int status) {
  switch (status) {
    case NVFP4_OK: return "ok";
    case NVFP4_ERR_NULL: return "null pointer";
    case NVFP4_ERR_SHAPE: return "invalid shape";
    case NVFP4_ERR_ENUM: return "invalid enum value";
    case NVFP4_ERR_HIP: return "HIP launch failed";
    case NVFP4_ERR_ALIGN: return "misaligned pointer";
    case NVFP4_ERR_VALUE: return "scalar argument out of range";
    default: return "unknown status";
  }
}

}  // extern "C"
