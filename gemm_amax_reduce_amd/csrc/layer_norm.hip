// layer_norm.hip -- layer norm over the rows of a matrix for gfx950, forward
// and backward, with the tensor maximum for the quantizer and the reduction
// of the weight and bias gradients.
//
//   m = sum x / C,  v = sum (x - m)^2 / C,  r = 1 / sqrt(v + eps)
//   y = (x - m) r w + b
//   a = dy w,  h = (x - m) r
//   dx = r (a - mean(a) - h mean(a h)),  dw = sum_rows dy h,  db = sum_rows dy
//
// Every pass is bound by HBM: 2 matrices move forward, 3 backward, against
// some 10 operations per element.  So a row is read once and stays in
// registers (8 elements per 16- or 32-byte load, VPT such vectors a thread)
// while its statistics are reduced over the workgroup; the variance is the
// sum of squared differences from the mean, taken in a second sweep over the
// registers, so that no digits cancel.  All sums are binary32.
#include "nvfp4_kernels.h"
#include "row_common.h"

#include <algorithm>

namespace nvfp4 {

namespace {

constexpr int kMaxThreads = 1024;
constexpr int kMaxWaves = kMaxThreads / 64;

__global__ void k_amax_init(uint32_t *amax) {
  if (threadIdx.x == 0) *amax = 0;
}

// |value as stored| as a bit pattern (NaN > Inf > finite).
template <typename T> __device__ __forceinline__ uint32_t absmax8(const Row8<T> &r) {
  float v[8];
  r.get(v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

// One workgroup per row, rows blockIdx.x, blockIdx.x + gridDim.x, ...; the
// threads keep their columns' weights and biases over all of them.
template <typename X, typename Y, int VPT>
__global__ __launch_bounds__(kMaxThreads) void k_ln_forward(const X *x, int64_t ldx, const void *w, const void *b, int w_bf16, Y *y,
                                       int64_t ldy, float *mean, float *rstd, uint32_t *amax, int64_t rows,
                                       int64_t cols, float eps) {
  __shared__ float part[2][2][kMaxWaves];
  __shared__ uint32_t umax[kMaxWaves];
  const int64_t step = (int64_t)blockDim.x * 8;
  const int64_t c0 = (int64_t)threadIdx.x * 8;
  float wv[VPT][8], bv[VPT][8];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    load_param8(wv[j], w, w_bf16, c0 + j * step, cols, 1.0f);
    load_param8(bv[j], b, w_bf16, c0 + j * step, cols, 0.0f);
  }
  uint32_t top = 0;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, turn ^= 1) {
    float v[VPT][8];
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      Row8<X> q;
      load_row8(q, x + row * ldx, c0 + j * step, cols);
      q.get(v[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[j][i];
    }
    const float m = block_sum(s, part[turn][0]) / (float)cols;
    float s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int64_t left = cols - (c0 + j * step);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[j][i] = i < left ? v[j][i] - m : 0.0f;
        s2 = __builtin_fmaf(v[j][i], v[j][i], s2);
      }
    }
    const float var = block_sum(s2, part[turn][1]) / (float)cols;
    const float r = 1.0f / __builtin_sqrtf(var + eps);
    if (threadIdx.x == 0) {
      mean[row] = m;
      rstd[row] = r;
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int64_t at = c0 + j * step;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = __builtin_fmaf(v[j][i] * r, wv[j][i], bv[j][i]);
      Row8<Y> q;
      q.set(v[j]);
      store_row8(q, y + row * ldy, at, cols);
      if (amax && at < cols) {
        // past the end v = fma(0, 1, 0) = 0 (or a NaN that the row holds anyway)
        top = max(top, absmax8(q));
      }
    }
  }
  if (amax) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
    if ((threadIdx.x & 63) == 0) umax[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < (int)(blockDim.x >> 6); ++i) top = max(top, umax[i]);
      // the value only grows, so a workgroup that cannot raise it skips the atomic
      if (top > __hip_atomic_load(amax, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) atomicMax(amax, top);
    }
  }
}

// Rows wider than the registers of a workgroup hold: the row is read three
// times (the second and third time from the caches).
template <typename X, typename Y>
__global__ __launch_bounds__(kMaxThreads) void k_ln_forward_wide(const X *x, int64_t ldx, const void *w, const void *b, int w_bf16,
                                            Y *y, int64_t ldy, float *mean, float *rstd, uint32_t *amax,
                                            int64_t rows, int64_t cols, float eps) {
  __shared__ float part[2][2][kMaxWaves];
  const int64_t step = (int64_t)blockDim.x * 8;
  const int64_t c0 = (int64_t)threadIdx.x * 8;
  uint32_t top = 0;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, turn ^= 1) {
    const X *xr = x + row * ldx;
    float s = 0.0f, v[8];
    for (int64_t at = c0; at < cols; at += step) {
      Row8<X> q;
      load_row8(q, xr, at, cols);
      q.get(v);
      float t = 0.0f;   // vector by vector, so that a long row's sum keeps its digits
#pragma unroll
      for (int i = 0; i < 8; ++i) t += v[i];
      s += t;
    }
    const float m = block_sum(s, part[turn][0]) / (float)cols;
    float s2 = 0.0f;
    for (int64_t at = c0; at < cols; at += step) {
      Row8<X> q;
      load_row8(q, xr, at, cols);
      q.get(v);
      float t = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = at + i < cols ? v[i] - m : 0.0f;
        t = __builtin_fmaf(d, d, t);
      }
      s2 += t;
    }
    const float var = block_sum(s2, part[turn][1]) / (float)cols;
    const float r = 1.0f / __builtin_sqrtf(var + eps);
    if (threadIdx.x == 0) {
      mean[row] = m;
      rstd[row] = r;
    }
    for (int64_t at = c0; at < cols; at += step) {
      Row8<X> q;
      load_row8(q, xr, at, cols);
      q.get(v);
      float wv[8], bv[8];
      load_param8(wv, w, w_bf16, at, cols, 1.0f);
      load_param8(bv, b, w_bf16, at, cols, 0.0f);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = at + i < cols ? __builtin_fmaf((v[i] - m) * r, wv[i], bv[i]) : 0.0f;
      Row8<Y> o;
      o.set(v);
      store_row8(o, y + row * ldy, at, cols);
      top = max(top, absmax8(o));
    }
  }
  if (amax) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
    if ((threadIdx.x & 63) == 0) atomicMax(amax, top);
  }
}

// Backward, first kernel: the two row sums (mean of a, mean of a h).
template <typename X, typename D>
__global__ __launch_bounds__(kMaxThreads) void k_ln_backward_rows(const D *dy, int64_t lddy, const X *x, int64_t ldx, const float *mean,
                                             const float *rstd, const void *w, int w_bf16, float2 *sums,
                                             int64_t rows, int64_t cols) {
  __shared__ float part[2][2][kMaxWaves];
  const int64_t step = (int64_t)blockDim.x * 8;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, turn ^= 1) {
    const float m = mean[row], r = rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t at = (int64_t)threadIdx.x * 8; at < cols; at += step) {
      Row8<X> qx;
      Row8<D> qd;
      load_row8(qx, x + row * ldx, at, cols);
      load_row8(qd, dy + row * lddy, at, cols);
      float xv[8], dv[8], wv[8];
      qx.get(xv);
      qd.get(dv);
      load_param8(wv, w, w_bf16, at, cols, 1.0f);
      float t1 = 0.0f, t2 = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = dv[i] * wv[i];        // 0 past the end: dy is
        t1 += a;
        t2 = __builtin_fmaf(a, (xv[i] - m) * r, t2);
      }
      s1 += t1;
      s2 += t2;
    }
    const float a1 = block_sum(s1, part[turn][0]) / (float)cols;
    const float a2 = block_sum(s2, part[turn][1]) / (float)cols;
    if (threadIdx.x == 0) sums[row] = make_float2(a1, a2);
  }
}

// Backward, second kernel: dx, and this workgroup's rows' share of dw and db
// for its 8 * blockDim.x columns.  partial: [gridDim.y][2][cols].
template <typename X, typename D>
__global__ __launch_bounds__(256) void k_ln_backward_cols(const D *dy, int64_t lddy, const X *x, int64_t ldx,
                                                          const float *mean, const float *rstd, const void *w,
                                                          int w_bf16, const float2 *sums, X *dx, int64_t lddx,
                                                          float *partial, int64_t rows, int64_t cols) {
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (at >= cols) return;
  float wv[8], dw[8], db[8];
  load_param8(wv, w, w_bf16, at, cols, 1.0f);
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = db[i] = 0.0f;
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const float m = mean[row], r = rstd[row];
    const float2 s = sums[row];
    Row8<X> qx;
    Row8<D> qd;
    load_row8(qx, x + row * ldx, at, cols);
    load_row8(qd, dy + row * lddy, at, cols);
    float xv[8], dv[8];
    qx.get(xv);
    qd.get(dv);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float h = (xv[i] - m) * r;
      dw[i] = __builtin_fmaf(dv[i], h, dw[i]);
      db[i] += dv[i];
      xv[i] = r * __builtin_fmaf(-h, s.y, __builtin_fmaf(dv[i], wv[i], -s.x));
    }
    qx.set(xv);
    store_row8(qx, dx + row * lddx, at, cols);
  }
  Row8<float> q;
  q.set(dw);
  store_row8(q, partial + (int64_t)blockIdx.y * 2 * cols, at, cols);
  q.set(db);
  store_row8(q, partial + ((int64_t)blockIdx.y * 2 + 1) * cols, at, cols);
}

// Backward, last kernel: dw and db from the partial sums, in a fixed order.
// 64 columns per workgroup (of the 2 cols that dw and db make together), 4
// interleaved shares of the partials added at the end.
__global__ __launch_bounds__(256) void k_ln_backward_sum(const float *partial, int64_t parts, int64_t cols, void *dw,
                                                         void *db, int g_bf16) {
  __shared__ float share[4][64];
  const int lane = threadIdx.x & 63, group = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < 2 * cols)
    for (int64_t p = group; p < parts; p += 4) s += partial[p * 2 * cols + c];
  share[group][lane] = s;
  __syncthreads();
  if (group == 0 && c < 2 * cols) {
    s = (share[0][lane] + share[1][lane]) + (share[2][lane] + share[3][lane]);
    void *out = c < cols ? dw : db;
    const int64_t k = c < cols ? c : c - cols;
    if (!out) return;
    if (g_bf16) ((uint16_t *)out)[k] = (uint16_t)pack_bf16(s, 0.0f);
    else ((float *)out)[k] = s;
  }
}

int threads_for(int64_t vectors, int vpt) {
  const int64_t t = (vectors + vpt - 1) / vpt;
  return (int)std::min<int64_t>(kMaxThreads, (t + 63) / 64 * 64);
}

template <typename X, typename Y>
void forward(const void *x, int64_t ldx, const void *w, const void *b, int w_bf16, void *y, int64_t ldy, float *mean,
             float *rstd, uint32_t *amax, int64_t rows, int64_t cols, float eps, hipStream_t stream) {
  const int64_t vectors = (cols + 7) / 8;
  const unsigned grid = (unsigned)std::min<int64_t>(rows, (int64_t)device_cus() * 8);
  const X *xp = (const X *)x;
  Y *yp = (Y *)y;
  if (vectors <= kMaxThreads)
    k_ln_forward<X, Y, 1><<<grid, threads_for(vectors, 1), 0, stream>>>(xp, ldx, w, b, w_bf16, yp, ldy, mean, rstd,
                                                                       amax, rows, cols, eps);
  else if (vectors <= 2 * kMaxThreads)
    k_ln_forward<X, Y, 2><<<grid, threads_for(vectors, 2), 0, stream>>>(xp, ldx, w, b, w_bf16, yp, ldy, mean, rstd,
                                                                       amax, rows, cols, eps);
  else
    k_ln_forward_wide<X, Y><<<grid, kMaxThreads, 0, stream>>>(xp, ldx, w, b, w_bf16, yp, ldy, mean, rstd, amax, rows,
                                                             cols, eps);
}

// Rows' shares of the column sums: one per workgroup row of the grid.
int64_t backward_parts(int64_t rows, int64_t cols) {
  const int64_t col_groups = (cols + 2047) / 2048;
  const int64_t want = std::max<int64_t>(1, (int64_t)device_cus() * 8 / col_groups);
  return std::min<int64_t>(std::min<int64_t>((rows + 7) / 8, want), 2048);
}

template <typename X, typename D>
void backward(const void *dy, int64_t lddy, const void *x, int64_t ldx, const float *mean, const float *rstd,
              const void *w, int w_bf16, void *dx, int64_t lddx, void *dw, void *db, int g_bf16, void *workspace,
              int64_t rows, int64_t cols, hipStream_t stream) {
  const int64_t parts = backward_parts(rows, cols);
  float2 *sums = (float2 *)workspace;
  float *partial = (float *)workspace + 2 * rows;
  if (rows > 0) {
    const unsigned grid = (unsigned)std::min<int64_t>(rows, (int64_t)device_cus() * 8);
    k_ln_backward_rows<X, D><<<grid, threads_for((cols + 7) / 8, 1), 0, stream>>>(
        (const D *)dy, lddy, (const X *)x, ldx, mean, rstd, w, w_bf16, sums, rows, cols);
    k_ln_backward_cols<X, D><<<dim3((unsigned)((cols + 2047) / 2048), (unsigned)parts), 256, 0, stream>>>(
        (const D *)dy, lddy, (const X *)x, ldx, mean, rstd, w, w_bf16, sums, (X *)dx, lddx, partial, rows, cols);
  }
  if (dw || db)
    k_ln_backward_sum<<<(unsigned)((2 * cols + 63) / 64), 256, 0, stream>>>(partial, parts, cols, dw, db, g_bf16);
}

}  // namespace

hipError_t launch_layer_norm(const void *x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, const void *w,
                             const void *b, int w_dtype, float eps, void *y, int y_dtype, int64_t ldy, float *mean,
                             float *rstd, float *amax, hipStream_t stream) {
  if (amax) k_amax_init<<<1, 64, 0, stream>>>((uint32_t *)amax);
  if (rows > 0) {
    uint32_t *um = (uint32_t *)amax;
    const int wb = w_dtype == 1;
    if (x_dtype == 1 && y_dtype == 1)
      forward<uint16_t, uint16_t>(x, ldx, w, b, wb, y, ldy, mean, rstd, um, rows, cols, eps, stream);
    else if (x_dtype == 1)
      forward<uint16_t, float>(x, ldx, w, b, wb, y, ldy, mean, rstd, um, rows, cols, eps, stream);
    else if (y_dtype == 1)
      forward<float, uint16_t>(x, ldx, w, b, wb, y, ldy, mean, rstd, um, rows, cols, eps, stream);
    else
      forward<float, float>(x, ldx, w, b, wb, y, ldy, mean, rstd, um, rows, cols, eps, stream);
  }
  return hipGetLastError();
}

int64_t layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  return 8 * rows + 8 * cols * backward_parts(rows, cols);
}

hipError_t launch_layer_norm_backward(const void *dy, int dy_dtype, int64_t lddy, const void *x, int x_dtype,
                                      int64_t ldx, const float *mean, const float *rstd, const void *w, int w_dtype,
                                      void *dx, int64_t lddx, void *dw, void *db, int g_dtype, void *workspace,
                                      int64_t rows, int64_t cols, hipStream_t stream) {
  const int wb = w_dtype == 1, gb = g_dtype == 1;
  if (x_dtype == 1 && dy_dtype == 1)
    backward<uint16_t, uint16_t>(dy, lddy, x, ldx, mean, rstd, w, wb, dx, lddx, dw, db, gb, workspace, rows, cols, stream);
  else if (x_dtype == 1)
    backward<uint16_t, float>(dy, lddy, x, ldx, mean, rstd, w, wb, dx, lddx, dw, db, gb, workspace, rows, cols, stream);
  else if (dy_dtype == 1)
    backward<float, uint16_t>(dy, lddy, x, ldx, mean, rstd, w, wb, dx, lddx, dw, db, gb, workspace, rows, cols, stream);
  else
    backward<float, float>(dy, lddy, x, ldx, mean, rstd, w, wb, dx, lddx, dw, db, gb, workspace, rows, cols, stream);
  return hipGetLastError();
}

}  // namespace nvfp4
