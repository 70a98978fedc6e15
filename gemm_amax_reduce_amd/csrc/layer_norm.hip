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
//
// Measured on one MI355X, kernels alone: forward 1 x 5120 bf16 3.3 us
// (latency), 4096 x 5120 bf16 with the tensor maximum 18.8 us (4.5 TB/s) and
// 1.6 to 4 us for joining it, 16384 x 8192 bf16 81 us (6.6 TB/s); backward 8192 x
// 5120 bf16 53 us (4.7 TB/s) and 4.8 us for the sums over rows, 1537 x 5003
// f32 19.4 (4.7 TB/s) and 4.0, 32768 x 8192 bf16 303 (5.3 TB/s) and 4.8; any
// width, forward 4096 x 20480 bf16 110 us (3.0 TB/s), backward 49 + 91 + 11 us.
#include "nvfp4_kernels.h"
#include "row_common.h"

#include <algorithm>

namespace nvfp4 {

namespace {

constexpr int kMaxThreads = 1024;
constexpr int kMaxWaves = kMaxThreads / 64;

// top becomes the wave's maximum, left in the wave's place of `share` (LDS).
__device__ __forceinline__ void wave_umax_to(uint32_t *share, uint32_t &top) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
  if ((threadIdx.x & 63) == 0) share[threadIdx.x >> 6] = top;
}

// The tensor maximum from the workgroups' own.  (Atomics on one word take
// some 10 ns each, and the workgroups come to their ends together: whole calls
// of 4096 x 5120 take 22.8 us with atomics, 19.9 so, of 8192 x 512 33 and 19.)
constexpr int kJoinThreads = 1024;
__global__ __launch_bounds__(kJoinThreads) void k_amax_join(const uint32_t *part, int n, uint32_t *amax) {
  __shared__ uint32_t share[kJoinThreads / 64];
  uint32_t top = 0;
  for (int i = threadIdx.x; i < n; i += kJoinThreads) top = max(top, part[i]);
  wave_umax_to(share, top);
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 1; i < kJoinThreads / 64; ++i) top = max(top, share[i]);
    *amax = top;
  }
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
// threads keep their columns' weights and biases over all of them, and a row
// is fetched while the one before it is worked on.
template <typename X, typename Y, int VPT, bool ONCE>
__global__ __launch_bounds__(kMaxThreads) void k_ln_forward(const X *x, int64_t ldx, const void *w, const void *b,
                                                            int w_bf16, Y *y, int64_t ldy, float *mean, float *rstd,
                                                            uint32_t *amax, int64_t rows, int64_t cols, float eps,
                                                            int threads) {
  __shared__ float part[2][2][kMaxWaves];
  __shared__ uint32_t umax[kMaxWaves];
  const int waves = threads >> 6;
  const float inv = 1.0f / (float)cols;
  constexpr bool kSplit = sizeof(X) + sizeof(Y) > 4;
  Piece<kSplit> sp[VPT];
  float wv[VPT][8], bv[VPT][8];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    sp[j] = Piece<kSplit>(Piece<kSplit>::start(threadIdx.x + j * threads), (uint32_t)cols);
    param_piece(wv[j], w, w_bf16, sp[j], 1.0f);
    param_piece(bv[j], b, w_bf16, sp[j], 0.0f);
  }
  uint32_t top = 0;
  int turn = 0;
  Row8<X> next[VPT];
  int64_t row = blockIdx.x;
#pragma unroll
  for (int j = 0; j < VPT; ++j) load_piece<ONCE>(next[j], x + row * ldx, sp[j]);
  while (row < rows) {
    float v[VPT][8];
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      next[j].get(v[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) s += sp[j].mine(i) ? v[j][i] : 0.0f;
    }
    const int64_t later = row + gridDim.x, fetch = min(later, rows - 1);
#pragma unroll
    for (int j = 0; j < VPT; ++j) load_piece<ONCE>(next[j], x + fetch * ldx, sp[j]);
    __builtin_amdgcn_sched_barrier(0);       // the loads go out before this row's work, not after it
    const float m = block_sum(s, part[turn][0], waves) * inv;
    float s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[j][i] -= m;
        const float d = sp[j].mine(i) ? v[j][i] : 0.0f;
        s2 = __builtin_fmaf(d, d, s2);
      }
    }
    const float var = block_sum(s2, part[turn][1], waves) * inv;
    const float r = 1.0f / __builtin_sqrtf(var + eps);
    if (threadIdx.x == 0) {
      mean[row] = m;
      rstd[row] = r;
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = __builtin_fmaf(v[j][i] * r, wv[j][i], bv[j][i]);
      Row8<Y> q;
      q.set(v[j]);
      store_piece(q, y + row * ldy, sp[j]);
      if (amax) top = max(top, absmax8(q));
    }
    row = later;
    turn ^= 1;
  }
  if (amax) {
    wave_umax_to(umax, top);
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < waves; ++i) top = max(top, umax[i]);
      amax[blockIdx.x] = top;
    }
  }
}

// Rows wider than the registers of a workgroup hold, or narrower than one
// vector: the row is read three times (the second and third from the caches).
template <typename X, typename Y>
__global__ __launch_bounds__(kMaxThreads) void k_ln_forward_wide(const X *x, int64_t ldx, const void *w, const void *b,
                                                                 int w_bf16, Y *y, int64_t ldy, float *mean,
                                                                 float *rstd, uint32_t *amax, int64_t rows,
                                                                 int64_t cols, float eps, int threads) {
  __shared__ float part[2][2][kMaxWaves];
  const int waves = threads >> 6;
  const int64_t step = (int64_t)threads * 8;
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
    const float m = block_sum(s, part[turn][0], waves) / (float)cols;
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
    const float var = block_sum(s2, part[turn][1], waves) / (float)cols;
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
    __shared__ uint32_t umax[kMaxWaves];
    wave_umax_to(umax, top);
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < waves; ++i) top = max(top, umax[i]);
      amax[blockIdx.x] = top;
    }
  }
}

// Backward where a row fits the registers.  A workgroup has `groups` groups
// of `tpr` threads, each of which walks rows of its own: x and dy of a row
// are read once and stay in registers between the reduction of the two row
// sums and dx, the next row's are fetched meanwhile, and every thread adds
// up dw and db of its columns over all its rows.  At the end the groups'
// sums meet in LDS, and the workgroup leaves one partial row of dw and one of
// db, or, if it is the only one, dw and db themselves (each may be null).
// partial: [gridDim.x][2][cols]; dynamic LDS: (groups - 1) * cols floats.
template <typename X, typename D, int VPT, int THREADS, bool ONCE>
__global__ __launch_bounds__(THREADS) void k_ln_backward(const D *dy, int64_t lddy, const X *x, int64_t ldx,
                                                         const float *mean, const float *rstd, const void *w,
                                                         int w_bf16, X *dx, int64_t lddx, float *partial, void *dw_out,
                                                         void *db_out, int g_bf16, int64_t rows, int64_t cols, int tpr,
                                                         int groups) {
  __shared__ float2 part[2][kMaxWaves];
  extern __shared__ float sums[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wpr = tpr >> 6;
  const int group = wave / wpr, t = threadIdx.x - group * tpr;
  const int64_t stride = (int64_t)gridDim.x * groups;
  const float inv = 1.0f / (float)cols;
  constexpr bool kSplit = sizeof(X) + sizeof(D) > 4;
  Piece<kSplit> sp[VPT];
  float wv[VPT][8], dw[VPT][8], db[VPT][8];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    sp[j] = Piece<kSplit>(Piece<kSplit>::start(t + j * tpr), (uint32_t)cols);
    param_piece(wv[j], w, w_bf16, sp[j], 1.0f);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = db[j][i] = 0.0f;
  }
  Row8<X> xn[VPT];
  Row8<D> dn[VPT];
  float mn, rn;
  const auto fetch = [&](int64_t r) {
    r = min(r, rows - 1);              // (past the last row: fetched, not used)
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      load_piece<ONCE>(xn[j], x + r * ldx, sp[j]);
      load_piece<ONCE>(dn[j], dy + r * lddy, sp[j]);
    }
    mn = mean[r];
    rn = rstd[r];
  };
  int64_t row = (int64_t)blockIdx.x * groups + group;
  fetch(row);
  // the workgroup's groups make the same number of turns (barriers)
  int turn = 0;
  for (int64_t first = (int64_t)blockIdx.x * groups; first < rows; first += stride, row += stride, turn ^= 1) {
    const float m = mn, r = rn;
    float s1 = 0.0f, s2 = 0.0f;
    Row8<X> xc[VPT];
    Row8<D> dc[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      xc[j] = xn[j];
      dc[j] = dn[j];
    }
    fetch(row + stride);
    __builtin_amdgcn_sched_barrier(0);       // the loads go out before this row's work, not after it
    if (row < rows) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        float xv[8], dv[8];
        xc[j].get(xv);
        dc[j].get(dv);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float h = (xv[i] - m) * r, a = sp[j].mine(i) ? dv[i] * wv[j][i] : 0.0f;
          dw[j][i] = __builtin_fmaf(dv[i], h, dw[j][i]);
          db[j][i] += dv[i];
          s1 += a;
          // (a stays out of the sum as it is: 0 times an h that is not finite would enter it)
          s2 = sp[j].mine(i) ? __builtin_fmaf(a, h, s2) : s2;
        }
      }
    }
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if (wpr > 1) {
      if ((threadIdx.x & 63) == 0) part[turn][wave] = make_float2(s1, s2);
      __syncthreads();
      s1 = s2 = 0.0f;
      for (int i = 0; i < wpr; ++i) {
        const float2 p = part[turn][group * wpr + i];
        s1 += p.x;
        s2 += p.y;
      }
    }
    s1 *= inv;
    s2 *= inv;
    if (row < rows) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        // h and a once more, from the row as it was read: to keep them over the
        // reduction would take twice the registers for 16-bit types
        float o[8], xv[8], dv[8];
        xc[j].get(xv);
        dc[j].get(dv);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          o[i] = r * __builtin_fmaf(-(xv[i] - m) * r, s2, __builtin_fmaf(dv[i], wv[j][i], -s1));
        Row8<X> q;
        q.set(o);
        store_piece(q, dx + row * lddx, sp[j]);
      }
    }
  }
  // dw, then db
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (groups > 1) {
      __syncthreads();
      if (group > 0) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
          Row8<float> q;
          q.set(k ? db[j] : dw[j]);
          store_piece(q, sums + (int64_t)(group - 1) * cols, sp[j]);
        }
      }
      __syncthreads();
    }
    if (group == 0) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = k ? db[j][i] : dw[j][i];
        for (int g = 1; g < groups; ++g) {
          Row8<float> q;
          float u[8];
          load_piece(q, sums + (int64_t)(g - 1) * cols, sp[j]);
          q.get(u);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += u[i];
        }
        void *const out = gridDim.x > 1 ? partial + ((int64_t)blockIdx.x * 2 + k) * cols : k ? db_out : dw_out;
        if (!out) continue;
        if (gridDim.x == 1 && g_bf16) {
          Row8<uint16_t> q;
          q.set(v);
          store_piece(q, (uint16_t *)out, sp[j]);
        } else {
          Row8<float> q;
          q.set(v);
          store_piece(q, (float *)out, sp[j]);
        }
      }
    }
  }
}

// Wider rows, first kernel: the two row sums (mean of a, mean of a h).
template <typename X, typename D>
__global__ __launch_bounds__(kMaxThreads) void k_ln_backward_rows(const D *dy, int64_t lddy, const X *x, int64_t ldx,
                                                                  const float *mean, const float *rstd, const void *w,
                                                                  int w_bf16, float2 *sums, int64_t rows,
                                                                  int64_t cols, int threads) {
  __shared__ float part[2][2][kMaxWaves];
  const int waves = threads >> 6;
  const int64_t step = (int64_t)threads * 8;
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
    const float a1 = block_sum(s1, part[turn][0], waves) / (float)cols;
    const float a2 = block_sum(s2, part[turn][1], waves) / (float)cols;
    if (threadIdx.x == 0) sums[row] = make_float2(a1, a2);
  }
}

// Wider rows, second kernel: dx, and this workgroup's rows' share of dw and
// db for its 2048 columns.  partial: [gridDim.y][2][cols].
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

// Backward, last kernel: dw and db from the partial rows, in a fixed order:
// 64 columns per workgroup (from `first` on, of the 2 cols that dw and db make
// together), 16 interleaved shares of the rows, added at the end.
constexpr int kShares = 16;
__global__ __launch_bounds__(64 * kShares) void k_ln_backward_sum(const float *partial, int64_t parts, int64_t cols,
                                                                  int64_t first, void *dw, void *db, int g_bf16) {
  __shared__ float share[kShares][64];
  const int lane = threadIdx.x & 63, group = threadIdx.x >> 6;
  const int64_t c = first + (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < 2 * cols) {
    const float *p = partial + c;
#pragma unroll 8
    for (int64_t k = group; k < parts; k += kShares) s += p[k * 2 * cols];
  }
  share[group][lane] = s;
  __syncthreads();
  if (group == 0 && c < 2 * cols) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < kShares; ++i) s += share[i][lane];
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

// Threads of a row for the kernels that take any width, and how many such
// workgroups: 32 waves a CU, one wave a row where that holds it (forward of
// 65536 x 6: 60 us, in workgroups of 1024 threads 760).
int any_width_threads(int64_t cols) { return cols < 8 ? 64 : kMaxThreads; }
unsigned any_width_grid(int64_t rows, int64_t cols) {
  return (unsigned)std::min<int64_t>(rows, (int64_t)device_cus() * (32 * 64 / any_width_threads(cols)));
}

// How a forward pass is cut: vectors per thread (0 = the wide kernel),
// threads and number of the workgroups.
struct ForwardCut {
  int vpt, threads;
  unsigned grid;
};
ForwardCut forward_cut(int64_t rows, int64_t cols, bool amax) {
  const int64_t vectors = (cols + 7) / 8;
  ForwardCut c;
  // one 8-element vector a thread where that makes a workgroup of up to 256
  // threads, else two (fewer waves to wait for at a row's two reductions)
  c.vpt = cols < 8 ? 0 : vectors <= 256 ? 1 : vectors <= 2 * kMaxThreads ? 2 : 0;
  c.threads = c.vpt ? threads_for(vectors, c.vpt) : any_width_threads(cols);
  // the maximum over a few rows: one workgroup, whose own it is (4 x 5120: 13.4
  // us a call, with a second kernel 17.4)
  if (amax && rows <= 4) {
    c.grid = (unsigned)std::min<int64_t>(rows, 1);
    return c;
  }
  if (!c.vpt) {
    c.grid = any_width_grid(rows, cols);
    return c;
  }
  // one round of workgroups, 16 waves a CU (4096 x 5120: 18.7 us, with 20 waves
  // 21.7, one workgroup a row 22)
  c.grid = (unsigned)std::min<int64_t>(rows, (int64_t)device_cus() * std::max(1, 16 * 64 / c.threads));
  return c;
}

// amax: a place for each workgroup's maximum, or null
template <typename X, typename Y>
void forward(const ForwardCut &c, const void *x, int64_t ldx, const void *w, const void *b, int w_bf16, void *y,
             int64_t ldy, float *mean, float *rstd, uint32_t *amax, int64_t rows, int64_t cols, float eps,
             hipStream_t stream) {
  const X *xp = (const X *)x;
  Y *yp = (Y *)y;
  const auto launch = [&](auto kernel) {
    kernel<<<c.grid, c.threads, 0, stream>>>(xp, ldx, w, b, w_bf16, yp, ldy, mean, rstd, amax, rows, cols, eps,
                                             c.threads);
  };
  const bool once = reads_once(rows * cols * (int64_t)(sizeof(X) + sizeof(Y)));
  if (c.vpt == 1) with_flag(once, [&](auto o) { launch(k_ln_forward<X, Y, 1, o.value>); });
  else if (c.vpt == 2) with_flag(once, [&](auto o) { launch(k_ln_forward<X, Y, 2, o.value>); });
  else launch(k_ln_forward_wide<X, Y>);
}

// How a backward pass is cut: vectors per thread (0 = the two kernels for
// wider rows, which also take those of less than one vector), threads a row,
// rows a workgroup works on at a time, and the partial rows of dw and db, one
// per workgroup (per workgroup row of the grid for wider rows).
struct BackCut {
  int vpt, tpr, groups;
  int64_t parts;
};
// Threads of a workgroup, by the registers that a thread takes (121 with two
// bf16 vectors each of x and dy, 160 with f32, 210 with four bf16 vectors).
constexpr int back_threads(int vpt, bool narrow) { return vpt == 4 ? 512 : narrow ? 1024 : 768; }
BackCut back_cut(int64_t rows, int64_t cols, bool narrow) {      // narrow: x and dy are both bf16
  const int64_t vectors = (cols + 7) / 8;
  BackCut c;
  // (four vectors of f32 do not fit the registers of 512 threads)
  c.vpt = cols < 8 ? 0 : vectors <= 64 ? 1 : vectors <= 1024 ? 2 : vectors <= 2048 && narrow ? 4 : 0;
  if (c.vpt) {
    c.tpr = threads_for(vectors, c.vpt);
    c.groups = std::max(1, back_threads(c.vpt, narrow) / c.tpr);
    const int64_t rounds = (rows + c.groups - 1) / c.groups;
    // one workgroup a CU, and two rounds for it at least: what the partial
    // rows cost to write and add up stays below a pass over the data.  Up to
    // four rounds one workgroup does without partial rows and the kernel that
    // adds them (6 x 5120 bf16: 13.5 us a call, in two kernels 17.3).
    c.parts = rounds <= 4 ? std::min<int64_t>(rounds, 1) : std::min((rounds + 1) / 2, (int64_t)device_cus());
  } else {
    c.tpr = c.groups = 0;
    const int64_t col_groups = (cols + 2047) / 2048;
    const int64_t want = std::max<int64_t>(1, (int64_t)device_cus() * 8 / col_groups);
    c.parts = std::min<int64_t>((rows + 7) / 8, want);
  }
  return c;
}

template <typename X, typename D>
void backward(const void *dy, int64_t lddy, const void *x, int64_t ldx, const float *mean, const float *rstd,
              const void *w, int w_bf16, void *dx, int64_t lddx, void *dw, void *db, int g_bf16, void *workspace,
              int64_t rows, int64_t cols, hipStream_t stream) {
  const BackCut c = back_cut(rows, cols, sizeof(X) + sizeof(D) == 4);
  const D *dp = (const D *)dy;
  const X *xp = (const X *)x;
  X *op = (X *)dx;
  float *partial = (float *)workspace + (c.vpt ? 0 : 2 * rows);
  if (rows > 0 && c.vpt) {
    const size_t lds = (size_t)(c.groups - 1) * cols * sizeof(float);
    const auto launch = [&](auto kernel) {
      kernel<<<(unsigned)c.parts, c.tpr * c.groups, lds, stream>>>(dp, lddy, xp, ldx, mean, rstd, w, w_bf16, op, lddx,
                                                                  partial, dw, db, g_bf16, rows, cols, c.tpr,
                                                                  c.groups);
    };
    constexpr bool narrow = sizeof(X) + sizeof(D) == 4;
    with_flag(reads_once(rows * cols * (int64_t)(2 * sizeof(X) + sizeof(D))), [&](auto o) {
      if (c.vpt == 1) launch(k_ln_backward<X, D, 1, back_threads(1, narrow), o.value>);
      else if (c.vpt == 2) launch(k_ln_backward<X, D, 2, back_threads(2, narrow), o.value>);
      else if constexpr (narrow) launch(k_ln_backward<X, D, 4, back_threads(4, true), o.value>);
    });
  } else if (rows > 0) {
    float2 *sums = (float2 *)workspace;
    const int threads = any_width_threads(cols);
    k_ln_backward_rows<X, D><<<any_width_grid(rows, cols), threads, 0, stream>>>(dp, lddy, xp, ldx, mean, rstd, w, w_bf16,
                                                                                sums, rows, cols, threads);
    k_ln_backward_cols<X, D><<<dim3((unsigned)((cols + 2047) / 2048), (unsigned)c.parts), 256, 0, stream>>>(
        dp, lddy, xp, ldx, mean, rstd, w, w_bf16, sums, op, lddx, partial, rows, cols);
  }
  if ((dw || db) && !(rows > 0 && c.vpt && c.parts == 1)) {
    // a grid's threads are counted in 32 bits
    constexpr int64_t kMost = (int64_t)64 << 21;
    for (int64_t first = 0; first < 2 * cols; first += kMost)
      k_ln_backward_sum<<<(unsigned)((std::min(2 * cols - first, kMost) + 63) / 64), 64 * kShares, 0, stream>>>(
          partial, c.parts, cols, first, dw, db, g_bf16);
  }
}

}  // namespace

int64_t layer_norm_workspace_bytes(int64_t rows, int64_t cols) {
  const int64_t grid = forward_cut(rows, cols, true).grid;
  return grid > 1 ? 4 * grid : 0;
}

hipError_t launch_layer_norm(const void *x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, const void *w,
                             const void *b, int w_dtype, float eps, void *y, int y_dtype, int64_t ldy, float *mean,
                             float *rstd, float *amax, void *workspace, hipStream_t stream) {
  const ForwardCut c = forward_cut(rows, cols, amax != nullptr);
  // (a single workgroup's maximum is the tensor's)
  uint32_t *part = (uint32_t *)(amax && c.grid > 1 ? workspace : amax);
  if (rows > 0) {
    const int wb = w_dtype == 1;
    if (x_dtype == 1 && y_dtype == 1)
      forward<uint16_t, uint16_t>(c, x, ldx, w, b, wb, y, ldy, mean, rstd, part, rows, cols, eps, stream);
    else if (x_dtype == 1)
      forward<uint16_t, float>(c, x, ldx, w, b, wb, y, ldy, mean, rstd, part, rows, cols, eps, stream);
    else if (y_dtype == 1)
      forward<float, uint16_t>(c, x, ldx, w, b, wb, y, ldy, mean, rstd, part, rows, cols, eps, stream);
    else
      forward<float, float>(c, x, ldx, w, b, wb, y, ldy, mean, rstd, part, rows, cols, eps, stream);
  }
  if (amax && c.grid != 1) k_amax_join<<<1, kJoinThreads, 0, stream>>>(part, (int)c.grid, (uint32_t *)amax);
  return hipGetLastError();
}

int64_t layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  const auto need = [&](const BackCut &c) {
    return c.vpt ? (c.parts > 1 ? 8 * cols * c.parts : 0) : 8 * rows + 8 * cols * c.parts;
  };
  return std::max(need(back_cut(rows, cols, false)), need(back_cut(rows, cols, true)));     // whatever the types
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
