// rms_norm.hip -- root-mean-square norm over the rows of a matrix for gfx950,
// with the residual's addition in front of it and its result in f32, bf16 or
// MXFP8; and the backward pass.
//
//   h = x + residual (rounded to the residual stream's type; x itself without one)
//   r = 1 / sqrt(sum h^2 / C + eps),  y = h w r
//   a = dy w,  n = h r:   dx = r (a - n sum(a n) / C) (+ dh),  dw = sum_rows dy n
//
// Every pass is bound by HBM: a row is read once and stays in registers (VPT
// vectors of 8 elements a thread) while its sum is reduced over the
// workgroup, and the next row is fetched meanwhile.  What is normed is h as
// it is stored, so that the backward pass, which reads it, sees the same.
// The products are formed as (h w) r: with bf16 h and w the first of them is
// exact in binary32, so an output before its own rounding carries one
// rounding and the error of r.
//
// MXFP8 blocks are 32 columns of a row: 4 lanes of 8 columns (8 lanes of 4
// where a matrix is f32), whose maximum takes two (three) exchanges inside a
// row of 16 lanes.  The result equals mxfp8_quantize of the f32 norm.
//
// Measured: one row of 5120 with a residual, bf16, 2.7 us; 4096 x 5120 bf16 with
// a float32 residual to MXFP8 46 us (230 MB at 5.0 TB/s, what a large copy
// reaches); backward 8192 x 5120 bf16 with the residual's gradient 61 us (5.5
// TB/s) and 5 us for adding up the workgroups' dw, 1537 x 5003 float32 18 us (5.1
// TB/s) and 4.
#include "mx8_scale.h"
#include "nvfp4_kernels.h"
#include "row_common.h"

#include <algorithm>

namespace nvfp4 {

namespace {

constexpr int kMaxThreads = 1024;
constexpr int kMaxWaves = kMaxThreads / 64;
// Threads of a workgroup by vectors a thread: four of them (with the next
// row's x and residual) do not fit 1024 threads' share of the registers.
constexpr int forward_threads(int vpt) { return vpt == 4 ? 768 : kMaxThreads; }

// Where a result goes: rows of f32 or bf16, or MXFP8 codes and scales.
template <typename Y> struct Out {
  Y *y;
  int64_t ldy;
};
struct Mx8 {};
template <> struct Out<Mx8> {
  uint8_t *codes, *scales;
  int64_t cols;
};

// The maximum of |v| over groups of 4 or 8 lanes, as bits (NaN on top).
template <int LANES> __device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));
  if (LANES == 8) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true));
  return v;
}
__device__ __forceinline__ uint32_t mx8_codes4(const float *v, float inv) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, lo, true);
}
__device__ __forceinline__ uint32_t absmax4(const float *v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

template <typename Y, bool SPLIT>
__device__ __forceinline__ void put(const Out<Y> &o, int64_t row, const float *v, const Piece<SPLIT> &p) {
  Row8<Y> q;
  q.set(v);
  store_piece(q, o.y + row * o.ldy, p);
}
// (cols % 32 == 0: the lanes of a block are all of the row or all past it)
__device__ __forceinline__ void put(const Out<Mx8> &o, int64_t row, const float *v, const Piece<false> &p) {
  const int e = mx8_exp(lanes_max<4>(max(absmax4(v), absmax4(v + 4))));
  const float inv = pow2f_mx8(-e);
  if (p.dup) return;
  *reinterpret_cast<uint2 *>(o.codes + row * o.cols + p.a) = make_uint2(mx8_codes4(v, inv), mx8_codes4(v + 4, inv));
  if (p.a % 32 == 0) o.scales[row * (o.cols / 32) + p.a / 32] = (uint8_t)(e + 127);
}
__device__ __forceinline__ void put(const Out<Mx8> &o, int64_t row, const float *v, const Piece<true> &p) {
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint32_t at = half ? p.b : p.a;
    const int e = mx8_exp(lanes_max<8>(absmax4(v + 4 * half)));
    if (half ? p.db : p.da) continue;
    *reinterpret_cast<uint32_t *>(o.codes + row * o.cols + at) = mx8_codes4(v + 4 * half, pow2f_mx8(-e));
    if (at % 32 == 0) o.scales[row * (o.cols / 32) + at / 32] = (uint8_t)(e + 127);
  }
}

// One workgroup per row, rows blockIdx.x, blockIdx.x + gridDim.x, ...  res
// and h may be one matrix: a row's loads have all arrived at its sum's barrier
// (or in its one wave), behind which it is stored.
template <typename X, typename R, typename Y, bool RES, int VPT, bool ONCE>
__global__ __launch_bounds__(forward_threads(VPT)) void k_rms_forward(const X *x, int64_t ldx, const R *res, int64_t ldr,
                                                                      R *h, int64_t ldh, const void *w, int w_bf16,
                                                                      Out<Y> out, float *rstd, int64_t rows,
                                                                      int64_t cols, float eps, int threads) {
  __shared__ float part[2][kMaxWaves];
  const int waves = threads >> 6;
  const float inv = 1.0f / (float)cols;
  constexpr bool kSplit = sizeof(X) > 2 || (RES && sizeof(R) > 2) || std::is_same<Y, float>::value;
  constexpr bool kHold = VPT <= 2;             // the weights stay in registers
  Piece<kSplit> sp[VPT];
  float wv[kHold ? VPT : 1][8];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    sp[j] = Piece<kSplit>(Piece<kSplit>::start(threadIdx.x + j * threads), (uint32_t)cols);
    if constexpr (kHold) param_piece(wv[j], w, w_bf16, sp[j], 1.0f);
  }
  int turn = 0;
  Row8<X> xn[VPT];
  Row8<R> rn[VPT];
  const auto fetch = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      load_piece<ONCE>(xn[j], x + row * ldx, sp[j]);
      if constexpr (RES) load_piece<ONCE>(rn[j], res + row * ldr, sp[j]);
    }
  };
  int64_t row = blockIdx.x;
  fetch(row);
  while (row < rows) {
    float v[VPT][8];
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      xn[j].get(v[j]);
      if constexpr (RES) {
        float u[8];
        rn[j].get(u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] += u[i];
        rn[j].set(v[j]);
        rn[j].get(v[j]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = sp[j].mine(i) ? v[j][i] : 0.0f;
        s = __builtin_fmaf(d, d, s);
      }
    }
    Row8<R> hv[VPT];
    if constexpr (RES) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) hv[j] = rn[j];
    }
    const int64_t later = row + gridDim.x;
    if (later < rows) fetch(later);
    __builtin_amdgcn_sched_barrier(0);       // the loads go out before this row's work, not after it
    const float r = 1.0f / __builtin_sqrtf(__builtin_fmaf(block_sum(s, part[turn], waves), inv, eps));
    if (threadIdx.x == 0) rstd[row] = r;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if constexpr (RES) store_piece(hv[j], h + row * ldh, sp[j]);
      float wr[8];
      if constexpr (!kHold) param_piece(wr, w, w_bf16, sp[j], 1.0f);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = v[j][i] * (kHold ? wv[kHold ? j : 0][i] : wr[i]) * r;
      put(out, row, v[j], sp[j]);
    }
    row = later;
    turn ^= 1;
  }
}

template <typename Y>
__device__ __forceinline__ void put_any(const Out<Y> &o, int64_t row, const float *v, int64_t at, int64_t cols) {
  Row8<Y> q;
  q.set(v);
  store_row8(q, o.y + row * o.ldy, at, cols);
}
__device__ __forceinline__ void put_any(const Out<Mx8> &o, int64_t row, const float *v, int64_t at, int64_t) {
  const int e = mx8_exp(lanes_max<4>(max(absmax4(v), absmax4(v + 4))));
  const float inv = pow2f_mx8(-e);
  *reinterpret_cast<uint2 *>(o.codes + row * o.cols + at) = make_uint2(mx8_codes4(v, inv), mx8_codes4(v + 4, inv));
  if (at % 32 == 0) o.scales[row * (o.cols / 32) + at / 32] = (uint8_t)(e + 127);
}

// Rows wider than the registers of a workgroup hold, or narrower than one
// vector: read twice, the second time (h, by the thread that wrote it) from
// the caches.
template <typename X, typename R, typename Y, bool RES>
__global__ __launch_bounds__(kMaxThreads) void k_rms_forward_any(const X *x, int64_t ldx, const R *res, int64_t ldr,
                                                                 R *h, int64_t ldh, const void *w, int w_bf16,
                                                                 Out<Y> out, float *rstd, int64_t rows, int64_t cols,
                                                                 float eps, int threads) {
  __shared__ float part[2][kMaxWaves];
  const int waves = threads >> 6;
  const int64_t step = (int64_t)threads * 8;
  const int64_t c0 = (int64_t)threadIdx.x * 8;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, turn ^= 1) {
    float s = 0.0f, v[8];
    for (int64_t at = c0; at < cols; at += step) {
      Row8<X> q;
      load_row8(q, x + row * ldx, at, cols);
      q.get(v);
      if constexpr (RES) {
        Row8<R> u;
        float uv[8];
        load_row8(u, res + row * ldr, at, cols);
        u.get(uv);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += uv[i];
        u.set(v);
        u.get(v);
        store_row8(u, h + row * ldh, at, cols);
      }
      float t = 0.0f;   // vector by vector, so that a long row's sum keeps its digits
#pragma unroll
      for (int i = 0; i < 8; ++i) t = __builtin_fmaf(v[i], v[i], t);
      s += t;
    }
    const float r = 1.0f / __builtin_sqrtf(block_sum(s, part[turn], waves) / (float)cols + eps);
    if (threadIdx.x == 0) rstd[row] = r;
    for (int64_t at = c0; at < cols; at += step) {
      if constexpr (RES) {
        Row8<R> q;
        load_row8(q, (const R *)h + row * ldh, at, cols);
        q.get(v);
      } else {
        Row8<X> q;
        load_row8(q, x + row * ldx, at, cols);
        q.get(v);
      }
      float wv[8];
      load_param8(wv, w, w_bf16, at, cols, 1.0f);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] * wv[i] * r;
      put_any(out, row, v, at, cols);
    }
  }
}

// Backward where a row fits the registers.  A workgroup has `groups` groups
// of `tpr` threads, each of which walks rows of its own: h and dy of a row are
// read once and stay in registers between the reduction of the row's sum and
// dx, the next row's are fetched meanwhile, and every thread adds up dw of its
// columns over all its rows.  At the end the groups' sums meet in LDS, and the
// workgroup leaves one partial row of dw, or, if it is the only one, dw itself.
// partial: [gridDim.x][cols]; dynamic LDS: (groups - 1) * cols floats.
template <typename X, typename D, bool DH, int VPT, int THREADS, bool ONCE>
__global__ __launch_bounds__(THREADS) void k_rms_backward(const D *dy, int64_t lddy, const X *x, int64_t ldx,
                                                          const float *rstd, const void *w, int w_bf16, const X *dh,
                                                          int64_t lddh, X *dx, int64_t lddx, float *partial,
                                                          void *dw_out, int g_bf16, int64_t rows, int64_t cols, int tpr,
                                                          int groups) {
  __shared__ float part[2][kMaxWaves];
  extern __shared__ float sums[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wpr = tpr >> 6;
  const int group = wave / wpr, t = threadIdx.x - group * tpr;
  const int64_t stride = (int64_t)gridDim.x * groups;
  const float inv = 1.0f / (float)cols;
  constexpr bool kSplit = sizeof(X) + sizeof(D) > 4;
  Piece<kSplit> sp[VPT];
  float wv[VPT][8], dw[VPT][8];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    sp[j] = Piece<kSplit>(Piece<kSplit>::start(t + j * tpr), (uint32_t)cols);
    param_piece(wv[j], w, w_bf16, sp[j], 1.0f);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.0f;
  }
  Row8<X> xn[VPT];
  Row8<D> dn[VPT];
  float rn;
  const auto fetch = [&](int64_t r) {
    r = min(r, rows - 1);              // (past the last row: fetched, not used)
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      load_piece<ONCE>(xn[j], x + r * ldx, sp[j]);
      load_piece<ONCE>(dn[j], dy + r * lddy, sp[j]);
    }
    rn = rstd[r];
  };
  int64_t row = (int64_t)blockIdx.x * groups + group;
  fetch(row);
  // the workgroup's groups make the same number of turns (barriers)
  int turn = 0;
  for (int64_t first = (int64_t)blockIdx.x * groups; first < rows; first += stride, row += stride, turn ^= 1) {
    const float r = rn;
    float s = 0.0f;
    Row8<X> xc[VPT], hc[VPT];
    Row8<D> dc[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      xc[j] = xn[j];
      dc[j] = dn[j];
      if constexpr (DH) load_piece<ONCE>(hc[j], dh + min(row, rows - 1) * lddh, sp[j]);
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
          const float n = xv[i] * r, a = dv[i] * wv[j][i];
          dw[j][i] = __builtin_fmaf(dv[i], n, dw[j][i]);
          s = sp[j].mine(i) ? __builtin_fmaf(a, n, s) : s;
        }
      }
    }
    s = wave_sum(s);
    if (wpr > 1) {
      if ((threadIdx.x & 63) == 0) part[turn][wave] = s;
      __syncthreads();
      s = 0.0f;
      for (int i = 0; i < wpr; ++i) s += part[turn][group * wpr + i];
    }
    s *= inv;
    if (row < rows) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        float o[8], xv[8], dv[8], hv[8];
        xc[j].get(xv);
        dc[j].get(dv);
        if constexpr (DH) hc[j].get(hv);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float d = __builtin_fmaf(dv[i], wv[j][i], -(xv[i] * r) * s);
          o[i] = DH ? __builtin_fmaf(d, r, hv[i]) : d * r;
        }
        Row8<X> q;
        q.set(o);
        store_piece(q, dx + row * lddx, sp[j]);
      }
    }
  }
  if (groups > 1) {
    __syncthreads();
    if (group > 0) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        Row8<float> q;
        q.set(dw[j]);
        store_piece(q, sums + (int64_t)(group - 1) * cols, sp[j]);
      }
    }
    __syncthreads();
  }
  if (group == 0) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      for (int g = 1; g < groups; ++g) {
        Row8<float> q;
        float u[8];
        load_piece(q, sums + (int64_t)(g - 1) * cols, sp[j]);
        q.get(u);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[j][i] += u[i];
      }
      void *const out = gridDim.x > 1 ? partial + (int64_t)blockIdx.x * cols : dw_out;
      if (!out) continue;
      if (gridDim.x == 1 && g_bf16) {
        Row8<uint16_t> q;
        q.set(dw[j]);
        store_piece(q, (uint16_t *)out, sp[j]);
      } else {
        Row8<float> q;
        q.set(dw[j]);
        store_piece(q, (float *)out, sp[j]);
      }
    }
  }
}

// Any width, first kernel: the row sum.
template <typename X, typename D>
__global__ __launch_bounds__(kMaxThreads) void k_rms_backward_rows(const D *dy, int64_t lddy, const X *x, int64_t ldx,
                                                                   const float *rstd, const void *w, int w_bf16,
                                                                   float *sums, int64_t rows, int64_t cols,
                                                                   int threads) {
  __shared__ float part[2][kMaxWaves];
  const int waves = threads >> 6;
  const int64_t step = (int64_t)threads * 8;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, turn ^= 1) {
    const float r = rstd[row];
    float s = 0.0f;
    for (int64_t at = (int64_t)threadIdx.x * 8; at < cols; at += step) {
      Row8<X> qx;
      Row8<D> qd;
      load_row8(qx, x + row * ldx, at, cols);
      load_row8(qd, dy + row * lddy, at, cols);
      float xv[8], dv[8], wv[8];
      qx.get(xv);
      qd.get(dv);
      load_param8(wv, w, w_bf16, at, cols, 1.0f);
      float t = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) t = __builtin_fmaf(dv[i] * wv[i], xv[i] * r, t);
      s += t;
    }
    const float mean = block_sum(s, part[turn], waves) / (float)cols;
    if (threadIdx.x == 0) sums[row] = mean;
  }
}

// Any width, second kernel: dx, and this workgroup's rows' share of dw for its
// 2048 columns.  partial: [gridDim.y][cols].
template <typename X, typename D>
__global__ __launch_bounds__(256) void k_rms_backward_cols(const D *dy, int64_t lddy, const X *x, int64_t ldx,
                                                           const float *rstd, const void *w, int w_bf16,
                                                           const float *sums, const X *dh, int64_t lddh, X *dx,
                                                           int64_t lddx, float *partial, int64_t rows, int64_t cols) {
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (at >= cols) return;
  float wv[8], dw[8];
  load_param8(wv, w, w_bf16, at, cols, 1.0f);
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = 0.0f;
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const float r = rstd[row], s = sums[row];
    Row8<X> qx, qh;
    Row8<D> qd;
    load_row8(qx, x + row * ldx, at, cols);
    load_row8(qd, dy + row * lddy, at, cols);
    if (dh) load_row8(qh, dh + row * lddh, at, cols);
    else qh.zero();
    float xv[8], dv[8], hv[8];
    qx.get(xv);
    qd.get(dv);
    qh.get(hv);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n = xv[i] * r;
      dw[i] = __builtin_fmaf(dv[i], n, dw[i]);
      xv[i] = __builtin_fmaf(__builtin_fmaf(dv[i], wv[i], -n * s), r, hv[i]);
    }
    qx.set(xv);
    store_row8(qx, dx + row * lddx, at, cols);
  }
  Row8<float> q;
  q.set(dw);
  store_row8(q, partial + (int64_t)blockIdx.y * cols, at, cols);
}

// dw from the partial rows, in a fixed order: 64 columns per workgroup (from
// `first` on), 16 interleaved shares of the rows, added at the end.
constexpr int kShares = 16;
__global__ __launch_bounds__(64 * kShares) void k_rms_backward_sum(const float *partial, int64_t parts, int64_t cols,
                                                                   int64_t first, void *dw, int g_bf16) {
  __shared__ float share[kShares][64];
  const int lane = threadIdx.x & 63, group = threadIdx.x >> 6;
  const int64_t c = first + (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int64_t k = group; k < parts; k += kShares) s += partial[k * cols + c];
  }
  share[group][lane] = s;
  __syncthreads();
  if (group == 0 && c < cols) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < kShares; ++i) s += share[i][lane];
    if (g_bf16) ((uint16_t *)dw)[c] = (uint16_t)pack_bf16(s, 0.0f);
    else ((float *)dw)[c] = s;
  }
}

int threads_for(int64_t vectors, int vpt, int most) {
  const int64_t t = (vectors + vpt - 1) / vpt;
  return (int)std::min<int64_t>(most, (t + 63) / 64 * 64);
}
// The kernels that take any width: 32 waves a CU, one wave a row below 8 columns.
int any_width_threads(int64_t cols) { return cols < 8 ? 64 : kMaxThreads; }
unsigned any_width_grid(int64_t rows, int64_t cols) {
  return (unsigned)std::min<int64_t>(rows, (int64_t)device_cus() * (32 * 64 / any_width_threads(cols)));
}

// How a forward pass is cut: vectors per thread (0 = the kernel for any
// width), threads and number of the workgroups: one round of them, 16 waves a
// CU.
struct ForwardCut {
  int vpt, threads;
  unsigned grid;
};
ForwardCut forward_cut(int64_t rows, int64_t cols) {
  const int64_t vectors = (cols + 7) / 8;
  ForwardCut c;
  c.vpt = cols < 8                             ? 0
          : vectors <= 256                     ? 1
          : vectors <= 2 * forward_threads(2)  ? 2
          : vectors <= 4 * forward_threads(4)  ? 4
                                               : 0;
  c.threads = c.vpt ? threads_for(vectors, c.vpt, forward_threads(c.vpt)) : any_width_threads(cols);
  c.grid = c.vpt ? (unsigned)std::min<int64_t>(rows, (int64_t)device_cus() * std::max(1, 16 * 64 / c.threads))
                 : any_width_grid(rows, cols);
  return c;
}

template <typename X, typename R, typename Y, bool RES>
void forward(const RmsForward &a, const Out<Y> &out, hipStream_t stream) {
  const ForwardCut c = forward_cut(a.rows, a.cols);
  const auto launch = [&](auto kernel) {
    kernel<<<c.grid, c.threads, 0, stream>>>((const X *)a.x, a.ldx, (const R *)a.res, a.ldr, (R *)a.h, a.ldh, a.w,
                                             a.w_dtype == 1, out, a.rstd, a.rows, a.cols, a.eps, c.threads);
  };
  const int64_t each = sizeof(X) + (RES ? 2 * sizeof(R) : 0) + (std::is_same<Y, Mx8>::value ? 1 : sizeof(Y));
  with_flag(reads_once(a.rows * a.cols * each), [&](auto o) {
    if (c.vpt == 1) launch(k_rms_forward<X, R, Y, RES, 1, o.value>);
    else if (c.vpt == 2) launch(k_rms_forward<X, R, Y, RES, 2, o.value>);
    else if (c.vpt == 4) launch(k_rms_forward<X, R, Y, RES, 4, o.value>);
  });
  if (!c.vpt) launch(k_rms_forward_any<X, R, Y, RES>);
}
template <typename X, typename Y> void forward_x(const RmsForward &a, const Out<Y> &out, hipStream_t stream) {
  if (!a.res) forward<X, X, Y, false>(a, out, stream);
  else if (a.r_dtype == 1) forward<X, uint16_t, Y, true>(a, out, stream);
  else forward<X, float, Y, true>(a, out, stream);
}
template <typename Y> hipError_t forward_y(const RmsForward &a, const Out<Y> &out, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  if (a.x_dtype == 1) forward_x<uint16_t>(a, out, stream);
  else forward_x<float>(a, out, stream);
  return hipGetLastError();
}

// How a backward pass is cut: vectors per thread (0 = the two kernels for any
// width), threads a row, rows a workgroup works on at a time, and the partial
// rows of dw, one per workgroup (per workgroup row of the grid for any width).
struct BackCut {
  int vpt, tpr, groups;
  int64_t parts;
};
constexpr int back_threads(int vpt, bool narrow) { return vpt == 4 ? 512 : narrow ? 1024 : 768; }
BackCut back_cut(int64_t rows, int64_t cols, bool narrow) {      // narrow: h and dy are both bf16
  const int64_t vectors = (cols + 7) / 8;
  BackCut c;
  c.vpt = cols < 8 ? 0 : vectors <= 64 ? 1 : vectors <= 1024 ? 2 : vectors <= 2048 && narrow ? 4 : 0;
  if (c.vpt) {
    c.tpr = threads_for(vectors, c.vpt, back_threads(c.vpt, narrow));
    c.groups = std::max(1, back_threads(c.vpt, narrow) / c.tpr);
    const int64_t rounds = (rows + c.groups - 1) / c.groups;
    // one workgroup a CU, and two rounds for it at least; up to four rounds one
    // workgroup does without partial rows and the kernel that adds them
    c.parts = rounds <= 4 ? std::min<int64_t>(rounds, 1) : std::min((rounds + 1) / 2, (int64_t)device_cus());
  } else {
    c.tpr = c.groups = 0;
    const int64_t col_groups = (cols + 2047) / 2048;
    const int64_t want = std::max<int64_t>(1, (int64_t)device_cus() * 8 / col_groups);
    c.parts = std::min<int64_t>((rows + 7) / 8, want);
  }
  return c;
}

template <typename X, typename D> void backward(const RmsBackward &a, hipStream_t stream) {
  constexpr bool narrow = sizeof(X) + sizeof(D) == 4;
  const BackCut c = back_cut(a.rows, a.cols, narrow);
  const D *dy = (const D *)a.dy;
  const X *x = (const X *)a.h, *dh = (const X *)a.dh;
  X *dx = (X *)a.dx;
  float *partial = (float *)a.ws + (c.vpt ? 0 : a.rows);
  const int wb = a.w_dtype == 1, gb = a.g_dtype == 1;
  if (a.rows > 0 && c.vpt) {
    const size_t lds = (size_t)(c.groups - 1) * a.cols * sizeof(float);
    const auto launch = [&](auto kernel) {
      kernel<<<(unsigned)c.parts, c.tpr * c.groups, lds, stream>>>(dy, a.lddy, x, a.ldh, a.rstd, a.w, wb, dh, a.lddh, dx,
                                                                  a.lddx, partial, a.dw, gb, a.rows, a.cols, c.tpr,
                                                                  c.groups);
    };
    const int64_t each = (dh ? 3 : 2) * sizeof(X) + sizeof(D);
    with_flag(reads_once(a.rows * a.cols * each), [&](auto o) {
      with_flag(dh != nullptr, [&](auto d) {
        if (c.vpt == 1) launch(k_rms_backward<X, D, d.value, 1, back_threads(1, narrow), o.value>);
        else if (c.vpt == 2) launch(k_rms_backward<X, D, d.value, 2, back_threads(2, narrow), o.value>);
        else if constexpr (narrow) launch(k_rms_backward<X, D, d.value, 4, back_threads(4, true), o.value>);
      });
    });
  } else if (a.rows > 0) {
    float *sums = (float *)a.ws;
    const int threads = any_width_threads(a.cols);
    k_rms_backward_rows<X, D><<<any_width_grid(a.rows, a.cols), threads, 0, stream>>>(dy, a.lddy, x, a.ldh, a.rstd, a.w,
                                                                                      wb, sums, a.rows, a.cols, threads);
    k_rms_backward_cols<X, D><<<dim3((unsigned)((a.cols + 2047) / 2048), (unsigned)c.parts), 256, 0, stream>>>(
        dy, a.lddy, x, a.ldh, a.rstd, a.w, wb, sums, dh, a.lddh, dx, a.lddx, partial, a.rows, a.cols);
  }
  if (a.dw && !(a.rows > 0 && c.vpt && c.parts == 1)) {
    // a grid's threads are counted in 32 bits
    constexpr int64_t kMost = (int64_t)64 << 21;
    for (int64_t first = 0; first < a.cols; first += kMost)
      k_rms_backward_sum<<<(unsigned)((std::min(a.cols - first, kMost) + 63) / 64), 64 * kShares, 0, stream>>>(
          partial, c.parts, a.cols, first, a.dw, gb);
  }
}

}  // namespace

hipError_t launch_rms_norm(const RmsForward &a, void *y, int y_dtype, int64_t ldy, hipStream_t stream) {
  if (y_dtype == 1) return forward_y(a, Out<uint16_t>{(uint16_t *)y, ldy}, stream);
  return forward_y(a, Out<float>{(float *)y, ldy}, stream);
}
hipError_t launch_rms_norm_mx8(const RmsForward &a, uint8_t *codes, uint8_t *scales, hipStream_t stream) {
  return forward_y(a, Out<Mx8>{codes, scales, a.cols}, stream);
}

int64_t rms_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  const auto need = [&](const BackCut &c) {
    return c.vpt ? (c.parts > 1 ? 4 * cols * c.parts : 0) : 4 * (rows + cols * c.parts);
  };
  return std::max(need(back_cut(rows, cols, false)), need(back_cut(rows, cols, true)));     // whatever the types
}
hipError_t launch_rms_norm_backward(const RmsBackward &a, hipStream_t stream) {
  if (a.h_dtype == 1 && a.dy_dtype == 1) backward<uint16_t, uint16_t>(a, stream);
  else if (a.h_dtype == 1) backward<uint16_t, float>(a, stream);
  else if (a.dy_dtype == 1) backward<float, uint16_t>(a, stream);
  else backward<float, float>(a, stream);
  return hipGetLastError();
}

}  // namespace nvfp4
