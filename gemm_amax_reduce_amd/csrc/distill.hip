// distill.hip -- distillation from a teacher's top logits for gfx950: the
// loss, its gradient, and both in one call.
//
//   p     = softmax(t / tau) over a row's valid entries (index inside the
//           vocabulary, teacher logit above -inf)
//   lse   = log sum_v exp(z_v / tau)
//   loss  = tau^2 sum_k p_k (log p_k - (z_{i_k} / tau - lse))
//   dz_v  = weight tau (exp(z_v / tau - lse) - sum_{k: i_k = v} p_k)
//
// A row without a valid entry has loss 0 and gradient 0 whatever z holds.
// Bound by HBM: the student's logits are read (and, for a gradient, written)
// once or twice, an exponential and some ten operations each; the teacher's
// lists are small.  Rows are cut into segments of the vocabulary, so that
// few rows still fill the GPU; each segment leaves its running maximum and
// sum, and the segments are joined in a fixed order.
#include "nvfp4_kernels.h"
#include "row_common.h"

#include <algorithm>

namespace nvfp4 {

namespace {

constexpr int kDT = 256;             // threads of a workgroup
constexpr int kMaxTop = 1024;        // entries of a teacher's list
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// Statistics of a set of logits: their maximum m, and the sum of
// 2^((z - m) scale) with scale = log2(e) / tau.  The difference comes before
// the product, so that logits of the type's lowest value do not overflow and
// large ones keep their digits.  join: of two disjoint sets.
__device__ __forceinline__ float2 join(float2 a, float2 b, float scale) {
  const float m = fmaxf(a.x, b.x);
  // nothing seen yet on either side: -inf - -inf would be NaN
  const float sa = a.x == m ? a.y : a.y * __builtin_amdgcn_exp2f((a.x - m) * scale);
  const float sb = b.x == m ? b.y : b.y * __builtin_amdgcn_exp2f((b.x - m) * scale);
  return make_float2(m, sa + sb);
}

// Statistics of one segment of one row.
template <typename T>
__global__ __launch_bounds__(kDT) void k_distill_stats(const T *z, int64_t ldz, int64_t V, int64_t seg_len,
                                                       float scale, float2 *part) {
  __shared__ float2 share[kDT / 64];
  const int64_t row = blockIdx.y, seg = blockIdx.x;
  const T *zr = z + row * ldz;
  const int64_t end = min(V, (seg + 1) * seg_len);
  float2 st = make_float2(-INFINITY, 0.0f);
  for (int64_t at = seg * seg_len + threadIdx.x * 8; at < end; at += kDT * 8) {
    Row8<T> q;
    load_row8(q, zr, at, end);
    float v[8];
    q.get(v);
    float m = st.x;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = at + i < end ? v[i] : -INFINITY;
      m = fmaxf(m, v[i]);
    }
    if (m > -INFINITY) {             // fmaxf passes a NaN by: it enters through the sum
      float s = st.x == m ? st.y : st.y * __builtin_amdgcn_exp2f((st.x - m) * scale);
#pragma unroll
      for (int i = 0; i < 8; ++i) s += __builtin_amdgcn_exp2f((v[i] - m) * scale);
      st = make_float2(m, s);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (v[i] != v[i]) st.y = v[i];
    }
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1)
    st = join(st, make_float2(__shfl_xor(st.x, off, 64), __shfl_xor(st.y, off, 64)), scale);
  if ((threadIdx.x & 63) == 0) share[threadIdx.x >> 6] = st;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kDT / 64; ++w) st = join(st, share[w], scale);
    part[row * gridDim.x + seg] = st;
  }
}

// A row's teacher list in LDS: the binary logarithm of p, and the index (-1
// where invalid); load_teacher returns whether any entry is valid.  p itself
// is 2^lp where it is used: log p taken from p would be -inf for the
// smallest shares.
struct Teacher {
  float lp[kMaxTop];
  int32_t at[kMaxTop];
  float share[2][kDT / 64];
};
__device__ __forceinline__ bool load_teacher(Teacher &te, const void *idx, int idx64, const void *t, int t_bf16,
                                             int64_t row, int top, int64_t V, float scale) {
  float m = -INFINITY;
  bool any = false;
  for (int k = threadIdx.x; k < top; k += kDT) {
    const int64_t e = row * top + k;
    const int64_t i = idx64 ? ((const int64_t *)idx)[e] : (int64_t)((const int32_t *)idx)[e];
    const float v = t_bf16 ? bf16_bits_f32(((const uint16_t *)t)[e]) : ((const float *)t)[e];
    const bool ok = i >= 0 && i < V && v != -INFINITY;
    te.at[k] = ok ? (int32_t)i : -1;
    te.lp[k] = v;
    if (ok) m = fmaxf(m, v);
    any |= ok;
  }
  m = wave_fmax(m);
  if ((threadIdx.x & 63) == 0) te.share[0][threadIdx.x >> 6] = m;
  const bool some = __syncthreads_or(any);
  for (int w = 0; w < kDT / 64; ++w) m = fmaxf(m, te.share[0][w]);
  float s = 0.0f;
  for (int k = threadIdx.x; k < top; k += kDT) {
    const float d = (te.lp[k] - m) * scale;
    te.lp[k] = d;
    s += te.at[k] >= 0 ? __builtin_amdgcn_exp2f(d) : 0.0f;
  }
  const float l = __builtin_amdgcn_logf(block_sum(s, te.share[1], kDT / 64));
  for (int k = threadIdx.x; k < top; k += kDT) te.lp[k] -= l;
  __syncthreads();
  return some;
}

__device__ __forceinline__ float share_of(float z, float top_z, float scale, float l2) {
  return __builtin_amdgcn_exp2f(__builtin_fmaf(z - top_z, scale, -l2));
}

// Loss and log-sum-exp of a row from its segments' statistics (part != null),
// and, with GRAD, the gradient of one segment.  Without part the log-sum-exp
// is read from lse and no loss is formed.  grid: (segments or 1, rows).
template <typename T, bool GRAD>
__global__ __launch_bounds__(kDT) void k_distill_finish(const T *z, int64_t ldz, int64_t V, int64_t seg_len,
                                                        int segments, const float2 *part, const void *idx, int idx64,
                                                        const void *t, int t_bf16, int top, float tau,
                                                        const float *weight, float *loss, float *lse, T *dz,
                                                        int64_t lddz) {
  __shared__ Teacher te;
  __shared__ float sums[kDT / 64];
  const int64_t row = blockIdx.y, seg = blockIdx.x;
  const float scale = kLog2e / tau;
  const T *zr = z + row * ldz;
  const bool some = load_teacher(te, idx, idx64, t, t_bf16, row, top, V, scale);
  // exp(z / tau - lse) = 2^((z - top) scale - l2)
  float top_z, l2;
  if (part) {
    float2 st = part[row * segments];
    for (int s = 1; s < segments; ++s) st = join(st, part[row * segments + s], scale);
    top_z = st.x;
    l2 = __builtin_amdgcn_logf(st.y);
    if (seg == 0) {
      float a = 0.0f;
      if (some)
        for (int k = threadIdx.x; k < top; k += kDT) {
          const float p = __builtin_amdgcn_exp2f(te.lp[k]);
          if (te.at[k] < 0 || p == 0.0f) continue;      // 0 log 0 = 0
          const float q = (to_float(zr[te.at[k]]) - top_z) * scale - l2;    // log2 of the student's share
          a = __builtin_fmaf(p, te.lp[k] - q, a);
        }
      a = block_sum(a, sums, kDT / 64);
      if (threadIdx.x == 0) {
        loss[row] = some ? tau * tau * kLn2 * a : 0.0f;
        lse[row] = top_z / tau + l2 * kLn2;
      }
    }
  } else {
    top_z = lse[row] * tau;
    l2 = 0.0f;
  }
  if (!GRAD) return;
  const float c = some ? weight[row] * tau : 0.0f;
  T *dr = dz + row * lddz;
  const int64_t begin = seg * seg_len, end = min(V, begin + seg_len);
  for (int64_t at = begin + threadIdx.x * 8; at < end; at += kDT * 8) {
    Row8<T> q;
    load_row8(q, zr, at, end);
    float v[8];
    q.get(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c == 0.0f ? 0.0f : c * share_of(v[i], top_z, scale, l2);
    q.set(v);
    store_row8(q, dr, at, end);
  }
  if (c == 0.0f) return;
  // the listed entries again, with the teacher's share; an index that is
  // listed twice takes the sum of its shares, in list order, so its writers
  // store the same value
  __syncthreads();
  for (int k = threadIdx.x; k < top; k += kDT) {
    const int32_t i = te.at[k];
    if (i < begin || i >= end) continue;
    float p = 0.0f;
    for (int j = 0; j < top; ++j)
      if (te.at[j] == i) p += __builtin_amdgcn_exp2f(te.lp[j]);
    const float g = c * (share_of(to_float(zr[i]), top_z, scale, l2) - p);
    store_one(dr + i, g);
  }
}

struct Split {
  int64_t seg_len;
  int segments;
};
// Segments of a row: enough workgroups to fill the GPU, none shorter than
// four loads of every thread, their starts at whole 8-element vectors.
Split split_for(int64_t T, int64_t V) {
  const int64_t vec = (int64_t)kDT * 8;
  const int64_t want = std::max<int64_t>(1, (int64_t)device_cus() * 8 / std::max<int64_t>(1, T));
  int64_t s = std::max<int64_t>(1, std::min<int64_t>(want, V / (4 * vec)));
  const int64_t len = ((V + s - 1) / s + vec - 1) / vec * vec;
  return {len, (int)((V + len - 1) / len)};
}

template <typename T>
void run(const void *z, int64_t rows, int64_t V, int64_t ldz, const void *idx, int idx64, const void *t, int t_bf16,
         int top, float tau, const float *weight, float *loss, float *lse, void *dz, int64_t lddz, void *workspace,
         bool stats, hipStream_t stream) {
  const Split sp = split_for(rows, V);
  float2 *part = stats ? (float2 *)workspace : nullptr;
  // rows on the grid's y dimension, 65535 at most per launch
  for (int64_t r = 0; r < rows; r += 65535) {
    const unsigned n = (unsigned)std::min<int64_t>(65535, rows - r);
    const T *zr = (const T *)z + r * ldz;
    const char *ir = (const char *)idx + r * top * (idx64 ? 8 : 4);
    const char *tr = (const char *)t + r * top * (t_bf16 ? 2 : 4);
    float2 *pr = part ? part + r * sp.segments : nullptr;
    if (stats)
      k_distill_stats<T><<<dim3(sp.segments, n), kDT, 0, stream>>>(zr, ldz, V, sp.seg_len, kLog2e / tau, pr);
    if (dz)
      k_distill_finish<T, true><<<dim3(sp.segments, n), kDT, 0, stream>>>(
          zr, ldz, V, sp.seg_len, sp.segments, pr, ir, idx64, tr, t_bf16, top, tau, weight + r,
          loss ? loss + r : nullptr, lse + r, (T *)dz + r * lddz, lddz);
    else
      k_distill_finish<T, false><<<dim3(1, n), kDT, 0, stream>>>(zr, ldz, V, sp.seg_len, sp.segments, pr, ir, idx64,
                                                                 tr, t_bf16, top, tau, nullptr, loss + r, lse + r,
                                                                 nullptr, 0);
  }
}

}  // namespace

int distill_max_top() { return kMaxTop; }

int64_t distill_workspace_bytes(int64_t rows, int64_t V) { return 8 * rows * split_for(rows, V).segments; }

hipError_t launch_distill(const void *z, int z_dtype, int64_t rows, int64_t V, int64_t ldz, const void *idx, int idx64,
                          const void *t, int t_dtype, int top, float tau, const float *weight, float *loss, float *lse,
                          void *dz, int64_t lddz, void *workspace, bool stats, hipStream_t stream) {
  if (rows > 0) {
    if (z_dtype == 1)
      run<uint16_t>(z, rows, V, ldz, idx, idx64, t, t_dtype == 1, top, tau, weight, loss, lse, dz, lddz, workspace,
                    stats, stream);
    else
      run<float>(z, rows, V, ldz, idx, idx64, t, t_dtype == 1, top, tau, weight, loss, lse, dz, lddz, workspace, stats,
                 stream);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
