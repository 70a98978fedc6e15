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
// lists are small.  A row that fits the registers of a workgroup is read once
// for everything.  Longer rows, and few of them, are cut into segments of the
// vocabulary, so that they fill the GPU; each segment leaves its running
// maximum and sum, and the segments are joined in a fixed order.
//
// Measured on one MI355X, kernels alone: whole rows, loss 24 x 32768 bf16 6.1
// us (1.6 MB: latency), 8192 x 32768 bf16 87 us (6.1 TB/s), loss and gradient
// 4096 x 131072 bf16 451 us (4.8 TB/s), 2048 x 50016 f32 172 us (4.8 TB/s); in
// segments, 777 x 50021 f32 statistics 26 us (5.9 TB/s), loss 4.3 to 4.9 us,
// gradient 58 us (5.4 TB/s), 1024 x 131072 bf16 loss 50 us (5.4 TB/s).
#include "nvfp4_kernels.h"
#include "row_common.h"

#include <algorithm>

namespace nvfp4 {

namespace {

constexpr int kDT = 256;             // threads of a segment's workgroup
constexpr int kRowThreads = 1024;    // threads of a row's workgroup, at most
constexpr int kMaxWaves = kRowThreads / 64;
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

// exp(z / tau - lse), with lse = top_z / tau + l2 ln 2
__device__ __forceinline__ float share_of(float z, float top_z, float scale, float l2) {
  return __builtin_amdgcn_exp2f(__builtin_fmaf(z - top_z, scale, -l2));
}

// f32 logits go by split pieces, so that loads and stores cover whole lines.
template <typename T> using Cols = Piece<sizeof(T) == 4>;
template <typename T> __device__ __forceinline__ bool is_ragged(int64_t n) { return n & (sizeof(T) == 4 ? 3 : 7); }

// The sum of 2^((v - m) scale) over 8 values, those of others left out; a NaN
// gives NaN.  m is finite: with -inf, of values all masked, -inf - -inf would
// be NaN.
template <bool SPLIT>
__device__ __forceinline__ float exp_sum8(const float *v, float m, float scale, const Piece<SPLIT> &p, bool ragged) {
  float e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = __builtin_amdgcn_exp2f((v[i] - m) * scale);
  if (!ragged) return p.sum_mine(((e[0] + e[1]) + e[2]) + e[3], ((e[4] + e[5]) + e[6]) + e[7]);
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += p.mine(i) ? e[i] : 0.0f;
  return s;
}

// A row's teacher list in LDS: the binary logarithm of p, and the index (-1
// where invalid).  p itself is 2^lp where it is used: log p taken from p
// would be -inf for the smallest shares.
// z: the student's logits at the list.
struct Teacher {
  alignas(16) int32_t at[kMaxTop];
  float lp[kMaxTop], z[kMaxTop];
  float share[2][kMaxWaves];
};
struct List {
  const void *idx, *t;
  int idx64, t_bf16, top;
  // the lists of the rows from `row` on
  List from(int64_t row) const {
    return {(const char *)idx + row * top * (idx64 ? 8 : 4), (const char *)t + row * top * (t_bf16 ? 2 : 4), idx64,
            t_bf16, top};
  }
  __device__ __forceinline__ int64_t index(int64_t row, int k) const {
    const int64_t e = row * top + k;
    return idx64 ? ((const int64_t *)idx)[e] : (int64_t)((const int32_t *)idx)[e];
  }
  __device__ __forceinline__ float logit(int64_t row, int k) const {
    const int64_t e = row * top + k;
    return t_bf16 ? bf16_bits_f32(((const uint16_t *)t)[e]) : ((const float *)t)[e];
  }
};
// The thread's first entry, fetched before anything else.
struct Entry {
  int64_t i = -1;
  float v = 0.0f;
  __device__ __forceinline__ Entry(const List &l, int64_t row) {
    if ((int)threadIdx.x < l.top) {
      i = l.index(row, threadIdx.x);
      v = l.logit(row, threadIdx.x);
    }
  }
};
// Returns whether any entry is valid; all threads see the list then.
template <typename T>
__device__ __forceinline__ bool load_teacher(Teacher &te, const List &l, Entry e, const T *zr, int64_t row, int64_t V,
                                             float scale, int threads) {
  const int waves = threads >> 6;
  float m = -INFINITY;
  bool any = false;
  for (int k = threadIdx.x; k < (l.top + 3) / 4 * 4; k += threads) {
    if (k >= l.top) {                  // filled up to whole vectors of four
      te.at[k] = -1;
      continue;
    }
    if (k != (int)threadIdx.x) {
      e.i = l.index(row, k);
      e.v = l.logit(row, k);
    }
    const bool ok = e.i >= 0 && e.i < V && e.v != -INFINITY;
    te.at[k] = ok ? (int32_t)e.i : -1;
    te.lp[k] = e.v;
    te.z[k] = ok ? to_float(zr[e.i]) : 0.0f;
    if (ok) m = fmaxf(m, e.v);
    any |= ok;
  }
  m = wave_fmax(m);
  if ((threadIdx.x & 63) == 0) te.share[0][threadIdx.x >> 6] = m;
  const bool some = __syncthreads_or(any);
  for (int w = 0; w < waves; ++w) m = fmaxf(m, te.share[0][w]);
  float s = 0.0f;
  for (int k = threadIdx.x; k < l.top; k += threads) {
    const float d = (te.lp[k] - m) * scale;
    te.lp[k] = d;
    s += te.at[k] >= 0 ? __builtin_amdgcn_exp2f(d) : 0.0f;
  }
  const float n = __builtin_amdgcn_logf(block_sum(s, te.share[1], waves));
  for (int k = threadIdx.x; k < l.top; k += threads) te.lp[k] -= n;
  __syncthreads();
  return some;
}

// The sum over the list of p (log2 p - log2 q).
__device__ __forceinline__ float list_sum(const Teacher &te, int top, float top_z, float scale, float l2, int threads) {
  float a = 0.0f;
  for (int k = threadIdx.x; k < top; k += threads) {
    const float p = __builtin_amdgcn_exp2f(te.lp[k]);
    if (te.at[k] < 0 || p == 0.0f) continue;      // 0 log 0 = 0
    const float q = (te.z[k] - top_z) * scale - l2;    // log2 of the student's share
    a = __builtin_fmaf(p, te.lp[k] - q, a);
  }
  return a;
}

// The gradient at the listed entries of [begin, end), stored over what the
// student's share alone gave.  An index that is listed twice takes the sum
// of its shares, in list order, so its writers store the same value.
template <typename T>
__device__ __forceinline__ void list_gradient(const Teacher &te, T *dr, int top, int64_t begin, int64_t end, float c,
                                              float top_z, float scale, float l2, int threads) {
  __syncthreads();
  for (int k = threadIdx.x; k < top; k += threads) {
    const int32_t i = te.at[k];
    if (i < begin || i >= end) continue;
    int same = 0;
#pragma unroll 4
    for (int j = 0; j < (top + 3) / 4; ++j) {
      const int4 a = *reinterpret_cast<const int4 *>(te.at + 4 * j);
      same += (a.x == i) + (a.y == i) + (a.z == i) + (a.w == i);
    }
    float p = 0.0f;
    if (same == 1) {
      p = __builtin_amdgcn_exp2f(te.lp[k]);
    } else {
      for (int j = 0; j < top; ++j) p += te.at[j] == i ? __builtin_amdgcn_exp2f(te.lp[j]) : 0.0f;
    }
    store_one(dr + i, c * (share_of(te.z[k], top_z, scale, l2) - p));
  }
}

// The thread's j-th piece of a row of V >= 8 elements.  `from` is made opaque
// before each use of all of them, so that a use computes the positions anew
// instead of keeping VPT of them.
template <typename T> struct Vectors {
  uint32_t from, step, n;
  __device__ __forceinline__ Vectors(int threads, int64_t V)
      : from(Cols<T>::start(threadIdx.x)), step(threads * 8), n((uint32_t)V) {}
  __device__ __forceinline__ void anew() { asm volatile("" : "+v"(from)); }
  __device__ __forceinline__ Cols<T> operator[](int j) const { return Cols<T>(from + j * step, n); }
};

// A whole row in the registers of one workgroup: read once, written once.
// Its vectors of 8 are dealt out VPT to a thread.  The list is fetched first
// and worked on while the row arrives.
template <typename T, int VPT, bool GRAD, bool ONCE>
__global__ __launch_bounds__(kRowThreads) void k_distill_row(const T *z, int64_t ldz, int64_t V, List list, float tau,
                                                             const float *weight, float *loss, float *lse, T *dz,
                                                             int64_t lddz, int threads) {
  __shared__ Teacher te;
  __shared__ float part[3][kMaxWaves];
  const int64_t row = blockIdx.x;
  const int waves = threads >> 6;
  const float scale = kLog2e / tau;
  const bool ragged = is_ragged<T>(V);
  const T *zr = z + row * ldz;
  const Entry first(list, row);
  Vectors<T> vec(threads, V);
  Row8<T> q[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) load_piece<ONCE>(q[j], zr, vec[j]);
  __builtin_amdgcn_sched_barrier(0);
  const bool some = load_teacher(te, list, first, zr, row, V, scale, threads);
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    float v[8];
    q[j].get(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, v[i]);
  }
  m = wave_fmax(m);
  if ((threadIdx.x & 63) == 0) part[0][threadIdx.x >> 6] = m;
  __syncthreads();
  for (int w = 0; w < waves; ++w) m = fmaxf(m, part[0][w]);
  float s = 0.0f;
  const float base = m > -INFINITY ? m : 0.0f;       // a row masked as a whole: its sum is 0
  vec.anew();
#pragma unroll
  for (int j = 0; j < VPT; ++j) q[j].keep_packed();
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    float v[8];
    q[j].get(v);
    s += exp_sum8(v, base, scale, vec[j], ragged);
  }
  s = block_sum(s, part[1], waves);
  const float l2 = __builtin_amdgcn_logf(s);
  float a = some ? list_sum(te, list.top, m, scale, l2, threads) : 0.0f;
  a = block_sum(a, part[2], waves);
  if (threadIdx.x == 0) {
    loss[row] = some ? tau * tau * kLn2 * a : 0.0f;
    lse[row] = m / tau + l2 * kLn2;
  }
  if (!GRAD) return;
  const float c = some ? weight[row] * tau : 0.0f;
  T *dr = dz + row * lddz;
  vec.anew();
#pragma unroll
  for (int j = 0; j < VPT; ++j) q[j].keep_packed();
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    float v[8];
    q[j].get(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c * share_of(v[i], m, scale, l2);
    if (c == 0.0f)                     // the same for the whole row: zeros even where a logit is NaN
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    q[j].set(v);
    store_piece(q[j], dr, vec[j]);
  }
  if (c != 0.0f) list_gradient(te, dr, list.top, 0, V, c, m, scale, l2, threads);
}

// Statistics of n logits by a workgroup of kDT threads, in every thread; kBatch
// vectors of a thread in flight together.  A vector that passes the end is
// moved back inside.  share: LDS.
constexpr int kBatch = 4;
template <typename T, bool ONCE>
__device__ __forceinline__ float2 span_stats(const T *zr, int64_t n, float scale, float2 *share) {
  float2 st = make_float2(-INFINITY, 0.0f);
  if (n < 8) {                       // less than a vector: an element a thread
    if ((int64_t)threadIdx.x < n) {
      const float v = to_float(zr[threadIdx.x]);
      st = v != v ? make_float2(-INFINITY, v) : make_float2(v, v > -INFINITY ? 1.0f : 0.0f);
    }
  } else {
    const bool ragged = is_ragged<T>(n);
    for (uint32_t at = 0; at < (uint32_t)n; at += kBatch * kDT * 8) {
      Row8<T> q[kBatch];
      Cols<T> sp[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        sp[j] = Cols<T>(at + j * kDT * 8 + Cols<T>::start(threadIdx.x), (uint32_t)n);
        load_piece<ONCE>(q[j], zr, sp[j]);
      }
      float m = st.x;
      float v[kBatch][8];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        q[j].get(v[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, v[j][i]);
      }
      // fmaxf passes a NaN by: it enters through the sum.  (m = -inf: all were
      // masked so far, and -inf - -inf would be NaN.)
      if (m > -INFINITY) {
        float s = st.x == m ? st.y : st.y * __builtin_amdgcn_exp2f((st.x - m) * scale);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) s += exp_sum8(v[j], m, scale, sp[j], ragged);
        st = make_float2(m, s);
      } else {
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (v[j][i] != v[j][i]) st.y = v[j][i];
      }
    }
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1)
    st = join(st, make_float2(__shfl_xor(st.x, off, 64), __shfl_xor(st.y, off, 64)), scale);
  if ((threadIdx.x & 63) == 0) share[threadIdx.x >> 6] = st;
  __syncthreads();
  st = share[0];
  for (int w = 1; w < kDT / 64; ++w) st = join(st, share[w], scale);
  return st;
}

// Without a gradient, for few rows, or for rows that registers do not hold:
// statistics of one segment of one row.
template <typename T, bool ONCE>
__global__ __launch_bounds__(kDT) void k_distill_stats(const T *z, int64_t ldz, int64_t V, int64_t seg_len,
                                                       float scale, float2 *part) {
  __shared__ float2 share[kDT / 64];
  const int64_t row = blockIdx.y, seg = blockIdx.x;
  const int64_t begin = seg * seg_len, n = min(V - begin, seg_len);
  const float2 st = span_stats<T, ONCE>(z + row * ldz + begin, n, scale, share);
  if (threadIdx.x == 0) part[row * gridDim.x + seg] = st;
}

// A saved log-sum-exp, rounded to binary32, leaves a share an error of
// |lse| 2^-23 of itself: 2^-11 here.  From there on (a row that lies as a whole
// at a mask's value, up to the type's lowest, whose lse may have overflowed)
// the gradient's workgroups form the row's statistics anew.
constexpr float kFarLse = 4096.0f;

// Loss and log-sum-exp of a row from its segments' statistics (part != null),
// and, with GRAD, the gradient of one segment.  Without part the log-sum-exp
// is read from lse and no loss is formed.  grid: (segments or 1, rows).
template <typename T, bool GRAD, bool ONCE>
__global__ __launch_bounds__(kDT) void k_distill_finish(const T *z, int64_t ldz, int64_t V, int64_t seg_len,
                                                        int segments, const float2 *part, List list, float tau,
                                                        const float *weight, float *loss, float *lse, T *dz,
                                                        int64_t lddz) {
  __shared__ Teacher te;
  __shared__ float sums[kDT / 64];
  const int64_t row = blockIdx.y, seg = blockIdx.x;
  const float scale = kLog2e / tau;
  const T *zr = z + row * ldz;
  const bool some = load_teacher(te, list, Entry(list, row), zr, row, V, scale, kDT);
  float top_z, l2;
  if (part) {
    float2 st = part[row * segments];
    for (int s = 1; s < segments; ++s) st = join(st, part[row * segments + s], scale);
    top_z = st.x;
    l2 = __builtin_amdgcn_logf(st.y);
    if (seg == 0) {
      float a = some ? list_sum(te, list.top, top_z, scale, l2, kDT) : 0.0f;
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
  if (!part && c != 0.0f && fabsf(lse[row]) >= kFarLse) {
    __shared__ float2 share[kDT / 64];
    const float2 st = span_stats<T, false>(zr, V, scale, share);
    top_z = st.x;
    l2 = __builtin_amdgcn_logf(st.y);
  }
  T *dr = dz + row * lddz;
  const int64_t begin = seg * seg_len, end = min(V, begin + seg_len), n = end - begin;
  const auto gradient = [&](Row8<T> &q) {
    float v[8];
    q.get(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c * share_of(v[i], top_z, scale, l2);
    if (c == 0.0f)                     // the same for the whole row: zeros even where a logit is NaN
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    q.set(v);
  };
  if (n < 8) {
    if (threadIdx.x == 0) {
      Row8<T> q;
      load_row8(q, zr + begin, 0, n);
      gradient(q);
      store_row8(q, dr + begin, 0, n);
    }
  } else {
    for (uint32_t at = 0; at < (uint32_t)n; at += kBatch * kDT * 8) {
      Row8<T> q[kBatch];
      Cols<T> sp[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        sp[j] = Cols<T>(at + j * kDT * 8 + Cols<T>::start(threadIdx.x), (uint32_t)n);
        load_piece<ONCE>(q[j], zr + begin, sp[j]);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        gradient(q[j]);
        store_piece(q[j], dr + begin, sp[j]);
      }
    }
  }
  if (c != 0.0f) list_gradient(te, dr, list.top, begin, end, c, top_z, scale, l2, kDT);
}

struct Split {
  int64_t seg_len;
  int segments;
};
// Segments of a row: enough workgroups to fill the GPU twice over (16 a CU;
// loss and gradient of 777 rows of 50021 f32: 1 segment 94 us, 2 85, 5 84, 10
// 83.5), a longer vocabulary at least
// one per 32768 elements, none shorter than four loads of every thread, their
// starts at whole 8-element vectors.
Split split_for(int64_t T, int64_t V) {
  const int64_t vec = (int64_t)kDT * 8;
  const int64_t want = std::max<int64_t>(V / 32768, (int64_t)device_cus() * 16 / std::max<int64_t>(1, T));
  const int64_t s = std::max<int64_t>(1, std::min<int64_t>(want, V / (4 * vec)));
  const int64_t len = ((V + s - 1) / s + vec - 1) / vec * vec;
  return {len, (int)((V + len - 1) / len)};
}

// Vectors per thread of the one-workgroup-a-row form; 0 where the segments'
// form is taken: rows that 1024 threads do not hold in 64 registers each, or
// shorter than a vector; and, of rows above 128 KB, a loss alone (2048 x 50016
// f32: 75 us in segments, 89 in rows) or too few for the CUs (24 x 65536 bf16
// with the gradient: 10.8 us in segments, 12.5 in rows; 128 rows 19.5 and
// 19.3, 512 rows 46 and 31).
int row_vectors(int64_t rows, int64_t V, int size, bool gradient) {
  const int64_t vectors = (V + 7) / 8;
  if (V < 8) return 0;
  if (V * size > (128 << 10) && (!gradient || rows < device_cus() / 2)) return 0;
  if (vectors <= 4 * 256) return 4;
  if (vectors <= 8 * kRowThreads) return 8;
  return vectors <= 16 * kRowThreads && size == 2 ? 16 : 0;
}

template <typename T, int VPT>
void rows_of(const T *z, int64_t rows, int64_t V, int64_t ldz, const List &list, float tau, const float *weight,
             float *loss, float *lse, T *dz, int64_t lddz, hipStream_t stream) {
  int threads = (int)(((V + 7) / 8 + VPT - 1) / VPT + 63) / 64 * 64;
  // two workgroups of 13 to 15 waves do not share a CU, two of 16 do (8192 x
  // 50016 bf16: loss 211 -> 165 us, with the gradient 368 -> 328)
  if (threads > 768) threads = kRowThreads;
  const bool once = reads_once(2 * rows * V * (int64_t)sizeof(T));
  with_flag(once, [&](auto o) {
    const auto launch = [&](auto kernel) {
      // a grid's threads are counted in 32 bits
      constexpr int64_t kMost = 1 << 21;
      for (int64_t r = 0; r < rows; r += kMost)
        kernel<<<(unsigned)std::min(rows - r, kMost), threads, 0, stream>>>(
            z + r * ldz, ldz, V, list.from(r), tau, dz ? weight + r : nullptr, loss + r, lse + r,
            dz ? dz + r * lddz : nullptr, lddz, threads);
    };
    if (dz) launch(k_distill_row<T, VPT, true, o.value>);
    else if constexpr (VPT < 16) launch(k_distill_row<T, VPT, false, o.value>);      // (longer rows: see row_vectors)
  });
}

template <typename T>
void run(const void *zv, int64_t rows, int64_t V, int64_t ldz, List list, float tau, const float *weight, float *loss,
         float *lse, void *dz, int64_t lddz, void *workspace, bool stats, hipStream_t stream) {
  const T *z = (const T *)zv;
  const int vpt = stats ? row_vectors(rows, V, sizeof(T), dz != nullptr) : 0;
  if (vpt == 4) rows_of<T, 4>(z, rows, V, ldz, list, tau, weight, loss, lse, (T *)dz, lddz, stream);
  else if (vpt == 8) rows_of<T, 8>(z, rows, V, ldz, list, tau, weight, loss, lse, (T *)dz, lddz, stream);
  else if (vpt == 16)
    rows_of<uint16_t, 16>((const uint16_t *)zv, rows, V, ldz, list, tau, weight, loss, lse, (uint16_t *)dz, lddz, stream);
  if (vpt) return;
  const Split sp = split_for(rows, V);
  const bool once = reads_once(2 * rows * V * (int64_t)sizeof(T));       // (after a loss comes its gradient)
  float2 *part = stats ? (float2 *)workspace : nullptr;
  // rows on the grid's y dimension, 65535 at most per launch
  for (int64_t r = 0; r < rows; r += 65535) {
    const unsigned n = (unsigned)std::min<int64_t>(65535, rows - r);
    const T *zr = z + r * ldz;
    const List lr = list.from(r);
    float2 *pr = part ? part + r * sp.segments : nullptr;
    with_flag(once, [&](auto o) {
      if (stats)
        k_distill_stats<T, o.value><<<dim3(sp.segments, n), kDT, 0, stream>>>(zr, ldz, V, sp.seg_len, kLog2e / tau, pr);
      if (dz)
        k_distill_finish<T, true, o.value><<<dim3(sp.segments, n), kDT, 0, stream>>>(
            zr, ldz, V, sp.seg_len, sp.segments, pr, lr, tau, weight + r, loss ? loss + r : nullptr, lse + r,
            (T *)dz + r * lddz, lddz);
    });
    if (!dz)
      k_distill_finish<T, false, false><<<dim3(1, n), kDT, 0, stream>>>(zr, ldz, V, sp.seg_len, sp.segments, pr, lr,
                                                                        tau, nullptr, loss + r, lse + r, nullptr, 0);
  }
}

}  // namespace

int distill_max_top() { return kMaxTop; }

int64_t distill_workspace_bytes(int64_t rows, int64_t V) {
  // none where every type's rows go whole through one workgroup
  return row_vectors(rows, V, 4, false) ? 0 : 8 * rows * split_for(rows, V).segments;
}

hipError_t launch_distill(const void *z, int z_dtype, int64_t rows, int64_t V, int64_t ldz, const void *idx, int idx64,
                          const void *t, int t_dtype, int top, float tau, const float *weight, float *loss, float *lse,
                          void *dz, int64_t lddz, void *workspace, bool stats, hipStream_t stream) {
  if (rows > 0) {
    const List list = {idx, t, idx64, t_dtype == 1, top};
    if (z_dtype == 1) run<uint16_t>(z, rows, V, ldz, list, tau, weight, loss, lse, dz, lddz, workspace, stats, stream);
    else run<float>(z, rows, V, ldz, list, tau, weight, loss, lse, dz, lddz, workspace, stats, stream);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
