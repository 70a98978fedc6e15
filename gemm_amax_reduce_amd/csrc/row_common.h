// row_common.h -- pieces shared by the kernels that walk rows of a bf16 or
// f32 matrix (layer norm, matrix-vector products, distillation): 8-element
// loads and stores at any element alignment, bf16 rounding that keeps NaN,
// wave and workgroup reductions.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace nvfp4 {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// Rows may start at any element (odd widths, padded strides): gfx950 takes
// 16-byte global accesses at any address, so one form serves every row and
// the types only promise the element's own alignment.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ float bf16_bits_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

__device__ __forceinline__ float to_float(uint16_t v) { return bf16_bits_f32(v); }
__device__ __forceinline__ float to_float(float v) { return v; }

// Two f32 to two bf16, nearest even, NaN kept (one v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2_t v = __builtin_convertvector((f32x2_t){a, b}, bf16x2_t);
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ void store_one(uint16_t *p, float v) { *p = (uint16_t)pack_bf16(v, 0.0f); }
__device__ __forceinline__ void store_one(float *p, float v) { *p = v; }

// 8 consecutive elements, as they lie in memory (load, store) and as f32
// (get, set).
template <typename T> struct Row8;
template <> struct Row8<uint16_t> {
  u32x4_a4 r;
  __device__ __forceinline__ void load(const uint16_t *p) { r = *reinterpret_cast<const u32x4_a2 *>(p); }
  // the first n < 8 elements, zero beyond
  __device__ __forceinline__ void load_part(const uint16_t *p, int n) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    r = (u32x4_a4){w[0], w[1], w[2], w[3]};
  }
  __device__ __forceinline__ void zero() { r = (u32x4_a4){0, 0, 0, 0}; }
  // Opaque to the compiler: what was computed from the raw bits before is
  // computed anew after it, instead of being kept in twice the registers.
  __device__ __forceinline__ void keep_packed() { asm volatile("" : "+v"(r)); }
  __device__ __forceinline__ void get(float *v) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(r[i] << 16);
      v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ void set(const float *v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  }
  __device__ __forceinline__ void store(uint16_t *p) const { *reinterpret_cast<u32x4_a2 *>(p) = r; }
  __device__ __forceinline__ void store_part(uint16_t *p, int n) const {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = (uint16_t)(r[i >> 1] >> (16 * (i & 1)));
  }
};
template <> struct Row8<float> {
  f32x4_a4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = *reinterpret_cast<const f32x4_a4 *>(p);
    b = *reinterpret_cast<const f32x4_a4 *>(p + 4);
  }
  __device__ __forceinline__ void load_part(const float *p, int n) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) v[i] = p[i];
    set(v);
  }
  __device__ __forceinline__ void zero() { a = b = (f32x4_a4){0, 0, 0, 0}; }
  __device__ __forceinline__ void keep_packed() {}
  __device__ __forceinline__ void get(float *v) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
  __device__ __forceinline__ void set(const float *v) {
    a = (f32x4_a4){v[0], v[1], v[2], v[3]};
    b = (f32x4_a4){v[4], v[5], v[6], v[7]};
  }
  __device__ __forceinline__ void store(float *p) const {
    *reinterpret_cast<f32x4_a4 *>(p) = a;
    *reinterpret_cast<f32x4_a4 *>(p + 4) = b;
  }
  __device__ __forceinline__ void store_part(float *p, int n) const {
    float v[8];
    get(v);
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = v[i];
  }
};

// 8 elements of a row of n elements from position at; zero past the end.
template <typename T>
__device__ __forceinline__ void load_row8(Row8<T> &r, const T *row, int64_t at, int64_t n) {
  if (at + 8 <= n) r.load(row + at);
  else if (at < n) r.load_part(row + at, (int)(n - at));
  else r.zero();
}
template <typename T>
__device__ __forceinline__ void store_row8(const Row8<T> &r, T *row, int64_t at, int64_t n) {
  if (at + 8 <= n) r.store(row + at);
  else if (at < n) r.store_part(row + at, (int)(n - at));
}

// Whether a call that moves that many bytes reads its matrices past the
// caches' usual order (nontemporal): above the 256 MB that the last cache
// holds, what is read only pushes out what was written, which whoever is next
// reads.  Each followed by a pass over its result, us: layer norm backward of
// 32768 x 8192 bf16 518 -> 489, distillation's gradient of 4096 x 50016 bf16
// 340 -> 312, of 512 x 131072 f32 179 -> 154; 4096 x 5120 bf16, which fits,
// would go from 58 to 64.
inline bool reads_once(int64_t bytes) { return bytes > ((int64_t)256 << 20); }
// f(std::true_type) or f(std::false_type)
template <typename F> inline void with_flag(bool flag, F f) {
  if (flag) f(std::true_type());
  else f(std::false_type());
}

// A thread's 8 columns of rows of n >= 8 elements (n below 2^31), the q-th of
// the row.  16-bit types take 8 in a row, one 16-byte load.  With SPLIT, for
// kernels of which a matrix is f32, they are two times 4, and a wave's 512
// lie in two blocks of 256, lane after lane: each load then covers whole
// lines.  (32 bytes a lane in two loads leave every line to both of them: a
// copy like that reaches 5.1 TB/s, lane after lane 5.9.)
//
// Where columns would pass the row's end they are moved back onto its last 4
// or 8, so that every load and store is a whole one: the first of them then
// belong to other threads as well, and only sums over the row have to leave
// them out (a duplicate store writes the same value).
template <bool SPLIT> struct Piece;
template <> struct Piece<false> {
  uint32_t a;
  int dup;                       // how many of the 8 are others'
  Piece() = default;
  static __device__ __forceinline__ uint32_t start(uint32_t q) { return q * 8; }
  __device__ __forceinline__ Piece(uint32_t from, uint32_t n) {
    a = min(from, n - 8);
    dup = (int)min(from - a, 8u);
  }
  __device__ __forceinline__ bool mine(int i) const { return i >= dup; }
  // of two sums, over the first 4 and the last 4, where rows are whole pieces
  __device__ __forceinline__ float sum_mine(float lo, float hi) const { return dup ? 0.0f : lo + hi; }
};
template <> struct Piece<true> {
  uint32_t a, b;                 // positions of the first and the last 4
  int da, db;                    // how many of each are others'
  Piece() = default;
  static __device__ __forceinline__ uint32_t start(uint32_t q) { return (q & ~63u) * 8 + (q & 63u) * 4; }
  __device__ __forceinline__ Piece(uint32_t from, uint32_t n) {
    a = min(from, n - 4);
    b = min(from + 256, n - 4);
    da = (int)min(from - a, 4u);
    db = (int)min(from + 256 - b, 4u);
  }
  __device__ __forceinline__ bool mine(int i) const { return i < 4 ? i >= da : i - 4 >= db; }
  __device__ __forceinline__ float sum_mine(float lo, float hi) const { return (da ? 0.0f : lo) + (db ? 0.0f : hi); }
};
// ONCE: past the caches' usual order.  (A template's choice: two branches of
// one kernel are merged into the plain load.)
template <typename V, bool ONCE, typename T> __device__ __forceinline__ V load_as(const T *p) {
  const V *v = reinterpret_cast<const V *>(p);
  return ONCE ? __builtin_nontemporal_load(v) : *v;
}
template <bool ONCE = false, typename T>
__device__ __forceinline__ void load_piece(Row8<T> &r, const T *row, const Piece<false> &p) {
  if constexpr (sizeof(T) == 2) {
    r.r = load_as<u32x4_a2, ONCE>(row + p.a);
  } else {
    r.a = load_as<f32x4_a4, ONCE>(row + p.a);
    r.b = load_as<f32x4_a4, ONCE>(row + p.a + 4);
  }
}
template <bool ONCE = false, typename T>
__device__ __forceinline__ void load_piece(Row8<T> &r, const T *row, const Piece<true> &p) {
  if constexpr (sizeof(T) == 2) {
    const u32x2_a2 x = load_as<u32x2_a2, ONCE>(row + p.a), y = load_as<u32x2_a2, ONCE>(row + p.b);
    r.r = (u32x4_a4){x[0], x[1], y[0], y[1]};
  } else {
    r.a = load_as<f32x4_a4, ONCE>(row + p.a);
    r.b = load_as<f32x4_a4, ONCE>(row + p.b);
  }
}
template <typename T> __device__ __forceinline__ void store_piece(const Row8<T> &r, T *row, const Piece<false> &p) {
  if (p.dup < 8) r.store(row + p.a);
}
__device__ __forceinline__ void store_piece(const Row8<uint16_t> &r, uint16_t *row, const Piece<true> &p) {
  if (p.da < 4) *reinterpret_cast<u32x2_a2 *>(row + p.a) = (u32x2_a2){r.r[0], r.r[1]};
  if (p.db < 4) *reinterpret_cast<u32x2_a2 *>(row + p.b) = (u32x2_a2){r.r[2], r.r[3]};
}
__device__ __forceinline__ void store_piece(const Row8<float> &r, float *row, const Piece<true> &p) {
  if (p.da < 4) *reinterpret_cast<f32x4_a4 *>(row + p.a) = r.a;
  if (p.db < 4) *reinterpret_cast<f32x4_a4 *>(row + p.b) = r.b;
}
// Of a parameter vector of n elements (f32 or bf16 by a wave-uniform flag),
// `fill` where it is absent.
template <bool SPLIT>
__device__ __forceinline__ void param_piece(float *v, const void *p, int is_bf16, const Piece<SPLIT> &at, float fill) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = fill;
  if (!p) return;
  if (is_bf16) {
    Row8<uint16_t> r;
    load_piece(r, (const uint16_t *)p, at);
    r.get(v);
  } else {
    Row8<float> r;
    load_piece(r, (const float *)p, at);
    r.get(v);
  }
}

// A parameter vector (f32 or bf16 by a wave-uniform flag), 8 from position
// at, `fill` past the end and where the vector is absent.
__device__ __forceinline__ void load_param8(float *v, const void *p, int is_bf16, int64_t at, int64_t n, float fill) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = fill;
  if (!p || at >= n) return;
  if (is_bf16) {
    Row8<uint16_t> r;
    load_row8(r, (const uint16_t *)p, at, n);
    r.get(v);
  } else {
    Row8<float> r;
    load_row8(r, (const float *)p, at, n);
    r.get(v);
  }
}

// Reductions over the wave, the result in every lane: four exchanges inside a
// row of 16 lanes ride on the operation (DPP: pairs, quads, mirrored halves,
// mirrored rows), then the rows and the halves are swapped.  Both operands
// of a commutative operation only change places between lanes, so every
// lane has the same bits.
template <int CTRL> __device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <typename Op> __device__ __forceinline__ float wave_reduce(float v, Op op) {
  v = op(v, dpp<0xB1>(v));      // quad_perm 1,0,3,2
  v = op(v, dpp<0x4E>(v));      // quad_perm 2,3,0,1
  v = op(v, dpp<0x141>(v));     // row_half_mirror
  v = op(v, dpp<0x140>(v));     // row_mirror
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_int(v), __float_as_int(v), false, false);
  v = op(__int_as_float(p[0]), __int_as_float(p[1]));
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_int(v), __float_as_int(v), false, false);
  return op(__int_as_float(q[0]), __int_as_float(q[1]));
}
__device__ __forceinline__ float wave_sum(float v) {
  return wave_reduce(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float wave_fmax(float v) {
  return wave_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}

// The sum over the workgroup's `waves` waves, in every thread; the order of
// additions is fixed.  part: LDS, one float per wave; the caller leaves a
// barrier between two uses of the same array.  (The number of waves is an
// argument: blockDim reads as a vector load with its own wait on this
// target, and in a loop that would stall whatever is being fetched ahead.)
__device__ __forceinline__ float block_sum(float v, float *part, int waves) {
  v = wave_sum(v);
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < waves; ++i) s += part[i];
  return s;
}

}  // namespace nvfp4
