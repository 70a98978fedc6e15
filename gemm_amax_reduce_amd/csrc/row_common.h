// row_common.h -- pieces shared by the kernels that walk rows of a bf16 or
// f32 matrix (layer norm, matrix-vector products, distillation): 8-element
// loads and stores at any element alignment, bf16 rounding that keeps NaN,
// wave and workgroup reductions.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// Rows may start at any element (odd widths, padded strides): gfx950 takes
// 16-byte global accesses at any address, so one form serves every row and
// the types only promise the element's own alignment.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
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

// A thread's 8 columns of rows of n >= 8 elements, from position at on.  Where
// they pass the row's end they are moved back onto its last 8, so that every
// load and store is a whole one: the first `dup` of them then belong to other
// threads as well, and only sums over the row have to leave them out (a
// duplicate store writes the same value).  dup = 8: all of them.
struct Span {
  int64_t at;
  int dup;
  Span() = default;
  __device__ __forceinline__ Span(int64_t from, int64_t n) {
    at = min(from, n - 8);
    dup = (int)min(from - at, (int64_t)8);
  }
  __device__ __forceinline__ bool mine(int i) const { return i >= dup; }
};

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
