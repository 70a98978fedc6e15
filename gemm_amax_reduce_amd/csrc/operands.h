// operands.h -- operands of the products that leave activations unquantized:
// 4-bit weights and their block scales decoded to bf16, float32 activations
// as three bf16 parts.
#pragma once
#include "nvfp4_device.h"
#include "row_common.h"

namespace nvfp4 {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint16_t u16_a1 __attribute__((aligned(1)));

// The scales of a lane's 32 k, as loaded and as two factors (k 0-15, 16-31).
template <bool MX> struct Scale;
template <> struct Scale<false> {
  static constexpr int kPerByte = 16;
  uint32_t raw;
  __device__ __forceinline__ void load(const uint8_t *p) { raw = *reinterpret_cast<const u16_a1 *>(p); }
  __device__ __forceinline__ float lo() const { return __builtin_amdgcn_cvt_f32_fp8((int)raw, 0); }
  __device__ __forceinline__ float hi() const { return __builtin_amdgcn_cvt_f32_fp8((int)raw, 1); }
};
template <> struct Scale<true> {
  static constexpr int kPerByte = 32;
  uint32_t raw;
  __device__ __forceinline__ void load(const uint8_t *p) { raw = *p; }
  // 2^(e - 127); e = 0 is the denormal 2^-127 and e = 255 NaN (both by the next bit below the exponent's)
  __device__ __forceinline__ float lo() const {
    return __uint_as_float(raw << 23 | (raw - 1 < 254 ? 0u : 0x00400000u));
  }
  __device__ __forceinline__ float hi() const { return lo(); }
  // From 253 on a weight, at most 6 times as large, may pass bf16's range.  A
  // quarter of the scale, 2^-129 to 2^125, keeps all weights in it (the
  // smallest as denormals, exact).
  static constexpr uint32_t kFar = 253;
  __device__ __forceinline__ float quarter() const {
    return raw == 255 ? lo() : __builtin_amdgcn_ldexpf(1.0f, (int)raw - 129);
  }
};

// 8 codes (one word) as 8 bf16: NVFP4 codes times the block scale s (exact
// in f32 and in bf16), MXFP4 by the conversion's own power-of-two scale.
template <bool MX> __device__ __forceinline__ bf16x8_t decode8(uint32_t w, float s) {
  u32x4_t v;
  if (MX) {
    v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
    v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
    v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
    v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  } else {
    const float2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    const float2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const float2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
    const float2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    v[0] = pack_bf16(a.x * s, a.y * s);
    v[1] = pack_bf16(b.x * s, b.y * s);
    v[2] = pack_bf16(c.x * s, c.y * s);
    v[3] = pack_bf16(d.x * s, d.y * s);
  }
  return __builtin_bit_cast(bf16x8_t, v);
}

// The three bf16 parts of 8 float32 values, a pair in each word.
struct Parts {
  u32x4_t v[3];
};
__device__ __forceinline__ Parts split8(const f32x4_t &a, const f32x4_t &b) {
  constexpr uint32_t kHigh = 0xFFFF0000u;
  const float f[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  uint32_t hi[8];
  float r[8];
  float odd = 0.0f;                                  // NaN if a remainder is, so where an x is Inf or NaN
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi[i] = __float_as_uint(f[i]) & kHigh;
    r[i] = f[i] - __uint_as_float(hi[i]);
    odd += r[i];
  }
  if (odd != odd) {
    // an Inf or NaN goes whole into the first part (with the quiet bit set
    // for a NaN, whose payload may lie below), the others are 0 then
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (f[i] != f[i]) hi[i] |= 0x00400000u;
      if ((__float_as_uint(f[i]) & 0x7F800000u) == 0x7F800000u) r[i] = 0.0f;
    }
  }
  Parts out;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t r0 = __float_as_uint(r[2 * i]), r1 = __float_as_uint(r[2 * i + 1]);
    const float lo0 = r[2 * i] - __uint_as_float(r0 & kHigh), lo1 = r[2 * i + 1] - __uint_as_float(r1 & kHigh);
    out.v[0][i] = __builtin_amdgcn_perm(hi[2 * i + 1], hi[2 * i], 0x07060302u);
    out.v[1][i] = __builtin_amdgcn_perm(r1, r0, 0x07060302u);
    out.v[2][i] = __builtin_amdgcn_perm(__float_as_uint(lo1), __float_as_uint(lo0), 0x07060302u);
  }
  return out;
}

// The same with hi and mid rounded to nearest: what is left over after two
// parts is at most 2^-17 of the value (2^-15 above, on one side).
__device__ __forceinline__ Parts split8_nearest(const Row8<float> &q) {
  float f[8], rest[8];
  q.get(f);
  Parts out;
  float odd = 0.0f;                                // NaN if a part is not finite
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t p = pack_bf16(f[2 * i], f[2 * i + 1]);
    out.v[0][i] = p;
    rest[2 * i] = f[2 * i] - bf16_lo(p);
    rest[2 * i + 1] = f[2 * i + 1] - bf16_hi(p);
    odd += rest[2 * i] * 0.0f + rest[2 * i + 1] * 0.0f;
    p = pack_bf16(rest[2 * i], rest[2 * i + 1]);
    out.v[1][i] = p;
    out.v[2][i] = pack_bf16(rest[2 * i] - bf16_lo(p), rest[2 * i + 1] - bf16_hi(p));
  }
  // (an Inf or NaN, or a value that rounds beyond bf16's largest)
  if (odd != odd) return split8((f32x4_t)q.a, (f32x4_t)q.b);
  return out;
}

// 8 rows of a lane's column, from rows of bf16 in LDS `pitch` bytes apart, by
// two transposing reads: 16 lanes name 4 rows of 16 columns (each 4 columns of
// one row) and leave with those rows of a column each; the second read takes
// the next 4 rows.
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
__device__ __forceinline__ bf16x8_t lds_column(const char *from, int pitch) {
  const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)from);
  const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(from + 4 * pitch));
  return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// 8 elements as MFMA operands: a bf16 value, or the parts of a float32 one.
template <typename T> struct Operand;
template <> struct Operand<uint16_t> {
  static constexpr int kParts = 1;
  bf16x8_t v[1];
  __device__ __forceinline__ void set(const Row8<uint16_t> &q) { v[0] = __builtin_bit_cast(bf16x8_t, (u32x4_t)q.r); }
};
template <> struct Operand<float> {
  static constexpr int kParts = 3;
  bf16x8_t v[3];
  __device__ __forceinline__ void set(const Row8<float> &q) {
    const Parts p = split8_nearest(q);
#pragma unroll
    for (int i = 0; i < 3; ++i) v[i] = __builtin_bit_cast(bf16x8_t, p.v[i]);
  }
};
// acc += the product of two operands (of the parts those that count).
template <typename A, typename B>
__device__ __forceinline__ void multiply16(f32x4_t &acc, const Operand<A> &a, const Operand<B> &b) {
#pragma unroll
  for (int p = 0; p < Operand<A>::kParts; ++p)
#pragma unroll
    for (int q = 0; q < Operand<B>::kParts; ++q)
      if (p + q < 3) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[p], b.v[q], acc, 0, 0, 0);
}

}  // namespace nvfp4
