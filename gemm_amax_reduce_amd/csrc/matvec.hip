// matvec.hip -- products of a few rows of activations with a 4-bit weight
// matrix for gfx950 (the single-token form of the linear layer):
//
//   NVFP4   y[t][n] = g * sum_k x[t][k] * e2m1(code[n][k]) * e4m3(scale[n][k/16])
//   MXFP4   y[t][n] =     sum_k x[t][k] * e2m1(code[n][k]) * 2^(scale[n][k/32] - 127)
//
// The weights are read once and everything else is small, so the kernel is
// bound by the N * K / 2 bytes of codes and the scales beside them.  A tile
// is 16 weight rows; its waves split K in steps of 128 and multiply on the
// 16x16x32 bf16 MFMA with the weights as the A operand and up to 16 tokens
// as the B operand, so 1 to 16 tokens cost the same instructions.  A lane
// holds 32 consecutive k of one weight row -- one 16-byte load of codes, and
// whole scale groups -- and takes them in four MFMAs; the k order of an MFMA
// is free as long as both operands agree on it.
//
// A decoded weight q * S has at most 6 significant bits (2 of E2M1, 4 of
// E4M3) and an exponent in bf16's range, so it is exact in bf16, and so is
// bf16 x.  A float32 x is split into three bf16 parts, x = hi + mid + lo,
// each of 8 bits: exact for every value whose low part does not fall below
// the bf16 range.  Products are exact in binary32 and added there; the
// tensor scale g is applied once to the sum.
#include "nvfp4_device.h"
#include "nvfp4_kernels.h"
#include "row_common.h"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef u32x4_t u32x4_a8 __attribute__((aligned(8)));

constexpr int kTileRows = 16;    // weight rows of a tile
constexpr int kTokens = 16;      // tokens of a tile
constexpr int kStepK = 128;      // k of one wave step: 4 lanes a row, 32 each
constexpr int kMvWaves = 8;

// 8 codes (one word) times the group's scale as 8 bf16.
template <bool MX> struct Decode;
template <> struct Decode<false> {
  __device__ __forceinline__ static u32x4_t run(uint32_t w, float s) {
    const float2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    const float2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const float2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
    const float2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    return (u32x4_t){pack_bf16(a.x * s, a.y * s), pack_bf16(b.x * s, b.y * s), pack_bf16(c.x * s, c.y * s),
                     pack_bf16(d.x * s, d.y * s)};
  }
};
template <> struct Decode<true> {
  __device__ __forceinline__ static u32x4_t run(uint32_t w, float s) {
    const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
    const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
    const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
    const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
    return (u32x4_t){__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, c),
                     __builtin_bit_cast(uint32_t, d)};
  }
};

// 8 consecutive x as NP bf16 operands whose sum is x.
template <typename X> struct Parts;
template <> struct Parts<uint16_t> {
  static constexpr int kCount = 1;
  __device__ __forceinline__ static void load(u32x4_t *p, const uint16_t *x) {
    p[0] = *reinterpret_cast<const u32x4_a2 *>(x);
  }
};
template <> struct Parts<float> {
  static constexpr int kCount = 3;
  __device__ __forceinline__ static void load(u32x4_t *p, const float *x) {
    const f32x4_a4 a = *reinterpret_cast<const f32x4_a4 *>(x), b = *reinterpret_cast<const f32x4_a4 *>(x + 4);
    const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t hi[2], mid[2], lo[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float f = v[2 * i + j];
        hi[j] = __float_as_uint(f);
        // an Inf or NaN goes whole into the first part (its top bits with
        // the quiet bit set for a NaN), the others are 0 then
        const bool finite = (hi[j] & 0x7F800000u) != 0x7F800000u;
        if (f != f) hi[j] |= 0x00400000u;
        hi[j] &= 0xFFFF0000u;
        const float r = finite ? f - __uint_as_float(hi[j]) : 0.0f;
        mid[j] = __float_as_uint(r) & 0xFFFF0000u;
        lo[j] = __float_as_uint(r - __uint_as_float(mid[j])) & 0xFFFF0000u;
      }
      p[0][i] = (hi[0] >> 16) | hi[1];
      p[1][i] = (mid[0] >> 16) | mid[1];
      p[2][i] = (lo[0] >> 16) | lo[1];
    }
  }
};

template <bool MX, typename X>
__global__ __launch_bounds__(64 * kMvWaves) void k_matvec(const uint8_t *codes, const uint8_t *scales,
                                                          const float *meta, int64_t N, int64_t K, const X *x,
                                                          int64_t tokens, int64_t ldx, void *y, int y_bf16,
                                                          int64_t ldy) {
  constexpr int kGroup = MX ? 32 : 16;
  __shared__ f32x4_t part[kMvWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, quarter = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * kTileRows, t0 = (int64_t)blockIdx.y * kTokens;
  const int64_t n = min(n0 + r, N - 1);              // rows past the end repeat the last one and are not stored
  const uint8_t *crow = codes + n * (K / 2);
  const uint8_t *srow = scales + n * (K / kGroup);
  const bool token = t0 + r < tokens;
  const X *xrow = x + (token ? t0 + r : 0) * ldx;
  f32x4_t acc = {0, 0, 0, 0};
  for (int64_t k = (int64_t)wave * kStepK + quarter * 32; k - quarter * 32 < K; k += kMvWaves * kStepK) {
    u32x4_t c = {0, 0, 0, 0};
    float s0 = 0.0f, s1 = 0.0f;
    int words = 0;                                    // groups of 8 k that lie inside the row
    if (k + 32 <= K) {
      c = *reinterpret_cast<const u32x4_a8 *>(crow + k / 2);
      words = 4;
    } else if (!MX && k + 16 <= K) {
      const u32x2_t h = *reinterpret_cast<const u32x2_t *>(crow + k / 2);
      c = (u32x4_t){h[0], h[1], 0, 0};
      words = 2;
    }
    if (MX) {
      // 2^(e - 127) as a float; e = 0 is the denormal 2^-127
      if (words) {
        const uint32_t e = srow[k / 32];
        s0 = s1 = __uint_as_float(e ? e << 23 : 0x00400000u);
      }
    } else {
      if (words) s0 = e4m3_to_f32(srow[k / 16]);
      if (words == 4) s1 = e4m3_to_f32(srow[k / 16 + 1]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x4_t b[Parts<X>::kCount];
#pragma unroll
      for (int p = 0; p < Parts<X>::kCount; ++p) b[p] = (u32x4_t){0, 0, 0, 0};
      if (token && j < words) Parts<X>::load(b, xrow + k + 8 * j);
      const bf16x8_t a = __builtin_bit_cast(bf16x8_t, Decode<MX>::run(c[j], j < 2 ? s0 : s1));
#pragma unroll
      for (int p = 0; p < Parts<X>::kCount; ++p)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8_t, b[p]), acc, 0, 0, 0);
    }
  }
  // lane: token t0 + (lane & 15), weight rows n0 + 4 * (lane >> 4) + i
  part[wave][lane] = acc;
  __syncthreads();
  if (wave == 0 && token) {
    for (int w = 1; w < kMvWaves; ++w) acc += part[w][lane];
    const float g = MX ? 1.0f : meta[1];
    const int64_t nn = n0 + 4 * quarter;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (nn + i >= N) break;
      const float v = acc[i] * g;
      const int64_t at = (t0 + r) * ldy + nn + i;
      if (y_bf16) ((uint16_t *)y)[at] = (uint16_t)pack_bf16(v, 0.0f);
      else ((float *)y)[at] = v;
    }
  }
}

template <bool MX, typename X>
void matvec(const uint8_t *codes, const uint8_t *scales, const float *meta, int64_t N, int64_t K, const void *x,
            int64_t tokens, int64_t ldx, void *y, int y_bf16, int64_t ldy, hipStream_t stream) {
  const dim3 grid((unsigned)((N + kTileRows - 1) / kTileRows), (unsigned)((tokens + kTokens - 1) / kTokens));
  k_matvec<MX, X><<<grid, 64 * kMvWaves, 0, stream>>>(codes, scales, meta, N, K, (const X *)x, tokens, ldx, y, y_bf16,
                                                      ldy);
}

}  // namespace

hipError_t launch_matvec(bool mx, const uint8_t *codes, const uint8_t *scales, const float *meta, int64_t N, int64_t K,
                         const void *x, int x_dtype, int64_t tokens, int64_t ldx, void *y, int y_dtype, int64_t ldy,
                         hipStream_t stream) {
  if (N > 0 && tokens > 0) {
    const int yb = y_dtype == 1;
    if (mx && x_dtype == 1) matvec<true, uint16_t>(codes, scales, meta, N, K, x, tokens, ldx, y, yb, ldy, stream);
    else if (mx) matvec<true, float>(codes, scales, meta, N, K, x, tokens, ldx, y, yb, ldy, stream);
    else if (x_dtype == 1) matvec<false, uint16_t>(codes, scales, meta, N, K, x, tokens, ldx, y, yb, ldy, stream);
    else matvec<false, float>(codes, scales, meta, N, K, x, tokens, ldx, y, yb, ldy, stream);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
