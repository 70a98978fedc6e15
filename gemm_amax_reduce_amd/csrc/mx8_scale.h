// mx8_scale.h -- the block scale of MXFP8, for the kernels that write it.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

// Smallest e with amax <= 448 * 2^e for the bit pattern of amax >= 0:
// 448 * 2^e = 1.75 * 2^(e+8), so for amax = m * 2^E (m in [1, 2)) e = E - 8
// when m <= 1.75 and E - 7 otherwise; zero and subnormal maxima fit e = -127.
__device__ __forceinline__ int mx8_exp(uint32_t amax_bits) {
  if (amax_bits < 0x00800000u) return -127;
  const int E = (int)(amax_bits >> 23) - 127;
  const int e = (amax_bits & 0x7FFFFFu) <= 0x600000u ? E - 8 : E - 7;
  return e < -127 ? -127 : (e > 127 ? 127 : e);
}

// 2^n as binary32 for n in [-127, 127] (2^-127 is subnormal).
__device__ __forceinline__ float pow2f_mx8(int n) {
  return n >= -126 ? __uint_as_float((uint32_t)(n + 127) << 23) : __uint_as_float(0x00400000u);
}

}  // namespace nvfp4
