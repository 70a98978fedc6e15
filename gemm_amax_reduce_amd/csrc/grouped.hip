// grouped.hip -- matrix products grouped by expert for gfx950: rows of
// unquantized activations, in ragged groups, each with 4-bit weights of its own
//
//   y[t][n] = g sum_k x[t][k] w_e[n][k]      for t in group e
//
// and the gradient of the weights, dw_e[n][k] = sum over t in group e of
// dy[t][n] x[t][k].
//
// Weights are decoded to bf16, where e2m1(code) e4m3(scale) is exact, and
// multiplied on the 32x32x16 bf16 MFMA with the weights as the A operand, so
// that a lane ends up with 16 consecutive n of a token; float32 activations
// are three bf16 parts.  A workgroup's tile is 128 NF weight rows (its four
// waves have NF fragments of 32 each, so every weight is decoded by one wave)
// by 32 MF tokens, which all of its waves read from LDS.
#include "gemm_common.h"
#include "groups.h"
#include "nvfp4_kernels.h"
#include "operands.h"

#include <algorithm>
#include <type_traits>

namespace nvfp4 {

namespace {

typedef uint32_t u32x4_a8 __attribute__((ext_vector_type(4), aligned(8)));
typedef uint32_t u32x2_a8 __attribute__((ext_vector_type(2), aligned(8)));

constexpr int kThreads = 256;
constexpr int kStage = 128;                        // k of one LDS buffer
constexpr int kXcds = 8;

// Where a call's weights lie: expert e's row n starts at n * pitch + e * step
// bytes of codes (experts one after the other, or side by side in each row).
struct Stack {
  const uint8_t *codes, *scales;
  const float *meta;
  int64_t N, K;
  int64_t code_pitch, code_step, scale_pitch, scale_step;
};

template <typename X> struct Rows {
  const X *p;
  int64_t ld;
};

// 16 outputs n .. n + 15 of a token, none from N on.
__device__ __forceinline__ void store16(void *y, int y_bf16, int64_t row, int64_t n, int64_t N, const float *v) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (y_bf16) {
      Row8<uint16_t> q;
      q.set(v + 8 * i);
      store_row8(q, (uint16_t *)y + row, n + 8 * i, N);
    } else {
      Row8<float> q;
      q.set(v + 8 * i);
      store_row8(q, (float *)y + row, n + 8 * i, N);
    }
  }
}

// Zeros in the rows of y that no group has.
__device__ void zero_rest(const Groups &g, void *y, int y_bf16, int64_t ldy, int64_t N) {
  const int64_t first = g.at(0), last = max(g.at(g.count), first), rest = first + g.rows - last;
  for (int64_t i = blockIdx.x; i < rest; i += gridDim.x) {
    const int64_t row = (i < first ? i : last + i - first) * ldy;
    for (int64_t n = threadIdx.x; n < N; n += blockDim.x) {
      if (y_bf16) ((uint16_t *)y)[row + n] = 0;
      else ((float *)y)[row + n] = 0.0f;
    }
  }
}

// XP: bf16 parts of an activation (1: bf16, 3: float32).
template <bool MX, typename X, int NF, int MF>
__global__ __launch_bounds__(kThreads, NF * MF >= 16 ? 1 : NF * MF >= 4 ? 2 : 4) void
k_grouped(Stack w, Groups g, Rows<X> x, void *y, int y_bf16, int64_t ldy, int tiles_n, int fill) {
  constexpr int kXP = sizeof(X) == 2 ? 1 : 3;
  constexpr int BN = 128 * NF, BM = 32 * MF;
  constexpr int kG = Scale<MX>::kPerByte, kSB = kStage / kG;        // scale bytes of a row and stage
  constexpr int kCodes = BN * kStage / 2, kScales = BN * 8, kPart = BM * kStage * 2;
  constexpr int kBuffer = kCodes + kScales + kXP * kPart;
  constexpr int kCL = BN * 4 / kThreads;                            // 16-byte pieces of codes a thread loads
  constexpr int kXL = BM * 16 / kThreads;                           // 8-element pieces of x
  constexpr int kSL = (BN + kThreads - 1) / kThreads;               // scale rows
  __shared__ __align__(16) char lds[2 * kBuffer];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5;

  if (fill) zero_rest(g, y, y_bf16, ldy, w.N);
  const int total = count_tiles(g, BM) * tiles_n;
  // workgroups are dealt to the XCDs in turn: each gets a run of tiles
  const int quota = (total + kXcds - 1) / kXcds, local = blockIdx.x / kXcds;
  const int index = (int)(blockIdx.x % kXcds) * quota + local;
  if (local >= quota || index >= total) return;
  const GroupTile t = find_tile(g, BM, tiles_n, index);
  if (t.e < 0) return;
  // up to 8 tiles of tokens with one tile of weights after the other
  const int per = 8 * tiles_n, first_m = t.local / per * 8, gsz = min(t.tiles - first_m, 8);
  const int64_t m0 = t.begin + (int64_t)(first_m + t.local % per % gsz) * BM;
  const int64_t n0 = (int64_t)(t.local % per / gsz) * BN;

  const int stages = (int)((w.K + kStage - 1) / kStage);
  const uint8_t *const codes = w.codes + t.e * w.code_step, *const scales = w.scales + t.e * w.scale_step;

  // ---- from memory to registers
  const uint8_t *crow[kCL], *srow[kSL];
  const X *xrow[kXL];
  bool live[kXL];
#pragma unroll
  for (int i = 0; i < kCL; ++i)
    crow[i] = codes + min(n0 + (tid + i * kThreads) / 4, w.N - 1) * w.code_pitch + 16 * (tid & 3);
#pragma unroll
  for (int i = 0; i < kSL; ++i) srow[i] = scales + min(n0 + tid + i * kThreads, w.N - 1) * w.scale_pitch;
#pragma unroll
  for (int i = 0; i < kXL; ++i) {
    const int64_t row = m0 + tid / 16 + 16 * i;
    live[i] = row < t.end;
    xrow[i] = x.p + min(row, t.end - 1) * x.ld + 8 * (tid & 15);
  }
  u32x4_t creg[kCL];
  uint64_t sreg[kSL];
  Row8<X> xreg[kXL];
  const auto load = [&](int s) {
    const int64_t k0 = (int64_t)s * kStage;
    if (k0 + kStage <= w.K) {
#pragma unroll
      for (int i = 0; i < kCL; ++i) creg[i] = *reinterpret_cast<const u32x4_a8 *>(crow[i] + k0 / 2);
#pragma unroll
      for (int i = 0; i < kSL; ++i) {
        sreg[i] = 0;
        __builtin_memcpy(&sreg[i], srow[i] + k0 / kG, kSB);
      }
#pragma unroll
      for (int i = 0; i < kXL; ++i) xreg[i].load(xrow[i] + k0);
    } else {
      // the last stage of K % 128 != 0: zeros past K (a scale of 1 for MXFP4)
      const int64_t left = w.K - k0;
#pragma unroll
      for (int i = 0; i < kCL; ++i) {
        const int at = 32 * (tid & 3);
        u32x2_a8 lo = {0, 0}, hi = {0, 0};
        if (at < left) lo = *reinterpret_cast<const u32x2_a8 *>(crow[i] + k0 / 2);
        if (at + 16 < left) hi = *reinterpret_cast<const u32x2_a8 *>(crow[i] + k0 / 2 + 8);
        creg[i] = (u32x4_t){lo[0], lo[1], hi[0], hi[1]};
      }
#pragma unroll
      for (int i = 0; i < kSL; ++i) {
        sreg[i] = MX ? 0x7F7F7F7F7F7F7F7Full : 0;
        for (int b = 0; b < kSB; ++b)
          if (b * kG < left) sreg[i] = (sreg[i] & ~(0xFFull << (8 * b))) | (uint64_t)srow[i][k0 / kG + b] << (8 * b);
      }
#pragma unroll
      for (int i = 0; i < kXL; ++i) {
        if (8 * (tid & 15) < left) xreg[i].load(xrow[i] + k0);
        else xreg[i].zero();
      }
    }
  };

  // ---- from registers to LDS.  Codes: 4 pieces a row, piece c in slot
  // c ^ (row / 16 % 4); x: 16 pieces a row, piece p in slot p ^ (row % 16): the
  // 8 lanes of a 16-byte read that go together fall on all banks.
  const auto put = [&](int s) {
    char *const buf = lds + (s & 1) * kBuffer;
#pragma unroll
    for (int i = 0; i < kCL; ++i) {
      const int row = (tid + i * kThreads) / 4;
      *reinterpret_cast<u32x4_t *>(buf + row * 64 + 16 * ((tid & 3) ^ ((row >> 4) & 3))) = creg[i];
    }
#pragma unroll
    for (int i = 0; i < kSL; ++i)
      if (BN % kThreads == 0 || tid + i * kThreads < BN)
        *reinterpret_cast<uint64_t *>(buf + kCodes + (tid + i * kThreads) * 8) = sreg[i];
#pragma unroll
    for (int i = 0; i < kXL; ++i) {
      const int row = tid / 16 + 16 * i;
      char *const at = buf + kCodes + kScales + row * 256 + 16 * ((tid & 15) ^ (row & 15));
      if constexpr (kXP == 1) {
        *reinterpret_cast<u32x4_t *>(at) = live[i] ? (u32x4_t)xreg[i].r : (u32x4_t){0, 0, 0, 0};
      } else {
        if (!live[i]) xreg[i].zero();
        const Parts q = split8((f32x4_t)xreg[i].a, (f32x4_t)xreg[i].b);
#pragma unroll
        for (int p = 0; p < 3; ++p) *reinterpret_cast<u32x4_t *>(at + p * kPart) = q.v[p];
      }
    }
  };

  // ---- a stage's products.  Row r of fragment f is weight row f * 32 +
  // (r / 4 % 2) * 16 + r / 8 * 4 + r % 4 of the wave's, so that the lane's
  // results of a fragment are 16 consecutive n.  A lane's 32 codes of a half
  // stage are k 32 h .. 32 h + 31 of it, 8 an MFMA.
  float16_t acc[NF][MF];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[f][m][i] = 0.0f;
  const int wrow = wave * (32 * NF) + ((r >> 2) & 1) * 16 + (r >> 3) * 4 + (r & 3);
  const auto half_stage = [&](int s, int sub) {
    const char *const buf = lds + (s & 1) * kBuffer;
    u32x4_t c[NF];
    Scale<MX> sc[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int row = wrow + 32 * f;
      c[f] = *reinterpret_cast<const u32x4_t *>(buf + row * 64 + 16 * ((2 * sub + h) ^ ((row >> 4) & 3)));
      const char *const sp = buf + kCodes + row * 8 + (2 * sub + h) * (32 / kG);
      if (MX) sc[f].raw = *reinterpret_cast<const uint8_t *>(sp);
      else sc[f].raw = *reinterpret_cast<const uint16_t *>(sp);
    }
    // MXFP4 at a quarter: the largest scales' weights pass bf16's range
    // otherwise; scales too near either end for the conversion's own go by
    // products
    bool far = false;
    if constexpr (MX) {
#pragma unroll
      for (int f = 0; f < NF; ++f) far |= sc[f].raw - 3 >= 250;
      far = __any(far);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bf16x8_t a[NF];
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        if constexpr (MX) {
          if (far) a[f] = decode8<false>(c[f][j], sc[f].quarter());
          else a[f] = decode8<true>(c[f][j], __uint_as_float((sc[f].raw - 2) << 23));
        } else {
          a[f] = decode8<false>(c[f][j], j < 2 ? sc[f].lo() : sc[f].hi());
        }
      }
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        const int row = 32 * m + r;
        const char *const at = buf + kCodes + kScales + row * 256 + 16 * ((8 * sub + 4 * h + j) ^ (row & 15));
#pragma unroll
        for (int p = 0; p < kXP; ++p) {
          const bf16x8_t b = *reinterpret_cast<const bf16x8_t *>(at + p * kPart);
#pragma unroll
          for (int f = 0; f < NF; ++f) acc[f][m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[f], b, acc[f][m], 0, 0, 0);
        }
      }
    }
  };

  if (stages > 0) {
    load(0);
    put(0);
    if (stages > 1) load(1);
    __syncthreads();
    for (int s = 0; s < stages; ++s) {
      half_stage(s, 0);
      half_stage(s, 1);
      if (s + 1 < stages) put(s + 1);
      if (s + 2 < stages) load(s + 2);
      __syncthreads();
    }
  }

  const float scale = MX ? 4.0f : w.K > 0 ? w.meta[1] : 0.0f;      // (g of no weights may be anything)
#pragma unroll
  for (int m = 0; m < MF; ++m) {
    const int64_t row = m0 + 32 * m + r;
    if (row >= t.end) continue;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = acc[f][m][i] * scale;
      store16(y, y_bf16, row * ldy, n0 + wave * (32 * NF) + 32 * f + 16 * h, w.N, v);
    }
  }
}

// ------------------------------------------------- bf16, larger groups --

// The same tiles with both operands copied to LDS by DMA, a stage ahead, and
// the work of a K step (the 16 k of an MFMA) in a fixed order: each MFMA is
// followed by its share of decoding the next step's weights, so that one wave a
// SIMD keeps the matrix pipe busy.  A stage's copies go out over the first four
// of its eight steps; in the last one the wave waits for those of the stage
// behind, meets the others, and reads from it.
//
// x rows of a multiple of 4 bytes, from an address of one (the range check that
// makes rows past the group zeros works by words).
constexpr int wait_vm(int n) { return (n & 15) | (n >> 4) << 14 | 0x0F70; }
// A wait for those counts, and the workgroup's barrier.
template <int COUNTS> __device__ __forceinline__ void meet() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(COUNTS);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

template <bool MX, int NF, int MF>
__global__ __launch_bounds__(kThreads, NF * MF >= 16 ? 1 : 2) void
k_grouped_dma(Stack w, Groups g, Rows<uint16_t> x, void *y, int y_bf16, int64_t ldy, int tiles_n, int fill) {
  constexpr int BN = 128 * NF, BM = 32 * MF;
  constexpr int kG = Scale<MX>::kPerByte, kSB = kStage / kG;
  constexpr int kCodes = BN * kStage / 2, kScales = BN * 8, kBuffer = kCodes + kScales + BM * kStage * 2;
  constexpr int kCL = BN / 64, kXL = BM / 16;        // DMA instructions a wave and stage: 16 rows of codes, 4 of x each
  constexpr int kSL = (BN + kThreads - 1) / kThreads;
  __shared__ __align__(16) uint8_t lds[2 * kBuffer];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5;

  if (fill) zero_rest(g, y, y_bf16, ldy, w.N);
  const int total = count_tiles(g, BM) * tiles_n;
  const int quota = (total + kXcds - 1) / kXcds, local = blockIdx.x / kXcds;
  const int index = (int)(blockIdx.x % kXcds) * quota + local;
  if (local >= quota || index >= total) return;
  const GroupTile t = find_tile(g, BM, tiles_n, index);
  if (t.e < 0) return;
  const int per = 8 * tiles_n, first_m = t.local / per * 8, gsz = min(t.tiles - first_m, 8);
  const int64_t m0 = t.begin + (int64_t)(first_m + t.local % per % gsz) * BM;
  const int64_t n0 = (int64_t)(t.local % per / gsz) * BN;
  const int stages = (int)((w.K + kStage - 1) / kStage);

  // ---- copies.  Codes: lane l takes row l / 4, slot l % 4, which holds piece
  // (l % 4) ^ (row / 16 % 4); x: row l / 16, slot l % 16, which holds piece
  // (l % 16) ^ (row % 16).  A wave's instructions are BN / 4 rows of codes and
  // BM / 4 of x, from views of the tile's own rows.
  const uint32_t cp = (uint32_t)w.code_pitch, xp = (uint32_t)(x.ld * 2), kb = (uint32_t)w.K;
  const __amdgpu_buffer_rsrc_t cview =
      make_rsrc(w.codes + t.e * w.code_step + n0 * w.code_pitch,
                (uint32_t)(min((int64_t)BN, w.N - n0) - 1) * cp + kb / 2);
  const __amdgpu_buffer_rsrc_t xview =
      make_rsrc(x.p + m0 * x.ld, (uint32_t)(min((int64_t)BM, t.end - m0) - 1) * xp + kb * 2);
  const uint32_t crow = (uint32_t)(wave * (BN / 4) + (lane >> 2)) * cp, cpiece = (uint32_t)lane & 3;
  const uint32_t xrow = (uint32_t)(wave * (BM / 4) + (lane >> 4)) * xp, xpiece = (uint32_t)(lane & 15) ^ (lane >> 4);
  const uint8_t *srow[kSL];
#pragma unroll
  for (int i = 0; i < kSL; ++i)
    srow[i] = w.scales + t.e * w.scale_step + min(n0 + tid + i * kThreads, w.N - 1) * w.scale_pitch;
  uint64_t sreg[kSL];
  // part q of 4 of stage s (nothing past the last one)
  const auto copy = [&](int s, int q) {
    uint8_t *const buf = lds + (s & 1) * kBuffer;
    const uint32_t k0 = (uint32_t)s * kStage;
    const bool in = s < stages;
#pragma unroll
    for (int i = q * kCL / 4; i < (q + 1) * kCL / 4; ++i) {
      const uint32_t piece = cpiece ^ (uint32_t)((wave * (BN / 64) + i) & 3);
      const uint32_t at = !in || k0 + 32 * piece < kb ? crow + 16 * piece : kOutOfRange;
      dma16(cview, buf + (wave * (BN / 4) + 16 * i) * 64, at, in ? 16u * i * cp + k0 / 2 : kOutOfRange);
    }
#pragma unroll
    for (int i = q * kXL / 4; i < (q + 1) * kXL / 4; ++i) {
      const uint32_t piece = xpiece ^ (uint32_t)((wave * (BM / 4) + 4 * i) & 15);
      const uint32_t at = !in || k0 + 8 * piece < kb ? xrow + 16 * piece : kOutOfRange;
      dma16(xview, buf + kCodes + kScales + (wave * (BM / 4) + 4 * i) * 256, at, in ? 4u * i * xp + k0 * 2 : kOutOfRange);
    }
    if (q == 0 && in) {
      if ((int64_t)k0 + kStage <= w.K) {
#pragma unroll
        for (int i = 0; i < kSL; ++i) {
          sreg[i] = 0;
          __builtin_memcpy(&sreg[i], srow[i] + k0 / kG, kSB);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kSL; ++i) {
          sreg[i] = MX ? 0x7F7F7F7F7F7F7F7Full : 0;
          for (int b = 0; b < kSB; ++b)
            if (k0 + b * kG < kb)
              sreg[i] = (sreg[i] & ~(0xFFull << (8 * b))) | (uint64_t)srow[i][k0 / kG + b] << (8 * b);
        }
      }
    }
  };
  const auto put_scales = [&](int s) {
#pragma unroll
    for (int i = 0; i < kSL; ++i)
      if (BN % kThreads == 0 || tid + i * kThreads < BN)
        *reinterpret_cast<uint64_t *>(lds + (s & 1) * kBuffer + kCodes + (tid + i * kThreads) * 8) = sreg[i];
  };

  // ---- operands.  Half stage p (0, 1) of a stage is four K steps.
  float16_t acc[NF][MF];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[f][m][i] = 0.0f;
  const int wrow = wave * (32 * NF) + ((r >> 2) & 1) * 16 + (r >> 3) * 4 + (r & 3);
  u32x4_t c[2][NF];
  Scale<MX> sc[2][NF];
  bool far[2] = {false, false};
  bf16x8_t a[2][NF], b[2][MF];
  const auto read_codes = [&](int s, int p) {
    const uint8_t *const buf = lds + (s & 1) * kBuffer;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int row = wrow + 32 * f;
      c[p][f] = *reinterpret_cast<const u32x4_t *>(buf + row * 64 + 16 * ((2 * p + h) ^ ((row >> 4) & 3)));
      const uint8_t *const sp = buf + kCodes + row * 8 + (2 * p + h) * (32 / kG);
      if (MX) sc[p][f].raw = *sp;
      else sc[p][f].raw = *reinterpret_cast<const uint16_t *>(sp);
    }
  };
  const auto read_x = [&](int s, int p, int j, int into) {
    const uint8_t *const buf = lds + (s & 1) * kBuffer + kCodes + kScales;
#pragma unroll
    for (int m = 0; m < MF; ++m)
      b[into][m] = *reinterpret_cast<const bf16x8_t *>(buf + (32 * m + r) * 256 + 16 * ((8 * p + 4 * h + j) ^ (r & 15)));
  };
  const auto check_far = [&](int p) {
    if constexpr (MX) {
      bool any = false;
#pragma unroll
      for (int f = 0; f < NF; ++f) any |= sc[p][f].raw - 3 >= 250;
      far[p] = __any(any);
    }
  };
  // a quarter of a fragment's 8 weights (MXFP4: all of them for quarter 0)
  const auto decode = [&](int p, int j, int f, int quarter, int into) {
    if constexpr (MX) {
      if (quarter) return;
      if (far[p]) a[into][f] = decode8<false>(c[p][f][j], sc[p][f].quarter());
      else a[into][f] = decode8<true>(c[p][f][j], __uint_as_float((sc[p][f].raw - 2) << 23));
    } else {
      const float s = j < 2 ? sc[p][f].lo() : sc[p][f].hi();
      const uint32_t code = c[p][f][j];
      const float2_t v = quarter == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 0)
                         : quarter == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 1)
                         : quarter == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 2)
                                        : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 3);
      const bf16x2_t q = __builtin_convertvector((f32x2_t){v.x * s, v.y * s}, bf16x2_t);
      a[into][f][2 * quarter] = q[0];
      a[into][f][2 * quarter + 1] = q[1];
    }
  };
  constexpr int NU = NF * MF, ND = 4 * NF;           // MFMAs and quarters to decode of a K step
  // K step j of half p of stage s: operands of `cur` are there; the next step's
  // go to the other.
  const auto step = [&](int s, auto half, auto kstep) {
    constexpr int p = decltype(half)::value, j = decltype(kstep)::value;
    constexpr int cur = j & 1, nxt = cur ^ 1, np = j == 3 ? p ^ 1 : p, nj = (j + 1) & 3;
    if constexpr (p == 1 && j == 3) {
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(wait_vm(0));       // this wave's copies of the next stage
      put_scales(s + 1);
      __syncthreads();
      read_codes(s + 1, 0);
      read_x(s + 1, 0, 0, nxt);
    } else {
      if constexpr (p == 0) copy(s + 1, j);
      if constexpr (p == 0 && j == 2) read_codes(s, 1);
      read_x(s, np, nj, nxt);
    }
    constexpr int kLag = j == 3 && NU >= 4 ? NU / 4 : 0;      // codes just read are not there yet
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      const int m = i / NF, f = (m & 1) ? NF - 1 - i % NF : i % NF;
      acc[f][m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[cur][f], b[cur][m], acc[f][m], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      if (j == 3 && i == kLag) check_far(np);
      if (i >= kLag) {
        const int d0 = (i - kLag) * ND / (NU - kLag), d1 = (i - kLag + 1) * ND / (NU - kLag);
#pragma unroll
        for (int d = d0; d < d1; ++d) decode(np, nj, d / 4, d % 4, nxt);
      }
    }
  };

  if (stages > 0) {
#pragma unroll
    for (int q = 0; q < 4; ++q) copy(0, q);
    __builtin_amdgcn_s_waitcnt(wait_vm(0));
    put_scales(0);
    __syncthreads();
    read_codes(0, 0);
    read_x(0, 0, 0, 0);
    check_far(0);
#pragma unroll
    for (int d = 0; d < ND; ++d) decode(0, 0, d / 4, d % 4, 0);
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I3 = std::integral_constant<int, 3>;
    for (int s = 0; s < stages; ++s) {
      step(s, I0{}, I0{});
      step(s, I0{}, I1{});
      step(s, I0{}, I2{});
      step(s, I0{}, I3{});
      step(s, I1{}, I0{});
      step(s, I1{}, I1{});
      step(s, I1{}, I2{});
      step(s, I1{}, I3{});
    }
    __builtin_amdgcn_sched_barrier(0);
  }

  const float scale = MX ? 4.0f : w.K > 0 ? w.meta[1] : 0.0f;
#pragma unroll
  for (int m = 0; m < MF; ++m) {
    const int64_t row = m0 + 32 * m + r;
    if (row >= t.end) continue;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = acc[f][m][i] * scale;
      store16(y, y_bf16, row * ldy, n0 + wave * (32 * NF) + 32 * f + 16 * h, w.N, v);
    }
  }
}

// Weight rows and tokens of a tile, in fragments of 32 (times 4 waves).
struct GroupedCut {
  int nf, mf;
};
GroupedCut grouped_cut(const Stack &w, int experts, int64_t tokens, bool f32) {
  const int64_t each = (tokens + experts - 1) / experts;      // rows of a group, on average
  if (each <= 40) return {1, 1};
  if (each <= 128 || f32) return {2, 2};
  return {4, 4};
}

template <bool MX, typename X, int NF, int MF>
hipError_t grouped(const Stack &w, const Groups &g, const Rows<X> &x, void *y, int y_bf16, int64_t ldy, int fill,
                   hipStream_t stream) {
  constexpr int BN = 128 * NF, BM = 32 * MF;
  const int64_t tiles_n = (w.N + BN - 1) / BN, tiles_m = g.rows / BM + std::min<int64_t>(g.count, g.rows);
  const unsigned grid = (unsigned)((tiles_n * tiles_m + kXcds - 1) / kXcds * kXcds);
  if constexpr (sizeof(X) == 2 && NF > 1) {
    // copies by DMA: words, and offsets inside a tile below 2^31
    if ((uintptr_t)x.p % 4 == 0 && x.ld % 2 == 0 && x.ld < (1LL << 22) && w.code_pitch < (1LL << 21)) {
      k_grouped_dma<MX, NF, MF><<<grid, kThreads, 0, stream>>>(w, g, x, y, y_bf16, ldy, (int)tiles_n, fill);
      return hipGetLastError();
    }
  }
  k_grouped<MX, X, NF, MF><<<grid, kThreads, 0, stream>>>(w, g, x, y, y_bf16, ldy, (int)tiles_n, fill);
  return hipGetLastError();
}
template <bool MX, typename X>
hipError_t grouped_x(const Stack &w, const Groups &g, const Rows<X> &x, void *y, int y_bf16, int64_t ldy, int fill,
                     hipStream_t stream) {
  const GroupedCut c = grouped_cut(w, g.count, g.rows, sizeof(X) == 4);
  if (c.nf == 1) return grouped<MX, X, 1, 1>(w, g, x, y, y_bf16, ldy, fill, stream);
  if constexpr (sizeof(X) == 2)
    if (c.nf == 4) return grouped<MX, X, 4, 4>(w, g, x, y, y_bf16, ldy, fill, stream);
  return grouped<MX, X, 2, 2>(w, g, x, y, y_bf16, ldy, fill, stream);
}

// ------------------------------------------------------ weight gradient --

// Tokens run along the reduction here, and lie down the columns of both
// operands: a stage's rows go to LDS as they are, and the lanes fetch columns
// with transposing reads (16 lanes take 4 rows of 16 columns, and each leaves
// with 4 rows of its own column).  Rows of LDS are 64 bytes longer than their
// columns, so that the 4 rows of two such neighbours fall on different banks.
// Of the parts of two float32 operands the products from hi hi to mid mid are
// taken; those left out are below 2^-25 of the whole.
// Tiles of a group that an XCD takes: a run of an eighth of every group's, since
// groups differ in length.  The grid has this for each XCD and group.
__host__ __device__ __forceinline__ int wgrad_quota(int tiles) { return (tiles + kXcds - 1) / kXcds; }

// A workgroup's tile is 64 FN columns of dy (n) by 64 FK columns of x, two by
// two waves; every group's tiles are written, zeros for a group without rows.
template <typename D, typename X, int FN, int FK, int TOKENS>
__global__ __launch_bounds__(kThreads) void k_grouped_wgrad(Groups g, Rows<D> dy, Rows<X> x, void *dw, int dw_bf16,
                                                            int64_t N, int64_t K, int tiles_n, int tiles_k) {
  constexpr int kDP = sizeof(D) == 2 ? 1 : 3, kXP = sizeof(X) == 2 ? 1 : 3;
  constexpr int TN = 64 * FN, TK = 64 * FK;
  constexpr int kRowD = TN * 2 + 64, kRowX = TK * 2 + 64;            // bytes of a row in LDS
  constexpr int kPartD = TOKENS * kRowD, kPartX = TOKENS * kRowX;
  constexpr int kBuffer = kDP * kPartD + kXP * kPartX;
  constexpr int kDL = TOKENS * (TN / 8) / kThreads, kXL = TOKENS * (TK / 8) / kThreads;
  __shared__ __align__(16) char lds[2 * kBuffer];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  const int tiles = tiles_n * tiles_k, quota = wgrad_quota(tiles);
  const int e = blockIdx.x / kXcds / quota, at = (int)(blockIdx.x % kXcds) * quota + (int)(blockIdx.x / kXcds) % quota;
  if (at >= tiles) return;
  const int per = 8 * tiles_k, first_n = at / per * 8, gsz = min(tiles_n - first_n, 8);
  const int64_t n0 = (int64_t)(first_n + at % per % gsz) * TN, k0 = (int64_t)(at % per / gsz) * TK;
  const int64_t begin = g.at(e), end = max(g.at(e + 1), begin);
  const bool inside = n0 + TN <= N && k0 + TK <= K;
  const int stages = (int)((end - begin + TOKENS - 1) / TOKENS);

  Row8<D> dreg[kDL];
  Row8<X> xreg[kXL];
  const auto load = [&](int s) {
    const int64_t t0 = begin + (int64_t)s * TOKENS;
    if (inside && t0 + TOKENS <= end) {
#pragma unroll
      for (int i = 0; i < kDL; ++i) {
        const int p = tid + i * kThreads;
        dreg[i].load(dy.p + (t0 + p / (TN / 8)) * dy.ld + n0 + p % (TN / 8) * 8);
      }
#pragma unroll
      for (int i = 0; i < kXL; ++i) {
        const int p = tid + i * kThreads;
        xreg[i].load(x.p + (t0 + p / (TK / 8)) * x.ld + k0 + p % (TK / 8) * 8);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kDL; ++i) {
        const int p = tid + i * kThreads;
        const int64_t row = t0 + p / (TN / 8);
        load_row8(dreg[i], dy.p + row * dy.ld, n0 + p % (TN / 8) * 8, row < end ? N : 0);
      }
#pragma unroll
      for (int i = 0; i < kXL; ++i) {
        const int p = tid + i * kThreads;
        const int64_t row = t0 + p / (TK / 8);
        load_row8(xreg[i], x.p + row * x.ld, k0 + p % (TK / 8) * 8, row < end ? K : 0);
      }
    }
  };
  const auto put_one = [&](char *to, int part, const auto &q) {
    if constexpr (sizeof(q) == 16) {
      *reinterpret_cast<u32x4_t *>(to) = q.r;
    } else {
      const Parts v = split8_nearest(q);
#pragma unroll
      for (int p = 0; p < 3; ++p) *reinterpret_cast<u32x4_t *>(to + p * part) = v.v[p];
    }
  };
  const auto put = [&](int s) {
    char *const buf = lds + (s & 1) * kBuffer;
#pragma unroll
    for (int i = 0; i < kDL; ++i) {
      const int p = tid + i * kThreads;
      put_one(buf + p / (TN / 8) * kRowD + p % (TN / 8) * 16, kPartD, dreg[i]);
    }
#pragma unroll
    for (int i = 0; i < kXL; ++i) {
      const int p = tid + i * kThreads;
      put_one(buf + kDP * kPartD + p / (TK / 8) * kRowX + p % (TK / 8) * 16, kPartX, xreg[i]);
    }
  };

  float16_t acc[FN][FK];
#pragma unroll
  for (int f = 0; f < FN; ++f)
#pragma unroll
    for (int q = 0; q < FK; ++q)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[f][q][i] = 0.0f;
  // a lane's 8 rows (8 h .. 8 h + 7 of an MFMA's 16) of its column of a
  // fragment of 32, by two reads; it names 4 columns of one row
  const int col = 16 * ((lane >> 4) & 1) + 4 * (lane & 3), trow = 8 * (lane >> 5) + ((lane >> 2) & 3);
  const auto products = [&](int s) {
    const char *const dbuf = lds + (s & 1) * kBuffer + trow * kRowD + ((wave >> 1) * (32 * FN) + col) * 2;
    const char *const xbuf = lds + (s & 1) * kBuffer + kDP * kPartD + trow * kRowX + ((wave & 1) * (32 * FK) + col) * 2;
#pragma unroll
    for (int ks = 0; ks < TOKENS / 16; ++ks) {
      bf16x8_t a[kDP][FN], b[kXP][FK];
#pragma unroll
      for (int p = 0; p < kDP; ++p)
#pragma unroll
        for (int f = 0; f < FN; ++f) a[p][f] = lds_column(dbuf + p * kPartD + ks * 16 * kRowD + f * 64, kRowD);
#pragma unroll
      for (int p = 0; p < kXP; ++p)
#pragma unroll
        for (int f = 0; f < FK; ++f) b[p][f] = lds_column(xbuf + p * kPartX + ks * 16 * kRowX + f * 64, kRowX);
#pragma unroll
      for (int p = 0; p < kDP; ++p)
#pragma unroll
        for (int q = 0; q < kXP; ++q) {
          if (p + q > 2) continue;
#pragma unroll
          for (int f = 0; f < FN; ++f)
#pragma unroll
            for (int k = 0; k < FK; ++k)
              acc[f][k] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[p][f], b[q][k], acc[f][k], 0, 0, 0);
        }
    }
  };

  if (stages > 0) {
    load(0);
    put(0);
    if (stages > 1) load(1);
    __syncthreads();
    for (int s = 0; s < stages; ++s) {
      products(s);
      if (s + 1 < stages) put(s + 1);
      if (s + 2 < stages) load(s + 2);
      __syncthreads();
    }
  }

  // register i of a fragment is row 8 (i / 4) + 4 h + i % 4, the lane its column
  const int64_t base = (int64_t)e * N;
#pragma unroll
  for (int f = 0; f < FN; ++f)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int64_t n = n0 + (wave >> 1) * (32 * FN) + 32 * f + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3);
      if (n >= N) continue;
#pragma unroll
      for (int q = 0; q < FK; ++q) {
        const int64_t k = k0 + (wave & 1) * (32 * FK) + 32 * q + (lane & 31);
        if (k >= K) continue;
        if (dw_bf16) ((uint16_t *)dw)[(base + n) * K + k] = (uint16_t)pack_bf16(acc[f][q][i], 0.0f);
        else ((float *)dw)[(base + n) * K + k] = acc[f][q][i];
      }
    }
}

// The 4 x 4 transpose over the lanes of a quad and four registers: lane j is
// left with the j-th register of each of them.
__device__ __forceinline__ f32x4_t quad_turn(float a, float b, float c, float d) {
  const int lane = threadIdx.x;
  const bool odd = lane & 1, high = lane & 2;
  // lanes 1 apart, then 2 (every exchange by all lanes, the choice after it)
  const float an = dpp<0xB1>(a), bn = dpp<0xB1>(b), cn = dpp<0xB1>(c), dn = dpp<0xB1>(d);
  const float a1 = odd ? bn : a, b1 = odd ? b : an, c1 = odd ? dn : c, d1 = odd ? d : cn;
  const float af = dpp<0x4E>(a1), bf = dpp<0x4E>(b1), cf = dpp<0x4E>(c1), df = dpp<0x4E>(d1);
  return (f32x4_t){high ? cf : a1, high ? df : b1, high ? c1 : af, high ? d1 : bf};
}
// 4 neighbouring elements k .. k + 3 of a row of K.
__device__ __forceinline__ void store4(void *out, int bf16, int64_t row, int64_t k, int64_t K, const f32x4_t &v) {
  if (k + 4 <= K) {
    if (bf16) *reinterpret_cast<u32x2_a2 *>((uint16_t *)out + row + k) = (u32x2_a2){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    else *reinterpret_cast<f32x4_a4 *>((float *)out + row + k) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      if (k + i >= K) continue;
      if (bf16) ((uint16_t *)out)[row + k + i] = (uint16_t)pack_bf16(v[i], 0.0f);
      else ((float *)out)[row + k + i] = v[i];
    }
  }
}

// bf16 operands of whole words: tiles of 128 columns of dy by 256 of x, two
// workgroups a CU, so that one multiplies while the other stores; copied to
// LDS by DMA two stages of 32 tokens ahead, the columns of the next 16 tokens
// fetched between the MFMAs of these.  Chunk c (32 bytes, 16 columns) of row t
// lies in place c ^ (2 (t % 4)), so that the 4 rows of a transposing read's
// two neighbouring chunks fall on different banks.
constexpr int kWgTokens = 32, kWgRing = 3, kWgRowD = 256, kWgRowX = 512;
constexpr int kWgStageD = kWgTokens * kWgRowD, kWgStage = kWgStageD + kWgTokens * kWgRowX;
constexpr int kWgCopies = kWgStage / 4096;         // DMA instructions a wave and stage
// One of the two half stages of 16 tokens: `from` is where the operands of the
// next one lie (the stage itself, or the one behind), `to` where this stage's
// copies go, which is another place of the ring.  (Two pointers that do not
// meet: a transposing read would else wait for every copy under way.)
struct WgOperands {
  bf16x8_t a[2][2], b[2][4];
};
struct WgCopy {
  __amdgpu_buffer_rsrc_t dv, xv;
  uint32_t dat, xat[2], dp, xp;              // lane offsets (x: of even and odd instructions), a row's bytes
  int wave;
  // copy i of 6 of a stage at `to`: 4 rows of dy, or 2 of x; a wave's are 8 rows
  __device__ __forceinline__ void run(int i, uint8_t *to) const {
    if (i < 2)
      dma16(dv, to + (8 * wave + 4 * i) * kWgRowD, dat, (uint32_t)(8 * wave + 4 * i) * dp);
    else
      dma16(xv, to + kWgStageD + (8 * wave + 2 * (i - 2)) * kWgRowX, xat[i & 1], (uint32_t)(8 * wave + 2 * (i - 2)) * xp);
  }
};
template <int P>
__device__ __forceinline__ void wg_half(const char *__restrict__ from, uint8_t *__restrict__ to, float16_t (&acc)[2][4],
                                        WgOperands &o, const uint32_t (&dat)[2], const uint32_t (&xat)[4],
                                        const WgCopy &c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    __builtin_amdgcn_sched_barrier(0);
    const int f = i / 4, q = (f & 1) ? 3 - i % 4 : i % 4;
    acc[f][q] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(o.a[P][f], o.b[P][q], acc[f][q], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
    if (i < 2) o.a[P ^ 1][i] = lds_column(from + dat[i], kWgRowD);
    else if (i < 6) o.b[P ^ 1][i - 2] = lds_column(from + xat[i - 2], kWgRowX);
    if (P == 0 && i >= 2) c.run(i - 2, to);
  }
}
__global__ __launch_bounds__(kThreads, 2) void k_grouped_wgrad_dma(Groups g, Rows<uint16_t> dy, Rows<uint16_t> x, void *dw,
                                                                   int dw_bf16, int64_t N, int64_t K, int tiles_n,
                                                                   int tiles_k) {
  __shared__ __align__(16) uint8_t lds[kWgRing * kWgStage];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tiles = tiles_n * tiles_k, quota = wgrad_quota(tiles);
  const int e = blockIdx.x / kXcds / quota, at = (int)(blockIdx.x % kXcds) * quota + (int)(blockIdx.x / kXcds) % quota;
  if (at >= tiles) return;
  const int per = 16 * tiles_k, first_n = at / per * 16, gsz = min(tiles_n - first_n, 16);
  const int64_t n0 = (int64_t)(first_n + at % per % gsz) * 128, k0 = (int64_t)(at % per / gsz) * 256;
  const int64_t begin = uniform64(g.at(e)), end = max(uniform64(g.at(e + 1)), begin);
  const int stages = (int)((end - begin + kWgTokens - 1) / kWgTokens);

  // an instruction copies 1 KB: 4 rows of dy, lane l slot l % 16 (16 bytes) of
  // row l / 16, or 2 of x, slot l % 32 of row l / 32
  WgCopy c;
  c.wave = wave;
  c.dp = (uint32_t)(dy.ld * 2);
  c.xp = (uint32_t)(x.ld * 2);
  c.dat = (uint32_t)(lane >> 4) * c.dp + 16 * (uint32_t)((lane & 15) ^ (4 * (lane >> 4)));
#pragma unroll
  for (int i = 0; i < 2; ++i)
    c.xat[i] = (uint32_t)(lane >> 5) * c.xp + 16 * (uint32_t)((lane & 31) ^ (4 * (2 * i + (lane >> 5))));
  const auto aim = [&](int s) {
    const int64_t t0 = begin + (int64_t)s * kWgTokens, rows = min(end - t0, (int64_t)kWgTokens);
    const auto view = [&](const Rows<uint16_t> &m, uint32_t pitch, int64_t c0, int64_t cols, int64_t most) {
      return make_rsrc(m.p + (rows > 0 ? t0 * m.ld + c0 : 0),
                       rows > 0 ? (uint32_t)(rows - 1) * pitch + (uint32_t)min(cols - c0, most) * 2 : 0u);
    };
    c.dv = view(dy, c.dp, n0, N, 128);
    c.xv = view(x, c.xp, k0, K, 256);
  };

  float16_t acc[2][4];
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[f][q][i] = 0.0f;
  // the lane's 4 columns of one row of a transposing read, for each fragment
  const int trow = 8 * (lane >> 5) + ((lane >> 2) & 3), turn = 2 * ((lane >> 2) & 3);
  uint32_t dat[2], xat[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    const int chunk = 2 * f + ((lane >> 4) & 1);
    if (f < 2) dat[f] = trow * kWgRowD + 32 * (((wave >> 1) * 4 + chunk) ^ turn) + 8 * (lane & 3);
    xat[f] = kWgStageD + trow * kWgRowX + 32 * (((wave & 1) * 8 + chunk) ^ turn) + 8 * (lane & 3);
  }
  // (a half stage's operands lie 16 rows on, of both matrices)
  uint32_t dat1[2], xat1[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    if (f < 2) dat1[f] = dat[f] + 16 * kWgRowD;
    xat1[f] = xat[f] + 16 * kWgRowX;
  }
  WgOperands o;
  if (stages > 0) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      aim(s);
#pragma unroll
      for (int i = 0; i < kWgCopies; ++i) c.run(i, lds + s * kWgStage);
    }
    meet<(wait_vm(kWgCopies) & ~0x0F00)>();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < 2) o.a[0][i] = lds_column((const char *)lds + dat[i], kWgRowD);
      o.b[0][i] = lds_column((const char *)lds + xat[i], kWgRowX);
    }
    int now = 0, next = kWgStage, free = 2 * kWgStage;           // places of this stage, the next, and the one behind it
    for (int s = 0; s < stages; ++s) {
      aim(s + 2);
      wg_half<0>((const char *)lds + now, lds + free, acc, o, dat1, xat1, c);
      // this wave's copies of the next stage (those of one more stay under way,
      // which a fence would wait for) and its reads of this one
      meet<(wait_vm(kWgCopies) & ~0x0F00)>();
      wg_half<1>((const char *)lds + next, lds + free, acc, o, dat, xat, c);
      const int was = now;
      now = next;
      next = free;
      free = was;
    }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(wait_vm(0));        // nothing is left that writes LDS
  }
  // register i of a fragment is row 8 (i / 4) + 4 h + i % 4, the lane its
  // column; turned over the quads a lane has 4 neighbours of fragment lane % 4
  // (stores of 16 bytes a lane, whole lines: with 4 the wave's 128 of them held
  // the copies of the CU's other workgroup up, 530 -> 480 us)
  const int64_t base = (int64_t)e * N, k = k0 + (wave & 1) * 128 + 32 * (lane & 3) + (lane & 28);
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int64_t n = n0 + (wave >> 1) * 64 + 32 * f + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3);
      const f32x4_t v = quad_turn(acc[f][0][i], acc[f][1][i], acc[f][2][i], acc[f][3][i]);
      if (n < N && k < K) store4(dw, dw_bf16, (base + n) * K, k, K, v);
    }
}

template <typename D, typename X>
hipError_t wgrad(const Groups &g, const Rows<D> &dy, const Rows<X> &x, void *dw, int dw_bf16, int64_t N, int64_t K,
                 hipStream_t stream) {
  constexpr bool narrow = sizeof(D) + sizeof(X) == 4;
  constexpr int F = narrow ? 4 : 2, kTokens = narrow ? 64 : 16;
  const int64_t tn = (N + 64 * F - 1) / (64 * F), tk = (K + 64 * F - 1) / (64 * F);
  const unsigned grid = (unsigned)(wgrad_quota((int)(tn * tk)) * kXcds * g.count);
  if constexpr (narrow) {
    const auto words = [](const Rows<uint16_t> &m, int64_t cols) {
      return (uintptr_t)m.p % 4 == 0 && m.ld % 2 == 0 && cols % 2 == 0 && m.ld < (1LL << 24);
    };
    if (words(dy, N) && words(x, K)) {
      const int64_t rows = (N + 127) / 128;
      k_grouped_wgrad_dma<<<(unsigned)(wgrad_quota((int)(rows * tk)) * kXcds * g.count), kThreads, 0, stream>>>(
          g, dy, x, dw, dw_bf16, N, K, (int)rows, (int)tk);
      return hipGetLastError();
    }
  }
  k_grouped_wgrad<D, X, F, F, kTokens><<<grid, kThreads, 0, stream>>>(g, dy, x, dw, dw_bf16, N, K, (int)tn, (int)tk);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_wgrad(const GroupedWgrad &p, hipStream_t stream) {
  if (p.n == 0 || p.k == 0) return hipSuccess;
  const Groups g = {p.offsets, p.index_bits == 64, (int)p.experts, p.rows, 0};
  const int b = p.dw_dtype == 1;
  const auto run = [&](auto *d, auto *x) {
    using D = std::remove_const_t<std::remove_pointer_t<decltype(d)>>;
    using X = std::remove_const_t<std::remove_pointer_t<decltype(x)>>;
    return wgrad<D, X>(g, {d, p.lddy}, {x, p.ldx}, p.dw, b, p.n, p.k, stream);
  };
  if (p.dy_dtype == 1 && p.x_dtype == 1) return run((const uint16_t *)p.dy, (const uint16_t *)p.x);
  if (p.dy_dtype == 1) return run((const uint16_t *)p.dy, (const float *)p.x);
  if (p.x_dtype == 1) return run((const float *)p.dy, (const uint16_t *)p.x);
  return run((const float *)p.dy, (const float *)p.x);
}

int64_t grouped_workspace_bytes(int64_t experts, int64_t n, int64_t k, int64_t rows, bool f32) { return 0; }

hipError_t launch_grouped(const GroupedProduct &p, hipStream_t stream) {
  if (p.n == 0 || p.rows == 0) return hipSuccess;
  const int64_t block = p.mx ? 32 : 16, rows = p.transposed ? 1 : p.n;
  const int64_t pitch = p.transposed ? p.experts * p.k : p.k, step = rows * p.k;
  const Stack w = {p.codes, p.scales, p.meta, p.n, p.k, pitch / 2, step / 2, pitch / block, step / block};
  const Groups g = {p.offsets, p.index_bits == 64, (int)p.experts, p.rows, 0};
  const int yb = p.y_dtype == 1;
  if (p.x_dtype == 1) {
    const Rows<uint16_t> x = {(const uint16_t *)p.x, p.ldx};
    return p.mx ? grouped_x<true>(w, g, x, p.y, yb, p.ldy, p.fill, stream)
                : grouped_x<false>(w, g, x, p.y, yb, p.ldy, p.fill, stream);
  }
  const Rows<float> x = {(const float *)p.x, p.ldx};
  return p.mx ? grouped_x<true>(w, g, x, p.y, yb, p.ldy, p.fill, stream)
              : grouped_x<false>(w, g, x, p.y, yb, p.ldy, p.fill, stream);
}

}  // namespace nvfp4
