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
// are three bf16 parts, made once per call (k_parts).  A workgroup's tile is
// 32 NF weight rows a wave, so that every weight is decoded by one wave, by 32
// MF tokens, which all of its waves read from LDS; codes, scales and tokens are
// copied there by DMA a stage ahead, and the decoding lies between the MFMAs.
// Groups of few rows take the matrix-vector product's tiles instead
// (grouped_tiles_fit, in matvec.hip), which read the weights once and are bound
// by that.
//
// Bound by the matrix pipe where groups are long: 4096 rows of 8 experts
// 20480 x 5120 in bf16 take 800 to 816 us (NVFP4; 1050 to 1075 TFLOP/s, a large bf16
// product of the library reaches 1440), of which partly filled tiles at the groups' ends
// are an eighth, decoding a tenth and the LDS traffic of the copies a fifth.
// 1531 float32 rows of 24 experts transposed, 5120 x 1280 (three products each):
// 101 to 107 us, bound by copies that are one stage ahead (60 KB a CU on their
// way), and 7.5 for the parts.
//
// The weight gradient has tokens along the reduction: both operands lie in LDS
// as they come, by DMA three stages deep, and reach the lanes by transposing
// reads.  8192 rows of 8 experts 5120 x 5120 in bf16: 498 us (863 TFLOP/s);
// float32 operands go as three parts each, six products (777 rows of 16 experts
// 1283 x 2050: 63 to 71 us, 168 MB of results among them, and 9 to 11 for the parts).
#include "gemm_common.h"
#include "groups.h"
#include "nvfp4_kernels.h"
#include "operands.h"

#include <algorithm>
#include <type_traits>

namespace nvfp4 {

namespace {

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

// Activations as the kernel copies them: bf16 rows of whole words.  Where a
// call's own are not (float32, or rows at odd places), they are brought to
// that first: [parts][rows][K] in the workspace.
template <typename X>
__global__ __launch_bounds__(256) void k_parts(const X *x, int64_t ldx, int64_t rows, int64_t K, uint16_t *out) {
  const int64_t pieces = K / 8, all = rows * pieces;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    const int64_t at = i / pieces * K + i % pieces * 8;
    Row8<X> q;
    q.load(x + i / pieces * ldx + i % pieces * 8);
    if constexpr (sizeof(X) == 2) {
      *reinterpret_cast<u32x4_t *>(out + at) = q.r;
    } else {
      const Parts p = split8((f32x4_t)q.a, (f32x4_t)q.b);
#pragma unroll
      for (int k = 0; k < 3; ++k) *reinterpret_cast<u32x4_t *>(out + k * rows * K + at) = p.v[k];
    }
  }
}

// Both operands are copied to LDS by DMA, a stage ahead, and the work of a K
// step (the 16 k of an MFMA) goes in a fixed order: each MFMA is followed by
// its share of decoding the next step's weights, so that one wave a SIMD keeps
// the matrix pipe busy.  A stage's copies go out over the first four of its
// eight steps; in the last one the wave waits for those of the stage behind,
// meets the others, and reads from it.
// XP: parts of x (3: float32), `part` elements apart.
template <bool MX, int XP, int WAVES, int NF, int MF>
__global__ __launch_bounds__(64 * WAVES, WAVES == 4 && NF * MF * XP < 12 ? 2 : 1) void
k_grouped(Stack w, Groups g, Rows<uint16_t> x, int64_t part, void *y, int y_bf16, int64_t ldy, int tiles_n, int fill) {
  constexpr int BN = 32 * WAVES * NF, BM = 32 * MF;
  constexpr int kG = Scale<MX>::kPerByte, kSB = kStage / kG;
  constexpr int kCodes = BN * kStage / 2, kScales = BN * 8, kPart = BM * kStage * 2, kBuffer = kCodes + kScales + XP * kPart;
  // DMA instructions a wave and stage: 16 rows of codes, 4 of a part of x each
  constexpr int kCL = BN / WAVES / 16, kXL = BM / WAVES / 4;
  constexpr int kSL = NF / 2;                        // weight rows of a lane, whose scales it fetches: its wave's own
  static_assert(kXL >= 1 && kSL >= 1, "a wave copies whole instructions");
  // (one array for all: with two of them every read would wait for the copies
  // under way)
  __shared__ __align__(16) uint8_t lds[2 * kBuffer + 4 * WAVES];
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
  // (codes: a view for each instruction's 16 rows, whose offsets stay small
  // however long the stack's rows are)
  const auto cview = [&](int i) {
    const int64_t row = n0 + wave * (BN / WAVES) + 16 * i, rows = min(w.N - row, (int64_t)16);
    return make_rsrc(w.codes + t.e * w.code_step + row * w.code_pitch, rows > 0 ? (uint32_t)(rows - 1) * cp + kb / 2 : 0u);
  };
  const int64_t xfirst = m0 + wave * (BM / WAVES), xrows = min(t.end - xfirst, (int64_t)(BM / WAVES));
  const auto xview = [&](int p) {
    return make_rsrc(x.p + p * part + xfirst * x.ld, xrows > 0 ? (uint32_t)(xrows - 1) * xp + kb * 2 : 0u);
  };
  const uint32_t crow = (uint32_t)(lane >> 2) * cp, cpiece = (uint32_t)lane & 3;
  const uint32_t xrow = (uint32_t)(lane >> 4) * xp, xpiece = (uint32_t)(lane & 15) ^ (lane >> 4);
  const uint8_t *srow[kSL];
#pragma unroll
  for (int i = 0; i < kSL; ++i)
    srow[i] = w.scales + t.e * w.scale_step + min(n0 + wave * (32 * NF) + lane + 64 * i, w.N - 1) * w.scale_pitch;
  uint64_t sreg[kSL];
  // instruction u of a stage's kC copies (nothing past the last stage); the
  // scales, by way of registers, with the first
  constexpr int kC = kCL + XP * kXL;
  const auto copy = [&](int s, int u) {
    uint8_t *const buf = lds + (s & 1) * kBuffer;
    const uint32_t k0 = (uint32_t)s * kStage;
    const bool in = s < stages;
    if (u < kCL) {
      const uint32_t piece = cpiece ^ (uint32_t)((wave * (BN / WAVES / 16) + u) & 3);
      const uint32_t at = !in || k0 + 32 * piece < kb ? crow + 16 * piece : kOutOfRange;
      dma16(cview(u), buf + (wave * (BN / WAVES) + 16 * u) * 64, at, in ? k0 / 2 : kOutOfRange);
    } else {
      const int p = (u - kCL) / kXL, i = (u - kCL) % kXL;
      const uint32_t piece = xpiece ^ (uint32_t)((wave * (BM / WAVES) + 4 * i) & 15);
      const uint32_t at = !in || k0 + 8 * piece < kb ? xrow + 16 * piece : kOutOfRange;
      dma16(xview(p), buf + kCodes + kScales + p * kPart + (wave * (BM / WAVES) + 4 * i) * 256, at,
            in ? 4u * i * xp + k0 * 2 : kOutOfRange);
    }
    if (u == 0 && in) {
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
      *reinterpret_cast<uint64_t *>(lds + (s & 1) * kBuffer + kCodes + (wave * (32 * NF) + lane + 64 * i) * 8) = sreg[i];
  };

  // ---- operands.  Half stage p (0, 1) of a stage is four K steps.
  float16_t acc[NF][MF];
  const int wrow = wave * (32 * NF) + ((r >> 2) & 1) * 16 + (r >> 3) * 4 + (r & 3);
  u32x4_t c[2][NF];
  Scale<MX> sc[2][NF];
  bf16x8_t a[2][NF], b[2][XP][MF];
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
  const auto read_x = [&](int s, int p, int j, int u, int into) {
    const uint8_t *const buf = lds + (s & 1) * kBuffer + kCodes + kScales;
    const int k = u / MF, m = u % MF;
    b[into][k][m] = *reinterpret_cast<const bf16x8_t *>(buf + k * kPart + (32 * m + r) * 256 +
                                                        16 * ((8 * p + 4 * h + j) ^ (r & 15)));
  };
  // a quarter of a fragment's 8 weights (MXFP4: all of them for quarter 0)
  // MXFP4 weights are decoded at a quarter: those of the largest scales would
  // pass bf16's range.  Where a scale lies too near either end for the
  // conversion's own (and is not that of zeros), the tile is done once more, FAR,
  // by products.
  uint32_t ends = 0;
  const auto check = [&](int p) {
    if constexpr (MX) {
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const uint32_t raw = sc[p][f].raw, any = (c[p][f][0] | c[p][f][1] | c[p][f][2] | c[p][f][3]) & 0x77777777u;
        ends |= raw >= 253 ? 1u : raw < 3 ? any : 0u;
      }
    }
  };
  const auto decode = [&](int p, int j, int f, int quarter, int into, auto far) {
    if constexpr (MX) {
      if (quarter) return;
      if constexpr (far.value) a[into][f] = decode8<false>(c[p][f][j], sc[p][f].quarter());
      else a[into][f] = decode8<true>(c[p][f][j], __uint_as_float((max(sc[p][f].raw, 3u) - 2) << 23));
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
  constexpr int NU = NF * MF * XP, ND = 4 * NF;      // MFMAs and quarters to decode of a K step
  // K step j of half p of stage s: operands of `cur` are there; the next step's
  // go to the other.
  const auto step = [&](int s, auto half, auto kstep, auto far) {
    constexpr int p = decltype(half)::value, j = decltype(kstep)::value;
    constexpr int cur = j & 1, nxt = cur ^ 1, np = j == 3 ? p ^ 1 : p, nj = (j + 1) & 3;
    if constexpr (p == 1 && j == 3) {
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(wait_vm(0));       // this wave's copies of the next stage
      put_scales(s + 1);
      __syncthreads();
      read_codes(s + 1, 0);
    } else if constexpr (p == 0 && j == 2) {
      read_codes(s, 1);
    }
    constexpr int kLag = j == 3 && NU >= 4 ? NU / 4 : 0;      // codes just read are not there yet
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      // snake order: one operand stays the same to the next MFMA
      const int k = i / (NF * MF), m = i / NF % MF, f = (m & 1) ? NF - 1 - i % NF : i % NF;
      acc[f][m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[cur][f], b[cur][k][m], acc[f][m], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      // the next step's x in the first half of the step, copies over all of it
      constexpr int kHalf = (NU + 1) / 2;
      if (i < kHalf) {
#pragma unroll
        for (int u = i * XP * MF / kHalf; u < (i + 1) * XP * MF / kHalf; ++u)
          read_x(p == 1 && j == 3 ? s + 1 : s, np, nj, u, nxt);
      }
      if (p == 0) {
#pragma unroll
        for (int u = (j * NU + i) * kC / (4 * NU); u < (j * NU + i + 1) * kC / (4 * NU); ++u) copy(s + 1, u);
      }
      if (j == 3 && i == kLag && !far.value) check(np);
      if (i >= kLag) {
        const int d0 = (i - kLag) * ND / (NU - kLag), d1 = (i - kLag + 1) * ND / (NU - kLag);
#pragma unroll
        for (int d = d0; d < d1; ++d) decode(np, nj, d / 4, d % 4, nxt, far);
      }
    }
  };

  const auto run = [&](auto far) {
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[f][m][i] = 0.0f;
#pragma unroll
    for (int u = 0; u < kC; ++u) copy(0, u);
    __builtin_amdgcn_s_waitcnt(wait_vm(0));
    put_scales(0);
    __syncthreads();
    read_codes(0, 0);
#pragma unroll
    for (int u = 0; u < XP * MF; ++u) read_x(0, 0, 0, u, 0);
    if (!far.value) check(0);
#pragma unroll
    for (int d = 0; d < ND; ++d) decode(0, 0, d / 4, d % 4, 0, far);
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I3 = std::integral_constant<int, 3>;
    for (int s = 0; s < stages; ++s) {
      step(s, I0{}, I0{}, far);
      step(s, I0{}, I1{}, far);
      step(s, I0{}, I2{}, far);
      step(s, I0{}, I3{}, far);
      step(s, I1{}, I0{}, far);
      step(s, I1{}, I1{}, far);
      step(s, I1{}, I2{}, far);
      step(s, I1{}, I3{}, far);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  if (stages == 0) {
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[f][m][i] = 0.0f;
  } else {
    run(std::false_type());
    if constexpr (MX) {
      uint32_t *const far = reinterpret_cast<uint32_t *>(lds + 2 * kBuffer);
      const bool any = __any(ends != 0);
      if (lane == 0) far[wave] = any;
      __syncthreads();
      uint32_t all = 0;
#pragma unroll
      for (int i = 0; i < WAVES; ++i) all |= far[i];
      if (__builtin_amdgcn_readfirstlane(all)) run(std::true_type());
    }
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

template <bool MX, int XP, int WAVES, int NF, int MF>
hipError_t grouped(const Stack &w, const Groups &g, const Rows<uint16_t> &x, int64_t part, void *y, int y_bf16, int64_t ldy,
                   int fill, hipStream_t stream) {
  constexpr int BN = 32 * WAVES * NF, BM = 32 * MF;
  const int64_t tiles_n = (w.N + BN - 1) / BN, tiles_m = g.rows / BM + std::min<int64_t>(g.count, g.rows);
  k_grouped<MX, XP, WAVES, NF, MF><<<(unsigned)((tiles_n * tiles_m + kXcds - 1) / kXcds * kXcds), 64 * WAVES, 0, stream>>>(
      w, g, x, part, y, y_bf16, ldy, (int)tiles_n, fill);
  return hipGetLastError();
}

// Whether a call's x is copied from where it lies.
bool copied_as_is(const void *x, int64_t ldx, bool f32) {
  return !f32 && (uintptr_t)x % 4 == 0 && ldx % 2 == 0 && ldx < (1LL << 24);
}

template <bool MX>
hipError_t grouped_tiles(const GroupedProduct &p, const Stack &w, const Groups &g, hipStream_t stream) {
  const bool f32 = p.x_dtype == 0;
  Rows<uint16_t> x = {(const uint16_t *)p.x, p.ldx};
  const int64_t part = p.rows * p.k;
  if (p.k > 0 && !copied_as_is(p.x, p.ldx, f32)) {
    const unsigned grid = (unsigned)std::min<int64_t>((part / 8 + 255) / 256, 1 << 14);
    if (f32) k_parts<<<grid, 256, 0, stream>>>((const float *)p.x, p.ldx, p.rows, p.k, (uint16_t *)p.ws);
    else k_parts<<<grid, 256, 0, stream>>>((const uint16_t *)p.x, p.ldx, p.rows, p.k, (uint16_t *)p.ws);
    x = {(const uint16_t *)p.ws, p.k};
  }
  const int yb = p.y_dtype == 1;
  const int64_t groups = std::min(p.experts, p.rows), each = (p.rows + groups - 1) / groups;
  if (f32) {
    // tiles of 512 x 32 against 256 x 64, us, 24 groups of 5120 x 1280: 64 rows
    // each 86 / 80, as many on average with few groups alike 113 / 128, 256 each
    // 315 / 288
    if (each <= 96) return grouped<MX, 3, 8, 2, 1>(w, g, x, part, p.y, yb, p.ldy, p.fill, stream);
    return grouped<MX, 3, 4, 2, 2>(w, g, x, part, p.y, yb, p.ldy, p.fill, stream);
  }
  // tiles of 512 x 128 where groups fill them and there are some for most CUs,
  // else of 256 x 64; us, 16 groups of 4096 x 4096 of unlike sizes, 64 rows on
  // average 98 / 81, 96 97 / 122, 128 104 / 125, 512 308 / 339
  const int64_t large = (w.N + 511) / 512 * (p.rows / 128 + groups / 2);
  if (each > 80 && 8 * large >= 5 * device_cus())
    return grouped<MX, 1, 8, 2, 4>(w, g, x, part, p.y, yb, p.ldy, p.fill, stream);
  return grouped<MX, 1, 4, 2, 2>(w, g, x, part, p.y, yb, p.ldy, p.fill, stream);
}

// Whether a product goes by the matvec's tiles, which read the weights once for
// every 16 rows of a group, at some 6 TB/s from whichever memory holds them,
// behind a start of 6 us; the tiles here take some 1.5 us a stage of 128 k for
// every two a CU.  us, 16 groups of 4096 x 4096, 4 rows each on average 38 /
// 54, 16 50 / 56, 32 71 / 80, 64 110 / 81.
bool by_matvec_tiles(int64_t experts, int64_t n, int64_t k, int64_t rows) {
  if (!grouped_tiles_fit(experts, k, rows)) return false;
  const int64_t groups = std::min(experts, rows);
  const double reads = (double)(rows / 16 + groups) * n * k * 0.53 / 6.0e6;
  const double rounds = std::max(1.0, (double)((n + 255) / 256) * (rows / 64 + groups / 2) / (2 * device_cus()));
  return reads < rounds * 1.5 * ((k + kStage - 1) / kStage);
}

// ------------------------------------------------------ weight gradient --

// Tokens run along the reduction here, and lie down the columns of both
// operands: a stage's rows go to LDS as they are, by DMA, and the lanes fetch
// columns with transposing reads (16 lanes take 4 rows of 16 columns, and each
// leaves with 4 rows of its own column), those of the next 16 tokens between the
// MFMAs of these.  Chunk c (32 bytes, 16 columns) of row t lies in place
// c ^ (2 (t % 4)), so that the 4 rows of a transposing read's two neighbouring
// chunks fall on different banks.  Of the parts of two float32 operands the
// products from hi hi to mid mid are taken; those left out are below 2^-25 of
// the whole.
//
// Two workgroups a CU, so that one multiplies while the other stores: tiles of
// 128 columns of dy by 256 of x and stages of 32 tokens for bf16, 128 by 128
// and 16 tokens for the parts of float32.

// Operands as the kernel copies them: rows of whole words.  Others are brought
// to that first: [parts][rows][round8(cols)] in the workspace, zeros behind a
// row's end.
int64_t round8(int64_t v) { return (v + 7) / 8 * 8; }
// Both operands in one launch where they are of one type: its start counts (777
// rows of 1283 and 2050 columns in two launches 14 us, in one 9 to 11).
template <typename X> struct Pad {
  const X *x;
  int64_t ld, cols;
  uint16_t *out;
};
template <typename X>
__global__ __launch_bounds__(256) void k_pad(Pad<X> first, Pad<X> second, int64_t rows) {
  const int64_t before = rows * ((first.cols + 7) / 8), every = before + rows * ((second.cols + 7) / 8);
  for (int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x; j < every; j += (int64_t)gridDim.x * 256) {
    const Pad<X> m = j < before ? first : second;
    const int64_t pieces = (m.cols + 7) / 8, all = rows * pieces, i = j < before ? j : j - before;
    Row8<X> q;
    load_row8(q, m.x + i / pieces * m.ld, i % pieces * 8, m.cols);
    if constexpr (sizeof(X) == 2) {
      *reinterpret_cast<u32x4_t *>(m.out + i * 8) = q.r;
    } else {
      const Parts p = split8_nearest(q);
#pragma unroll
      for (int k = 0; k < 3; ++k) *reinterpret_cast<u32x4_t *>(m.out + (k * all + i) * 8) = p.v[k];
    }
  }
}

// A matrix as the kernel copies it, with an even number of columns; its parts
// lie `part` elements apart.
struct Operand16 {
  const uint16_t *p;
  int64_t ld, cols, part;
};

// The tiles of a group that an XCD takes: a run of an eighth of every group's,
// since groups differ in length.  The grid has this for each XCD and group.
__host__ __device__ __forceinline__ int wgrad_quota(int tiles) { return (tiles + kXcds - 1) / kXcds; }

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
// 4 neighbouring elements k .. of a row of K.
__device__ __forceinline__ void store4(void *out, int bf16, int64_t row, int64_t k, int64_t K, const f32x4_t &v) {
  if (k + 4 <= K) {
    if (bf16) *reinterpret_cast<u32x2_a2 *>((uint16_t *)out + row + k) = (u32x2_a2){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    else *reinterpret_cast<f32x4_a4 *>((float *)out + row + k) = v;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (k + i >= K) continue;
    if (bf16) ((uint16_t *)out)[row + k + i] = (uint16_t)pack_bf16(v[i], 0.0f);
    else ((float *)out)[row + k + i] = v[i];
  }
}

// DP, XP: parts of dy and x; FK: fragments of 32 columns of x a wave (the tile
// is two waves of 64 columns of dy by two of 32 FK of x).
template <int DP, int XP, int FK, int TOKENS> struct Wgrad {
  static constexpr int kTK = 64 * FK, kRing = 3;
  static constexpr int kRowD = 256, kRowX = 2 * kTK;                  // bytes of a row in LDS
  static constexpr int kPartD = TOKENS * kRowD, kPartX = TOKENS * kRowX;
  static constexpr int kX = DP * kPartD, kStage = kX + XP * kPartX;
  // DMA instructions (1 KB: 4 rows of 256 bytes, or 2 of 512) a wave: of a
  // part, of a stage; a wave copies TOKENS / 4 rows
  static constexpr int kID = kPartD / 4096, kIX = kPartX / 4096, kCopies = DP * kID + XP * kIX;
  static constexpr int kPairs = DP * XP == 9 ? 6 : DP * XP;           // products of parts that count
  static constexpr int kMfma = kPairs * 2 * FK, kReads = 2 * DP + FK * XP;

  struct Operands {
    bf16x8_t a[2][DP][2], b[2][XP][FK];
  };
  struct Copy {
    __amdgpu_buffer_rsrc_t dv[DP], xv[XP];
    uint32_t dat, xat[2], dp, xp;            // lane offsets (x: of even and odd instructions), a row's bytes
    int wave;
    // copy u of a stage at `to`
    __device__ __forceinline__ void run(int u, uint8_t *to) const {
      const int row = wave * (TOKENS / 4);
      if (u < DP * kID) {
        const int p = u / kID, r = row + 4 * (u % kID);
        dma16(dv[p], to + p * kPartD + r * kRowD, dat, (uint32_t)r * dp);
      } else {
        const int p = (u - DP * kID) / kIX, i = (u - DP * kID) % kIX, r = row + 1024 / kRowX * i;
        dma16(xv[p], to + kX + p * kPartX + r * kRowX, xat[i & 1], (uint32_t)r * xp);
      }
    }
  };
  // The MFMAs of 16 tokens, whose operands are set P: `from` is where those of
  // the next 16 lie, `to` where copies go, which is another place of the ring.
  // (Two pointers that do not meet: a transposing read would else wait for every
  // copy under way.)
  template <int P, bool COPY>
  static __device__ __forceinline__ void step(const char *__restrict__ from, uint8_t *__restrict__ to,
                                              float16_t (&acc)[2][FK], Operands &o, const uint32_t (&dat)[2],
                                              const uint32_t (&xat)[FK], const Copy &c) {
#pragma unroll
    for (int i = 0; i < kMfma; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      // pairs of parts (0 0) (0 1) (0 2) (1 0) (1 1) (2 0), as far as there are parts
      const int pair = i / (2 * FK), u = i % (2 * FK), f = u / FK, q = (f & 1) ? FK - 1 - u % FK : u % FK;
      const int p = XP == 1 ? pair : DP == 1 ? 0 : pair < 3 ? 0 : pair < 5 ? 1 : 2;
      const int k = XP == 1 ? 0 : DP == 1 ? pair : pair < 3 ? pair : pair < 5 ? pair - 3 : 0;
      acc[f][q] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(o.a[P][p][f], o.b[P][k][q], acc[f][q], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      // the reads in the first three quarters, the copies after the first two MFMAs
      constexpr int kSlots = kMfma * 3 / 4;
      if (i < kSlots) {
#pragma unroll
        for (int r = i * kReads / kSlots; r < (i + 1) * kReads / kSlots; ++r) {
          if (r < 2 * DP) o.a[P ^ 1][r / 2][r % 2] = lds_column(from + r / 2 * kPartD + dat[r % 2], kRowD);
          else o.b[P ^ 1][(r - 2 * DP) / FK][(r - 2 * DP) % FK] =
                   lds_column(from + (r - 2 * DP) / FK * kPartX + xat[(r - 2 * DP) % FK], kRowX);
        }
      }
      if (COPY && i >= 2) {
#pragma unroll
        for (int r = (i - 2) * kCopies / (kMfma - 2); r < (i - 1) * kCopies / (kMfma - 2); ++r) c.run(r, to);
      }
    }
  }
};

// Every group's tiles are written, zeros for a group without rows; with several
// shares of a group's tokens (gridDim.y) the sums go to partial[share] instead.
template <int DP, int XP, int FK, int TOKENS>
__global__ __launch_bounds__(kThreads, 2) void k_grouped_wgrad(Groups g, Operand16 dy, Operand16 x, void *dw, int dw_bf16,
                                                               float *partial, int64_t N, int64_t K, int tiles_n,
                                                               int tiles_k) {
  using W = Wgrad<DP, XP, FK, TOKENS>;
  __shared__ __align__(16) uint8_t lds[W::kRing * W::kStage];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tiles = tiles_n * tiles_k, quota = wgrad_quota(tiles);
  const int e = blockIdx.x / kXcds / quota, at = (int)(blockIdx.x % kXcds) * quota + (int)(blockIdx.x / kXcds) % quota;
  if (at >= tiles) return;
  const int per = 16 * tiles_k, first_n = at / per * 16, gsz = min(tiles_n - first_n, 16);
  const int64_t n0 = (int64_t)(first_n + at % per % gsz) * 128, k0 = (int64_t)(at % per / gsz) * W::kTK;
  int64_t begin = uniform64(g.at(e)), end = max(uniform64(g.at(e + 1)), begin);
  if (gridDim.y > 1) {
    // a share is a run of whole stages
    const int64_t all = (end - begin + TOKENS - 1) / TOKENS, from = all * blockIdx.y / gridDim.y, to = all * (blockIdx.y + 1) / gridDim.y;
    end = min(end, begin + to * TOKENS);
    begin = min(begin + from * TOKENS, end);
  }
  const int stages = (int)((end - begin + TOKENS - 1) / TOKENS);

  typename W::Copy c;
  c.wave = wave;
  c.dp = (uint32_t)(dy.ld * 2);
  c.xp = (uint32_t)(x.ld * 2);
  // lane l copies slot l % 16 (16 bytes) of row l / 16, or l % 32 of row l / 32
  c.dat = (uint32_t)(lane >> 4) * c.dp + 16 * (uint32_t)((lane & 15) ^ (4 * (lane >> 4)));
#pragma unroll
  for (int i = 0; i < 2; ++i)
    c.xat[i] = FK == 4 ? (uint32_t)(lane >> 5) * c.xp + 16 * (uint32_t)((lane & 31) ^ (4 * (2 * i + (lane >> 5))))
                       : (uint32_t)(lane >> 4) * c.xp + 16 * (uint32_t)((lane & 15) ^ (4 * (lane >> 4)));
  const auto aim = [&](int s) {
    const int64_t t0 = begin + (int64_t)s * TOKENS, rows = min(end - t0, (int64_t)TOKENS);
    const auto view = [&](const Operand16 &m, int p, uint32_t pitch, int64_t c0, int64_t most) {
      return make_rsrc(m.p + (rows > 0 ? p * m.part + t0 * m.ld + c0 : 0),
                       rows > 0 ? (uint32_t)(rows - 1) * pitch + (uint32_t)most * 2 : 0u);
    };
#pragma unroll
    for (int p = 0; p < DP; ++p) c.dv[p] = view(dy, p, c.dp, n0, min(dy.cols - n0, (int64_t)128));
#pragma unroll
    for (int p = 0; p < XP; ++p) c.xv[p] = view(x, p, c.xp, k0, min(x.cols - k0, (int64_t)W::kTK));
  };

  float16_t acc[2][FK];
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int q = 0; q < FK; ++q)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[f][q][i] = 0.0f;
  // the lane's 4 columns of one row of a transposing read, for each fragment, in
  // the first 16 tokens of a stage and the second
  const int trow = 8 * (lane >> 5) + ((lane >> 2) & 3), turn = 2 * ((lane >> 2) & 3);
  uint32_t dat[2][2], xat[2][FK];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int f = 0; f < FK; ++f) {
      const int chunk = 2 * f + ((lane >> 4) & 1);
      if (f < 2) dat[h][f] = (trow + 16 * h) * W::kRowD + 32 * (((wave >> 1) * 4 + chunk) ^ turn) + 8 * (lane & 3);
      xat[h][f] = W::kX + (trow + 16 * h) * W::kRowX + 32 * (((wave & 1) * 2 * FK + chunk) ^ turn) + 8 * (lane & 3);
    }
  typename W::Operands o;
  if (stages > 0) {
    const auto place = [&](int turn_of) { return lds + turn_of * W::kStage; };
    constexpr int kLead = TOKENS == 32 ? 2 : 3;          // stages copied before the first is used
#pragma unroll
    for (int s = 0; s < kLead; ++s) {
      aim(s);
#pragma unroll
      for (int i = 0; i < W::kCopies; ++i) c.run(i, place(s));
    }
    constexpr int kStay = wait_vm((kLead - 1) * W::kCopies) & ~0x0F00;
    meet<kStay>();
#pragma unroll
    for (int p = 0; p < DP; ++p)
#pragma unroll
      for (int f = 0; f < 2; ++f) o.a[0][p][f] = lds_column((const char *)lds + p * W::kPartD + dat[0][f], W::kRowD);
#pragma unroll
    for (int p = 0; p < XP; ++p)
#pragma unroll
      for (int f = 0; f < FK; ++f) o.b[0][p][f] = lds_column((const char *)lds + p * W::kPartX + xat[0][f], W::kRowX);
    int now = 0, next = 1, last = 2;             // places of this stage, the next, and the one behind it
    const auto move = [&]() {
      const int was = now;
      now = next;
      next = last;
      last = was;
    };
    if constexpr (TOKENS == 32) {
      for (int s = 0; s < stages; ++s) {
        aim(s + 2);
        W::template step<0, true>((const char *)place(now), place(last), acc, o, dat[1], xat[1], c);
        // this wave's copies of the next stage (those of one more stay under way,
        // which a fence would wait for) and its reads of this one
        meet<(wait_vm(W::kCopies) & ~0x0F00)>();
        W::template step<1, false>((const char *)place(next), place(last), acc, o, dat[0], xat[0], c);
        move();
      }
    } else {
      // (the stage's own operands are in registers: its place takes the copies)
      for (int s = 0; s < stages; s += 2) {
        meet<(wait_vm(W::kCopies) & ~0x0F00)>();
        aim(s + 3);
        W::template step<0, true>((const char *)place(next), place(now), acc, o, dat[0], xat[0], c);
        move();
        if (s + 1 >= stages) break;
        meet<(wait_vm(W::kCopies) & ~0x0F00)>();
        aim(s + 4);
        W::template step<1, true>((const char *)place(next), place(now), acc, o, dat[0], xat[0], c);
        move();
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(wait_vm(0));        // nothing is left that writes LDS
  }
  // register i of a fragment is row 8 (i / 4) + 4 h + i % 4, the lane its
  // column; turned over the quads (pairs) a lane has neighbours of fragment
  // lane % 4 (stores of 16 bytes a lane, whole lines: with 4 the wave's 128 of
  // them held up the copies of the CU's other workgroup, 8192 rows of 8 experts
  // 5120 x 5120 530 -> 490 us)
  const bool split = gridDim.y > 1;
  void *const out = split ? (void *)(partial + (int64_t)blockIdx.y * g.count * N * K) : dw;
  const int bf16 = split ? 0 : dw_bf16;
  const int64_t base = (int64_t)e * N;
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int64_t n = n0 + (wave >> 1) * 64 + 32 * f + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3);
      if constexpr (FK == 4) {
        const int64_t k = k0 + (wave & 1) * 128 + 32 * (lane & 3) + (lane & 28);
        const f32x4_t v = quad_turn(acc[f][0][i], acc[f][1][i], acc[f][2][i], acc[f][3][i]);
        if (n < N && k < K) store4(out, bf16, (base + n) * K, k, K, v);
      } else {
        // two fragments: rows n and n + 1 of the pair (i, i + 1) make the quad's four
        if (i & 1) continue;
        const f32x4_t v = quad_turn(acc[f][0][i], acc[f][1][i], acc[f][0][i + 1], acc[f][1][i + 1]);
        const int64_t m = n + ((lane >> 1) & 1), k = k0 + (wave & 1) * 64 + 32 * (lane & 1) + (lane & 28);
        if (m < N && k < K) store4(out, bf16, (base + m) * K, k, K, v);
      }
    }
}

// The shares' sums, in their order.
__global__ __launch_bounds__(256) void k_wgrad_join(const float *partial, int shares, int64_t size, void *dw, int dw_bf16) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < size; i += (int64_t)gridDim.x * 256) {
    float v = 0.0f;
    for (int z = 0; z < shares; ++z) v += partial[z * size + i];
    if (dw_bf16) ((uint16_t *)dw)[i] = (uint16_t)pack_bf16(v, 0.0f);
    else ((float *)dw)[i] = v;
  }
}

// Shares of the tokens: until there is work for two workgroups a CU, at least
// 128 tokens of an average group each.
int wgrad_shares(int64_t experts, int64_t n, int64_t k, int64_t rows, bool narrow) {
  const int64_t tk = narrow ? 256 : 128, tiles = (n + 127) / 128 * ((k + tk - 1) / tk);
  const int64_t groups = std::max<int64_t>(1, std::min(experts, rows));
  const int64_t want = std::min(2 * (int64_t)device_cus() / (tiles * groups), rows / groups / 128);
  return (int)std::min<int64_t>(std::max<int64_t>(want, 1), 64);
}
// Whether a matrix is copied from where it lies.
bool words(const void *p, int64_t ld, int64_t cols, bool f32) {
  return !f32 && (uintptr_t)p % 4 == 0 && ld % 2 == 0 && cols % 2 == 0 && ld < (1LL << 24);
}

template <int DP, int XP> hipError_t wgrad(const GroupedWgrad &p, hipStream_t stream) {
  constexpr bool narrow = DP * XP == 1;
  constexpr int FK = narrow ? 4 : 2, kTokens = narrow ? 32 : 16;
  const int shares = wgrad_shares(p.experts, p.n, p.k, p.rows, narrow);
  float *const partial = (float *)p.ws;
  uint16_t *space = (uint16_t *)((char *)p.ws + (shares > 1 ? 4 * shares * p.experts * p.n * p.k : 0));
  space += (8 - (uintptr_t)space / 2 % 8) % 8;
  const auto ready = [&](const void *m, int64_t ld, int64_t cols, bool f32) {
    if (p.rows == 0 || words(m, ld, cols, f32)) return Operand16{(const uint16_t *)m, ld, cols, 0};
    const int64_t padded = round8(cols);
    const Operand16 o = {space, padded, padded, p.rows * padded};
    space += (f32 ? 3 : 1) * p.rows * padded;
    return o;
  };
  const Operand16 dy = ready(p.dy, p.lddy, p.n, DP == 3), x = ready(p.x, p.ldx, p.k, XP == 3);
  // an operand that is where it was takes no part
  const auto pad = [&](auto zero, bool with_dy, bool with_x) {
    using T = decltype(zero);
    Pad<T> a = {(const T *)p.dy, p.lddy, p.n, (uint16_t *)dy.p}, b = {(const T *)p.x, p.ldx, p.k, (uint16_t *)x.p};
    if (!with_dy || dy.p == p.dy) a.cols = 0;
    if (!with_x || x.p == p.x) b.cols = 0;
    const int64_t pieces = p.rows * (round8(a.cols) + round8(b.cols)) / 8;
    if (pieces > 0)
      k_pad<<<(unsigned)std::min<int64_t>((pieces + 255) / 256, 1 << 14), 256, 0, stream>>>(a, b, p.rows);
  };
  pad(0.0f, DP == 3, XP == 3);
  pad((uint16_t)0, DP == 1, XP == 1);
  const Groups g = {p.offsets, p.index_bits == 64, (int)p.experts, p.rows, 0};
  const int64_t tn = (p.n + 127) / 128, tk = (p.k + 64 * FK - 1) / (64 * FK);
  const dim3 grid((unsigned)(wgrad_quota((int)(tn * tk)) * kXcds * p.experts), (unsigned)shares);
  k_grouped_wgrad<DP, XP, FK, kTokens><<<grid, kThreads, 0, stream>>>(g, dy, x, p.dw, p.dw_dtype == 1, partial, p.n, p.k,
                                                                     (int)tn, (int)tk);
  if (shares > 1) {
    const int64_t size = p.experts * p.n * p.k;
    k_wgrad_join<<<(unsigned)std::min<int64_t>((size + 255) / 256, 1 << 14), 256, 0, stream>>>(partial, shares, size, p.dw,
                                                                                             p.dw_dtype == 1);
  }
  return hipGetLastError();
}

}  // namespace

int64_t grouped_wgrad_workspace_bytes(int64_t experts, int64_t n, int64_t k, int64_t rows, bool dy_f32, bool x_f32) {
  if (n == 0 || k == 0) return 0;
  const int shares = wgrad_shares(experts, n, k, rows, !dy_f32 && !x_f32);
  // (a bf16 matrix may lie at any place: room for a copy)
  return (shares > 1 ? 4 * shares * experts * n * k + 16 : 0) +
         2 * rows * (round8(n) * (dy_f32 ? 3 : 1) + round8(k) * (x_f32 ? 3 : 1));
}
hipError_t launch_grouped_wgrad(const GroupedWgrad &p, hipStream_t stream) {
  if (p.n == 0 || p.k == 0) return hipSuccess;
  if (p.dy_dtype == 1) return p.x_dtype == 1 ? wgrad<1, 1>(p, stream) : wgrad<1, 3>(p, stream);
  return p.x_dtype == 1 ? wgrad<3, 1>(p, stream) : wgrad<3, 3>(p, stream);
}

int64_t grouped_workspace_bytes(int64_t experts, int64_t n, int64_t k, int64_t rows, bool f32) {
  if (n == 0 || rows == 0 || k == 0) return 0;
  if (by_matvec_tiles(experts, n, k, rows)) return grouped_tiles_workspace_bytes(experts, n, k, rows, f32);
  // (a bf16 x may lie at any place: room for a copy)
  return rows * k * (f32 ? 6 : 2);
}

hipError_t launch_grouped(const GroupedProduct &p, hipStream_t stream) {
  if (p.n == 0 || p.rows == 0) return hipSuccess;
  const int64_t block = p.mx ? 32 : 16, rows = p.transposed ? 1 : p.n;
  const int64_t pitch = p.transposed ? p.experts * p.k : p.k, step = rows * p.k;
  const Stack w = {p.codes, p.scales, p.meta, p.n, p.k, pitch / 2, step / 2, pitch / block, step / block};
  if (by_matvec_tiles(p.experts, p.n, p.k, p.rows))
    return launch_grouped_tiles(p, w.code_pitch, w.code_step, w.scale_pitch, w.scale_step, stream);
  const Groups g = {p.offsets, p.index_bits == 64, (int)p.experts, p.rows, 0};
  return p.mx ? grouped_tiles<true>(p, w, g, stream) : grouped_tiles<false>(p, w, g, stream);
}

}  // namespace nvfp4
