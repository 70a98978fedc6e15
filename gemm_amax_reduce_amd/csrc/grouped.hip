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
