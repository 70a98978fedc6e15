// matvec.hip -- products of a few rows of activations with a 4-bit weight
// matrix for gfx950 (the single-token form of the linear layer):
//
//   NVFP4   y[t][n] = g * sum_k x[t][k] * e2m1(code[n][k]) * e4m3(scale[n][k/16])
//   MXFP4   y[t][n] =     sum_k x[t][k] * e2m1(code[n][k]) * 2^(scale[n][k/32] - 127)
//
// The weights are read once and everything else is small, so the kernels are
// bound by the N * K / 2 bytes of codes and the scales beside them.  Two
// forms, both with 32 consecutive k of one weight row per lane and load (16
// bytes of codes, whole scale groups):
//
//  * k_matvec_row, up to 4 tokens: a wave walks whole weight rows (contiguous
//    runs of 1 KB per load), its share of x stays in registers, and a pair
//    of products is one v_dot2_f32_bf16 on decoded codes; the block scale is
//    applied to a block's sum.  Half an instruction per weight and half a
//    one per product.
//  * k_matvec_tile, more tokens: tiles of 16 weight rows on the 16x16x32
//    bf16 MFMA with the weights as the A operand and up to 16 tokens as the
//    B operand, so 1 to 16 bf16 tokens cost the same (f32 tokens take three
//    columns each: one slab of 16 up to 5 of them, two up to 10, three up to
//    16).  A lane's 32 k enter four MFMAs; the k order of an MFMA is free as
//    long as both operands agree.
//    The block scale has to be multiplied into every weight here, about two
//    instructions per NVFP4 weight.
//
// A decoded weight q * S has at most 6 significant bits (2 of E2M1, 4 of
// E4M3) and an exponent in bf16's range (MXFP4 at a quarter where its scales
// are at their largest), so it is exact in bf16, and so is bf16 x.  A float32
// x is split into three bf16 parts, x = hi + mid + lo, each of 8 bits: exact
// for every value whose low part does not fall below the bf16 range.  Products
// are exact in binary32 and added there; the tensor scale g is applied once to
// the sum.
//
// Measured on one MI355X, kernels alone, two sets of weights in turn: rows, one
// bf16 token, NVFP4 5120 x 5120 5.4 us (2.7 TB/s: 2.3 us of reading behind a
// start of 3), 20480 x 5120 12.6 us (4.7 TB/s); tiles, 8 bf16 tokens, 131075 x
// 5120 73.9 us (5.1 TB/s), 5 f32 tokens of MXFP4 5120 x 20480 17.0 us and 3.9
// us for joining the ranges of K.  Whole calls with weights that no cache
// holds: one bf16 token 20480 x 5120 12.8 us, MXFP4 13.4, 131075 x 5120 58.2
// (6.5 TB/s) and 59.1; 8 bf16 tokens 20480 x 5120 17.3; f32, NVFP4, 16 tokens
// 20480 x 5120 (three slabs) 29.6, 8 tokens 131075 x 5120 (two slabs) 111.
#include "gemm_common.h"
#include "groups.h"
#include "nvfp4_device.h"
#include "nvfp4_kernels.h"
#include "operands.h"
#include "row_common.h"

#include <algorithm>
#include <type_traits>

namespace nvfp4 {

namespace {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_a8 __attribute__((ext_vector_type(4), aligned(8)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));
typedef uint32_t u32x2_a1 __attribute__((ext_vector_type(2), aligned(1)));

// ------------------------------------------------------------- operands --

// The same as 8 f16, where every q * S is exact, too: one conversion and one
// packed product for two weights, half of what the bf16 form takes.
__device__ __forceinline__ half8_t decode8_f16(uint32_t w, half2_t s) {
  half2_t v[4];
  v[0] = __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0)) * s;
  v[1] = __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1)) * s;
  v[2] = __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2)) * s;
  v[3] = __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3)) * s;
  return (half8_t){v[0][0], v[0][1], v[1][0], v[1][1], v[2][0], v[2][1], v[3][0], v[3][1]};
}

// 32 consecutive x of one token, 16-byte pieces.
template <typename X> struct Act {
  static constexpr int kPieces = 32 * sizeof(X) / 16;
  u32x4_t v[kPieces];
};

// A lane's last load of a row may reach past the end: it is moved back to the
// row's last 32 k, and meets zeros where it is not the row's own.  Makes k
// where to load from; returns by how many it was moved, 32 if nothing of the
// row is left.
__device__ __forceinline__ int last_window(int64_t &k, int64_t K) {
  const int64_t at = min(k, K - 32);
  const int drop = (int)min(k - at, (int64_t)32);
  k = at;
  return drop;
}

__device__ __forceinline__ void store_y(void *y, int y_bf16, int64_t at, float v) {
  if (y_bf16) ((uint16_t *)y)[at] = (uint16_t)pack_bf16(v, 0.0f);
  else ((float *)y)[at] = v;
}

// Up to 4 consecutive outputs, positions at .. at + 3, none from `end` on.
__device__ __forceinline__ void store_rows(void *y, int y_bf16, int64_t at, int64_t end, const f32x4_t &v) {
  if (at + 4 <= end && y_bf16) {
    *reinterpret_cast<u32x2_a2 *>((uint16_t *)y + at) = (u32x2_t){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
  } else if (at + 4 <= end) {
    *reinterpret_cast<f32x4_a4 *>((float *)y + at) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (at + i < end) store_y(y, y_bf16, at + i, v[i]);
  }
}

// ---------------------------------------------------- up to 16 tokens --

constexpr int kStepK = 128;      // k of one MFMA step: 4 lanes a row, 32 each
constexpr int kTokens = 16;      // tokens of a launch's y index
// Waves of a workgroup, at most, and those of them that multiply (three
// slabs: their sums take 6 KB of LDS a wave).  From three waves on (or with
// several slabs), one more adds up what the others leave: the additions'
// latency would else stand between one tile's barrier and the next.
constexpr int kTileWaves = 12;
constexpr int max_waves(int slabs) { return slabs == 3 ? 8 : kTileWaves - 1; }
bool has_helper(int waves, int slabs) { return waves > 2 || slabs > 1; }
constexpr int kTurnBytes = 4096; // 16 columns x 128 k of bf16

// The B operand's columns.  bf16: one column a token.  float32: three
// columns a token, the parts hi, mid and lo, so that one MFMA serves five
// tokens and the parts are added at the end.
template <typename X> constexpr int columns() { return sizeof(X) == 2 ? 1 : 3; }

// A workgroup holds the columns of all its tokens over its range of K in
// registers -- each wave a slice of SW steps -- and walks tiles of 16 weight
// rows, blockIdx.x, blockIdx.x + gridDim.x, ...: only codes and scales move
// in the loop, codes straight to the lanes that multiply them, a tile ahead.
// A tile's scales are fetched by the whole workgroup in rows' runs (a lane's
// own would be 2 bytes out of every line) and pass through LDS.
// The waves' sums of a tile meet in LDS, too, behind the tile's one barrier,
// and an extra wave adds and stores them meanwhile.  With more than
// one range of K (gridDim.z) the sums go to `partial` [z][token][n] instead.
// SL: 16-column slabs; grid: (tile walkers, tokens / 16, ranges of K).
//
// With groups (of tokens, each with weights of its own) the grid's y counts the
// groups' tiles of up to as many tokens as the slabs hold.  16 rows over 32
// experts of MXFP4 2048 x 5120: 19.5 us for the weights of some 12 experts (66
// MB) in one wave of workgroups, 3.4 TB/s behind a start of 6 us.
struct OneWeight {};
struct Experts {
  Groups g;
  int64_t code_pitch, code_step, scale_pitch, scale_step;      // bytes from row to row, from expert to expert
  int fill;                                                    // zeros in the rows of no group
};
// Zeros in the rows of y that no group has, by all of the grid's workgroups.
__device__ void zero_other_rows(const Groups &g, void *y, int y_bf16, int64_t ldy, int64_t N, int64_t block,
                                int64_t blocks) {
  const int64_t first = g.at(0), last = max(g.at(g.count), first), rest = first + g.rows - last;
  for (int64_t i = block; i < rest; i += blocks)
    for (int64_t n = threadIdx.x; n < N; n += blockDim.x) store_y(y, y_bf16, (i < first ? i : last + i - first) * ldy + n, 0.0f);
}
// Tokens that the slabs' columns hold.
template <typename X> constexpr int slab_tokens(int slabs) { return sizeof(X) == 2 ? 16 : 16 * slabs / 3; }

template <bool MX, typename X, int SL, int SW, bool HELPER, typename G>
__global__ __launch_bounds__(64 * kTileWaves) void k_matvec_tile(const uint8_t *codes, const uint8_t *scales,
                                                                 const float *meta, int64_t N, int64_t K, const X *x,
                                                                 int64_t tokens, int64_t ldx, void *y, int y_bf16,
                                                                 int64_t ldy, float *partial, int waves, int long_walk,
                                                                 G groups) {
  constexpr bool kGrouped = std::is_same<G, Experts>::value;
  constexpr int kC = columns<X>();
  constexpr int kG = Scale<MX>::kPerByte;
  constexpr int kSB = SW * kStepK / kG;              // scale bytes of a slice's row
  constexpr int kPiece = kSB / 4;                    // of which a thread fetches a quarter
  extern __shared__ __align__(16) char lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, quarter = lane >> 4;
  int64_t t0 = (int64_t)blockIdx.y * kTokens;
  int live = (int)min(tokens - t0, (int64_t)kTokens);
  int64_t code_pitch = K / 2, scale_pitch = K / kG;
  if constexpr (kGrouped) {
    if (groups.fill && !partial)
      zero_other_rows(groups.g, y, y_bf16, ldy, N, blockIdx.y * (int64_t)gridDim.x + blockIdx.x,
                      (int64_t)gridDim.y * gridDim.x);
    constexpr int kMost = slab_tokens<X>(SL);
    const GroupTile tile = find_tile(groups.g, kMost, 1, blockIdx.y);
    if (tile.e < 0) return;
    t0 = tile.begin + (int64_t)tile.local * kMost;
    live = (int)min(tile.end - t0, (int64_t)kMost);
    codes += tile.e * groups.code_step;
    scales += tile.e * groups.scale_step;
    code_pitch = groups.code_pitch;
    scale_pitch = groups.scale_pitch;
  }
  // a range's own k begin at `own`; one that would have only 16 of them (half a
  // lane's load, NVFP4) starts 16 before, and meets zeros there
  const int64_t own = (int64_t)blockIdx.z * waves * (SW * kStepK), kz = MX ? own : min(own, K - 32);
  const int64_t k0 = kz + wave * (SW * kStepK);
  const int64_t tiles = (N + 15) / 16, step = gridDim.x;

  constexpr int kSums = max_waves(SL) * SL * 64;                   // sums of one tile, waves that do not exist counted
  f32x4_t *const part = reinterpret_cast<f32x4_t *>(lds);          // [2][waves][SL][64]
  const float g = MX ? 1.0f : meta[1];
  // adds the waves' sums of a tile, a lane 4 weight rows of a token, and
  // stores them; they are read four waves' at a time (those of waves that do
  // not exist are left out)
  const auto finish = [&](int64_t tile, int turn) {
    if (row >= live) return;
    f32x4_t sum = {0, 0, 0, 0};
#pragma unroll
    for (int p = 0; p < kC; ++p) {
      const int col = row * kC + p;
      const f32x4_t *f = part + (turn & 1) * kSums + (col >> 4) * 64 + quarter * 16 + (col & 15);
      for (int w0 = 0; w0 < waves; w0 += 4) {
        f32x4_t v[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) v[w] = f[(w0 + w) * SL * 64];
#pragma unroll
        for (int w = 0; w < 4; ++w) sum += w0 + w < waves ? v[w] : (f32x4_t){0, 0, 0, 0};
      }
    }
    const int64_t n = 16 * tile + 4 * quarter;
    if (partial) store_rows(partial + ((int64_t)blockIdx.z * tokens + t0 + row) * N, 0, n, N, sum);
    else store_rows(y, y_bf16, (t0 + row) * ldy + n, (t0 + row) * ldy + N, sum * g);
  };
  if (HELPER && wave == waves) {
    // the extra wave only finishes tiles, while the others are at the next one
    __syncthreads();
    __syncthreads();
    int turn = 0;
    for (int64_t t = blockIdx.x; t < tiles; t += step, ++turn) {
      __syncthreads();
      finish(t, turn);
    }
    return;
  }

  // codes of one tile
  uint32_t k[SW];
  int half = 0;                                      // steps (as bits) in which the lane was moved back by 16
#pragma unroll
  for (int s = 0; s < SW; ++s) {
    int64_t at = k0 + s * kStepK + quarter * 32;
    half |= (last_window(at, K) == 16) << s;
    k[s] = (uint32_t)at;
  }
  // through a view of the tile's rows, which is empty past the last tile:
  // what lies outside reads as 0 and moves nothing
  const auto load_codes = [&](u32x4_t *c, int64_t tile) {
    const int64_t n0 = min(tile, tiles - 1) * 16;
    const uint32_t rows = tile < tiles ? (uint32_t)min(N - n0, (int64_t)16) : 0u;
    const __amdgpu_buffer_rsrc_t view =
        make_rsrc(codes + n0 * code_pitch, kGrouped ? rows ? (rows - 1) * (uint32_t)code_pitch + (uint32_t)(K / 2) : 0u
                                                    : rows * (uint32_t)(K / 2));
#pragma unroll
    for (int s = 0; s < SW; ++s)
      c[s] = __builtin_amdgcn_raw_buffer_load_b128(view, (uint32_t)row * (uint32_t)code_pitch + k[s] / 2, 0, 0);
  };
  // scales: piece `sp` of row `sr` of the tile's runs of waves * kSB bytes;
  // a piece that passes the row's end is fetched from before it and shifted
  const int pieces = waves * 4, sr = threadIdx.x / pieces, sp = threadIdx.x % pieces;
  const int64_t row_bytes = K / kG, want = kz / kG + sp * kPiece;
  const int over = (int)min(max(want + kPiece - row_bytes, (int64_t)0), (int64_t)kPiece);
  const uint32_t sfrom = (uint32_t)min(want, row_bytes - kPiece);
  const int shift = 8 * min(over, kPiece - 1);
  const uint64_t keep = over == kPiece ? 0 : ~(uint64_t)0;
  const int stride = waves * kSB + 4;                // + 4: the 16 rows' reads fall on different banks
  const auto load_scales = [&](int64_t tile) {
    const int64_t n0 = tile * 16;
    const uint32_t r = min((uint32_t)sr, (uint32_t)min(N - 1 - n0, (int64_t)15));
    uint64_t v = 0;
    const uint8_t *p = scales + n0 * scale_pitch + (r * (uint32_t)scale_pitch + sfrom);
    __builtin_memcpy(&v, p, kPiece);
    return v;
  };

  // x into registers, by way of LDS: an MFMA's lane wants 8 k of its own
  // column, which as a load would touch 64 places; so runs of k are loaded
  // and turned, a step at a time, in a region of the wave's own.  Piece p (8
  // k) of run i (32 k) of a column lies so that stores (4 pieces of 4 columns
  // or 4 runs) and reads (one piece of 16 columns) fall on all banks.
  bf16x8_t b[SW][4][SL];
  u32x4_t c0[SW], c1[SW];
  const int64_t first = blockIdx.x;
  const auto clamp = [&](int64_t t) { return t < tiles ? t : first; };
  load_codes(c0, first);
  const uint64_t sc_first = load_scales(first);
  uint64_t sc_next = load_scales(clamp(first + step));
  {
    char *const turn = lds + wave * (SL * kTurnBytes);
    const auto mine = [&](int64_t at) { return (uint32_t)(at - own) < (uint32_t)(K - own); };
    const auto slot = [&](int col, int i, int p) {
      return turn + (col >> 4) * kTurnBytes + i * 1024 + 16 * (4 * ((col & 15) ^ i) + (p ^ ((col & 15) >> 2)));
    };
    // a step's columns from LDS (past the last it is repeated: columns are
    // independent); a lane moved back by 16 finds its x in the other half
    const auto take = [&](int s) {
#pragma unroll
      for (int l = 0; l < SL; ++l)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          b[s][j][l] = *reinterpret_cast<const bf16x8_t *>(
              slot(min(16 * l + row, live * kC - 1), quarter, j ^ (((half >> s) & 1) << 1)));
    };
    if constexpr (sizeof(X) == 2) {
      // 64-byte runs, 4 lanes a token
      const int col = lane >> 2, piece = lane & 3;
      const X *xr = x + (t0 + min(col, live - 1)) * ldx;
      u32x4_t raw[SW][4];
#pragma unroll
      for (int s = 0; s < SW; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t at = k0 + s * kStepK + 32 * i + 8 * piece;
          const u32x4_t v = *reinterpret_cast<const u32x4_a2 *>(xr + (mine(at) ? at : 0));
          raw[s][i] = mine(at) ? v : (u32x4_t){0, 0, 0, 0};
        }
#pragma unroll
      for (int s = 0; s < SW; ++s) {
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<u32x4_t *>(slot(col, i, piece)) = raw[s][i];
        take(s);
      }
    } else {
      // a step of a token is 16 lanes' pieces; four tokens a load, the last
      // ones of all steps in one more
      constexpr int kT = 16 * SL / 3, kFull = kT / 4, kLeft = kT % 4;
      static_assert(kLeft == 0 || SW * kLeft == 4, "what is left of the steps fills one load");
      f32x4_t raw[SW * kFull + 1][2];
      const auto fetch = [&](f32x4_t *v, int token, int s) {
        const int64_t at = k0 + s * kStepK + 8 * (lane & 15);
        const X *from = x + (t0 + min(token, live - 1)) * ldx + (mine(at) ? at : 0);
        const f32x4_t v0 = *reinterpret_cast<const f32x4_a4 *>(from);
        const f32x4_t v1 = *reinterpret_cast<const f32x4_a4 *>(from + 4);
        v[0] = mine(at) ? v0 : (f32x4_t){0, 0, 0, 0};
        v[1] = mine(at) ? v1 : (f32x4_t){0, 0, 0, 0};
      };
      const auto put = [&](const Parts &q, int token) {
#pragma unroll
        for (int p = 0; p < 3; ++p)
          if (token < live) *reinterpret_cast<u32x4_t *>(slot(3 * token + p, (lane & 15) >> 2, lane & 3)) = q.v[p];
      };
      const int left_token = 4 * kFull + (kLeft ? quarter % (kLeft ? kLeft : 1) : 0);
      const int left_step = kLeft ? quarter / (kLeft ? kLeft : 1) : 0;
#pragma unroll
      for (int s = 0; s < SW; ++s)
#pragma unroll
        for (int i = 0; i < kFull; ++i) fetch(raw[s * kFull + i], 4 * i + quarter, s);
      Parts left;
      if (kLeft) {
        fetch(raw[SW * kFull], left_token, left_step);
        left = split8(raw[SW * kFull][0], raw[SW * kFull][1]);
      }
#pragma unroll
      for (int s = 0; s < SW; ++s) {
#pragma unroll
        for (int i = 0; i < kFull; ++i)
          put(split8(raw[s * kFull + i][0], raw[s * kFull + i][1]), 4 * i + quarter);
        if (kLeft && left_step == s) put(left, left_token);
        take(s);
      }
    }
  }
  // NVFP4: where a column's values span at most 29 binades they are as exact
  // in f16, moved by a power of two so that the largest lies in [2^14, 2^15)
  // and the smallest at 2^-14 or above (8 bits of f16's 11, no subnormals);
  // the weights decode in half the instructions there.  A wave whose columns
  // do not all allow it (or hold an Inf or NaN) stays with bf16.
  bool f16 = false;
  int move[SL];
#pragma unroll
  for (int l = 0; l < SL; ++l) move[l] = 0;
  if (!MX && long_walk) {
    bool fits = true;
#pragma unroll
    for (int l = 0; l < SL; ++l) {
      ushort2_t hi = {0, 0}, lo = {0xFFFF, 0xFFFF};       // of the magnitudes, and of those less 1 (0 becomes the largest)
#pragma unroll
      for (int s = 0; s < SW; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32x4_t w = __builtin_bit_cast(u32x4_t, b[s][j][l]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const ushort2_t m = __builtin_bit_cast(ushort2_t, (uint32_t)w[i] & 0x7FFF7FFFu);
            hi = __builtin_elementwise_max(hi, m);
            lo = __builtin_elementwise_min(lo, m - (ushort2_t){1, 1});
          }
        }
      int top = max((int)hi[0], (int)hi[1]), low = min((int)lo[0], (int)lo[1]);
      top = max(top, __shfl_xor(top, 16, 64));            // the column's other three lanes
      low = min(low, __shfl_xor(low, 16, 64));
      top = max(top, __shfl_xor(top, 32, 64));
      low = min(low, __shfl_xor(low, 32, 64));
      const int top_e = top >> 7, low_e = max((low + 1) >> 7, 1);
      fits &= top_e < 255 && (top == 0 || low_e >= top_e - 28);
      move[l] = top == 0 ? 0 : top_e - 127 - 14;
    }
    f16 = __all(fits);
    if (f16) {
#pragma unroll
      for (int l = 0; l < SL; ++l)
#pragma unroll
        for (int s = 0; s < SW; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const u32x4_t w = __builtin_bit_cast(u32x4_t, b[s][j][l]);
            half8_t h;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              h[2 * i] = (_Float16)__builtin_amdgcn_ldexpf(bf16_lo(w[i]), -move[l]);
              h[2 * i + 1] = (_Float16)__builtin_amdgcn_ldexpf(bf16_hi(w[i]), -move[l]);
            }
            b[s][j][l] = __builtin_bit_cast(bf16x8_t, h);
          }
    } else {
#pragma unroll
      for (int l = 0; l < SL; ++l) move[l] = 0;
    }
  }
  __syncthreads();

  char *const scale_lds = lds + 2 * kSums * sizeof(f32x4_t);       // [2][16][stride]
  const auto put_scales = [&](uint64_t v, int turn) {
    v = (v >> shift) & keep;
    __builtin_memcpy(scale_lds + (turn & 1) * 16 * stride + sr * stride + sp * kPiece, &v, kPiece);
  };
  put_scales(sc_first, 0);
  __syncthreads();

  int adder = 0;
  const auto work = [&](const u32x4_t *c, int64_t tile, int turn) {
    constexpr int kA = SL == 1 ? 2 : 1;       // one slab: two accumulators, so that MFMAs do not wait for each other
    f32x4_t acc[kA][SL];
#pragma unroll
    for (int l = 0; l < SL; ++l) acc[0][l] = acc[kA - 1][l] = (f32x4_t){0, 0, 0, 0};
    Scale<MX> sc[SW];
    const char *at = scale_lds + (turn & 1) * 16 * stride + row * stride;
#pragma unroll
    for (int s = 0; s < SW; ++s) {
      const uint32_t o = (k[s] - (uint32_t)kz) / kG;
      // NVFP4: the pair of a lane moved back starts at an odd byte; its
      // first scale meets only zeros, so the second's pair will do
      if (MX) sc[s].raw = *reinterpret_cast<const uint8_t *>(at + o);
      else sc[s].raw = (uint32_t)*reinterpret_cast<const uint16_t *>(at + ((o + 1) & ~1u)) << (((half >> s) & 1) * 8);
    }
    // MXFP4: weights of the scales from 2^126 on may pass bf16's range; where a
    // wave holds one, its tile is decoded at a quarter
    bool far = false;
    if constexpr (MX) {
      uint32_t top = sc[0].raw;
#pragma unroll
      for (int s = 1; s < SW; ++s) top = max(top, sc[s].raw);
      far = __any(top >= Scale<MX>::kFar);
    }
    if (!MX && f16) {
#pragma unroll
      for (int s = 0; s < SW; ++s) {
        const _Float16 lo = (_Float16)sc[s].lo(), hi = (_Float16)sc[s].hi();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const half8_t a = decode8_f16(c[s][j], j < 2 ? (half2_t){lo, lo} : (half2_t){hi, hi});
#pragma unroll
          for (int l = 0; l < SL; ++l)
            acc[j % kA][l] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, __builtin_bit_cast(half8_t, b[s][j][l]),
                                                                    acc[j % kA][l], 0, 0, 0);
        }
      }
    } else if (far) {
      if constexpr (MX) {
#pragma unroll
        for (int s = 0; s < SW; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bf16x8_t a = decode8<false>(c[s][j], sc[s].quarter());
#pragma unroll
            for (int l = 0; l < SL; ++l)
              acc[j % kA][l] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[s][j][l], acc[j % kA][l], 0, 0, 0);
          }
      }
    } else {
#pragma unroll
      for (int s = 0; s < SW; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bf16x8_t a = decode8<MX>(c[s][j], j < 2 ? sc[s].lo() : sc[s].hi());
#pragma unroll
          for (int l = 0; l < SL; ++l)
            acc[j % kA][l] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[s][j][l], acc[j % kA][l], 0, 0, 0);
        }
    }
    f32x4_t *const mine = part + (turn & 1) * kSums;
#pragma unroll
    for (int l = 0; l < SL; ++l) {
      f32x4_t v = kA == 2 ? acc[0][l] + acc[kA - 1][l] : acc[0][l];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __builtin_amdgcn_ldexpf(v[i], MX ? 2 * far : move[l]);
      mine[(wave * SL + l) * 64 + lane] = v;
    }
    put_scales(sc_next, turn + 1);
    __syncthreads();
    if (!HELPER) {
      if (wave == adder) finish(tile, turn);
      adder = adder + 1 < waves ? adder + 1 : 0;
    }
  };

  // one turn: the loads of a later tile, then this tile
  int turn = 0;
  const auto round = [&](const u32x4_t *now, u32x4_t *next, int64_t t) {
    load_codes(next, t + step);
    const uint64_t sc_later = load_scales(clamp(t + 2 * step));
    __builtin_amdgcn_sched_barrier(0);       // the loads go out before this tile's work, not after it
    work(now, t, turn++);
    sc_next = sc_later;
    return t + step < tiles;
  };
  for (int64_t t = first;; t += 2 * step) {
    if (!round(c0, c1, t)) break;
    if (!round(c1, c0, t + step)) break;
  }
}

// y = g times the sum of the ranges' partial sums, in their order.
__global__ __launch_bounds__(256) void k_matvec_join(const float *partial, int ranges, const float *meta, int64_t N,
                                                     int64_t tokens, void *y, int y_bf16, int64_t ldy) {
  const float g = meta ? meta[1] : 1.0f;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < N * tokens; i += (int64_t)gridDim.x * 256) {
    float sum = 0.0f;
    for (int z = 0; z < ranges; ++z) sum += partial[z * tokens * N + i];
    store_y(y, y_bf16, i / N * ldy + i % N, sum * g);
  }
}

// The same for the rows of groups; those of none become zeros or stay.
__global__ __launch_bounds__(256) void k_grouped_join(const float *partial, int ranges, const float *meta, int64_t N,
                                                      int64_t tokens, void *y, int y_bf16, int64_t ldy, Experts groups) {
  const float g = meta ? meta[1] : 1.0f;
  const int64_t first = groups.g.at(0), last = groups.g.at(groups.g.count);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < N * tokens; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / N;
    const bool own = t >= first && t < last;
    if (!own && !groups.fill) continue;
    float sum = 0.0f;
    if (own)
      for (int z = 0; z < ranges; ++z) sum += partial[z * tokens * N + i];
    store_y(y, y_bf16, t * ldy + i % N, own ? sum * g : 0.0f);
  }
}

// K below 128, where a row has less than a step's codes: one thread an output.
constexpr int64_t kShortK = 128;
template <bool MX, typename X>
__global__ __launch_bounds__(256) void k_matvec_short(const uint8_t *codes, const uint8_t *scales, const float *meta,
                                                      int64_t N, int64_t K, const X *x, int64_t tokens, int64_t ldx,
                                                      void *y, int y_bf16, int64_t ldy) {
  constexpr int kG = Scale<MX>::kPerByte;
  const float g = MX ? 1.0f : meta[1];
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < N * tokens; i += (int64_t)gridDim.x * 256) {
    const int64_t n = i % N, t = i / N;
    float sum = 0.0f;
    for (int k0 = 0; k0 < K; k0 += 16) {
      const u32x2_t c = *reinterpret_cast<const u32x2_t *>(codes + n * (K / 2) + k0 / 2);
      Scale<MX> sc;
      sc.raw = scales[n * (K / kG) + k0 / kG];
      float p = 0.0f;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float2_t q = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4((c[k >> 3] >> (4 * (k & 7))) & 15u, 1.0f, 0);
        p = __builtin_fmaf(to_float(x[t * ldx + k0 + k]), q.x, p);
      }
      sum = __builtin_fmaf(p, sc.lo(), sum);
    }
    store_y(y, y_bf16, t * ldy + n, K > 0 ? sum * g : 0.0f);      // (g of no weights may be anything)
  }
}
constexpr int64_t kFlatGrid = 1 << 16;

// ----------------------------------------------------- up to 4 tokens --

// A lane's products with 32 weights of one row: sum x q s.
template <bool MX> __device__ __forceinline__ float dot32(const u32x4_t &c, const Scale<MX> &s, const Act<uint16_t> &x) {
  float p[2] = {0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bf16x8_t q = decode8<true>(c[j], 1.0f);
    const u32x4_t qw = __builtin_bit_cast(u32x4_t, q);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[j >> 1] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, (uint32_t)qw[i]),
                                                  __builtin_bit_cast(bf16x2_t, (uint32_t)x.v[j][i]), p[j >> 1], false);
  }
  return MX ? (p[0] + p[1]) * s.lo() : __builtin_fmaf(p[0], s.lo(), p[1] * s.hi());
}
template <bool MX> __device__ __forceinline__ float dot32(const u32x4_t &c, const Scale<MX> &s, const Act<float> &x) {
  float p[2] = {0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2_t q[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[j], 1.0f, 0),
                           __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[j], 1.0f, 1),
                           __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[j], 1.0f, 2),
                           __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[j], 1.0f, 3)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32x4_t &v = x.v[2 * j + (i >> 1)];
      p[j >> 1] = __builtin_fmaf(q[i].x, __uint_as_float(v[2 * (i & 1)]), p[j >> 1]);
      p[j >> 1] = __builtin_fmaf(q[i].y, __uint_as_float(v[2 * (i & 1) + 1]), p[j >> 1]);
    }
  }
  return MX ? (p[0] + p[1]) * s.lo() : __builtin_fmaf(p[0], s.lo(), p[1] * s.hi());
}

constexpr int kWaveK = 64 * 32;         // k of one wave load

// C sums over the wave at once.  A swap of halves (then of odd and even rows
// of 16 lanes) between two values and one addition fold both of them into
// one register, each in its own lanes; what is left takes four additions
// with rotated lanes.  On return value i is v[i % slots] in the lanes of row
// (of 16) i / slots, for C >= 4; for C = 2 in the rows 0-1 and 2-3, for C = 1
// in all.
template <int C> constexpr int sum_slots() { return C >= 4 ? C / 4 : 1; }
template <int C> __device__ __forceinline__ int sum_row(int i) { return C >= 4 ? i / (C / 4) : 2 * i; }
template <int C> __device__ __forceinline__ void wave_sums(float *v) {
  static_assert(C == 1 || C == 2 || C % 4 == 0, "sums come in fours");
  constexpr int kHalf = C > 1 ? C / 2 : 1, kSlots = sum_slots<C>();
  // the pair of a register: another value, or itself where one is left
#pragma unroll
  for (int i = 0; i < kHalf; ++i) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_int(v[i]), __float_as_int(v[C > 1 ? i + kHalf : i]),
                                                    false, false);
    v[i] = __int_as_float(p[0]) + __int_as_float(p[1]);
  }
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_int(v[i]), __float_as_int(v[C >= 4 ? i + kSlots : i]),
                                                    false, false);
    v[i] = __int_as_float(p[0]) + __int_as_float(p[1]);
    v[i] += dpp<0xB1>(v[i]);
    v[i] += dpp<0x4E>(v[i]);
    v[i] += dpp<0x141>(v[i]);
    v[i] += dpp<0x140>(v[i]);
  }
}

// R weight rows' share of a wave: J loads each.
template <bool MX, int J, int R> struct RowPart {
  u32x4_t c[R][J];
  Scale<MX> s[R][J];
  __device__ __forceinline__ void load(const uint8_t *codes, const uint8_t *scales, int64_t n, int64_t N, int64_t K,
                                       const uint32_t *k) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = min(n + r, N - 1);          // past the end: the last one again, not stored
      const uint8_t *cr = codes + row * (K / 2), *sr = scales + row * (K / Scale<MX>::kPerByte);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        // read once (one token, 131075 x 5120: 66.2 -> 58.8 us, 20480 x 5120
        // 13.9 -> 13.3, the same where the weights stay in the last cache;
        // the tiles' loads of half a line lose by it: 72 -> 85)
        c[r][j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_a8 *>(cr + k[j] / 2));
        s[r][j].load(sr + k[j] / Scale<MX>::kPerByte);
      }
    }
  }
};

// The workgroup's waves hold J loads of each token's x: WK waves share a row
// (K <= WK * J * 2048), the others work on rows of their own, R at a time
// (so that every wave has some 3 KB in flight, twice).
constexpr int row_waves(int wk) { return wk == 3 ? 3 : 4; }
template <bool MX, typename X, int J, int WK, int R, int T>
__global__ __launch_bounds__(64 * row_waves(WK), T <= 2 ? 3 : 2) void
k_matvec_row(const uint8_t *codes, const uint8_t *scales, const float *meta, int64_t N, int64_t K, const X *x, int64_t ldx,
             void *y, int y_bf16, int64_t ldy) {
  constexpr int kWaves = row_waves(WK), kThreads = 64 * kWaves, kRows = kWaves / WK * R, kC = R * T;
  // x through LDS: a lane's 32 k would be a load of 64 lines of memory.  Each
  // of J T rounds takes the waves' j-th loads of one token; unit u (16 bytes)
  // lies at slot u with its lowest bits turned by the next ones, so that 16
  // lanes' reads of one piece each fall on all banks.
  constexpr int kUnit = 16 / sizeof(X), kPieces = Act<X>::kPieces;
  constexpr int kWaveUnits = kWaveK / kUnit, kLoads = WK * kWaveUnits / kThreads;
  __shared__ u32x4_t turned[WK * kWaveUnits];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kw = wave % WK;
  const auto slot = [](uint32_t u) { return u ^ ((u >> 4) & (kPieces - 1)); };
  u32x4_t raw[T][J][kLoads];
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int u = threadIdx.x + i * kThreads;
        const int64_t at = (int64_t)(u / kWaveUnits * J + j) * kWaveK + u % kWaveUnits * kUnit;
        const u32x4_t v = *reinterpret_cast<const u32x4_a2 *>(x + t * ldx + (at < K ? at : 0));
        raw[t][j][i] = at < K ? v : (u32x4_t){0, 0, 0, 0};
      }
  const float g = MX ? 1.0f : meta[1];
  const int64_t stride = (int64_t)gridDim.x * kRows;
  const int64_t mine = wave / WK * R, first = (int64_t)blockIdx.x * kRows + mine;
  __shared__ float share[2][kWaves][kC];
  uint32_t k[J];
  int half = 0;                                      // loads (as bits) that were moved back by 16
#pragma unroll
  for (int j = 0; j < J; ++j) {
    int64_t at = (int64_t)((kw * J + j) * 64 + lane) * 32;
    half |= (last_window(at, K) == 16) << j;
    k[j] = (uint32_t)at;
  }
  Act<X> xv[T][J];
  RowPart<MX, J, R> a, b;
  const auto finish = [&](const RowPart<MX, J, R> &p, int64_t n, int turn) {
    // sum i = (row i / T of the R, token i % T)
    float v[kC];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < T; ++t) {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < J; ++j) sum += dot32<MX>(p.c[r][j], p.s[r][j], xv[t][j]);
        v[r * T + t] = sum;
      }
    wave_sums<kC>(v);
    const auto store = [&](int i, float sum) {
      if (n + i / T < N) store_y(y, y_bf16, i % T * ldy + n + i / T, sum * g);
    };
    if (WK == 1) {
#pragma unroll
      for (int i = 0; i < kC; ++i)
        if (lane == 16 * sum_row<kC>(i)) store(i, v[i % sum_slots<kC>()]);
      return;
    }
#pragma unroll
    for (int i = 0; i < kC; ++i)
      if (lane == 16 * sum_row<kC>(i)) share[turn][wave][i] = v[i % sum_slots<kC>()];
    __syncthreads();
    if (kw == 0 && lane < kC) {
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < WK; ++w) sum += share[turn][wave + w][lane];
      store(lane, sum);
    }
  };
  a.load(codes, scales, first, N, K, k);
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (t + j) __syncthreads();
#pragma unroll
      for (int i = 0; i < kLoads; ++i) turned[slot(threadIdx.x + i * kThreads)] = raw[t][j][i];
      __syncthreads();
      // (moved back by 16: its x are the load's first half, zeros before them)
      const int swap = ((half >> j) & 1) * (kPieces / 2);
#pragma unroll
      for (int p = 0; p < kPieces; ++p) xv[t][j].v[p] = turned[slot(kw * kWaveUnits + lane * kPieces + (p ^ swap))];
    }
  // the workgroup's waves make the same number of turns (barriers)
  for (int64_t n = first; n - mine < N; n += 2 * stride) {
    b.load(codes, scales, n + stride, N, K, k);
    finish(a, n, 0);
    a.load(codes, scales, n + 2 * stride, N, K, k);
    finish(b, n + stride, 1);
  }
}

// ------------------------------------------------------------- launches --

// How a product of more than one token is cut: SL slabs of 16 columns, SW
// steps a wave (16 SL SW registers of x), `waves` of them a workgroup,
// `ranges` of K, and the workgroups that walk the tiles of one range.
struct Cut {
  int sl, sw, waves, ranges, walkers, long_walk;
};
Cut cut_of(int64_t N, int64_t K, int cols, int64_t blocks) {
  Cut c;
  c.sl = (cols + 15) / 16;
  c.sw = c.sl == 1 ? 4 : 2;
  const int64_t slices = (K + c.sw * kStepK - 1) / (c.sw * kStepK);
  const int most = max_waves(c.sl);
  c.ranges = (int)((slices + most - 1) / most);
  c.waves = (int)((slices + c.ranges - 1) / c.ranges);       // (the last range has a slice at least: waves <= most)
  // one round of workgroups: as many as fit the CUs' waves, the tiles dealt evenly
  const int64_t tiles = (N + 15) / 16;
  const int64_t room = (int64_t)device_cus() * (kTileWaves / (c.waves + has_helper(c.waves, c.sl)));
  const int64_t want = std::min(tiles, std::max<int64_t>(1, room / (c.ranges * blocks)));
  const int64_t per = (tiles + want - 1) / want;
  c.walkers = (int)((tiles + per - 1) / per);
  // bringing x to f16 pays from about 8 tiles on (1.3 us more at the start, a
  // fifth less a tile: 131075 x 5120 90 -> 77 us, 20480 x 5120 18.4 -> 19.7)
  c.long_walk = per >= 8;
  return c;
}
Cut cut_for(int64_t N, int64_t K, int64_t tokens, bool f32) {
  return cut_of(N, K, (int)std::min<int64_t>(tokens, kTokens) * (f32 ? 3 : 1), (tokens + kTokens - 1) / kTokens);
}

// What every launch of a product passes on.
template <typename X> struct Product {
  const uint8_t *codes, *scales;
  const float *meta;
  int64_t N, K;
  const X *x;
  int64_t tokens, ldx;
  void *y;
  int y_bf16;
  int64_t ldy;
  void *ws;
  hipStream_t stream;
};

template <bool MX, int SL, int SW, typename X, typename G>
void tile(const Cut &c, const Product<X> &p, int64_t blocks, const G &groups) {
  const dim3 grid((unsigned)c.walkers, (unsigned)blocks, (unsigned)c.ranges);
  const size_t run = c.waves * SW * kStepK / Scale<MX>::kPerByte;       // scale bytes of a row
  const size_t lds =
      std::max<size_t>(c.waves * SL * kTurnBytes, 2 * max_waves(SL) * SL * 64 * sizeof(f32x4_t) + 32 * (run + 4));
  float *partial = c.ranges > 1 ? (float *)p.ws : nullptr;
  const auto launch = [&](auto kernel, int waves) {
    kernel<<<grid, 64 * waves, lds, p.stream>>>(p.codes, p.scales, p.meta, p.N, p.K, p.x, p.tokens, p.ldx, p.y, p.y_bf16,
                                                p.ldy, partial, c.waves, c.long_walk, groups);
  };
  if (has_helper(c.waves, SL)) launch(k_matvec_tile<MX, X, SL, SW, true, G>, c.waves + 1);
  else if constexpr (SL == 1) launch(k_matvec_tile<MX, X, SL, SW, false, G>, c.waves);
  if constexpr (std::is_same<G, Experts>::value) {
    if (partial)
      k_grouped_join<<<(unsigned)std::min(kFlatGrid, (p.N * p.tokens + 255) / 256), 256, 0, p.stream>>>(
          partial, c.ranges, MX ? nullptr : p.meta, p.N, p.tokens, p.y, p.y_bf16, p.ldy, groups);
    return;
  }
  if (partial)
    k_matvec_join<<<(unsigned)std::min(kFlatGrid, (p.N * p.tokens + 255) / 256), 256, 0, p.stream>>>(
        partial, c.ranges, MX ? nullptr : p.meta, p.N, p.tokens, p.y, p.y_bf16, p.ldy);
}

template <bool MX, int J, int WK, int R, int T, typename X> void rows(const Product<X> &p) {
  // 12 waves a CU (one token, 20480 x 5120: 13.5 us, with 16 waves 14.7, 32
  // 16.1), the rows dealt evenly
  constexpr int kWaves = row_waves(WK);
  const int64_t per = kWaves / WK * R, turns = (p.N + per - 1) / per, slots = (int64_t)device_cus() * (12 / kWaves);
  const int64_t each = (turns + slots - 1) / slots;
  const unsigned grid = (unsigned)((turns + each - 1) / each);
  k_matvec_row<MX, X, J, WK, R, T><<<grid, 64 * kWaves, 0, p.stream>>>(p.codes, p.scales, p.meta, p.N, p.K, p.x, p.ldx,
                                                                      p.y, p.y_bf16, p.ldy);
}

// Products for k_matvec_row: tokens whose x fits the registers of a workgroup
// (one up to K = 24576, two in bf16 up to 16384, four up to 8192), of which
// more than one only up to 2e8 products (four in f32 1e8): each costs an
// instruction there, while the tiles' cost does not grow with the tokens.
// us, rows / tiles, for 2, 3, 4 tokens of NVFP4 in bf16: 5120 x 5120 7.9 8.9
// 10.3 / 10.3, 20480 x 2048 8.6 9.3 11.9 / 12.9, 10000 x 8192 13.9 16.0 18.4
// / 17.8, 20480 x 5120 18.6 22.6 27.1 / 17.4; in f32 5120 x 2048 6.3 7.3 8.9
// / 10.5, 5120 x 5120 9.3 11.2 15.3 / 12.5, 20480 x 5120 23.6 30.0 41.2 / 19.5.
// The limits lie between these sizes, one for 2 and 3 tokens of both types, and
// are not the break-evens themselves: 3 bf16 tokens of 10000 x 8192 go by tiles
// (17.8 against 16.0), and 2 or 3 f32 tokens go by rows up to 1e8 and 6.7e7
// weights where by the lines between the f32 figures tiles lead from some 6e7 and 3.5e7 on.
bool by_rows(int64_t N, int64_t K, int64_t tokens, bool f32) {
  if (K < kShortK) return false;
  if (tokens == 1) return K <= 12 * kWaveK;
  if (tokens > 4 || K > (tokens == 2 && !f32 ? 8 : 4) * kWaveK) return false;
  return N * K <= (f32 && tokens == 4 ? 100000000 : 200000000) / tokens;
}

template <bool MX, int T, typename X> void rows_of(const Product<X> &p) {
  const int64_t loads = (p.K + kWaveK - 1) / kWaveK;
  if constexpr (T == 1) {
    if (loads <= 1) rows<MX, 1, 1, 4, T>(p);
    else if (loads <= 2) rows<MX, 2, 1, 2, T>(p);
    else if (loads <= 3) rows<MX, 3, 1, 1, T>(p);
    else if (loads <= 4) rows<MX, 1, 4, 4, T>(p);
    else if (loads <= 8) rows<MX, 2, 4, 2, T>(p);
    else rows<MX, 3, 4, 1, T>(p);
  } else {
    if (loads <= 1) rows<MX, 1, 1, 4, T>(p);
    else if (loads <= 2) rows<MX, 1, 2, 4, T>(p);
    else if (loads <= 3) rows<MX, 1, 3, 4, T>(p);
    else if (loads <= 4) rows<MX, 1, 4, 4, T>(p);
    else if constexpr (T == 2 && sizeof(X) == 2) rows<MX, 2, 4, 2, T>(p);
  }
}

template <bool MX, typename X> void matvec(const Product<X> &p) {
  if (by_rows(p.N, p.K, p.tokens, sizeof(X) == 4)) {
    if (p.tokens == 1) rows_of<MX, 1>(p);
    else if (p.tokens == 2) rows_of<MX, 2>(p);
    else if (p.tokens == 3) rows_of<MX, 3>(p);
    else rows_of<MX, 4>(p);
  } else if (p.K < kShortK) {
    const unsigned grid = (unsigned)std::min(kFlatGrid, (p.N * p.tokens + 255) / 256);
    k_matvec_short<MX, X><<<grid, 256, 0, p.stream>>>(p.codes, p.scales, p.meta, p.N, p.K, p.x, p.tokens, p.ldx, p.y,
                                                     p.y_bf16, p.ldy);
  } else {
    const Cut c = cut_for(p.N, p.K, p.tokens, sizeof(X) == 4);
    const int64_t blocks = (p.tokens + kTokens - 1) / kTokens;
    if (c.sl == 1) tile<MX, 1, 4>(c, p, blocks, OneWeight());
    else if constexpr (sizeof(X) == 4)
      c.sl == 2 ? tile<MX, 2, 2>(c, p, blocks, OneWeight()) : tile<MX, 3, 2>(c, p, blocks, OneWeight());
  }
}

// Groups of few rows: the tiles of 16 weight rows, one walk over an expert's
// for up to as many tokens as the slabs hold (float32: 5, 10 or 16, by the
// groups' average).
struct GroupedCut {
  Cut cut;
  int64_t blocks;
};
GroupedCut grouped_cut(int64_t experts, int64_t N, int64_t K, int64_t rows, bool f32) {
  const int64_t groups = std::min(experts, rows), each = (rows + groups - 1) / groups;
  const int most = !f32 ? 16 : each <= 3 ? 5 : each <= 8 ? 10 : 16;
  GroupedCut c;
  c.blocks = rows / (f32 ? 16 * ((3 * most + 15) / 16) / 3 : 16) + groups;
  c.cut = cut_of(N, K, f32 ? 3 * most : 16, c.blocks);
  return c;
}

}  // namespace

// Whether the tiles can take a grouped product (a row holds a step's codes, the
// grid's y the groups' tiles).
bool grouped_tiles_fit(int64_t experts, int64_t K, int64_t rows) {
  return K >= kShortK && rows / 5 + std::min(experts, rows) <= 65535;
}
int64_t grouped_tiles_workspace_bytes(int64_t experts, int64_t N, int64_t K, int64_t rows, bool f32) {
  const GroupedCut c = grouped_cut(experts, N, K, rows, f32);
  return c.cut.ranges > 1 ? 4 * c.cut.ranges * rows * N : 0;
}
hipError_t launch_grouped_tiles(const GroupedProduct &g, int64_t code_pitch, int64_t code_step, int64_t scale_pitch,
                                int64_t scale_step, hipStream_t stream) {
  const Experts experts = {{g.offsets, g.index_bits == 64, (int)g.experts, g.rows, 0}, code_pitch, code_step,
                           scale_pitch, scale_step, g.fill};
  const GroupedCut c = grouped_cut(g.experts, g.n, g.k, g.rows, g.x_dtype == 0);
  const auto run = [&](auto *xt, auto mx) {
    using X = std::remove_const_t<std::remove_pointer_t<decltype(xt)>>;
    constexpr bool MX = decltype(mx)::value;
    const Product<X> p = {g.codes, g.scales, g.meta, g.n, g.k, xt, g.rows, g.ldx, g.y, g.y_dtype == 1, g.ldy, g.ws, stream};
    if constexpr (sizeof(X) == 2) {
      tile<MX, 1, 4>(c.cut, p, c.blocks, experts);
    } else {
      if (c.cut.sl == 1) tile<MX, 1, 4>(c.cut, p, c.blocks, experts);
      else if (c.cut.sl == 2) tile<MX, 2, 2>(c.cut, p, c.blocks, experts);
      else tile<MX, 3, 2>(c.cut, p, c.blocks, experts);
    }
  };
  with_flag(g.mx, [&](auto mx) {
    if (g.x_dtype == 1) run((const uint16_t *)g.x, mx);
    else run((const float *)g.x, mx);
  });
  return hipGetLastError();
}

int64_t matvec_workspace_bytes(int64_t N, int64_t K, int64_t tokens, bool f32) {
  if (N <= 0 || tokens <= 0 || K < kShortK || by_rows(N, K, tokens, f32)) return 0;
  const Cut c = cut_for(N, K, tokens, f32);
  return c.ranges > 1 ? 4 * c.ranges * tokens * N : 0;
}

hipError_t launch_matvec(bool mx, const uint8_t *codes, const uint8_t *scales, const float *meta, int64_t N, int64_t K,
                         const void *x, int x_dtype, int64_t tokens, int64_t ldx, void *y, int y_dtype, int64_t ldy,
                         void *ws, hipStream_t stream) {
  if (N > 0 && tokens > 0) {
    const auto run = [&](auto *xt) {
      using X = std::remove_const_t<std::remove_pointer_t<decltype(xt)>>;
      const Product<X> p = {codes, scales, meta, N, K, xt, tokens, ldx, y, y_dtype == 1, ldy, ws, stream};
      if (mx) matvec<true>(p);
      else matvec<false>(p);
    };
    if (x_dtype == 1) run((const uint16_t *)x);
    else run((const float *)x);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
