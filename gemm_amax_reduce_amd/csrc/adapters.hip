// adapters.hip -- low-rank adapters of many requests at once, beside a shared
// projection, for gfx950: rows come in segments (requests), each with an
// adapter (A [r][K], B [N][r], scale s) or none,
//
//   u = A x,  y = base + s B u
//
// and the backward pass,
//
//   g = s B^T dy,  dx = base + A^T g,  dA = sum g x^T,  dB = sum s dy u^T.
//
// The rank is small, so each product reads its wide matrix once and is bound
// by that: x and dy into r numbers a row (k_shrink), r numbers a row into base
// and y (k_expand), and both matrices into sums over rows (k_grad).  u and g
// are float32; every product runs on the bf16 MFMA with float32 operands as
// three bf16 parts each (about what binary32 products keep).
#include "gemm_common.h"
#include "groups.h"
#include "nvfp4_kernels.h"
#include "operands.h"

#include <algorithm>
#include <type_traits>

namespace nvfp4 {

namespace {

// The adapter of a segment: index[e], -1 where it names none.
struct Segments {
  Groups g;                // with the rows of no segment as the first and the last group
  const void *index;
  int adapters;
  __device__ __forceinline__ int adapter(int e) const {
    if (e < 1 || e >= g.count - 1) return -1;
    const int64_t v = g.is64 ? ((const int64_t *)index)[e - 1] : (int64_t)((const int32_t *)index)[e - 1];
    return v >= 0 && v < adapters ? (int)v : -1;
  }
};
// The first segment from e on with that adapter and rows of its own; count - 1
// if there is none.
__device__ __forceinline__ int next_of(const Segments &s, int adapter, int e) {
  const int lane = threadIdx.x & 63;
  for (; e < s.g.count - 1; e += 64) {
    const int mine = e + lane;
    bool hit = mine < s.g.count - 1 && s.adapter(mine) == adapter;
    if (hit) hit = s.g.size(mine) > 0;
    const uint64_t found = __ballot(hit);
    if (found) return __builtin_amdgcn_readfirstlane(e + (int)__builtin_ctzll(found));
  }
  return s.g.count - 1;
}

// --------------------------------------------------------------- shrink --

// out[t][j] = scale sum_c x[t][c] w[a][j][c] for a tile of 16 MT rows, zeros
// for those without an adapter.  The weights are the A operand of the 16x16x32
// MFMA, so that a lane has 4 neighbouring ranks of a row; 4 lanes hold 64 bytes
// of a row in one piece.  The workgroup's waves take 128 c each in turn, and
// their sums meet in LDS.  Bound by reading x, in pieces of 64 bytes, and by the
// two to three rounds of loads that a wave makes: 8192 rows of 5120 bf16, rank 16,
// 34 us (2.5 TB/s), 24 rows of as many adapters 9.4 us.  Twice the columns a wave
// and round, 20 us a call for the 24 rows instead of 19, and 200 instead of 193
// for the backward pass of 8192.
constexpr int kChunk = 128;
template <typename X, typename W, int RF, int MT>
__global__ __launch_bounds__(RF * MT > 4 ? 512 : 1024) void k_shrink(Segments s, const X *x, int64_t ldx, int64_t C, const W *w,
                                                                int rank, const float *scale, float *out, int waves) {
  extern __shared__ __align__(16) float sums[];        // [waves][16 MT][16 RF]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, quarter = lane >> 4;
  const GroupTile t = find_tile(s.g, 16 * MT, 1, blockIdx.x);
  if (t.e < 0) return;
  const int64_t t0 = t.begin + 16 * MT * (int64_t)t.local;
  const int live = (int)min(t.end - t0, (int64_t)(16 * MT));
  const int a = s.adapter(t.e);
  if (a < 0) {
    for (int i = threadIdx.x; i < live * rank; i += 64 * waves) out[t0 * rank + i] = 0.0f;
    return;
  }
  const X *xr[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) xr[m] = x + (t0 + min(16 * m + row, live - 1)) * ldx;
  const W *wr[RF];
#pragma unroll
  for (int f = 0; f < RF; ++f) wr[f] = w + ((int64_t)a * rank + min(16 * f + row, rank - 1)) * C;
  f32x4_t acc[MT][RF];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int f = 0; f < RF; ++f) acc[m][f] = (f32x4_t){0, 0, 0, 0};
  // (as many loads as the registers hold go out together)
  constexpr int kTogether = (MT * sizeof(X) + RF * sizeof(W)) > 16 ? (MT * sizeof(X) + RF * sizeof(W)) > 32 ? 1 : 2 : 4;
  const auto step = [&](int64_t c0, auto whole) {
#pragma unroll
    for (int i0 = 0; i0 < 4; i0 += kTogether) {
      Row8<X> xq[kTogether][MT];
      Row8<W> wq[kTogether][RF];
#pragma unroll
      for (int i = 0; i < kTogether; ++i) {
        const int64_t c = c0 + 32 * (i0 + i) + 8 * quarter;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if (whole.value) xq[i][m].load(xr[m] + c);
          else load_row8(xq[i][m], xr[m], c, C);
        }
#pragma unroll
        for (int f = 0; f < RF; ++f) {
          if (whole.value) wq[i][f].load(wr[f] + c);
          else load_row8(wq[i][f], wr[f], c, C);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < kTogether; ++i) {
        Operand<X> xo[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) xo[m].set(xq[i][m]);
#pragma unroll
        for (int f = 0; f < RF; ++f) {
          Operand<W> wo;
          wo.set(wq[i][f]);
#pragma unroll
          for (int m = 0; m < MT; ++m) multiply16(acc[m][f], wo, xo[m]);
        }
      }
    }
  };
  int64_t c0 = (int64_t)wave * kChunk;
  for (; c0 + kChunk <= C; c0 += (int64_t)waves * kChunk) step(c0, std::true_type());
  if (c0 < C) step(c0, std::false_type());
  constexpr int kPitch = 16 * RF;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int f = 0; f < RF; ++f)
      *reinterpret_cast<f32x4_t *>(sums + (wave * 16 * MT + 16 * m + row) * kPitch + 16 * f + 4 * quarter) = acc[m][f];
  __syncthreads();
  const float factor = scale ? scale[a] : 1.0f;
  for (int i = threadIdx.x; i < live * rank; i += 64 * waves) {
    const int at = i / rank * kPitch + i % rank;
    float v = 0.0f;
    for (int k = 0; k < waves; ++k) v += sums[k * 16 * MT * kPitch + at];
    out[t0 * rank + i] = v * factor;
  }
}

// --------------------------------------------------------------- expand --

// y[t][c] = base[t][c] + scale sum_j u[t][j] w[a][c][j] for 16 MT rows and
// `spans` times 256 columns, 64 of them a wave.  The weights are the A operand with its rows
// ordered so that a lane's results are two runs of 8 columns of a row, and 4
// lanes hold 64 bytes of it (bf16) in one piece.
//
// Loads are whole and unconditional wherever the columns (the ranks) allow it,
// by a choice that the wave makes as one: what a branch leaves zero in some lanes
// would wait for the loads of the others.
//
// Bound by HBM: 4099 rows of 20480 columns, bf16 base and result, rank 32: 97 us
// (336 MB, 3.5 TB/s); 8192 x 5120 48 us.  160 registers leave three waves a SIMD;
// four (and spilled registers) took 209 us instead of 133 for the whole call, which
// takes 125 to 133 from card to card.
template <typename T>
__device__ __forceinline__ void load_ranks(Row8<T> &q, const T *row, int at, int rank, bool eights) {
  if (eights) {
    q.load(row + (at < rank ? at : 0));
  } else {
    load_row8(q, row, at, rank);
  }
}
template <typename T> __device__ __forceinline__ void zero_unless(Row8<T> &q, bool keep) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) q.r[i] = keep ? q.r[i] : 0u;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q.a[i] = keep ? q.a[i] : 0.0f;
      q.b[i] = keep ? q.b[i] : 0.0f;
    }
  }
}

// BASE: 0 none, 1 f32, 2 bf16.
template <typename W, int MT, int BASE>
__global__ __launch_bounds__(256) void k_expand(Segments s, const float *u, int rank, const W *w, const float *scale,
                                                const void *base, int64_t ldb, void *y, int y_bf16, int64_t ldy, int64_t C,
                                                int tiles_c, int spans) {
  using B = std::conditional_t<BASE == 2, uint16_t, float>;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, quarter = lane >> 4;
  const GroupTile t = find_tile(s.g, 16 * MT, tiles_c, blockIdx.x);
  if (t.e < 0) return;
  const int64_t t0 = t.begin + 16 * MT * (int64_t)(t.local / tiles_c);
  const int live = (int)min(t.end - t0, (int64_t)(16 * MT));
  const int a = __builtin_amdgcn_readfirstlane(s.adapter(t.e));
  if (a < 0 && base == y) return;
  const float factor = a >= 0 && scale ? scale[a] : 1.0f;
  const bool eights = rank % 8 == 0;
  int64_t c0 = (int64_t)(t.local % tiles_c) * spans * 256 + 64 * wave;
  const int64_t end = min(C, c0 + spans * 256);
  for (; c0 < end; c0 += 256) {
    const int64_t mine = c0 + 8 * quarter;
    const bool inside = c0 + 64 <= C;
    Row8<B> bq[BASE ? MT : 1][2];
    if constexpr (BASE != 0) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const B *at = (const B *)base + (t0 + min(16 * m + row, live - 1)) * ldb;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (inside) bq[m][i].load(at + mine + 32 * i);
          else load_row8(bq[m][i], at, mine + 32 * i, C);
        }
      }
    }
    f32x4_t acc[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int f = 0; f < 4; ++f) acc[m][f] = (f32x4_t){0, 0, 0, 0};
    if (a >= 0) {
      for (int j0 = 0; j0 < rank; j0 += 32) {
        const int j = j0 + 8 * quarter;
        Row8<W> wq[4];
        Row8<float> uq[MT];
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const int64_t c = min(c0 + 32 * (f >> 1) + 8 * (row >> 2) + 4 * (f & 1) + (row & 3), C - 1);
          load_ranks(wq[f], w + ((int64_t)a * C + c) * rank, j, rank, eights);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) load_ranks(uq[m], u + (t0 + min(16 * m + row, live - 1)) * rank, j, rank, eights);
        __builtin_amdgcn_sched_barrier(0);
        Operand<W> wo[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          zero_unless(wq[f], j < rank);
          wo[f].set(wq[f]);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          zero_unless(uq[m], j < rank);
          Operand<float> uo;
          uo.set(uq[m]);
#pragma unroll
          for (int f = 0; f < 4; ++f) multiply16(acc[m][f], wo[f], uo);
        }
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (16 * m + row >= live) continue;
      const int64_t at = (t0 + 16 * m + row) * ldy;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v[8];
        if constexpr (BASE != 0) {
          bq[m][i].get(v);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = 0.0f;
        }
        if (a >= 0) {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = __builtin_fmaf(acc[m][2 * i + k / 4][k % 4], factor, v[k]);
        }
        if (y_bf16) {
          Row8<uint16_t> q;
          q.set(v);
          if (inside) q.store((uint16_t *)y + at + mine + 32 * i);
          else store_row8(q, (uint16_t *)y + at, mine + 32 * i, C);
        } else {
          Row8<float> q;
          q.set(v);
          if (inside) q.store((float *)y + at + mine + 32 * i);
          else store_row8(q, (float *)y + at, mine + 32 * i, C);
        }
      }
    }
  }
}

// ------------------------------------------------------------ gradients --

// Sums over the rows t of all segments of an adapter of x[t][c] g[t][j], x
// with C columns, as [r][C] (dA) or, with TURN, [C][r] (dB).  Rows run along
// the reduction: 32 of them a stage, of a segment, go to LDS as they lie, and
// the lanes fetch 8 rows of a column: by transposing reads where they are bf16
// (two 32-byte chunks of a row trade places by row, as in the grouped weight
// gradient), else, and g always, by 8 reads whose lanes are neighbours.
// grid: (256 columns, adapters, shares of the rows); with several shares
// partial sums go to partial[share][adapter][...].
//
// x of whole words goes to LDS by DMA, two stages ahead; x at odd places by way
// of registers, one stage ahead.
//
// 8192 rows of 5120 bf16 columns, rank 16, 6 adapters of unlike lengths: 38 to 50
// us (1.7 to 2.2 TB/s), bound by the longest adapter's shares, of which each
// stage costs the four waves the splitting of g into parts.  Its stages are dealt
// out in turn: runs of rows took 69 to 84 us, since segments begin and end inside
// them; twice the shares took 218 us a call instead of 211.
constexpr int kGradRows = 32, kGradCols = 256;
template <typename X, int RF, bool DMA> struct Grad {
  static constexpr int kRowX = kGradCols * sizeof(X), kX = kGradRows * kRowX;
  static constexpr int kG = kGradRows * 32 * RF * 4 + 256;            // g's rows lie together, a rank apart
  static constexpr int kStage = kX + kG, kRing = DMA ? 3 : 2;
  static_assert(kRing * kStage <= 160 * 1024, "the stages fit a CU's LDS");
  // DMA instructions (1 KB) a wave and stage: a wave copies 8 rows of x
  static constexpr int kIX = kX / 4096, kRows = 1024 / kRowX;
};
// Where a stage lies: rows at .. at + 31 of a segment that ends at `end`.
struct GradStage {
  int64_t at, end;
};

template <typename X, int RF, bool TURN, bool DMA>
__global__ __launch_bounds__(256) void k_grad(Segments s, const X *x, int64_t ldx, int64_t C, const float *g, int rank,
                                              const float *scale, void *out, int out_bf16, float *partial) {
  using T = Grad<X, RF, DMA>;
  constexpr bool kWide = sizeof(X) == 4;
  constexpr int kXP = Operand<X>::kParts;
  __shared__ __align__(16) uint8_t lds[T::kRing * T::kStage];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int a = blockIdx.y;
  const int64_t c0 = (int64_t)blockIdx.x * kGradCols;

  // the stages one after the other, every gridDim.z-th of the adapter's; past the
  // last one, empty ones
  const int shares = gridDim.z;
  int e = next_of(s, a, 1), before = 0;             // stages of earlier segments, modulo the shares
  GradStage now = {0, 0};
  const auto enter = [&]() {
    for (; e < s.g.count - 1; e = next_of(s, a, e + 1)) {
      const int64_t begin = uniform64(s.g.at(e)), end = uniform64(s.g.at(e + 1));
      const int skip = ((int)blockIdx.z - before + shares) % shares;
      now = {begin + (int64_t)skip * kGradRows, end};
      if (now.at < end) return;
      before = (int)((before + (end - begin + kGradRows - 1) / kGradRows) % shares);
    }
    now = {0, 0};
  };
  enter();
  // (one without rows leaves zeros, whatever its scale)
  const float factor = scale && now.at < now.end ? scale[a] : 1.0f;
  const auto advance = [&]() {
    if (now.at >= now.end) return;
    now.at += (int64_t)shares * kGradRows;
    if (now.at < now.end) return;
    before = (int)((before + (uniform64(s.g.size(e)) + kGradRows - 1) / kGradRows) % shares);
    e = next_of(s, a, e + 1);
    enter();
  };

  // ---- into LDS
  const uint32_t xp = (uint32_t)(ldx * sizeof(X));
  // lane l copies 16 bytes, l % kPer of row l / kPer; bf16 chunks (32 bytes)
  // turned by 2 (row % 4)
  constexpr int kPer = T::kRowX / 16 < 64 ? T::kRowX / 16 : 64;
  uint32_t xat[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    xat[i] = kWide ? 16 * (uint32_t)lane : (uint32_t)(lane / kPer) * xp + 16 * (uint32_t)((lane % kPer) ^ (4 * (2 * i + lane / kPer)));
  const auto copy = [&](uint8_t *buf) {
    const int64_t rows = min(now.end - now.at, (int64_t)kGradRows), cols = min(C - c0, (int64_t)kGradCols);
    const __amdgpu_buffer_rsrc_t xv = make_rsrc(x + (rows > 0 ? now.at * ldx + c0 : 0),
                                                rows > 0 ? (uint32_t)(rows - 1) * xp + (uint32_t)(cols * sizeof(X)) : 0u);
    const __amdgpu_buffer_rsrc_t gv = make_rsrc(g + (rows > 0 ? now.at * rank : 0), rows > 0 ? (uint32_t)rows * rank * 4 : 0u);
#pragma unroll
    for (int i = 0; i < T::kIX; ++i) {
      const int r = 8 * wave + i * T::kRows;
      if constexpr (kWide) {
        // (a view for each row, wherever it lies)
        const bool in = r < rows;
        dma16(make_rsrc(x + (in ? (now.at + r) * ldx + c0 : 0), in ? (uint32_t)cols * 4 : 0u), buf + r * T::kRowX, xat[0], 0);
      } else {
        dma16(xv, buf + r * T::kRowX, xat[i & 1], (uint32_t)r * xp);
      }
    }
    // g's 128 rank bytes, a KB an instruction, the same number for each wave
#pragma unroll
    for (int i = 0; i < RF; ++i) {
      const uint32_t at = (uint32_t)(4 * i + wave) * 1024;
      dma16(gv, buf + T::kX + at, 16 * (uint32_t)lane, at);
    }
  };
  // (bf16 at odd places)
  constexpr int kXL = kGradRows * (kGradCols / 8) / 256, kGL = kGradRows * 32 * RF / 256;
  Row8<X> xr[DMA ? 1 : kXL];
  float gr[DMA ? 1 : kGL];
  const auto load = [&]() {
    if constexpr (!DMA) {
#pragma unroll
      for (int i = 0; i < kXL; ++i) {
        const int p = tid + i * 256;
        const int64_t t = now.at + p / (kGradCols / 8);
        load_row8(xr[i], x + t * ldx, c0 + p % (kGradCols / 8) * 8, t < now.end ? C : 0);
      }
#pragma unroll
      for (int i = 0; i < kGL; ++i) {
        const int64_t p = tid + i * 256;
        gr[i] = p < min(now.end - now.at, (int64_t)kGradRows) * rank ? g[now.at * rank + p] : 0.0f;
      }
    }
  };
  const auto put = [&](uint8_t *buf) {
    if constexpr (!DMA) {
#pragma unroll
      for (int i = 0; i < kXL; ++i) {
        const int p = tid + i * 256, r = p / (kGradCols / 8), c = p % (kGradCols / 8);
        *reinterpret_cast<u32x4_t *>(buf + r * T::kRowX + 16 * (c ^ (4 * (r & 3)))) = xr[i].r;
      }
#pragma unroll
      for (int i = 0; i < kGL; ++i) *reinterpret_cast<float *>(buf + T::kX + 4 * (tid + i * 256)) = gr[i];
    }
  };

  float16_t acc[RF][2];
#pragma unroll
  for (int f = 0; f < RF; ++f)
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[f][q][i] = 0.0f;
  const int r = lane & 31, h = lane >> 5;
  uint32_t xcol[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int chunk = 4 * wave + 2 * q + ((lane >> 4) & 1);
    xcol[q] = kWide ? 8 * h * T::kRowX + 4 * (64 * wave + 32 * q + r)
                    : (8 * h + ((lane >> 2) & 3)) * T::kRowX + 32 * (chunk ^ (2 * ((lane >> 2) & 3))) + 8 * (lane & 3);
  }
  const auto eight = [&](const char *p, int pitch) {
    Row8<float> q;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const float *>(p + i * pitch);
    q.set(v);
    return q;
  };
  const auto products = [&](const char *buf) {
#pragma unroll
    for (int ks = 0; ks < kGradRows / 16; ++ks) {
      Operand<X> xo[2];
      Operand<float> go[RF];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const char *at = buf + xcol[q] + ks * 16 * T::kRowX;
        if constexpr (kWide) xo[q].set(eight(at, T::kRowX));
        else xo[q].v[0] = lds_column(at, T::kRowX);
      }
#pragma unroll
      for (int f = 0; f < RF; ++f) go[f].set(eight(buf + T::kX + ((16 * ks + 8 * h) * rank + 32 * f + r) * 4, rank * 4));
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int k = 0; k < kXP; ++k) {
          if (p + k > 2) continue;
#pragma unroll
          for (int f = 0; f < RF; ++f)
#pragma unroll
            for (int q = 0; q < 2; ++q)
              acc[f][q] = TURN ? __builtin_amdgcn_mfma_f32_32x32x16_bf16(xo[q].v[k], go[f].v[p], acc[f][q], 0, 0, 0)
                               : __builtin_amdgcn_mfma_f32_32x32x16_bf16(go[f].v[p], xo[q].v[k], acc[f][q], 0, 0, 0);
        }
    }
  };
  if (now.at < now.end) {
    if constexpr (DMA) {
      constexpr int kCopies = T::kIX + RF, kAhead = T::kRing - 1;
      GradStage at[T::kRing];                       // the stages in the ring
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        at[i] = now;
        copy(lds + i * T::kStage);
        advance();
      }
      int place = 0;
      while (at[0].at < at[0].end) {
        // this wave's copies of the stage (those behind it stay under way), and
        // every wave past its reads of the one before
        meet<(wait_vm((kAhead - 1) * kCopies) & ~0x0F00)>();
        const int free = place == 0 ? T::kRing - 1 : place - 1;
        at[kAhead] = now;
        copy(lds + free * T::kStage);
        advance();
        products((const char *)lds + place * T::kStage);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) at[i] = at[i + 1];
        place = place + 1 == T::kRing ? 0 : place + 1;
      }
      __builtin_amdgcn_s_waitcnt(wait_vm(0));       // nothing is left that writes LDS
    } else {
      int turn = 0;
      load();
      put(lds);
      advance();
      bool next = now.at < now.end;
      if (next) load();
      __syncthreads();
      for (;;) {
        products((const char *)lds + turn * T::kStage);
        if (!next) break;
        put(lds + (turn ^ 1) * T::kStage);
        advance();
        next = now.at < now.end;
        if (next) load();
        __syncthreads();
        turn ^= 1;
      }
    }
  }
  const int64_t size = (int64_t)rank * C;
  const int64_t first = gridDim.z > 1 ? ((int64_t)blockIdx.z * gridDim.y + a) * size : a * size;
  // register i of a fragment is its row 8 (i / 4) + 4 h + i % 4, the lane its column
#pragma unroll
  for (int f = 0; f < RF; ++f)
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int down = 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3), over = lane & 31;
        const int j = 32 * f + (TURN ? over : down);
        const int64_t c = c0 + 64 * wave + 32 * q + (TURN ? down : over);
        if (j >= rank || c >= C) continue;
        const int64_t to_at = first + (TURN ? c * rank + j : j * C + c);
        const float v = acc[f][q][i] * factor;
        if (gridDim.z > 1) partial[to_at] = v;
        else if (out_bf16) ((uint16_t *)out)[to_at] = (uint16_t)pack_bf16(v, 0.0f);
        else ((float *)out)[to_at] = v;
      }
}

// The shares' sums, in their order; zeros for an adapter that no segment has.
__global__ __launch_bounds__(256) void k_grad_join(Segments s, const float *partial, int shares, int64_t size, void *out,
                                                   int out_bf16) {
  const int a = blockIdx.y;
  const bool used = next_of(s, a, 1) < s.g.count - 1;
  const int64_t all = size * s.adapters;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < size; i += (int64_t)gridDim.x * 256) {
    float v = 0.0f;
    if (used)
      for (int z = 0; z < shares; ++z) v += partial[z * all + a * size + i];
    if (out_bf16) ((uint16_t *)out)[a * size + i] = (uint16_t)pack_bf16(v, 0.0f);
    else ((float *)out)[a * size + i] = v;
  }
}

// B as [r][N] and A as [K][r] for the adapters that a segment has: kTurn of the
// long side and the whole rank a workgroup, B's workgroups first, read and
// written as they lie.  (6 adapters of rank 16, 5120 + 5120: 5.4 us, mostly its
// start; two launches of square tiles took 20.)
constexpr int kTurn = 64;
template <typename W>
__global__ __launch_bounds__(256) void k_turn(Segments s, const W *b, W *b_turned, int64_t N, const W *a, W *a_turned,
                                              int64_t K, int rank) {
  extern __shared__ __align__(16) uint8_t turn_lds[];
  W *const tile = reinterpret_cast<W *>(turn_lds);       // [rank][kTurn + 1]
  const int adapter = blockIdx.y;
  if (next_of(s, adapter, 1) == s.g.count - 1) return;
  const int blocks_b = (int)((N + kTurn - 1) / kTurn);
  const bool first = (int)blockIdx.x < blocks_b;
  const int64_t L = first ? N : K, at = (int64_t)(first ? blockIdx.x : blockIdx.x - blocks_b) * kTurn;
  const int live = (int)min(L - at, (int64_t)kTurn);
  const int64_t base = (int64_t)adapter * rank * L;
  if (first) {
#pragma unroll 4
    for (int i = threadIdx.x; i < live * rank; i += 256) tile[i % rank * (kTurn + 1) + i / rank] = b[base + at * rank + i];
  } else {
#pragma unroll 4
    for (int i = threadIdx.x; i < kTurn * rank; i += 256)
      if (i % kTurn < live) tile[i / kTurn * (kTurn + 1) + i % kTurn] = a[base + i / kTurn * L + at + i % kTurn];
  }
  __syncthreads();
  if (first) {
    for (int i = threadIdx.x; i < kTurn * rank; i += 256)
      if (i % kTurn < live) b_turned[base + i / kTurn * L + at + i % kTurn] = tile[i / kTurn * (kTurn + 1) + i % kTurn];
  } else {
    for (int i = threadIdx.x; i < live * rank; i += 256) a_turned[base + at * rank + i] = tile[i % rank * (kTurn + 1) + i / rank];
  }
}

// -------------------------------------------------------------- launches --

template <typename X, typename W>
void shrink(const Segments &s, const X *x, int64_t ldx, int64_t C, const W *w, int rank, const float *scale, float *out,
            hipStream_t stream) {
  // 32 rows a tile where 16 would make more than two rounds of the CUs.  us a
  // call (K 5120, N 64; tiles of 16 rows / of 32) of rank 16, 32, 64: bf16 8200
  // rows 37 / 39, 54 / 49, 83 / 69, 32768 rows 105 / 98, 156 / 128, 244 / 170;
  // float32 x, bf16 weights 8200 rows 59 / 69, 74 / 109, 144 / 98, 32768 rows 169 /
  // 174, 216 / 278, 438 / 243.  (Float32 of rank up to 32 loses by it: the
  // registers of that form spill.  4099 bf16 rows would gain: 28 / 24, 39 / 29,
  // 59 / 39.)
  const bool pairs = s.g.rows > 16 * 2 * (int64_t)device_cus() && rank <= 64;
  const int64_t tile = pairs ? 32 : 16, tiles = s.g.rows / tile + std::min<int64_t>(s.g.count, s.g.rows);
  const auto launch = [&](auto kernel, int rf) {
    const int most = rf * (pairs ? 2 : 1) > 4 ? 8 : 16;
    const int64_t chunks = std::max<int64_t>(1, (C + kChunk - 1) / kChunk), rounds = (chunks + most - 1) / most;
    const int waves = (int)((chunks + rounds - 1) / rounds);
    kernel<<<(unsigned)tiles, 64 * waves, (size_t)waves * tile * 16 * rf * 4, stream>>>(s, x, ldx, C, w, rank, scale, out,
                                                                                       waves);
  };
  if (rank <= 16) pairs ? launch(k_shrink<X, W, 1, 2>, 1) : launch(k_shrink<X, W, 1, 1>, 1);
  else if (rank <= 32) pairs ? launch(k_shrink<X, W, 2, 2>, 2) : launch(k_shrink<X, W, 2, 1>, 2);
  else if (rank <= 64) pairs ? launch(k_shrink<X, W, 4, 2>, 4) : launch(k_shrink<X, W, 4, 1>, 4);
  else launch(k_shrink<X, W, 8, 1>, 8);
}

template <typename W>
void expand(const Segments &s, const float *u, int rank, const W *w, const float *scale, const void *base, int base_bf16,
            int64_t ldb, void *y, int y_bf16, int64_t ldy, int64_t C, hipStream_t stream) {
  const bool few = s.g.rows <= 16 * (int64_t)(s.g.count - 2);
  const int64_t tile = few ? 16 : 32;
  const int64_t tiles = s.g.rows / tile + std::min<int64_t>(s.g.count, s.g.rows), across = (C + 255) / 256;
  // several spans a workgroup where the CUs have 8 workgroups each without: finding
  // the rows is paid once (4099 rows of 20480 columns: 138 us a call with one span,
  // 132 with four, 136 with eight)
  const int spans = (int)std::max<int64_t>(1, std::min<int64_t>(4, tiles * across / (8 * (int64_t)device_cus())));
  const int tiles_c = (int)((across + spans - 1) / spans);
  const auto launch = [&](auto kernel) {
    kernel<<<(unsigned)(tiles * tiles_c), 256, 0, stream>>>(s, u, rank, w, scale, base, ldb, y, y_bf16, ldy, C, tiles_c,
                                                            spans);
  };
  with_flag(few, [&](auto f) {
    constexpr int MT = f.value ? 1 : 2;
    if (!base) launch(k_expand<W, MT, 0>);
    else if (base_bf16) launch(k_expand<W, MT, 2>);
    else launch(k_expand<W, MT, 1>);
  });
}

// Shares of the rows that the gradient kernels cut a sum into: until there is
// work for two rounds of the CUs, at least 256 rows each, and within 512 MB of
// partial sums.
int shares_of(int64_t rows, int64_t C, int64_t rank, int64_t adapters, int64_t segments) {
  const int64_t work = (C + kGradCols - 1) / kGradCols * std::min(adapters, segments);
  const int64_t want = std::min(2 * (int64_t)device_cus() / std::max<int64_t>(work, 1), rows / 256);
  const int64_t room = ((int64_t)512 << 20) / std::max<int64_t>(1, adapters * rank * C * 4);
  return (int)std::max<int64_t>(1, std::min(want, room));
}

template <typename X, bool TURN>
void grad(const Segments &s, int64_t segments, const X *x, int64_t ldx, int64_t C, const float *g, int rank,
          const float *scale, void *out, int out_bf16, float *partial, hipStream_t stream) {
  const int shares = shares_of(s.g.rows, C, rank, s.adapters, segments);
  const dim3 grid((unsigned)((C + kGradCols - 1) / kGradCols), (unsigned)s.adapters, (unsigned)shares);
  const auto launch = [&](auto kernel) {
    kernel<<<grid, 256, 0, stream>>>(s, x, ldx, C, g, rank, scale, out, out_bf16, partial);
  };
  const bool words = (uintptr_t)x % 4 == 0 && ldx * sizeof(X) % 4 == 0 && C * sizeof(X) % 4 == 0 && ldx < (1LL << 24);
  const auto of_rank = [&](auto dma) {
    if (rank <= 32) launch(k_grad<X, 1, TURN, dma.value>);
    else if (rank <= 64) launch(k_grad<X, 2, TURN, dma.value>);
    else launch(k_grad<X, 4, TURN, dma.value>);
  };
  if constexpr (sizeof(X) == 2) with_flag(words, of_rank);
  else of_rank(std::true_type());
  if (shares > 1) {
    const int64_t size = rank * C;
    k_grad_join<<<dim3((unsigned)std::min<int64_t>((size + 255) / 256, 1024), (unsigned)s.adapters), 256, 0, stream>>>(
        s, partial, shares, size, out, out_bf16);
  }
}

int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }

// The backward pass' scratch memory: B and A turned, g, and the partial sums
// (one after the other: dA's are added up before dB's are written).
struct BackwardSpace {
  int64_t b_turned, a_turned, g, partial, all;
};
BackwardSpace backward_space(int64_t rows, int64_t n, int64_t k, int64_t rank, int64_t adapters, int64_t segments,
                             int64_t wsize) {
  BackwardSpace s;
  s.b_turned = 0;
  s.a_turned = s.b_turned + round16(adapters * rank * n * wsize);
  s.g = s.a_turned + round16(adapters * rank * k * wsize);
  s.partial = s.g + round16(rows * rank * 4);
  const auto need = [&](int64_t C) {
    const int64_t shares = shares_of(rows, C, rank, adapters, segments);
    return shares > 1 ? shares * adapters * rank * C * 4 : 0;
  };
  s.all = s.partial + std::max(need(n), need(k));
  return s;
}

template <typename W> void forward_w(const AdapterForward &p, const Segments &s, hipStream_t stream) {
  const W *a = (const W *)p.w.a, *b = (const W *)p.w.b;
  const int rank = (int)p.w.rank;
  if (p.x_dtype == 1) shrink(s, (const uint16_t *)p.x, p.ldx, p.w.k, a, rank, nullptr, p.u, stream);
  else shrink(s, (const float *)p.x, p.ldx, p.w.k, a, rank, nullptr, p.u, stream);
  if (p.w.n > 0)
    expand(s, p.u, rank, b, p.w.scale, p.base, p.base_dtype == 1, p.ldb, p.y, p.y_dtype == 1, p.ldy, p.w.n, stream);
}

template <typename W> void backward_w(const AdapterBackward &p, const Segments &s, hipStream_t stream) {
  const AdapterWeights &w = p.w;
  const int rank = (int)w.rank, gb = p.g_dtype == 1;
  const BackwardSpace at = backward_space(s.g.rows, w.n, w.k, rank, w.adapters, w.segments, sizeof(W));
  char *const ws = (char *)p.ws;
  W *const bt = (W *)(ws + at.b_turned), *const aT = (W *)(ws + at.a_turned);
  float *const g = (float *)(ws + at.g), *const partial = (float *)(ws + at.partial);
  if (s.g.rows > 0) {
    const int64_t blocks = (w.n + kTurn - 1) / kTurn + (w.k + kTurn - 1) / kTurn;
    if (blocks > 0)
      k_turn<W><<<dim3((unsigned)blocks, (unsigned)w.adapters), 256, sizeof(W) * rank * (kTurn + 1), stream>>>(
          s, (const W *)w.b, bt, w.n, (const W *)w.a, aT, w.k, rank);
    if (p.dy_dtype == 1) shrink(s, (const uint16_t *)p.dy, p.lddy, w.n, bt, rank, w.scale, g, stream);
    else shrink(s, (const float *)p.dy, p.lddy, w.n, bt, rank, w.scale, g, stream);
    if (w.k > 0)
      expand(s, g, rank, aT, nullptr, p.base, p.base_dtype == 1, p.ldb, p.dx, p.dx_dtype == 1, p.lddx, w.k, stream);
  }
  if (w.k > 0) {
    if (p.x_dtype == 1) grad<uint16_t, false>(s, w.segments, (const uint16_t *)p.x, p.ldx, w.k, g, rank, nullptr, p.da, gb, partial, stream);
    else grad<float, false>(s, w.segments, (const float *)p.x, p.ldx, w.k, g, rank, nullptr, p.da, gb, partial, stream);
  }
  if (w.n > 0) {
    if (p.dy_dtype == 1) grad<uint16_t, true>(s, w.segments, (const uint16_t *)p.dy, p.lddy, w.n, p.u, rank, w.scale, p.db, gb, partial, stream);
    else grad<float, true>(s, w.segments, (const float *)p.dy, p.lddy, w.n, p.u, rank, w.scale, p.db, gb, partial, stream);
  }
}

Segments segments_of(const AdapterWeights &w, int64_t rows) {
  return {{w.offsets, w.index_bits == 64, (int)w.segments + 2, rows, 1}, w.index, (int)w.adapters};
}

}  // namespace

int64_t adapters_backward_workspace_bytes(int64_t rows, int64_t n, int64_t k, int64_t rank, int64_t adapters,
                                          int64_t segments, int w_dtype) {
  return backward_space(rows, n, k, rank, adapters, segments, w_dtype == 1 ? 2 : 4).all;
}

hipError_t launch_adapters(const AdapterForward &p, hipStream_t stream) {
  if (p.rows == 0) return hipSuccess;
  const Segments s = segments_of(p.w, p.rows);
  if (p.w.w_dtype == 1) forward_w<uint16_t>(p, s, stream);
  else forward_w<float>(p, s, stream);
  return hipGetLastError();
}

hipError_t launch_adapters_backward(const AdapterBackward &p, hipStream_t stream) {
  const Segments s = segments_of(p.w, p.rows);
  if (p.w.w_dtype == 1) backward_w<uint16_t>(p, s, stream);
  else backward_w<float>(p, s, stream);
  return hipGetLastError();
}

}  // namespace nvfp4
