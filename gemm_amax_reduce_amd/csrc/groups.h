// groups.h -- ragged groups of consecutive rows, given by offsets in device
// memory: group e is rows offsets[e] .. offsets[e + 1) - 1 of a matrix of
// `rows` rows, and rows in front of the first or behind the last belong to
// none.  The host knows only how many groups and rows there are, so grids are
// made for the most tiles that these can have, and a workgroup finds its own.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

// With `cover` the rows in front and behind are groups of their own, the first
// and the last of `count`.
struct Groups {
  const void *offsets;
  int is64;
  int count;
  int64_t rows;
  int cover;
  // where group i begins (i == count: where the last one ends), kept inside the
  // matrix whatever is stored there
  __device__ __forceinline__ int64_t at(int i) const {
    if (cover) {
      if (i == 0 || i == count) return i ? rows : 0;
      i -= 1;
    }
    const int64_t v = is64 ? ((const int64_t *)offsets)[i] : (int64_t)((const int32_t *)offsets)[i];
    return min(max(v, (int64_t)0), rows);
  }
  __device__ __forceinline__ int64_t size(int e) const { return max(at(e + 1) - at(e), (int64_t)0); }
};

// A tile of up to `tile` rows of a group; e < 0: none.
struct GroupTile {
  int e;
  int local;            // which of the group's tiles
  int tiles;            // how many it has
  int64_t begin, end;   // the group's rows
};

// A value that is the same in every lane, for the compiler to know.
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 |
                   (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}
__device__ __forceinline__ int wave_total(int v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}
// How many tiles all groups have.
__device__ __forceinline__ int count_tiles(const Groups &g, int tile) {
  const int lane = threadIdx.x & 63;
  int total = 0;
  for (int e0 = 0; e0 < g.count; e0 += 64) {
    const int e = e0 + lane;
    total += wave_total(e < g.count ? (int)((g.size(e) + tile - 1) / tile) : 0);
  }
  return __builtin_amdgcn_readfirstlane(total);
}
// The index-th of all tiles, counted over the groups in their order, found by a
// wave 64 groups at a time; every lane has the result.  `index` counts tiles of
// rows times `units` (the tiles of a row of tiles); local is the place among the
// group's tiles x units.
__device__ __forceinline__ GroupTile find_tile(const Groups &g, int tile, int units, int index) {
  const int lane = threadIdx.x & 63;
  GroupTile t = {-1, 0, 0, 0, 0};
  int before = 0;
  for (int e0 = 0; e0 < g.count; e0 += 64) {
    const int e = e0 + lane;
    const int tiles = e < g.count ? (int)((g.size(e) + tile - 1) / tile) : 0;
    int sum = tiles * units;                               // inclusive prefix over the wave
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int v = __shfl_up(sum, off, 64);
      if (lane >= off) sum += v;
    }
    const int all = __builtin_amdgcn_readfirstlane(__shfl(sum, 63, 64));      // (uniform, so that the branch is)
    if (index < before + all) {
      const uint64_t past = __ballot(before + sum > index);
      const int who = __builtin_ctzll(past);
      t.e = __builtin_amdgcn_readfirstlane(e0 + who);
      t.tiles = __builtin_amdgcn_readfirstlane(__shfl(tiles, who, 64));
      t.local = __builtin_amdgcn_readfirstlane(index - before - (__shfl(sum, who, 64) - t.tiles * units));
      t.begin = uniform64(g.at(t.e));
      t.end = uniform64(g.at(t.e + 1));
      return t;
    }
    before += all;
  }
  return t;
}

}  // namespace nvfp4
