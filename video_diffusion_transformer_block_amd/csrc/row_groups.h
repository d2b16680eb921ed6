// Rows grouped by expert: which expert's rows a tile of rows belongs to, from
// E + 1 row offsets in device memory.  Experts are taken in order, each cut
// into tiles of `bm` rows; a tile never spans two experts.
//
// An offset counts as the largest up to there, clamped to [0, T], so no
// offsets whatever reach past the T rows or give a row to two experts.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace vdtq {

struct RowTile {
  int expert, row0, rows;      // first row, and the expert's rows from there on (0: no such tile)
  int before, tiles;           // tiles of the experts before this one, and its own
};

// Running maximum and sum over the 64 lanes.
__device__ __forceinline__ int lanes_max(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o, 64);
    if (lane >= o) v = max(v, u);
  }
  return v;
}
__device__ __forceinline__ int lanes_sum(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o, 64);
    if (lane >= o) v += u;
  }
  return v;
}

// Calls f(e0, lo, hi, upto) for each 64 experts from e0: lane i's expert
// e0 + i has rows lo .. hi - 1, and `upto` counts the tiles up to and
// including its own within the 64.  f returns true to stop.  All lanes of a
// wavefront call this together.
template <class F>
__device__ __forceinline__ void each_group(const int32_t* offsets, int E, int T, int bm, F f) {
  const int lane = threadIdx.x & 63;
  int last = min(max(offsets[0], 0), T);
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = min(e0 + lane, E - 1);
    const int hi = max(last, lanes_max(min(offsets[e + 1], T)));
    int lo = __shfl_up(hi, 1, 64);
    if (lane == 0) lo = last;
    if (e0 + lane >= E) lo = hi;                      // no rows
    if (f(e0, lo, hi, lanes_sum((hi - lo + bm - 1) / bm))) return;
    last = __shfl(hi, 63, 64);
  }
}

// Tiles of all experts together.
__device__ __forceinline__ int row_tiles(const int32_t* offsets, int E, int T, int bm) {
  int n = 0;
  each_group(offsets, E, T, bm, [&](int, int, int, int upto) {
    n += __shfl(upto, 63, 64);
    return false;
  });
  return __builtin_amdgcn_readfirstlane(n);
}

// The tile among 64 experts from e0 (lane i: expert e0 + i, rows lo .. hi - 1,
// `upto` tiles with it) after `past` tiles of earlier ones.
__device__ __forceinline__ RowTile tile_among(int e0, int lo, int hi, int upto, int past, int bm, int t) {
  const int i = __builtin_ctzll(__ballot(past + upto > t));   // the first lane whose tiles reach past t
  const int before = past + (i ? __shfl(upto, i - 1, 64) : 0);
  const int row0 = __shfl(lo, i, 64) + (t - before) * bm;
  return RowTile{e0 + i, row0, __shfl(hi, i, 64) - row0, before, past + __shfl(upto, i, 64) - before};
}

__device__ __forceinline__ RowTile uniform(const RowTile& r) {
  return RowTile{(int)__builtin_amdgcn_readfirstlane(r.expert), (int)__builtin_amdgcn_readfirstlane(r.row0),
                 (int)__builtin_amdgcn_readfirstlane(r.rows), (int)__builtin_amdgcn_readfirstlane(r.before),
                 (int)__builtin_amdgcn_readfirstlane(r.tiles)};
}

// Tile t; no rows when there are not so many.
__device__ __forceinline__ RowTile row_tile(const int32_t* offsets, int E, int T, int bm, int t) {
  RowTile r{0, 0, 0, 0, 0};
  int past = 0;                                         // tiles of the 64s before
  each_group(offsets, E, T, bm, [&](int e0, int lo, int hi, int upto) {
    const int all = __shfl(upto, 63, 64);
    if (t >= past + all) {
      past += all;
      return false;
    }
    r = tile_among(e0, lo, hi, upto, past, bm, t);
    return true;
  });
  return uniform(r);
}

// The tile pick(tiles of all experts) asks for; none where it answers -1.
// The offsets of up to 64 experts are read once.
template <class F>
__device__ __forceinline__ RowTile pick_row_tile(const int32_t* offsets, int E, int T, int bm, F pick) {
  if (E <= 64) {
    RowTile r{0, 0, 0, 0, 0};
    each_group(offsets, E, T, bm, [&](int e0, int lo, int hi, int upto) {
      const int t = pick((int)__builtin_amdgcn_readfirstlane(__shfl(upto, 63, 64)));
      if (t >= 0) r = tile_among(e0, lo, hi, upto, 0, bm, t);
      return true;
    });
    return uniform(r);
  }
  const int t = pick(row_tiles(offsets, E, T, bm));
  return t >= 0 ? row_tile(offsets, E, T, bm, t) : RowTile{0, 0, 0, 0, 0};
}

}  // namespace vdtq
