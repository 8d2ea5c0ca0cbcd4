// rz_groups.h -- the rows of products grouped by expert, cut into tiles: device code
// shared by the grouped products.
#pragma once

#include "rz_device.h"

namespace rz {

// The rows [m0, m1) of one expert's tile.
struct Tile {
  int64_t m0, m1;
  int expert;  // -1: no such tile
};

// Tile t of the grouped product's row tiles, each `rows` high and within one
// expert's run.  Every wave works it out for itself: lane l counts the tiles of
// expert l and a running sum over the lanes finds the one that holds t.
// Offsets outside [0, m] are clamped.
__device__ __forceinline__ Tile find_tile(const int32_t* offsets, int experts, int64_t m_rows, int rows, int64_t t) {
  const int lane = threadIdx.x & 63;
  const int m = (int)m_rows;
  int before = 0;
  for (int e0 = 0; e0 < experts; e0 += 64) {
    const int e = e0 + lane;
    int lo = 0, hi = 0;
    if (e < experts) {
      lo = min(max(offsets[e], 0), m);
      hi = min(max(offsets[e + 1], lo), m);
    }
    const int cnt = (hi - lo + rows - 1) / rows;
    int sum = cnt;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(sum, o, 64);
      if (lane >= o) sum += up;
    }
    sum += before;
    const uint64_t hit = __ballot(sum > t);
    if (hit) {
      const int src = __builtin_ctzll(hit);
      const int first = __builtin_amdgcn_readlane(sum - cnt, src);
      const int l = __builtin_amdgcn_readlane(lo, src), h = __builtin_amdgcn_readlane(hi, src);
      const int m0 = l + (int)(t - first) * rows;
      return {m0, min(m0 + rows, h), e0 + src};
    }
    before = __builtin_amdgcn_readlane(sum, 63);
  }
  return {0, 0, -1};
}

// Number of row tiles, each `rows` high, of the grouped product.
__device__ __forceinline__ int live_tiles(const int32_t* offsets, int experts, int64_t m_rows, int rows) {
  const int lane = threadIdx.x & 63, m = (int)m_rows;
  int cnt = 0;
  for (int e = lane; e < experts; e += 64) {
    const int lo = min(max(offsets[e], 0), m), hi = min(max(offsets[e + 1], lo), m);
    cnt += (hi - lo + rows - 1) / rows;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) cnt += __shfl_xor(cnt, o, 64);
  return __builtin_amdgcn_readfirstlane(cnt);
}

// The same for a kernel that looks tiles up more than once: what lane l counts for expert l
// stays in registers, if there are no more than 64.
struct RowTiles {
  int lo, hi, cnt, sum;  // lane l: expert l's rows, its tiles, and those of the experts up to it
  int count;             // of all experts
};
__device__ __forceinline__ RowTiles row_tiles(const int32_t* offsets, int experts, int64_t m_rows, int rows) {
  const int lane = threadIdx.x & 63, m = (int)m_rows;
  RowTiles r = {};
  if (experts > 64) {
    r.count = live_tiles(offsets, experts, m_rows, rows);
    return r;
  }
  if (lane < experts) {
    r.lo = min(max(offsets[lane], 0), m);
    r.hi = min(max(offsets[lane + 1], r.lo), m);
  }
  r.cnt = r.sum = (r.hi - r.lo + rows - 1) / rows;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int up = __shfl_up(r.sum, o, 64);
    if (lane >= o) r.sum += up;
  }
  r.count = __builtin_amdgcn_readlane(r.sum, 63);
  return r;
}
__device__ __forceinline__ Tile find_tile(const RowTiles& r, const int32_t* offsets, int experts, int64_t m_rows, int rows,
                                          int64_t t) {
  if (experts > 64) return find_tile(offsets, experts, m_rows, rows, t);
  const uint64_t hit = __ballot(r.sum > t);
  if (!hit) return {0, 0, -1};
  const int src = __builtin_ctzll(hit);
  const int m0 = __builtin_amdgcn_readlane(r.lo, src) + (int)(t - __builtin_amdgcn_readlane(r.sum - r.cnt, src)) * rows;
  return {m0, min(m0 + rows, __builtin_amdgcn_readlane(r.hi, src)), src};
}

}  // namespace rz
