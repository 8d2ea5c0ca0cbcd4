// rz_i8_plan.h -- which kernel a product of 8-bit integer tensors runs on, and how it is
// cut: rules on sizes and the device's compute units.  Host code.  (In a namespace of its
// own: the MXFP4 products' rules have the same names.)
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "rz_i8_launch.h"

namespace rz {
namespace i8 {

// ---- tile kernel -------------------------------------------------------------
constexpr int kTileN = 256;   // rows of W of a tile
constexpr int kStepB = 128;   // bytes of a row and step

// How a product is cut: mt x nt tiles (grouped: as many row tiles as there are),
// the last `rest` of them each in `split` slices of K whose sums go to slots of `part`.
struct TilePlan {
  int high;  // rows of X of a tile
  int mt, nt;
  int full, rest, split;
  int halves;  // of the full tiles, 256 high, the last ones that are done as two of 128 each
  int first;   // the first of them
  int32_t* part;
};

// us that a step of a tile of 256 or 128 rows takes in a full round, and in one that
// leaves CUs (and power) to spare; what slices cost, their sums written and read.
inline double step_us(int high, bool full) { return high == 256 ? full ? 1.5 : 1.3 : full ? 0.9 : 0.8; }
inline double fold_us(int slices, int high) { return 4.0 + slices * high * (0.1 / 256); }
inline int steps_of(int64_t k) { return (int)((k + kStepB - 1) / kStepB); }

// The tiles of a product, `high` rows each, and its time in us.  The last, partly
// filled round of tiles is cut along K where that is quicker.
inline TilePlan tiles_of(int high, int64_t m, int64_t n, int64_t k, int64_t experts, double& us) {
  TilePlan p = {};
  const int cus = device_cu_count(), steps = steps_of(k);
  p.high = high;
  p.nt = (int)((n + kTileN - 1) / kTileN);
  p.mt = (int)((m + high - 1) / high + std::min(experts, m));
  p.full = (int)std::min((int64_t)p.mt * p.nt, (int64_t)INT32_MAX);  // more have no memory for their results
  p.split = 1;
  if (experts) {  // of about the same number of rows, whose last tile is half full
    const int64_t parts = std::min(experts, m);
    const double tiles = (double)p.nt * std::max(parts, m / high + parts / 2), rounds = std::floor(tiles / cus);
    us = (rounds * step_us(high, true) + (tiles > rounds * cus ? step_us(high, false) : 0)) * steps;
    return p;
  }
  const int rest = p.full % cus;
  double best = rest ? steps * step_us(high, false) : 0;
  for (int s = 2; s <= 8 && rest > 0 && rest * s <= cus && s <= steps; s++) {
    const double t = (steps + s - 1) / s * step_us(high, false) + fold_us(rest * s, high);
    if (t < best) best = t, p.split = s;
  }
  if (high == 256 && rest * 2 <= cus && steps * step_us(128, true) + 6.0 < best) {
    best = steps * step_us(128, true) + 6.0;
    p.halves = rest;
    p.split = 1;
  }
  us = p.full / cus * step_us(high, true) * steps + best;
  if (p.split > 1) p.rest = rest, p.full -= rest;
  return p;
}
inline TilePlan tile_plan(int64_t m, int64_t n, int64_t k, int64_t experts, double& us) {
  double low_us;
  const TilePlan p = tiles_of(256, m, n, k, experts, us), low = tiles_of(128, m, n, k, experts, low_us);
  if (low_us >= us + 1.0) return p;  // the larger tile's results take longer to store
  us = low_us;
  return low;
}
inline size_t tile_ws_bytes(const TilePlan& p) { return (size_t)p.rest * p.split * kTileN * p.high * 4; }

}  // namespace i8
}  // namespace rz
