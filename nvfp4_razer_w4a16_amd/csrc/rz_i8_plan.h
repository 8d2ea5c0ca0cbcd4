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

// ---- stream kernel -----------------------------------------------------------
constexpr int kSRows = 16, kChunkB = 2048;  // rows of a row tile, bytes of a row in a chunk

// How the line of all jobs' row tiles is cut: into pieces as even as can be, or, where
// that makes none longer by more than loading another job's X takes, two row tiles or
// so, every job into `per_job` pieces.
struct Cuts {
  uint32_t jobs, per_job;  // 0: even pieces of the line
  uint32_t share, extra;   // the first `extra` pieces are share + 1 tiles
};
__host__ __device__ __forceinline__ Cuts cuts_of(uint32_t tiles, uint32_t jobs, uint32_t grid, uint32_t rt) {
  const uint32_t line = tiles * jobs;
  Cuts c = {jobs, jobs ? grid / jobs : 0, line / grid, 0};
  const uint32_t most = c.per_job ? tiles / c.per_job : 0, rest = tiles - most * c.per_job;
  if (c.per_job && most + (rest ? 1 : 0) <= c.share + 2 * rt) {
    c.share = most;
    c.extra = rest;
  } else {
    c.per_job = 0;
    c.extra = line - c.share * grid;
  }
  return c;
}

// The chunks of a row: `ck` of them, each `pieces` 16-byte pieces, the last `last`.
struct StreamPlan {
  int ck, mt;  // ck = 0: not covered
  int rt;      // row tiles of a chunk
  int rows;    // of a job, at most 16 mt
  int pieces, last;
  int mul_pieces, mul_last;  // p / d = p * mul >> 20 for p < 2048
  Cuts cuts;                 // of a product without experts
  int mul_per_job;
};

// The stream kernel's shape for `m` rows, of each of `experts` on average if that is not 0.
inline StreamPlan stream_plan(int64_t m, int64_t n, int64_t k, int64_t experts) {
  StreamPlan p = {};
  int ck = 1;
  while ((int64_t)ck * kChunkB < k) ck *= 2;
  if (ck > 8) return p;  // X would not fit the registers
  // rows a job: X of CK chunks has to fit the registers; experts' rows scatter about the average
  const int64_t rows = experts ? (m + experts - 1) / experts * 3 / 2 : m;
  const int most = std::min(4, 8 / ck);
  p.mt = std::min(rows <= 16 ? 1 : rows <= 32 ? 2 : 4, most);
  p.rows = 16 * p.mt;
  if (!experts && m > p.rows) {
    // A power of two of jobs: workgroups that walk through the same piece of W are then
    // on one XCD and share its L2.
    int64_t jobs = 1;
    while (jobs < 32 && jobs * p.rows < m) jobs *= 2;
    if (jobs * p.rows >= m) p.rows = (int)((m + jobs - 1) / jobs);
  }
  p.ck = ck;
  // Short rows: several row tiles a chunk, if there is a chunk for every CU.
  const int64_t jobs = experts ? std::min(experts, m) : (m + p.rows - 1) / p.rows;
  p.rt = p.mt == 4 ? 1 : k <= kChunkB / 4 ? 4 : k <= kChunkB / 2 ? 2 : 1;
  while (p.rt > 1 && jobs * ((n + kSRows * p.rt - 1) / (kSRows * p.rt)) < device_cu_count()) p.rt /= 2;
  p.pieces = (int)(((k + ck - 1) / ck + 63) / 64 * 4);  // whole products' pieces
  p.last = (int)(k / 16) - p.pieces * (ck - 1);
  p.mul_pieces = (1 << 20) / p.pieces + 1;
  p.mul_last = (1 << 20) / p.last + 1;
  return p;
}

// Whether a product runs on the stream kernel: the shorter time of two estimates, in us.
// Both take what the kernel's own work and the read of W come to, one of them half
// hidden behind the other, and what a launch costs.
inline bool streams(int64_t m, int64_t n, int64_t k, int64_t experts, StreamPlan& p) {
  p = stream_plan(m, n, k, experts);
  if (!p.ck) return false;
  const int cus = device_cu_count();
  const int64_t parts = experts ? std::min(experts, m) : 1, rows = (m + parts - 1) / parts;  // W's used, rows each
  auto whole = [](double us) { return (int)std::min(us, 1e9); };
  const int read = whole((double)parts * n * k / 5e6);
  auto rounds = [&](int64_t units) { return (double)((units + cus - 1) / cus); };
  auto total = [&](double us, double fixed) {
    const int work = whole(us);
    return std::max(work, read) + std::min(work, read) / 2 + fixed;
  };
  const double stream = rounds(parts * ((rows + p.rows - 1) / p.rows) * ((n + kSRows * p.rt - 1) / (kSRows * p.rt))) *
                        (0.25 * p.mt + 0.3 * p.ck);
  double tile;
  tile_plan(m, n, k, experts, tile);
  return total(stream, 3.0 + 0.4 * p.ck * p.mt) <= total(tile, 4.0);  // X is loaded first
}

}  // namespace i8
}  // namespace rz
