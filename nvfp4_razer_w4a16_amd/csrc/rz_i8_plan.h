// rz_i8_plan.h -- which kernel a product of 8-bit integer tensors runs on, and how it is
// cut: rules on sizes and the device's compute units (`cus`).  Host code.  (In a namespace of its
// own: the MXFP4 products' rules have the same names.)
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

namespace rz {
namespace i8 {

// ---- tile kernel -------------------------------------------------------------
constexpr int kTileN = 256;   // rows of W of a tile
constexpr int kStepB = 128;   // bytes of a row and step

// How a product is cut: mt x nt tiles (grouped: as many row tiles as there are),
// the last `rest` of them each in `split` slices of K whose sums go to slots of `part`.
struct TilePlan {
  int cus;
  int high;  // rows of X of a tile
  int mt, nt;
  int full, rest, split;
  int halves;  // of the full tiles, 256 high, the last ones that are done as two of 128 each
  int first;   // the first of them
  int32_t* part;
};

// us that a round of `tiles` tiles takes: a step of 256 or 128 rows, the longer the more of
// them there are (they share the memory's and the card's power), and a tile's first loads
// and results; what slices cost, their sums written and read, and another launch.
// Measured, 256 rows, 128 rows, and as chosen here:
//   1024 x 14336 x 4096  57.8  72.0  57.8     512 x 28672 x 8192   111  143  111
//   2048 x 4096 x 4096   43.5  35.8  35.8     1024 x 4096 x 4096  42.0 28.0 28.0
//   2048 x 28672 x 8192   408   478   393     1024 x 4096 x 14336  119 76.5 76.4
//   8192 rows, 8 experts of 14336 x 4096  458  540  460
//   8192 rows, 64 experts of 1536 x 2048 71.2 73.4 73.2, 16384 rows 102 93.1 92.9
inline double round_us(int high, double tiles, int cus, int steps) {
  const double f = std::min(tiles / cus, 1.0);
  return high == 256 ? steps * (0.85 + 0.62 * f) + 10.0 : steps * (0.48 + 0.5 * f) + 6.0;
}
inline double fold_us(int slices, int high) { return 3.0 + slices * high * 2.5e-4; }
inline int steps_of(int64_t k) { return (int)((k + kStepB - 1) / kStepB); }

// The tiles of a product, `high` rows each, and its time in us.  The last, partly
// filled round of tiles is cut along K where that is quicker.
inline TilePlan tiles_of(int high, int64_t m, int64_t n, int64_t k, int64_t experts, int cus, double& us) {
  TilePlan p = {};
  const int steps = steps_of(k);
  p.cus = cus;
  p.high = high;
  p.nt = (int)((n + kTileN - 1) / kTileN);
  p.mt = (int)((m + high - 1) / high + std::min(experts, m));
  p.full = (int)std::min((int64_t)p.mt * p.nt, (int64_t)INT32_MAX);  // more have no memory for their results
  p.split = 1;
  auto rounds_us = [&](double tiles) {
    const double rounds = std::floor(tiles / cus), rest = tiles - rounds * cus;
    return rounds * round_us(high, cus, cus, steps) + (rest > 0 ? round_us(high, rest, cus, steps) : 0);
  };
  if (experts) {  // of about the same number of rows, whose last tile is half full
    const int64_t parts = std::min(experts, m);
    us = rounds_us((double)p.nt * std::max(parts, m / high + parts / 2));
    return p;
  }
  us = rounds_us(p.full);
  const int rest = p.full % cus;
  const double whole = rounds_us(p.full - rest);
  for (int s = 2; s <= 8 && rest > 0 && rest * s <= cus && s <= steps; s++) {
    const double t = whole + round_us(high, rest * s, cus, (steps + s - 1) / s) + fold_us(rest * s, high);
    if (t < us) us = t, p.split = s;
  }
  if (high == 256 && rest > 0 && rest * 2 <= cus) {
    const double t = whole + round_us(128, rest * 2, cus, steps) + 6.0;
    if (t < us) us = t, p.split = 1, p.halves = rest;
  }
  if (p.split > 1) p.rest = rest, p.full -= rest;
  return p;
}
inline TilePlan tile_plan(int64_t m, int64_t n, int64_t k, int64_t experts, int cus, double& us) {
  double low_us;
  const TilePlan p = tiles_of(256, m, n, k, experts, cus, us), low = tiles_of(128, m, n, k, experts, cus, low_us);
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
  int cus;
  int ck, mt;  // ck = 0: not covered
  int rt;      // row tiles of a chunk
  int rows;    // of a job, at most 16 mt
  int pieces, last;
  int mul_pieces, mul_last;  // p / d = p * mul >> 20 for p < 2048
  Cuts cuts;                 // of a product without experts
  int mul_per_job;
};

// The stream kernel's shape for `m` rows, of each of `experts` on average if that is not 0.
inline StreamPlan stream_plan(int64_t m, int64_t n, int64_t k, int64_t experts, int cus) {
  StreamPlan p = {};
  p.cus = cus;
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
  while (p.rt > 1 && jobs * ((n + kSRows * p.rt - 1) / (kSRows * p.rt)) < cus) p.rt /= 2;
  p.pieces = (int)(((k + ck - 1) / ck + 63) / 64 * 4);  // whole products' pieces
  p.last = (int)(k / 16) - p.pieces * (ck - 1);
  p.mul_pieces = (1 << 20) / p.pieces + 1;
  p.mul_last = (1 << 20) / p.last + 1;
  return p;
}

// Whether a product runs on the stream kernel: the shorter time of two estimates, in us.
// The stream kernel's work is its row tiles, whose sums meet in LDS, and half of the
// shorter of this and the read of W shows beside the other; the tile kernel's its rounds,
// and not quite half of the read shows.  Measured, stream and tile kernel:
//   27 x 28672 x 8192   51.1 and 65.1    128 x 28672 x 8192   81.9 and 68.1
//   128 x 14336 x 4096  22.3 and 24.2    256 x 14336 x 4096   31.7 and 28.6
//   256 x 4096 x 4096   17.7 and 21.1    1024 x 4096 x 4096   34.8 and 28.0
//   64 x 4096 x 14336   23.8 and 25.0    256 x 4096 x 14336   54.1 and 30.2
//   128 x 8192 x 1024   11.7 and 12.2    512 x 8192 x 1024    24.3 and 13.7
//   8 experts of 14336 x 4096, 64 rows each 116 and 106, 128 rows 207 and 143
//   64 experts of 1536 x 2048, 8 rows each 37.0 and 47.9, 32 rows 54.9 and 54.4
struct Estimate {
  double stream, tile;
};
inline Estimate estimate(int64_t m, int64_t n, int64_t k, int64_t experts, const StreamPlan& p) {
  const int cus = p.cus;
  const int64_t parts = experts ? std::min(experts, m) : 1, rows = (m + parts - 1) / parts;  // W's used, rows each
  const double read = (double)parts * n * k / 5e6;
  const int64_t jobs = (rows + p.rows - 1) / p.rows;  // of each W
  const double units = (double)parts * jobs * ((n + kSRows * p.rt - 1) / (kSRows * p.rt));
  const double work = std::ceil(units / cus) * (0.22 * p.mt + 0.4 * p.ck);
  // an expert's jobs read its W one after the other; those of one product side by side
  const double streamed = experts ? read * jobs : read;
  double tile;
  tile_plan(m, n, k, experts, cus, tile);
  return {std::max(work, streamed) + std::min(work, streamed) / 2 + 2.5 + 0.3 * p.ck * p.mt, tile + 0.45 * read};
}
inline bool streams(int64_t m, int64_t n, int64_t k, int64_t experts, int cus, StreamPlan& p) {
  p = stream_plan(m, n, k, experts, cus);
  if (!p.ck) return false;
  const Estimate e = estimate(m, n, k, experts, p);
  return e.stream <= e.tile;
}

}  // namespace i8
}  // namespace rz
