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
constexpr int kStepB = 128;   // bytes of a row and step

// How a product is cut: mt x nt tiles (grouped: as many row tiles as there are),
// the last `rest` of them each in `split` slices of K whose sums go to slots of `part`.
struct TilePlan {
  int cus;
  int wide, high;  // rows of W and of X of a tile: 256 x 256, 256 x 128 or 128 x 128
  int mt, nt;
  int full, rest, split;
  int halves;  // of the full tiles, 256 high, the last ones that are done as two of 128 each
  int first;   // the first of them
  int32_t* part;
};

// us that a round of `tiles` tiles takes: a step of K, the longer the more of them there are
// (they share the memory's and the card's power; two tiles of 128 x 128 on a CU its LDS), and
// a tile's first loads and results; what slices cost, their sums written and read, and another
// launch.  Measured, tiles of 256 x 256, 256 x 128, 128 x 128, and as chosen here:
//   1024 x 4096 x 4096   42.0 27.3 23.1 21.9   512 x 4096 x 4096   40.8 23.3 20.2 20.2
//   2048 x 4096 x 4096   43.5 35.7 36.7 35.3   1024 x 4096 x 14336  119 74.2 62.6 61.2
//   256 x 14336 x 4096   40.0 27.6 22.4 21.7   512 x 14336 x 4096  39.7 33.1 34.5 32.1
//   1024 x 14336 x 4096  57.8 76.1 78.2 57.5   512 x 28672 x 8192   111  140  154  109
//   2048 x 28672 x 480   66.4 59.9 58.1 58.1   2048 x 28672 x 1920  124  138  137  121
//   256 x 8192 x 1024    17.6 12.9 9.6 9.5     2048 x 28672 x 8192  408  476  508  393
//   8192 rows, 8 experts of 14336 x 4096  458  535  552  453
//   8192 rows, 64 experts of 1536 x 2048  71.2 73.2 71.5 71.1
inline int wgs_of(int wide) { return wide == 128 ? 2 : 1; }  // workgroups a CU
inline double round_us(int wide, int high, double tiles, int cus, int steps) {
  const double f = std::min(tiles / (cus * wgs_of(wide)), 1.0);
  if (wide == 128) return steps * (f <= 0.5 ? 0.43 + 0.2 * f : 0.55 + 0.47 * f) + 5.0;
  return high == 256 ? steps * (0.85 + 0.62 * f) + 10.0 : steps * (0.48 + 0.5 * f) + 6.0;
}
inline double fold_us(int slices, int wide, int high) { return (wide == 128 ? 6.0 : 3.0) + slices * (wide * high) * 1e-6; }
inline int steps_of(int64_t k) { return (int)((k + kStepB - 1) / kStepB); }

// The tiles of a product, `high` rows each, and its time in us.  The last, partly
// filled round of tiles is cut along K where that is quicker.
inline TilePlan tiles_of(int wide, int high, int64_t m, int64_t n, int64_t k, int64_t experts, int cus, double& us) {
  TilePlan p = {};
  const int steps = steps_of(k), slots = cus * wgs_of(wide);
  p.cus = cus;
  p.wide = wide;
  p.high = high;
  p.nt = (int)((n + wide - 1) / wide);
  p.mt = (int)((m + high - 1) / high + std::min(experts, m));
  p.full = (int)std::min((int64_t)p.mt * p.nt, (int64_t)INT32_MAX);  // more have no memory for their results
  p.split = 1;
  auto rounds_us = [&](double tiles) {
    const double rounds = std::floor(tiles / slots), rest = tiles - rounds * slots;
    if (wide == 128 && rounds > 0)  // the tiles of a last round share CUs all the same; starts overlap with ends
      return std::ceil(tiles / slots) * (round_us(wide, high, slots, cus, steps) - 0.8);
    return rounds * round_us(wide, high, slots, cus, steps) + (rest > 0 ? round_us(wide, high, rest, cus, steps) : 0);
  };
  if (experts) {  // of about the same number of rows, whose last tile is half full
    const int64_t parts = std::min(experts, m);
    us = rounds_us((double)p.nt * std::max(parts, m / high + parts / 2));
    return p;
  }
  us = rounds_us(p.full);
  const int rest = p.full % slots;
  const double whole = rounds_us(p.full - rest);
  for (int s = 2; s <= 8 && rest > 0 && rest * s <= slots && s <= steps; s++) {
    const double t = whole + round_us(wide, high, rest * s, cus, (steps + s - 1) / s) + fold_us(rest * s, wide, high);
    if (t < us) us = t, p.split = s;
  }
  if (high == 256 && rest > 0 && rest * 2 <= cus) {
    const double t = whole + round_us(256, 128, rest * 2, cus, steps) + 6.0;
    if (t < us) us = t, p.split = 1, p.halves = rest;
  }
  if (p.split > 1) p.rest = rest, p.full -= rest;
  return p;
}
inline TilePlan tile_plan(int64_t m, int64_t n, int64_t k, int64_t experts, int cus, double& us) {
  double low_us, small_us;
  TilePlan p = tiles_of(256, 256, m, n, k, experts, cus, us);
  const TilePlan low = tiles_of(256, 128, m, n, k, experts, cus, low_us);
  const TilePlan small = tiles_of(128, 128, m, n, k, experts, cus, small_us);
  if (low_us < us + 1.0) us = low_us, p = low;  // the larger tile's results take longer to store
  if (small_us < 0.96 * us) us = small_us, p = small;
  return p;
}
inline size_t tile_ws_bytes(const TilePlan& p) { return (size_t)p.rest * p.split * p.wide * p.high * 4; }

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
// The stream kernel's work is its row tiles, whose sums meet in LDS, beside the read of W, and
// its job's X that it loads first; the tile kernel's its rounds, and half of the read shows.
// Measured, stream kernel and the best of the tiles:
//   64 x 4096 x 4096    14.6 and 17.1    512 x 4096 x 4096   23.0 and 20.2
//   64 x 14336 x 4096   21.0 and 20.6    128 x 14336 x 4096  22.1 and 21.0
//   27 x 28672 x 8192   51.3 and 60.5    64 x 28672 x 8192   58.4 and 62.0
//   64 x 8192 x 1024    9.6 and 8.4      256 x 8192 x 1024   15.9 and 9.5
//   100 x 2000 x 2000   7.3 and 10.7     64 x 2048 x 8192    14.5 and 17.4
//   8 experts of 14336 x 4096, 16 rows each 96 and 116, 64 rows 116 and 123, 128 rows 204 and 146
//   64 experts of 1536 x 2048, 8 rows each 37.0 and 47.9, 32 rows 53.6 and 52.6
// Few rows above K = 16384, which have the tile kernel alone, were not measured: how those
// are cut follows from the fits above.
struct Estimate {
  double stream, tile;
};
inline Estimate estimate(int64_t m, int64_t n, int64_t k, int64_t experts, const StreamPlan& p) {
  const int cus = p.cus;
  const int64_t parts = experts ? std::min(experts, m) : 1;  // W's used
  const double rows = (double)m / parts, read = (double)parts * n * k / 6.5e6;
  // jobs of each W: experts' rows scatter about the average
  const double jobs = experts ? std::max(rows / p.rows + 0.5, 1.0) : (double)((m + p.rows - 1) / p.rows);
  const double units = parts * jobs * (double)((n + kSRows * p.rt - 1) / (kSRows * p.rt));
  const double work = std::ceil(units / cus) * (0.22 * p.mt + 0.4 * p.ck);
  // an expert's jobs read its W one after the other, of which the caches hold a part; those
  // of one product side by side
  const double streamed = experts ? read * (1.0 + jobs) / 2 : read;
  double tile;
  tile_plan(m, n, k, experts, cus, tile);
  return {std::max(work, streamed) + 0.4 * std::min(work, streamed) + 3.5 + 0.75 * p.ck * p.mt, tile + 0.55 * read};
}
inline bool streams(int64_t m, int64_t n, int64_t k, int64_t experts, int cus, StreamPlan& p) {
  p = stream_plan(m, n, k, experts, cus);
  if (!p.ck) return false;
  const Estimate e = estimate(m, n, k, experts, p);
  return e.stream <= e.tile;
}

}  // namespace i8
}  // namespace rz
