// rz_mx_plan.h -- which kernel a product of MXFP4 tensors runs on, and how it is cut:
// rules on sizes and the device's compute units.  Host code, but for cuts_of.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "rz_mx_launch.h"

namespace rz {

// ---- tile kernel -------------------------------------------------------------
constexpr int kTileN = 256;       // rows of W of a tile
constexpr int kWindow = 16;       // blocks of a window
constexpr int kWindowK = kWindow * 32;

// How a product is cut: mt x nt tiles (grouped: as many row tiles as there are),
// the last `rest` of them each in `split` slices of K whose fp32 sums go to slots
// of `part`.
struct TilePlan {
  int high;  // rows of X of a tile
  int mt, nt;
  int full, rest, split;
  float* part;
};

// us that a window of a tile of 256 or 128 rows takes in a full round, and in one that
// leaves CUs (and power) to spare; what slices cost, their sums written and read.
// Measured, 256 rows, 256 with K cut, 128 rows, 128 with K cut:
//   2048 x 28672 x 8192  262 272 325    -      1024 x 4096 x 14336  81.3 52.5 64.2 48.7
//   2048 x 4096 x 14336 82.7 78.3  74.3 -      1024 x 4096 x 4096   29.0  -   22.7  -
//   512 x 14336 x 4096  29.8   -   24.4 -      1024 x 14336 x 4096  35.7  -   44.2  -
//   64 experts of 1536 x 2048, 64 rows each 44.3 and (128) 38.4, 128 rows 48.3 and 52.8
inline double window_us(int high, bool full) { return high == 256 ? full ? 3.75 : 3.0 : full ? 2.5 : 2.2; }
inline double fold_us(int slices, int high) { return 4.0 + slices * high * (0.1 / 256); }
inline int windows_of(int64_t k) { return (int)((k + kWindowK - 1) / kWindowK); }

// The tiles of a product, `high` rows each, and its time in us.  The last, partly
// filled round of tiles is cut along K where that is quicker.
inline TilePlan tiles_of(int high, int64_t m, int64_t n, int64_t k, int64_t experts, double& us) {
  TilePlan p = {};
  const int cus = device_cu_count(), windows = windows_of(k);
  p.high = high;
  p.nt = (int)((n + kTileN - 1) / kTileN);
  p.mt = (int)((m + high - 1) / high + std::min(experts, m));
  p.full = (int)std::min((int64_t)p.mt * p.nt, (int64_t)INT32_MAX);  // more have no memory for their results
  p.split = 1;
  if (experts) {  // of about the same number of rows, whose last tile is half full
    const int64_t parts = std::min(experts, m);
    const double tiles = (double)p.nt * std::max(parts, m / high + parts / 2), rounds = std::floor(tiles / cus);
    us = (rounds * window_us(high, true) + (tiles > rounds * cus ? window_us(high, false) : 0)) * windows;
    return p;
  }
  const int rest = p.full % cus;
  double best = rest ? windows * window_us(high, false) : 0;
  for (int s = 2; s <= 8 && rest > 0 && rest * s <= cus && s <= windows; s++) {
    const double t = (windows + s - 1) / s * window_us(high, false) + fold_us(rest * s, high);
    if (t < best) best = t, p.split = s;
  }
  us = p.full / cus * window_us(high, true) * windows + best;
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
// so, every job into `per_job` pieces.  (64 experts of 1503 x 2080, 1000 rows: 32.0 us
// with pieces that cross jobs, 28.9 without.)
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
  int sc_pieces, mul_sc;     // 16-byte pieces of a row's scale bytes, 0 where they are not whole
  Cuts cuts;                 // of a product without experts
  int mul_per_job;
};

// Blocks of K that a row tile's scale area holds.
constexpr int stream_blocks(int ck) { return ck == 4 ? 480 : 128 * ck; }

// The stream kernel's shape for `m` rows, of each of `experts` on average if that is not 0.
inline StreamPlan stream_plan(int64_t m, int64_t n, int64_t k, int64_t experts) {
  StreamPlan p = {};
  const int64_t kb = k / 2;
  int ck = 1;
  while ((int64_t)ck * kChunkB < kb) ck *= 2;
  // Above 15360 elements a row's scale bytes would not fit LDS: the tile kernel takes such
  // products, cut along K where they have no experts (1 x 8192 x 15360 12.9 us, x 16384
  // 27.7, x 28672 40.2; 16 rows through 8 experts of 4096 x 14336 48.8, x 16384 100).
  if (ck > 4 || kb / 16 > stream_blocks(ck)) return p;
  // rows a job: X of CK chunks has to fit the registers; experts' rows scatter about the average
  const int64_t rows = experts ? (m + experts - 1) / experts * 3 / 2 : m;
  const int most = std::min(4, 8 / ck);
  p.mt = std::min(rows <= 16 ? 1 : rows <= 32 ? 2 : 4, most);
  p.rows = 16 * p.mt;
  if (!experts && m > p.rows) {
    // A power of two of jobs: workgroups that walk through the same piece of W are then
    // on one XCD and share its L2 (192 x 28672 x 8192 as three jobs 76 us, as four 61).
    int64_t jobs = 1;
    while (jobs < 32 && jobs * p.rows < m) jobs *= 2;
    if (jobs * p.rows >= m) p.rows = (int)((m + jobs - 1) / jobs);
  }
  p.ck = ck;
  // Short rows: several row tiles a chunk, if there is a chunk for every CU.  Not for
  // jobs of 64 rows, where the sums of a chunk take as long as two smaller ones' (64 x
  // 28672 x 2048: 15.2 us and, one row tile a chunk, 14.1).
  const int64_t jobs = experts ? std::min(experts, m) : (m + p.rows - 1) / p.rows;
  p.rt = p.mt == 4 ? 1 : kb <= kChunkB / 4 ? 4 : kb <= kChunkB / 2 ? 2 : 1;
  while (p.rt > 1 && jobs * ((n + kSRows * p.rt - 1) / (kSRows * p.rt)) < device_cu_count()) p.rt /= 2;
  p.pieces = (int)(((kb + ck - 1) / ck + 63) / 64 * 4);  // whole products' blocks
  p.last = (int)(kb / 16) - p.pieces * (ck - 1);
  p.mul_pieces = (1 << 20) / p.pieces + 1;
  p.mul_last = (1 << 20) / p.last + 1;
  const int nb = (int)(kb / 16);
  if (nb % 16 == 0) p.sc_pieces = nb / 16, p.mul_sc = (1 << 20) / p.sc_pieces + 1;
  return p;
}

// Whether a product runs on the stream kernel: K below a window of the tile kernel, which
// reads scale bytes a window at a time, whatever M is (2048 x 28672 x 480 215 us, x 512 on
// tiles 44.5; 256 x 14336 x 480 17.9, x 512 7.9), or the shorter time of two estimates, in
// us.  Both take what the kernel's own work and
// the read of W come to, one of them half hidden behind the other, and what a launch
// costs.  The stream kernel's work is its row tiles, whose sums meet in LDS; the tile
// kernel's its rounds of tiles.  Whole us are compared: of 24 products that fractions
// would move to the tile kernel 23 are slower there (7.2-9.7 us, and 8.5-10.9).
// Measured, stream and tile kernel:
//   128 x 28672 x 8192  40.5 and 47.1    256 x 28672 x 8192   60.0 and 54.3
//   128 x 14336 x 4096  16.0 and 22.6    256 x 14336 x 4096   22.6 and 22.9
//   512 x 4096 x 4096   16.0 and 22.1    1024 x 4096 x 4096   24.5 and 22.7
//   33 x 8192 x 1024     7.1 and  8.0    128 x 8192 x 1024    10.3 and  8.5
//   256 x 4096 x 14336  26.3 and 25.2    1024 x 4096 x 14336  66.2 and 48.6
//   8 experts of 14336 x 4096, 64 rows each 72.7 and 69.8, 128 rows 115 and 85
// One of them is misjudged: 256 x 4096 x 14336 streams.
inline bool streams(int64_t m, int64_t n, int64_t k, int64_t experts, StreamPlan& p) {
  p = stream_plan(m, n, k, experts);
  if (!p.ck) return false;
  const int cus = device_cu_count();
  if (k < kWindowK) return true;
  const int64_t parts = experts ? std::min(experts, m) : 1, rows = (m + parts - 1) / parts;  // W's used, rows each
  auto whole = [](double us) { return (int)std::min(us, 1e9); };
  const int read = whole((double)parts * n * (k / 2 + k / 32) / 5e6);
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

}  // namespace rz
