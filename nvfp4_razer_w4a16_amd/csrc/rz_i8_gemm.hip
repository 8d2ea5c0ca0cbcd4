// rz_i8_gemm.hip -- products of 8-bit integer tensors on gfx950: y[M, N] = X W^T with
// a scale for each row of X and of W, and the same grouped by expert.
//
// The sums are exact: 32-bit integers hold K products of two 8-bit codes for K up to
// 131056.  W rows are the A operand of v_mfma_i32_32x32x32_i8, X rows the B operand, so
// a lane ends with four consecutive columns of y.  Both operands are read as they
// are stored, 16 bytes of a row a lane; the order of K within a product is free as long
// as both agree.
//
// Out of range: rows are clamped to the last one (their results are not stored); pieces
// past K read as zeros.
#include <algorithm>
#include <type_traits>
#include <utility>

#include "rz_groups.h"
#include "rz_i8.h"
#include "rz_i8_launch.h"
#include "rz_i8_plan.h"

namespace rz {

namespace {

using namespace i8;

struct Args {
  const int8_t *xc, *wc;
  const float *xs, *ws;
  int64_t m, n, k, x_rows_total;
  void* y;
  const int32_t* offsets;
  const int32_t* x_rows;
  int experts;
};

// Memory from p on of which loads past `bytes` read zero.
typedef __amdgpu_buffer_rsrc_t Rsrc;
__device__ __forceinline__ Rsrc rsrc_of(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)bytes, 0x00020000);
}
constexpr uint32_t kPast = 0xFFFFFFF0u;  // past all that a descriptor holds

// 16 bytes a lane straight to LDS, lane i's at l + 16 i.
__device__ __forceinline__ void load_lds16(Rsrc r, uint32_t offset, uint8_t* l) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)l, 16, (int)offset, 0, 0, 0);
}

// The operand of s_waitcnt for at most VM loads and stores, and LGKM LDS accesses, under
// way.  (The builtin, which the compiler counts with: after waits that it does not know of
// it puts its own, for all loads, ahead of a loop's first LDS read.)
constexpr int vm_lgkm(int vm, int lgkm) { return (vm & 15) | (vm & 48) << 10 | 0x70 | lgkm << 8; }

// The workgroup's barrier.
__device__ __forceinline__ void meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// f(0), f(1) .. as compile-time constants, until one of them is false.
template <typename F, int... I> __device__ __forceinline__ bool for_each(F& f, std::integer_sequence<int, I...>) {
  return (f(std::integral_constant<int, I>{}) && ...);
}

// Place of tile `pos`: bands of eight row tiles, within a band the row tiles of
// one column tile side by side, so that what runs at one time shares few rows of
// W and X.
__device__ __forceinline__ void tile_place(int pos, int mt, int nt, int& im, int& in) {
  const int band = pos / (8 * nt), at = pos - band * 8 * nt;
  const int high = min(8, mt - band * 8);
  in = at / high;
  im = band * 8 + at - in * high;
}

// ---- tile kernel -------------------------------------------------------------
// A BN x BM tile of y (256 rows of W by 256 or 128 of X, or 128 by 128) per workgroup of
// four waves (2x2), each wave (BN/2) x (BM/2) in 32x32 accumulators, 128 bytes of K a step.
// As many workgroups as CUs, or twice as many of 128 x 128; each walks through the tiles.
// The larger a tile, the less of what LDS delivers a product takes; the smaller, the fewer
// products it takes to fill the card, and two workgroups hide each other's results.
//
// LDS: a ring of two steps of W and of three of X (160 KiB for 256 x 256), filled by
// direct-to-LDS loads of whole 128-byte row pieces.  A piece is eight 16-byte chunks;
// chunk c of row r lies at place c ^ (r & 7) ^ (r >> 3 & 1), so that 16 lanes of a
// fragment read (one chunk of 16 rows) cover all banks.  Direct loads write lane-linear,
// so the loading lane picks its chunk by the same rule.  Lane half h takes chunk 4h + i
// at product i.
//
// Schedule of a step (products 0..3): the fragments of the next product are read under
// this one's.  Under product 0 the X rows of the step after next are requested, into the
// place of the step before.  The barrier sits before product 3, whose fragments are then
// in registers: behind it the next step is complete (each wave has waited for its own
// loads, but for the X rows just requested) and nobody reads this step any more, so the W
// rows of the step after next go into its place.  W has a whole step to arrive, X two.
// A load takes the CU's address unit 16 cycles and the four waves come at once, so loads
// stand behind every other product (one behind each: 2048 x 28672 x 8192 450 us, and 421).
//
// Measured: 8192 cubed 403-409 us (2.7 POP/s), 2048 x 28672 x 8192 390-400 us, of which
// the last half-filled round, in halves, takes 72-77; a loop of products in registers
// alone runs at 3.47 POP/s on random codes (4.93 on zeros), a library's product of the
// first size at 2.2.  Bound by power, then by its results: a step takes 1.46 us, 2.95 POP/s
// (on zeros, which power does not hold down, 0.98 us, 4.4), and between two tiles lie some
// 10 us, half of them the stores of 256 CUs at once.  The matrix units are busy 72 % of
// the time.  Tiles of 128 x 128: 1024 x 4096 x 4096 22 us (256 x 128: 27), 256 x 8192 x 1024
// 9.6 us (12.9); with two on a CU its LDS is busy all the time, 1.05 us a step.
template <int BN, int BM, typename OT, bool GROUPED>
__global__ __launch_bounds__(256, BN == 256 ? 1 : 2) void i8_tile_kernel(Args a, TilePlan plan) {
  constexpr int NI = BN / 64, MI = BM / 64;      // 32-row fragments of a wave
  constexpr int NL = BN / 32, ML = BM / 32;      // direct loads of a wave and step
  __shared__ __attribute__((aligned(16))) uint8_t w0[BN * kStepB], w1[BN * kStepB];
  __shared__ __attribute__((aligned(16))) uint8_t x0[BM * kStepB], x1[BM * kStepB], x2[BM * kStepB];
  // scales of the tile's columns and rows, and which rows are padding: behind the results' place in x2
  // where that is large enough (and all other LDS taken); in w1, which is then loaded behind the
  // results, where two workgroups share the LDS
  constexpr int kOut = 4 * 32 * 128, kScales = (BN + BM) * 4 + 32;
  constexpr bool kInW1 = BN == 128;
  __shared__ __attribute__((aligned(16))) uint8_t own[BM == 256 || kInW1 ? 16 : kScales];
  static_assert(BM != 256 || kOut + kScales <= BM * kStepB, "x2 holds both");
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, l32 = lane & 31;
  const int wn = (wave & 1) * (BN / 2), wm = (wave >> 1) * (BM / 2);
  const int all_nb = (int)(a.k / 16);            // 16-byte pieces of a row
  auto w_place = [&](auto p) -> uint8_t* {
    constexpr int i = decltype(p)::value % 2;
    return i == 0 ? w0 : w1;
  };
  auto x_place = [&](auto p) -> uint8_t* {
    constexpr int i = decltype(p)::value % 3;
    return i == 0 ? x0 : i == 1 ? x1 : x2;
  };

  const bool gather = GROUPED && a.x_rows;
  const RowTiles tiles = GROUPED ? row_tiles(a.offsets, a.experts, a.m, BM) : RowTiles{};
  const int mt = GROUPED ? tiles.count : plan.mt;
  const int full = GROUPED ? mt * plan.nt : plan.full;
  const int items = full + plan.rest * plan.split;
  // Consecutive workgroups go to the eight XCDs in turn: of every round of tiles
  // each XCD takes adjacent ones.
  const int grid = gridDim.x, b = blockIdx.x;
  const int place = (b % 8) * (grid / 8) + min(b % 8, grid % 8) + b / 8;
  const int chunk = (lane & 7) ^ (lane >> 3) ^ (wave & 1);

  // Where a tile is.
  struct Spot {
    Tile t;
    int64_t n0;
    int b0, nb, slot;  // first piece and pieces of its slice of K; slot of `part` or -1
    __device__ int x_last() const { return (int)max(t.m1 - t.m0, (int64_t)1) - 1; }
  };
  auto locate = [&](int item) {
    int im, in, pos = item;
    Spot o;
    o.b0 = 0;
    o.nb = all_nb;
    o.slot = -1;
    if (!GROUPED && item >= full) {
      o.slot = item - full;
      pos = full + o.slot / plan.split;
      const int s = o.slot % plan.split, steps = (all_nb + 7) / 8;
      o.b0 = steps * s / plan.split * 8;
      o.nb = min(steps * (s + 1) / plan.split * 8, all_nb) - o.b0;
    }
    if (!GROUPED && BM == 128 && plan.halves) {  // half `item % 2` of a tile of twice the height
      tile_place(plan.first + item / 2, mt, plan.nt, im, in);
      im = 2 * im + item % 2;
    } else {
      tile_place(pos, mt, plan.nt, im, in);
    }
    if (GROUPED)
      o.t = find_tile(tiles, a.offsets, a.experts, a.m, BM, im);
    else  // a half behind the last row has none: what is read for it is the last one
      o.t = Tile{min((int64_t)im * BM, a.m), min((int64_t)(im + 1) * BM, a.m), 0};
    o.n0 = (int64_t)in * BN;
    return o;
  };
  // The rows of X of this lane's direct loads, from the tile's first or as they are gathered,
  // and of the scale that it passes on.
  struct Rows {
    int x[ML], scale;
  };
  auto rows_of = [&](const Spot& o) {
    Rows r;
    const int last = o.x_last();
#pragma unroll
    for (int i = 0; i < ML; i++) r.x[i] = min((4 * i + wave) * 8 + (lane >> 3), last);
    r.scale = min(tid % BM, last);
    if (gather) {
      const int32_t* p = a.x_rows + o.t.m0;
#pragma unroll
      for (int i = 0; i < ML; i++) r.x[i] = p[r.x[i]];
      r.scale = p[r.scale];
    }
    return r;
  };
  // What the loads of the tile at hand go by.
  Rsrc wc, xc;
  int nb;
  uint32_t ow[NL], ox[ML];                       // direct load i of this lane: bytes from wc, xc
  float sw, sx;                                  // of the tile's column, and row, tid
  bool none;                                     // that row is padding
  auto aim = [&](const Spot& o, const Rows& r) {
    const int64_t wr = (int64_t)o.t.expert * a.n + o.n0;
    const int w_rows = (int)min((int64_t)BN, a.n - o.n0);
    const int64_t first = gather ? 0 : min(o.t.m0, a.m - 1), span = gather ? a.x_rows_total : o.x_last() + 1;
    nb = o.nb;
    wc = rsrc_of(a.wc + wr * a.k + o.b0 * 16, w_rows * a.k - o.b0 * 16);
    xc = rsrc_of(a.xc + first * a.k + o.b0 * 16, span * a.k - o.b0 * 16);
#pragma unroll
    for (int i = 0; i < NL; i++) ow[i] = (uint32_t)(min((4 * i + wave) * 8 + (lane >> 3), w_rows - 1) * a.k);
#pragma unroll
    for (int i = 0; i < ML; i++) ox[i] = (uint32_t)(min((int64_t)max(r.x[i], 0), span - 1) * a.k);
    none = r.scale < 0 || r.scale >= span;
    sw = a.ws[wr + min(tid % BN, w_rows - 1)];
    sx = a.xs[first + (none ? 0 : r.scale)];
  };
  auto load_w = [&](int s, uint8_t* l) {
    const int piece = s * 8 + chunk;
#pragma unroll
    for (int i = 0; i < NL; i++) load_lds16(wc, piece < nb ? ow[i] + piece * 16 : kPast, l + (4 * i + wave) * 1024);
  };
  auto load_x = [&](int s, uint8_t* l) {
    const int piece = s * 8 + chunk;
#pragma unroll
    for (int i = 0; i < ML; i++) load_lds16(xc, piece < nb ? ox[i] + piece * 16 : kPast, l + (4 * i + wave) * 1024);
  };

  struct Frags {
    i32x4_t w[NI], x[MI];
  };
  auto read_frags = [&](const uint8_t* lw, const uint8_t* lx, int i) {
    Frags f;
    const int at = l32 * kStepB + ((4 * half + i) ^ (l32 & 7) ^ ((l32 >> 3) & 1)) * 16;
#pragma unroll
    for (int j = 0; j < NI; j++) f.w[j] = *(const i32x4_t*)(lw + (wn + j * 32) * kStepB + at);
#pragma unroll
    for (int j = 0; j < MI; j++) f.x[j] = *(const i32x4_t*)(lx + (wm + j * 32) * kStepB + at);
    return f;
  };
  i32x16_t acc[NI][MI];
  auto first_products = [&](const Frags& f) {
#pragma unroll
    for (int i = 0; i < NI; i++)
#pragma unroll
      for (int j = 0; j < MI; j++)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.w[i], f.x[j], i32x16_t{}, 0, 0, 0);
  };
  auto products = [&](const Frags& f) {
#pragma unroll
    for (int i = 0; i < NI; i++)
#pragma unroll
      for (int j = 0; j < MI; j++)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.w[i], f.x[j], acc[i][j], 0, 0, 0);
  };
  // Keeps the products before it from moving past the branches behind them, where
  // their operands would have to wait in registers.
  auto pin = [&]() {
#pragma unroll
    for (int i = 0; i < NI; i++)
#pragma unroll
      for (int j = 0; j < MI; j++) asm volatile("" : "+a"(acc[i][j]));
  };
  // The instruction order asked for: LDS reads, then memory loads, one at a time
  // between the products.
  auto spread = [&](int reads, int loads) {
#pragma unroll
    for (int i = 0; i < NI * MI; i++) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (i < reads) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      if (BN == 128 ? i < loads : i % 2 && i / 2 < loads) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  int item = place;
  if (item >= items) return;
  Spot spot = locate(item);
  Rows rows_at = rows_of(spot);
  aim(spot, rows_at);
  load_x(0, x0);
  load_w(0, w0);
  load_x(1, x1);
  load_w(1, w1);
  while (true) {
    const int steps = (nb + 7) / 8;
    int s = 0;
    __builtin_amdgcn_s_waitcnt(vm_lgkm(NL + ML, 0));
    meet();
    Frags f = read_frags(w0, x0, 0), g;
    // Where the next tile is: its row numbers arrive under this one's steps.
    item += grid;
    const Spot next = locate(min(item, items - 1));
    const Rows next_rows = rows_of(next);
    // position P of the rings: products 0 to 2 of step s, and the fragments of product 3
    auto front = [&](auto which) {
      constexpr int P = decltype(which)::value;  // 0 for the tile's first step alone
      uint8_t *lw = w_place(which), *lx = x_place(which);
      g = read_frags(lw, lx, 1);
      load_x(s + 2, x_place(std::integral_constant<int, P + 2>{}));
      if constexpr (P == 0)
        first_products(f);
      else
        products(f);
      spread(NI + MI, ML);
      f = read_frags(lw, lx, 2);
      products(g);
      spread(NI + MI, 0);
      g = read_frags(lw, lx, 3);
      products(f);
      spread(NI + MI, 0);
      pin();
    };
    // product 3 of step s behind the barrier.  The loads run past the slice's end, where
    // they read nothing of use.
    auto back = [&](auto which) {
      constexpr int P = decltype(which)::value;
      typedef std::integral_constant<int, P + 1> Next;
      __builtin_amdgcn_s_waitcnt(vm_lgkm(ML, 0));
      meet();
      f = read_frags(w_place(Next{}), x_place(Next{}), 0);
      load_w(s + 2, w_place(which));
      products(g);
      spread(NI + MI, NL);
      pin();
      s++;
    };
    auto step = [&](auto which) {
      back(which);
      front(std::integral_constant<int, decltype(which)::value + 1>{});
      return true;
    };
    auto last_steps = [&](auto which) {
      back(which);
      if (s >= steps) return false;
      front(std::integral_constant<int, decltype(which)::value + 1>{});
      return true;
    };
    front(std::integral_constant<int, 0>{});
    // Whole turns of both rings, then one to six steps.  (With a way out behind every step the
    // compiler waits for all loads at the loop's start, whose LDS any of the ways may have
    // loaded last.)
    for (int turns = (steps - 1) / 6; turns > 0; turns--) for_each(step, std::make_integer_sequence<int, 6>{});
    for_each(last_steps, std::make_integer_sequence<int, 6>{});

    // ---- this tile's results, under which the next one's first steps are loaded
    const Spot done = spot;
    uint8_t* scl = BM == 256 ? x2 + kOut : kInW1 ? w1 : own;
    __builtin_amdgcn_s_waitcnt(vm_lgkm(0, 0));  // nothing of this tile is under way
    meet();                                     // or read any more
    if (BN == 256 || tid < BN) *(float*)(scl + tid * 4) = sw;
    if (BM == 256 || tid < BM) *(float*)(scl + (BN + tid) * 4) = sx;
    if (GROUPED) *(uint64_t*)(scl + (BN + BM) * 4 + wave * 8) = __ballot(none);
    if (item < items) {
      spot = next;
      aim(next, next_rows);
      load_x(0, x0);
      load_w(0, w0);
      load_x(1, x1);
      if (!kInW1) load_w(1, w1);
    }
    __builtin_amdgcn_s_waitcnt(vm_lgkm(63, 0));
    meet();
    __builtin_amdgcn_sched_barrier(0);
    // The accumulators are taken out of their registers where they are written, not
    // all at once, and the addresses are worked out here, not kept from before the
    // loop: either would spill.
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int half = lane >> 5, l32 = lane & 31;
    if (!GROUPED && done.slot >= 0) {  // a slice's sums, in the order of the registers
      i32x4_t* p = (i32x4_t*)(plan.part + (int64_t)done.slot * BM * BN) + wave * (NI * MI * 4 * 64) + lane;
#pragma unroll
      for (int i = 0; i < NI; i++)
#pragma unroll
        for (int j = 0; j < MI; j++)
#pragma unroll
          for (int q = 0; q < 4; q++) {
            i32x16_t& c = acc[i][j];
            if (q == 0) asm volatile("" : "+a"(c));
            p[((i * MI + j) * 4 + q) * 64] = i32x4_t{c[q * 4], c[q * 4 + 1], c[q * 4 + 2], c[q * 4 + 3]};
          }
    } else {
      // Through LDS, in the third place of the ring of X, to be stored in whole 128-byte lines.
      typedef OT V4 __attribute__((ext_vector_type(4)));
      constexpr int kCols = 128 / sizeof(OT), kPer = 16 / sizeof(OT), kFr = kCols / 32;  // columns of a pass, a store
      const int rows = (int)(done.t.m1 - done.t.m0), cols = (int)min(a.n - done.n0, (int64_t)BN);
      uint8_t* o = x2 + wave * (32 * 128);
      const int r0 = lane >> 3, c0 = (lane & 7) * kPer;  // of a store within its 8 rows
      OT* y = (OT*)a.y + (done.t.m0 + wm + r0) * a.n + done.n0 + wn + c0;
      const float* csw = (const float*)scl + wn + half * 4;
      constexpr int kPasses = MI * NI / kFr;  // 32 rows and kCols columns each
      V4 v[kFr * 4];
      f32x4_t s4[kFr * 4];                    // scales of a pass's columns, the same for the passes of all rows
      auto convert = [&](int pass) {
        const int j = pass % MI, p = pass / MI, m = wm + j * 32 + l32;  // this lane's row
        if (j == 0)
#pragma unroll
          for (int i = 0; i < kFr * 4; i++) s4[i] = *(const f32x4_t*)(csw + p * kCols + i * 8);
        const float rsx = *(const float*)(scl + (BN + m) * 4);
        const bool zero = GROUPED && (scl[(BN + BM) * 4 + (m >> 3)] >> (m & 7) & 1);
#pragma unroll
        for (int i = 0; i < kFr; i++)
#pragma unroll
          for (int q = 0; q < 4; q++) {
            i32x16_t& c = acc[p * kFr + i][j];
            if (q == 0) asm volatile("" : "+a"(c));
#pragma unroll
            for (int e = 0; e < 4; e++) v[i * 4 + q][e] = mx_cvt<OT>(i8_scaled(c[q * 4 + e], rsx, s4[i * 4 + q][e]));
            if (zero) v[i * 4 + q] = V4{};
          }
      };
      convert(0);
#pragma unroll
      for (int pass = 0; pass < kPasses; pass++) {
        const int j = pass % MI, p = pass / MI;
#pragma unroll
        for (int i = 0; i < kFr; i++)
#pragma unroll
          for (int q = 0; q < 4; q++) {
            const int byte = (i * 32 + q * 8 + half * 4) * (int)sizeof(OT);
            *(V4*)(o + l32 * 128 + (((byte >> 4) ^ (l32 & 7)) << 4) + (byte & 15)) = v[i * 4 + q];
          }
        wave_lds_sync();
        const int n = wn + p * kCols + c0;
        u32x4_t line[4];
#pragma unroll
        for (int s = 0; s < 4; s++) line[s] = *(const u32x4_t*)(o + (s * 8 + r0) * 128 + ((lane & 7) ^ r0) * 16);
        if (pass + 1 < kPasses) convert(pass + 1);
#pragma unroll
        for (int s = 0; s < 4; s++)
          if (wm + j * 32 + s * 8 + r0 < rows && n + kPer <= cols)
            __builtin_memcpy(y + (int64_t)(j * 32 + s * 8) * a.n + p * kCols, &line[s], 16);
        if (cols % kPer) {  // the columns of a width that ends inside a store
#pragma unroll 1
          for (int s = 0; s < 4; s++) {
            const OT* e = (const OT*)(o + (s * 8 + r0) * 128 + ((lane & 7) ^ r0) * 16);
            if (wm + j * 32 + s * 8 + r0 < rows && n < cols && n + kPer > cols)
#pragma unroll 1
              for (int i = 0; n + i < cols; i++) y[(int64_t)(j * 32 + s * 8) * a.n + p * kCols + i] = e[i];
          }
        }
        wave_lds_sync();
      }
    }
    if (item >= items) return;
    if (kInW1) {
      meet();  // nobody reads the scales any more
      load_w(1, w1);
    }
  }
}

// ---- stream kernel -------------------------------------------------------------
// For few rows of X the product is a read of W.  A workgroup of eight waves owns 16
// W rows at a time (a "row tile", one contiguous piece of memory) and all of K,
// which the waves share in units of 256 bytes; each keeps its share of up to 16 MT
// rows of X (a "job") in registers for all the row tiles that the workgroup walks
// through, so that nothing but W is read in the loop.  The row
// tiles of all jobs stand in one line that is cut between the workgroups, however
// the rows are spread over the experts; a piece that crosses jobs loads the next
// one's X on the way.
//
// A row tile comes in CK chunks of up to 2048 bytes of K, 32 KiB each, by
// direct-to-LDS loads into a ring of RING buffers, RING - 1 chunks ahead: memory is
// read in long runs whatever K is, and what is under way costs no registers.  A chunk's
// 16-byte pieces lie in LDS as in memory but for an exchange within a row, piece c of
// row r at c ^ (r & mask), which spreads the rows over the banks where the row's length
// would not.  Rows of at most 1024 or 512 bytes come RT = two or four row tiles a chunk,
// each of which has four or two of the waves to share its K.
//
// Of a wave's sixteen pieces, lane group g = lane / 16 takes piece 4 i + g at product i, so
// that a load of X covers 64 bytes of each of 16 rows.  Pieces past the
// row or the chunk are zeros in X, whatever W's fragment holds there.  The scales of a
// row tile come to LDS the same way as W.  The waves' sums meet in LDS.  Loads past the
// last row return zero (the buffer descriptor ends there), so no load has a branch
// around it and a chunk's loads have a fixed number.
//
// Bound by the read of W: 1 x 14336 x 4096 13.4-14.2 us (58.8 MB, 4.1-4.4 TB/s, the ramp of a
// launch in it), 27 x 28672 x 8192 50.7-51.7 us (237 MB, 4.6 TB/s), 8 tokens through 2 of 8
// experts of 14336 x 4096, seven of them used, 77-78 us (411 MB, 5.3 TB/s; a copy of 1 GiB
// reaches 5.1).
constexpr int kSWaves = 8, kSLoads = kSRows * kChunkB / 1024 / kSWaves;

// Ring places.
constexpr int stream_ring(int mt) { return mt == 4 ? 3 : 4; }

template <int RT, int CK, int MT, bool GROUPED>
__global__ __launch_bounds__(64 * kSWaves, 2) void i8_stream_kernel(Args a, int y_dtype, StreamPlan plan) {
  constexpr int kRing = stream_ring(MT);
  static_assert(RT == 1 || CK == 1, "chunks of several row tiles hold whole rows");
  // Of the waves of a row tile, kAlong share its K and kX the job's rows; a wave has
  // kUnits times 256 bytes of K and kMT times 16 rows.
  constexpr int kX = !GROUPED && CK == 1 && MT > 1 ? 2 : 1, kAlong = kSWaves / RT / kX, kUnits = kX, kMT = MT / kX;
  constexpr int kRows = kSRows * RT;         // rows of W in a chunk
  constexpr int kPart = kSRows * 16 * kMT;   // sums of one wave
  constexpr int kSums = kSRows * 16 * MT;    // results of a row tile
  constexpr int kOuts = (RT * kSums + 64 * kSWaves - 1) / (64 * kSWaves);  // of a thread in a chunk
  // A round is whole row tiles and whole turns of the ring, and an even number of tiles
  // where there are two sets of sums.
  constexpr int kRound = CK >= 4 ? 2 * CK : kRing % 2 ? 2 * kRing : kRing;
  static_assert(kRound % kRing == 0 && kRound % CK == 0, "whole turns, whole row tiles");
  constexpr int kAreas = CK == 1 ? kRing : kRound / CK;  // places of scales, in turn for the round's row tiles
  // Row tiles that the scales are requested ahead: enough that the loads of kRing - 2
  // chunks are behind them when they are needed, behind the next row tile's first barrier.
  constexpr int kScAhead = CK == 1 ? kRing - 2 : 0;
  static_assert(kAreas > kScAhead + 1, "of four areas one is read, and the others loaded");
  __shared__ __attribute__((aligned(16))) uint8_t r0[kSRows * kChunkB], r1[kSRows * kChunkB], r2[kSRows * kChunkB],
      r3[kRing > 3 ? kSRows * kChunkB : 16];
  __shared__ __attribute__((aligned(16))) float a0[kRows], a1[kRows], a2[kAreas > 2 ? kRows : 4], a3[kAreas > 3 ? kRows : 4];
  // The waves' sums of a row tile are added behind the next chunk's barrier, where there
  // is a second set of them or a barrier more before the next tile's are written.
  constexpr int kParts = CK == 1 && (MT == 1 || kX == 2) ? 2 : 1;
  constexpr bool kDefer = CK > 1 || kParts == 2;
  __shared__ __attribute__((aligned(16))) int part[kParts * kSWaves * kPart];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kb = (int)a.k, nb = kb / 16;
  const int units = (int)((a.n + kSRows - 1) / kSRows);  // what the line is cut into
  auto ring = [&](auto p) -> uint8_t* {
    constexpr int i = decltype(p)::value % kRing;
    return i == 0 ? r0 : i == 1 ? r1 : i == 2 ? r2 : r3;
  };
  auto area = [&](auto tile) -> float* {
    constexpr int i = decltype(tile)::value % kAreas;
    return i == 0 ? a0 : i == 1 ? a1 : i == 2 ? a2 : a3;
  };
  // exchange of a row's pieces: within aligned groups, at most 16, that divide the row
  auto key = [](int pieces, int r) { return r & (min(pieces & -pieces, 16) - 1); };
  auto quotient = [](int p, int mul) { return (int)(((uint32_t)p * (uint32_t)mul) >> 20); };
  // direct load i of this lane: bytes from the chunk's first one, or past every end
  uint32_t off[kSLoads], off_last[kSLoads];
#pragma unroll
  for (int i = 0; i < kSLoads; i++) {
    const int p = (i * kSWaves + wave) * 64 + lane;
    auto offset = [&](int pieces, int mul) {
      const int r = quotient(p, mul), c = p - r * pieces;
      return r < kRows ? (uint32_t)(r * kb + (c ^ key(pieces, r)) * 16) : 0x7FFFFFFFu;
    };
    off_last[i] = offset(plan.last, plan.mul_last);
    off[i] = CK > 1 ? offset(plan.pieces, plan.mul_pieces) : off_last[i];
  }

  // this workgroup's piece of the line
  const uint32_t b = blockIdx.x;
  Cuts c = plan.cuts;
  if (GROUPED) c = cuts_of((uint32_t)units, (uint32_t)live_tiles(a.offsets, a.experts, a.m, plan.rows), gridDim.x, RT);
  int job, unit, left;
  if (c.per_job) {
    job = GROUPED ? (int)(b / c.per_job) : quotient((int)b, plan.mul_per_job);
    const uint32_t cut = b - (uint32_t)job * c.per_job;
    unit = (int)(c.share * cut + min(cut, c.extra));
    left = job < (int)c.jobs ? (int)(c.share + (cut < c.extra ? 1 : 0)) : 0;
  } else {
    const uint32_t start = c.share * b + min(b, c.extra);
    job = (int)(start / (uint32_t)units);
    unit = (int)(start - (uint32_t)job * (uint32_t)units);
    left = (int)(c.share + (b < c.extra ? 1 : 0));
  }
  for (; left > 0; job++, unit = 0) {
    Tile t;
    if (GROUPED)
      t = find_tile(a.offsets, a.experts, a.m, plan.rows, job);
    else
      t = Tile{(int64_t)job * plan.rows, min((int64_t)(job + 1) * plan.rows, a.m), 0};
    if (GROUPED && t.expert < 0) return;
    // its rows of W in this job: n_rows from n0 on, in `end` chunks or times CK
    const int taken = min(left, units - unit), n0 = unit * kSRows;
    const int n_rows = (int)min((int64_t)taken * kSRows, a.n - n0), end = (n_rows + kRows - 1) / kRows;
    left -= taken;
    int tile = 0;
    const int8_t* wc = a.wc + ((int64_t)t.expert * a.n + n0) * kb;
    const float* wsc = a.ws + (int64_t)t.expert * a.n + n0;
    auto rows_of = [&](int tile) { return tile < end ? min(n_rows - tile * kRows, kRows) : 0; };
    auto load_chunk = [&](int tile, int ck, uint8_t* l) {
      const int col = ck * plan.pieces * 16;
      const Rsrc r = rsrc_of(wc + (int64_t)tile * kRows * kb + col, max(rows_of(tile) * kb - col, 0));
#pragma unroll
      for (int i = 0; i < kSLoads; i++)
        load_lds16(r, ck == CK - 1 ? off_last[i] : off[i], l + (i * kSWaves + wave) * 1024);
    };
    auto load_scales = [&](int tile, float* l) {
      const Rsrc r = rsrc_of(wsc + (int64_t)tile * kRows, rows_of(tile) * 4);
      if (tid < kRows)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)l, 4, tid * 4, 0, 0, 0);
    };
    __syncthreads();  // the job before still reads the ring
    if constexpr (kScAhead > 0) load_scales(tile, a0);
    load_chunk(tile, 0, r0);
    __builtin_amdgcn_sched_barrier(0);
    // this wave's share of X
    i32x4_t fx[kMT][CK][kUnits][4];
    const int along = wave % kAlong, x_row = wave / kAlong % kX * 16 * kMT;
#pragma unroll
    for (int j = 0; j < kMT; j++) {
      int64_t row = min(t.m0 + x_row + 16 * j + (lane & 15), t.m1 - 1);
      if (GROUPED && a.x_rows) row = min((int64_t)max(a.x_rows[row], 0), a.x_rows_total - 1);
      const int8_t* pc = a.xc + row * kb;
#pragma unroll
      for (int u = 0; u < CK; u++)
#pragma unroll
        for (int v = 0; v < kUnits; v++)
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const int at = 16 * (along + v * kAlong) + 4 * i + (lane >> 4);  // of the chunk's pieces
            fx[j][u][v][i] = *(const i32x4_t*)(pc + min(u * plan.pieces + at, nb - 1) * 16);
          }
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (kScAhead > 1) load_scales(tile + 1, a1);
    load_chunk(tile + 1 / CK, 1 % CK, r1);
    if constexpr (kRing > 3) load_chunk(tile + 2 / CK, 2 % CK, r2);
    // Where the operands lie: worked out while the first loads are under way, hence
    // from a lane number that the compiler cannot follow up to the kernel's start.
    int at_lane = lane;
    asm volatile("" : "+v"(at_lane));
    const int g = at_lane >> 4, w_row = wave / (kAlong * kX) * kSRows + (at_lane & 15), mine = 16 * along + g;
    // fragment i of W in a chunk; the next unit's lie kAlong * 256
    // bytes on, as the exchange is within 16 pieces
    int fo[4], fo_last[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int c = mine + 4 * i;
      auto offset = [&](int pieces) {  // past the row: some other codes
        return min(w_row * pieces + (c ^ key(pieces, w_row)), kSRows * kChunkB / 16 - 1 - 16 * kAlong * (kUnits - 1)) * 16;
      };
      fo_last[i] = offset(plan.last);
      fo[i] = CK > 1 ? offset(plan.pieces) : fo_last[i];
    }
    // pieces that the chunk does not have add nothing
#pragma unroll
    for (int j = 0; j < kMT; j++)
#pragma unroll
      for (int u = 0; u < CK; u++)
#pragma unroll
        for (int v = 0; v < kUnits; v++)
#pragma unroll
          for (int i = 0; i < 4; i++)
            if (mine + 16 * v * kAlong + 4 * i >= (u == CK - 1 ? plan.last : plan.pieces)) fx[j][u][v][i] = i32x4_t{};

    // this thread's results: the scale of their row, and rows that padding leaves zero
    bool none[kOuts];
    float sx[kOuts];
#pragma unroll
    for (int i = 0; i < kOuts; i++) {
      none[i] = false;
      int64_t row = min(t.m0 + ((tid + i * 64 * kSWaves) % kSums >> 4), t.m1 - 1);
      if (GROUPED && a.x_rows) {
        row = a.x_rows[row];
        none[i] = row < 0 || row >= a.x_rows_total;
        if (none[i]) row = 0;
      }
      sx[i] = a.xs[row];
    }
    // y of a row tile, from set `set` of the waves' sums
    auto finish = [&](int tile, int set, const float* sw) {
#pragma unroll
      for (int i = 0; i < kOuts; i++) {
        const int o = tid + i * 64 * kSWaves;
        const int n = o & 15, m = (RT == 1 ? o : o % kSums) >> 4, at_tile = RT == 1 ? 0 : o / kSums;
        const int m_x = kX == 1 ? m : m % (16 * kMT);
        const int64_t row = t.m0 + m;
        const int col = tile * kRows + at_tile * kSRows + n;
        if (o >= RT * kSums || row >= t.m1 || col >= n_rows) continue;
        // lane (n / 4) * 16 + m % 16 of a wave holds it in element n % 4
        const int* p = part + ((set * RT + at_tile) * kX + (kX == 1 ? 0 : m / (16 * kMT))) * kAlong * kPart + (m_x >> 4) * 256 +
                       ((n >> 2) * 16 + (m_x & 15)) * 4 + (n & 3);
        int v[kAlong];
#pragma unroll
        for (int w = 0; w < kAlong; w++) v[w] = p[w * kPart];
        int sum = 0;
#pragma unroll
        for (int w = 0; w < kAlong; w++) sum += v[w];
        float r = i8_scaled(sum, sx[i], sw[at_tile * kSRows + n]);
        if (none[i]) r = 0.0f;
        const int64_t at = row * a.n + n0 + col;
        if (y_dtype == kF32) ((float*)a.y)[at] = r;
        else if (y_dtype == kF16) ((_Float16*)a.y)[at] = mx_cvt<_Float16>(r);
        else ((__bf16*)a.y)[at] = mx_cvt<__bf16>(r);
      }
    };
    auto meet_lds = [&]() {  // once this wave's LDS accesses are done
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      meet();
    };
    i32x4_t acc[kMT];
    // position P of a round: chunk P % CK of the row tile, ring place P % kRing;
    // false behind the last row tile
    auto chunk = [&](auto which) {
      constexpr int P = decltype(which)::value, ck = P % CK, ahead = ck + kRing - 1;
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kSLoads*(kRing - 2)) : "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      if constexpr (ck == 0) {
        load_scales(tile + kScAhead, area(std::integral_constant<int, P / CK + kScAhead>{}));
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < kMT; j++) acc[j] = i32x4_t{0, 0, 0, 0};
      }
      load_chunk(tile + ahead / CK, ahead % CK, ring(std::integral_constant<int, P + kRing - 1>{}));
      const uint8_t* l = ring(which);
      auto unit_of = [&](auto which_unit) {
        constexpr int v = decltype(which_unit)::value;
        if (v > 0 && 16 * (along + v * kAlong) >= plan.last) return false;  // the row ends before it
        i32x4_t f[4];
#pragma unroll
        for (int i = 0; i < 4; i++) f[i] = *(const i32x4_t*)(l + (ck == CK - 1 ? fo_last[i] : fo[i]) + v * kAlong * 256);
#pragma unroll
        for (int j = 0; j < kMT; j++) {
#pragma unroll
          for (int i = 0; i < 4; i++)
            acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f[i], fx[j][ck][v][i], acc[j], 0, 0, 0);
          asm volatile("" : "+v"(acc[j]));  // here, not behind the next barrier with all chunks' operands
        }
        return true;
      };
      for_each(unit_of, std::make_integer_sequence<int, kUnits>{});
      if constexpr (kDefer && ck == 0)
        if (tile > 0)
          finish(tile - 1, (P / CK + kParts - 1) % kParts, area(std::integral_constant<int, P / CK + kAreas - 1>{}));
      if constexpr (ck == CK - 1) {
        int* sums = part + (P / CK % kParts * kSWaves + wave) * kPart;
#pragma unroll
        for (int j = 0; j < kMT; j++) *(i32x4_t*)(sums + j * 256 + lane * 4) = acc[j];
        if constexpr (!kDefer) {
          meet_lds();
          finish(tile, 0, area(std::integral_constant<int, P / CK>{}));
        }
        return ++tile < end;
      }
      return true;
    };
    while (for_each(chunk, std::make_integer_sequence<int, kRound>{})) {
    }
    if constexpr (kDefer) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      meet_lds();
      const int last = (end - 1) % kAreas;
      finish(end - 1, (end - 1) % kParts, last == 0 ? a0 : last == 1 ? a1 : last == 2 ? a2 : a3);
    }
  }
}

template <int RT, int CK, int MT> hipError_t go_stream(const Args& a, int y_dtype, StreamPlan p, hipStream_t stream) {
  const int64_t tiles = (a.n + kSRows - 1) / kSRows, full = (a.m + p.rows - 1) / p.rows;
  const int64_t jobs = a.offsets ? std::min(full + a.experts, a.m) : full;
  const int64_t grid = std::min(tiles * jobs, (int64_t)p.cus);  // the ring fills a CU
  if (!a.offsets) {
    p.cuts = cuts_of((uint32_t)tiles, (uint32_t)jobs, (uint32_t)grid, RT);
    if (p.cuts.per_job) p.mul_per_job = (1 << 20) / (int)p.cuts.per_job + 1;
  }
  const dim3 blocks((unsigned)grid), threads(64 * kSWaves);
  if (a.offsets) hipLaunchKernelGGL((i8_stream_kernel<RT, CK, MT, true>), blocks, threads, 0, stream, a, y_dtype, p);
  else hipLaunchKernelGGL((i8_stream_kernel<RT, CK, MT, false>), blocks, threads, 0, stream, a, y_dtype, p);
  return hipGetLastError();
}

hipError_t run_stream(const Args& a, int y_dtype, const StreamPlan& p, hipStream_t s) {
  if (p.rt == 4) return p.mt == 1 ? go_stream<4, 1, 1>(a, y_dtype, p, s) : go_stream<4, 1, 2>(a, y_dtype, p, s);
  if (p.rt == 2) return p.mt == 1 ? go_stream<2, 1, 1>(a, y_dtype, p, s) : go_stream<2, 1, 2>(a, y_dtype, p, s);
  switch (p.mt * 16 + p.ck) {
    case 17: return go_stream<1, 1, 1>(a, y_dtype, p, s);
    case 18: return go_stream<1, 2, 1>(a, y_dtype, p, s);
    case 20: return go_stream<1, 4, 1>(a, y_dtype, p, s);
    case 24: return go_stream<1, 8, 1>(a, y_dtype, p, s);
    case 33: return go_stream<1, 1, 2>(a, y_dtype, p, s);
    case 34: return go_stream<1, 2, 2>(a, y_dtype, p, s);
    case 36: return go_stream<1, 4, 2>(a, y_dtype, p, s);
    case 65: return go_stream<1, 1, 4>(a, y_dtype, p, s);
    default: return go_stream<1, 2, 4>(a, y_dtype, p, s);
  }
}

// y of the split tiles: adds the slices' sums.  A thread takes 16 sums of one fragment
// in register order; the half-waves swap so that each lane stores runs of eight columns.
template <int BN, int BM, typename OT>
__global__ __launch_bounds__(256) void i8_fold_kernel(Args a, TilePlan plan) {
  constexpr int NI = BN / 64, MI = BM / 64;
  typedef OT V8 __attribute__((ext_vector_type(8)));
  const int lane = threadIdx.x & 63, half = lane >> 5, l32 = lane & 31;
  const int piece = blockIdx.x * 4 + (threadIdx.x >> 6);  // fragment of a tile
  const int tile = piece / (4 * NI * MI), frag = piece % (4 * NI * MI);
  const int wave = frag / (NI * MI), i = frag % (NI * MI) / MI, j = frag % MI;
  int im, in;
  tile_place(plan.full + tile, plan.mt, plan.nt, im, in);
  i32x4_t v[4] = {};
  const i32x4_t* p = (const i32x4_t*)plan.part + ((int64_t)tile * plan.split * 4 * NI * MI + frag) * 256 + lane;
  for (int s = 0; s < plan.split; s++, p += 4 * NI * MI * 256)
#pragma unroll
    for (int q = 0; q < 4; q++) v[q] += p[q * 64];
  const int64_t row = (int64_t)im * BM + (wave >> 1) * (BM / 2) + j * 32 + l32;
  const float sx = a.xs[min(row, a.m - 1)];
#pragma unroll
  for (int q = 0; q < 4; q += 2) {
    // of columns 8 q .. 8 q + 15 the lower half-wave stores the first eight, the upper the others
    i32x4_t other;
#pragma unroll
    for (int e = 0; e < 4; e++) other[e] = __shfl_xor(half ? v[q][e] : v[q + 1][e], 32, 64);
    const i32x4_t lo = half ? other : v[q], hi = half ? v[q + 1] : other;
    const int64_t n = (int64_t)in * BN + (wave & 1) * (BN / 2) + i * 32 + (q + half) * 8;
    if (row >= a.m || n >= a.n) continue;
    OT* y = (OT*)a.y + row * a.n + n;
    V8 o;
#pragma unroll
    for (int e = 0; e < 8; e++) o[e] = mx_cvt<OT>(i8_scaled(e < 4 ? lo[e] : hi[e - 4], sx, a.ws[min(n + e, a.n - 1)]));
    if (n + 8 <= a.n) {
      __builtin_memcpy(y, &o, sizeof(o));
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (n + e < a.n) y[e] = o[e];
    }
  }
}

template <int BN, int BM, typename OT, bool GROUPED> hipError_t go_tiles(const Args& a, const TilePlan& p, hipStream_t stream) {
  const int grid = std::min(p.full + p.rest * p.split, p.cus * wgs_of(BN));
  hipLaunchKernelGGL((i8_tile_kernel<BN, BM, OT, GROUPED>), dim3((unsigned)grid), dim3(256), 0, stream, a, p);
  return hipGetLastError();
}
template <typename OT, bool GROUPED> hipError_t any_tiles(const Args& a, const TilePlan& p, hipStream_t stream) {
  if (p.wide == 128) return go_tiles<128, 128, OT, GROUPED>(a, p, stream);
  return p.high == 256 ? go_tiles<256, 256, OT, GROUPED>(a, p, stream) : go_tiles<256, 128, OT, GROUPED>(a, p, stream);
}

template <int BN, int BM, typename OT> hipError_t go_fold(const Args& a, const TilePlan& p, hipStream_t stream) {
  hipLaunchKernelGGL((i8_fold_kernel<BN, BM, OT>), dim3((unsigned)(p.rest * (BN / 64) * (BM / 64))), dim3(256), 0, stream,
                     a, p);
  return hipGetLastError();
}

template <typename OT> hipError_t run(const Args& a, int cus, void* ws, hipStream_t stream) {
  double us;
  TilePlan p = tile_plan(a.m, a.n, a.k, a.offsets ? a.experts : 0, cus, us);
  p.part = (int32_t*)ws;
  if (a.offsets) return any_tiles<OT, true>(a, p, stream);
  TilePlan halves = p;
  if (p.halves) {  // the tiles of whole rounds, then the rest in halves
    halves.first = p.full - p.halves;
    halves.full = 2 * p.halves;
    p.full -= p.halves;
    p.halves = 0;
  }
  hipError_t e = hipSuccess;
  if (p.full + p.rest > 0) e = any_tiles<OT, false>(a, p, stream);
  if (e == hipSuccess && halves.halves) return go_tiles<256, 128, OT, false>(a, halves, stream);
  if (e != hipSuccess || !p.rest) return e;
  if (p.wide == 128) return go_fold<128, 128, OT>(a, p, stream);
  return p.high == 256 ? go_fold<256, 256, OT>(a, p, stream) : go_fold<256, 128, OT>(a, p, stream);
}

}  // namespace

size_t i8_gemm_ws_bytes(int64_t m, int64_t n, int64_t k, int64_t experts) {
  const int cus = device_cu_count();
  i8::StreamPlan p;
  double us;
  return i8::streams(m, n, k, experts, cus, p) ? 0 : i8::tile_ws_bytes(i8::tile_plan(m, n, k, experts, cus, us));
}

hipError_t launch_i8_gemm(const I8Gemm& g, void* ws, hipStream_t stream) {
  const Args a = {g.x.codes, g.w.codes, g.x.scales, g.w.scales, g.m, g.n, g.k, g.x.rows, g.y, g.offsets, g.x_rows,
                  g.experts};
  const int cus = device_cu_count();
  i8::StreamPlan p;
  if (i8::streams(g.m, g.n, g.k, g.offsets ? g.experts : 0, cus, p)) return run_stream(a, g.y_dtype, p, stream);
  if (g.y_dtype == kF32) return run<float>(a, cus, ws, stream);
  if (g.y_dtype == kF16) return run<_Float16>(a, cus, ws, stream);
  return run<__bf16>(a, cus, ws, stream);
}

}  // namespace rz
