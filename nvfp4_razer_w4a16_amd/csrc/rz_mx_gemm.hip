// rz_mx_gemm.hip -- products of MXFP4 tensors on gfx950: y[M, N] = X W^T, and
// the same grouped by expert.
//
// The matrix units take both operands as they are stored: 32 FP4 codes a lane
// and one scale byte for them (v_mfma_scale_f32_32x32x64_f8f6f4), accumulating
// in fp32.  The order of K within a product is free as long as both operands
// agree, so lane half h of MFMA i takes block 4h + i of a 256-element step: the
// four scale bytes a lane needs for one row are then one dword, and the MFMA
// picks the byte.  W rows are the A operand, X rows the B operand, so a lane
// ends with four consecutive columns of y.
//
// Out of range: rows are clamped to the last one (their results are not
// stored).  Blocks past K are read from the last block and get scale byte 0 on
// both sides: every FP4 code is finite, so they add at most 36 * 2^-254 = 0.
#include <algorithm>
#include <type_traits>
#include <utility>

#include "rz_mx.h"
#include "rz_mx_launch.h"
#include "rz_mx_plan.h"

namespace rz {

namespace {

struct Args {
  const uint8_t *xc, *xs, *wc, *ws;
  int64_t m, n, k, x_rows_total;
  void* y;
  const int32_t* offsets;
  const int32_t* x_rows;
  int experts;
};

// The rows [m0, m1) of one expert's tile.
struct Tile {
  int64_t m0, m1;
  int expert;  // -1: no such tile
};

// Tile t of the grouped product's row tiles, each `rows` high and within one
// expert's run.  Every wave works it out for itself: lane l counts the tiles of
// expert l and a running sum over the lanes finds the one that holds t.
// Offsets outside [0, m] are clamped.
__device__ __forceinline__ Tile find_tile(const Args& a, int rows, int64_t t) {
  const int lane = threadIdx.x & 63;
  const int m = (int)a.m;
  int before = 0;
  for (int e0 = 0; e0 < a.experts; e0 += 64) {
    const int e = e0 + lane;
    int lo = 0, hi = 0;
    if (e < a.experts) {
      lo = min(max(a.offsets[e], 0), m);
      hi = min(max(a.offsets[e + 1], lo), m);
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
__device__ __forceinline__ int live_tiles(const Args& a, int rows) {
  const int lane = threadIdx.x & 63, m = (int)a.m;
  int cnt = 0;
  for (int e = lane; e < a.experts; e += 64) {
    const int lo = min(max(a.offsets[e], 0), m), hi = min(max(a.offsets[e + 1], lo), m);
    cnt += (hi - lo + rows - 1) / rows;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) cnt += __shfl_xor(cnt, o, 64);
  return __builtin_amdgcn_readfirstlane(cnt);
}

// The scale bytes of blocks b .. b + 3 of a row of nb blocks, 0 past its end.
__device__ __forceinline__ uint32_t scales4(const uint8_t* row, int b, int nb) {
  uint32_t v = 0;
  if (b + 4 <= nb) {
    __builtin_memcpy(&v, row + b, 4);
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (b + i < nb) v |= (uint32_t)row[b + i] << (8 * i);
  }
  return v;
}

__device__ __forceinline__ i32x8_t frag(u32x4_t v) {
  return i32x8_t{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

// One MFMA of a step: byte i of both scale dwords.
template <int I> __device__ __forceinline__ f32x16_t mma(u32x4_t a, u32x4_t b, f32x16_t c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(frag(a), frag(b), c, 4, 4, I, (int)sa, I, (int)sb);
}

// Memory from p on of which loads past `bytes` read zero.
typedef __amdgpu_buffer_rsrc_t Rsrc;
__device__ __forceinline__ Rsrc rsrc_of(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)bytes, 0x00020000);
}

// ---- tile kernel -------------------------------------------------------------
// A kTileN x BM tile of y (256 rows of W, BM = 256 or 128 of X) per workgroup of four
// waves (2x2), each wave (BN/2) x (BM/2) in 32x32 accumulators, 256 elements of K a step; two
// steps are a "window", whose scale bytes are 16 bytes a row.  As many workgroups
// as CUs; each walks through the tiles.
//
// LDS: two steps' codes, filled by direct-to-LDS loads of whole 128-byte row
// pieces (64-byte pieces, four of them in flight, took 1.7 times as long: a line
// is fetched whole and gone before its other half is asked for).  A piece is eight
// 16-byte chunks; chunk c of row r lies at place c ^ (r & 7) ^ (r >> 3 & 1), so
// that 16 lanes of a fragment read (one chunk of 16 rows) cover all banks.  Direct
// loads write lane-linear, so the loading lane picks its chunk by the same rule.  Lane half h
// takes chunk 4h + i at product i; scale bytes pass through registers, a window
// ahead.
//
// Schedule of a step (products 0..3): the fragments of the next product are read
// under this one's.  The barrier sits before the last product, whose fragments are
// then in registers: behind it the next step is complete (each wave has waited for
// its own loads) and nobody reads this one any more, so the step after next is
// loaded in its place, half of it under the last product and half under the next
// step's first (a load takes the CU's address unit 16 cycles; all 64 under one
// product, 512 cycles, would stall it).  The loads run on into the next tile, so
// they are under way while this tile's results go through LDS to be stored in whole
// 128-byte lines.
//
// Measured: 2048 x 28672 x 8192 in bf16 262-277 us (3.5-3.7 PFLOP/s, the last of its
// rounds half full), 8192 cubed 4.0-4.4 PFLOP/s; a loop of products in registers alone
// runs at 6.2-6.7 (random codes).  Bound by its schedule, then by power: on zeros,
// which power does not hold down, it reaches 5.0-5.4 and that loop 9.7, and the matrix
// units are busy 62 % of the time.  Half of a step's loads go out under its first
// product and have the next two, some 0.7 us, to arrive; one wave a SIMD has nothing
// else to run while it waits for them.
constexpr int kStepB = 128;   // code bytes of a row and step

// 16 bytes a lane straight to LDS, lane i's at l + 16 i.  (The buffer form: behind
// the global one the compiler waits for every load under way.)
__device__ __forceinline__ void load_lds16(Rsrc r, uint32_t offset, uint8_t* l) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)l, 16, (int)offset, 0, 0, 0);
}

// The workgroup's barrier, once this wave's loads have arrived.
__device__ __forceinline__ void wait_and_meet() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
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

template <int BM, typename OT, bool GROUPED>
__global__ __launch_bounds__(256, 1) void mx_tile_kernel(Args a, TilePlan plan) {
  constexpr int BN = kTileN;
  constexpr int NI = BN / 64, MI = BM / 64;      // 32-row fragments of a wave
  constexpr int NL = BN / 32, ML = BM / 32;      // direct loads of a wave and step
  __shared__ __attribute__((aligned(16))) uint8_t s0[(BN + BM) * kStepB], s1[(BN + BM) * kStepB];
  __shared__ __attribute__((aligned(16))) uint8_t scl[(BN + BM) * kWindow];
  __shared__ __attribute__((aligned(16))) uint8_t out[4 * 32 * 128];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, l32 = lane & 31;
  const int wn = (wave & 1) * (BN / 2), wm = (wave >> 1) * (BM / 2);
  const int all_nb = (int)(a.k / kMxBlock);
  const int64_t kb = a.k / 2;

  // ---- the tile at hand
  int64_t n0;
  Tile t;
  int b0, nb, slot;                              // first block and blocks of its slice of K; slot of `part` or -1
  Rsrc wc, xc;
  const uint8_t *psw, *psx;
  uint32_t ow[NL], ox[ML];                       // direct load i of this lane: bytes from wc, xc
  const int mt = GROUPED ? live_tiles(a, BM) : plan.mt;
  const int full = GROUPED ? mt * plan.nt : plan.full;
  const int items = full + plan.rest * plan.split;
  // Consecutive workgroups go to the eight XCDs in turn: of every round of tiles
  // each XCD takes adjacent ones.
  const int grid = gridDim.x, b = blockIdx.x;
  const int place = (b % 8) * (grid / 8) + min(b % 8, grid % 8) + b / 8;
  const int chunk = (lane & 7) ^ (lane >> 3) ^ (wave & 1);
  auto set_tile = [&](int item) {
    int im, in, pos = item;
    b0 = 0;
    nb = all_nb;
    slot = -1;
    if (!GROUPED && item >= full) {
      slot = item - full;
      pos = full + slot / plan.split;
      const int s = slot % plan.split, windows = (all_nb + kWindow - 1) / kWindow;
      b0 = windows * s / plan.split * kWindow;
      nb = min(windows * (s + 1) / plan.split * kWindow, all_nb) - b0;
    }
    tile_place(pos, mt, plan.nt, im, in);
    if (GROUPED)
      t = find_tile(a, BM, im);
    else
      t = Tile{(int64_t)im * BM, min((int64_t)(im + 1) * BM, a.m), 0};
    n0 = (int64_t)in * BN;
    const int64_t w0 = (int64_t)t.expert * a.n + n0;
    const int w_rows = (int)min((int64_t)BN, a.n - n0), x_rows = (int)(t.m1 - t.m0);
    // X rows, from row x0: of this lane's direct loads and of its scale bytes
    int64_t xr[ML + 1];
#pragma unroll
    for (int i = 0; i <= ML; i++) xr[i] = min(i < ML ? (4 * i + wave) * 8 + (lane >> 3) : tid % BM, x_rows - 1);
    if (GROUPED && a.x_rows) {
#pragma unroll
      for (int i = 0; i <= ML; i++) xr[i] = a.x_rows[t.m0 + xr[i]];
#pragma unroll
      for (int i = 0; i <= ML; i++) xr[i] = min(max(xr[i], (int64_t)0), a.x_rows_total - 1);
    }
    const bool gather = GROUPED && a.x_rows;
    const int64_t x0 = gather ? 0 : t.m0, x_span = gather ? a.x_rows_total : x_rows;
    wc = rsrc_of(a.wc + w0 * kb + b0 * 16, w_rows * kb - b0 * 16);
    xc = rsrc_of(a.xc + x0 * kb + b0 * 16, x_span * kb - b0 * 16);
#pragma unroll
    for (int i = 0; i < NL; i++) ow[i] = (uint32_t)(min((4 * i + wave) * 8 + (lane >> 3), w_rows - 1) * kb);
#pragma unroll
    for (int i = 0; i < ML; i++) ox[i] = (uint32_t)(xr[i] * kb);
    psw = a.ws + (w0 + min(tid, w_rows - 1)) * all_nb + b0;
    psx = a.xs + (x0 + xr[ML]) * all_nb + b0;
  };
  // A step's loads go out in two parts, the X rows' behind the W rows'.
  struct XLoads {
    Rsrc r;
    uint32_t at[ML];
  };
  auto load_w = [&](int s, uint8_t* l) {
    const uint32_t col = (uint32_t)min(s * 8 + chunk, nb - 1) * 16;
#pragma unroll
    for (int i = 0; i < NL; i++) load_lds16(wc, ow[i] + col, l + (4 * i + wave) * 1024);
    XLoads x;
    x.r = xc;
#pragma unroll
    for (int i = 0; i < ML; i++) x.at[i] = ox[i] + col;
    return x;
  };
  auto load_x = [&](const XLoads& x, uint8_t* l) {
#pragma unroll
    for (int i = 0; i < ML; i++) load_lds16(x.r, x.at[i], l + BN * kStepB + (4 * i + wave) * 1024);
  };
  // scale bytes: thread i carries row i of either side.  A window that K does not
  // fill is read further left and moved down, with zeros behind.
  struct Window {
    u32x4_t w, x;
    int skip;  // bytes ahead of the window's first
  };
  auto load_window = [&](int w) {
    Window v;
    const int b = min(w * kWindow, all_nb - b0 - kWindow);
    v.skip = w * kWindow - b;
    __builtin_memcpy(&v.w, psw + b, 16);
    __builtin_memcpy(&v.x, psx + b, 16);
    return v;
  };
  auto moved = [&](u32x4_t v, int skip) {
    if (skip & 8) v = u32x4_t{v[2], v[3], 0, 0};
    if (skip & 4) v = u32x4_t{v[1], v[2], v[3], 0};
    const uint32_t n = (uint32_t)skip & 3;
    return u32x4_t{__builtin_amdgcn_alignbyte(v[1], v[0], n), __builtin_amdgcn_alignbyte(v[2], v[1], n),
                   __builtin_amdgcn_alignbyte(v[3], v[2], n), __builtin_amdgcn_alignbyte(0u, v[3], n)};
  };
  auto store_window = [&](const Window& v) {
    *(u32x4_t*)(scl + tid * 16) = moved(v.w, v.skip);
    if (BM == 256 || tid < BM) *(u32x4_t*)(scl + (BN + tid) * 16) = moved(v.x, v.skip);
  };

  struct Frags {
    u32x4_t w[NI], x[MI];
  };
  struct Scales {
    uint32_t w[NI], x[MI];
  };
  auto read_frags = [&](const uint8_t* l, int i) {
    Frags f;
    const int at = l32 * kStepB + ((4 * half + i) ^ (l32 & 7) ^ ((l32 >> 3) & 1)) * 16;
#pragma unroll
    for (int j = 0; j < NI; j++) f.w[j] = *(const u32x4_t*)(l + (wn + j * 32) * kStepB + at);
#pragma unroll
    for (int j = 0; j < MI; j++) f.x[j] = *(const u32x4_t*)(l + (BN + wm + j * 32) * kStepB + at);
    return f;
  };
  auto read_scales = [&](int step) {  // of the window
    Scales d;
    const int at = l32 * 16 + step * 8 + half * 4;
#pragma unroll
    for (int i = 0; i < NI; i++) d.w[i] = *(const uint32_t*)(scl + (wn + i * 32) * 16 + at);
#pragma unroll
    for (int i = 0; i < MI; i++) d.x[i] = *(const uint32_t*)(scl + (BN + wm + i * 32) * 16 + at);
    return d;
  };
  f32x16_t acc[NI][MI];
  auto products = [&](auto ii, const Frags& f, const Scales& d) {
    constexpr int I = decltype(ii)::value;
#pragma unroll
    for (int i = 0; i < NI; i++)
#pragma unroll
      for (int j = 0; j < MI; j++) acc[i][j] = mma<I>(f.w[i], f.x[j], acc[i][j], d.w[i], d.x[j]);
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
      if (i < reads - NI * MI) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      if (i < loads) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      if (i < loads - NI * MI) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  typedef std::integral_constant<int, 0> C0;
  typedef std::integral_constant<int, 1> C1;
  typedef std::integral_constant<int, 2> C2;
  typedef std::integral_constant<int, 3> C3;
  // A step from `l` with its first fragments f; returns the next step's, from
  // `next`.  `late` issues the loads that the step before left, `behind` those
  // that wait for the barrier.
  auto run_step = [&](const uint8_t* l, const uint8_t* next, Frags f, const Scales& d, auto late, auto behind) {
    Frags g = read_frags(l, 1);
    late();
    products(C0{}, f, d);
    spread(NI + MI, ML + 2);
    f = read_frags(l, 2);
    products(C1{}, g, d);
    spread(NI + MI, 0);
    g = read_frags(l, 3);
    products(C2{}, f, d);
    spread(NI + MI, 0);
    pin();
    wait_and_meet();
    behind();
    f = read_frags(next, 0);
    products(C3{}, g, d);
    spread(2 * (NI + MI), NL);
    pin();
    return f;
  };

  int item = place;
  if (item >= items) return;
  set_tile(item);
  load_x(load_w(0, s0), s0);
  XLoads x = load_w(1, s1);
  store_window(load_window(0));
  wait_and_meet();
  Frags f = read_frags(s0, 0);
  Scales d0 = read_scales(0), d1 = read_scales(1);
  while (true) {
#pragma unroll
    for (int i = 0; i < NI; i++)
#pragma unroll
      for (int j = 0; j < MI; j++)
#pragma unroll
        for (int e = 0; e < 16; e++) acc[i][j][e] = 0.0f;
    const Tile done = t;
    const int64_t dn0 = n0;
    const int dslot = slot, windows = (nb + kWindow - 1) / kWindow;
    item += grid;
    // The loads run a window ahead, in the tile's last one into the next tile (the
    // last tile's go to waste).  K that ends inside a window is filled up with
    // blocks of scale 0.
#pragma unroll 1
    for (int w = 0; w < windows; w++) {
      int next = w + 1;
      if (next == windows) {
        next = 0;
        if (item < items) set_tile(item);
      }
      const Window v = load_window(next);
      f = run_step(s0, s1, f, d0, [&]() { load_x(x, s1); }, [&]() {
        store_window(v);  // ahead of the loads, so that none is waited for
        __builtin_amdgcn_sched_barrier(0);
        x = load_w(next * 2, s0);
      });
      f = run_step(s1, s0, f, d1, [&]() { load_x(x, s0); }, [&]() {
        d0 = read_scales(0);
        x = load_w(next * 2 + 1, s1);
      });
      d1 = read_scales(1);
    }

    // ---- this tile's results
    // The accumulators are taken out of their registers where they are written, not
    // all at once, and the addresses are worked out here, not kept from before the
    // loop: either would spill.
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int half = lane >> 5, l32 = lane & 31;
    if (!GROUPED && dslot >= 0) {  // a slice's sums, in the order of the registers
      f32x4_t* p = (f32x4_t*)(plan.part + (int64_t)dslot * BM * BN) + wave * (NI * MI * 4 * 64) + lane;
#pragma unroll
      for (int i = 0; i < NI; i++)
#pragma unroll
        for (int j = 0; j < MI; j++)
#pragma unroll
          for (int q = 0; q < 4; q++) {
            f32x16_t& c = acc[i][j];
            if (q == 0) asm volatile("" : "+a"(c));
            p[((i * MI + j) * 4 + q) * 64] = f32x4_t{c[q * 4], c[q * 4 + 1], c[q * 4 + 2], c[q * 4 + 3]};
          }
    } else {
      typedef OT V4 __attribute__((ext_vector_type(4)));
      constexpr int kCols = 128 / sizeof(OT), kPer = 16 / sizeof(OT), kFr = kCols / 32;  // columns of a pass, a store
      const int rows = (int)(done.m1 - done.m0), cols = (int)min(a.n - dn0, (int64_t)BN);
      uint8_t* o = out + wave * (32 * 128);
      const int r0 = lane >> 3, c0 = (lane & 7) * kPer;  // of a store within its 8 rows
      OT* y = (OT*)a.y + (done.m0 + wm + r0) * a.n + dn0 + wn + c0;
#pragma unroll
      for (int j = 0; j < MI; j++) {
        bool none = false;
        if (GROUPED && a.x_rows && wm + j * 32 + l32 < rows) {
          const int64_t r = a.x_rows[done.m0 + wm + j * 32 + l32];
          none = r < 0 || r >= a.x_rows_total;
        }
#pragma unroll
        for (int p = 0; p < NI / kFr; p++) {
#pragma unroll
          for (int i = 0; i < kFr; i++)
#pragma unroll
            for (int q = 0; q < 4; q++) {
              f32x16_t& c = acc[p * kFr + i][j];
              if (q == 0) asm volatile("" : "+a"(c));
              V4 v = {mx_cvt<OT>(c[q * 4]), mx_cvt<OT>(c[q * 4 + 1]), mx_cvt<OT>(c[q * 4 + 2]), mx_cvt<OT>(c[q * 4 + 3])};
              if (GROUPED && none) v = V4{};
              const int byte = (i * 32 + q * 8 + half * 4) * (int)sizeof(OT);
              *(V4*)(o + l32 * 128 + (((byte >> 4) ^ (l32 & 7)) << 4) + (byte & 15)) = v;
            }
          wave_lds_sync();
          const int n = wn + p * kCols + c0;
          u32x4_t v[4];
#pragma unroll
          for (int s = 0; s < 4; s++) v[s] = *(const u32x4_t*)(o + (s * 8 + r0) * 128 + ((lane & 7) ^ r0) * 16);
#pragma unroll
          for (int s = 0; s < 4; s++)
            if (wm + j * 32 + s * 8 + r0 < rows && n + kPer <= cols)
              __builtin_memcpy(y + (int64_t)(j * 32 + s * 8) * a.n + p * kCols, &v[s], 16);
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
    }
    if (item >= items) return;
  }
}

// ---- stream kernel -------------------------------------------------------------
// For few rows of X the product is a read of W.  A workgroup of eight waves owns 16
// W rows at a time (a "row tile", one contiguous piece of memory) and all of K,
// which the waves share in units of 512 elements; each keeps its share of up to 16 MT
// rows of X (a "job") in registers for all the row tiles that the workgroup walks
// through, so that nothing but W is read in the loop.  The row
// tiles of all jobs stand in one line that is cut between the workgroups, however
// the rows are spread over the experts; a piece that crosses jobs loads the next
// one's X on the way.
//
// A row tile comes in CK chunks of up to 4096 elements of K, 32 KiB each, by
// direct-to-LDS loads into a ring of RING buffers, RING - 1 chunks ahead: memory is
// read in long runs whatever K is (pieces of 256 bytes a row, turned through
// registers, took up to 1.5 times as long where rows do not start on whole lines),
// and what is under way costs no registers.  A chunk's 16-byte pieces lie in LDS as
// in memory but for an exchange within a row, piece c of row r at c ^ (r & mask),
// which spreads the rows over the banks where the row's length would not.
//
// Rows of at most 2048 or 1024 elements come RT = two or four row tiles a chunk, each
// of which has four or two of the waves to share its K: a chunk keeps its size, its
// one barrier and its number of sums.  (128 experts of 2048 x 768, 4 rows each: 40.7 us
// with one row tile a chunk, 25.8 with four; 16 x 28672 x 2048: 9.8 and 8.5.)
//
// Of a wave's sixteen blocks, lane group g = lane / 16 takes the four from 4 g on, one
// a product: K is summed in another order, the same for both operands.  So a lane's
// four pieces of a row are 64 bytes in one run and its four scale bytes one dword.
// (With block 4 s + g at product s they were four bytes in four places, and 27 rows of
// 8192 took 32.0 us, 64 rows 40, against 28.9 and 34.4.)  The scale bytes of a row
// tile are contiguous too and come the same way (through registers they would have
// to be waited for, and all chunks under way with them: loads finish in order).
// The waves' sums meet in LDS.  Loads past the last row return zero (the buffer
// descriptor ends there), so no load has a branch around it and a chunk's loads
// have a fixed number.
//
// Bound by the read of W: 27 x 28672 x 8192 28.6-30.1 us (125 MB, 4.2-4.4 TB/s; a copy
// of 1 GiB reaches 5.06), 1 x 14336 x 4096 8.3-8.5 us (31 MB, 3.7 TB/s: a third of it is
// the ramp of a launch).  With one or two such weights in turn, which the 256 MB behind
// the L2 caches hold, 24.2-24.6 and 7.4-7.9.
constexpr int kSWaves = 8, kSLoads = kSRows * kChunkB / 1024 / kSWaves;

template <int I> __device__ __forceinline__ f32x4_t mma16(u32x4_t a, u32x4_t b, f32x4_t c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag(a), frag(b), c, 4, 4, I, (int)sa, I, (int)sb);
}

// f(0), f(1) .. as compile-time constants, until one of them is false.
template <typename F, int... I> __device__ __forceinline__ bool for_each(F& f, std::integer_sequence<int, I...>) {
  return (f(std::integral_constant<int, I>{}) && ...);
}

// Ring places.
constexpr int stream_ring(int mt) { return mt == 4 ? 3 : 4; }

template <int RT, int CK, int MT, bool GROUPED>
__global__ __launch_bounds__(64 * kSWaves, 2) void mx_stream_kernel(Args a, int y_dtype, StreamPlan plan) {
  constexpr int kRing = stream_ring(MT);
  static_assert(RT == 1 || CK == 1, "chunks of several row tiles hold whole rows");
  // Of the waves of a row tile, kAlong share its K and kX the job's rows; a wave has
  // kUnits times 512 elements of K and kMT times 16 rows.  Sharing the rows reads W's
  // fragments twice from LDS, but leaves room for a second set of sums: 128 x 14336 x
  // 4096 17.0 us without and 16.0 with it, 27 rows 10.3 and 9.8.  (64 experts of 1503 x
  // 2080, 1000 rows: 29.8 and 31.7.)
  constexpr int kX = !GROUPED && CK == 1 && MT > 1 ? 2 : 1, kAlong = kSWaves / RT / kX, kUnits = kX, kMT = MT / kX;
  constexpr int kRows = kSRows * RT;         // rows of W in a chunk
  constexpr int kPart = kSRows * 16 * kMT;   // fp32 sums of one wave
  constexpr int kSums = kSRows * 16 * MT;    // results of a row tile
  constexpr int kOuts = (RT * kSums + 64 * kSWaves - 1) / (64 * kSWaves);  // of a thread in a chunk
  // A round is whole row tiles and whole turns of the ring, and an even number of tiles
  // where there are two sets of sums.
  constexpr int kRound = CK == 4 ? 8 : kRing % 2 ? 2 * kRing : kRing;
  constexpr int kAreas = CK == 1 ? kRing : kRound / CK;  // scale areas, in turn for the round's row tiles
  // Row tiles that the scale bytes are requested ahead: enough that the loads of
  // kRing - 2 chunks are behind them when they are needed.
  constexpr int kScAhead = CK == 1 ? kRing - 2 : 1;
  constexpr int kArea = (kSRows * stream_blocks(CK) + 4 + 15) & ~15;
  static_assert(kArea <= 1024 * kSWaves && kAreas > kScAhead, "one load a wave");
  __shared__ __attribute__((aligned(16))) uint8_t r0[kSRows * kChunkB], r1[kSRows * kChunkB], r2[kSRows * kChunkB],
      r3[kRing > 3 ? kSRows * kChunkB : 16];
  __shared__ __attribute__((aligned(16))) uint8_t a0[kArea], a1[kArea], a2[kAreas > 2 ? kArea : 16], a3[kAreas > 3 ? kArea : 16];
  // The waves' sums of a row tile are added behind the next chunk's barrier, where there
  // is a second set of them or a barrier more before the next tile's are written.
  constexpr int kParts = CK == 1 && (MT == 1 || kX == 2) ? 2 : 1;
  constexpr bool kDefer = CK > 1 || kParts == 2;
  __shared__ __attribute__((aligned(16))) float part[kParts * kSWaves * kPart];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nb = (int)(a.k / kMxBlock), kb = nb * 16;
  const int units = (int)((a.n + kSRows - 1) / kSRows);  // what the line is cut into
  auto ring = [&](auto p) -> uint8_t* {
    constexpr int i = decltype(p)::value % kRing;
    return i == 0 ? r0 : i == 1 ? r1 : i == 2 ? r2 : r3;
  };
  auto area = [&](auto tile) -> uint8_t* {
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
  // the scale bytes' pieces are exchanged likewise, by their place in the area
  auto sc_place = [&](int piece) {
    return plan.sc_pieces ? piece ^ key(plan.sc_pieces, quotient(piece, plan.mul_sc)) : piece;
  };
  const uint32_t sc_from = (uint32_t)sc_place(tid) * 16;

  // this workgroup's piece of the line
  const uint32_t b = blockIdx.x;
  Cuts c = plan.cuts;
  if (GROUPED) c = cuts_of((uint32_t)units, (uint32_t)live_tiles(a, plan.rows), gridDim.x, RT);
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
      t = find_tile(a, plan.rows, job);
    else
      t = Tile{(int64_t)job * plan.rows, min((int64_t)(job + 1) * plan.rows, a.m), 0};
    if (GROUPED && t.expert < 0) return;
    // its rows of W in this job: n_rows from n0 on, in `end` chunks or times CK
    const int taken = min(left, units - unit), n0 = unit * kSRows;
    const int n_rows = (int)min((int64_t)taken * kSRows, a.n - n0), end = (n_rows + kRows - 1) / kRows;
    left -= taken;
    int tile = 0;
    const uint8_t* wc = a.wc + ((int64_t)t.expert * a.n + n0) * kb;
    const uint8_t* wsc = a.ws + ((int64_t)t.expert * a.n + n0) * nb;
    auto rows_of = [&](int tile) { return tile < end ? min(n_rows - tile * kRows, kRows) : 0; };
    auto load_chunk = [&](int tile, int ck, uint8_t* l) {
      const int col = ck * plan.pieces * 16;
      const Rsrc r = rsrc_of(wc + (int64_t)tile * kRows * kb + col, max(rows_of(tile) * kb - col, 0));
#pragma unroll
      for (int i = 0; i < kSLoads; i++)
        load_lds16(r, ck == CK - 1 ? off_last[i] : off[i], l + (i * kSWaves + wave) * 1024);
    };
    // A row tile's scale bytes, in whole dwords: up to three bytes on either side
    // are not its own and not looked at.  Wave i takes bytes 1024 i on; dwords that
    // hold none of the tile's bytes read zero.
    const int skew = (int)((uintptr_t)wsc & 3);  // of every row tile: 16 rows are whole dwords
    auto load_scales = [&](int tile, uint8_t* l) {
      const int rows = rows_of(tile);
      const Rsrc r = rsrc_of(wsc + (int64_t)tile * kRows * nb - skew, rows ? (rows * nb + skew + 3) & ~3 : 0);
      if (tid * 16 < kArea) load_lds16(r, sc_from, l + wave * 1024);
    };
    __syncthreads();  // the job before still reads the ring
    load_scales(tile, a0);
    load_chunk(tile, 0, r0);
    __builtin_amdgcn_sched_barrier(0);
    // this wave's share of X
    u32x4_t fx[kMT][CK][kUnits][4];
    uint32_t dx[kMT][CK][kUnits];
    const int along = wave % kAlong, x_row = wave / kAlong % kX * 16 * kMT;
#pragma unroll
    for (int j = 0; j < kMT; j++) {
      int64_t row = min(t.m0 + x_row + 16 * j + (lane & 15), t.m1 - 1);
      if (GROUPED && a.x_rows) row = min((int64_t)max(a.x_rows[row], 0), a.x_rows_total - 1);
      const uint8_t *pc = a.xc + row * kb, *ps = a.xs + row * nb;
#pragma unroll
      for (int u = 0; u < CK; u++)
#pragma unroll
        for (int v = 0; v < kUnits; v++) {
          const int b = u * plan.pieces + 16 * (along + v * kAlong) + 4 * (lane >> 4);  // the first of its four blocks
#pragma unroll
          for (int i = 0; i < 4; i++) fx[j][u][v][i] = *(const u32x4_t*)(pc + min(b + i, nb - 1) * 16);
          dx[j][u][v] = scales4(ps, b, nb);
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
    const int g = at_lane >> 4, w_row = wave / (kAlong * kX) * kSRows + (at_lane & 15), mine = 16 * along + 4 * g;
    // of its blocks' scale bytes, those that the chunk has: past the row, scale 0
    auto kept = [&](int left) { return left >= 4 ? ~0u : left <= 0 ? 0u : ~(~0u << 8 * left); };
    uint32_t keep[kUnits], keep_last[kUnits];
#pragma unroll
    for (int v = 0; v < kUnits; v++) {
      keep_last[v] = kept(plan.last - mine - 16 * v * kAlong);
      keep[v] = CK > 1 ? kept(plan.pieces - mine - 16 * v * kAlong) : keep_last[v];
    }
    // fragment i of W in a chunk; the next unit's lie kAlong * 256
    // bytes on, as the exchange is within 16 pieces
    int fo[4], fo_last[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int c = mine + i;
      auto offset = [&](int pieces) {  // past the row: some other codes
        return min(w_row * pieces + (c ^ key(pieces, w_row)), kSRows * kChunkB / 16 - 1 - 16 * kAlong * (kUnits - 1)) * 16;
      };
      fo_last[i] = offset(plan.last);
      fo[i] = CK > 1 ? offset(plan.pieces) : fo_last[i];
    }
    // this lane's four scale bytes in the area: the two dwords that hold them
    const int sc_shift = (skew + w_row * nb) & 3;
    int so[CK][kUnits][2];
#pragma unroll
    for (int u = 0; u < CK; u++)
#pragma unroll
      for (int v = 0; v < kUnits; v++)
#pragma unroll
        for (int i = 0; i < 2; i++) {
          const int at = min(((skew + w_row * nb + u * plan.pieces + mine + 16 * v * kAlong) & ~3) + 4 * i, kArea - 4);
          so[u][v][i] = sc_place(at >> 4) * 16 + (at & 15);
        }
#pragma unroll
    for (int j = 0; j < kMT; j++)
#pragma unroll
      for (int u = 0; u < CK; u++)
#pragma unroll
        for (int v = 0; v < kUnits; v++) dx[j][u][v] &= u == CK - 1 ? keep_last[v] : keep[v];

    // this thread's results: rows that padding leaves zero
    bool none[kOuts];
#pragma unroll
    for (int i = 0; i < kOuts; i++) {
      none[i] = false;
      const int64_t row = t.m0 + ((tid + i * 64 * kSWaves) % kSums >> 4);
      if (GROUPED && a.x_rows && row < t.m1) {
        const int64_t r = a.x_rows[row];
        none[i] = r < 0 || r >= a.x_rows_total;
      }
    }
    // y of a row tile, from set `set` of the waves' sums
    auto finish = [&](int tile, int set) {
#pragma unroll
      for (int i = 0; i < kOuts; i++) {
        const int o = tid + i * 64 * kSWaves;
        const int n = o & 15, m = (RT == 1 ? o : o % kSums) >> 4, at_tile = RT == 1 ? 0 : o / kSums;
        const int m_x = kX == 1 ? m : m % (16 * kMT);
        const int64_t row = t.m0 + m;
        const int col = tile * kRows + at_tile * kSRows + n;
        if (o >= RT * kSums || row >= t.m1 || col >= n_rows) continue;
        // lane (n / 4) * 16 + m % 16 of a wave holds it in element n % 4
        const float* p = part + ((set * RT + at_tile) * kX + (kX == 1 ? 0 : m / (16 * kMT))) * kAlong * kPart + (m_x >> 4) * 256 +
                         ((n >> 2) * 16 + (m_x & 15)) * 4 + (n & 3);
        float v[kAlong];
#pragma unroll
        for (int w = 0; w < kAlong; w++) v[w] = p[w * kPart];
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kAlong; w++) sum += v[w];
        if (none[i]) sum = 0.0f;
        const int64_t at = row * a.n + n0 + col;
        if (y_dtype == kF32) ((float*)a.y)[at] = sum;
        else if (y_dtype == kF16) ((_Float16*)a.y)[at] = mx_cvt<_Float16>(sum);
        else ((__bf16*)a.y)[at] = mx_cvt<__bf16>(sum);
      }
    };
    auto meet = [&]() {  // once this wave's LDS accesses are done
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    };
    f32x4_t acc[kMT];
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
        for (int j = 0; j < kMT; j++) acc[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      }
      load_chunk(tile + ahead / CK, ahead % CK, ring(std::integral_constant<int, P + kRing - 1>{}));
      const uint8_t* l = ring(which);
      const uint8_t* ds = area(std::integral_constant<int, P / CK>{});
      auto unit_of = [&](auto which_unit) {
        constexpr int v = decltype(which_unit)::value;
        if (v > 0 && 16 * (along + v * kAlong) >= plan.last) return false;  // the row ends before it
        u32x4_t f[4];
#pragma unroll
        for (int i = 0; i < 4; i++) f[i] = *(const u32x4_t*)(l + (ck == CK - 1 ? fo_last[i] : fo[i]) + v * kAlong * 256);
        const uint32_t d0 = *(const uint32_t*)(ds + so[ck][v][0]), d1 = *(const uint32_t*)(ds + so[ck][v][1]);
        const uint32_t dw = __builtin_amdgcn_alignbyte(d1, d0, sc_shift) & (ck == CK - 1 ? keep_last[v] : keep[v]);
#pragma unroll
        for (int j = 0; j < kMT; j++) {
          acc[j] = mma16<0>(f[0], fx[j][ck][v][0], acc[j], dw, dx[j][ck][v]);
          acc[j] = mma16<1>(f[1], fx[j][ck][v][1], acc[j], dw, dx[j][ck][v]);
          acc[j] = mma16<2>(f[2], fx[j][ck][v][2], acc[j], dw, dx[j][ck][v]);
          acc[j] = mma16<3>(f[3], fx[j][ck][v][3], acc[j], dw, dx[j][ck][v]);
          asm volatile("" : "+v"(acc[j]));  // here, not behind the next barrier with all chunks' operands
        }
        return true;
      };
      for_each(unit_of, std::make_integer_sequence<int, kUnits>{});
      if constexpr (kDefer && ck == 0)
        if (tile > 0) finish(tile - 1, (P / CK + kParts - 1) % kParts);
      if constexpr (ck == CK - 1) {
        float* sums = part + (P / CK % kParts * kSWaves + wave) * kPart;
#pragma unroll
        for (int j = 0; j < kMT; j++) *(f32x4_t*)(sums + j * 256 + lane * 4) = acc[j];
        if constexpr (!kDefer) {
          meet();
          finish(tile, 0);
        }
        return ++tile < end;
      }
      return true;
    };
    while (for_each(chunk, std::make_integer_sequence<int, kRound>{})) {
    }
    if constexpr (kDefer) {
      meet();
      finish(end - 1, (end - 1) % kParts);
    }
  }
}

template <int RT, int CK, int MT> hipError_t go_stream(const Args& a, int y_dtype, StreamPlan p, hipStream_t stream) {
  const int64_t tiles = (a.n + kSRows - 1) / kSRows, full = (a.m + p.rows - 1) / p.rows;
  const int64_t jobs = a.offsets ? std::min(full + a.experts, a.m) : full;
  const int64_t grid = std::min(tiles * jobs, (int64_t)device_cu_count());  // the ring fills a CU
  if (!a.offsets) {
    p.cuts = cuts_of((uint32_t)tiles, (uint32_t)jobs, (uint32_t)grid, RT);
    if (p.cuts.per_job) p.mul_per_job = (1 << 20) / (int)p.cuts.per_job + 1;
  }
  const dim3 blocks((unsigned)grid), threads(64 * kSWaves);
  if (a.offsets) hipLaunchKernelGGL((mx_stream_kernel<RT, CK, MT, true>), blocks, threads, 0, stream, a, y_dtype, p);
  else hipLaunchKernelGGL((mx_stream_kernel<RT, CK, MT, false>), blocks, threads, 0, stream, a, y_dtype, p);
  return hipGetLastError();
}

hipError_t run_stream(const Args& a, int y_dtype, const StreamPlan& p, hipStream_t s) {
  if (p.rt == 4) return p.mt == 1 ? go_stream<4, 1, 1>(a, y_dtype, p, s) : go_stream<4, 1, 2>(a, y_dtype, p, s);
  if (p.rt == 2) return p.mt == 1 ? go_stream<2, 1, 1>(a, y_dtype, p, s) : go_stream<2, 1, 2>(a, y_dtype, p, s);
  switch (p.mt * 16 + p.ck) {
    case 17: return go_stream<1, 1, 1>(a, y_dtype, p, s);
    case 18: return go_stream<1, 2, 1>(a, y_dtype, p, s);
    case 20: return go_stream<1, 4, 1>(a, y_dtype, p, s);
    case 33: return go_stream<1, 1, 2>(a, y_dtype, p, s);
    case 34: return go_stream<1, 2, 2>(a, y_dtype, p, s);
    case 36: return go_stream<1, 4, 2>(a, y_dtype, p, s);
    case 65: return go_stream<1, 1, 4>(a, y_dtype, p, s);
    default: return go_stream<1, 2, 4>(a, y_dtype, p, s);
  }
}

// y of the split tiles: adds the slices' sums, slice by slice.  A thread takes 16
// sums of one fragment in register order; the half-waves swap so that each lane
// stores runs of eight columns.
template <int BM, typename OT>
__global__ __launch_bounds__(256) void mx_fold_kernel(Args a, TilePlan plan) {
  constexpr int BN = kTileN;
  constexpr int NI = BN / 64, MI = BM / 64;
  typedef OT V8 __attribute__((ext_vector_type(8)));
  const int lane = threadIdx.x & 63, half = lane >> 5, l32 = lane & 31;
  const int piece = blockIdx.x * 4 + (threadIdx.x >> 6);  // fragment of a tile
  const int tile = piece / (4 * NI * MI), frag = piece % (4 * NI * MI);
  const int wave = frag / (NI * MI), i = frag % (NI * MI) / MI, j = frag % MI;
  int im, in;
  tile_place(plan.full + tile, plan.mt, plan.nt, im, in);
  f32x4_t v[4] = {};
  const f32x4_t* p = (const f32x4_t*)plan.part + ((int64_t)tile * plan.split * 4 * NI * MI + frag) * 256 + lane;
  for (int s = 0; s < plan.split; s++, p += 4 * NI * MI * 256)
#pragma unroll
    for (int q = 0; q < 4; q++) v[q] += p[q * 64];
  const int64_t row = (int64_t)im * BM + (wave >> 1) * (BM / 2) + j * 32 + l32;
#pragma unroll
  for (int q = 0; q < 4; q += 2) {
    // of columns 8 q .. 8 q + 15 the lower half-wave stores the first eight, the upper the others
    f32x4_t other;
#pragma unroll
    for (int e = 0; e < 4; e++) other[e] = __shfl_xor(half ? v[q][e] : v[q + 1][e], 32, 64);
    const f32x4_t lo = half ? other : v[q], hi = half ? v[q + 1] : other;
    const int64_t n = (int64_t)in * BN + (wave & 1) * (BN / 2) + i * 32 + (q + half) * 8;
    if (row >= a.m || n >= a.n) continue;
    OT* y = (OT*)a.y + row * a.n + n;
    V8 o;
#pragma unroll
    for (int e = 0; e < 8; e++) o[e] = mx_cvt<OT>(e < 4 ? lo[e] : hi[e - 4]);
    if (n + 8 <= a.n) {
      __builtin_memcpy(y, &o, sizeof(o));
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (n + e < a.n) y[e] = o[e];
    }
  }
}

template <int BM, typename OT, bool GROUPED> hipError_t go_tiles(const Args& a, const TilePlan& p, hipStream_t stream) {
  const int grid = std::min(p.full + p.rest * p.split, device_cu_count());
  hipLaunchKernelGGL((mx_tile_kernel<BM, OT, GROUPED>), dim3((unsigned)grid), dim3(256), 0, stream, a, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !p.rest) return e;
  hipLaunchKernelGGL((mx_fold_kernel<BM, OT>), dim3((unsigned)(p.rest * (kTileN / 64) * (BM / 64))), dim3(256), 0,
                     stream, a, p);
  return hipGetLastError();
}

template <typename OT> hipError_t run(const Args& a, void* ws, hipStream_t stream) {
  double us;
  TilePlan p = tile_plan(a.m, a.n, a.k, a.offsets ? a.experts : 0, us);
  p.part = (float*)ws;
  if (p.high == 256) return a.offsets ? go_tiles<256, OT, true>(a, p, stream) : go_tiles<256, OT, false>(a, p, stream);
  return a.offsets ? go_tiles<128, OT, true>(a, p, stream) : go_tiles<128, OT, false>(a, p, stream);
}

}  // namespace

size_t mx_gemm_ws_bytes(int64_t m, int64_t n, int64_t k, int64_t experts) {
  StreamPlan p;
  double us;
  return streams(m, n, k, experts, p) ? 0 : tile_ws_bytes(tile_plan(m, n, k, experts, us));
}

hipError_t launch_mx_gemm(const MxGemm& g, void* ws, size_t, hipStream_t stream) {
  if (g.m == 0 || g.n == 0) return hipSuccess;
  const Args a = {g.x.codes, g.x.scales, g.w.codes, g.w.scales, g.m, g.n, g.k, g.x.rows, g.y, g.offsets, g.x_rows,
                  g.experts};
  StreamPlan p;
  if (streams(g.m, g.n, g.k, g.offsets ? g.experts : 0, p)) return run_stream(a, g.y_dtype, p, stream);
  if (g.y_dtype == kF32) return run<float>(a, ws, stream);
  if (g.y_dtype == kF16) return run<_Float16>(a, ws, stream);
  return run<__bf16>(a, ws, stream);
}

}  // namespace rz
