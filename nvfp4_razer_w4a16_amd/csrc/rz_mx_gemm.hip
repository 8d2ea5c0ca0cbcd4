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
#include <type_traits>

#include "rz_mx.h"
#include "rz_mx_launch.h"

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
  if (!a.offsets) {
    const int64_t m0 = t * rows;
    return {m0, min(m0 + rows, a.m), m0 < a.m ? 0 : -1};
  }
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
      const int first = __shfl(sum - cnt, src, 64);
      const int l = __shfl(lo, src, 64), h = __shfl(hi, src, 64);
      const int m0 = l + (int)(t - first) * rows;
      return {m0, min(m0 + rows, h), e0 + src};
    }
    before = __shfl(sum, 63, 64);
  }
  return {0, 0, -1};
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

// Stores y[row][n .. n + 3] (those below nn), rounded once.
template <typename OT>
__device__ __forceinline__ void store4(OT* y, int64_t row, int64_t n, int64_t nn, const float (&v)[4]) {
  typedef OT V __attribute__((ext_vector_type(4)));
  OT* p = y + row * nn + n;
  if ((nn & 3) == 0 && n + 4 <= nn) {
    *(V*)p = V{mx_cvt<OT>(v[0]), mx_cvt<OT>(v[1]), mx_cvt<OT>(v[2]), mx_cvt<OT>(v[3])};
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (n + i < nn) p[i] = mx_cvt<OT>(v[i]);
  }
}

// ---- tile kernel -------------------------------------------------------------
// A BN x BM tile of y (BN rows of W, BM of X) per workgroup of four waves (2x2),
// each wave (BN/2) x (BM/2) in 32x32 accumulators, 256 elements of K a step.
//
// LDS: two buffers of a step's codes, filled by direct-to-LDS loads of whole
// 128-byte row pieces.  A piece is eight 16-byte chunks; chunk c of row r lies at
// place c ^ (r & 7), so the lanes of a fragment read (one chunk of 32 rows)
// spread over the banks.  Direct loads write lane-linear, so the loading lane
// picks its chunk by the same rule.  Scale bytes come through registers, 16
// bytes a row (two steps, a "window"), into one LDS area.
//
// Schedule of a step (four sub-steps of 64 elements): the fragments of the next
// sub-step are read while the products of this one run.  The barrier sits before
// the last sub-step, whose fragments are then in registers: behind it the next
// step's buffer is complete and this step's is free, so the loads of the step
// after next and the first fragments of the next step go out under its products.
constexpr int kStep = 256, kRowB = kStep / 2;

typedef __attribute__((address_space(1))) const void* GlobalPtr;
typedef __attribute__((address_space(3))) void* LdsPtr;
__device__ __forceinline__ void load_lds16(const uint8_t* g, uint8_t* l) {
  __builtin_amdgcn_global_load_lds((GlobalPtr)g, (LdsPtr)l, 16, 0, 0);
}

// Number of the tile that workgroup b computes: consecutive workgroups go to the
// eight XCDs in turn, so each XCD gets a contiguous run of tiles (and its L2 the
// W rows that the run shares).
__device__ __forceinline__ int64_t xcd_tile(int64_t b, int64_t tiles) {
  const int64_t per = tiles / 8, extra = tiles % 8, x = b % 8, i = b / 8;
  return x * per + min(x, extra) + i;
}

template <int BN, int BM, typename OT>
__global__ __launch_bounds__(256, BN * BM > 128 * 128 ? 1 : 2) void mx_tile_kernel(Args a, int64_t m_tiles) {
  constexpr int NI = BN / 64, MI = BM / 64;  // 32-row fragments of a wave
  __shared__ __attribute__((aligned(16))) uint8_t w0[BN * kRowB], x0[BM * kRowB], w1[BN * kRowB], x1[BM * kRowB];
  __shared__ __attribute__((aligned(16))) uint8_t scw[BN * 16], scx[BM * 16];
  const int64_t id = xcd_tile(blockIdx.x, gridDim.x);
  const Tile t = find_tile(a, BM, id % m_tiles);
  if (t.expert < 0) return;
  const int64_t n0 = id / m_tiles * BN;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nb = (int)(a.k / kMxBlock);
  const int64_t kb = a.k / 2;
  const int steps = (nb + 7) / 8;
  auto w_row = [&](int r) { return (int64_t)t.expert * a.n + min(n0 + r, a.n - 1); };
  auto x_row = [&](int r) -> int64_t {
    const int64_t row = min(t.m0 + r, t.m1 - 1);
    return a.x_rows ? min((int64_t)max(a.x_rows[row], 0), a.x_rows_total - 1) : row;
  };
  // direct loads: instruction i of a wave fills rows (4 i + wave) * 8 ..+7
  const int chunk = (lane & 7) ^ (lane >> 3);
  const uint8_t* wc = a.wc + ((int64_t)t.expert * a.n + n0) * kb;
  const int64_t x_first = a.x_rows ? 0 : t.m0;
  const uint8_t* xc = a.xc + x_first * kb;
  uint32_t ow[BN / 32], ox[BM / 32];  // the rows' bytes, from the tile's first row (gathered ones from X's)
#pragma unroll
  for (int i = 0; i < BN / 32; i++) ow[i] = (uint32_t)(min((int64_t)((4 * i + wave) * 8 + (lane >> 3)), a.n - 1 - n0) * kb);
#pragma unroll
  for (int i = 0; i < BM / 32; i++) ox[i] = (uint32_t)((x_row((4 * i + wave) * 8 + (lane >> 3)) - x_first) * kb);
  auto load_step = [&](int s, uint8_t* lw, uint8_t* lx) {
    const uint32_t col = (uint32_t)min(s * 8 + chunk, nb - 1) * 16;
#pragma unroll
    for (int i = 0; i < BN / 32; i++) load_lds16(wc + (uint64_t)(ow[i] + col), lw + (4 * i + wave) * 1024);
#pragma unroll
    for (int i = 0; i < BM / 32; i++) load_lds16(xc + (uint64_t)(ox[i] + col), lx + (4 * i + wave) * 1024);
  };
  // scale bytes: thread i carries row i of either tile, 16 blocks (a window) at a time
  const uint8_t* psw = a.ws + w_row(tid % BN) * nb;
  const uint8_t* psx = a.xs + x_row(tid % BM) * nb;
  struct Window {
    u32x4_t w, x;
  };
  auto load_window = [&](int b) {
    Window v;
    __builtin_memcpy(&v.w, psw + b, 16);
    __builtin_memcpy(&v.x, psx + b, 16);
    return v;
  };
  auto store_window = [&](const Window& v) {
    if (BN == 256 || tid < BN) *(u32x4_t*)(scw + tid * 16) = v.w;
    if (BM == 256 || tid < BM) *(u32x4_t*)(scx + tid * 16) = v.x;
  };
  auto tail_window = [&](int b) {  // zeros from the end of K on
#pragma unroll 1
    for (int i = 0; i < 16; i++) {
      const int c = min(b + i, nb - 1);
      if (tid < BN) scw[tid * 16 + i] = b + i < nb ? psw[c] : 0;
      if (tid < BM) scx[tid * 16 + i] = b + i < nb ? psx[c] : 0;
    }
  };

  const int wn = (wave & 1) * (BN / 2), wm = (wave >> 1) * (BM / 2);
  const int half = lane >> 5, l32 = lane & 31;
  struct Frags {
    u32x4_t w[NI], x[MI];
  };
  struct Dwords {
    uint32_t w[NI], x[MI];
  };
  auto read_frags = [&](const uint8_t* lw, const uint8_t* lx, int kk) {
    Frags f;
    const int place = ((half * 4 + kk) ^ (l32 & 7)) * 16;
#pragma unroll
    for (int i = 0; i < NI; i++) f.w[i] = *(const u32x4_t*)(lw + (wn + i * 32 + l32) * kRowB + place);
#pragma unroll
    for (int i = 0; i < MI; i++) f.x[i] = *(const u32x4_t*)(lx + (wm + i * 32 + l32) * kRowB + place);
    return f;
  };
  auto read_scales = [&](int step) {  // of the window
    Dwords d;
#pragma unroll
    for (int i = 0; i < NI; i++) d.w[i] = *(const uint32_t*)(scw + (wn + i * 32 + l32) * 16 + step * 8 + half * 4);
#pragma unroll
    for (int i = 0; i < MI; i++) d.x[i] = *(const uint32_t*)(scx + (wm + i * 32 + l32) * 16 + step * 8 + half * 4);
    return d;
  };
  f32x16_t acc[NI][MI];
#pragma unroll
  for (int i = 0; i < NI; i++)
#pragma unroll
    for (int j = 0; j < MI; j++)
#pragma unroll
      for (int e = 0; e < 16; e++) acc[i][j][e] = 0.0f;
  auto products = [&](auto kk, const Frags& f, const Dwords& d) {
    constexpr int I = decltype(kk)::value;
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
  typedef std::integral_constant<int, 0> K0;
  typedef std::integral_constant<int, 1> K1;
  typedef std::integral_constant<int, 2> K2;
  typedef std::integral_constant<int, 3> K3;
  // One step from buffer (lw, lx), f its first fragments; `behind` runs after the
  // barrier and returns the next step's first fragments.
  // The instruction order asked for: a sub-step's LDS reads, then the direct loads,
  // one at a time between its products.
  auto spread = [&](int reads, int loads) {
#pragma unroll
    for (int i = 0; i < NI * MI; i++) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (i < reads) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      if (i < loads) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto step = [&](const uint8_t* lw, const uint8_t* lx, Frags f, const Dwords& d, auto behind) {
    Frags g = read_frags(lw, lx, 1);
    products(K0{}, f, d);
    spread(NI + MI, 2);
    f = read_frags(lw, lx, 2);
    products(K1{}, g, d);
    spread(NI + MI, 0);
    g = read_frags(lw, lx, 3);
    products(K2{}, f, d);
    spread(NI + MI, 0);
    pin();
    __syncthreads();
    f = behind();
    products(K3{}, g, d);
    spread(NI * MI, (BN + BM) / 32);
    pin();
    return f;
  };

  load_step(0, w0, x0);
  if (steps > 1) load_step(1, w1, x1);
  if (nb >= 16)
    store_window(load_window(0));
  else
    tail_window(0);
  __syncthreads();
  Frags f = read_frags(w0, x0, 0);
  Dwords da = read_scales(0), db = read_scales(1);
  int s = 0;
  // Two steps (a window) a round.  While the next window lies within K there is
  // nothing to ask on the way, and the loads spread between the products.
  for (; s * 8 + 32 <= nb; s += 2) {
    const Window v = load_window(s * 8 + 16);
    f = step(w0, x0, f, da, [&]() {
      store_window(v);  // ahead of the loads, which the compiler would have it wait for
      __builtin_amdgcn_sched_barrier(0);
      load_step(s + 2, w0, x0);
      return read_frags(w1, x1, 0);
    });
    f = step(w1, x1, f, db, [&]() {
      load_step(s + 3, w1, x1);
      da = read_scales(0);
      return read_frags(w0, x0, 0);
    });
    db = read_scales(1);
  }
  // the last ones, where K may end
  for (; s < steps; s += 2) {
    f = step(w0, x0, f, da, [&]() {
      if (s + 2 < steps) load_step(s + 2, w0, x0);
      tail_window(s * 8 + 16);
      return read_frags(w1, x1, 0);
    });
    if (s + 1 == steps) break;
    f = step(w1, x1, f, db, [&]() {
      if (s + 3 < steps) load_step(s + 3, w1, x1);
      da = read_scales(0);
      return read_frags(w0, x0, 0);
    });
    db = read_scales(1);
  }
#pragma unroll
  for (int j = 0; j < MI; j++) {
    const int64_t row = t.m0 + wm + j * 32 + l32;
    if (row >= t.m1) continue;
    bool none = false;
    if (a.x_rows) {
      const int64_t r = a.x_rows[row];
      none = r < 0 || r >= a.x_rows_total;
    }
#pragma unroll
    for (int i = 0; i < NI; i++)
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int64_t n = n0 + wn + i * 32 + q * 8 + half * 4;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; e++) v[e] = none ? 0.0f : acc[i][j][q * 4 + e];
        if (n < a.n) store4((OT*)a.y, row, n, a.n, v);
      }
  }
}

// ---- stream kernel -------------------------------------------------------------
// For few rows of X the product is a read of W.  A workgroup owns 16 W rows at a
// time (a "row tile") and all of K; each of its up to eight waves takes U units
// of 512 elements of K and keeps its share of up to 16 MT rows of X in registers
// for all the row tiles that the workgroup walks through, so that nothing but W
// is read in the loop.
//
// A unit (16 rows x 256 bytes) is loaded with four instructions that each cover
// 256 contiguous bytes of four rows, four units ahead of their use, and turned
// through a wave's own LDS stage into the operand's layout (chunk c of row r at
// place c ^ r: no bank conflicts either way).  Group g = lane / 16 takes block
// 4g + s of a unit at MFMA s, so its scale bytes are one dword.  The scale bytes
// of a row tile are one contiguous piece of memory; the workgroup loads it a
// tile ahead and hands it round in LDS.  The waves' partial sums meet in LDS,
// one barrier a row tile (both areas are double-buffered).
//
// Reads past the last W row return zero (the buffer descriptor ends there), so
// the loop has no branch around a load.
constexpr int kSRows = 16, kSUnit = 512, kSAhead = 4, kSMaxWaves = 8;

typedef __amdgpu_buffer_rsrc_t Rsrc;
__device__ __forceinline__ Rsrc rsrc_of(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)bytes, 0x00020000);
}

template <int I> __device__ __forceinline__ f32x4_t mma16(u32x4_t a, u32x4_t b, f32x4_t c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag(a), frag(b), c, 4, 4, I, (int)sa, I, (int)sb);
}

template <int U, int MT>
__global__ __launch_bounds__(64 * kSMaxWaves, U * MT == 1 ? 4 : 2) void mx_stream_kernel(Args a, int y_dtype, int waves) {
  constexpr int kPart = kSRows * 16 * MT;  // fp32 sums of one wave
  constexpr int kChunks = U / 4 + 1;       // 16-byte chunks of a tile's scale bytes a thread carries: nb + 1 <= 16 U waves + 1
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const Tile t = find_tile(a, 16 * MT, blockIdx.y);
  if (t.expert < 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nb = (int)(a.k / kMxBlock), kb = nb * 16;
  const int g = lane >> 4, l16 = lane & 15;
  uint8_t* stage = smem + wave * (kSRows * 256);
  float* part = (float*)(smem + waves * (kSRows * 256));            // [2][waves][kPart]
  uint8_t* sc = (uint8_t*)(part + 2 * waves * kPart);                // [2][sc_bytes]
  const int sc_bytes = (kSRows * nb + 4 + 15 + 4) & ~15;             // a tile's scale bytes, dword-aligned start
  const int unit0 = wave * U;
  const uint8_t* wc = a.wc + (int64_t)t.expert * a.n * kb;
  const uint8_t* wsc = a.ws + (int64_t)t.expert * a.n * nb;
  const int tiles = (int)((a.n + kSRows - 1) / kSRows);

  // this wave's share of X
  u32x4_t fx[MT][U][4];
  uint32_t dx[MT][U];
  const int64_t last = t.m1 - 1;
#pragma unroll
  for (int j = 0; j < MT; j++) {
    int64_t row = min(t.m0 + 16 * j + l16, last);
    if (a.x_rows) row = min((int64_t)max(a.x_rows[row], 0), a.x_rows_total - 1);
    const uint8_t *pc = a.xc + row * kb, *ps = a.xs + row * nb;
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int b = (unit0 + u) * 16 + 4 * g;
#pragma unroll
      for (int s = 0; s < 4; s++) fx[j][u][s] = *(const u32x4_t*)(pc + min(b + s, nb - 1) * 16);
      dx[j][u] = scales4(ps, b, nb);
    }
  }

  // W units: slot i of a round is unit i % U of row tile i / U of the round
  constexpr int kRound = U > kSAhead ? U : kSAhead, kTilesRound = kRound / U;
  u32x4_t fw[kSAhead][4];
  int voff[4];
#pragma unroll
  for (int i = 0; i < 4; i++) voff[i] = (4 * i + g) * kb + l16 * 16;
  const int step = (int)gridDim.x;
  auto load_unit = [&](int tile, int u, u32x4_t (&v)[4]) {
    const int n0 = tile * kSRows, col = (unit0 + u) * 256;
    const int rows = min(max((int)a.n - n0, 0), kSRows);
    const Rsrc r = rsrc_of(wc + (int64_t)n0 * kb + col, max(rows * kb - col, 0));
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = __builtin_amdgcn_raw_buffer_load_b128(r, voff[i], 0, 0);
  };
  // A row tile's scale bytes, from the dword that holds its first one; thread i
  // carries 16 bytes of every 16 * (threads).  Dwords that hold none of the bytes
  // read zero.
  struct Scales {
    u32x4_t v[kChunks];
  };
  auto load_scales = [&](int tile) {
    const int n0 = tile * kSRows, rows = min(max((int)a.n - n0, 0), kSRows);
    const uint8_t* p = wsc + (int64_t)n0 * nb;
    const int skew = (int)((uintptr_t)p & 3);
    const Rsrc r = rsrc_of(p - skew, rows ? (rows * nb + skew + 3) & ~3 : 0);
    Scales s;
#pragma unroll
    for (int i = 0; i < kChunks; i++)
      s.v[i] = __builtin_amdgcn_raw_buffer_load_b128(r, (i * 64 * waves + tid) * 16, 0, 0);
    return s;
  };
  auto keep_scales = [&](const Scales& s, int buf) {
#pragma unroll
    for (int i = 0; i < kChunks; i++) {
      const int at = (i * 64 * waves + tid) * 16;
      if (at < sc_bytes) *(u32x4_t*)(sc + buf * sc_bytes + at) = s.v[i];
    }
  };
  auto skew_of = [&](int tile) { return (int)((uintptr_t)(wsc + (int64_t)tile * kSRows * nb) & 3); };

  int tile = blockIdx.x;
#pragma unroll
  for (int i = 0; i < kSAhead; i++) load_unit(tile + i / U * step, i % U, fw[i]);
  keep_scales(load_scales(tile), 0);
  __syncthreads();

  f32x4_t acc[MT];
  int buf = 0;
  // row tile RT of a round
  auto row_tile = [&](auto which) {
      constexpr int rt = decltype(which)::value;
      const Scales next_sc = load_scales(tile + step);
      const int skew = skew_of(tile);
#pragma unroll
      for (int j = 0; j < MT; j++) acc[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < U; u++) {
        constexpr int kA = kSAhead;
        const int slot = (rt * U + u) % kA;
#pragma unroll
        for (int i = 0; i < 4; i++)
          *(u32x4_t*)(stage + (4 * i + g) * 256 + ((l16 ^ (4 * i + g)) * 16)) = fw[slot][i];
        const int ahead = u + kA;  // the unit that takes this slot
        load_unit(tile + ahead / U * step, ahead % U, fw[slot]);
        // scale bytes of blocks b .. b + 3 of row l16, 0 past K
        const int b = (unit0 + u) * 16 + 4 * g, at = skew + l16 * nb + b;
        const uint32_t* q = (const uint32_t*)(sc + buf * sc_bytes) + (min(at, sc_bytes - 8) >> 2);
        uint32_t dw = __builtin_amdgcn_alignbyte(q[1], q[0], (uint32_t)at & 3u);
        const int have = nb - b;
        dw = have >= 4 ? dw : have <= 0 ? 0u : dw & ((1u << (8 * have)) - 1u);
        wave_lds_sync();
        u32x4_t f[4];
#pragma unroll
        for (int s = 0; s < 4; s++) f[s] = *(const u32x4_t*)(stage + l16 * 256 + (((4 * g + s) ^ l16) * 16));
#pragma unroll
        for (int j = 0; j < MT; j++) {
          acc[j] = mma16<0>(f[0], fx[j][u][0], acc[j], dw, dx[j][u]);
          acc[j] = mma16<1>(f[1], fx[j][u][1], acc[j], dw, dx[j][u]);
          acc[j] = mma16<2>(f[2], fx[j][u][2], acc[j], dw, dx[j][u]);
          acc[j] = mma16<3>(f[3], fx[j][u][3], acc[j], dw, dx[j][u]);
        }
        // the products stay here: moved down, all units' fragments would wait in registers
#pragma unroll
        for (int j = 0; j < MT; j++) asm volatile("" : "+v"(acc[j]));
        wave_lds_sync();
      }
      float* mine = part + (buf * waves + wave) * kPart;
#pragma unroll
      for (int j = 0; j < MT; j++) *(f32x4_t*)(mine + j * 256 + lane * 4) = acc[j];
      keep_scales(next_sc, buf ^ 1);
      __syncthreads();
      for (int o = tid; o < kPart; o += 64 * waves) {
        const int n = o & 15, m = o >> 4;  // lane (n / 4) * 16 + m % 16 holds it in element n % 4
        const float* p = part + buf * waves * kPart + (m >> 4) * 256 + ((n >> 2) * 16 + (m & 15)) * 4 + (n & 3);
        float v = 0.0f;
        for (int w = 0; w < waves; w++) v += p[w * kPart];
        const int64_t row = t.m0 + m, col = (int64_t)tile * kSRows + n;
        if (row < t.m1 && col < a.n) {
          if (a.x_rows) {
            const int64_t r = a.x_rows[row];
            if (r < 0 || r >= a.x_rows_total) v = 0.0f;
          }
          const int64_t at = row * a.n + col;
          if (y_dtype == kF32) ((float*)a.y)[at] = v;
          else if (y_dtype == kF16) ((_Float16*)a.y)[at] = mx_cvt<_Float16>(v);
          else ((__bf16*)a.y)[at] = mx_cvt<__bf16>(v);
        }
      }
      buf ^= 1;
      tile += step;
      return tile < tiles;
  };
  if (tile >= tiles) return;
  while (true) {
    if (!row_tile(std::integral_constant<int, 0>{})) return;
    if constexpr (kTilesRound > 1)
      if (!row_tile(std::integral_constant<int, 1>{})) return;
    if constexpr (kTilesRound > 2) {
      if (!row_tile(std::integral_constant<int, 2>{})) return;
      if (!row_tile(std::integral_constant<int, 3>{})) return;
    }
  }
}

// The stream kernel's shape for a product: U units a wave, waves, MT.
struct StreamPlan {
  int u, waves, mt;  // u = 0: not covered
};
StreamPlan stream_plan(int64_t rows, int64_t k) {
  const int64_t units = (k + kSUnit - 1) / kSUnit;
  const int mt = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  int u = 1;
  while ((int64_t)u * kSMaxWaves < units) u *= 2;
  if (u * mt > 8) return {0, 0, 0};  // X would not fit the registers
  return {u, (int)((units + u - 1) / u), mt};
}

template <int U, int MT> hipError_t go_stream(const Args& a, int y_dtype, const StreamPlan& p, hipStream_t stream) {
  const int nb = (int)(a.k / kMxBlock);
  const int sc_bytes = (kSRows * nb + 4 + 15 + 4) & ~15;
  const size_t lds = (size_t)p.waves * (kSRows * 256 + 2 * 4 * kSRows * 16 * MT) + 2 * sc_bytes;
  const int64_t tiles = (a.n + kSRows - 1) / kSRows;
  const int64_t jobs = a.offsets ? min((a.m + 16 * MT - 1) / (16 * MT) + a.experts, a.m) : (a.m + 16 * MT - 1) / (16 * MT);
  const int64_t slots = (int64_t)device_cu_count() * 2;
  int64_t per = (tiles * jobs + slots - 1) / slots;  // row tiles a workgroup
  if (a.offsets) per = min(per, (int64_t)4);         // many of the jobs may be empty
  const int64_t gx = (tiles + per - 1) / per;
  auto kern = mx_stream_kernel<U, MT>;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kern, dim3((unsigned)gx, (unsigned)jobs), dim3(64 * p.waves), lds, stream, a, y_dtype, p.waves);
  return hipGetLastError();
}

hipError_t run_stream(const Args& a, int y_dtype, const StreamPlan& p, hipStream_t s) {
  switch (p.mt * 16 + p.u) {
    case 17: return go_stream<1, 1>(a, y_dtype, p, s);
    case 18: return go_stream<2, 1>(a, y_dtype, p, s);
    case 20: return go_stream<4, 1>(a, y_dtype, p, s);
    case 24: return go_stream<8, 1>(a, y_dtype, p, s);
    case 33: return go_stream<1, 2>(a, y_dtype, p, s);
    case 34: return go_stream<2, 2>(a, y_dtype, p, s);
    case 36: return go_stream<4, 2>(a, y_dtype, p, s);
    case 65: return go_stream<1, 4>(a, y_dtype, p, s);
    default: return go_stream<2, 4>(a, y_dtype, p, s);
  }
}

template <int BN, int BM, typename OT> hipError_t go_tile(const Args& a, hipStream_t stream) {
  const int64_t nt = (a.n + BN - 1) / BN;
  const int64_t mt = (a.m + BM - 1) / BM + (a.offsets ? min((int64_t)a.experts, a.m) : 0);
  hipLaunchKernelGGL((mx_tile_kernel<BN, BM, OT>), dim3((unsigned)(nt * mt)), dim3(256), 0, stream, a, mt);
  return hipGetLastError();
}

template <typename OT> hipError_t run(const Args& a, hipStream_t stream) {
  return go_tile<256, 256, OT>(a, stream);
}

}  // namespace

size_t mx_gemm_ws_bytes(int64_t, int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_mx_gemm(const MxGemm& g, void*, size_t, hipStream_t stream) {
  if (g.m == 0 || g.n == 0) return hipSuccess;
  const Args a = {g.x.codes, g.x.scales, g.w.codes, g.w.scales, g.m, g.n, g.k, g.x.rows, g.y, g.offsets, g.x_rows,
                  g.experts};
  // rows of one product: of one expert, on average
  const int64_t rows = g.offsets ? (g.m + g.experts - 1) / g.experts : g.m;
  if (rows <= 64) {
    const StreamPlan p = stream_plan(rows, g.k);
    if (p.u) return run_stream(a, g.y_dtype, p, stream);
  }
  if (g.y_dtype == kF32) return run<float>(a, stream);
  if (g.y_dtype == kF16) return run<_Float16>(a, stream);
  return run<__bf16>(a, stream);
}

}  // namespace rz
