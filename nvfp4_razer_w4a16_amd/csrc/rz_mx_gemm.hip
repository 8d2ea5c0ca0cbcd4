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
// A 128x128 tile of y per workgroup of four waves (2x2), 256 elements of K a
// step through LDS.  A tile row is 128 bytes of codes, eight 16-byte chunks;
// chunk c of row r lies at place c ^ (r & 7), so the lanes of a fragment read
// (one chunk of 32 rows) spread over the banks.
constexpr int kT = 128, kStep = 256, kRowB = kStep / 2;

template <typename OT> __global__ __launch_bounds__(256) void mx_tile_kernel(Args a) {
  __shared__ __attribute__((aligned(16))) uint8_t lw[kT * kRowB], lx[kT * kRowB];
  const Tile t = find_tile(a, kT, blockIdx.y);
  if (t.expert < 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t n0 = (int64_t)blockIdx.x * kT;
  const int nb = (int)(a.k / kMxBlock);
  const int64_t kb = a.k / 2;  // code bytes of a row
  auto w_row = [&](int r) { return (int64_t)t.expert * a.n + min(n0 + r, a.n - 1); };
  auto x_row = [&](int r) -> int64_t {
    const int64_t row = min(t.m0 + r, t.m1 - 1);
    return a.x_rows ? min((int64_t)max(a.x_rows[row], 0), a.x_rows_total - 1) : row;
  };
  // this thread's four chunks of either tile
  const uint8_t *pw[4], *px[4];
  int place[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int r = i * 32 + (tid >> 3);
    pw[i] = a.wc + w_row(r) * kb;
    px[i] = a.xc + x_row(r) * kb;
    place[i] = r * kRowB + (((tid & 7) ^ (r & 7)) * 16);
  }
  const int wn = (wave & 1) * 64, wm = (wave >> 1) * 64;
  const int half = lane >> 5, l32 = lane & 31;
  const uint8_t *sw[2], *sx[2];
#pragma unroll
  for (int i = 0; i < 2; i++) {
    sw[i] = a.ws + w_row(wn + i * 32 + l32) * nb;
    sx[i] = a.xs + x_row(wm + i * 32 + l32) * nb;
  }
  f32x16_t acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; i++)
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
      for (int e = 0; e < 16; e++) acc[i][j][e] = 0.0f;
  const int steps = (nb + 7) / 8;
  for (int s = 0; s < steps; s++) {
    const int c = min(s * 8 + (tid & 7), nb - 1);
    u32x4_t vw[4], vx[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      vw[i] = *(const u32x4_t*)(pw[i] + c * 16);
      vx[i] = *(const u32x4_t*)(px[i] + c * 16);
    }
    uint32_t dw[2], dx[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
      dw[i] = scales4(sw[i], s * 8 + half * 4, nb);
      dx[i] = scales4(sx[i], s * 8 + half * 4, nb);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; i++) {
      *(u32x4_t*)(lw + place[i]) = vw[i];
      *(u32x4_t*)(lx + place[i]) = vx[i];
    }
    __syncthreads();
    auto sub = [&](auto kk) {
      constexpr int I = decltype(kk)::value;
      u32x4_t fw[2], fx[2];
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const int rw = wn + i * 32 + l32, rx = wm + i * 32 + l32;
        fw[i] = *(const u32x4_t*)(lw + rw * kRowB + (((half * 4 + I) ^ (rw & 7)) * 16));
        fx[i] = *(const u32x4_t*)(lx + rx * kRowB + (((half * 4 + I) ^ (rx & 7)) * 16));
      }
#pragma unroll
      for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 2; j++) acc[i][j] = mma<I>(fw[i], fx[j], acc[i][j], dw[i], dx[j]);
    };
    sub(std::integral_constant<int, 0>{});
    sub(std::integral_constant<int, 1>{});
    sub(std::integral_constant<int, 2>{});
    sub(std::integral_constant<int, 3>{});
  }
#pragma unroll
  for (int j = 0; j < 2; j++) {
    const int64_t row = t.m0 + wm + j * 32 + l32;
    if (row >= t.m1) continue;
    bool none = false;
    if (a.x_rows) {
      const int64_t r = a.x_rows[row];
      none = r < 0 || r >= a.x_rows_total;
    }
#pragma unroll
    for (int i = 0; i < 2; i++)
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

template <typename OT> hipError_t run(const Args& a, hipStream_t stream) {
  const int64_t gx = (a.n + kT - 1) / kT;
  const int64_t gy = (a.m + kT - 1) / kT + (a.offsets ? min((int64_t)a.experts, a.m) : 0);
  hipLaunchKernelGGL(mx_tile_kernel<OT>, dim3((unsigned)gx, (unsigned)gy), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

size_t mx_gemm_ws_bytes(int64_t, int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_mx_gemm(const MxGemm& g, void*, size_t, hipStream_t stream) {
  if (g.m == 0 || g.n == 0) return hipSuccess;
  const Args a = {g.x.codes, g.x.scales, g.w.codes, g.w.scales, g.m, g.n, g.k, g.x.rows, g.y, g.offsets, g.x_rows,
                  g.experts};
  if (g.y_dtype == kF32) return run<float>(a, stream);
  if (g.y_dtype == kF16) return run<_Float16>(a, stream);
  return run<__bf16>(a, stream);
}

}  // namespace rz
