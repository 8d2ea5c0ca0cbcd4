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

#include "rz_groups.h"
#include "rz_i8.h"
#include "rz_i8_launch.h"

namespace rz {

namespace {

struct Args {
  const int8_t *xc, *wc;
  const float *xs, *ws;
  int64_t m, n, k, x_rows_total;
  void* y;
  const int32_t* offsets;
  const int32_t* x_rows;
  int experts;
};

// A 64x64 tile of y per workgroup of four waves, a 32x32 quarter each.
template <typename OT, bool GROUPED> __device__ void i8_tile(const Args& a, int64_t im, int64_t in) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5, l32 = lane & 31;
  Tile t = {im * 64, min(im * 64 + 64, a.m), 0};
  if (GROUPED) t = find_tile(a.offsets, a.experts, a.m, 64, im);
  if (t.expert < 0) return;
  const int64_t n0 = in * 64 + (wave & 1) * 32, m = t.m0 + (wave >> 1) * 32 + l32;
  if (n0 >= a.n) return;
  const int64_t wr = t.expert * a.n + min(n0 + l32, a.n - 1);
  int64_t xr = min(m, t.m1 - 1);
  bool none = false;
  if (GROUPED && a.x_rows) {
    xr = a.x_rows[xr];
    none = xr < 0 || xr >= a.x_rows_total;
    if (none) xr = 0;
  }
  const int8_t *pw = a.wc + wr * a.k, *px = a.xc + xr * a.k;
  i32x16_t acc = {};
  for (int64_t k = half * 16; k - half * 16 < a.k; k += 32) {
    i32x4_t fw = {}, fx = {};
    if (k < a.k) {
      fw = *(const i32x4_t*)(pw + k);
      fx = *(const i32x4_t*)(px + k);
    }
    acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw, fx, acc, 0, 0, 0);
  }
  if (m >= t.m1) return;
  const float sx = a.xs[xr];
  OT* y = (OT*)a.y + m * a.n;
#pragma unroll
  for (int i = 0; i < 16; i++) {
    const int64_t n = n0 + 8 * (i >> 2) + 4 * half + (i & 3);
    if (n < a.n) y[n] = none ? (OT)0.0f : mx_cvt<OT>(i8_scaled(acc[i], sx, a.ws[t.expert * a.n + n]));
  }
}

template <typename OT, bool GROUPED> __global__ __launch_bounds__(256) void i8_tile_kernel(Args a, int64_t mt, int64_t nt) {
  for (int64_t i = blockIdx.x; i < mt * nt; i += gridDim.x) i8_tile<OT, GROUPED>(a, i / nt, i % nt);
}

template <typename OT> hipError_t run(const Args& a, hipStream_t stream) {
  const int64_t mt = (a.m + 63) / 64 + (a.offsets ? std::min((int64_t)a.experts, a.m) : 0), nt = (a.n + 63) / 64;
  const dim3 grid((unsigned)std::min(mt * nt, (int64_t)1 << 20));
  if (a.offsets) hipLaunchKernelGGL((i8_tile_kernel<OT, true>), grid, dim3(256), 0, stream, a, mt, nt);
  else hipLaunchKernelGGL((i8_tile_kernel<OT, false>), grid, dim3(256), 0, stream, a, mt, nt);
  return hipGetLastError();
}

}  // namespace

size_t i8_gemm_ws_bytes(int64_t, int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_i8_gemm(const I8Gemm& g, void*, hipStream_t stream) {
  const Args a = {g.x.codes, g.w.codes, g.x.scales, g.w.scales, g.m, g.n, g.k, g.x.rows, g.y, g.offsets, g.x_rows,
                  g.experts};
  if (g.y_dtype == kF32) return run<float>(a, stream);
  if (g.y_dtype == kF16) return run<_Float16>(a, stream);
  return run<__bf16>(a, stream);
}

}  // namespace rz
