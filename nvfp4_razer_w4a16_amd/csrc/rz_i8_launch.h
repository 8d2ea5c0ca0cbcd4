// rz_i8_launch.h -- internal launcher interface of the 8-bit integer operators.
// Host-only declarations; no torch types.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace rz {

struct I8View {
  int64_t rows, cols;
  int8_t* codes;   // rows * cols bytes
  float* scales;   // rows
};

// x: [rows, cols] with `stride` elements from row to row.  gated: x is
// [rows, 2 * cols], the encoded value is silu(x[:, c]) * x[:, cols + c].
hipError_t launch_i8_quantize(const void* x, int dtype, int64_t stride, bool gated, const I8View& out,
                              hipStream_t stream);
hipError_t launch_i8_dequant(const I8View& t, void* out, int out_dtype, hipStream_t stream);

struct I8Gemm {
  I8View x, w;
  void* y;
  int y_dtype;
  int64_t m, n, k;           // output rows, columns (of one expert), reduction length
  const int32_t* offsets;    // device, experts + 1 row offsets, or NULL for one product
  const int32_t* x_rows;     // device, m row numbers of x, or NULL
  int experts;
};
size_t i8_gemm_ws_bytes(int64_t m, int64_t n, int64_t k, int64_t experts);
hipError_t launch_i8_gemm(const I8Gemm& g, void* ws, hipStream_t stream);

int device_cu_count();

}  // namespace rz
