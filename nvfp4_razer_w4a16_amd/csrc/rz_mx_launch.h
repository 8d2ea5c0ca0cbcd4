// rz_mx_launch.h -- internal launcher interface of the MXFP4 operators and the
// block norm.  Host-only declarations; no torch types.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace rz {

struct MxView {
  int64_t rows, cols;
  uint8_t* codes;   // rows * cols / 2 bytes
  uint8_t* scales;  // rows * cols / 32 bytes
};

// x: [rows, cols] with `stride` elements from row to row.  gated: x is
// [rows, 2 * cols], the packed value is silu(x[:, c]) * x[:, cols + c].
hipError_t launch_mx_quantize(const void* x, int dtype, int64_t stride, bool gated, const MxView& out,
                              hipStream_t stream);
hipError_t launch_mx_dequant(const MxView& t, void* out, int out_dtype, hipStream_t stream);

struct MxGemm {
  MxView x, w;
  void* y;
  int y_dtype;
  int64_t m, n, k;           // output rows, columns (of one expert), reduction length
  const int32_t* offsets;    // device, experts + 1 row offsets, or NULL for one product
  const int32_t* x_rows;     // device, m row numbers of x, or NULL
  int experts;
};
size_t mx_gemm_ws_bytes(int64_t m, int64_t n, int64_t k, int64_t experts);
hipError_t launch_mx_gemm(const MxGemm& g, void* ws, size_t ws_bytes, hipStream_t stream);

struct BlockNorm {
  int64_t rows, cols;
  const void *y, *h;         // [rows, cols]; y may be NULL
  int64_t y_stride, h_stride;
  int dtype;                 // of y, h, the weights, the gate and the 16/32-bit outputs
  const void *post, *pre;    // [cols] or NULL: no weight
  const void* gate;          // [gate_rows, cols] or NULL
  int64_t gate_rows;
  float scale, eps;
  bool norm_y;               // whether y is normalised
  void *h_out, *x_out;       // [rows, cols], either may be NULL
  MxView packed;             // codes NULL: no packed output
};
// Lanes that a row of the block norm is spread over.
inline int block_norm_lanes(int64_t cols) { return cols <= 1024 ? 64 : cols <= 8192 ? 256 : 1024; }
// Threads of its workgroups: short rows share one.
inline int block_norm_threads(int64_t cols) { return block_norm_lanes(cols) < 256 ? 256 : block_norm_lanes(cols); }
hipError_t launch_block_norm(const BlockNorm& b, hipStream_t stream);

int device_cu_count();

}  // namespace rz
