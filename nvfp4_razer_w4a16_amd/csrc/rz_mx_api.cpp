// rz_mx_api.cpp -- the extern "C" entry points of the MXFP4 operators and the
// block norm (see include/librazer.h).
//
// Host-side argument checks, synchronous, before anything is enqueued; then the
// launchers on the caller's stream.  No allocation, no synchronisation, no
// exceptions cross the ABI.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "../../include/librazer.h"
#include "rz_mx_launch.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool dtype_ok(int dt) { return dt == RAZER_F32 || dt == RAZER_F16 || dt == RAZER_BF16; }
int64_t dtype_size(int dt) { return dt == RAZER_F32 ? 4 : 2; }

constexpr int64_t kMaxElems = (int64_t)1 << 34;   // 8 elements a thread, a launch has fewer than 2^32 threads
constexpr int64_t kMaxGemmRows = (int64_t)1 << 30;
constexpr int64_t kMaxGemmK = (int64_t)1 << 23;   // the rows of a tile within 32 bits
constexpr int64_t kMaxNormCols = 32768;           // 1024 threads of at most four 8-element chunks

razer_status check_mx(const razer_mx* t) {
  if (!t || t->rows < 0 || t->cols < 0 || t->cols % 32 != 0) return RAZER_E_INVALID;
  if (t->cols > 0 && t->rows > INT64_MAX / 4 / t->cols) return RAZER_E_INVALID;
  if (t->rows * t->cols > 0 && (!t->codes || !t->scales || !aligned(t->codes, 16))) return RAZER_E_INVALID;
  return RAZER_OK;
}

// A [rows, cols] operand of `stride` elements from row to row: 16-byte rows.
bool strided_ok(const void* p, int64_t stride, int64_t cols, int dt) {
  if (!p || !aligned(p, 16) || stride < cols || stride >= INT64_MAX / 8) return false;
  return stride * dtype_size(dt) % 16 == 0;
}

rz::MxView view_of(const razer_mx* t) { return {t->rows, t->cols, t->codes, t->scales}; }

razer_status status_of(hipError_t e) { return e == hipSuccess ? RAZER_OK : RAZER_E_HIP; }

razer_status quantize(const void* x, razer_dtype dt, int64_t stride, bool gated, const razer_mx* out, void* stream) {
  const razer_status s = check_mx(out);
  if (s != RAZER_OK) return s;
  if (!dtype_ok(dt)) return RAZER_E_INVALID;
  if (out->rows * out->cols == 0) return RAZER_OK;
  if (!strided_ok(x, stride, out->cols * (gated ? 2 : 1), dt) || out->rows > INT64_MAX / 16 / stride)
    return RAZER_E_INVALID;
  if (out->rows * out->cols > kMaxElems || out->cols > INT32_MAX) return RAZER_E_UNSUPPORTED;
  return status_of(rz::launch_mx_quantize(x, dt, stride, gated, view_of(out), (hipStream_t)stream));
}

// The sizes a product accepts; `m` output rows.
razer_status check_gemm(const razer_mx* x, const razer_mx* w, int64_t m, razer_dtype y_dt) {
  razer_status s = check_mx(x);
  if (s != RAZER_OK) return s;
  s = check_mx(w);
  if (s != RAZER_OK) return s;
  if (!dtype_ok(y_dt) || x->cols != w->cols || m < 0) return RAZER_E_INVALID;
  if (x->cols == 0 || x->cols > kMaxGemmK || m > kMaxGemmRows || w->rows > kMaxGemmRows) return RAZER_E_UNSUPPORTED;
  return RAZER_OK;
}

}  // namespace

extern "C" {

razer_status razer_mx_quantize(const void* x, razer_dtype x_dt, int64_t x_stride, const razer_mx* out, void* stream) {
  return quantize(x, x_dt, x_stride, false, out, stream);
}

razer_status razer_mx_quantize_gated(const void* gu, razer_dtype gu_dt, int64_t gu_stride, const razer_mx* out,
                                     void* stream) {
  return quantize(gu, gu_dt, gu_stride, true, out, stream);
}

razer_status razer_mx_dequant(const razer_mx* t, void* out, razer_dtype out_dt, void* stream) {
  const razer_status s = check_mx(t);
  if (s != RAZER_OK) return s;
  if (!dtype_ok(out_dt)) return RAZER_E_INVALID;
  if (t->rows * t->cols == 0) return RAZER_OK;
  if (!out || !aligned(out, 16)) return RAZER_E_INVALID;
  if (t->rows * t->cols > kMaxElems) return RAZER_E_UNSUPPORTED;
  return status_of(rz::launch_mx_dequant(view_of(t), out, out_dt, (hipStream_t)stream));
}

razer_status razer_mx_gemm(const razer_mx* x, const razer_mx* w, void* y, razer_dtype y_dt, void* ws, size_t ws_bytes,
                           void* stream) {
  const razer_status s = check_gemm(x, w, x ? x->rows : 0, y_dt);
  if (s != RAZER_OK) return s;
  if (x->rows == 0 || w->rows == 0) return RAZER_OK;
  if (!y || !aligned(y, 16)) return RAZER_E_INVALID;
  const size_t need = rz::mx_gemm_ws_bytes(x->rows, w->rows, x->cols, 0);
  if (need > 0 && (!ws || ws_bytes < need || !aligned(ws, 16))) return RAZER_E_INVALID;
  const rz::MxGemm g = {view_of(x), view_of(w), y,       y_dt,    x->rows, w->rows,
                        x->cols,    nullptr,    nullptr, 0};
  return status_of(rz::launch_mx_gemm(g, ws, ws_bytes, (hipStream_t)stream));
}

razer_status razer_mx_gemm_grouped(const razer_mx* x, const razer_mx* w, const int32_t* offsets, int64_t experts,
                                   const int32_t* x_rows, int64_t m, void* y, razer_dtype y_dt, void* ws,
                                   size_t ws_bytes, void* stream) {
  const razer_status s = check_gemm(x, w, m, y_dt);
  if (s != RAZER_OK) return s;
  if (experts < 1 || experts > RAZER_MX_MAX_EXPERTS || w->rows % experts != 0) return RAZER_E_INVALID;
  if (m == 0 || w->rows == 0) return RAZER_OK;
  if (!x_rows && m != x->rows) return RAZER_E_INVALID;
  if (x->rows == 0 || !offsets || !aligned(offsets, 4) || !aligned(x_rows, 4)) return RAZER_E_INVALID;
  if (x->rows > kMaxGemmRows || (x_rows && x->rows * x->cols / 2 > UINT32_MAX)) return RAZER_E_UNSUPPORTED;
  if (!y || !aligned(y, 16)) return RAZER_E_INVALID;
  const size_t need = rz::mx_gemm_ws_bytes(m, w->rows / experts, x->cols, experts);
  if (need > 0 && (!ws || ws_bytes < need || !aligned(ws, 16))) return RAZER_E_INVALID;
  const rz::MxGemm g = {view_of(x), view_of(w), y,      y_dt,        m, w->rows / experts,
                        x->cols,    offsets,    x_rows, (int)experts};
  return status_of(rz::launch_mx_gemm(g, ws, ws_bytes, (hipStream_t)stream));
}

razer_status razer_block_norm(const razer_norm* a, void* stream) {
  if (!a || !dtype_ok(a->dtype) || a->rows < 0 || a->cols < 0 || a->cols % 32 != 0) return RAZER_E_INVALID;
  if (a->flags & ~(uint32_t)RAZER_NORM_POST) return RAZER_E_INVALID;
  if (a->cols > 0 && a->rows > INT64_MAX / 16 / a->cols) return RAZER_E_INVALID;
  if (a->gate && (a->gate_rows < 1 || a->rows % a->gate_rows != 0)) return RAZER_E_INVALID;
  if (a->packed) {
    const razer_status s = check_mx(a->packed);
    if (s != RAZER_OK) return s;
    if (a->packed->rows != a->rows || a->packed->cols != a->cols) return RAZER_E_INVALID;
  }
  if (a->rows * a->cols == 0) return RAZER_OK;
  if (!a->y && ((a->flags & RAZER_NORM_POST) || a->gate)) return RAZER_E_INVALID;
  if (!a->h_out && !a->x_out && !a->packed) return RAZER_E_INVALID;
  if (!strided_ok(a->h, a->h_stride, a->cols, a->dtype) || a->rows > INT64_MAX / 16 / a->h_stride)
    return RAZER_E_INVALID;
  if (a->y && (!strided_ok(a->y, a->y_stride, a->cols, a->dtype) || a->rows > INT64_MAX / 16 / a->y_stride))
    return RAZER_E_INVALID;
  const void* others[] = {a->post_weight, a->pre_weight, a->gate, a->h_out, a->x_out};
  for (const void* p : others)
    if (!aligned(p, 16)) return RAZER_E_INVALID;
  const int lanes = rz::block_norm_lanes(a->cols), threads = rz::block_norm_threads(a->cols);
  if (a->cols > kMaxNormCols || a->rows > (int64_t)(UINT32_MAX / threads) * (threads / lanes)) return RAZER_E_UNSUPPORTED;
  rz::BlockNorm b = {};
  b.rows = a->rows;
  b.cols = a->cols;
  b.y = a->y;
  b.h = a->h;
  b.y_stride = a->y_stride;
  b.h_stride = a->h_stride;
  b.dtype = a->dtype;
  b.post = a->post_weight;
  b.pre = a->pre_weight;
  b.gate = a->gate;
  b.gate_rows = a->gate_rows;
  b.scale = a->residual_scale;
  b.eps = a->eps;
  b.norm_y = (a->flags & RAZER_NORM_POST) != 0;
  b.h_out = a->h_out;
  b.x_out = a->x_out;
  if (a->packed) b.packed = view_of(a->packed);
  return status_of(rz::launch_block_norm(b, (hipStream_t)stream));
}

size_t razer_mx_workspace_bytes(int64_t m, int64_t n, int64_t k, int64_t experts) {
  if (m <= 0 || n <= 0 || k <= 0 || experts < 0) return 0;
  if (m > kMaxGemmRows || n > kMaxGemmRows || k > kMaxGemmK || experts > RAZER_MX_MAX_EXPERTS) return 0;  // refused
  return rz::mx_gemm_ws_bytes(m, n, k, experts);
}

}  // extern "C"
