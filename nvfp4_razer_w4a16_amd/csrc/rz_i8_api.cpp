// rz_i8_api.cpp -- the extern "C" entry points of the 8-bit integer operators, the
// routing to experts and the combination of their rows (see include/librazer.h).
//
// Host-side argument checks, synchronous, before anything is enqueued; then the
// launchers on the caller's stream.  No allocation, no synchronisation, no
// exceptions cross the ABI.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "../../include/librazer.h"
#include "rz_i8_launch.h"
#include "rz_moe_launch.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool dtype_ok(int dt) { return dt == RAZER_F32 || dt == RAZER_F16 || dt == RAZER_BF16; }
int64_t dtype_size(int dt) { return dt == RAZER_F32 ? 4 : 2; }

constexpr int64_t kMaxElems = (int64_t)1 << 34;   // 8 elements a thread, a launch has fewer than 2^32 threads
                                                  // (in each dimension: the combination, of 4 or 8, has two)
constexpr int64_t kMaxGemmRows = (int64_t)1 << 30;
constexpr int64_t kMaxPairs = (int64_t)1 << 30;   // of a token and a place
constexpr int64_t kMaxTokens = (int64_t)1 << 26;  // blocks of 1024 threads, 16 or 32 tokens each, in one launch
// Every block reads the sums of all groups of blocks, which grows with the square of the
// tokens: 8 of 256 experts of 65536 tokens 44 of the 127 us of a call, of 2^20 1.5 of 2.5 ms.
constexpr int64_t kMaxOrdered = (int64_t)1 << 20;

razer_status check_i8(const razer_i8* t) {
  if (!t || t->rows < 0 || t->cols < 0 || t->cols % 16 != 0) return RAZER_E_INVALID;
  if (t->cols > 0 && t->rows > INT64_MAX / 16 / t->cols) return RAZER_E_INVALID;
  if (t->rows * t->cols > 0 && (!t->codes || !aligned(t->codes, 16))) return RAZER_E_INVALID;
  if (t->rows > 0 && (!t->scales || !aligned(t->scales, 4))) return RAZER_E_INVALID;
  return RAZER_OK;
}

// A [rows, cols] operand of `stride` elements from row to row: 16-byte rows.
bool strided_ok(const void* p, int64_t stride, int64_t cols, int dt) {
  if (!p || !aligned(p, 16) || stride < cols || stride >= INT64_MAX / 8) return false;
  return stride * dtype_size(dt) % 16 == 0;
}

// A [rows, cols] operand of any stride: elements aligned, addresses within 64 bits.
bool rows_ok(const void* p, int64_t rows, int64_t stride, int64_t cols, int dt) {
  return p && aligned(p, (uintptr_t)dtype_size(dt)) && stride >= cols && (rows == 0 || stride <= INT64_MAX / 16 / rows);
}

rz::I8View view_of(const razer_i8* t) { return {t->rows, t->cols, t->codes, t->scales}; }

razer_status status_of(hipError_t e) { return e == hipSuccess ? RAZER_OK : RAZER_E_HIP; }

razer_status quantize(const void* x, razer_dtype dt, int64_t stride, bool gated, const razer_i8* out, void* stream) {
  const razer_status s = check_i8(out);
  if (s != RAZER_OK) return s;
  if (!dtype_ok(dt)) return RAZER_E_INVALID;
  if (out->rows == 0) return RAZER_OK;
  if (out->cols == 0) return RAZER_E_UNSUPPORTED;  // rows without elements have no maximum
  if (out->cols > INT64_MAX / 8) return RAZER_E_INVALID;
  if (!strided_ok(x, stride, out->cols * (gated ? 2 : 1), dt) || out->rows > INT64_MAX / 16 / stride)
    return RAZER_E_INVALID;
  if (out->rows > kMaxElems / out->cols || out->cols > INT32_MAX) return RAZER_E_UNSUPPORTED;
  return status_of(rz::launch_i8_quantize(x, dt, stride, gated, view_of(out), (hipStream_t)stream));
}

// The sizes a product accepts; `m` output rows.
razer_status check_gemm(const razer_i8* x, const razer_i8* w, int64_t m, razer_dtype y_dt) {
  razer_status s = check_i8(x);
  if (s != RAZER_OK) return s;
  s = check_i8(w);
  if (s != RAZER_OK) return s;
  if (!dtype_ok(y_dt) || x->cols != w->cols || m < 0) return RAZER_E_INVALID;
  if (x->cols == 0 || x->cols > RAZER_I8_MAX_K || m > kMaxGemmRows || w->rows > kMaxGemmRows)
    return RAZER_E_UNSUPPORTED;
  return RAZER_OK;
}

}  // namespace

extern "C" {

razer_status razer_i8_quantize(const void* x, razer_dtype x_dt, int64_t x_stride, const razer_i8* out, void* stream) {
  return quantize(x, x_dt, x_stride, false, out, stream);
}

razer_status razer_i8_quantize_gated(const void* gu, razer_dtype gu_dt, int64_t gu_stride, const razer_i8* out,
                                     void* stream) {
  return quantize(gu, gu_dt, gu_stride, true, out, stream);
}

razer_status razer_i8_dequant(const razer_i8* t, void* out, razer_dtype out_dt, void* stream) {
  const razer_status s = check_i8(t);
  if (s != RAZER_OK) return s;
  if (!dtype_ok(out_dt)) return RAZER_E_INVALID;
  if (t->rows == 0 || t->cols == 0) return RAZER_OK;
  if (!out || !aligned(out, 16)) return RAZER_E_INVALID;
  if (t->rows > kMaxElems / t->cols || t->cols > INT32_MAX) return RAZER_E_UNSUPPORTED;
  return status_of(rz::launch_i8_dequant(view_of(t), out, out_dt, (hipStream_t)stream));
}

razer_status razer_i8_gemm(const razer_i8* x, const razer_i8* w, void* y, razer_dtype y_dt, void* ws, size_t ws_bytes,
                           void* stream) {
  const razer_status s = check_gemm(x, w, x ? x->rows : 0, y_dt);
  if (s != RAZER_OK) return s;
  if (x->rows == 0 || w->rows == 0) return RAZER_OK;
  if (!y || !aligned(y, 16)) return RAZER_E_INVALID;
  const size_t need = rz::i8_gemm_ws_bytes(x->rows, w->rows, x->cols, 0);
  if (need > 0 && (!ws || ws_bytes < need || !aligned(ws, 16))) return RAZER_E_INVALID;
  const rz::I8Gemm g = {view_of(x), view_of(w), y,       y_dt,    x->rows, w->rows,
                        x->cols,    nullptr,    nullptr, 0};
  return status_of(rz::launch_i8_gemm(g, ws, (hipStream_t)stream));
}

razer_status razer_i8_gemm_grouped(const razer_i8* x, const razer_i8* w, const int32_t* offsets, int64_t experts,
                                   const int32_t* x_rows, int64_t m, void* y, razer_dtype y_dt, void* ws,
                                   size_t ws_bytes, void* stream) {
  const razer_status s = check_gemm(x, w, m, y_dt);
  if (s != RAZER_OK) return s;
  if (experts < 1 || experts > RAZER_MX_MAX_EXPERTS || w->rows % experts != 0) return RAZER_E_INVALID;
  if (m == 0 || w->rows == 0) return RAZER_OK;
  if (!x_rows && m != x->rows) return RAZER_E_INVALID;
  if (x->rows == 0 || !offsets || !aligned(offsets, 4) || !aligned(x_rows, 4)) return RAZER_E_INVALID;
  if (x->rows > kMaxGemmRows || (x_rows && x->rows * x->cols > UINT32_MAX)) return RAZER_E_UNSUPPORTED;
  if (!y || !aligned(y, 16)) return RAZER_E_INVALID;
  const size_t need = rz::i8_gemm_ws_bytes(m, w->rows / experts, x->cols, experts);
  if (need > 0 && (!ws || ws_bytes < need || !aligned(ws, 16))) return RAZER_E_INVALID;
  const rz::I8Gemm g = {view_of(x), view_of(w), y,      y_dt,        m, w->rows / experts,
                        x->cols,    offsets,    x_rows, (int)experts};
  return status_of(rz::launch_i8_gemm(g, ws, (hipStream_t)stream));
}

size_t razer_i8_workspace_bytes(int64_t m, int64_t n, int64_t k, int64_t experts) {
  if (m <= 0 || n <= 0 || k <= 0 || experts < 0) return 0;
  if (m > kMaxGemmRows || n > kMaxGemmRows || k > RAZER_I8_MAX_K || experts > RAZER_MX_MAX_EXPERTS) return 0;  // refused
  return rz::i8_gemm_ws_bytes(m, n, k, experts);
}

razer_status razer_moe_route(const razer_route* a, void* ws, size_t ws_bytes, void* stream) {
  if (!a || a->tokens < 0 || a->experts < 1 || a->top < 1 || a->groups < 1 || a->groups > RAZER_MOE_MAX_GROUPS)
    return RAZER_E_INVALID;
  if (a->experts > RAZER_MOE_MAX_EXPERTS || a->top > RAZER_MOE_MAX_TOP) return RAZER_E_UNSUPPORTED;
  if (a->experts % a->groups != 0 || a->groups_kept < 1 || a->groups_kept > a->groups) return RAZER_E_INVALID;
  if (a->group_best < 1 || a->group_best > 2 || a->top > a->experts / a->groups * a->groups_kept) return RAZER_E_INVALID;
  if (a->score != RAZER_SCORE_SOFTMAX && a->score != RAZER_SCORE_SIGMOID) return RAZER_E_INVALID;
  if (!dtype_ok(a->dtype) || (a->flags & ~(uint32_t)RAZER_ROUTE_RENORM)) return RAZER_E_INVALID;
  const bool order = a->offsets != nullptr;
  if (order ? a->tokens > 0 && (!a->rows || !a->slots) : a->rows || a->slots) return RAZER_E_INVALID;
  const void* words[] = {a->bias, a->chosen, a->weights, a->offsets, a->rows, a->slots};
  for (const void* p : words)
    if (!aligned(p, 4)) return RAZER_E_INVALID;
  if (a->tokens >= kMaxPairs / a->top || a->tokens > (order ? kMaxOrdered : kMaxTokens)) return RAZER_E_UNSUPPORTED;
  if (a->tokens > 0) {
    if (!a->chosen || !a->weights || !rows_ok(a->logits, a->tokens, a->stride, a->experts, a->dtype))
      return RAZER_E_INVALID;
  } else if (!order) {
    return RAZER_OK;
  }
  const size_t need = order ? rz::moe_route_ws_bytes(a->tokens, a->experts, a->top) : 0;
  if (need > 0 && (!ws || ws_bytes < need || !aligned(ws, 16))) return RAZER_E_INVALID;
  rz::MoeRoute r = {};
  r.tokens = a->tokens;
  r.stride = a->stride;
  r.experts = a->experts;
  r.top = a->top;
  r.groups = a->groups;
  r.kept = a->groups_kept;
  r.best = a->group_best;
  r.sigmoid = a->score == RAZER_SCORE_SIGMOID;
  r.renorm = (a->flags & RAZER_ROUTE_RENORM) != 0;
  r.dtype = a->dtype;
  r.scale = a->scale;
  r.logits = a->logits;
  r.bias = a->bias;
  r.chosen = a->chosen;
  r.weights = a->weights;
  r.offsets = a->offsets;
  r.rows = a->rows;
  r.slots = a->slots;
  return status_of(rz::launch_moe_route(r, ws, (hipStream_t)stream));
}

size_t razer_moe_workspace_bytes(int64_t tokens, int64_t experts, int64_t top) {
  if (tokens < 0 || experts < 1 || experts > RAZER_MOE_MAX_EXPERTS || top < 1 || top > RAZER_MOE_MAX_TOP) return 0;
  if (tokens > kMaxOrdered || tokens >= kMaxPairs / top) return 0;  // refused
  return rz::moe_route_ws_bytes(tokens, experts, top);
}

razer_status razer_moe_combine(const razer_combine* a, void* stream) {
  if (!a || a->tokens < 0 || a->cols < 0 || a->y_rows < 0 || a->top < 1 || !dtype_ok(a->dtype)) return RAZER_E_INVALID;
  if (a->top > RAZER_MOE_MAX_TOP) return RAZER_E_UNSUPPORTED;
  if (a->tokens == 0 || a->cols == 0) return RAZER_OK;
  if (a->tokens > INT64_MAX / 16 / a->cols) return RAZER_E_INVALID;
  if (a->tokens >= kMaxPairs / a->top || a->y_rows > INT32_MAX || a->cols > INT32_MAX || a->tokens > kMaxElems / a->cols)
    return RAZER_E_UNSUPPORTED;
  if (a->y_rows > 0 && !rows_ok(a->y, a->y_rows, a->y_stride, a->cols, a->dtype)) return RAZER_E_INVALID;
  if (a->add && !rows_ok(a->add, a->tokens, a->add_stride, a->cols, a->dtype)) return RAZER_E_INVALID;
  if (!a->slots || !a->weights || !aligned(a->slots, 4) || !aligned(a->weights, 4)) return RAZER_E_INVALID;
  if (!a->out || !aligned(a->out, (uintptr_t)dtype_size(a->dtype))) return RAZER_E_INVALID;
  const rz::MoeCombine c = {a->tokens, a->cols, a->y_rows,  a->y_stride, a->add_stride, (int)a->top,
                            a->dtype,  a->y,    a->slots,   a->weights,  a->add,        a->out};
  return status_of(rz::launch_moe_combine(c, (hipStream_t)stream));
}

}  // extern "C"
