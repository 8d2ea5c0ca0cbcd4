// i8_host_check.cpp -- test infrastructure only (tests/test_i8_sanitizers.py): a host
// build of rz_i8_api.cpp against stub launchers, run under AddressSanitizer and
// UndefinedBehaviorSanitizer.  Every entry point is called with accepted arguments and
// with sizes at the ends of 64 bits (fake, never dereferenced device addresses); the
// stubs count the launches.  Exit status 0 and no sanitizer report means clean.
#include <hip/hip_runtime.h>

#include <stdint.h>
#include <stdio.h>

#include "../../include/librazer.h"
#include "rz_i8_launch.h"
#include "rz_moe_launch.h"

namespace {
int g_launches = 0, g_fail = 0;
hipError_t g_status = hipSuccess;
hipError_t counted() {
  g_launches++;
  return g_status;
}
}  // namespace

namespace rz {
hipError_t launch_i8_quantize(const void*, int, int64_t, bool, const I8View&, hipStream_t) { return counted(); }
hipError_t launch_i8_dequant(const I8View&, void*, int, hipStream_t) { return counted(); }
size_t i8_gemm_ws_bytes(int64_t m, int64_t n, int64_t, int64_t) { return m >= 512 ? (size_t)m * (size_t)n : 0; }
hipError_t launch_i8_gemm(const I8Gemm&, void*, hipStream_t) { return counted(); }
size_t moe_route_ws_bytes(int64_t tokens, int64_t experts, int64_t) { return (size_t)(tokens * experts); }
hipError_t launch_moe_route(const MoeRoute&, void*, hipStream_t) { return counted(); }
hipError_t launch_moe_combine(const MoeCombine&, hipStream_t) { return counted(); }
}  // namespace rz

namespace {

void expect(razer_status got, razer_status want, int launches, const char* what) {
  if (got != want || g_launches != launches) {
    fprintf(stderr, "i8_host_check: %s: got %d after %d launches, want %d after %d\n", what, (int)got, g_launches,
            (int)want, launches);
    g_fail = 1;
  }
  g_launches = 0;
}
#define ACCEPT(call) expect(call, RAZER_OK, 1, #call)
#define NOTHING(call) expect(call, RAZER_OK, 0, #call)
#define REFUSE(call) expect(call, RAZER_E_INVALID, 0, #call)
#define TOO_MUCH(call) expect(call, RAZER_E_UNSUPPORTED, 0, #call)

int8_t* fake(uintptr_t a) { return (int8_t*)a; }
razer_i8 i8(int64_t rows, int64_t cols) { return {rows, cols, fake(0x10000), (float*)fake(0x20004)}; }

const int64_t kEnds[] = {INT64_MIN, -1, INT64_MAX, INT64_MAX - 15, (int64_t)1 << 62, (int64_t)1 << 40};

void encoders() {
  void* x = fake(0x40000);
  razer_i8 t = i8(3, 64);
  ACCEPT(razer_i8_quantize(x, RAZER_F16, 64, &t, nullptr));
  ACCEPT(razer_i8_quantize(x, RAZER_F32, 68, &t, nullptr));
  ACCEPT(razer_i8_quantize_gated(x, RAZER_BF16, 128, &t, nullptr));
  ACCEPT(razer_i8_dequant(&t, x, RAZER_F32, nullptr));
  REFUSE(razer_i8_quantize(x, RAZER_F16, 64, nullptr, nullptr));
  REFUSE(razer_i8_dequant(nullptr, x, RAZER_F32, nullptr));
  for (int64_t v : kEnds) {
    razer_i8 r = i8(v, 64), c = i8(3, v);
    razer_i8_quantize(x, RAZER_F16, 64, &r, nullptr), razer_i8_quantize(x, RAZER_F16, v, &c, nullptr);
    razer_i8_quantize_gated(x, RAZER_F32, v, &r, nullptr), razer_i8_quantize_gated(x, RAZER_F32, v, &c, nullptr);
    razer_i8_dequant(&r, x, RAZER_F16, nullptr), razer_i8_dequant(&c, x, RAZER_F16, nullptr);
    expect(RAZER_OK, RAZER_OK, 0, "an end of 64 bits is launched");
    razer_i8_quantize(x, RAZER_F16, v, &t, nullptr);
    g_launches = 0;
  }
  razer_i8 large = i8((int64_t)1 << 20, (int64_t)1 << 14);
  ACCEPT(razer_i8_quantize(x, RAZER_F16, large.cols, &large, nullptr));
  TOO_MUCH((large.rows++, razer_i8_quantize(x, RAZER_F16, large.cols, &large, nullptr)));
  g_status = hipErrorInvalidValue;
  expect(razer_i8_quantize(x, RAZER_F16, 64, &t, nullptr), RAZER_E_HIP, 1, "a failed launch");
  g_status = hipSuccess;
}

void products() {
  razer_i8 x = i8(8, 128), w = i8(12, 128), tall = i8(512, 128);
  void *y = fake(0x50000), *ws = fake(0x60000);
  ACCEPT(razer_i8_gemm(&x, &w, y, RAZER_F16, nullptr, 0, nullptr));
  ACCEPT(razer_i8_gemm(&tall, &w, y, RAZER_BF16, ws, 512 * 12, nullptr));
  REFUSE(razer_i8_gemm(&tall, &w, y, RAZER_BF16, ws, 512 * 12 - 1, nullptr));
  REFUSE(razer_i8_gemm(&tall, &w, y, RAZER_BF16, nullptr, 512 * 12, nullptr));
  REFUSE(razer_i8_gemm(&tall, &w, y, RAZER_BF16, fake(0x60004), 512 * 12, nullptr));
  const int32_t *off = (const int32_t*)fake(0x70000), *rows = (const int32_t*)fake(0x80004);
  ACCEPT(razer_i8_gemm_grouped(&x, &w, off, 3, nullptr, 8, y, RAZER_F32, nullptr, 0, nullptr));
  ACCEPT(razer_i8_gemm_grouped(&x, &w, off, 4, rows, 100, y, RAZER_F32, nullptr, 0, nullptr));
  razer_i8 wide = i8((int64_t)1 << 25, 128);  // 4 GiB of codes
  TOO_MUCH(razer_i8_gemm_grouped(&wide, &w, off, 3, rows, 8, y, RAZER_F32, nullptr, 0, nullptr));
  wide.rows--;
  ACCEPT(razer_i8_gemm_grouped(&wide, &w, off, 3, rows, 8, y, RAZER_F32, nullptr, 0, nullptr));
  for (int64_t v : kEnds) {
    razer_i8 r = i8(v, 128), c = i8(8, v);
    razer_i8_gemm(&r, &w, y, RAZER_F32, ws, SIZE_MAX, nullptr), razer_i8_gemm(&x, &r, y, RAZER_F32, ws, SIZE_MAX, nullptr);
    razer_i8_gemm(&c, &c, y, RAZER_F32, ws, SIZE_MAX, nullptr);
    razer_i8_gemm_grouped(&x, &w, off, v, rows, 8, y, RAZER_F32, ws, SIZE_MAX, nullptr);
    razer_i8_gemm_grouped(&x, &w, off, 3, rows, v, y, RAZER_F32, ws, SIZE_MAX, nullptr);
    razer_i8_gemm_grouped(&r, &w, off, 3, rows, 8, y, RAZER_F32, ws, SIZE_MAX, nullptr);
    razer_i8_workspace_bytes(v, 8, 64, 0), razer_i8_workspace_bytes(8, v, 64, 2), razer_i8_workspace_bytes(8, 8, v, v);
    expect(RAZER_OK, RAZER_OK, 0, "an end of 64 bits is launched");
  }
}

void routes() {
  int32_t* word = (int32_t*)fake(0x90000);
  razer_route a = {};
  a.tokens = 6, a.stride = 40, a.experts = 32, a.top = 2, a.groups = 4, a.groups_kept = 2, a.group_best = 2;
  a.score = RAZER_SCORE_SIGMOID, a.dtype = RAZER_BF16, a.scale = 1, a.logits = word, a.chosen = word;
  a.weights = (float*)word;
  ACCEPT(razer_moe_route(&a, nullptr, 0, nullptr));
  razer_route b = a;
  b.offsets = b.rows = b.slots = word, b.bias = (float*)word, b.flags = RAZER_ROUTE_RENORM;
  ACCEPT(razer_moe_route(&b, word, 6 * 32, nullptr));
  REFUSE(razer_moe_route(&b, word, 6 * 32 - 1, nullptr));
  REFUSE(razer_moe_route(&b, nullptr, 6 * 32, nullptr));
  razer_route c = b;
  c.tokens = 0, c.logits = nullptr, c.chosen = c.rows = c.slots = nullptr, c.weights = nullptr;
  ACCEPT(razer_moe_route(&c, nullptr, 0, nullptr));
  const int32_t ends[] = {INT32_MIN, -1, INT32_MAX, 1 << 30};
  for (int64_t v : kEnds) {
    razer_route r = b, s = b;
    r.tokens = v;
    razer_moe_route(&r, word, SIZE_MAX, nullptr);
    expect(RAZER_OK, RAZER_OK, 0, "an end of 64 bits is launched");
    s.stride = v;
    razer_moe_route(&s, word, SIZE_MAX, nullptr);
    razer_moe_workspace_bytes(v, 8, 2), razer_moe_workspace_bytes(8, v, 2), razer_moe_workspace_bytes(8, 8, v);
    g_launches = 0;
  }
  for (int32_t v : ends) {
    razer_route r[6] = {b, b, b, b, b, b};
    r[0].experts = v, r[1].top = v, r[2].groups = v, r[3].groups_kept = v, r[4].group_best = v, r[5].score = v;
    for (razer_route& x : r) razer_moe_route(&x, word, SIZE_MAX, nullptr);
    expect(RAZER_OK, RAZER_OK, 0, "an end of 32 bits is launched");
  }

  razer_combine d = {};
  d.tokens = 6, d.top = 2, d.cols = 64, d.y_rows = 12, d.y_stride = 64, d.dtype = RAZER_F16, d.y = word;
  d.slots = word, d.weights = (float*)word, d.out = word;
  ACCEPT(razer_moe_combine(&d, nullptr));
  d.add = word, d.add_stride = 80;
  ACCEPT(razer_moe_combine(&d, nullptr));
  for (int64_t v : kEnds) {
    razer_combine r[5] = {d, d, d, d, d};
    r[0].tokens = v, r[1].top = v, r[2].cols = v, r[3].y_rows = v, r[4].y_rows = 1 << 30, r[4].y_stride = v;
    for (razer_combine& x : r) razer_moe_combine(&x, nullptr);
    g_launches = 0;
    razer_combine e = d;
    e.tokens = v, e.cols = v;
    razer_moe_combine(&e, nullptr);
    expect(RAZER_OK, RAZER_OK, 0, "an end of 64 bits is launched");
  }
}

}  // namespace

int main() {
  encoders();
  products();
  routes();
  if (!g_fail) printf("i8_host_check: ok\n");
  return g_fail;
}
