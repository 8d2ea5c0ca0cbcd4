// mx_host_check.cpp -- test infrastructure only (tests/test_mx_sanitizers.py): a
// host build of rz_mx_api.cpp against stub launchers, run under AddressSanitizer
// and UndefinedBehaviorSanitizer.  Every entry point is called with rejected and
// with accepted arguments, sizes at the ends of 64 bits among them (fake, never
// dereferenced device addresses); the stubs count the launches.  Exit status 0
// and no sanitizer report means clean.
#include <hip/hip_runtime.h>

#include <stdint.h>
#include <stdio.h>

#include "../../include/librazer.h"
#include "rz_mx_launch.h"

namespace {
int g_launches = 0, g_fail = 0;
hipError_t g_status = hipSuccess;
hipError_t counted() {
  g_launches++;
  return g_status;
}
}  // namespace

namespace rz {
hipError_t launch_mx_quantize(const void*, int, int64_t, bool, const MxView&, hipStream_t) { return counted(); }
hipError_t launch_mx_dequant(const MxView&, void*, int, hipStream_t) { return counted(); }
size_t mx_gemm_ws_bytes(int64_t m, int64_t n, int64_t, int64_t) { return m >= 512 ? (size_t)m * (size_t)n : 0; }
hipError_t launch_mx_gemm(const MxGemm&, void*, size_t, hipStream_t) { return counted(); }
hipError_t launch_block_norm(const BlockNorm&, hipStream_t) { return counted(); }
int device_cu_count() { return 256; }
}  // namespace rz

namespace {

void expect(razer_status got, razer_status want, int launches, const char* what) {
  if (got != want || g_launches != launches) {
    fprintf(stderr, "mx_host_check: %s: got %d after %d launches, want %d after %d\n", what, (int)got, g_launches,
            (int)want, launches);
    g_fail = 1;
  }
  g_launches = 0;
}
#define ACCEPT(call) expect(call, RAZER_OK, 1, #call)
#define NOTHING(call) expect(call, RAZER_OK, 0, #call)
#define REFUSE(call) expect(call, RAZER_E_INVALID, 0, #call)
#define TOO_MUCH(call) expect(call, RAZER_E_UNSUPPORTED, 0, #call)

uint8_t* fake(uintptr_t a) { return (uint8_t*)a; }
razer_mx mx(int64_t rows, int64_t cols) { return {rows, cols, fake(0x10000), fake(0x20001)}; }

const int64_t kEnds[] = {INT64_MIN, -1, INT64_MAX, INT64_MAX - 31, (int64_t)1 << 62, (int64_t)1 << 40};

void encoders() {
  void* x = fake(0x40000);
  razer_mx t = mx(3, 64);
  ACCEPT(razer_mx_quantize(x, RAZER_F16, 64, &t, nullptr));
  ACCEPT(razer_mx_quantize(x, RAZER_F32, 68, &t, nullptr));
  ACCEPT(razer_mx_quantize_gated(x, RAZER_BF16, 128, &t, nullptr));
  ACCEPT(razer_mx_dequant(&t, x, RAZER_F32, nullptr));
  REFUSE(razer_mx_quantize_gated(x, RAZER_BF16, 64, &t, nullptr));
  REFUSE(razer_mx_quantize(x, RAZER_F16, 63, &t, nullptr));
  REFUSE(razer_mx_quantize(x, RAZER_F16, 68, &t, nullptr));
  REFUSE(razer_mx_quantize(fake(0x40002), RAZER_F16, 64, &t, nullptr));
  REFUSE(razer_mx_quantize(nullptr, RAZER_F16, 64, &t, nullptr));
  REFUSE(razer_mx_quantize(x, (razer_dtype)9, 64, &t, nullptr));
  REFUSE(razer_mx_quantize(x, RAZER_F16, 64, nullptr, nullptr));
  REFUSE(razer_mx_dequant(nullptr, x, RAZER_F32, nullptr));
  REFUSE(razer_mx_dequant(&t, nullptr, RAZER_F32, nullptr));
  REFUSE(razer_mx_dequant(&t, fake(0x40004), RAZER_F32, nullptr));
  REFUSE(razer_mx_dequant(&t, x, (razer_dtype)-1, nullptr));
  for (int64_t v : kEnds) {
    razer_mx r = mx(v, 64), c = mx(3, v);
    razer_mx_quantize(x, RAZER_F16, 64, &r, nullptr), razer_mx_quantize(x, RAZER_F16, v, &c, nullptr);
    razer_mx_quantize_gated(x, RAZER_F32, v, &r, nullptr), razer_mx_quantize_gated(x, RAZER_F32, v, &c, nullptr);
    razer_mx_dequant(&r, x, RAZER_F16, nullptr), razer_mx_dequant(&c, x, RAZER_F16, nullptr);
    expect(RAZER_OK, RAZER_OK, 0, "an end of 64 bits is launched");
    razer_mx_quantize(x, RAZER_F16, v, &t, nullptr);
    g_launches = 0;
  }
  razer_mx none = {0, 64, nullptr, nullptr}, odd = mx(3, 48), bare = {3, 64, nullptr, fake(1)};
  NOTHING(razer_mx_quantize(nullptr, RAZER_F16, 0, &none, nullptr));
  NOTHING(razer_mx_dequant(&none, nullptr, RAZER_F16, nullptr));
  REFUSE(razer_mx_quantize(x, RAZER_F16, 64, &odd, nullptr));
  REFUSE(razer_mx_quantize(x, RAZER_F16, 64, &bare, nullptr));
  razer_mx large = mx((int64_t)1 << 20, (int64_t)1 << 15);
  TOO_MUCH((large.rows++, razer_mx_quantize(x, RAZER_F16, large.cols, &large, nullptr)));
  g_status = hipErrorInvalidValue;
  expect(razer_mx_quantize(x, RAZER_F16, 64, &t, nullptr), RAZER_E_HIP, 1, "a failed launch");
  g_status = hipSuccess;
}

void products() {
  razer_mx x = mx(8, 128), w = mx(12, 128), other = mx(12, 96), none = mx(0, 128), flat = mx(8, 0);
  void *y = fake(0x50000), *ws = fake(0x60000);
  ACCEPT(razer_mx_gemm(&x, &w, y, RAZER_F16, nullptr, 0, nullptr));
  REFUSE(razer_mx_gemm(nullptr, &w, y, RAZER_F16, nullptr, 0, nullptr));
  REFUSE(razer_mx_gemm(&x, nullptr, y, RAZER_F16, nullptr, 0, nullptr));
  REFUSE(razer_mx_gemm(&x, &other, y, RAZER_F16, nullptr, 0, nullptr));
  REFUSE(razer_mx_gemm(&x, &w, nullptr, RAZER_F16, nullptr, 0, nullptr));
  REFUSE(razer_mx_gemm(&x, &w, fake(0x50008), RAZER_F16, nullptr, 0, nullptr));
  REFUSE(razer_mx_gemm(&x, &w, y, (razer_dtype)7, nullptr, 0, nullptr));
  NOTHING(razer_mx_gemm(&none, &w, nullptr, RAZER_F16, nullptr, 0, nullptr));
  NOTHING(razer_mx_gemm(&x, &none, nullptr, RAZER_F16, nullptr, 0, nullptr));
  razer_mx flat_w = mx(12, 0);
  TOO_MUCH(razer_mx_gemm(&flat, &flat_w, y, RAZER_F16, nullptr, 0, nullptr));
  razer_mx long_x = mx(1, ((int64_t)1 << 23) + 32);
  TOO_MUCH(razer_mx_gemm(&long_x, &long_x, y, RAZER_F16, nullptr, 0, nullptr));
  razer_mx many = mx(((int64_t)1 << 30) + 1, 128);
  TOO_MUCH(razer_mx_gemm(&many, &w, y, RAZER_F16, ws, SIZE_MAX, nullptr));
  TOO_MUCH(razer_mx_gemm(&x, &many, y, RAZER_F16, ws, SIZE_MAX, nullptr));
  razer_mx tall = mx(512, 128);  // the stub asks for 512 * 12 bytes
  ACCEPT(razer_mx_gemm(&tall, &w, y, RAZER_BF16, ws, 512 * 12, nullptr));
  REFUSE(razer_mx_gemm(&tall, &w, y, RAZER_BF16, ws, 512 * 12 - 1, nullptr));
  REFUSE(razer_mx_gemm(&tall, &w, y, RAZER_BF16, nullptr, 512 * 12, nullptr));
  REFUSE(razer_mx_gemm(&tall, &w, y, RAZER_BF16, fake(0x60004), 512 * 12, nullptr));

  const int32_t *off = (const int32_t*)fake(0x70000), *rows = (const int32_t*)fake(0x80004);
  ACCEPT(razer_mx_gemm_grouped(&x, &w, off, 3, nullptr, 8, y, RAZER_F32, nullptr, 0, nullptr));
  ACCEPT(razer_mx_gemm_grouped(&x, &w, off, 4, rows, 100, y, RAZER_F32, nullptr, 0, nullptr));
  REFUSE(razer_mx_gemm_grouped(&x, &w, off, 3, nullptr, 7, y, RAZER_F32, nullptr, 0, nullptr));
  REFUSE(razer_mx_gemm_grouped(&x, &w, off, 5, nullptr, 8, y, RAZER_F32, nullptr, 0, nullptr));
  REFUSE(razer_mx_gemm_grouped(&x, &w, off, 0, nullptr, 8, y, RAZER_F32, nullptr, 0, nullptr));
  REFUSE(razer_mx_gemm_grouped(&x, &w, off, RAZER_MX_MAX_EXPERTS + 1, rows, 8, y, RAZER_F32, nullptr, 0, nullptr));
  REFUSE(razer_mx_gemm_grouped(&x, &w, nullptr, 3, nullptr, 8, y, RAZER_F32, nullptr, 0, nullptr));
  REFUSE(razer_mx_gemm_grouped(&x, &w, (const int32_t*)fake(0x70002), 3, nullptr, 8, y, RAZER_F32, nullptr, 0, nullptr));
  REFUSE(razer_mx_gemm_grouped(&x, &w, off, 3, (const int32_t*)fake(0x80001), 8, y, RAZER_F32, nullptr, 0, nullptr));
  REFUSE(razer_mx_gemm_grouped(&none, &w, off, 3, rows, 8, y, RAZER_F32, nullptr, 0, nullptr));
  NOTHING(razer_mx_gemm_grouped(&x, &w, nullptr, 3, rows, 0, nullptr, RAZER_F32, nullptr, 0, nullptr));
  razer_mx wide = mx((int64_t)1 << 26, 128);  // 4 GiB of codes
  TOO_MUCH(razer_mx_gemm_grouped(&wide, &w, off, 3, rows, 8, y, RAZER_F32, nullptr, 0, nullptr));
  wide.rows--;
  ACCEPT(razer_mx_gemm_grouped(&wide, &w, off, 3, rows, 8, y, RAZER_F32, nullptr, 0, nullptr));
  for (int64_t v : kEnds) {
    razer_mx r = mx(v, 128), c = mx(8, v);
    razer_mx_gemm(&r, &w, y, RAZER_F32, ws, SIZE_MAX, nullptr), razer_mx_gemm(&x, &r, y, RAZER_F32, ws, SIZE_MAX, nullptr);
    razer_mx_gemm(&c, &c, y, RAZER_F32, ws, SIZE_MAX, nullptr);
    razer_mx_gemm_grouped(&x, &w, off, v, rows, 8, y, RAZER_F32, ws, SIZE_MAX, nullptr);
    razer_mx_gemm_grouped(&x, &w, off, 3, rows, v, y, RAZER_F32, ws, SIZE_MAX, nullptr);
    razer_mx_gemm_grouped(&r, &w, off, 3, rows, 8, y, RAZER_F32, ws, SIZE_MAX, nullptr);
    razer_mx_workspace_bytes(v, 8, 64, 0), razer_mx_workspace_bytes(8, v, 64, 2), razer_mx_workspace_bytes(8, 8, v, v);
    expect(RAZER_OK, RAZER_OK, 0, "an end of 64 bits is launched");
  }
}

void norms() {
  razer_mx t = mx(6, 64);
  razer_norm a = {};
  a.rows = 6, a.cols = 64, a.dtype = RAZER_BF16, a.h = fake(0x90000), a.h_stride = 64, a.x_out = fake(0xa0000);
  a.residual_scale = 1, a.eps = 1e-5f;
  ACCEPT(razer_block_norm(&a, nullptr));
  razer_norm b = a;
  b.y = fake(0xb0000), b.y_stride = 72, b.gate = fake(0xc0000), b.gate_rows = 3, b.flags = RAZER_NORM_POST;
  b.x_out = nullptr, b.packed = &t;
  ACCEPT(razer_block_norm(&b, nullptr));
  REFUSE(razer_block_norm(nullptr, nullptr));
  razer_norm c;
#define WITH(base, change) (c = base, change, razer_block_norm(&c, nullptr))
  REFUSE(WITH(a, c.x_out = nullptr));
  REFUSE(WITH(a, c.h = nullptr));
  REFUSE(WITH(a, c.h_stride = 60));
  REFUSE(WITH(a, c.h_stride = 68));
  REFUSE(WITH(a, c.dtype = 5));
  REFUSE(WITH(a, c.flags = 2));
  REFUSE(WITH(a, c.flags = RAZER_NORM_POST));
  REFUSE(WITH(a, c.cols = 40));
  REFUSE(WITH(a, c.x_out = fake(0xa0008)));
  REFUSE(WITH(b, c.gate_rows = 4));
  REFUSE(WITH(b, c.gate_rows = 0));
  REFUSE(WITH(b, c.y = nullptr));
  REFUSE(WITH(b, c.y_stride = 8));
  REFUSE(WITH(b, (t.rows = 5)));
  t.rows = 6;
  NOTHING(WITH(a, c.rows = 0));
  TOO_MUCH(WITH(a, (c.cols = 32800, c.h_stride = 32800)));
  for (int64_t v : kEnds) {
    WITH(a, c.rows = v), WITH(a, c.cols = v), WITH(b, c.gate_rows = v), WITH(b, (c.rows = v, c.cols = v));
    expect(RAZER_OK, RAZER_OK, 0, "an end of 64 bits is launched");
    WITH(a, c.h_stride = v), WITH(b, c.y_stride = v);
    g_launches = 0;
  }
}

}  // namespace

int main() {
  encoders();
  products();
  norms();
  if (!g_fail) printf("mx_host_check: ok\n");
  return g_fail;
}
