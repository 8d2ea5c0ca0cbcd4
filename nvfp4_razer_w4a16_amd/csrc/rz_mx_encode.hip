// rz_mx_encode.hip -- MXFP4 encoder, gated encoder and decoder on gfx950.
//
// Per 32-element block: amax = max |x_j|, scale X = 2^(floor(log2 amax) - 2),
// code_j = x_j / X rounded to FP4-E2M1 {0, 0.5, 1, 1.5, 2, 3, 4, 6}, halves to
// the even code, magnitudes above 6 to 6.  Division by a power of two is exact
// and the rounding one hardware conversion (v_cvt_scalef32_pk_fp4_*), so the
// bytes follow from the definition alone.  The gated form packs
// silu(g) * u = g * u / (1 + exp(-g)), formed in fp32 and never stored.
//
// Bound by memory: a 16-bit element costs 2 bytes read and 0.53 written and
// about two vector instructions.  A lane takes 8 elements (one 16-byte load of
// a 16-bit type), so four neighbouring lanes hold a block and two quad
// permutations give them its amax; no LDS, no second pass.  Measured: 14336 x 4096
// in fp32 59.9 us (266 MB, 4.4 TB/s) and back to fp32 44-46 us (5.8-6.1 TB/s); the
// gated form of 2041 x 14336 from bf16 26.0-26.8 us (133 MB, 5.0-5.1 TB/s; a copy of
// 1 GiB reaches 5.06); one row of 4096 1.9 us, the time of any launch.
#include "rz_mx.h"
#include "rz_mx_launch.h"

namespace rz {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = kMxChunk;

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

template <typename T, bool GATED>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(const T* __restrict__ x, int64_t stride, int64_t chunks,
                                                               FastDiv cpr, int64_t cols, uint32_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales) {
  const int64_t first = (int64_t)blockIdx.x * kThreads;
  const int64_t row0 = first / cpr.d;  // uniform; the thread's own row follows from 32-bit arithmetic
  const uint32_t c0 = (uint32_t)(first - row0 * cpr.d) + threadIdx.x;
  const uint32_t dr = fast_div(c0, cpr);
  const int64_t at = first + threadIdx.x;
  const bool live = at < chunks;  // whole quads: a row has a multiple of four chunks
  const T* p = x + (row0 + dr) * stride + (int64_t)(c0 - dr * cpr.d) * kPer;
  float v[kPer];
  if (live) {
    Chunk<T> a;
    a.load(p);
    if constexpr (GATED) {
      Chunk<T> b;
      b.load(p + cols);
#pragma unroll
      for (int i = 0; i < kPer; i++) v[i] = silu_mul(a.at(i), b.at(i));
    } else {
#pragma unroll
      for (int i = 0; i < kPer; i++) v[i] = a.at(i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; i++) v[i] = 0.0f;
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kPer; i++) top = max(top, f2u(v[i]) & 0x7FFFFFFFu);
  top = quad_max(top);
  const uint32_t byte = mx_scale_byte(top);
  const uint32_t out = mx_codes8(v, byte);
  if (!live) return;
  codes[at] = out;
  if ((threadIdx.x & 3) == 0) scales[at >> 2] = (uint8_t)byte;
}

template <typename OT>
__global__ __launch_bounds__(kThreads) void mx_dequant_kernel(const uint32_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales, int64_t chunks,
                                                              OT* __restrict__ out) {
  typedef OT V __attribute__((ext_vector_type(8)));
  const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (at >= chunks) return;
  const float s = mx_scale_value(scales[at >> 2]);
  const uint32_t c = codes[at];
  V v;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float q = 0.5f * (float)fp4_mag_x2((c >> (4 * i)) & 7u) * s;
    v[i] = mx_cvt<OT>(((c >> (4 * i)) & 8u) ? -q : q);
  }
  *(V*)(out + at * 8) = v;
}

template <typename T>
hipError_t run_quantize(const T* x, int64_t stride, bool gated, const MxView& out, hipStream_t stream) {
  const int64_t chunks = out.rows * (out.cols / kPer);
  if (chunks == 0) return hipSuccess;
  const int64_t grid = (chunks + kThreads - 1) / kThreads;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  const FastDiv cpr = make_fastdiv((uint32_t)(out.cols / kPer));
  if (gated)
    hipLaunchKernelGGL((mx_quantize_kernel<T, true>), dim3((unsigned)grid), dim3(kThreads), 0, stream, x, stride,
                       chunks, cpr, out.cols, (uint32_t*)out.codes, out.scales);
  else
    hipLaunchKernelGGL((mx_quantize_kernel<T, false>), dim3((unsigned)grid), dim3(kThreads), 0, stream, x, stride,
                       chunks, cpr, out.cols, (uint32_t*)out.codes, out.scales);
  return hipGetLastError();
}

template <typename OT> hipError_t run_dequant(const MxView& t, OT* out, hipStream_t stream) {
  const int64_t chunks = t.rows * (t.cols / kPer);
  if (chunks == 0) return hipSuccess;
  const int64_t grid = (chunks + kThreads - 1) / kThreads;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  hipLaunchKernelGGL(mx_dequant_kernel<OT>, dim3((unsigned)grid), dim3(kThreads), 0, stream, (const uint32_t*)t.codes,
                     t.scales, chunks, out);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(const void* x, int dtype, int64_t stride, bool gated, const MxView& out,
                              hipStream_t stream) {
  if (dtype == kF32) return run_quantize((const float*)x, stride, gated, out, stream);
  if (dtype == kF16) return run_quantize((const _Float16*)x, stride, gated, out, stream);
  return run_quantize((const __bf16*)x, stride, gated, out, stream);
}

hipError_t launch_mx_dequant(const MxView& t, void* out, int out_dtype, hipStream_t stream) {
  if (out_dtype == kF32) return run_dequant(t, (float*)out, stream);
  if (out_dtype == kF16) return run_dequant(t, (_Float16*)out, stream);
  return run_dequant(t, (__bf16*)out, stream);
}

}  // namespace rz
