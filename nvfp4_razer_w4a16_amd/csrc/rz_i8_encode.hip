// rz_i8_encode.hip -- encoder, gated encoder and decoder of 8-bit integer tensors on
// gfx950.
//
// Per row: amax = max |x_c|, scale = amax / 127, code_c = rint(x_c * (127 / amax)),
// one fp32 rounding an operation.  |x_c| <= amax makes |x_c * (127 / amax)| at most
// 127 (1 + 2^-23), which rounds to 127: no clamp.  Below 2^-64 both sides of the
// quotient are first multiplied by 2^64, exactly, which keeps 127 / amax finite.
// Adding 1.5 * 2^23 rounds a value of less than 2^22 to a whole number, halves to even,
// and leaves that number's low byte in the sum's low byte.
// The gated form encodes silu(g) * u = g * u / (1 + exp(-g)), formed in fp32 and never
// stored.
//
// Bound by memory: the row lives in the registers of 64 to 1024 lanes between its
// maximum and its codes, so x is read once; rows of more than 32768 are read twice.
// Measured: the gated form of 2041 x 14336 from bf16 28.6-30.1 us (146 MB, 4.9-5.1 TB/s; a
// copy of 1 GiB reaches 5.1) and back to bf16 13.5-14.2 us (88 MB, 6.2-6.5 TB/s, the codes
// still in the cache behind the L2s); one row of 4096 2.2 and 1.8 us, the time of any launch.
#include <algorithm>

#include "rz_i8.h"
#include "rz_i8_launch.h"

namespace rz {

namespace {

constexpr int kPer = kMxChunk;

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

template <typename T, bool GATED> struct Loader {
  Chunk<T> a, b;
  __device__ __forceinline__ void load(const T* p, int64_t cols) {
    a.load(p);
    if constexpr (GATED) b.load(p + cols);
  }
  __device__ __forceinline__ void values(float (&v)[kPer]) const {
#pragma unroll
    for (int i = 0; i < kPer; i++) v[i] = GATED ? silu_mul(a.at(i), b.at(i)) : a.at(i);
  }
};

__device__ __forceinline__ uint32_t top_of(const float (&v)[kPer]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kPer; i++) top = max(top, f2u(v[i]) & 0x7FFFFFFFu);
  return top;
}

// What a row's codes are formed with, from its largest magnitude's bits.
struct RowScale {
  float pre, inverse, scale;
};
__device__ __forceinline__ RowScale row_scale(uint32_t top) {
  const float amax = u2f(top);
  RowScale r;
  r.pre = amax < 0x1p-64f ? 0x1p64f : 1.0f;
  if (top >= 0x7F800000u) {
    r.inverse = 0.0f;
    r.scale = u2f(0x7FC00000u);
  } else {
    r.inverse = amax > 0.0f ? 127.0f / (amax * r.pre) : 0.0f;
    r.scale = amax / 127.0f;
  }
  return r;
}

__device__ __forceinline__ u32x2_t codes8(const float (&v)[kPer], const RowScale& r, bool bad) {
  uint32_t q[kPer];
#pragma unroll
  for (int i = 0; i < kPer; i++) q[i] = f2u(v[i] * r.pre * r.inverse + 12582912.0f);
  u32x2_t o;
#pragma unroll
  for (int i = 0; i < 2; i++)
    o[i] = (q[4 * i] & 255u) | (q[4 * i + 1] & 255u) << 8 | (q[4 * i + 2] & 255u) << 16 | q[4 * i + 3] << 24;
  return bad ? u32x2_t{0u, 0u} : o;
}

// The maximum over the LANES threads of a row.
template <int LANES> __device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* lds) {
  v = wave_max_u32(v);
  if constexpr (LANES > 64) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < LANES / 64; i++) v = max(v, lds[i]);
    __syncthreads();
  }
  return v;
}

// LANES threads a row, CH chunks of 8 elements each; CH = 0: rows of any length, read twice.
template <typename T, bool GATED, int LANES, int CH>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES) void i8_quantize_kernel(const T* __restrict__ x, int64_t stride,
                                                                                int64_t rows, int64_t cols,
                                                                                u32x2_t* __restrict__ codes,
                                                                                float* __restrict__ scales) {
  constexpr int kRows = LANES < 256 ? 256 / LANES : 1;  // rows of a workgroup
  __shared__ uint32_t lds[LANES / 64];
  const int lane = threadIdx.x % LANES, chunks = (int)(cols / kPer);
  for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / LANES; row < rows; row += (int64_t)gridDim.x * kRows) {
    const T* p = x + row * stride;
    uint32_t top = 0;
    if constexpr (CH > 0) {
      Loader<T, GATED> raw[CH];
#pragma unroll
      for (int i = 0; i < CH; i++)
        if (lane + i * LANES < chunks) raw[i].load(p + (int64_t)(lane + i * LANES) * kPer, cols);
      float v[CH][kPer];
#pragma unroll
      for (int i = 0; i < CH; i++)
        if (lane + i * LANES < chunks) {
          raw[i].values(v[i]);
          top = max(top, top_of(v[i]));
        }
      top = row_max<LANES>(top, lds);
      const RowScale r = row_scale(top);
#pragma unroll
      for (int i = 0; i < CH; i++)
        if (lane + i * LANES < chunks) codes[row * chunks + lane + i * LANES] = codes8(v[i], r, top >= 0x7F800000u);
      if (lane == 0) scales[row] = r.scale;
    } else {
      float v[kPer];
      for (int c = lane; c < chunks; c += LANES) {
        Loader<T, GATED> raw;
        raw.load(p + (int64_t)c * kPer, cols);
        raw.values(v);
        top = max(top, top_of(v));
      }
      top = row_max<LANES>(top, lds);
      const RowScale r = row_scale(top);
      for (int c = lane; c < chunks; c += LANES) {
        Loader<T, GATED> raw;
        raw.load(p + (int64_t)c * kPer, cols);
        raw.values(v);
        codes[row * chunks + c] = codes8(v, r, top >= 0x7F800000u);
      }
      if (lane == 0) scales[row] = r.scale;
    }
  }
}

template <typename OT>
__global__ __launch_bounds__(256) void i8_dequant_kernel(const u32x2_t* __restrict__ codes,
                                                         const float* __restrict__ scales, int64_t chunks, FastDiv cpr,
                                                         OT* __restrict__ out) {
  typedef OT V __attribute__((ext_vector_type(8)));
  const int64_t first = (int64_t)blockIdx.x * 256;
  const int64_t row0 = first / cpr.d;  // uniform; the thread's own row follows from 32-bit arithmetic
  const uint32_t c0 = (uint32_t)(first - row0 * cpr.d) + threadIdx.x;
  const int64_t at = first + threadIdx.x;
  if (at >= chunks) return;
  const float s = scales[row0 + fast_div(c0, cpr)];
  const u32x2_t c = codes[at];
  V v;
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = mx_cvt<OT>(rounded((float)((int)(c[i >> 2] << (24 - 8 * (i & 3))) >> 24) * s));
  *(V*)(out + at * 8) = v;
}

template <typename T, bool GATED, int LANES, int CH>
hipError_t go(const T* x, int64_t stride, const I8View& out, hipStream_t stream) {
  constexpr int threads = LANES < 256 ? 256 : LANES, rows = threads / LANES;
  const int64_t grid = std::min((out.rows + rows - 1) / rows, (int64_t)1 << 21);  // below 2^32 threads
  hipLaunchKernelGGL((i8_quantize_kernel<T, GATED, LANES, CH>), dim3((unsigned)grid), dim3(threads), 0, stream, x,
                     stride, out.rows, out.cols, (u32x2_t*)out.codes, out.scales);
  return hipGetLastError();
}

template <typename T, bool GATED>
hipError_t run_quantize(const T* x, int64_t stride, const I8View& out, hipStream_t stream) {
  const int64_t chunks = out.cols / kPer;
  if (chunks <= 64) return go<T, GATED, 64, 1>(x, stride, out, stream);
  if (chunks <= 256) return go<T, GATED, 64, 4>(x, stride, out, stream);
  if (chunks <= 512) return go<T, GATED, 256, 2>(x, stride, out, stream);
  if (chunks <= 1024) return go<T, GATED, 256, 4>(x, stride, out, stream);
  if (chunks <= 2048) return go<T, GATED, 512, 4>(x, stride, out, stream);
  if (chunks <= 4096) return go<T, GATED, 1024, 4>(x, stride, out, stream);
  return go<T, GATED, 1024, 0>(x, stride, out, stream);
}
template <typename T>
hipError_t run_quantize(const T* x, int64_t stride, bool gated, const I8View& out, hipStream_t stream) {
  return gated ? run_quantize<T, true>(x, stride, out, stream) : run_quantize<T, false>(x, stride, out, stream);
}

template <typename OT> hipError_t run_dequant(const I8View& t, OT* out, hipStream_t stream) {
  const int64_t chunks = t.rows * (t.cols / kPer), grid = (chunks + 255) / 256;
  hipLaunchKernelGGL(i8_dequant_kernel<OT>, dim3((unsigned)grid), dim3(256), 0, stream, (const u32x2_t*)t.codes,
                     t.scales, chunks, make_fastdiv((uint32_t)(t.cols / kPer)), out);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_i8_quantize(const void* x, int dtype, int64_t stride, bool gated, const I8View& out,
                              hipStream_t stream) {
  if (dtype == kF32) return run_quantize((const float*)x, stride, gated, out, stream);
  if (dtype == kF16) return run_quantize((const _Float16*)x, stride, gated, out, stream);
  return run_quantize((const __bf16*)x, stride, gated, out, stream);
}

hipError_t launch_i8_dequant(const I8View& t, void* out, int out_dtype, hipStream_t stream) {
  if (out_dtype == kF32) return run_dequant(t, (float*)out, stream);
  if (out_dtype == kF16) return run_dequant(t, (_Float16*)out, stream);
  return run_dequant(t, (__bf16*)out, stream);
}

}  // namespace rz
