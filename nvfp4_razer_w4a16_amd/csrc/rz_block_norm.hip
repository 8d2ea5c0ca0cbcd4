// rz_block_norm.hip -- the step between two blocks of a transformer on gfx950:
//
//   h' = h + s * gate . N(y; post)        N(v; w) = v * w / sqrt(mean(v^2) + eps)
//   x  = N(h'; pre)
//
// in one pass: y and h are read once, h' and x (as values, packed to MXFP4, or
// both) written once.  Everything between is fp32 and stays in registers: a
// row's second mean is taken over the unrounded h', and x is packed from the
// unrounded norm.
//
// Bound by memory.  A lane holds chunks of 8 elements (16-byte accesses of
// 16-bit types); a row is spread over 64, 256 or 1024 lanes so that a lane has
// at most four chunks, and short rows share a workgroup.  All loads of a row,
// the weights' among them, are requested before the first sum is needed.
// Measured: 4096 x 8192 in bf16 with four gates 48.6 us (268 MB, 5.5 TB/s); one row
// of 4096 in fp16, packed, 4.1 us (two barriers and the launch).
#include "rz_mx.h"
#include "rz_mx_launch.h"

namespace rz {

namespace {

template <typename T> struct Args {
  int64_t rows;
  int chunks;                // of a row
  const T *y, *h;
  int64_t y_stride, h_stride;
  const T *post, *pre, *gate;
  int64_t rows_per_gate;
  float scale, eps, inv_cols;
  int norm_y;
  T *h_out, *x_out;
  uint32_t* codes;
  uint8_t* scales;
};

// Sum over the TPR lanes of a row; `part` is one float per wave of the workgroup.
template <int TPR> __device__ __forceinline__ float row_sum(float v, float* part) {
  v = wave_sum_f32(v);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < TPR / 64; i++) v += part[i];
  }
  return v;
}

template <typename T> __device__ __forceinline__ void store_chunk(T* p, const float (&v)[kMxChunk]) {
  if constexpr (sizeof(T) == 4) {
    *(f32x4_t*)p = f32x4_t{v[0], v[1], v[2], v[3]};
    *(f32x4_t*)(p + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
  } else {
    typedef T V __attribute__((ext_vector_type(8)));
    V o;
#pragma unroll
    for (int i = 0; i < kMxChunk; i++) o[i] = mx_cvt<T>(v[i]);
    *(V*)p = o;
  }
}

template <typename T, int TPR, int CH>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void block_norm_kernel(Args<T> a) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR, kRows = kThreads / TPR;
  __shared__ float part[2][kThreads / 64];
  const int lane = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
  if (row >= a.rows) return;  // whole waves, and whole workgroups where a row needs barriers
  const int64_t cols = (int64_t)a.chunks * kMxChunk;
  const T* gate = a.gate + row / a.rows_per_gate * cols;
  float h[CH][kMxChunk], ss = 0.0f;
  Chunk<T> cy[CH], ch[CH], cpost[CH], cgate[CH], cpre[CH];
  const bool want_x = a.x_out || a.codes;
  constexpr bool kEarly = CH * sizeof(T) <= 8;  // four fp32 chunks of everything would spill
#pragma unroll
  for (int i = 0; i < CH; i++) {
    const int c = lane + i * TPR;
    if (c >= a.chunks) continue;
    if (a.y) cy[i].load(a.y + row * a.y_stride + c * kMxChunk);
    ch[i].load(a.h + row * a.h_stride + c * kMxChunk);
  }
#pragma unroll
  for (int i = 0; i < CH; i++) {
    const int c = lane + i * TPR;
    if (c >= a.chunks) continue;
    if (!kEarly) continue;
    if (a.y && a.post) cpost[i].load(a.post + c * kMxChunk);
    if (a.y && a.gate) cgate[i].load(gate + c * kMxChunk);
    if (want_x && a.pre) cpre[i].load(a.pre + c * kMxChunk);
  }
  float r = a.scale;
  if (a.y && a.norm_y) {
#pragma unroll
    for (int i = 0; i < CH; i++)
      if (lane + i * TPR < a.chunks)
#pragma unroll
        for (int j = 0; j < kMxChunk; j++) ss += cy[i].at(j) * cy[i].at(j);
    r *= rsqrtf(row_sum<TPR>(ss, part[0]) * a.inv_cols + a.eps);
  }
  ss = 0.0f;
#pragma unroll
  for (int i = 0; i < CH; i++) {
    const int c = lane + i * TPR;
    if (c >= a.chunks) continue;
    if (!kEarly && a.y && a.post) cpost[i].load(a.post + c * kMxChunk);
    if (!kEarly && a.y && a.gate) cgate[i].load(gate + c * kMxChunk);
#pragma unroll
    for (int j = 0; j < kMxChunk; j++) {
      float v = ch[i].at(j);
      if (a.y) {
        float t = cy[i].at(j) * r;
        if (a.post) t *= cpost[i].at(j);
        if (a.gate) t *= cgate[i].at(j);
        v += t;
      }
      h[i][j] = v;
      ss += v * v;
    }
    if (a.h_out) store_chunk(a.h_out + row * cols + c * kMxChunk, h[i]);
  }
  if (!want_x) return;
  r = rsqrtf(row_sum<TPR>(ss, part[1]) * a.inv_cols + a.eps);
#pragma unroll
  for (int i = 0; i < CH; i++) {
    const int c = lane + i * TPR;
    if (c >= a.chunks) continue;  // whole quads: a row has a multiple of four chunks
    if (!kEarly && a.pre) cpre[i].load(a.pre + c * kMxChunk);
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < kMxChunk; j++) {
      h[i][j] *= r;
      if (a.pre) h[i][j] *= cpre[i].at(j);
      top = max(top, f2u(h[i][j]) & 0x7FFFFFFFu);
    }
    if (a.x_out) store_chunk(a.x_out + row * cols + c * kMxChunk, h[i]);
    if (a.codes) {
      const uint32_t byte = mx_scale_byte(quad_max(top));
      const int64_t at = row * a.chunks + c;
      a.codes[at] = mx_codes8(h[i], byte);
      if ((lane & 3) == 0) a.scales[at >> 2] = (uint8_t)byte;
    }
  }
}

template <typename T, int TPR, int CH> hipError_t go(const Args<T>& a, hipStream_t stream) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR, kRows = kThreads / TPR;
  const int64_t grid = (a.rows + kRows - 1) / kRows;
  hipLaunchKernelGGL((block_norm_kernel<T, TPR, CH>), dim3((unsigned)grid), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

template <typename T> hipError_t run(const BlockNorm& b, hipStream_t stream) {
  const Args<T> a = {b.rows,
                     (int)(b.cols / kMxChunk),
                     (const T*)b.y,
                     (const T*)b.h,
                     b.y_stride,
                     b.h_stride,
                     (const T*)b.post,
                     (const T*)b.pre,
                     (const T*)b.gate,
                     b.gate ? b.rows / b.gate_rows : 1,
                     b.scale,
                     b.eps,
                     1.0f / (float)b.cols,
                     b.norm_y,
                     (T*)b.h_out,
                     (T*)b.x_out,
                     (uint32_t*)b.packed.codes,
                     b.packed.scales};
  const int c = a.chunks;
  switch (block_norm_lanes(b.cols)) {
    case 64: return c <= 64 ? go<T, 64, 1>(a, stream) : go<T, 64, 2>(a, stream);
    case 256: return c <= 256 ? go<T, 256, 1>(a, stream) : c <= 512 ? go<T, 256, 2>(a, stream) : go<T, 256, 4>(a, stream);
    default: return c <= 2048 ? go<T, 1024, 2>(a, stream) : go<T, 1024, 4>(a, stream);
  }
}

}  // namespace

hipError_t launch_block_norm(const BlockNorm& b, hipStream_t stream) {
  if (b.rows == 0 || b.cols == 0) return hipSuccess;
  if (b.dtype == kF32) return run<float>(b, stream);
  if (b.dtype == kF16) return run<_Float16>(b, stream);
  return run<__bf16>(b, stream);
}

}  // namespace rz
