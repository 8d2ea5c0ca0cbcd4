// rz_mx.h -- device-side helpers of the microscaled 4-bit (MXFP4) kernels.
//
// The format: 32-element blocks along a row, FP4-E2M1 elements (two a byte, the
// even column in the low half) and one E8M0 scale byte a block: byte b < 255
// stands for 2^(b - 127), 255 for NaN.
#pragma once

#include "rz_device.h"

namespace rz {

constexpr int kMxBlock = 32;
constexpr uint32_t kMxNanScale = 255u;

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

// 2^(b - 127) as fp32: byte 0 is the subnormal 2^-127, 255 NaN.
__device__ __forceinline__ float mx_scale_value(uint32_t b) {
  return b == 0u ? u2f(0x00400000u) : b == kMxNanScale ? u2f(0x7FC00000u) : u2f(b << 23);
}

// The scale byte of a block whose largest magnitude has fp32 bits `amax` (sign
// clear): 2^(floor(log2 amax) - 2), so that the largest magnitude lands in
// [4, 8), the binade of FP4's largest value 6.  Below 2^-125 (and for a zero
// block) the byte is 0; an infinity or NaN gives 255.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
  const int e = (int)(amax >> 23);
  return e == 255 ? kMxNanScale : (uint32_t)max(e - 2, 0);
}

// FP4 codes of a chunk for a block of scale byte `byte`, value i in bits
// 4i .. 4i+3: one conversion a pair divides by the scale, rounds to nearest even
// and saturates at 6.  The conversion takes the scale's exponent bits alone.  A
// NaN block's codes are 0.
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8], uint32_t byte) {
  const float s = u2f(byte << 23);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
  return byte == kMxNanScale ? 0u : c;
}

// A lane's share of a row: eight elements, so that four neighbouring lanes hold
// a block.
constexpr int kMxChunk = 8;

// max over the four lanes of a quad
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));  // lanes 1 0 3 2
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
  return v;
}

template <typename T> struct Chunk;
template <> struct Chunk<float> {
  f32x4_t a, b;
  __device__ void load(const float* p) {
    a = *(const f32x4_t*)p;
    b = *(const f32x4_t*)(p + 4);
  }
  __device__ float at(int i) const { return i < 4 ? a[i] : b[i - 4]; }
};
template <> struct Chunk<_Float16> {
  typedef _Float16 V __attribute__((ext_vector_type(8)));
  V v;
  __device__ void load(const _Float16* p) { v = *(const V*)p; }
  __device__ float at(int i) const { return (float)v[i]; }
};
template <> struct Chunk<__bf16> {
  u32x4_t v;
  __device__ void load(const __bf16* p) { v = *(const u32x4_t*)p; }
  __device__ float at(int i) const {
    const uint32_t w = v[i >> 1];
    return u2f((i & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
};

// Stores round once, to nearest even.
template <typename T> __device__ __forceinline__ T mx_cvt(float v) { return (T)v; }

// n / d for n < 2^31 by a multiplication: the quotient of a thread's place by the
// chunks of a row.  With s = ceil(log2 d) the multiplier floor(2^32 (2^s - d) / d) + 1
// is the round-up method of Granlund and Montgomery, "Division by Invariant Integers
// using Multiplication" (1994); its sum mulhi(n, mul) + n stays within 32 bits for
// such n.
struct FastDiv {
  uint32_t d, mul, shift;
};
inline FastDiv make_fastdiv(uint32_t d) {
  uint32_t s = 0;
  while (s < 31 && (1u << s) < d) s++;
  const uint64_t m = ((((uint64_t)1 << s) - d) << 32) / d + 1;
  return {d, (uint32_t)m, s};
}
__device__ __forceinline__ uint32_t fast_div(uint32_t n, const FastDiv& f) {
  return (__umulhi(n, f.mul) + n) >> f.shift;
}

}  // namespace rz
