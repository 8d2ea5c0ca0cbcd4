// rz_i8.h -- device-side helpers of the 8-bit integer kernels.
#pragma once

#include "rz_mx.h"

namespace rz {

typedef int i32x16_t __attribute__((ext_vector_type(16)));

// A product that is rounded to fp32 before anything else happens to it: the compiler
// would form a product and its rounding to f16 in one operation (v_fma_mixlo_f16) of one
// rounding, whatever it is told of contraction.
__device__ __forceinline__ float rounded(float v) {
  asm("" : "+v"(v));
  return v;
}

// y = sum * sx * sw, in this order everywhere: one rounding for the sum (above 2^24)
// and one a product, so that a result does not depend on the kernel that forms it.
__device__ __forceinline__ float i8_scaled(int sum, float sx, float sw) { return rounded((float)sum * sx * sw); }

}  // namespace rz
