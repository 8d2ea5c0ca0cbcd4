// rz_moe_launch.h -- internal launcher interface of the routing to experts and of the
// combination of their rows.  Host-only declarations; no torch types.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace rz {

struct MoeRoute {
  int64_t tokens, stride;
  int experts, top, groups, kept, best;
  bool sigmoid, renorm;
  int dtype;
  float scale;
  const void* logits;
  const float* bias;   // or NULL
  int32_t* chosen;
  float* weights;
  int32_t *offsets, *rows, *slots;  // all or none
};
size_t moe_route_ws_bytes(int64_t tokens, int64_t experts, int64_t top);
hipError_t launch_moe_route(const MoeRoute& r, void* ws, hipStream_t stream);

struct MoeCombine {
  int64_t tokens, cols, y_rows, y_stride, add_stride;
  int top, dtype;
  const void* y;
  const int32_t* slots;
  const float* weights;
  const void* add;     // or NULL
  void* out;
};
hipError_t launch_moe_combine(const MoeCombine& c, hipStream_t stream);

}  // namespace rz
