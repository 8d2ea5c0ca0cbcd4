// rz_moe.hip -- routing of tokens to experts and the combination of the experts' rows
// on gfx950.
//
// Route: s = softmax(l) or sigmoid(l), c = s + bias, the `top` largest c of the groups
// kept, weights s (over their sum) times a scale.  Scores and their comparisons are in
// fp64: of 256 experts the last chosen and the first not chosen lie within an fp32
// rounding of each other once in some ten thousand tokens, and the choice would then
// depend on how exp rounds.
// Order: the pairs (token, place) sorted by expert, then token.
// Combine: out[t] = add[t] + sum_j w[t, j] y[slots[t, j]], bound by memory.
#include <algorithm>

#include "rz_mx.h"
#include "rz_moe_launch.h"

namespace rz {

namespace {

constexpr int kWaves = 4;
constexpr double kNone = -__builtin_inf();

template <typename T> __device__ __forceinline__ T wave_max(T v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = max(v, __shfl_xor(v, o, 64));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// A wave a token; lane l holds experts l, l + 64 ...
template <typename T, int V> __global__ __launch_bounds__(64 * kWaves) void route_kernel(MoeRoute a) {
  __shared__ double keys[kWaves][64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
  if (t >= a.tokens) return;
  const T* row = (const T*)a.logits + t * a.stride;
  float l[V], m = -__builtin_inff();
  bool bad = false;
#pragma unroll
  for (int v = 0; v < V; v++) {
    const int e = lane + 64 * v;
    l[v] = e < a.experts ? (float)row[e] : -__builtin_inff();
    bad |= !(l[v] < __builtin_inff());
    m = max(m, l[v]);
  }
  bad = __ballot(bad) != 0;
  double s[V], c[V];
  if (a.sigmoid) {
#pragma unroll
    for (int v = 0; v < V; v++) s[v] = 1.0 / (1.0 + exp(-(double)l[v]));
  } else {
    m = wave_max(m);
    if (m == -__builtin_inff()) m = 0.0f;
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < V; v++) {
      s[v] = exp((double)l[v] - (double)m);
      sum += s[v];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int v = 0; v < V; v++) s[v] /= sum;
  }
#pragma unroll
  for (int v = 0; v < V; v++) {
    const int e = lane + 64 * v;
    c[v] = s[v] + (a.bias && e < a.experts ? (double)a.bias[e] : 0.0);
    if (!(c[v] > kNone) || l[v] == -__builtin_inff()) c[v] = kNone;
  }
  if (a.groups > 1) {
    // lane g scores group g
    const int size = a.experts / a.groups;
#pragma unroll
    for (int v = 0; v < V; v++) keys[wave][lane + 64 * v] = c[v];
    wave_lds_sync();
    double first = kNone, second = kNone;
    for (int i = 0; lane < a.groups && i < size; i++) {
      const double k = keys[wave][lane * size + i];
      second = max(second, min(first, k));
      first = max(first, k);
    }
    const double score = a.best == 2 && second > kNone ? first + second : first;
    int before = 0;
    for (int g = 0; g < a.groups; g++) {
      const double other = __shfl(score, g, 64);
      before += other > score || (other == score && g < lane);
    }
    const uint64_t kept = __ballot(lane < a.groups && before < a.kept);
#pragma unroll
    for (int v = 0; v < V; v++)
      if (!(kept >> ((lane + 64 * v) / size & 63) & 1)) c[v] = kNone;
  }
  // one choice a turn; lane j keeps the j-th
  int chosen = -1;
  double weight = 0.0;
  for (int j = 0; j < a.top; j++) {
    double best = kNone;
    int at = 0;
#pragma unroll
    for (int v = 0; v < V; v++)
      if (c[v] > best) {
        best = c[v];
        at = lane + 64 * v;
      }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const double other = __shfl_xor(best, o, 64);
      const int other_at = __shfl_xor(at, o, 64);
      if (other > best || (other == best && other_at < at)) {
        best = other;
        at = other_at;
      }
    }
    if (!(best > kNone)) break;
    double w = 0.0;
#pragma unroll
    for (int v = 0; v < V; v++)
      if (at == lane + 64 * v) {
        w = s[v];
        c[v] = kNone;
      }
    w = __shfl(w, at & 63, 64);
    if (lane == j) {
      chosen = at;
      weight = w;
    }
  }
  if (a.renorm) {
    const double sum = wave_sum(weight);
    weight = sum > 0.0 ? weight / sum : 0.0;
  }
  if (lane >= a.top) return;
  float w = (float)(weight * (double)a.scale);
  if (bad) {
    chosen = -1;
    w = __builtin_nanf("");
  } else if (chosen < 0) {
    w = 0.0f;
  }
  a.chosen[t * a.top + lane] = chosen;
  a.weights[t * a.top + lane] = w;
}

// How often each expert, a workgroup's number, was chosen.
__global__ __launch_bounds__(256) void count_kernel(const int32_t* chosen, int pairs, int32_t* counts) {
  __shared__ int32_t part[4];
  int n = 0;
  for (int i = threadIdx.x; i < pairs; i += 256) n += chosen[i] == (int)blockIdx.x;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o, 64);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = n;
  __syncthreads();
  if (threadIdx.x == 0) counts[blockIdx.x] = part[0] + part[1] + part[2] + part[3];
}

// Workgroup e places expert e's pairs; the last one what belongs to none.
__global__ __launch_bounds__(256) void place_kernel(MoeRoute a, int pairs, const int32_t* counts) {
  __shared__ int32_t part[4], seen[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = blockIdx.x;
  int base = 0;
  for (int i = threadIdx.x; i < e; i += 256) base += counts[i];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) base += __shfl_xor(base, o, 64);
  if (lane == 0) part[wave] = base;
  __syncthreads();
  base = part[0] + part[1] + part[2] + part[3];
  if (threadIdx.x == 0) a.offsets[e] = base;
  if (e == a.experts) {
    for (int i = threadIdx.x; i < pairs; i += 256) {
      if (a.chosen[i] < 0) a.slots[i] = -1;
      if (i >= base) a.rows[i] = -1;
    }
    return;
  }
  for (int i0 = 0; i0 < pairs; i0 += 256) {
    const int i = i0 + threadIdx.x;
    const bool mine = i < pairs && a.chosen[i] == e;
    const uint64_t all = __ballot(mine);
    if (lane == 0) seen[wave] = __popcll(all);
    __syncthreads();
    int at = base + __popcll(all & ((1ull << lane) - 1));
    for (int w = 0; w < wave; w++) at += seen[w];
    if (mine) {
      a.slots[i] = at;
      a.rows[at] = i / a.top;
    }
    base += seen[0] + seen[1] + seen[2] + seen[3];
    __syncthreads();
  }
}

template <typename T> hipError_t run_route(const MoeRoute& a, hipStream_t stream) {
  if (a.tokens == 0) return hipSuccess;
  const dim3 grid((unsigned)((a.tokens + kWaves - 1) / kWaves)), threads(64 * kWaves);
  const int e = a.experts;
  if (e <= 64) hipLaunchKernelGGL((route_kernel<T, 1>), grid, threads, 0, stream, a);
  else if (e <= 128) hipLaunchKernelGGL((route_kernel<T, 2>), grid, threads, 0, stream, a);
  else if (e <= 256) hipLaunchKernelGGL((route_kernel<T, 4>), grid, threads, 0, stream, a);
  else if (e <= 512) hipLaunchKernelGGL((route_kernel<T, 8>), grid, threads, 0, stream, a);
  else hipLaunchKernelGGL((route_kernel<T, 16>), grid, threads, 0, stream, a);
  return hipGetLastError();
}

// N elements of a row a thread, at once where N > 1.
template <typename T, int N> __global__ __launch_bounds__(256) void combine_kernel(MoeCombine a) {
  typedef T V __attribute__((ext_vector_type(N)));
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * N;
  if (c >= a.cols) return;
  for (int64_t t = blockIdx.y; t < a.tokens; t += gridDim.y) {
    float v[N];
    if (a.add) {
      const V add = *(const V*)((const T*)a.add + t * a.add_stride + c);
#pragma unroll
      for (int i = 0; i < N; i++) v[i] = (float)add[i];
    } else {
#pragma unroll
      for (int i = 0; i < N; i++) v[i] = 0.0f;
    }
    for (int j = 0; j < a.top; j++) {
      const int64_t s = a.slots[t * a.top + j];
      const float w = a.weights[t * a.top + j];
      V y = {};
      if (s >= 0 && s < a.y_rows) y = *(const V*)((const T*)a.y + s * a.y_stride + c);
#pragma unroll
      for (int i = 0; i < N; i++) v[i] += w * (float)y[i];
    }
    V o;
#pragma unroll
    for (int i = 0; i < N; i++) o[i] = mx_cvt<T>(v[i]);
    *(V*)((T*)a.out + t * a.cols + c) = o;
  }
}

template <typename T> hipError_t run_combine(const MoeCombine& a, hipStream_t stream) {
  constexpr int kAll = 16 / sizeof(T);
  const uintptr_t any = (uintptr_t)a.y | (uintptr_t)a.add | (uintptr_t)a.out | (uintptr_t)(a.cols * sizeof(T)) |
                        (uintptr_t)(a.y_stride * sizeof(T)) | (uintptr_t)(a.add ? a.add_stride * sizeof(T) : 0);
  const int n = any & 15 ? 1 : kAll;
  const dim3 grid((unsigned)((a.cols + 256 * n - 1) / (256 * n)), (unsigned)std::min(a.tokens, (int64_t)65535));
  if (n == 1) hipLaunchKernelGGL((combine_kernel<T, 1>), grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((combine_kernel<T, kAll>), grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

size_t moe_route_ws_bytes(int64_t, int64_t experts, int64_t) { return (size_t)experts * 4; }

hipError_t launch_moe_route(const MoeRoute& a, void* ws, hipStream_t stream) {
  const hipError_t e = a.dtype == kF32   ? run_route<float>(a, stream)
                       : a.dtype == kF16 ? run_route<_Float16>(a, stream)
                                         : run_route<__bf16>(a, stream);
  if (e != hipSuccess || !a.offsets) return e;
  const int pairs = (int)(a.tokens * a.top);
  hipLaunchKernelGGL(count_kernel, dim3((unsigned)a.experts), dim3(256), 0, stream, a.chosen, pairs, (int32_t*)ws);
  hipLaunchKernelGGL(place_kernel, dim3((unsigned)a.experts + 1), dim3(256), 0, stream, a, pairs, (const int32_t*)ws);
  return hipGetLastError();
}

hipError_t launch_moe_combine(const MoeCombine& c, hipStream_t stream) {
  if (c.dtype == kF32) return run_combine<float>(c, stream);
  if (c.dtype == kF16) return run_combine<_Float16>(c, stream);
  return run_combine<__bf16>(c, stream);
}

}  // namespace rz
