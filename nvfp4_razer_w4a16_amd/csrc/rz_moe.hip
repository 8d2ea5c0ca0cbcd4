// rz_moe.hip -- routing of tokens to experts and the combination of the experts' rows
// on gfx950.
//
// Route: s = softmax(l) or sigmoid(l), c = s + bias, the `top` largest c of the groups
// kept, weights s (over their sum) times a scale.  Scores and their comparisons are in
// fp64: of 256 experts the last chosen and the first not chosen lie within an fp32
// rounding of each other once in some ten thousand tokens, and the choice would then
// depend on how exp rounds.
// Order: the pairs (token, place) sorted by expert, then token.
// Combine: out[t] = add[t] + sum_j w[t, j] y[slots[t, j]].
//
// Route and order are bound by instructions and by launches: 8192 tokens of 256 experts,
// 8 of them out of 4 of 8 groups by sigmoid, 17.3-17.7 us of route (690 vector
// instructions a token: 300 for logits and fp64 scores, 165 for the groups, 25 for each
// choice) and 6.6 us of order; 333 tokens of 64 experts 4.3 and 5.2 us; one token, in one
// launch, 6.2 us of latency.  (Comparing fp64 scores across the wave took 33-43 us.)
// Combine is bound by memory: 8192 tokens of 8 rows of 4096 in bf16 131-134 us (671 MB, 5.0-5.1
// TB/s; a copy of 1 GiB reaches 5.1), 4124 of 3 rows of 746 in f32 11.7 us (4.2 TB/s; an element
// a thread took 18.7).  A thread takes 16 bytes of a row and adds up its
// token's rows in registers, so that every row is read once and nothing meets elsewhere.
#include <algorithm>

#include "rz_mx.h"
#include "rz_moe_launch.h"

namespace rz {

namespace {

constexpr double kNone = -__builtin_inf();
constexpr float kNone32 = -__builtin_inff();

// ---- over a wave: row shifts by 1, 2, 4, 8, then lane 15 and 31 of the rows before, to
// lane 63; lanes without a source combine with `old`
template <int CTRL> __device__ __forceinline__ int dpp(int old, int v) {
  return __builtin_amdgcn_update_dpp(old, v, CTRL, 0xF, 0xF, false);
}
template <int CTRL> __device__ __forceinline__ float dpp(float old, float v) {
  return u2f((uint32_t)dpp<CTRL>((int)f2u(old), (int)f2u(v)));
}
template <int CTRL> __device__ __forceinline__ double dpp(double old, double v) {
  const uint64_t o = __builtin_bit_cast(uint64_t, old), n = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)dpp<CTRL>((int)(uint32_t)o, (int)(uint32_t)n);
  const uint32_t hi = (uint32_t)dpp<CTRL>((int)(uint32_t)(o >> 32), (int)(uint32_t)(n >> 32));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return u2f((uint32_t)__builtin_amdgcn_readlane((int)f2u(v), lane));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t n = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)n, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(n >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <typename T> __device__ __forceinline__ T wave_max(T v) {
  v = max(v, dpp<0x111>(v, v));
  v = max(v, dpp<0x112>(v, v));
  v = max(v, dpp<0x114>(v, v));
  v = max(v, dpp<0x118>(v, v));
  v = max(v, dpp<0x142>(v, v));
  v = max(v, dpp<0x143>(v, v));
  return lane_value(v, 63);
}
// The same of whole numbers, 0 where a lane has no source: a step is one instruction.
__device__ __forceinline__ uint32_t wave_max_key(uint32_t v) {
  v = max(v, (uint32_t)dpp<0x111>(0, (int)v));
  v = max(v, (uint32_t)dpp<0x112>(0, (int)v));
  v = max(v, (uint32_t)dpp<0x114>(0, (int)v));
  v = max(v, (uint32_t)dpp<0x118>(0, (int)v));
  v = max(v, (uint32_t)dpp<0x142>(0, (int)v));
  v = max(v, (uint32_t)dpp<0x143>(0, (int)v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
// A whole number above 0 for each float but NaN, in the floats' order (zeros as one).
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = f2u(f + 0.0f);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp<0x111>(0.0, v);
  v += dpp<0x112>(0.0, v);
  v += dpp<0x114>(0.0, v);
  v += dpp<0x118>(0.0, v);
  // lane 15 of a row holds the row's sum: rows 1 and 3 add the row before, then rows 2 and 3 lane 31's
  const double row = dpp<0x142>(0.0, v);
  if (threadIdx.x & 16) v += row;
  const double half = dpp<0x143>(0.0, v);
  if (threadIdx.x & 32) v += half;
  return lane_value(v, 63);
}

// A wave's row of logits, or the bias: lane l holds experts l, l + 64 ...
template <typename T, int V> __device__ __forceinline__ void load_row(const T* row, int experts, float none, float (&l)[V]) {
#pragma unroll
  for (int v = 0; v < V; v++) {
    const int e = (threadIdx.x & 63) + 64 * v;
    l[v] = row && e < experts ? (float)row[e] : none;
  }
}

// The experts of one token: lane j's place j, -1 and 0 for none (lanes from `top` on too).
// `keys` is LDS of 64 V.
//
// Turns of choice compare the fp32 roundings of c, as whole numbers in their order:
// rounding keeps the order, so only entries of an equal rounding are compared in fp64.
template <int V>
__device__ __forceinline__ void route_token(const MoeRoute& a, const float (&l)[V], const float (&bias)[V], double* keys,
                                            int& chosen, float& weight) {
  const int lane = threadIdx.x & 63;
  float m = kNone32;
  bool bad = false;
#pragma unroll
  for (int v = 0; v < V; v++) {
    bad |= !(l[v] < __builtin_inff());
    m = fmaxf(m, l[v]);
  }
  chosen = -1;
  weight = 0.0f;
  if (__ballot(bad)) {
    weight = __builtin_nanf("");
    return;
  }
  double s[V], c[V];
  if (a.sigmoid) {
#pragma unroll
    for (int v = 0; v < V; v++) s[v] = 1.0 / (1.0 + exp(-(double)l[v]));
  } else {
    m = wave_max(m);
    if (m == kNone32) return;
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < V; v++) {
      s[v] = exp((double)l[v] - (double)m);
      sum += s[v];
    }
    const double inverse = 1.0 / wave_sum(sum);
#pragma unroll
    for (int v = 0; v < V; v++) s[v] *= inverse;
  }
#pragma unroll
  for (int v = 0; v < V; v++) {
    c[v] = s[v] + (double)bias[v];
    if (!(c[v] > kNone) || l[v] == kNone32) c[v] = kNone;
  }
  if (a.groups > 1) {
    // 64 / groups lanes (a power of two) score a group
    const int size = a.experts / a.groups;
    int per = 64;
    while (per * a.groups > 64) per >>= 1;
    const int group = lane / per;
#pragma unroll
    for (int v = 0; v < V; v++) keys[lane + 64 * v] = c[v];
    wave_lds_sync();
    double first = kNone, second = kNone;
    if (group < a.groups)
      for (int i = lane % per; i < size; i += per) {
        const double k = keys[group * size + i];
        second = max(second, min(first, k));
        first = max(first, k);
      }
    for (int o = 1; o < per; o <<= 1) {
      const double f = __shfl_xor(first, o, 64), g = __shfl_xor(second, o, 64);
      second = max(max(second, g), min(first, f));
      first = max(first, f);
    }
    const double score = a.best == 2 && second > kNone ? first + second : first;
    int before = 0;  // groups that are better
    if (a.groups <= per) {  // a lane compares its group with one other
      const int g = lane % per;
      const double other = __shfl(score, min(g, a.groups - 1) * per, 64);
      const uint64_t better = __ballot(g < a.groups && (other > score || (other == score && g < group)));
      before = __popc((uint32_t)(better >> (group * per & 63)) & (uint32_t)((1ull << per) - 1));
    } else {
      for (int g = 0; g < a.groups; g++) {
        const double other = lane_value(score, g * per);
        before += other > score || (other == score && g < group);
      }
    }
    const uint64_t kept = __ballot(before < a.kept);
    const uint32_t mul = (1u << 20) / (uint32_t)size + 1;  // e / size for e < 1024
#pragma unroll
    for (int v = 0; v < V; v++) {
      const int g = (int)((uint32_t)(lane + 64 * v) * mul >> 20);
      if (!(kept >> (g * per & 63) & 1)) c[v] = kNone;
    }
    wave_lds_sync();  // the next token writes the keys again
  }
  uint32_t key[V];  // 0: none
#pragma unroll
  for (int v = 0; v < V; v++) key[v] = c[v] == kNone ? 0 : order_key((float)c[v]);
  for (int j = 0; j < a.top; j++) {
    uint32_t best = key[0];
#pragma unroll
    for (int v = 1; v < V; v++) best = max(best, key[v]);
    best = wave_max_key(best);
    if (best == 0) break;
    int at = -1, count = 0;
#pragma unroll
    for (int v = V - 1; v >= 0; v--) {
      const uint64_t equal = __ballot(key[v] == best);
      count += __popcll(equal);
      if (equal) at = 64 * v + __builtin_ctzll(equal);
    }
    if (count == 1) {
#pragma unroll
      for (int v = 0; v < V; v++) key[v] = key[v] == best ? 0 : key[v];
    } else {
      double most = kNone;
#pragma unroll
      for (int v = 0; v < V; v++)
        if (key[v] == best) most = max(most, c[v]);
      most = wave_max(most);
#pragma unroll
      for (int v = V - 1; v >= 0; v--) {
        const uint64_t equal = __ballot(key[v] == best && c[v] == most);
        if (equal) at = 64 * v + __builtin_ctzll(equal);
      }
#pragma unroll
      for (int v = 0; v < V; v++)
        if (lane + 64 * v == at) key[v] = 0;
    }
    if (lane == j) chosen = at;
  }
  // the chosen experts' scores, from the lanes that hold them
  double mine = 0.0;
#pragma unroll
  for (int v = 0; v < V; v++) {
    const double w = __shfl(s[v], chosen & 63, 64);
    if (chosen >> 6 == v) mine = w;
  }
  if (a.renorm) {
    const double sum = wave_sum(mine);
    mine = sum > 0.0 ? mine / sum : 0.0;
  }
  weight = chosen < 0 ? 0.0f : (float)(mine * (double)a.scale);
}

// ---- order ---------------------------------------------------------------------
// Tokens are taken in blocks of at most 32.  The route kernel leaves how often each
// expert occurs in a block, a byte each; the place kernel adds up what stands before its
// own block, of many blocks by way of the sums of 64 at a time.  Within a block, an expert
// has a bit for each token (it occurs once a token at most), and the bits below a token's
// count the pairs before it.  All of it is integers, so the order in which waves come
// changes nothing.
constexpr int kPairs = 512;          // most pairs of a block
constexpr int kDirect = 256;         // blocks whose counts every block adds up for itself
constexpr int kGroup = 64;           // otherwise: blocks of a group
// Tokens that one workgroup of eight or 16 waves routes and orders.  Two a wave are as quick
// as two launches for up to 64 experts alone; 16 waves of more than 256 do not fit the
// registers.  One workgroup and two launches, us captured and called one by one: 32 tokens of
// 64 experts 8.4, 10.4 and 8.8, 14.7; 16 of 256 (of groups) 10.8, 11.3 and 11.3, 15.2; 32 of
// 256 16.9, 15.8 and 11.6, 15.1.
constexpr int most_alone(int experts) { return experts <= 64 ? 32 : experts <= 256 ? 16 : 8; }

struct OrderPlan {
  int per;              // tokens of a block
  int blocks, groups;   // groups 0: none
  int row;              // bytes of a block's counts, whole dwords
  size_t counts, sums;  // bytes of the counts and of the groups' sums
};
// blocks 0: one workgroup for all.  (Without an order nothing asks for one, and the second of
// two tokens would wait.)
OrderPlan order_plan(int64_t tokens, int64_t experts, int64_t top, bool order) {
  OrderPlan p = {};
  if (tokens <= (order ? most_alone((int)experts) : 8)) return p;
  p.per = (int)std::min(std::max((tokens + 255) / 256, (int64_t)4), std::min((int64_t)32, kPairs / top));
  p.blocks = (int)((tokens + p.per - 1) / p.per);
  p.groups = p.blocks > kDirect ? (p.blocks + kGroup - 1) / kGroup : 0;
  p.row = ((int)experts + 3) & ~3;
  p.counts = ((size_t)p.blocks * p.row + 15) & ~(size_t)15;
  p.sums = (size_t)p.groups * p.row * 4;
  return p;
}

// The exclusive prefix sum of start[0 .. n) over the workgroup's N threads, in place;
// returns the total.  `part` is LDS of N / 64.
template <int N> __device__ __forceinline__ int prefix(int* start, int n, int* part) {
  constexpr int kEach = 1024 / N;  // experts a thread, n <= 1024
  const int tid = threadIdx.x, lane = tid & 63;
  int v[kEach], sum = 0;
#pragma unroll
  for (int i = 0; i < kEach; i++) {
    v[i] = tid * kEach + i < n ? start[tid * kEach + i] : 0;
    sum += v[i];
  }
  int scan = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int up = __shfl_up(scan, o, 64);
    if (lane >= o) scan += up;
  }
  if (lane == 63) part[tid >> 6] = scan;
  __syncthreads();
  int before = scan - sum, total = 0;
#pragma unroll
  for (int w = 0; w < N / 64; w++) {
    if (w < tid >> 6) before += part[w];
    total += part[w];
  }
#pragma unroll
  for (int i = 0; i < kEach; i++) {
    if (tid * kEach + i < n) start[tid * kEach + i] = before;
    before += v[i];
  }
  __syncthreads();
  return total;
}

// The places of the list's pairs, from `start` for each expert; `bits` is LDS of an int an expert.
template <int N>
__device__ __forceinline__ void place(const MoeRoute& a, const int* list, int n, int64_t first, const int* start, uint32_t* bits) {
  for (int e = threadIdx.x; e < a.experts; e += N) bits[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += N)
    if (list[i] >= 0) atomicOr(&bits[list[i]], 1u << i / a.top);
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += N) {
    const int e = list[i], t = i / a.top;
    int at = -1;
    if (e >= 0) {
      at = start[e] + __popc(bits[e] & ((1u << t) - 1));
      a.rows[at] = (int)(first / a.top) + t;
    }
    a.slots[first + i] = at;
  }
}

// All of a few tokens' routing and order.
template <typename T, int V, int WAVES> __global__ __launch_bounds__(64 * WAVES) void route_one_kernel(MoeRoute a) {
  constexpr int N = 64 * WAVES, kTokens = most_alone(64 * V);
  __shared__ double keys[WAVES][64 * V];
  __shared__ __attribute__((aligned(16))) int list[kTokens * 32], start[1024], part[WAVES];
  __shared__ uint32_t bits[1024];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = (int)a.tokens * a.top;
  float bias[V];
  if (wave < a.tokens) load_row(a.bias, a.experts, 0.0f, bias);
  for (int t = wave; t < a.tokens; t += WAVES) {
    int chosen;
    float w, l[V];
    load_row((const T*)a.logits + t * a.stride, a.experts, kNone32, l);
    route_token(a, l, bias, keys[wave], chosen, w);
    if (lane < a.top) {
      a.chosen[t * a.top + lane] = chosen;
      a.weights[t * a.top + lane] = w;
      list[t * a.top + lane] = chosen;
    }
  }
  if (!a.offsets) return;
  for (int e = tid; e < a.experts; e += N) start[e] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += N)
    if (list[i] >= 0) atomicAdd(&start[list[i]], 1);
  __syncthreads();
  const int total = prefix<N>(start, a.experts, part);
  for (int e = tid; e < a.experts; e += N) a.offsets[e] = start[e];
  if (tid == 0) a.offsets[a.experts] = total;
  for (int i = tid; i < n; i += N)
    if (i >= total) a.rows[i] = -1;
  place<N>(a, list, n, 0, start, bits);
}

// A block's tokens, a wave a token, and the counts of their experts.  A token is some 5 us
// of latency to a wave: most of it is hidden where a SIMD has several.
constexpr int most_waves(int v) { return v <= 4 ? 16 : v <= 8 ? 8 : 4; }
template <typename T, int V>
__global__ __launch_bounds__(64 * most_waves(V)) void route_kernel(MoeRoute a, OrderPlan plan, uint8_t* counts) {
  __shared__ double keys[most_waves(V)][64 * V];
  __shared__ int found[64 * V];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, threads = blockDim.x, waves = threads >> 6;
  if (counts) {
    for (int e = tid; e < 64 * V; e += threads) found[e] = 0;
    __syncthreads();
  }
  const int64_t first = (int64_t)blockIdx.x * plan.per, end = min(first + plan.per, a.tokens);
  const T* row = (const T*)a.logits + (first + wave) * a.stride;
  float next[V], bias[V];
  load_row(a.bias, a.experts, 0.0f, bias);
  load_row(first + wave < end ? row : nullptr, a.experts, kNone32, next);
  for (int64_t t = first + wave; t < end; t += waves) {
    int chosen;
    float w, l[V];
#pragma unroll
    for (int v = 0; v < V; v++) l[v] = next[v];
    row += waves * a.stride;
    load_row(t + waves < end ? row : nullptr, a.experts, kNone32, next);  // under this token's work
    route_token(a, l, bias, keys[wave], chosen, w);
    if (lane < a.top) {
      a.chosen[t * a.top + lane] = chosen;
      a.weights[t * a.top + lane] = w;
      if (counts && chosen >= 0) atomicAdd(&found[chosen], 1);
    }
  }
  if (!counts) return;
  __syncthreads();
  for (int e = tid; e < plan.row; e += threads) counts[(int64_t)blockIdx.x * plan.row + e] = (uint8_t)found[e];
}

// Counts of blocks [lo, hi), two in a register: sums of at most 256 blocks stay within 16
// bits.  `shares` threads take the blocks of each dword in turn.
struct Counts {
  uint32_t even = 0, odd = 0;
  __device__ __forceinline__ void add(uint32_t c) {
    even += c & 0x00FF00FF;
    odd += c >> 8 & 0x00FF00FF;
  }
};
// f(i, p[i * stride]) for i = lo, lo + step .. below hi, 16 loads at a time under way (a
// plain loop waits for each: its length differs from lane to lane).
template <typename T, typename F>
__device__ __forceinline__ void for_rows(const T* p, int lo, int hi, int step, int stride, F f) {
  for (int i = lo; i < hi; i += 16 * step) {
    T v[16];
#pragma unroll
    for (int k = 0; k < 16; k++) v[k] = p[(int64_t)min(i + k * step, hi - 1) * stride];
#pragma unroll
    for (int k = 0; k < 16; k++)
      if (i + k * step < hi) f(i + k * step, v[k]);
  }
}
__device__ __forceinline__ int count_of(const uint32_t* even, const uint32_t* odd, int e) {
  return (int)((e & 1 ? odd : even)[e >> 2] >> (e & 2) * 8 & 0xFFFF);
}

// The sums of a group's counts.
__global__ __launch_bounds__(256) void sum_kernel(OrderPlan plan, const uint32_t* counts, int* sums) {
  __shared__ uint32_t even[256], odd[256];
  const int tid = threadIdx.x, words = plan.row / 4, shares = 256 / words, share = tid / words, w = tid - share * words;
  even[tid] = odd[tid] = 0;
  __syncthreads();
  const int lo = blockIdx.x * kGroup, hi = min(lo + kGroup, plan.blocks);
  if (share < shares) {
    Counts c;
    for_rows(counts + w, lo + share, hi, shares, words, [&](int, uint32_t v) { c.add(v); });
    atomicAdd(&even[w], c.even);
    atomicAdd(&odd[w], c.odd);
  }
  __syncthreads();
  for (int e = tid; e < plan.row; e += 256) sums[(int64_t)blockIdx.x * plan.row + e] = count_of(even, odd, e);
}

// The places of a block's pairs.
constexpr int kPlace = 512;
static_assert(kPairs <= kPlace, "a pair a thread");
__global__ __launch_bounds__(kPlace) void place_kernel(MoeRoute a, OrderPlan plan, const uint32_t* counts, const int* sums) {
  __shared__ int list[kPairs], all[1024], start[1024], part[kPlace / 64];
  __shared__ uint32_t even[256], odd[256], even0[256], odd0[256], bits[1024];
  const int tid = threadIdx.x, b = blockIdx.x;
  const int64_t first = (int64_t)b * plan.per * a.top, pairs = a.tokens * a.top;
  const int n = (int)min((int64_t)plan.per * a.top, pairs - first);
  // all loads first: counts before this block and, where there are no groups, in all (of
  // the others' groups their sums)
  const int mine = tid < n ? a.chosen[first + tid] : -1;
  const int lo = plan.groups ? b / kGroup * kGroup : 0, hi = plan.groups ? b : plan.blocks;
  const int words = plan.row / 4, shares = kPlace / words, share = tid / words, w = tid - share * words;
  Counts c, before;
  if (share < shares)
    for_rows(counts + w, lo + share, hi, shares, words, [&](int i, uint32_t v) {
      c.add(v);
      before.add(i < b ? v : 0);
    });
  if (tid < n) list[tid] = mine;
  for (int e = tid; e < plan.row; e += kPlace) all[e] = start[e] = 0;
  if (tid < 256) even[tid] = odd[tid] = even0[tid] = odd0[tid] = 0;
  __syncthreads();
  if (share < shares) {
    atomicAdd(&even[w], c.even);
    atomicAdd(&odd[w], c.odd);
    atomicAdd(&even0[w], before.even);
    atomicAdd(&odd0[w], before.odd);
  }
  if (plan.groups) {
    const int shares = max(kPlace / plan.row, 1), share = tid / plan.row;
    for (int e = tid - share * plan.row; share < shares && e < plan.row; e += kPlace) {
      int total = 0, before = 0;
      for_rows(sums + e, share, plan.groups, shares, plan.row, [&](int g, int v) {
        total += v;
        before += g < b / kGroup ? v : 0;
      });
      atomicAdd(&all[e], total);
      atomicAdd(&start[e], before);
    }
  }
  __syncthreads();
  for (int e = tid; e < a.experts; e += kPlace) {
    if (!plan.groups) all[e] = count_of(even, odd, e);
    start[e] += count_of(even0, odd0, e);
  }
  __syncthreads();
  const int total = prefix<kPlace>(all, a.experts, part);
  for (int e = tid; e < a.experts; e += kPlace) {
    start[e] += all[e];
    if (b == 0) a.offsets[e] = all[e];
  }
  if (b == 0 && tid == 0) a.offsets[a.experts] = total;
  for (int i = tid; i < n; i += kPlace)  // this block's share of the rows that hold none
    if (first + i >= total) a.rows[first + i] = -1;
  __syncthreads();
  place<kPlace>(a, list, n, first, start, bits);
}

// offsets of no tokens
__global__ __launch_bounds__(256) void empty_kernel(MoeRoute a) {
  for (int e = threadIdx.x; e <= a.experts; e += 256) a.offsets[e] = 0;
}

template <typename T, int V> hipError_t go_route(const MoeRoute& a, const OrderPlan& p, uint8_t* counts, hipStream_t s) {
  if (!p.blocks) {
    if constexpr (V <= 4)
      if (a.tokens > 8) {
        hipLaunchKernelGGL((route_one_kernel<T, V, 16>), dim3(1), dim3(64 * 16), 0, s, a);
        return hipGetLastError();
      }
    hipLaunchKernelGGL((route_one_kernel<T, V, 8>), dim3(1), dim3(64 * 8), 0, s, a);
  } else
    hipLaunchKernelGGL((route_kernel<T, V>), dim3((unsigned)p.blocks), dim3(64 * std::min(p.per, most_waves(V))), 0, s, a,
                       p, counts);
  return hipGetLastError();
}
template <typename T> hipError_t run_route(const MoeRoute& a, const OrderPlan& p, uint8_t* counts, hipStream_t s) {
  const int e = a.experts;
  if (e <= 64) return go_route<T, 1>(a, p, counts, s);
  if (e <= 128) return go_route<T, 2>(a, p, counts, s);
  if (e <= 256) return go_route<T, 4>(a, p, counts, s);
  if (e <= 512) return go_route<T, 8>(a, p, counts, s);
  return go_route<T, 16>(a, p, counts, s);
}

// N elements of a row a thread, 2^shift threads a row (or a piece of it).  ALIGNED: rows at
// multiples of 16 bytes, of whole pieces; otherwise loads and stores cross lines, and where
// a row's last piece is shorter its thread takes the row's last N elements and stores what
// is its own (the others may be another thread's result already).  WAVE: a wave has one row, whose slots and weights then take
// scalar loads.
template <typename T, int N, bool ALIGNED, bool WAVE> __global__ __launch_bounds__(256) void combine_kernel(MoeCombine a, int shift) {
  typedef T V __attribute__((ext_vector_type(N)));
  const int64_t own = (((int64_t)blockIdx.x << shift) + (threadIdx.x & ((1u << shift) - 1))) * N;
  if (own >= a.cols) return;
  const int64_t c = ALIGNED ? own : min(own, max(a.cols - N, (int64_t)0));
  const int skip = (int)(own - c), end = (int)min(a.cols - c, (int64_t)N);
  auto load = [&](const void* rows, int64_t at) {
    const T* p = (const T*)rows + at;
    V v = {};
    if (ALIGNED) {
      v = *(const V*)p;
    } else if (end == N) {
      __builtin_memcpy(&v, p, sizeof(V));
    } else {  // rows shorter than a piece
#pragma unroll
      for (int i = 0; i < N - 1; i++)
        if (i < end) v[i] = p[i];
    }
    return v;
  };
  const int64_t step = (int64_t)gridDim.y * (256 >> shift);
  const int row = WAVE ? __builtin_amdgcn_readfirstlane((int)threadIdx.x >> shift) : (int)threadIdx.x >> shift;
  for (int64_t t = (int64_t)blockIdx.y * (256 >> shift) + row; t < a.tokens; t += step) {
    float v[N];
    if (a.add) {
      const V add = load(a.add, t * a.add_stride + c);
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
      if (s >= 0 && s < a.y_rows) y = load(a.y, s * a.y_stride + c);
#pragma unroll
      for (int i = 0; i < N; i++) v[i] += w * (float)y[i];
    }
    V o;
#pragma unroll
    for (int i = 0; i < N; i++) o[i] = mx_cvt<T>(v[i]);
    T* out = (T*)a.out + t * a.cols + c;
    if (ALIGNED) {
      *(V*)out = o;
    } else if (skip == 0 && end == N) {
      __builtin_memcpy(out, &o, sizeof(V));
    } else {
#pragma unroll
      for (int i = 0; i < N; i++)
        if (i >= skip && i < end) out[i] = o[i];
    }
  }
}

template <typename T> hipError_t run_combine(const MoeCombine& a, hipStream_t stream) {
  constexpr int N = 16 / sizeof(T);
  const uintptr_t any = (uintptr_t)a.y | (uintptr_t)a.add | (uintptr_t)a.out | (uintptr_t)(a.cols * sizeof(T)) |
                        (uintptr_t)(a.y_stride * sizeof(T)) | (uintptr_t)(a.add ? a.add_stride * sizeof(T) : 0);
  const int64_t pieces = (a.cols + N - 1) / N;
  int shift = 0;
  while (shift < 8 && 1 << shift < pieces) shift++;
  const int64_t rows = 256 >> shift;
  const dim3 grid((unsigned)((pieces + (1 << shift) - 1) >> shift), (unsigned)std::min((a.tokens + rows - 1) / rows, (int64_t)65535));
  const bool aligned = !(any & 15), wave = shift >= 6;
  if (aligned && wave) hipLaunchKernelGGL((combine_kernel<T, N, true, true>), grid, dim3(256), 0, stream, a, shift);
  else if (aligned) hipLaunchKernelGGL((combine_kernel<T, N, true, false>), grid, dim3(256), 0, stream, a, shift);
  else if (wave) hipLaunchKernelGGL((combine_kernel<T, N, false, true>), grid, dim3(256), 0, stream, a, shift);
  else hipLaunchKernelGGL((combine_kernel<T, N, false, false>), grid, dim3(256), 0, stream, a, shift);
  return hipGetLastError();
}

}  // namespace

size_t moe_route_ws_bytes(int64_t tokens, int64_t experts, int64_t top) {
  const OrderPlan p = order_plan(tokens, experts, top, true);
  return p.counts + p.sums;
}

hipError_t launch_moe_route(const MoeRoute& a, void* ws, hipStream_t stream) {
  if (a.tokens == 0) {
    if (a.offsets) hipLaunchKernelGGL(empty_kernel, dim3(1), dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  const OrderPlan p = order_plan(a.tokens, a.experts, a.top, a.offsets != nullptr);
  uint8_t* counts = a.offsets ? (uint8_t*)ws : nullptr;
  const hipError_t e = a.dtype == kF32   ? run_route<float>(a, p, counts, stream)
                       : a.dtype == kF16 ? run_route<_Float16>(a, p, counts, stream)
                                         : run_route<__bf16>(a, p, counts, stream);
  if (e != hipSuccess || !a.offsets || !p.blocks) return e;
  int* sums = (int*)((uint8_t*)ws + p.counts);
  if (p.groups) hipLaunchKernelGGL(sum_kernel, dim3((unsigned)p.groups), dim3(256), 0, stream, p, (const uint32_t*)counts, sums);
  hipLaunchKernelGGL(place_kernel, dim3((unsigned)p.blocks), dim3(kPlace), 0, stream, a, p,
                     (const uint32_t*)counts, sums);
  return hipGetLastError();
}

hipError_t launch_moe_combine(const MoeCombine& c, hipStream_t stream) {
  if (c.dtype == kF32) return run_combine<float>(c, stream);
  if (c.dtype == kF16) return run_combine<_Float16>(c, stream);
  return run_combine<__bf16>(c, stream);
}

}  // namespace rz
