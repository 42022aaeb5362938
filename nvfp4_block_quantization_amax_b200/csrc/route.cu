// route.cu -- routing of tokens to experts and its gradient.
//
//   s = softmax(z) or sigmoid(z),  c = s + bias (the order of the experts),
//   the k largest c of the groups that are kept, w = s or s / sum of the
//   chosen s, times scale.
// The gradient with g_j = scale dw_j and p_j = w_j / scale:
//   softmax           dz_i = s_i (g_i - sum_j s_j g_j)             every i
//   sigmoid           dz_i = g_i s_i (1 - s_i)                     chosen i
//   softmax, renorm.  dz_i = p_i (g_i - sum_j p_j g_j)             chosen i
//   sigmoid, renorm.  dz_i = (1 - s_i) p_i (g_i - sum_j p_j g_j)   chosen i
//
// The order is that of the values in 64 bits, so that equal results come from
// any machine that computes them so.  It is found on values in 32 bits with a
// bound of their error (error_of); rows in which that bound does not part the
// choices are looked at in 64 bits.  How many those are goes by the values: with
// a bias, or without bias and groups, mostly below one in a hundred; scores in
// groups without a bias have more the farther the logits are apart, since the
// bound goes by the largest score: 32768 tokens, logits of standard deviation 1.5
// / 3 / 5 / 8: 160 experts, softmax, 3 of 8 groups 46 / 46 / 73 / 103 us (bf16), 34
// / 41 / 59 / 108 (fp32); 256 experts, sigmoid, 4 of 8 groups of pairs 36 / 36 / 70
// / 170, with a bias 34 / 36 / 32 / 35.
//
// What bounds the choice is its instructions, not memory: of 32768 tokens of 256
// experts (sigmoid, bias, 4 of 8 groups, 8 choices) 36 us (34 to 38 with the
// rows that are in doubt), 528 warp instructions per token at half the issue
// rate, and an end at which few warps still finish such rows (an SM is active
// 56 thousand cycles on average, 98 at most); the logits alone are 5.1 us at the
// measured rate, the same without bias and groups 18 to 20 us.  The gradient is
// bound by its launch and its zeros: 11.6 us for the same sizes (5.6).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cfloat>
#include <cstdint>

#include "launch.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

constexpr int kWarps = 4;
constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename Z>
__device__ __forceinline__ float lowest();
template <>
__device__ __forceinline__ float lowest<float>() { return -FLT_MAX; }
template <>
__device__ __forceinline__ float lowest<__nv_bfloat16>() { return __uint_as_float(0xFF7F0000u); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// Finite floats in their order as unsigned numbers above 0 (-0 counts as 0).
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(__fadd_rn(f, 0.0f));
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Merge two descending pairs: (a1, a2) becomes the two largest of the four.
template <typename F>
__device__ __forceinline__ void merge_two(F& a1, F& a2, F b1, F b2) {
  const F low = a1 < b1 ? a1 : b1;
  const F two = a2 < b2 ? b2 : a2;
  a1 = a1 < b1 ? b1 : a1;
  a2 = low < two ? two : low;
}

// A group's value from its two largest (-inf: there is none).  A sum below the
// finite numbers of 32 bits becomes the lowest, which still stands above a group
// without any; groups as near as that are parted in 64 bits.
__device__ __forceinline__ float group_value(float first, float second, bool pair) {
  return pair && second > -INFINITY ? fmaxf(first + second, -FLT_MAX) : first;
}
__device__ __forceinline__ double group_value(double first, double second, bool pair) {
  return pair && second > -INFINITY ? first + second : first;
}

// Finite numbers in their order as unsigned ones above 0, -inf as 0.
__device__ __forceinline__ unsigned long long ordered(double v) {
  if (!(v > -INFINITY)) return 0ull;
  const long long u = __double_as_longlong(v + 0.0);
  return static_cast<unsigned long long>(u ^ ((u >> 63) | static_cast<long long>(0x8000000000000000ull)));
}

// The choice in 64 bits, by the whole warp, for rows whose values in 32 bits
// are too near to one another to be ordered: lane j < k gets the j-th expert,
// or -1.  c: E doubles of shared memory.
template <typename Z>
__device__ __noinline__ int choose_exactly(const Z* __restrict__ z, const RouteArgs& a, double* c, int lane) {
  const float low = lowest<Z>();
  const int E = static_cast<int>(a.E), k = static_cast<int>(a.k), G = static_cast<int>(a.groups), n = E / G;
  const double none = -INFINITY;
  const bool direct = !a.bias && G == 1, softmax = a.score == NVFP4_ROUTE_SOFTMAX;
  float m = -INFINITY;
  double sum = 0.0;
  if (!direct && softmax) {
    for (int e = lane; e < E; e += 32) m = fmaxf(m, as_float(z[e]));
    m = warp_max(m);
#pragma unroll 4
    for (int e = lane; e < E; e += 32) sum += exp(static_cast<double>(as_float(z[e])) - m);
    sum = warp_sum(sum);
  }
#pragma unroll 8
  for (int e = lane; e < E; e += 32) {
    const float v = as_float(z[e]);
    double s = v;
    if (!direct) s = softmax ? exp(s - m) / sum : 1.0 / (1.0 + exp(-s));
    bool open = v > low;
    if (a.bias) {
      const float b = __ldg(a.bias + e);
      s += b;
      open &= b > -FLT_MAX;
    }
    c[e] = open ? s : none;
  }
  __syncwarp();
  unsigned kept = 1u;
  int lanes = 32;   // of a group
  if (G > 1) {
    while (lanes * G > 32) lanes >>= 1;
    const int g = lane / lanes;
    double a1 = none, a2 = none;
    if (g < G)
      for (int i = lane % lanes; i < n; i += lanes) merge_two(a1, a2, c[g * n + i], none);
    for (int o = lanes >> 1; o; o >>= 1) {
      const double b1 = __shfl_xor_sync(kAll, a1, o), b2 = __shfl_xor_sync(kAll, a2, o);
      merge_two(a1, a2, b1, b2);
    }
    const double mine = group_value(a1, a2, a.flags & NVFP4_ROUTE_GROUP_PAIR);
    int better = 0;
    for (int h = 0; h < G; ++h) {
      const double v = __shfl_sync(kAll, mine, h * lanes);
      better += v > mine || (v == mine && h < g);
    }
    kept = __ballot_sync(kAll, g < G && better < a.kept);
  }
  // values as ordered numbers, and this lane's largest with its expert
  unsigned long long* const key = reinterpret_cast<unsigned long long*>(c);
  unsigned long long best = 0ull;
  int at = E;
#pragma unroll 4
  for (int e = lane; e < E; e += 32) {
    const unsigned long long v = kept >> (e / n * lanes & 31) & 1u ? ordered(c[e]) : 0ull;
    key[e] = v;
    if (v > best) {
      best = v;
      at = e;
    }
  }
  int mine = -1;
  for (int j = 0; j < k; ++j) {
    const unsigned high = static_cast<unsigned>(best >> 32), top = __reduce_max_sync(kAll, high);
    if (top == 0u) break;
    const unsigned lo = high == top ? static_cast<unsigned>(best) : 0u, next = __reduce_max_sync(kAll, lo);
    const int e = __reduce_min_sync(kAll, high == top && lo == next ? at : E);
    if (lane == j) mine = e;
    if (at == e) {
      key[e] = 0ull;
      best = 0ull;
      at = E;
#pragma unroll 8
      for (int i = lane; i < E; i += 32) {
        const unsigned long long v = key[i];
        if (v > best) {
          best = v;
          at = i;
        }
      }
    }
  }
  return mine;
}

// Scores of lane j's choice (e < 0: none) as factors of the weights: r with
// sum r over the choices for renormalised weights, r = s without.  For
// renormalised weights a common factor is taken out, so that scores which are
// all below the smallest number still share out: softmax r = exp(z - max),
// sigmoid r = exp(z - m) / (1 + exp(z)) with m = min(max z, 0).
// top: the largest z of the choices (renormalised) or of the row (softmax).
__device__ __forceinline__ float share_at(float z, bool got, float top, int score, bool renorm, float row_sum) {
  if (!got) return 0.0f;
  if (score == NVFP4_ROUTE_SOFTMAX) {
    const float e = expf(z - top);
    return renorm ? e : __fdiv_rn(e, row_sum);
  }
  if (z > 0.0f) return __fdiv_rn(1.0f, 1.0f + expf(-z));
  return __fdiv_rn(expf(renorm ? z - fminf(top, 0.0f) : z), 1.0f + expf(z));
}

__device__ __forceinline__ float share_of(float z, bool got, int score, bool renorm, float row_max, float row_sum) {
  return share_at(z, got, renorm ? warp_max(got ? z : -INFINITY) : row_max, score, renorm, row_sum);
}

// Bound of |32-bit c - c| (see the figures behind route_kernel); share: the
// largest score, most_c: no less than any |c|.
__device__ __forceinline__ float error_of(bool softmax, float share, float most_c) {
  return (softmax ? 0x1p-18f * share : 0x1.8p-22f) + 0x1.1p-24f * most_c + FLT_MIN;
}

// Rows that have to be looked at in 64 bits wait until a warp has been through
// its others (the code for them would cost those registers).  Until then the
// first choice holds a mark: kDoubtful, if the row has to be chosen again, or
// mark - e for a first choice e, if the choices, and the expert behind them,
// whose number lies in the place of the first weight, only have to be put in
// order.  kTied in that place: the choices stand if no other expert belongs
// above the last one.
constexpr int kDoubtful = -2, kMark = -3, kTied = -2;

// The choices of a row (lane j: the j-th, or -1) with their weights.
template <typename Z>
__device__ __forceinline__ void write_row(const RouteArgs& a, int64_t t, const Z* row, int mine, int lane) {
  const int k = static_cast<int>(a.k);
  const bool softmax = a.score == NVFP4_ROUTE_SOFTMAX, renorm = a.flags & NVFP4_ROUTE_RENORM;
  float row_max = -INFINITY, row_sum = 0.0f;
  if (softmax && !renorm) {
    for (int e = lane; e < a.E; e += 32) row_max = fmaxf(row_max, as_float(row[e]));
    row_max = fmaxf(warp_max(row_max), -FLT_MAX);
    for (int e = lane; e < a.E; e += 32) row_sum += ex2((as_float(row[e]) - row_max) * kLog2e);
    row_sum = warp_sum(row_sum);
  }
  const bool got = mine >= 0;
  const float share = share_of(got ? as_float(row[mine]) : 0.0f, got, a.score, renorm, row_max, row_sum);
  const float sum = renorm ? warp_sum(share) : 1.0f;
  if (lane < k) {
    a.ids[t * k + lane] = mine;
    a.weights[t * k + lane] = got ? a.scale * (renorm ? __fdiv_rn(share, sum) : share) : 0.0f;
  }
}

template <typename Z>
__device__ __noinline__ void finish_exactly(const RouteArgs& a, int64_t t, double* c, int lane) {
  const Z* const row = static_cast<const Z*>(a.logits) + t * a.ldl;
  write_row<Z>(a, t, row, choose_exactly<Z>(row, a, c, lane), lane);
  __syncwarp();   // c is free
}

// Put the choices of a row and the expert behind them in order, by their values
// in 64 bits; c: 32 numbers of shared memory.  Adds 2.7 us to a call
// (choose_exactly with the weights, 256 experts: up to 7.6).  Not for softmax scores with
// a bias or groups: they need the whole row.
template <typename Z>
__device__ __noinline__ void settle(const RouteArgs& a, int64_t t, double* c, int lane) {
  const Z* const row = static_cast<const Z*>(a.logits) + t * a.ldl;
  const int k = static_cast<int>(a.k);
  const bool direct = !a.bias && a.groups == 1;
  int e[2] = {lane < k ? a.ids[t * k + lane] : -1, __float_as_int(a.weights[t * k])};   // of this lane, and the last one
  if (lane == 0) e[0] = kMark - e[0];
  double v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool is = e[i] >= 0;
    v[i] = is ? as_float(row[e[i]]) : 0.0f;
    if (!direct) v[i] = 1.0 / (1.0 + exp(-v[i])) + (is && a.bias ? __ldg(a.bias + e[i]) : 0.0f);
    if (!is) v[i] = -INFINITY;
  }
  const auto before = [](double x, int ex, double y, int ey) { return x > y || (x == y && ex < ey); };
  int better = before(v[1], e[1], v[0], e[0]);
  for (int j = 0; j < k; ++j) {
    const double o = __shfl_sync(kAll, v[0], j);
    const int eo = __shfl_sync(kAll, e[0], j);
    better += eo >= 0 && before(o, eo, v[0], e[0]);
  }
  int* const order = reinterpret_cast<int*>(c);
  const int place = __popc(__ballot_sync(kAll, e[0] >= 0 && before(v[0], e[0], v[1], e[1])));   // of the last one
  order[lane] = -1;
  __syncwarp();
  if (e[0] >= 0 && better < k) order[better] = e[0];
  if (lane == 0 && e[1] >= 0 && place < k) order[place] = e[1];
  __syncwarp();
  write_row<Z>(a, t, row, lane < k ? order[lane] : -1, lane);
  __syncwarp();   // c is free
}

// A row where the last choice and the expert behind it are equal and others are
// as close to them: the choices stand if those are no more than equal.  An
// expert that is unlike the last choice and not surely below it (error_of) has
// to be a choice itself, so both are counted.  Softmax scores need the whole
// row.  Logits without a bias or groups do not come here.
template <typename Z>
__device__ __noinline__ void finish_tied(const RouteArgs& a, int64_t t, double* c, int lane) {
  if (a.score == NVFP4_ROUTE_SOFTMAX) return finish_exactly<Z>(a, t, c, lane);
  const Z* const row = static_cast<const Z*>(a.logits) + t * a.ldl;
  const int k = static_cast<int>(a.k), E = static_cast<int>(a.E);
  const int id = lane < k ? a.ids[t * k + lane] : -1, mine = lane ? id : kMark - id;
  const int last = __shfl_sync(kAll, mine, k - 1);
  const float z_last = as_float(row[last]), b_last = a.bias ? __ldg(a.bias + last) : 0.0f;
  const float c_last = rcp(1.0f + ex2(-kLog2e * z_last)) + b_last;
  const auto above = [&](int e) {
    const float z = as_float(row[e]), b = a.bias ? __ldg(a.bias + e) : 0.0f;
    if ((z == z_last && b == b_last) || !(z > lowest<Z>()) || !(b > -FLT_MAX)) return false;
    const float v = rcp(1.0f + ex2(-kLog2e * z)) + b;
    return v - c_last > -2.0f * error_of(false, 1.0f, 1.0f + fmaxf(fabsf(b), fabsf(b_last)));
  };
  int n = 0;
  for (int e = lane; e < E; e += 32) n += above(e);
  if (__reduce_add_sync(kAll, n) != __popc(__ballot_sync(kAll, mine >= 0 && above(mine)))) return finish_exactly<Z>(a, t, c, lane);
  write_row<Z>(a, t, row, mine, lane);
}

template <typename Z>
__device__ __forceinline__ void finish(const RouteArgs& a, int64_t t, int mark, double* c, int lane) {
  if (mark == kDoubtful) finish_exactly<Z>(a, t, c, lane);
  else if (__float_as_int(a.weights[t * a.k]) == kTied) finish_tied<Z>(a, t, c, lane);
  else settle<Z>(a, t, c, lane);
}

// One warp per row; expert e is value e / 32 of lane e % 32, so that a row is
// read in whole lines whatever its alignment, and equal values come in the
// order (value, lane) = the experts' order.
// V: values per lane, the power of two from E / 32 on.  kDirect: no bias and
// no groups, so that the order is that of the logits themselves.
//
// The order is found on 32-bit keys: the value in its order, the low log2 V
// bits replaced by V - 1 - i for value i of the lane, so that a lane's keys
// differ and the largest one names its place.  A round takes the largest key
// of the warp; the lane that held it moves on to its second largest, which
// every lane keeps, and looks for a third only when it wins again.
// Values as near as the error of their 32-bit form (delta), or with the same
// key, may stand in the wrong order; rows with such a pair among the chosen
// and the next one, or with such groups, are chosen again in 64 bits.  Equal
// inputs are in order; but where the last choice and the next one are equal,
// any expert behind them that is as near may be unlike them and belong above
// both (`tied`).  Logits that are ordered as they are show it at once (bf16 has
// no two values as near); other values wait for finish_tied.
template <typename Z, bool kDirect>
constexpr bool kTies = !(kDirect && sizeof(Z) == 2);
template <int V>
constexpr int kRouteCtas = V <= 8 ? 8 : V == 16 ? 5 : 3;   // per SM

template <typename Z, int V, bool kDirect>
__global__ void __launch_bounds__(kWarps * 32, kRouteCtas<V>) route_kernel(const __grid_constant__ RouteArgs a) {
  extern __shared__ double route_smem[];
  pdl_entry();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = static_cast<int>(a.E), k = static_cast<int>(a.k), G = static_cast<int>(a.groups), n = E / G;
  double* const c64 = route_smem + static_cast<size_t>(warp) * max(E, 16);   // E values, or 32 numbers
  float* const c32 = reinterpret_cast<float*>(c64);   // padded: expert e at e + e / 32 <= 2 E - 1
  const Z* const logits = static_cast<const Z*>(a.logits);
  const float low = lowest<Z>();
  const bool softmax = a.score == NVFP4_ROUTE_SOFTMAX, renorm = a.flags & NVFP4_ROUTE_RENORM;
  const bool whole = softmax && (!kDirect || !renorm);   // needs the row's maximum and sum
  const unsigned inverse = ((1u << 20) + n - 1) / n;      // e / n = e inverse / 2^20 for e < 1024
  int span = 1;                                           // lanes that hold a choice, to a power of two
  while (span < k) span <<= 1;

  float bias[kDirect ? 1 : V];
  float bmax = 0.0f;
  bool bad_bias = false;
  if (!kDirect) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 32 + lane;
      bias[i] = a.bias && e < E ? __ldg(a.bias + e) : 0.0f;
      bad_bias |= !(bias[i] <= FLT_MAX);
      if (bias[i] > -FLT_MAX) bmax = fmaxf(bmax, fabsf(bias[i]));
    }
    bmax = warp_max(bmax);
  }

  bool doubts = false;   // uniform in the warp
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * kWarps) {
    const Z* const row = logits + t * a.ldl;
    float z[V];
    bool bad = bad_bias;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 32 + lane;
      z[i] = i < V / 2 || e < E ? as_float(row[e]) : -INFINITY;   // E > 16 V
    }
#pragma unroll
    for (int i = 0; i < V; ++i) bad |= !(z[i] <= FLT_MAX);
    if (__any_sync(kAll, bad)) {
      if (lane == 0 && a.status) *a.status = kStatusNonFinite;
      if (lane < k) {
        a.ids[t * k + lane] = -1;
        a.weights[t * k + lane] = 0.0f;
      }
      continue;
    }
    float row_max = -INFINITY, row_sum = 0.0f;
    float c[V];
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = z[i];
    if (whole) {
#pragma unroll
      for (int i = 0; i < V; ++i) row_max = fmaxf(row_max, z[i]);
      row_max = fmaxf(warp_max(row_max), -FLT_MAX);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float e = ex2((z[i] - row_max) * kLog2e);
        if (!kDirect) c[i] = e;
        row_sum += e;
      }
      row_sum = warp_sum(row_sum);
    }
    // bound of the error of a key's value
    float delta = 0.0f, most_c = 0.0f;   // most_c >= |c|
    if (!kDirect) {
      const float share = softmax ? rcp(fmaxf(row_sum, FLT_MIN)) : 1.0f;
      most_c = share + bmax;
      delta = error_of(softmax, share, most_c) + 0x1p-23f * static_cast<float>(V) * most_c;
      if (softmax) {
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = __fmaf_rn(c[i], share, bias[i]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = rcp(1.0f + ex2(-kLog2e * z[i])) + bias[i];
      }
    }
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool open = z[i] > low && (kDirect || bias[i] > -FLT_MAX);
      key[i] = open ? (ordered(c[i]) & ~static_cast<uint32_t>(V - 1)) | static_cast<uint32_t>(V - 1 - i) : 0u;
    }
    bool near = false;   // uniform in the warp
    if (!kDirect && G > 1) {
      // lane g * lanes: the two largest values of group g
      int lanes = 1;
      float a1 = -INFINITY, a2 = -INFINITY;
      if ((n & 31) == 0) {
        // whole registers: the warp's largest key and the largest without it
        uint32_t k1 = 0u, k2 = 0u;
        int g = 0, left = n >> 5;
        uint32_t m1 = 0u, m2 = 0u;   // of this lane
#pragma unroll
        for (int i = 0; i < V; ++i) {
          m2 = max(m2, min(m1, key[i]));
          m1 = max(m1, key[i]);
          if (--left == 0) {
            const uint32_t w1 = __reduce_max_sync(kAll, m1);
            const int src = __ffs(__ballot_sync(kAll, m1 == w1)) - 1;
            const uint32_t w2 = __reduce_max_sync(kAll, lane == src ? m2 : m1);
            if (lane == g) {
              k1 = w1;
              k2 = w2;
            }
            ++g;
            left = n >> 5;
            m1 = m2 = 0u;
          }
        }
        if (k1) a1 = from_ordered(k1);
        if (k2) a2 = from_ordered(k2);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = i * 32 + lane;
          if (i < V / 2 || e < E) c32[e + i] = key[i] ? c[i] : -INFINITY;
        }
        __syncwarp();
        lanes = 32;
        while (lanes * G > 32) lanes >>= 1;
        const int g = lane / lanes;
        if (g < G)
          for (int i = lane % lanes; i < n; i += lanes) {
            const int e = g * n + i;
            merge_two(a1, a2, c32[e + (e >> 5)], -INFINITY);
          }
        __syncwarp();   // c32 is written again in the next row
        for (int o = lanes >> 1; o; o >>= 1) {
          const float b1 = __shfl_xor_sync(kAll, a1, o), b2 = __shfl_xor_sync(kAll, a2, o);
          merge_two(a1, a2, b1, b2);
        }
      }
      const int g = lane / lanes;
      const float mine = group_value(a1, a2, a.flags & NVFP4_ROUTE_GROUP_PAIR);
      int better = 0;
      for (int h = 0; h < G; ++h) {
        const float v = __shfl_sync(kAll, mine, h * lanes);
        better += v > mine || (v == mine && h < g);
      }
      const bool keep = g < G && better < a.kept;
      const unsigned kept = __ballot_sync(kAll, keep);
      const float least = -warp_max(keep ? -mine : -INFINITY), most = warp_max(keep || g >= G ? -INFINITY : mine);
      near = most >= -FLT_MAX && !(least - most > 4.0f * delta + 0x1p-21f * most_c);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const unsigned of = (static_cast<unsigned>(i * 32 + lane) * inverse >> 20) * lanes;
        if (!(kept >> (of & 31u) & 1u)) key[i] = 0u;   // of >= 32: no expert
      }
    }
    uint32_t top = 0u, second = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      second = max(second, min(top, key[i]));
      top = max(top, key[i]);
    }
    bool spent = false;        // second is no longer known
    uint32_t my_key = 0u, w = 0u;   // lane j: the j-th choice's
    int my_src = 0, src = 0;
    uint32_t behind = 0u;   // the key behind the last choice's next
    for (int j = 0; j <= k + 1; ++j) {
      behind = __reduce_max_sync(kAll, top);
      if (j > k) break;
      w = behind;
      if (w == 0u) break;
      src = __ffs(__ballot_sync(kAll, top == w)) - 1;
      if (lane == j) {
        my_key = w;
        my_src = src;
      }
      if (lane == src) {
        if (spent) {
          // keys below w wrap to numbers above those that do not
          uint32_t most = 0u;
#pragma unroll
          for (int i = 0; i < V; ++i) most = max(most, key[i] - w);
          top = w + most < w ? w + most : 0u;
        } else {
          top = second;
          spent = true;
        }
      }
    }
    // w, src: the one behind the last choice (w = 0: none)
    const bool had = lane < k && my_key;
    uint32_t next_key = __shfl_down_sync(kAll, my_key, 1);
    int next_src = __shfl_down_sync(kAll, my_src, 1);
    if (lane == k - 1) {
      next_key = w;
      next_src = src;
    }
    int mine = had ? (V - 1 - static_cast<int>(my_key & (V - 1))) * 32 + my_src : -1;
    // neighbours that may stand in the wrong order; equal inputs do not
    const auto close = [&](uint32_t above, uint32_t below) {
      return kDirect ? (above ^ below) < static_cast<uint32_t>(V) : !(from_ordered(above) - from_ordered(below) > 2.0f * delta);
    };
    bool unsure = false, tied = false;
    if (had && next_key && close(my_key, next_key)) {
      const int next = (V - 1 - static_cast<int>(next_key & (V - 1))) * 32 + next_src;
      unsure = !(as_float(row[mine]) == as_float(row[next]) && (kDirect || !a.bias || __ldg(a.bias + mine) == __ldg(a.bias + next)));
      tied = kTies<Z, kDirect> && !unsure && lane == k - 1 && behind && close(my_key, behind);
    }
    if (kDirect && kTies<Z, kDirect> && __any_sync(kAll, tied)) {
      const uint32_t last = __shfl_sync(kAll, my_key, k - 1);
      const float z_last = as_float(row[__shfl_sync(kAll, mine, k - 1)]);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (key[i] && key[i] <= last && close(last, key[i])) unsure |= as_float(row[i * 32 + lane]) > z_last;
      tied = false;
    }
    if (near || __any_sync(kAll, unsure || tied)) {
      // the choices and the next one are all there is to it where what is behind
      // them is further below; softmax values need the whole row
      const uint32_t last = __shfl_sync(kAll, my_key, k - 1);
      const bool only_tied = !near && !__any_sync(kAll, unsure);
      const bool whole_row = !only_tied && (near || (!kDirect && softmax) || (last && behind && close(last, behind)));
      const int next = only_tied ? kTied : w ? (V - 1 - static_cast<int>(w & (V - 1))) * 32 + src : -1;
      if (lane < k && !whole_row) a.ids[t * k + lane] = lane ? mine : kMark - mine;
      if (lane == 0) {
        if (whole_row) a.ids[t * k] = kDoubtful;
        a.weights[t * k] = __int_as_float(next);
      }
      doubts = true;
      continue;
    }
    const bool got = mine >= 0;
    const float share = share_of(got ? as_float(row[mine]) : 0.0f, got, a.score, renorm, row_max, row_sum);
    float sum = share;
    if (renorm)
      for (int o = span >> 1; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    if (lane < k) {
      a.ids[t * k + lane] = mine;
      a.weights[t * k + lane] = got ? a.scale * (renorm ? __fdiv_rn(share, sum) : share) : 0.0f;
    }
  }
  if (doubts) {
    __syncwarp();
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < a.T; t += static_cast<int64_t>(gridDim.x) * kWarps) {
      const int mark = __shfl_sync(kAll, lane == 0 ? a.ids[t * k] : 0, 0);
      if (mark <= kDoubtful) finish<Z>(a, t, mark, c64, lane);
    }
  }
}
// error_of, in u = 2^-24, half a step of 32 bits.  ex2.approx is off by 4 u,
// rcp.approx by 2 u, both relative.
//   sigmoid: log2 e and its product with z are rounded, 1.25 |z| u relative to
// exp(-z), which reaches s with the factor 1 - s; 1 + exp(-z) and its reciprocal
// add 3 u s.  s (1 - s) <= 1/4 and s (1 - s) |z| <= 0.23 make that less than
// 4.4 u; the code takes 6.
//   softmax, d = max - z: d is rounded too, so exp(-d) is off by (4 + 2.25 d) u
// relative, that is by at most 4 u of the largest score's (at d = 0).  What all
// scores of a row share comes on top: the sum's terms, 4 + 2.25 times their mean
// d, which is at most ln 1024 (the entropy less the sum's logarithm); its
// additions, 31 in a lane and 5 across them; the reciprocal, 2.  In all
// 4 + (4 + 15.6) + 36 + 2 < 62 u of the largest score; the code takes 64.
//   c is rounded once more, u |c|.  The keys drop log2 V bits of c: 2 V u |c|.
// A sum of two is rounded by u of up to 2 |c|.

// ---------------------------------------------------------------------------
// Many rows.  What a row costs beyond its values (reductions, rounds, the
// weights) is a warp instruction each, so four rows share a warp: eight lanes
// per row, expert e being value e / 8 of lane e % 8.  A lane keeps its four
// largest keys in order, a round takes the largest of the eight lanes, and the
// lane that held it moves on; one that has used up its four looks through its
// values again.  k <= 8 (lane j of a row ends up with choice j) and at most
// eight groups (lane g adds up group g, from shared memory).
// ---------------------------------------------------------------------------
constexpr int kShare = 8;                 // lanes of a row
constexpr int kRowsOfWarp = 32 / kShare;
template <int V>
constexpr int kManyCtas = V <= 16 ? 7 : 5;   // per SM

__device__ __forceinline__ float share_sum(float v) {
#pragma unroll
  for (int o = kShare / 2; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float share_max(float v) {
#pragma unroll
  for (int o = kShare / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// Values of a row in shared memory, four free ones after each 32: lanes that
// read 16 bytes of different groups then meet different banks.
__device__ __forceinline__ int place(int e) { return e + (e >> 5) * 4; }

template <typename Z, int V, bool kDirect>
__global__ void __launch_bounds__(kWarps * 32, kManyCtas<V>) route_many_kernel(const __grid_constant__ RouteArgs a) {
  constexpr int kPitch = V * kShare + V + 8;   // of a row's values in shared memory; rows 8 banks apart
  // a warp's values in 32 bits (four rows), and in 64 (one row at a time)
  __shared__ __align__(16) double values[kWarps][kDirect ? V * kShare : kRowsOfWarp * kPitch / 2];
  __shared__ __align__(16) float biases[kDirect ? 1 : V * kShare];
  __shared__ int bad_bias;
  __shared__ float most_bias[kWarps];
  __shared__ uint8_t holder[kWarps][kRowsOfWarp][kShare + 1];
  pdl_entry();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = lane & (kShare - 1), r = lane / kShare;
  const int E = static_cast<int>(a.E), k = static_cast<int>(a.k), G = static_cast<int>(a.groups), n = E / G;
  const Z* const logits = static_cast<const Z*>(a.logits);
  const float low = lowest<Z>();
  const bool softmax = a.score == NVFP4_ROUTE_SOFTMAX, renorm = a.flags & NVFP4_ROUTE_RENORM;
  const bool whole = softmax && (!kDirect || !renorm);
  const unsigned inverse = ((1u << 20) + n - 1) / n;
  const unsigned before = ((1u << lane) - 1u) & (0xFFu << (lane & 24));   // lanes of this row in front of this one
  float* const c32 = reinterpret_cast<float*>(values[warp]) + (kDirect ? 0 : r * kPitch);

  float bmax = 0.0f;
  if (!kDirect) {
    if (tid == 0) bad_bias = 0;
    __syncthreads();
    bool bad = false;
    for (int e = tid; e < V * kShare; e += kWarps * 32) {
      const float b = a.bias && e < E ? __ldg(a.bias + e) : 0.0f;
      bad |= !(b <= FLT_MAX);
      biases[e] = b > -FLT_MAX ? b : -INFINITY;
      if (b > -FLT_MAX) bmax = fmaxf(bmax, fabsf(b));
    }
    bmax = warp_max(bmax);
    if (bad) bad_bias = 1;
    if (lane == 0) most_bias[warp] = bmax;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) bmax = fmaxf(bmax, most_bias[i]);
  }

  bool doubts = false;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kRowsOfWarp; t0 < a.T;
       t0 += static_cast<int64_t>(gridDim.x) * (kWarps * kRowsOfWarp)) {
    const int64_t t = t0 + r < a.T ? t0 + r : a.T - 1;   // rows behind the last are the last again, and not written
    const Z* const row = logits + t * a.ldl;
    float c[V];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * kShare + sub;
      c[i] = i < V / 2 || e < E ? as_float(row[e]) : -INFINITY;   // E > 4 V
    }
#pragma unroll
    for (int i = 0; i < V; ++i) bad |= !(c[i] <= FLT_MAX);
    if (!kDirect) bad |= bad_bias != 0;
    bad = __ballot_sync(kAll, bad) >> (lane & 24) & 0xFFu;
    float row_max = -INFINITY, row_sum = 0.0f;
    if (whole) {
#pragma unroll
      for (int i = 0; i < V; ++i) row_max = fmaxf(row_max, c[i]);
      row_max = fmaxf(share_max(row_max), -FLT_MAX);
#pragma unroll
      for (int i = 0; i < V; ++i) row_sum += ex2((c[i] - row_max) * kLog2e);
      row_sum = share_sum(row_sum);
    }
    // |32-bit c - c| <= fine, and delta for the c of a key
    float fine = 0.0f, delta = 0.0f, most_c = 0.0f;
    if (!kDirect) {
      const float share = softmax ? rcp(fmaxf(row_sum, FLT_MIN)) : 1.0f;
      most_c = share + bmax;
      fine = error_of(softmax, share, most_c);
      delta = fine + 0x1p-23f * static_cast<float>(V) * most_c;
      if (softmax) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          c[i] = c[i] > low ? __fmaf_rn(ex2((c[i] - row_max) * kLog2e), share, biases[i * kShare + sub]) : -INFINITY;
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = c[i] > low ? rcp(1.0f + ex2(-kLog2e * c[i])) + biases[i * kShare + sub] : -INFINITY;
      }
    }
    bool near = false;   // the same in a row's lanes
    unsigned kept = 0xFFu;
    if (!kDirect && G > 1) {
#pragma unroll
      for (int i = 0; i < V; ++i) c32[i * kShare + sub + i / 4 * 4] = c[i];
      __syncwarp();
      float a1 = -INFINITY, a2 = -INFINITY;
      const auto add = [&](float v) {
        a2 = fmaxf(a2, fminf(a1, v));
        a1 = fmaxf(a1, v);
      };
      if (sub < G) {
        const int first = sub * n;
        if ((n & 3) == 0) {
#pragma unroll 4
          for (int i = first; i < first + n; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(c32 + place(i));
            add(v.x);
            add(v.y);
            add(v.z);
            add(v.w);
          }
        } else {
          for (int i = first; i < first + n; ++i) add(c32[place(i)]);
        }
      }
      const bool pair = a.flags & NVFP4_ROUTE_GROUP_PAIR;
      const float mine = group_value(a1, a2, pair);   // -inf from lanes without a group
      int better = 0;
#pragma unroll
      for (int o = 1; o < kShare; ++o) {
        const float v = __shfl_xor_sync(kAll, mine, o);
        better += v > mine || (v == mine && (sub ^ o) < sub);
      }
      const bool keep = better < a.kept;
      kept = __ballot_sync(kAll, keep) >> (lane & 24) & 0xFFu;
      const float least = -share_max(keep ? -mine : -INFINITY), most = share_max(keep ? -INFINITY : mine);
      near = !bad && most >= -FLT_MAX && !(least - most > 4.0f * fine + 0x1p-22f * most_c);
    }
    uint32_t key[V];
    uint32_t l0 = 0u, l1 = 0u, l2 = 0u, l3 = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      bool open = kDirect ? c[i] > low : c[i] > -FLT_MAX;
      if (!kDirect && G > 1) open &= kept >> (static_cast<unsigned>(i * kShare + sub) * inverse >> 20 & 31u) & 1u;
      uint32_t v = open ? (ordered(c[i]) & ~static_cast<uint32_t>(V - 1)) | static_cast<uint32_t>(V - 1 - i) : 0u;
      key[i] = v;
      const uint32_t d0 = min(l0, v);
      l0 = max(l0, v);
      const uint32_t d1 = min(l1, d0);
      l1 = max(l1, d0);
      const uint32_t d2 = min(l2, d1);
      l2 = max(l2, d1);
      l3 = max(l3, d2);
    }
    uint32_t my_key = 0u, w = 0u, behind = 0u;   // behind: the key behind the last choice's next
    for (int j = 0; j <= k + 1; ++j) {
      behind = l0;
#pragma unroll
      for (int o = kShare / 2; o; o >>= 1) behind = max(behind, __shfl_xor_sync(kAll, behind, o));
      if (j > k) break;
      w = behind;
      const unsigned held = __ballot_sync(kAll, l0 == w);
      if (sub == j) my_key = w;
      if (l0 == w && !(held & before)) {
        holder[warp][r][j] = static_cast<uint8_t>(sub);
        l0 = l1;
        l1 = l2;
        l2 = l3;
        l3 = 0u;
        if (l0 == 0u) {
          // keys below w wrap to numbers above those that do not
          uint32_t most = 0u;
#pragma unroll
          for (int i = 0; i < V; ++i) most = max(most, key[i] - w);
          l0 = w + most < w ? w + most : 0u;
        }
      }
    }
    __syncwarp();
    const bool had = sub < k && my_key;
    uint32_t next_key = __shfl_down_sync(kAll, my_key, 1);
    if (sub == k - 1) next_key = w;
    int mine = had ? (V - 1 - static_cast<int>(my_key & (V - 1))) * kShare + holder[warp][r][sub] : -1;
    // Neighbours whose keys do not part them: equal inputs are in order; of two
    // that are both choices, so are those whose values themselves part them (any
    // other expert's key is below both); the rest is unsure.
    const auto close = [&](uint32_t above, uint32_t below) {
      return kDirect ? (above ^ below) < static_cast<uint32_t>(V) : !(from_ordered(above) - from_ordered(below) > 2.0f * delta);
    };
    bool unsure = false, tied = false;
    if (had && next_key && close(my_key, next_key)) {
      const int next = (V - 1 - static_cast<int>(next_key & (V - 1))) * kShare + holder[warp][r][sub + 1];
      const float z1 = as_float(row[mine]), z2 = as_float(row[next]);
      float c1 = z1, c2 = z2;
      bool equal = z1 == z2;
      if (!kDirect) {
        const float b1 = biases[mine], b2 = biases[next];
        equal &= b1 == b2;
        if (!softmax) {
          c1 = rcp(1.0f + ex2(-kLog2e * z1)) + b1;
          c2 = rcp(1.0f + ex2(-kLog2e * z2)) + b2;
        }
      }
      unsure = !equal && !((kDirect || !softmax) && sub + 1 < k && c1 - c2 > 2.0f * fine);
      tied = kTies<Z, kDirect> && equal && sub == k - 1 && behind && close(my_key, behind);
    }
    if (kDirect && kTies<Z, kDirect> && __any_sync(kAll, tied)) {
      const int from = (lane & 24) + k - 1;
      const uint32_t last = __shfl_sync(kAll, my_key, from);
      const int at = __shfl_sync(kAll, mine, from);
      if (__shfl_sync(kAll, tied, from)) {
        const float z_last = as_float(row[at]);
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (key[i] && key[i] <= last && close(last, key[i])) unsure |= as_float(row[i * kShare + sub]) > z_last;
      }
      tied = false;
    }
    // its vote also parts the uses of values
    const bool only_tied = !(__ballot_sync(kAll, unsure) >> (lane & 24) & 0xFFu) && !near;   // of the row, if it is
    const bool later = ((__ballot_sync(kAll, tied) >> (lane & 24) & 0xFFu) || !only_tied) && !bad;
    doubts |= later;
    const uint32_t last = __shfl_sync(kAll, my_key, (lane & 24) + k - 1);
    // as in the kernel above
    const bool whole_row = !only_tied && (near || (!kDirect && softmax) || (last && behind && close(last, behind)));
    if (bad) mine = -1;
    const bool got = mine >= 0;
    const float z = got ? as_float(row[mine]) : 0.0f;
    const float top = renorm ? share_max(got ? z : -INFINITY) : row_max;
    const float share = share_at(z, got, top, a.score, renorm, row_sum);
    const float sum = renorm ? share_sum(share) : 1.0f;
    if (t0 + r < a.T) {
      if (bad && sub == 0 && a.status) *a.status = kStatusNonFinite;
      if (later) {
        if (sub < k) a.ids[t * k + sub] = sub ? mine : whole_row ? kDoubtful : kMark - mine;
        if (sub == 0)
          a.weights[t * k] =
              __int_as_float(only_tied ? kTied : w ? (V - 1 - static_cast<int>(w & (V - 1))) * kShare + holder[warp][r][k] : -1);
      } else if (sub < k) {
        a.ids[t * k + sub] = mine;
        a.weights[t * k + sub] = got ? a.scale * (renorm ? __fdiv_rn(share, sum) : share) : 0.0f;
      }
    }
  }
  if (__any_sync(kAll, doubts)) {
    __syncwarp();
    for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kRowsOfWarp; t0 < a.T;
         t0 += static_cast<int64_t>(gridDim.x) * (kWarps * kRowsOfWarp)) {
      const int mark = sub == 0 && t0 + r < a.T ? a.ids[(t0 + r) * k] : 0;
      for (unsigned rows = __ballot_sync(kAll, mark <= kDoubtful); rows; rows &= rows - 1u) {
        const int from = __ffs(rows) - 1;
        finish<Z>(a, t0 + from / kShare, __shfl_sync(kAll, mark, from), values[warp], lane);
      }
    }
  }
}

template <typename Z, int V>
cudaError_t route_many_launch_v(const RouteArgs& a, cudaStream_t st) {
  const bool direct = !a.bias && a.groups == 1;
  constexpr int rows = kWarps * kRowsOfWarp;
  const unsigned grid =
      static_cast<unsigned>(std::min<int64_t>((a.T + rows - 1) / rows, static_cast<int64_t>(sm_count()) * kManyCtas<V>));
  note_launch();
  return direct ? launch_k(route_many_kernel<Z, V, true>, dim3(grid), dim3(kWarps * 32), 0, st, 1, a)
                : launch_k(route_many_kernel<Z, V, false>, dim3(grid), dim3(kWarps * 32), 0, st, 1, a);
}

// From here on four rows share a warp.  One row a warp / four rows a warp, us,
// without and with bias and groups: 64 experts, 2048 tokens 3.3 / 3.1 and
// 4.7 / 4.5, 32768 tokens 24 / 8.5 and 37 / 16; 256 experts, 512 tokens 3.1 / 4.0
// and 4.5 / 8.0, 2048 3.7 / 3.9 and 7.8 / 8.2, 4096 5.1 / 4.7 and 13.7 / 11.3, 32768
// 27 / 18 and 52 / 36; 512 experts, 32768 tokens 46 / 36 and 77 / 95 (not built).
// One bound for all sizes, which gives away up to 0.4 us at 256 experts.  Up to 32
// experts a row is one value per lane: 32768 tokens of 8, 16 and 32 experts take
// 13.4, 13.4 and 16.4 us (eight lanes a row: not built); more than 8 choices or
// groups stay on the first kernel as well.
constexpr int64_t kManyRows = 2048;

template <typename Z, int V>
cudaError_t route_launch_v(const RouteArgs& a, cudaStream_t st) {
  const bool direct = !a.bias && a.groups == 1;
  const size_t smem = static_cast<size_t>(kWarps) * std::max<int64_t>(a.E, 16) * sizeof(double);
  const int64_t want = (a.T + kWarps - 1) / kWarps;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(want, static_cast<int64_t>(sm_count()) * kRouteCtas<V>));
  note_launch();
  return direct ? launch_k(route_kernel<Z, V, true>, dim3(grid), dim3(kWarps * 32), smem, st, 1, a)
                : launch_k(route_kernel<Z, V, false>, dim3(grid), dim3(kWarps * 32), smem, st, 1, a);
}

template <typename Z>
cudaError_t route_launch_z(const RouteArgs& a, cudaStream_t st) {
  if (a.T >= kManyRows && a.k <= kShare && a.groups <= kShare && a.E > 32 && a.E <= 256)
    return a.E <= 64    ? route_many_launch_v<Z, 8>(a, st)
           : a.E <= 128 ? route_many_launch_v<Z, 16>(a, st)
                        : route_many_launch_v<Z, 32>(a, st);
  return a.E <= 32    ? route_launch_v<Z, 1>(a, st)
         : a.E <= 64  ? route_launch_v<Z, 2>(a, st)
         : a.E <= 128 ? route_launch_v<Z, 4>(a, st)
         : a.E <= 256 ? route_launch_v<Z, 8>(a, st)
         : a.E <= 512 ? route_launch_v<Z, 16>(a, st)
                      : route_launch_v<Z, 32>(a, st);
}

// ---------------------------------------------------------------------------
// Gradient.  Softmax scores without renormalisation reach every expert: one
// warp per row writes s_e (0 - sum s g) for all and then the choices' s_i (g_i -
// sum s g) on top.  Otherwise a row is zeros but for its choices: a CTA
// computes the choices of its rows, `span` lanes each, fills all of them with
// zeros in 16-byte pieces and puts the choices' values on top.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Sum of `v` over the choices j < k of the `span` lanes of a row that name
// lane's own expert; *first: whether none before it does.
__device__ __forceinline__ float sum_of_same(int id, float v, int k, int span, bool* first) {
  float sum = 0.0f;
  const int sub = threadIdx.x & (span - 1), from = threadIdx.x & 31 & ~(span - 1);
  *first = id >= 0;
  for (int j = 0; j < k; ++j) {
    const int other = __shfl_sync(kAll, id, from + j);
    const float part = __shfl_sync(kAll, v, from + j);
    if (other == id) {
      sum += part;
      *first &= j >= sub;
    }
  }
  return sum;
}

template <typename Z, int V>
__global__ void __launch_bounds__(kWarps * 32)
    route_backward_kernel(const __grid_constant__ RouteArgs a, const float* __restrict__ dweights, Z* dlogits, int64_t ldd) {
  pdl_entry();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = static_cast<int>(a.E), k = static_cast<int>(a.k);
  const Z* const logits = static_cast<const Z*>(a.logits);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * kWarps) {
    const Z* const row = logits + t * a.ldl;
    int id = lane < k ? __ldg(a.ids + t * k + lane) : -1;
    if (id < -1 || id >= E) {
      if (a.status) *a.status = kStatusArg;
      id = -1;
    }
    const bool got = id >= 0, live = __any_sync(kAll, got);
    float z[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 32 + lane;
      z[i] = i < V / 2 || e < E ? as_float(row[e]) : -INFINITY;   // E > 16 V
    }
    const float mine = got ? as_float(row[id]) : 0.0f, g = got ? a.scale * __ldg(dweights + t * k + lane) : 0.0f;
    float row_max = -INFINITY, row_sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) row_max = fmaxf(row_max, z[i]);
    row_max = warp_max(row_max);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      z[i] = ex2((z[i] - row_max) * kLog2e);
      row_sum += z[i];
    }
    row_sum = warp_sum(row_sum);
    const float p = share_at(mine, got, row_max, NVFP4_ROUTE_SOFTMAX, false, row_sum);
    const float dot = warp_sum(got ? p * g : 0.0f);
    bool first;
    const float sum = sum_of_same(id, g, k, 32, &first);
    const float all = live ? -__fdiv_rn(dot, row_sum) : 0.0f;
    Z* const out = dlogits + t * ldd;
    __syncwarp();   // dlogits may be the logits
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 32 + lane;
      if (i < V / 2 || e < E) put(out + e, live ? z[i] * all : 0.0f);   // a row without a choice may hold anything
    }
    __syncwarp();
    if (first) put(out + id, p * (sum - dot));
  }
}

template <typename Z, int V>
cudaError_t route_backward_launch_v(const RouteArgs& a, const float* dweights, void* dlogits, int64_t ldd, cudaStream_t st) {
  const int64_t want = (a.T + kWarps - 1) / kWarps;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(want, static_cast<int64_t>(sm_count()) * 12));
  return launch_k(route_backward_kernel<Z, V>, dim3(grid), dim3(kWarps * 32), 0, st, 1, a, dweights, static_cast<Z*>(dlogits), ldd);
}

constexpr int kFillThreads = 256;

template <typename Z>
__global__ void __launch_bounds__(kFillThreads) route_backward_sparse_kernel(const __grid_constant__ RouteArgs a,
                                                                             const float* __restrict__ dweights, Z* dlogits,
                                                                             int64_t ldd, int span) {
  pdl_entry();
  const int tid = threadIdx.x, sub = tid % span, rows = kFillThreads / span;
  const int E = static_cast<int>(a.E), k = static_cast<int>(a.k);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * rows, t = t0 + tid / span;
  const int64_t left = a.T - t0 < rows ? a.T - t0 : rows;
  const bool softmax = a.score == NVFP4_ROUTE_SOFTMAX, renorm = a.flags & NVFP4_ROUTE_RENORM;
  int id = t < a.T && sub < k ? __ldg(a.ids + t * k + sub) : -1;
  if (id < -1 || id >= E) {
    if (a.status) *a.status = kStatusArg;
    id = -1;
  }
  const bool got = id >= 0;
  const float z = got ? as_float(static_cast<const Z*>(a.logits)[t * a.ldl + id]) : 0.0f;
  float g = got ? a.scale * __ldg(dweights + t * k + sub) : 0.0f;
  float top = got ? z : -INFINITY;
  for (int o = span >> 1; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
  float p = share_at(z, got, top, a.score, renorm, 1.0f);
  if (renorm) {
    float sum = p;
    for (int o = span >> 1; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    p = got ? __fdiv_rn(p, sum) : 0.0f;
    float dot = got ? p * g : 0.0f;
    for (int o = span >> 1; o; o >>= 1) dot += __shfl_xor_sync(kAll, dot, o);
    g -= dot;
  }
  // 1 - sigmoid(z)
  if (!softmax) p *= z > 0.0f ? __fdiv_rn(expf(-z), 1.0f + expf(-z)) : __fdiv_rn(1.0f, 1.0f + expf(z));
  const float mine = got ? p * g : 0.0f;
  // an expert that is named more than once: the first one puts the sum
  bool first;
  const float sum = sum_of_same(id, mine, k, span, &first);
  __syncthreads();   // dlogits may be the logits
  if (ldd == E && (reinterpret_cast<uintptr_t>(dlogits) & 15) == 0) {
    // rows * E values are whole 16-byte pieces: rows is a multiple of 8
    const int64_t values = left * E, pieces = values / (16 / sizeof(Z));
    Z* const base = dlogits + t0 * E;
    for (int64_t i = tid; i < pieces; i += kFillThreads) reinterpret_cast<uint4*>(base)[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int64_t i = pieces * (16 / sizeof(Z)) + tid; i < values; i += kFillThreads) put(base + i, 0.0f);
  } else {
    for (int64_t r = tid >> 5; r < left; r += kFillThreads / 32)
      for (int e = tid & 31; e < E; e += 32) put(dlogits + (t0 + r) * ldd + e, 0.0f);
  }
  __syncthreads();
  if (first) put(dlogits + t * ldd + id, sum);
}

template <typename Z>
cudaError_t route_backward_launch_z(const RouteArgs& a, const float* dweights, void* dlogits, int64_t ldd, cudaStream_t st) {
  note_launch();
  if (a.score != NVFP4_ROUTE_SOFTMAX || a.flags & NVFP4_ROUTE_RENORM) {
    int span = 1;
    while (span < a.k) span <<= 1;
    const int rows = kFillThreads / span;
    return launch_k(route_backward_sparse_kernel<Z>, dim3(static_cast<unsigned>((a.T + rows - 1) / rows)), dim3(kFillThreads), 0,
                    st, 1, a, dweights, static_cast<Z*>(dlogits), ldd, span);
  }
  return a.E <= 32    ? route_backward_launch_v<Z, 1>(a, dweights, dlogits, ldd, st)
         : a.E <= 64  ? route_backward_launch_v<Z, 2>(a, dweights, dlogits, ldd, st)
         : a.E <= 128 ? route_backward_launch_v<Z, 4>(a, dweights, dlogits, ldd, st)
         : a.E <= 256 ? route_backward_launch_v<Z, 8>(a, dweights, dlogits, ldd, st)
         : a.E <= 512 ? route_backward_launch_v<Z, 16>(a, dweights, dlogits, ldd, st)
                      : route_backward_launch_v<Z, 32>(a, dweights, dlogits, ldd, st);
}

}  // namespace

cudaError_t route_launch(const RouteArgs& a, cudaStream_t st) {
  return a.fp32 ? route_launch_z<float>(a, st) : route_launch_z<__nv_bfloat16>(a, st);
}

cudaError_t route_backward_launch(const RouteArgs& a, const float* dweights, void* dlogits, int64_t ldd, cudaStream_t st) {
  return a.fp32 ? route_backward_launch_z<float>(a, dweights, dlogits, ldd, st)
                : route_backward_launch_z<__nv_bfloat16>(a, dweights, dlogits, ldd, st);
}

}  // namespace nvfp4
