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
// One warp per token; expert e is value e / 32 of lane e % 32, so that a row
// is read in whole lines whatever its alignment, and equal values come in the
// order (value, lane) = the experts' order.
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

// A group's value from its two largest (-inf: there is none).
template <typename F>
__device__ __forceinline__ F group_value(F first, F second, bool pair) {
  return pair && second > -FLT_MAX ? first + second : first;
}

// The choice in 64 bits, for rows whose values in 32 bits are too near to one
// another to be ordered: lane j < k gets the j-th expert, or -1.
template <typename Z>
__device__ __noinline__ int choose_exactly(const Z* __restrict__ z, const RouteArgs& a, double* c, int lane) {
  const float low = lowest<Z>();
  const int E = static_cast<int>(a.E), k = static_cast<int>(a.k), G = static_cast<int>(a.groups), n = E / G;
  const double none = -INFINITY;
  const bool direct = !a.bias && G == 1;
  float m = -INFINITY;
  double sum = 0.0;
  if (!direct && a.score == NVFP4_ROUTE_SOFTMAX) {
    for (int e = lane; e < E; e += 32) m = fmaxf(m, as_float(z[e]));
    m = warp_max(m);
    for (int e = lane; e < E; e += 32) sum += exp(static_cast<double>(as_float(z[e])) - m);
    sum = warp_sum(sum);
  }
#pragma unroll 4
  for (int e = lane; e < E; e += 32) {
    const float v = as_float(z[e]);
    double s = v;
    if (!direct) s = a.score == NVFP4_ROUTE_SOFTMAX ? exp(s - m) / sum : 1.0 / (1.0 + exp(-s));
    bool open = v > low;
    if (a.bias) {
      const float b = __ldg(a.bias + e);
      s += b;
      open &= b > -FLT_MAX;
    }
    c[e] = open ? s : none;
  }
  __syncwarp();
  if (G > 1) {
    int lanes = 32;   // of a group
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
    const unsigned kept = __ballot_sync(kAll, g < G && better < a.kept);
    for (int e = lane; e < E; e += 32)
      if (!(kept >> (e / n * lanes) & 1u)) c[e] = none;
    __syncwarp();
  }
  int mine = -1;
  for (int j = 0; j < k; ++j) {
    double best = none;
    int at = E;
    for (int e = lane; e < E; e += 32)
      if (c[e] > best) {
        best = c[e];
        at = e;
      }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const double v = __shfl_xor_sync(kAll, best, o);
      const int i = __shfl_xor_sync(kAll, at, o);
      if (v > best || (v == best && i < at)) {
        best = v;
        at = i;
      }
    }
    if (at == E) break;   // the same in every lane
    if (lane == j) mine = at;
    if (lane == (at & 31)) c[at] = none;
    __syncwarp();
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
// and the next one, or with such groups, are chosen again in 64 bits.
template <int V>
constexpr int kRouteCtas = V <= 8 ? 8 : V == 16 ? 5 : 3;   // per SM

template <typename Z, int V, bool kDirect>
__global__ void __launch_bounds__(kWarps * 32, kRouteCtas<V>) route_kernel(const __grid_constant__ RouteArgs a) {
  extern __shared__ double route_smem[];
  pdl_entry();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = static_cast<int>(a.E), k = static_cast<int>(a.k), G = static_cast<int>(a.groups), n = E / G;
  double* const c64 = route_smem + static_cast<size_t>(warp) * E;
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
    // |32-bit c - c| <= delta: see the figures behind the kernel
    float delta = 0.0f, most_c = 0.0f;   // most_c >= |c|
    if (!kDirect) {
      const float share = softmax ? rcp(fmaxf(row_sum, FLT_MIN)) : 1.0f;
      most_c = share + bmax;
      delta = (softmax ? 0x1p-18f * share : 0x1p-20f) + 0x1p-23f * static_cast<float>(V) * most_c + FLT_MIN;
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
    for (int j = 0; j <= k; ++j) {
      w = __reduce_max_sync(kAll, top);
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
    bool unsure = false;
    if (had && next_key &&
        (kDirect ? (my_key ^ next_key) < static_cast<uint32_t>(V) : !(from_ordered(my_key) - from_ordered(next_key) > 2.0f * delta))) {
      const int next = (V - 1 - static_cast<int>(next_key & (V - 1))) * 32 + next_src;
      unsure = !(as_float(row[mine]) == as_float(row[next]) && (kDirect || !a.bias || __ldg(a.bias + mine) == __ldg(a.bias + next)));
    }
    if (near || __any_sync(kAll, unsure)) {
      __syncwarp();
      mine = choose_exactly<Z>(row, a, c64, lane);
      __syncwarp();
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
}
// delta.  ex2.approx and rcp.approx are off by 2^-22 and 2^-23 relative; the
// exponent's rounding makes that |z| 2^-23.5 more.  sigmoid: s (1 - s) |z| <=
// 0.23, in all below 2^-21.  softmax with d = z - max: exp(-d) d <= 0.37 of
// the largest share, and the row's sum is off by (mean d + 1) 2^-22 <=
// (ln 1024 + 1) 2^-22 relative: below 2^-19 of the largest share.  The keys
// drop log2 V bits of c: 2^-23 V |c|, and c's own rounding is in the slack.

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
constexpr int kManyCtas = V <= 16 ? 7 : V == 32 ? 5 : 4;   // per SM

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

template <typename Z, int V, bool kDirect>
__global__ void __launch_bounds__(kWarps * 32, kManyCtas<V>) route_many_kernel(const __grid_constant__ RouteArgs a) {
  constexpr int kPitch = V * kShare + V / 4;   // of a row's values in shared memory: one free after each 32
  static_assert(V % 4 == 0);
  // a warp's values in 32 bits (four rows) or in 64 (one row at a time)
  constexpr int kValues = kDirect ? V * kShare : kRowsOfWarp * (kPitch + 8) / 2;
  __shared__ double values[kWarps][kValues < kRowsOfWarp * 32 ? kRowsOfWarp * 32 : kValues];
  __shared__ int16_t doubtful[kWarps][kRowsOfWarp][32];   // experts that may be among the choices
  __shared__ int doubts[kWarps][kRowsOfWarp];
  __shared__ int16_t order[kWarps][kRowsOfWarp][kShare];
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
  float* const c32 = reinterpret_cast<float*>(values[warp]) + (kDirect ? 0 : r * (kPitch + 8));   // rows 8 banks apart

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
    float delta = 0.0f, most_c = 0.0f;
    if (!kDirect) {
      const float share = softmax ? rcp(fmaxf(row_sum, FLT_MIN)) : 1.0f;
      most_c = share + bmax;
      delta = (softmax ? 0x1p-18f * share : 0x1p-20f) + 0x1p-23f * static_cast<float>(V) * most_c + FLT_MIN;
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
      for (int i = 0; i < V; ++i) c32[i * kShare + sub + i / 4] = c[i];
      __syncwarp();
      float a1 = -INFINITY, a2 = -INFINITY;
      if (sub < G) {
        const int first = sub * n;
        for (int i = first; i < first + n; ++i) {
          const float v = c32[i + (i >> 5)];
          a2 = fmaxf(a2, fminf(a1, v));
          a1 = fmaxf(a1, v);
        }
      }
      __syncwarp();
      const float mine = group_value(a1, a2, a.flags & NVFP4_ROUTE_GROUP_PAIR);   // -inf from lanes without a group
      int better = 0;
#pragma unroll
      for (int o = 1; o < kShare; ++o) {
        const float v = __shfl_xor_sync(kAll, mine, o);
        better += v > mine || (v == mine && (sub ^ o) < sub);
      }
      const bool keep = better < a.kept;
      kept = __ballot_sync(kAll, keep) >> (lane & 24) & 0xFFu;
      const float least = -share_max(keep ? -mine : -INFINITY), most = share_max(keep ? -INFINITY : mine);
      near = most >= -FLT_MAX && !(least - most > 4.0f * delta + 0x1p-21f * most_c);
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
    uint32_t my_key = 0u, w = 0u;
    for (int j = 0; j <= k; ++j) {
      w = l0;
#pragma unroll
      for (int o = kShare / 2; o; o >>= 1) w = max(w, __shfl_xor_sync(kAll, w, o));
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
    bool unsure = false;
    if (had && next_key &&
        (kDirect ? (my_key ^ next_key) < static_cast<uint32_t>(V) : !(from_ordered(my_key) - from_ordered(next_key) > 2.0f * delta))) {
      const int next = (V - 1 - static_cast<int>(next_key & (V - 1))) * kShare + holder[warp][r][sub + 1];
      unsure = !(as_float(row[mine]) == as_float(row[next]) && (kDirect || !a.bias || __ldg(a.bias + mine) == __ldg(a.bias + next)));
    }
    unsure = (__ballot_sync(kAll, unsure) >> (lane & 24) & 0xFFu) && !near && !bad;   // of the row
    if (__any_sync(kAll, unsure)) {
      // every expert whose 32-bit value could belong to a choice, in 64 bits
      const uint32_t last = __reduce_min_sync(0xFFu << (lane & 24), had ? my_key : 0xFFFFFFFFu);
      const uint32_t least = (kDirect ? last : ordered(from_ordered(last) - 2.0f * delta)) & ~static_cast<uint32_t>(V - 1);
      if (sub == 0) doubts[warp][r] = 0;
      __syncwarp();
      if (unsure) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (key[i] && key[i] >= least) {
            const int at = atomicAdd(&doubts[warp][r], 1);
            if (at < 32) doubtful[warp][r][at] = static_cast<int16_t>(i * kShare + sub);
          }
      }
      __syncwarp();
      const int number = doubts[warp][r];
      if (unsure && number > 32) {   // as many equal ones: the whole row
        near = true;
        unsure = false;
      }
      double* const v64 = values[warp] + r * 32;
      double sum64 = 1.0;
      if (!kDirect && softmax) {
        sum64 = 0.0;
        if (unsure)
          for (int e = sub; e < E; e += kShare) sum64 += exp(static_cast<double>(as_float(row[e])) - row_max);
#pragma unroll
        for (int o = kShare / 2; o; o >>= 1) sum64 += __shfl_xor_sync(kAll, sum64, o);
      }
      if (unsure)
        for (int m = sub; m < number; m += kShare) {
          const int e = doubtful[warp][r][m];
          double v = as_float(row[e]);
          if (!kDirect) {
            v = softmax ? exp(v - row_max) / sum64 : 1.0 / (1.0 + exp(-v));
            if (a.bias) v += __ldg(a.bias + e);
          }
          v64[m] = v;
        }
      __syncwarp();
      if (unsure)
        for (int m = sub; m < number; m += kShare) {
          const int e = doubtful[warp][r][m];
          const double v = v64[m];
          int better = 0;
          for (int i = 0; i < number; ++i) better += v64[i] > v || (v64[i] == v && doubtful[warp][r][i] < e);
          if (better < k) order[warp][r][better] = static_cast<int16_t>(e);
        }
      __syncwarp();
      if (unsure && had) mine = order[warp][r][sub];
    }
    const unsigned again = __ballot_sync(kAll, near && !bad);   // its votes also part the uses of values
    for (unsigned rows = again; rows;) {
      const int of = (__ffs(rows) - 1) / kShare;
      rows &= ~(0xFFu << (of * kShare));
      const int64_t u = t0 + of < a.T ? t0 + of : a.T - 1;
      const int e = choose_exactly<Z>(logits + u * a.ldl, a, values[warp], lane);
      __syncwarp();
      const int moved = __shfl_sync(kAll, e, sub);   // lane j of the warp has choice j
      if (r == of) mine = sub < k ? moved : -1;
    }
    if (bad) mine = -1;
    const bool got = mine >= 0;
    const float z = got ? as_float(row[mine]) : 0.0f;
    const float top = renorm ? share_max(got ? z : -INFINITY) : row_max;
    const float share = share_at(z, got, top, a.score, renorm, row_sum);
    const float sum = renorm ? share_sum(share) : 1.0f;
    if (t0 + r < a.T) {
      if (bad && sub == 0 && a.status) *a.status = kStatusNonFinite;
      if (sub < k) {
        a.ids[t * k + sub] = mine;
        a.weights[t * k + sub] = got ? a.scale * (renorm ? __fdiv_rn(share, sum) : share) : 0.0f;
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

// From here on four rows share a warp.
constexpr int64_t kManyRows = 2048;

template <typename Z, int V>
cudaError_t route_launch_v(const RouteArgs& a, cudaStream_t st) {
  const bool direct = !a.bias && a.groups == 1;
  const size_t smem = static_cast<size_t>(kWarps) * a.E * sizeof(double);
  const int64_t want = (a.T + kWarps - 1) / kWarps;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(want, static_cast<int64_t>(sm_count()) * kRouteCtas<V>));
  note_launch();
  return direct ? launch_k(route_kernel<Z, V, true>, dim3(grid), dim3(kWarps * 32), smem, st, 1, a)
                : launch_k(route_kernel<Z, V, false>, dim3(grid), dim3(kWarps * 32), smem, st, 1, a);
}

template <typename Z>
cudaError_t route_launch_z(const RouteArgs& a, cudaStream_t st) {
  if (a.T >= kManyRows && a.k <= kShare && a.groups <= kShare && a.E > 32 && a.E <= 512)
    return a.E <= 64    ? route_many_launch_v<Z, 8>(a, st)
           : a.E <= 128 ? route_many_launch_v<Z, 16>(a, st)
           : a.E <= 256 ? route_many_launch_v<Z, 32>(a, st)
                        : route_many_launch_v<Z, 64>(a, st);
  return a.E <= 32    ? route_launch_v<Z, 1>(a, st)
         : a.E <= 64  ? route_launch_v<Z, 2>(a, st)
         : a.E <= 128 ? route_launch_v<Z, 4>(a, st)
         : a.E <= 256 ? route_launch_v<Z, 8>(a, st)
         : a.E <= 512 ? route_launch_v<Z, 16>(a, st)
                      : route_launch_v<Z, 32>(a, st);
}

// ---------------------------------------------------------------------------
// Gradient.  Softmax scores without renormalisation reach every expert: one
// warp per row, the chosen experts' parts put together in shared memory in the
// order of the choices (an expert that is named twice gets both).  Otherwise a
// row is zeros but for its choices: a CTA computes the choices of its rows,
// `span` lanes each, fills all of them with zeros in 16-byte pieces and then
// puts the choices' values on top.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename Z>
__global__ void __launch_bounds__(kWarps * 32) route_backward_kernel(const __grid_constant__ RouteArgs a, const float* __restrict__ dweights,
                                                                     Z* dlogits, int64_t ldd) {
  extern __shared__ float grad_smem[];
  pdl_entry();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = static_cast<int>(a.E), k = static_cast<int>(a.k);
  float* const d = grad_smem + static_cast<size_t>(warp) * E;
  const Z* const logits = static_cast<const Z*>(a.logits);

  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * kWarps) {
    const Z* const row = logits + t * a.ldl;
    int id = lane < k ? __ldg(a.ids + t * k + lane) : -1;
    const bool wrong = id < -1 || id >= E;
    if (wrong) {
      if (a.status) *a.status = kStatusArg;
      id = -1;
    }
    const bool got = id >= 0;
    const float z = got ? as_float(row[id]) : 0.0f;
    const float g = got ? a.scale * __ldg(dweights + t * k + lane) : 0.0f;
    float row_max = -INFINITY, row_sum = 0.0f;
    const bool live = __any_sync(kAll, got);
    if (live) {
      for (int e = lane; e < E; e += 32) row_max = fmaxf(row_max, as_float(row[e]));
      row_max = warp_max(row_max);
      for (int e = lane; e < E; e += 32) row_sum += ex2((as_float(row[e]) - row_max) * kLog2e);
      row_sum = warp_sum(row_sum);
    }
    const float p = share_at(z, got, row_max, NVFP4_ROUTE_SOFTMAX, false, row_sum);
    const float dot = warp_sum(got ? p * g : 0.0f);
    for (int e = lane; e < E; e += 32) d[e] = 0.0f;
    __syncwarp();
    for (int j = 0; j < k; ++j) {
      const int e = __shfl_sync(kAll, id, j);
      const float v = __shfl_sync(kAll, g, j);
      if (e >= 0 && lane == (e & 31)) d[e] += v;
    }
    __syncwarp();
    Z* const out = dlogits + t * ldd;
    for (int e = lane; e < E; e += 32) {
      put(out + e, live ? __fdiv_rn(ex2((as_float(row[e]) - row_max) * kLog2e), row_sum) * (d[e] - dot) : 0.0f);
    }
    __syncwarp();
  }
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
  float sum = 0.0f;
  bool first = got;
  for (int j = 0; j < k; ++j) {
    const int from = (tid & 31 & ~(span - 1)) + j;
    const int other = __shfl_sync(kAll, id, from);
    const float v = __shfl_sync(kAll, mine, from);
    if (other == id) {
      sum += v;
      first &= j >= sub;
    }
  }
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
  const int64_t want = (a.T + kWarps - 1) / kWarps;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(want, static_cast<int64_t>(sm_count()) * 16));
  return launch_k(route_backward_kernel<Z>, dim3(grid), dim3(kWarps * 32), static_cast<size_t>(kWarps) * a.E * sizeof(float),
                  st, 1, a, dweights, static_cast<Z*>(dlogits), ldd);
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
