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
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
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
    double mine = none;   // lane g: the value of group g
    for (int g = 0; g < G; ++g) {
      double a1 = none, a2 = none;
      for (int i = lane; i < n; i += 32) merge_two(a1, a2, c[g * n + i], none);
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const double b1 = __shfl_xor_sync(kAll, a1, o), b2 = __shfl_xor_sync(kAll, a2, o);
        merge_two(a1, a2, b1, b2);
      }
      if (lane == g) mine = group_value(a1, a2, a.flags & NVFP4_ROUTE_GROUP_PAIR);
    }
    int better = 0;
    for (int g = 0; g < G; ++g) {
      const double v = __shfl_sync(kAll, mine, g);
      better += v > mine || (v == mine && g < lane);
    }
    const unsigned kept = __ballot_sync(kAll, lane < G && better < a.kept);
    for (int e = lane; e < E; e += 32)
      if (!(kept >> (e / n) & 1u)) c[e] = none;
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
__device__ __forceinline__ float share_of(float z, bool got, int score, bool renorm, float row_max, float row_sum) {
  const float top = renorm ? warp_max(got ? z : -INFINITY) : row_max;
  if (!got) return 0.0f;
  if (score == NVFP4_ROUTE_SOFTMAX) {
    const float e = expf(z - top);
    return renorm ? e : __fdiv_rn(e, row_sum);
  }
  if (z > 0.0f) return __fdiv_rn(1.0f, 1.0f + expf(-z));
  return __fdiv_rn(expf(renorm ? z - fminf(top, 0.0f) : z), 1.0f + expf(z));
}

// V: values per lane, the power of two from E / 32 on.  kDirect: no bias and
// no groups, so that the order is that of the logits themselves.
//
// The order is found on 32-bit keys: the value in its order, the low log2 V
// bits replaced by V - 1 - i for value i of the lane, so that a lane's keys
// differ and the largest one names its place.  A round takes the largest key
// of the warp; the lane that held it moves on to its largest key below.
// Values as near as the error of their 32-bit form (delta), or with the same
// key, may stand in the wrong order; rows with such a pair among the chosen
// and the next one, or with such groups, are chosen again in 64 bits.
template <typename Z, int V, bool kDirect>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const __grid_constant__ RouteArgs a) {
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

  float bias[V];
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
      z[i] = e < E ? as_float(row[e]) : -INFINITY;
      bad |= !(z[i] <= FLT_MAX);
    }
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
    // |32-bit c - c| <= delta: see the figures at the end of the kernel
    float delta = 0.0f, most_c = 0.0f;   // most_c >= |c|
    if (!kDirect) {
      const float share = softmax ? rcp(fmaxf(row_sum, FLT_MIN)) : 1.0f;
      most_c = share + bmax;
      delta = (softmax ? 0x1p-18f * share : 0x1p-20f) + 0x1p-23f * static_cast<float>(V) * most_c + FLT_MIN;
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = (softmax ? c[i] * share : rcp(1.0f + ex2(-kLog2e * z[i]))) + bias[i];
    }
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool open = z[i] > low && (kDirect || bias[i] > -FLT_MAX);
      key[i] = open ? (ordered(c[i]) & ~static_cast<uint32_t>(V - 1)) | static_cast<uint32_t>(V - 1 - i) : 0u;
    }
    bool near = false;   // uniform in the warp
    if (!kDirect && G > 1) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        if (e < E) c32[e + i] = key[i] ? c[i] : -INFINITY;
      }
      __syncwarp();
      int lanes = 32;   // of a group
      while (lanes * G > 32) lanes >>= 1;
      const int g = lane / lanes;
      float a1 = -INFINITY, a2 = -INFINITY;
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
      for (int i = 0; i < V; ++i)
        if (!(kept >> ((i * 32 + lane) / n * lanes & 31) & 1u)) key[i] = 0u;
    }
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) top = max(top, key[i]);
    uint32_t my_key = 0u, next_key = 0u;   // lane j: the j-th choice's and the one behind it
    int mine = -1, next = -1;
    uint32_t w = 0u;
    for (int j = 0; j <= k; ++j) {
      w = __reduce_max_sync(kAll, top);
      const int src = __ffs(__ballot_sync(kAll, top == w)) - 1;
      const int e = w ? (V - 1 - static_cast<int>(w & (V - 1))) * 32 + src : -1;
      if (lane == j) {
        my_key = w;
        mine = e;
      }
      if (lane == j - 1) {
        next_key = w;
        next = e;
      }
      if (lane == src) {
        // keys below w wrap to numbers above those that do not
        uint32_t most = 0u;
#pragma unroll
        for (int i = 0; i < V; ++i) most = max(most, key[i] - w);
        top = w + most < w ? w + most : 0u;
      }
      if (w == 0u) break;
    }
    if (lane >= k) mine = next = -1;
    // neighbours that may stand in the wrong order; equal inputs do not
    bool unsure = false;
    if (mine >= 0 && next >= 0) {
      const bool equal = as_float(row[mine]) == as_float(row[next]) &&
                         (kDirect || !a.bias || __ldg(a.bias + mine) == __ldg(a.bias + next));
      unsure = !equal && (kDirect ? (my_key ^ next_key) < static_cast<uint32_t>(V)
                                  : !(from_ordered(my_key) - from_ordered(next_key) > 2.0f * delta));
    }
    if (near || __any_sync(kAll, unsure)) {
      __syncwarp();
      mine = choose_exactly<Z>(row, a, c64, lane);
      __syncwarp();
    }
    const bool got = mine >= 0;
    const float share = share_of(got ? as_float(row[mine]) : 0.0f, got, a.score, renorm, row_max, row_sum);
    const float sum = renorm ? warp_sum(share) : 1.0f;
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

template <typename Z, int V>
cudaError_t route_launch_v(const RouteArgs& a, cudaStream_t st) {
  const bool direct = !a.bias && a.groups == 1;
  const size_t smem = static_cast<size_t>(kWarps) * a.E * sizeof(double);
  const int64_t want = (a.T + kWarps - 1) / kWarps;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(want, static_cast<int64_t>(sm_count()) * 16));
  note_launch();
  return direct ? launch_k(route_kernel<Z, V, true>, dim3(grid), dim3(kWarps * 32), smem, st, 1, a)
                : launch_k(route_kernel<Z, V, false>, dim3(grid), dim3(kWarps * 32), smem, st, 1, a);
}

template <typename Z>
cudaError_t route_launch_z(const RouteArgs& a, cudaStream_t st) {
  return a.E <= 32    ? route_launch_v<Z, 1>(a, st)
         : a.E <= 64  ? route_launch_v<Z, 2>(a, st)
         : a.E <= 128 ? route_launch_v<Z, 4>(a, st)
         : a.E <= 256 ? route_launch_v<Z, 8>(a, st)
         : a.E <= 512 ? route_launch_v<Z, 16>(a, st)
                      : route_launch_v<Z, 32>(a, st);
}

// ---------------------------------------------------------------------------
// Gradient.  The chosen experts' entries are put together in shared memory, in
// the order of the choices (an expert that is named twice gets both parts).
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
  const bool softmax = a.score == NVFP4_ROUTE_SOFTMAX, renorm = a.flags & NVFP4_ROUTE_RENORM;
  const bool whole = softmax && !renorm;

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
    float g = got ? a.scale * __ldg(dweights + t * k + lane) : 0.0f;
    float row_max = 0.0f, row_sum = 1.0f;
    const bool live = __any_sync(kAll, got);
    if (whole && live) {
      row_max = -INFINITY;
      for (int e = lane; e < E; e += 32) row_max = fmaxf(row_max, as_float(row[e]));
      row_max = warp_max(row_max);
      row_sum = 0.0f;
      for (int e = lane; e < E; e += 32) row_sum += ex2((as_float(row[e]) - row_max) * kLog2e);
      row_sum = warp_sum(row_sum);
    }
    float p = share_of(z, got, a.score, renorm, row_max, row_sum);
    if (renorm) p = live ? __fdiv_rn(p, warp_sum(p)) : 0.0f;
    const float dot = softmax || renorm ? warp_sum(got ? p * g : 0.0f) : 0.0f;
    // 1 - sigmoid(z)
    const float other = softmax ? 1.0f : z > 0.0f ? __fdiv_rn(expf(-z), 1.0f + expf(-z)) : __fdiv_rn(1.0f, 1.0f + expf(z));
    if (!whole) g = got ? other * p * (g - dot) : 0.0f;
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
      float v = d[e];
      if (whole) v = live ? __fdiv_rn(ex2((as_float(row[e]) - row_max) * kLog2e), row_sum) * (v - dot) : 0.0f;
      put(out + e, v);
    }
    __syncwarp();
  }
}

template <typename Z>
cudaError_t route_backward_launch_z(const RouteArgs& a, const float* dweights, void* dlogits, int64_t ldd, cudaStream_t st) {
  const int64_t want = (a.T + kWarps - 1) / kWarps;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(want, static_cast<int64_t>(sm_count()) * 16));
  note_launch();
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
