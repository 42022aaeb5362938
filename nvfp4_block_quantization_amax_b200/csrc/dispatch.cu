// dispatch.cu -- token rows to their experts and back.
//
//   sort:      offsets[e] = number of pairs (token, choice) with an expert
//              below e; rows[t, j] = offsets[e] + number of earlier pairs of
//              e = ids[t, j]                                  (-1: no expert)
//   dispatch:  xs[rows[t, j]] = x[t]
//   combine:   out[t] = res[t] + sum_j w[t, j] y[rows[t, j]]
//   backward:  dy[rows[t, j]] = w[t, j] dout[t],
//              dw[t, j] = <dout[t], y[rows[t, j]]>
//
// The row kernels are bound by memory: every row passes once, in 16-byte
// pieces, one thread per piece and token, so that a token's row is read once
// for its k copies (dispatch, backward) and its k rows are on their way at the
// same time (combine).  A token takes the power of two of threads from C / 8
// on, at most a CTA.  Sums are fp32, in the order of the choices.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>

#include "launch.cuh"
#include "nvfp4_internal.h"

namespace cg = cooperative_groups;

namespace nvfp4 {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;

// ---------------------------------------------------------------------------
// sort: one cluster; each warp takes a run of consecutive pairs
// ---------------------------------------------------------------------------
constexpr int kSortCtas = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;

// The expert of pair p, -1 for none and behind the last pair; an id outside
// -1 .. E - 1 counts as -1 and sets the status.
__device__ __forceinline__ int expert_of(const int32_t* __restrict__ ids, int64_t p, int64_t P, int E, int32_t* status) {
  if (p >= P) return -1;
  const int id = __ldg(ids + p);
  if (id >= 0 && id < E) return id;
  if (id != -1 && status) *status = kStatusArg;
  return -1;
}

__global__ void __launch_bounds__(kSortThreads) sort_kernel(const int32_t* __restrict__ ids, int64_t P, int E,
                                                            int32_t* __restrict__ offsets, int32_t* __restrict__ rows,
                                                            int32_t* status) {
  extern __shared__ int sort_smem[];
  pdl_entry();
  int* const hist = sort_smem;                      // [warps][E]: counts, then where the warp's next pair goes
  int* const total = sort_smem + kSortWarps * E;    // [E]: this CTA's counts, read by the cluster
  __shared__ int warp_sum[kSortWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, rank = static_cast<int>(cluster.block_rank());
  const int64_t warps = kSortCtas * kSortWarps;
  const int64_t run = ((P + warps - 1) / warps + 31) / 32 * 32;
  const int64_t from = (rank * kSortWarps + w) * run, to = from + run < P ? from + run : P;
  int* const mine = hist + w * E;
  for (int e = lane; e < E; e += 32) mine[e] = 0;
  __syncwarp();
  for (int64_t p = from; p < to; p += 32) {
    const int e = expert_of(ids, p + lane, P, E, status);
    const unsigned same = __match_any_sync(kAll, e);
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  if (tid < E) {
    int sum = 0;
    for (int i = 0; i < kSortWarps; ++i) {
      const int v = hist[i * E + tid];
      hist[i * E + tid] = sum;
      sum += v;
    }
    total[tid] = sum;
  }
  cluster.sync();
  int all = 0, before = 0;
  if (tid < E)
    for (int r = 0; r < kSortCtas; ++r) {
      const int v = cluster.map_shared_rank(total, r)[tid];
      before += r < rank ? v : 0;
      all += v;
    }
  int incl = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kAll, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[w] = incl;
  __syncthreads();
  int base = incl - all;
  for (int i = 0; i < w; ++i) base += warp_sum[i];
  if (tid < E) {
    if (rank == 0) {
      offsets[tid] = base;
      if (tid == E - 1) offsets[E] = base + all;
    }
    for (int i = 0; i < kSortWarps; ++i) hist[i * E + tid] += base + before;
  }
  cluster.sync();   // the others have read total; hist is complete
  for (int64_t p = from; p < to; p += 32) {
    const int e = expert_of(ids, p + lane, P, E, nullptr);
    const unsigned same = __match_any_sync(kAll, e);
    const int at = e >= 0 ? mine[e] + __popc(same & ((1u << lane) - 1u)) : -1;
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
    if (p + lane < P) rows[p + lane] = at;
  }
}

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256;

// Place of pair p among R rows; -1 where it has none, and for a place outside
// -1 .. R - 1, which sets the status.  Without a list it is p itself.
__device__ __forceinline__ int64_t place_of(const RowArgs& a, int64_t p) {
  if (!a.rows) return p;
  const int r = __ldg(a.rows + p);
  if (r >= 0 && r < a.R) return r;
  if (r != -1 && a.status) *a.status = kStatusArg;
  return -1;
}

__device__ __forceinline__ float2 widen(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t narrow(float x, float y) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint4 load16(const __nv_bfloat16* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ void store16(__nv_bfloat16* p, uint4 v) { *reinterpret_cast<uint4*>(p) = v; }

// s += w v of eight values
__device__ __forceinline__ void add_scaled(float* s, float w, uint4 v) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = widen(u[i]);
    s[2 * i] = __fmaf_rn(w, f.x, s[2 * i]);
    s[2 * i + 1] = __fmaf_rn(w, f.y, s[2 * i + 1]);
  }
}
__device__ __forceinline__ uint4 narrow8(const float* s) {
  return make_uint4(narrow(s[0], s[1]), narrow(s[2], s[3]), narrow(s[4], s[5]), narrow(s[6], s[7]));
}

__global__ void __launch_bounds__(kRowThreads) dispatch_kernel(const RowArgs a, int per_token) {
  pdl_entry();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRowThreads / per_token) + threadIdx.x / per_token;
  if (t >= a.T) return;
  const int k = static_cast<int>(a.k);
  for (int64_t c = (threadIdx.x % per_token) * 8; c < a.C; c += per_token * 8) {
    const uint4 v = load16(a.in + t * a.ldi + c);
    for (int j = 0; j < k; ++j) {
      const int64_t r = place_of(a, t * k + j);
      if (r >= 0) store16(a.out + r * a.ldo + c, v);
    }
  }
}

constexpr int kTogether = 8;   // rows of a token on their way at the same time

__global__ void __launch_bounds__(kRowThreads) combine_kernel(const RowArgs a, int per_token) {
  pdl_entry();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRowThreads / per_token) + threadIdx.x / per_token;
  if (t >= a.T) return;
  const int k = static_cast<int>(a.k);
  for (int64_t c = (threadIdx.x % per_token) * 8; c < a.C; c += per_token * 8) {
    float s[8] = {};
    if (a.in) add_scaled(s, 1.0f, *reinterpret_cast<const uint4*>(a.in + t * a.ldi + c));   // may be out
    for (int j0 = 0; j0 < k; j0 += kTogether) {
      uint4 v[kTogether];
      bool got[kTogether];
#pragma unroll
      for (int j = 0; j < kTogether; ++j) {
        const int64_t r = j0 + j < k ? place_of(a, t * k + j0 + j) : -1;
        got[j] = r >= 0;
        if (got[j]) v[j] = load16(a.y + r * a.ldy + c);
      }
#pragma unroll
      for (int j = 0; j < kTogether; ++j)
        if (got[j]) add_scaled(s, a.weights ? __ldg(a.weights + t * k + j0 + j) : 1.0f, v[j]);
    }
    store16(a.out + t * a.ldo + c, narrow8(s));
  }
}

// per_token threads of one token; the sums of dw go through shared memory when
// they are more than a warp's.
__global__ void __launch_bounds__(kRowThreads) combine_backward_kernel(const RowArgs a, int per_token) {
  __shared__ float part[kRowThreads / 32][kTogether];
  pdl_entry();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRowThreads / per_token) + threadIdx.x / per_token;
  const int k = static_cast<int>(a.k), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool live = t < a.T;
  for (int j0 = 0; j0 < k; j0 += kTogether) {
    float dot[kTogether] = {};
    if (live) {
      int64_t r[kTogether];
      float w[kTogether];
#pragma unroll
      for (int j = 0; j < kTogether; ++j) {
        r[j] = j0 + j < k ? place_of(a, t * k + j0 + j) : -1;
        w[j] = a.weights && r[j] >= 0 ? __ldg(a.weights + t * k + j0 + j) : 1.0f;
      }
      for (int64_t c = (threadIdx.x % per_token) * 8; c < a.C; c += per_token * 8) {
        float d[8] = {};
        add_scaled(d, 1.0f, load16(a.in + t * a.ldi + c));
        uint4 v[kTogether];
        if (a.dweights) {
#pragma unroll
          for (int j = 0; j < kTogether; ++j)
            if (r[j] >= 0) v[j] = load16(a.y + r[j] * a.ldy + c);
        }
#pragma unroll
        for (int j = 0; j < kTogether; ++j) {
          if (r[j] < 0) continue;
          if (a.dweights) {
            const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 f = widen(u[i]);
              dot[j] = __fmaf_rn(d[2 * i], f.x, dot[j]);
              dot[j] = __fmaf_rn(d[2 * i + 1], f.y, dot[j]);
            }
          }
          if (a.out) {
            float s[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = w[j] * d[i];
            store16(a.out + r[j] * a.ldo + c, narrow8(s));
          }
        }
      }
    }
    if (!a.dweights) continue;
    const int width = per_token < 32 ? per_token : 32;
#pragma unroll
    for (int j = 0; j < kTogether; ++j)
      for (int o = width >> 1; o; o >>= 1) dot[j] += __shfl_xor_sync(kAll, dot[j], o);
    const int own = threadIdx.x % per_token;
    if (per_token > 32) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kTogether; ++j)
        if (lane == 0) part[warp][j] = dot[j];
      __syncthreads();
      if (live && own < kTogether && j0 + own < k) {
        float s = 0.0f;
        for (int i = 0; i < per_token / 32; ++i) s += part[warp + i][own];
        a.dweights[t * k + j0 + own] = s;
      }
    } else if (live && own == 0) {
#pragma unroll
      for (int j = 0; j < kTogether; ++j)
        if (j0 + j < k) a.dweights[t * k + j0 + j] = dot[j];
    }
  }
}

int threads_per_token(int64_t C) {
  int n = 1;
  while (n < kRowThreads && n * 8 < C) n *= 2;
  return n;
}

template <typename Kernel>
cudaError_t rows_launch(Kernel kernel, const RowArgs& a, cudaStream_t st) {
  const int per_token = threads_per_token(a.C), tokens = kRowThreads / per_token;
  note_launch();
  return launch_k(kernel, dim3(static_cast<unsigned>((a.T + tokens - 1) / tokens)), dim3(kRowThreads), 0, st, 1, a, per_token);
}

}  // namespace

cudaError_t sort_launch(const int32_t* ids, int64_t P, int64_t E, int32_t* offsets, int32_t* rows, int32_t* status,
                        cudaStream_t st) {
  const size_t smem = static_cast<size_t>(kSortWarps + 1) * E * sizeof(int);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  note_launch();
  return launch_k(sort_kernel, dim3(kSortCtas), dim3(kSortThreads), smem, st, kSortCtas, ids, P, static_cast<int>(E), offsets,
                  rows, status);
}

cudaError_t dispatch_rows_launch(const RowArgs& a, cudaStream_t st) { return rows_launch(dispatch_kernel, a, st); }
cudaError_t combine_launch(const RowArgs& a, cudaStream_t st) { return rows_launch(combine_kernel, a, st); }
cudaError_t combine_backward_launch(const RowArgs& a, cudaStream_t st) { return rows_launch(combine_backward_kernel, a, st); }

}  // namespace nvfp4
