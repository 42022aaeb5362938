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
//
// 16384 tokens, 8 choices, C = 4096, and what memory alone takes at the measured
// rate, us: copying 198 (185: 5.98 TB/s, 1.07 GB of it written), the sort in
// front of it 16; combine, 6 choices, 16301 tokens 158 (143: 5.6 to 5.9 TB/s);
// backward 403 (349: 5.96 TB/s, half read, half written).  64 tokens: 3.8 and 5.1,
// a launch and two or three dependent loads.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <atomic>
#include <cstdint>

#include "launch.cuh"
#include "nvfp4_internal.h"
#include "smem.cuh"

namespace cg = cooperative_groups;

namespace nvfp4 {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;

// ---------------------------------------------------------------------------
// sort: one cluster; each warp takes a run of consecutive pairs, and counts
// them while it notes each one's rank among its run's.  One cluster needs no
// memory of its own and one launch; it is bound by its instructions on eight SMs
// (126 per 32 pairs; 131072 pairs of 64 experts 16 us, of 1024 22, 524288 pairs
// 59).  With match.any for the ballots, and again in the second pass: 34 and 142.
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

// Lanes with the same e, found bit by bit (match.any takes several times as long).
template <int kBits>
__device__ __forceinline__ unsigned same_as(int e) {
  unsigned same = kAll;
#pragma unroll
  for (int b = 0; b < kBits; ++b) {
    const bool one = e >> b & 1;
    const unsigned v = __ballot_sync(kAll, one);
    same &= one ? v : ~v;
  }
  return same;
}

template <int kBits>   // of E - 1
__global__ void __launch_bounds__(kSortThreads) sort_kernel(const int32_t* __restrict__ ids, int64_t P, int E,
                                                            int32_t* __restrict__ offsets, int32_t* rows, int32_t* status) {
  extern __shared__ int sort_smem[];
  pdl_entry();
  int* const hist = sort_smem;                      // [warps][E]: counts, then those of the warps before
  int* const total = sort_smem + kSortWarps * E;    // [E]: this CTA's counts, read by the cluster
  int* const start = total + E;                     // [E]: where this CTA's pairs of an expert go
  __shared__ int warp_sum[kSortWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, rank = static_cast<int>(cluster.block_rank());
  const int64_t warps = kSortCtas * kSortWarps;
  const int64_t run = ((P + warps - 1) / warps + 31) / 32 * 32;
  const int64_t from = (rank * kSortWarps + w) * run, to = from + run < P ? from + run : P;
  int* const mine = hist + w * E;
  for (int e = lane; e < E; e += 32) mine[e] = 0;
  __syncwarp();
  constexpr int kAhead = 4;
  for (int64_t p0 = from; p0 < to; p0 += 32 * kAhead) {
    int id[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t p = p0 + i * 32 + lane;
      id[i] = expert_of(ids, p, to, E, status);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t p = p0 + i * 32 + lane;
      const int e = id[i];
      const unsigned same = same_as<kBits>(e) & __ballot_sync(kAll, e >= 0);
      const unsigned before = same & ((1u << lane) - 1u);
      const int at = e >= 0 ? mine[e] + __popc(before) : -1;
      __syncwarp();
      if (e >= 0 && !before) mine[e] += __popc(same);
      __syncwarp();
      if (p < to) rows[p] = at;
    }
  }
  __syncthreads();
  if (tid < E) {
    int sum = 0;
#pragma unroll 8
    for (int i = 0; i < kSortWarps; ++i) {
      const int v = hist[i * E + tid];
      hist[i * E + tid] = sum;
      sum += v;
    }
    total[tid] = sum;
  }
  cluster.sync();
  int all = 0, before = 0;
  if (tid < E) {
#pragma unroll
    for (int r = 0; r < kSortCtas; ++r) {
      const int v = cluster.map_shared_rank(total, r)[tid];
      before += r < rank ? v : 0;
      all += v;
    }
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
    start[tid] = base + before;
  }
  cluster.sync();   // the others have read total; start is complete
  for (int64_t p0 = from; p0 < to; p0 += 32 * kAhead) {
    int id[kAhead], at[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t p = p0 + i * 32 + lane;
      at[i] = p < to ? rows[p] : -1;
      id[i] = at[i] >= 0 ? __ldg(ids + p) : 0;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (at[i] >= 0) rows[p0 + i * 32 + lane] = at[i] + mine[id[i]] + start[id[i]];
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
__device__ __forceinline__ uint4 load16_once(const __nv_bfloat16* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }
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

// Few pairs: every CTA counts for itself where its tokens' rows go (the pairs
// with a lower expert and the earlier ones with the same), one warp per pair,
// and copies them; the experts' offsets are shared out over all warps.  What it
// costs is the rounds that a CTA makes (a token at a time, eight choices at a
// time) over all pairs, against the sort and the copy.  C = 4096, 64 experts,
// us for rounds x pairs:
//   1 choice    1024 tokens  4 x 1024   6.0 /  8.8   1536  6 x 1536   9.2 /  9.4
//               2048         7 x 2048  11.3 / 10.0   4096 14 x 4096  28.0 / 13.4
//   2 choices   1024         4 x 2048   9.2 /  9.8   1500  6 x 3000  15.9 / 11.0
//   4 choices    512         2 x 2048   6.7 /  9.8    750  3 x 3000  11.3 / 11.1
//   6 choices    500         2 x 3000   9.5 / 10.7    682  3 x 4092  14.5 / 11.9
//   8 choices    256         1 x 2048   5.6 /  9.2    512  2 x 4096  11.3 / 12.4
//  16 choices    256         2 x 4096  11.6 / 11.8
//  32 choices     64         4 x 2048  10.4 / 12.0    128  4 x 4096  15.1 / 12.3
constexpr int kFewPairs = 4096;                      // shared memory
constexpr int64_t kFewWork = 9 * 1024;               // rounds x pairs
constexpr int kFewThreads = 256;

__global__ void __launch_bounds__(kFewThreads) dispatch_few_kernel(const RowArgs a, const int32_t* __restrict__ ids, int E,
                                                                   int32_t* __restrict__ offsets, int32_t* __restrict__ rows) {
  __shared__ int id[kFewPairs];
  __shared__ int place[kFewThreads];
  pdl_entry();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = static_cast<int>(a.k), P = static_cast<int>(a.T) * k;
  for (int p = tid; p < P; p += kFewThreads) {
    const int e = __ldg(ids + p);
    const bool is = e >= 0 && e < E;
    if (!is && e != -1 && a.status) *a.status = kStatusArg;
    id[p] = is ? e : E;   // behind all others
  }
  __syncthreads();
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    for (int j = warp; j < k; j += kFewThreads / 32) {
      const int p = t * k + j, e = id[p];
      int n = 0;
      for (int q = lane; q < P; q += 32) n += id[q] < e + (q < p);
      n = __reduce_add_sync(kAll, n);
      if (lane == 0) {
        n = e < E ? n : -1;
        place[j] = n;
        rows[p] = n;
      }
    }
    __syncthreads();
    if (a.in)
      for (int64_t c = tid * 8; c < a.C; c += kFewThreads * 8) {
        const uint4 v = load16(a.in + t * a.ldi + c);
        for (int j = 0; j < k; ++j)
          if (place[j] >= 0) store16(a.out + place[j] * a.ldo + c, v);
      }
    __syncthreads();
  }
  for (int e = blockIdx.x * (kFewThreads / 32) + warp; e <= E; e += gridDim.x * (kFewThreads / 32)) {
    int n = 0;
    for (int q = lane; q < P; q += 32) n += id[q] < e;
    n = __reduce_add_sync(kAll, n);
    if (lane == 0) offsets[e] = n;
  }
}

constexpr int kTogether = 8;   // rows of a token on their way at the same time
// The same in the backward pass, which holds the sums as well: 4 rows and four
// CTAs per SM 402 us for the sizes above, 8 and two 402, 8 and three (spills)
// 435, 4 and three 422, 2 and six 468; at C = 1024, 65536 tokens 389, 441, 450, 416, 414.
constexpr int kBack = 4;

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
        if (got[j]) v[j] = load16_once(a.y + r * a.ldy + c);
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
__global__ void __launch_bounds__(kRowThreads, 4) combine_backward_kernel(const RowArgs a, int per_token) {
  __shared__ float part[kRowThreads / 32][kBack];
  pdl_entry();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRowThreads / per_token) + threadIdx.x / per_token;
  const int k = static_cast<int>(a.k), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool live = t < a.T;
  for (int j0 = 0; j0 < k; j0 += kBack) {
    float dot[kBack] = {};
    if (live) {
      int64_t r[kBack];
      float w[kBack];
#pragma unroll
      for (int j = 0; j < kBack; ++j) {
        r[j] = j0 + j < k ? place_of(a, t * k + j0 + j) : -1;
        w[j] = a.weights && r[j] >= 0 ? __ldg(a.weights + t * k + j0 + j) : 1.0f;
      }
      for (int64_t c = (threadIdx.x % per_token) * 8; c < a.C; c += per_token * 8) {
        float d[8] = {};
        add_scaled(d, 1.0f, load16(a.in + t * a.ldi + c));
        uint4 v[kBack];
        if (a.dweights) {
#pragma unroll
          for (int j = 0; j < kBack; ++j)
            if (r[j] >= 0) v[j] = load16(a.y + r[j] * a.ldy + c);
        }
#pragma unroll
        for (int j = 0; j < kBack; ++j) {
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
    for (int j = 0; j < kBack; ++j)
      for (int o = width >> 1; o; o >>= 1) dot[j] += __shfl_xor_sync(kAll, dot[j], o);
    const int own = threadIdx.x % per_token;
    if (per_token > 32) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kBack; ++j)
        if (lane == 0) part[warp][j] = dot[j];
      __syncthreads();
      if (live && own < kBack && j0 + own < k) {
        float s = 0.0f;
        for (int i = 0; i < per_token / 32; ++i) s += part[warp + i][own];
        a.dweights[t * k + j0 + own] = s;
      }
    } else if (live && own == 0) {
#pragma unroll
      for (int j = 0; j < kBack; ++j)
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
cudaError_t rows_launch(Kernel kernel, const RowArgs& a, cudaStream_t st, int per_token) {
  const int tokens = kRowThreads / per_token;
  note_launch();
  return launch_k(kernel, dim3(static_cast<unsigned>((a.T + tokens - 1) / tokens)), dim3(kRowThreads), 0, st, 1, a, per_token);
}

template <int kBits>
cudaError_t sort_launch(const RowArgs& a, const int32_t* ids, int64_t P, int64_t E, int32_t* offsets, int32_t* rows,
                        cudaStream_t st) {
  constexpr auto bytes = [](int64_t experts) { return static_cast<size_t>(kSortWarps + 2) * experts * sizeof(int); };
  constexpr size_t most = bytes(int64_t(1) << kBits);
  if constexpr (most > 48 * 1024) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(sort_kernel<kBits>, most, done);
    if (e != cudaSuccess) return e;
  }
  note_launch();
  return launch_k(sort_kernel<kBits>, dim3(kSortCtas), dim3(kSortThreads), bytes(E), st, kSortCtas, ids, P, static_cast<int>(E),
                  offsets, rows, a.status);
}

}  // namespace

// Without rows to copy (in null) only the places and offsets.
cudaError_t dispatch_launch(const RowArgs& a, const int32_t* ids, int64_t E, int32_t* offsets, int32_t* rows, cudaStream_t st) {
  const int64_t P = a.T * a.k;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(std::max<int64_t>(a.T, 32), 2 * sm_count()));
  const int64_t rounds = (a.T + grid - 1) / grid * ((a.k + kFewThreads / 32 - 1) / (kFewThreads / 32));
  if (P <= kFewPairs && rounds * P <= kFewWork) {
    note_launch();
    return launch_k(dispatch_few_kernel, dim3(grid), dim3(kFewThreads), 0, st, 1, a, ids, static_cast<int>(E), offsets, rows);
  }
  const cudaError_t e = E <= 64    ? sort_launch<6>(a, ids, P, E, offsets, rows, st)
                        : E <= 256 ? sort_launch<8>(a, ids, P, E, offsets, rows, st)
                                   : sort_launch<10>(a, ids, P, E, offsets, rows, st);
  if (e != cudaSuccess || !a.in) return e;
  RowArgs copy = a;
  copy.status = nullptr;   // what is wrong has been said
  return rows_launch(dispatch_kernel, copy, st, threads_per_token(a.C));
}

cudaError_t combine_launch(const RowArgs& a, cudaStream_t st) {
  return rows_launch(combine_kernel, a, st, threads_per_token(a.C));
}

cudaError_t combine_backward_launch(const RowArgs& a, cudaStream_t st) {
  // A warp per token where that fills the GPU: no barrier between its rows (437
  // us for the sizes above, a CTA per token 481, both with 8 rows); 64 tokens take
  // 7.3 with a CTA each.
  int per_token = threads_per_token(a.C);
  while (per_token > 32 && a.T * per_token > static_cast<int64_t>(sm_count()) * 2048) per_token /= 2;
  return rows_launch(combine_backward_kernel, a, st, per_token);
}

}  // namespace nvfp4
