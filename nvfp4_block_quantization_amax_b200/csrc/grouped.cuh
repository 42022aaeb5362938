// grouped.cuh -- ragged groups of rows described on the device.
//
// T rows are sorted by group: group e owns rows offsets[e] .. offsets[e+1]-1
// (device int32, offsets[0] >= 0, offsets[E] <= T).  The host never reads the
// offsets, so every kernel builds the table it needs in shared memory: the
// offsets and two exclusive prefix sums of per-group unit counts (rows padded
// to a tile), by which a unit index is mapped back to its group.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "nvfp4_internal.h"

namespace nvfp4 {

constexpr int kMaxGroups = 1024;

// The most rows that groups of T rows in all take up, each group padded to a
// multiple of `step` (a group without rows takes none).
inline int64_t grouped_capacity(int64_t T, int64_t E, int64_t step) {
  return (T + (T < E ? T : E) * (step - 1)) / step * step;
}

__host__ __device__ constexpr size_t group_table_bytes(int E) { return 3u * (static_cast<size_t>(E) + 1u) * sizeof(int); }

struct GroupTable {
  int* off;   // [E + 1] offsets
  int* pa;    // [E + 1] exclusive prefix of ceil(rows / step_a)
  int* pb;    // [E + 1] exclusive prefix of ceil(rows / step_b)
  int E;
  __device__ __forceinline__ int rows(int e) const { return off[e + 1] - off[e]; }
};

// Build the table with all NT threads of the CTA; ends with a barrier.
// Offsets that decrease or leave [0, T] make every group empty and set
// NVFP4_ERR_ARG (first CTA), so a bad table never addresses memory.
// mem: group_table_bytes(E) bytes of shared memory.
template <int NT>
__device__ __forceinline__ GroupTable build_group_table(const int32_t* __restrict__ offsets, int E, int64_t T,
                                                        int step_a, int step_b, int* mem, int32_t* status,
                                                        bool report) {
  GroupTable t{mem, mem + (E + 1), mem + 2 * (E + 1), E};
  __shared__ int warp_a[NT / 32], warp_b[NT / 32];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  bool bad = false;
  for (int e = tid; e <= E; e += NT) {
    const int o = __ldg(offsets + e);
    bad |= o < 0 || o > T || (e > 0 && __ldg(offsets + e - 1) > o);
    t.off[e] = o;
  }
  const bool invalid = __syncthreads_or(bad);
  if (invalid) {
    for (int e = tid; e <= E; e += NT) t.off[e] = 0;
    if (report && tid == 0 && status) *status = kStatusArg;
    __syncthreads();
  }
  // each thread sums a run of consecutive groups, then a block-wide scan
  const int per = (E + NT - 1) / NT;
  const int e0 = tid * per < E ? tid * per : E, e1 = e0 + per < E ? e0 + per : E;
  int sa = 0, sb = 0;
  for (int e = e0; e < e1; ++e) {
    const int r = t.off[e + 1] - t.off[e];
    sa += (r + step_a - 1) / step_a;
    sb += (r + step_b - 1) / step_b;
  }
  int ia = sa, ib = sb;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int ua = __shfl_up_sync(0xFFFFFFFFu, ia, o), ub = __shfl_up_sync(0xFFFFFFFFu, ib, o);
    if (lane >= o) {
      ia += ua;
      ib += ub;
    }
  }
  if (lane == 31) {
    warp_a[w] = ia;
    warp_b[w] = ib;
  }
  __syncthreads();
  int ba = ia - sa, bb = ib - sb;
  for (int i = 0; i < w; ++i) {
    ba += warp_a[i];
    bb += warp_b[i];
  }
  for (int e = e0; e < e1; ++e) {
    t.pa[e] = ba;
    t.pb[e] = bb;
    const int r = t.off[e + 1] - t.off[e];
    ba += (r + step_a - 1) / step_a;
    bb += (r + step_b - 1) / step_b;
    if (e + 1 == E) {
      t.pa[E] = ba;
      t.pb[E] = bb;
    }
  }
  __syncthreads();
  return t;
}

// The group that holds unit u of prefix p (p[e] <= u < p[e + 1]); 0 <= u < p[E].
__device__ __forceinline__ int find_group(const int* p, int E, int u) {
  int lo = 0, hi = E;   // p[lo] <= u < p[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p[mid] <= u) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace nvfp4
