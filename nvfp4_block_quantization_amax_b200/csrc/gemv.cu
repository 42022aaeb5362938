// gemv.cu -- products of a few bf16 rows with NVFP4 weights.
//
//   y[p, n] = alpha_e sum_k x[p / rep, k] q[e, n, k] Delta[e, n, k / 16],   e = ids[p]
//
// What bounds it is the weight, 0.5625 bytes per value, read once for all rows
// that need it.  q Delta has at most 6 significant bits (2 of E2M1, 4 of
// E4M3), so it is exact in bf16, and mma.sync m16n8k16 multiplies it with bf16
// x into fp32: weight rows are the 16 rows of a product, up to 8 x rows its
// columns.  A warp reads codes straight from memory into the operand's
// registers.  The order of k within a product is free as long as both
// operands share it: lane c of a quad takes 32 consecutive k (16 bytes of
// codes, 2 scales) of each 128, and the codes i and i + 4 of a word, which sit
// in its two halves, are one register's pair.
//
// A code's bits s, e e, m go to a bf16's bits 15, 8 7, 6, which is
// q 2^-126 (denormals included), by one masked multiply; times Delta 2^118 that
// is q Delta 2^-8, normal and exact.
//
// A CTA takes 32 weight rows, 8 b + g and 32, 64, 96 further of a 128-row
// atom: with that choice 16 bytes of the scale layout hold the scales of a
// lane's four rows.  Its 8 warps share out K; their sums are added in order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>

#include "launch.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTileRows = 32;

__device__ __forceinline__ void mma16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Two E4M3 bytes as bf16 pairs (each in both halves), times 2^118.
__device__ __forceinline__ void scale_pairs(uint32_t two, uint32_t* s) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<unsigned short>(two)));
  const __half2 v = *reinterpret_cast<const __half2*>(&h);
  const __nv_bfloat162 lo = __float2bfloat162_rn(__low2float(v) * 0x1p118f);
  const __nv_bfloat162 hi = __float2bfloat162_rn(__high2float(v) * 0x1p118f);
  s[0] = *reinterpret_cast<const uint32_t*>(&lo);
  s[1] = *reinterpret_cast<const uint32_t*>(&hi);
}

// The eight codes of a word times their scale: pairs (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ void decode(uint32_t w, uint32_t s, uint32_t* q) {
  const uint32_t v = w >> 8;
  q[0] = mul2(((w & 0x000F000Fu) * 0x1040u) & 0x81C081C0u, s);
  q[1] = mul2(((w & 0x00F000F0u) * 0x0104u) & 0x81C081C0u, s);
  q[2] = mul2(((v & 0x000F000Fu) * 0x1040u) & 0x81C081C0u, s);
  q[3] = mul2(((v & 0x00F000F0u) * 0x0104u) & 0x81C081C0u, s);
}

struct Weights {   // of one lane and 128 values of K
  uint4 code[4];   // rows 32 i + 8 b + g
  uint4 scale;
};

// NT: groups of eight x rows at a time.
template <int NT, typename Out>
__global__ void __launch_bounds__(kThreads) gemv_kernel(const GemvArgs a) {
  __shared__ float part[kWarps][NT * 8][kTileRows + 1];
  __shared__ int list[1024];            // pairs of this CTA's expert
  __shared__ uint32_t used[32];         // experts that occur
  __shared__ int counts[kWarps], found;
  pdl_entry();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int P = static_cast<int>(a.P);
  const int64_t N = a.N, K = a.K;
  const int64_t atom = blockIdx.x >> 2, quarter = blockIdx.x & 3;
  Out* const out = static_cast<Out*>(a.out);
  int expert = 0, members = P;
  if (a.ids) {
    // the blockIdx.y-th expert that occurs, and its pairs in order
    if (tid < 32) used[tid] = 0u;
    if (tid == 0) found = -1;
    __syncthreads();
    for (int p = tid; p < P; p += kThreads) {
      const int id = __ldg(a.ids + p);
      if (id >= 0 && id < a.E) atomicOr(&used[id >> 5], 1u << (id & 31));
      else if (id != -1 && a.status) *a.status = kStatusArg;
    }
    __syncthreads();
    if (warp == 0) {
      const uint32_t bits = used[lane];
      int upto = __popc(bits);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += v;
      }
      const int skip = static_cast<int>(blockIdx.y) - (upto - __popc(bits));
      if (skip >= 0 && skip < __popc(bits)) {
        uint32_t rest = bits;
        for (int i = 0; i < skip; ++i) rest &= rest - 1u;
        found = lane * 32 + __ffs(rest) - 1;
      }
    }
    __syncthreads();
    expert = found;
    // rows of pairs without an expert are zeros
    if (blockIdx.y == 0)
      for (int p = warp; p < P; p += kWarps) {
        const int id = __ldg(a.ids + p);
        if (id < 0 || id >= a.E) out[p * a.ldo + atom * 128 + (lane >> 3) * 32 + quarter * 8 + (lane & 7)] = Out(0.0f);
      }
    if (expert < 0) return;
    members = 0;
    for (int p0 = 0; p0 < P; p0 += kThreads) {
      const int p = p0 + tid;
      const bool is = p < P && __ldg(a.ids + p) == expert;
      const unsigned vote = __ballot_sync(0xFFFFFFFFu, is);
      if (lane == 0) counts[warp] = __popc(vote);
      __syncthreads();
      int at = members;
      for (int i = 0; i < kWarps; ++i) {
        if (i < warp) at += counts[i];
        members += counts[i];
      }
      if (is) list[at + __popc(vote & ((1u << lane) - 1u))] = p;
      __syncthreads();
    }
  }

  const int64_t row0 = atom * 128 + quarter * 8 + g;
  const uint8_t* const codes = a.W + (expert * N + row0) * (K / 2) + c * 16;
  const uint8_t* const scales = a.sW + (expert * N * (K / 16)) + (atom * (K / 64) + (c >> 1)) * 512 + (quarter * 8 + g) * 16;
  const float alpha = __ldg(a.alphaW + expert);
  const int chunks = static_cast<int>((K + 127) / 128);

  auto fetch = [&](int kc, Weights& w) {
    if (kc < chunks && kc * 128 + c * 32 < K) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w.code[i] = __ldg(reinterpret_cast<const uint4*>(codes + i * 32 * (K / 2) + kc * 64));
      w.scale = __ldg(reinterpret_cast<const uint4*>(scales + static_cast<int64_t>(kc) * 1024));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w.code[i] = make_uint4(0u, 0u, 0u, 0u);
      w.scale = make_uint4(0u, 0u, 0u, 0u);
    }
  };

  for (int m0 = 0; m0 < members; m0 += NT * 8) {
    const __nv_bfloat16* x[NT];
    bool has[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int m = m0 + i * 8 + g;
      has[i] = m < members;
      const int64_t p = !has[i] ? 0 : a.ids ? list[m] : m;
      x[i] = a.x + p / a.rep * a.ldx + c * 32;
    }
    float acc[NT][2][4] = {};
    constexpr int kDepth = 3;
    Weights w[kDepth];
#pragma unroll
    for (int s = 0; s < kDepth - 1; ++s) fetch(warp + s * kWarps, w[s]);
    for (int kc0 = warp; kc0 < chunks; kc0 += kWarps * kDepth) {
#pragma unroll
      for (int s = 0; s < kDepth; ++s) {
        const int kc = kc0 + s * kWarps;
        fetch(kc + (kDepth - 1) * kWarps, w[(s + kDepth - 1) % kDepth]);
        if (kc >= chunks) continue;
        const bool inside = kc * 128 + c * 32 < K;
        uint32_t sc[4][2];
        const uint32_t sw[4] = {w[s].scale.x, w[s].scale.y, w[s].scale.z, w[s].scale.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) scale_pairs(c & 1 ? sw[i] >> 16 : sw[i] & 0xFFFFu, sc[i]);
#pragma unroll
        for (int word = 0; word < 4; ++word) {
          uint32_t q[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t u[4] = {w[s].code[i].x, w[s].code[i].y, w[s].code[i].z, w[s].code[i].w};
            decode(u[word], sc[i][word >> 1], q[i]);
          }
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (inside && has[i]) v = __ldg(reinterpret_cast<const uint4*>(x[i] + kc * 128 + word * 8));
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t lo = half ? v.y : v.x, hi = half ? v.w : v.z;
              const uint32_t b0 = __byte_perm(lo, hi, 0x5410), b1 = __byte_perm(lo, hi, 0x7632);
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                const uint32_t op[4] = {q[2 * m][2 * half], q[2 * m + 1][2 * half], q[2 * m][2 * half + 1],
                                        q[2 * m + 1][2 * half + 1]};
                mma16(acc[i][m], op, b0, b1);
              }
            }
          }
        }
      }
    }
    __syncthreads();   // part is read until here in the round before
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 4; ++h)
          // weight row: 32 (2 m + h / 2) + g; x row 2 c + h % 2 of the group
          part[warp][i * 8 + 2 * c + (h & 1)][(2 * m + (h >> 1)) * 8 + g] = acc[i][m][h];
    __syncthreads();
    for (int v = tid; v < NT * 8 * kTileRows; v += kThreads) {
      const int m = v / kTileRows, r = v % kTileRows;
      if (m0 + m >= members) break;
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) s += part[i][m][r];
      const int64_t p = a.ids ? list[m0 + m] : m0 + m;
      out[p * a.ldo + atom * 128 + (r >> 3) * 32 + quarter * 8 + (r & 7)] = Out(s * 256.0f * alpha);
    }
  }
}

template <int NT>
cudaError_t launch_nt(const GemvArgs& a, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.N / kTileRows), static_cast<unsigned>(a.ids ? std::min(a.P, a.E) : 1));
  note_launch();
  return a.fp32 ? launch_k(gemv_kernel<NT, float>, grid, dim3(kThreads), 0, st, 1, a)
                : launch_k(gemv_kernel<NT, __nv_bfloat16>, grid, dim3(kThreads), 0, st, 1, a);
}

}  // namespace

cudaError_t gemv_launch(const GemvArgs& a, cudaStream_t st) {
  return a.P <= 8 ? launch_nt<1>(a, st) : a.P <= 16 ? launch_nt<2>(a, st) : launch_nt<4>(a, st);
}

}  // namespace nvfp4
