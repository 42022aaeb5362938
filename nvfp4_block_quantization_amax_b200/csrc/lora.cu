// lora.cu -- low-rank adapters of many requests beside a shared projection.
//
//   forward:   h[t] = A_a x[t],   out[t] = y[t] + s_a B_a h[t],    a = ids[t]
//   backward:  g[t] = B_a^T dy[t],  dx[t] = dx0[t] + s_a A_a^T g[t],
//              dA_a = s_a sum_{ids[t] = a} g[t] x[t]^T,
//              dB_a = s_a sum_{ids[t] = a} dy[t] h[t]^T
// y is the projection's bf16 result (nvfp4_gemm of the frozen weight); A_a
// [r, K] and B_a [N, r] are bf16.  ids[t] = -1: the token has no adapter.
//
// Three kernels, each used in both directions:
//   shrink  (x, A) -> h and (dy, B) -> g: contraction over the long axis,
//           split over CTAs into fp32 partial sums;
//   expand  (h, B) + y -> out and (g, A) + dx0 -> dx: contraction over the
//           rank; sums the partials first, in their order;
//   outer   (g, x) -> dA and (h, dy) -> dB: contraction over one adapter's
//           tokens.
// The products are small (2 T r (K + N) flops) beside the rows that pass
// through memory, so they run on mma.sync with bf16 operands and fp32 sums.
// h and g are kept in fp32; where they are an operand of a product they enter
// as the sum of two bf16 numbers (16 bits of mantissa, error 2^-17), which
// costs one more product of the rank's size instead of bf16's 2^-9.
// Adapters are found tile by tile: a tile of 64 tokens loops over the
// adapters that occur in it, so tokens of one request (in a row) share one
// pass and any order is right.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>

#include "launch.cuh"
#include "nvfp4_internal.h"
#include "tile.cuh"

namespace nvfp4 {
namespace {

constexpr int kRows = 64;      // tokens of a tile
constexpr int kStep = 64;      // columns of a shrink stage
constexpr int kCols = 128;     // columns of an expand / outer tile
constexpr int kStagesL = 3;
constexpr int kMaxSplit = 32;

struct AdapterIds {
  const int32_t* ids;
  int64_t T;
  int n;
  int32_t* status;
};

// Adapter of token t: -1 for none, for rows past the last token, and for an
// id that names no adapter (which also sets the status).
__device__ __forceinline__ int adapter_of(const AdapterIds& a, int64_t t, bool report) {
  if (t >= a.T) return -1;
  const int id = __ldg(a.ids + t);
  if (id >= 0 && id < a.n) return id;
  if (id != -1 && report && a.status) *a.status = kStatusArg;
  return -1;
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void ldsm4(uint32_t* r, const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(smem_addr(p)) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t* r, const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(smem_addr(p)) : "memory");
}
// d += a (16 x 16) b (16 x 8), bf16 operands, fp32 sums
__device__ __forceinline__ void mma16(float* d, const uint32_t* a, const uint32_t* b) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

__device__ __forceinline__ void copy16(void* smem, const void* gmem, bool valid) {
  const int bytes = valid ? 16 : 0;   // 0: the 16 bytes become zero, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_addr(smem)), "l"(gmem), "r"(bytes) : "memory");
}

// v = hi + lo up to 2^-17 |v| (an infinity or NaN is all in hi: its lo would
// be a NaN of its own)
__device__ __forceinline__ void split_bf16(float v, __nv_bfloat16& hi, __nv_bfloat16& lo) {
  hi = __float2bfloat16_rn(v);
  const float rest = __fsub_rn(v, __bfloat162float(hi));
  lo = __float2bfloat16_rn(fabsf(rest) <= 3.402823466e38f ? rest : 0.0f);
}

// The adapters of a tile of 64 tokens: ids[64] (-1: none) and the list of the
// distinct ones.  All threads call it (NT >= 64); ends with a barrier.
struct TileAdapters {
  int ids[kRows];
  int list[kRows];
  int count;
};
__device__ __forceinline__ void tile_adapters(TileAdapters& ta, const AdapterIds& a, int64_t row0, bool report) {
  const int t = threadIdx.x;
  __shared__ uint32_t firsts[2];
  if (t < kRows) ta.ids[t] = adapter_of(a, row0 + t, report);
  __syncthreads();
  bool first = false;
  if (t < kRows) {
    const int id = ta.ids[t];
    first = id >= 0;
    for (int j = 0; j < t; ++j) first = first && ta.ids[j] != id;
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, first);
    if ((t & 31) == 0) firsts[t >> 5] = m;
  }
  __syncthreads();
  if (t < kRows) {
    const uint32_t below = firsts[t >> 5] & ((1u << (t & 31)) - 1u);
    if (first) ta.list[__popc(below) + (t >= 32 ? __popc(firsts[0]) : 0)] = ta.ids[t];
    if (t == 0) ta.count = __popc(firsts[0]) + __popc(firsts[1]);
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// shrink: part[split][t][j] = sum over this split's columns of z[t, c] W[j, c]
// TRANS: W is stored [C, r] (c-major), else [r, C].
// ---------------------------------------------------------------------------
template <int RP, bool TRANS>
struct ShrinkSmem {
  static constexpr int R = 16 * RP;
  static constexpr int ZB = kRows * (kStep + 8) * 2;
  static constexpr int WB = (TRANS ? kStep * (R + 8) : R * (kStep + 8)) * 2;
  static constexpr int BYTES = kStagesL * (ZB + WB);
};

template <int RP, bool TRANS>
__global__ void __launch_bounds__(128) lora_shrink_kernel(const __nv_bfloat16* __restrict__ z, int64_t ldz,
                                                          const __nv_bfloat16* __restrict__ W, const AdapterIds a,
                                                          int64_t C, int r, int64_t per_split,
                                                          float* __restrict__ part) {
  pdl_entry();
  using S = ShrinkSmem<RP, TRANS>;
  constexpr int R = S::R;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ TileAdapters ta;
  const int th = threadIdx.x, lane = th & 31, warp = th >> 5;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kRows;
  const int64_t c_begin = blockIdx.y * per_split;
  const int64_t c_end = c_begin + per_split < C ? c_begin + per_split : C;
  const int steps = static_cast<int>((c_end - c_begin + kStep - 1) / kStep);
  tile_adapters(ta, a, row0, blockIdx.y == 0);
  float* mine = part + static_cast<int64_t>(blockIdx.y) * a.T * r;

  auto load = [&](int st, int step, const __nv_bfloat16* w) {
    uint8_t* base = dyn + st * (S::ZB + S::WB);
    const int64_t c0 = c_begin + static_cast<int64_t>(step) * kStep;
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // 64 rows x 8 chunks
      const int k = th + 128 * i, row = k >> 3, ch = k & 7;
      const bool ok = row0 + row < a.T && c0 + 8 * ch < c_end && ta.ids[row] >= 0;
      copy16(base + row * (kStep + 8) * 2 + 16 * ch, ok ? z + (row0 + row) * ldz + c0 + 8 * ch : z, ok);
    }
    uint8_t* wb = base + S::ZB;
    if constexpr (!TRANS) {
      for (int k = th; k < R * 8; k += 128) {
        const int j = k >> 3, ch = k & 7;
        const bool ok = j < r && c0 + 8 * ch < c_end;
        copy16(wb + j * (kStep + 8) * 2 + 16 * ch, ok ? w + j * C + c0 + 8 * ch : w, ok);
      }
    } else {
      for (int k = th; k < kStep * (R / 8); k += 128) {
        const int c = k / (R / 8), ch = k % (R / 8);
        const bool ok = c0 + c < c_end && 8 * ch < r;
        copy16(wb + c * (R + 8) * 2 + 16 * ch, ok ? w + (c0 + c) * r + 8 * ch : w, ok);
      }
    }
    cp_async_commit();
  };

  for (int u = 0; u < ta.count; ++u) {
    const int id = ta.list[u];
    const __nv_bfloat16* w = W + static_cast<int64_t>(id) * r * C;
    float sum[2 * RP][4];
#pragma unroll
    for (int i = 0; i < 2 * RP; ++i) sum[i][0] = sum[i][1] = sum[i][2] = sum[i][3] = 0.0f;
#pragma unroll
    for (int p = 0; p < kStagesL - 1; ++p) {
      if (p < steps) load(p, p, w);
      else cp_async_commit();
    }
    for (int s = 0; s < steps; ++s) {
      cp_async_wait<kStagesL - 2>();
      __syncthreads();
      if (s + kStagesL - 1 < steps) load((s + kStagesL - 1) % kStagesL, s + kStagesL - 1, w);
      else cp_async_commit();
      const uint8_t* base = dyn + (s % kStagesL) * (S::ZB + S::WB);
      const __nv_bfloat16* zs = reinterpret_cast<const __nv_bfloat16*>(base);
      const __nv_bfloat16* ws = reinterpret_cast<const __nv_bfloat16*>(base + S::ZB);
      // this stage's sums start from zero and are added to the running ones:
      // the tensor core truncates as it adds, so its runs are kept short
      float acc[2 * RP][4];
#pragma unroll
      for (int i = 0; i < 2 * RP; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
#pragma unroll
      for (int kk = 0; kk < kStep; kk += 16) {
        uint32_t af[4];
        ldsm4(af, zs + (16 * warp + (lane & 15)) * (kStep + 8) + kk + (lane >> 4) * 8);
#pragma unroll
        for (int p = 0; p < RP; ++p) {
          uint32_t bf[4];
          if constexpr (!TRANS)
            ldsm4(bf, ws + (16 * p + (lane & 7) + ((lane >> 4) << 3)) * (kStep + 8) + kk + ((lane >> 3) & 1) * 8);
          else
            ldsm4_t(bf, ws + (kk + (lane & 7) + ((lane >> 3) & 1) * 8) * (R + 8) + 16 * p + (lane >> 4) * 8);
          mma16(acc[2 * p], af, bf);
          mma16(acc[2 * p + 1], af, bf + 2);
        }
      }
#pragma unroll
      for (int i = 0; i < 2 * RP; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[i][e] = __fadd_rn(sum[i][e], acc[i][e]);
    }
    __syncthreads();   // every warp has read the last stage before the next adapter's loads
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int row = 16 * warp + (lane >> 2) + 8 * half;
      if (ta.ids[row] == id) {
#pragma unroll
        for (int i = 0; i < 2 * RP; ++i) {
          const int j = 8 * i + 2 * (lane & 3);
          if (j < r)
            *reinterpret_cast<float2*>(mine + (row0 + row) * r + j) = make_float2(sum[i][2 * half], sum[i][2 * half + 1]);
        }
      }
    }
  }
  // tokens without an adapter
  for (int k = th; k < kRows * r; k += 128) {
    const int row = k / r;
    if (ta.ids[row] < 0 && row0 + row < a.T) mine[(row0 + row) * r + (k - row * r)] = 0.0f;
  }
}

// ---------------------------------------------------------------------------
// expand: out[t, c] = base[t, c] + s_a sum_j w[t, j] W[c, j], w = sum of the
// partials; w itself goes to w_out.  TRANS: W is stored [r, C], else [C, r].
// A CTA takes 64 tokens and `per_cta` column tiles.
// ---------------------------------------------------------------------------
template <int RP, bool TRANS>
struct ExpandSmem {
  static constexpr int R = 16 * RP;
  static constexpr int HB = kRows * (R + 8) * 2;
  static constexpr int WB = (TRANS ? R * (kCols + 8) : kCols * (R + 8)) * 2;
  static constexpr int DB = kRows * (kCols + 4) * 4;
  static constexpr int BYTES = 2 * HB + WB + DB;
};

template <int RP, bool TRANS>
__global__ void __launch_bounds__(128) lora_expand_kernel(const float* __restrict__ part, int splits,
                                                          const __nv_bfloat16* __restrict__ W,
                                                          const float* __restrict__ scaling, const AdapterIds a,
                                                          int64_t C, int r, int per_cta,
                                                          const __nv_bfloat16* __restrict__ in, int64_t ldi,
                                                          __nv_bfloat16* __restrict__ out, int64_t ldo,
                                                          float* __restrict__ w_out) {
  pdl_entry();
  using S = ExpandSmem<RP, TRANS>;
  constexpr int R = S::R;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ TileAdapters ta;
  __nv_bfloat16* hh = reinterpret_cast<__nv_bfloat16*>(dyn);
  __nv_bfloat16* hl = reinterpret_cast<__nv_bfloat16*>(dyn + S::HB);
  __nv_bfloat16* ws = reinterpret_cast<__nv_bfloat16*>(dyn + 2 * S::HB);
  float* delta = reinterpret_cast<float*>(dyn + 2 * S::HB + S::WB);
  const int th = threadIdx.x, lane = th & 31, warp = th >> 5;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kRows;
  tile_adapters(ta, a, row0, false);
  // the sum of the partials, in their order
  for (int k = th; k < kRows * R; k += 128) {
    const int row = k / R, j = k % R;
    float v = 0.0f;
    if (row0 + row < a.T && j < r) {
      const int64_t at = (row0 + row) * r + j;
      for (int s = 0; s < splits; ++s) v = __fadd_rn(v, __ldcg(part + s * a.T * r + at));
      if (w_out && blockIdx.y == 0) w_out[at] = v;
    }
    split_bf16(v, hh[row * (R + 8) + j], hl[row * (R + 8) + j]);
  }
  if (!out) return;   // only the sum was asked for
  __syncthreads();

  for (int i = 0; i < per_cta; ++i) {
    const int64_t c0 = (static_cast<int64_t>(blockIdx.y) * per_cta + i) * kCols;
    if (c0 >= C) break;
    // this warp's rows of the base: lane l takes 16 bytes l % 16 of rows 2 p + l / 16
    const int piece = lane & 15;
    const bool col_ok = c0 + 8 * piece < C;
    uint4 y[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const int64_t t = row0 + 16 * warp + 2 * p + (lane >> 4);
      y[p] = make_uint4(0u, 0u, 0u, 0u);
      if (in && col_ok && t < a.T) y[p] = __ldcg(reinterpret_cast<const uint4*>(in + t * ldi + c0 + 8 * piece));
    }
    // tokens without an adapter add nothing
    float* mine = delta + 16 * warp * (kCols + 4);
    for (int row = 0; row < 16; ++row)
      if (ta.ids[16 * warp + row] < 0)
        *reinterpret_cast<float4*>(mine + row * (kCols + 4) + 4 * lane) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int u = 0; u < ta.count; ++u) {
      const int id = ta.list[u];
      const __nv_bfloat16* w = W + static_cast<int64_t>(id) * r * C;
      __syncthreads();   // the previous weights have been read
      if constexpr (!TRANS) {
        for (int k = th; k < kCols * (R / 8); k += 128) {
          const int c = k / (R / 8), ch = k % (R / 8);
          const bool ok = c0 + c < C && 8 * ch < r;
          copy16(ws + c * (R + 8) + 8 * ch, ok ? w + (c0 + c) * r + 8 * ch : w, ok);
        }
      } else {
        for (int k = th; k < R * (kCols / 8); k += 128) {
          const int j = k / (kCols / 8), ch = k % (kCols / 8);
          const bool ok = j < r && c0 + 8 * ch < C;
          copy16(ws + j * (kCols + 8) + 8 * ch, ok ? w + j * C + c0 + 8 * ch : w, ok);
        }
      }
      cp_async_commit();
      cp_async_wait<0>();
      __syncthreads();
      bool any = false;
      for (int row = 0; row < 16; ++row) any |= ta.ids[16 * warp + row] == id;
      if (!any) continue;   // uniform over the warp
      const float s = __ldg(scaling + id);
#pragma unroll
      for (int nb = 0; nb < kCols; nb += 16) {
        float acc[2][4] = {};
#pragma unroll
        for (int kk = 0; kk < R; kk += 16) {
          uint32_t ah[4], al[4], bf[4];
          ldsm4(ah, hh + (16 * warp + (lane & 15)) * (R + 8) + kk + (lane >> 4) * 8);
          ldsm4(al, hl + (16 * warp + (lane & 15)) * (R + 8) + kk + (lane >> 4) * 8);
          if constexpr (!TRANS)
            ldsm4(bf, ws + (nb + (lane & 7) + ((lane >> 4) << 3)) * (R + 8) + kk + ((lane >> 3) & 1) * 8);
          else
            ldsm4_t(bf, ws + (kk + (lane & 7) + ((lane >> 3) & 1) * 8) * (kCols + 8) + nb + (lane >> 4) * 8);
          mma16(acc[0], al, bf);
          mma16(acc[1], al, bf + 2);
          mma16(acc[0], ah, bf);
          mma16(acc[1], ah, bf + 2);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int row = (lane >> 2) + 8 * half;
          if (ta.ids[16 * warp + row] == id) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
              *reinterpret_cast<float2*>(mine + row * (kCols + 4) + nb + 8 * q + 2 * (lane & 3)) =
                  make_float2(__fmul_rn(s, acc[q][2 * half]), __fmul_rn(s, acc[q][2 * half + 1]));
          }
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const int row = 2 * p + (lane >> 4);
      const int64_t t = row0 + 16 * warp + row;
      const float* d = mine + row * (kCols + 4) + 8 * piece;
      const float4 d0 = *reinterpret_cast<const float4*>(d), d1 = *reinterpret_cast<const float4*>(d + 4);
      const float dv[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
      const uint32_t yw[4] = {y[p].x, y[p].y, y[p].z, y[p].w};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(__fadd_rn(__uint_as_float(yw[j] << 16), dv[2 * j]),
                                                       __fadd_rn(__uint_as_float(yw[j] & 0xFFFF0000u), dv[2 * j + 1]));
        o[j] = *reinterpret_cast<const uint32_t*>(&b);
      }
      // a token without an adapter keeps the base's bits (a NaN's payload, a zero's sign)
      if (col_ok && t < a.T)
        *reinterpret_cast<uint4*>(out + t * ldo + c0 + 8 * piece) =
            ta.ids[16 * warp + row] < 0 ? y[p] : make_uint4(o[0], o[1], o[2], o[3]);
    }
    __syncwarp();
  }
}

// ---------------------------------------------------------------------------
// outer: P[a][j, c] = s_a sum_{ids[t] = a} w[t, j] z[t, c] over a range of
// row tiles.  Rows of other adapters are not read (their slots are zero, so a
// NaN there reaches nothing).  COLS_FIRST: P is stored [C, r], else [r, C].
// grid: column tile, adapter, split.
// ---------------------------------------------------------------------------
constexpr int kOuterNT = 256;

template <int RP>
struct OuterSmem {
  static constexpr int R = 16 * RP;
  static constexpr int ZB = kRows * (kCols + 8) * 2;
  static constexpr int HB = kRows * (R + 8) * 2;
  static constexpr int BYTES = 2 * (ZB + 2 * HB);
};

__device__ __forceinline__ void store_out(void* dst, int64_t at, float v, bool fp32) {
  if (fp32) static_cast<float*>(dst)[at] = v;
  else static_cast<__nv_bfloat16*>(dst)[at] = __float2bfloat16_rn(v);
}

template <int RP, bool COLS_FIRST>
__global__ void __launch_bounds__(kOuterNT) lora_outer_kernel(const float* __restrict__ w,
                                                              const __nv_bfloat16* __restrict__ z, int64_t ldz,
                                                              const float* __restrict__ scaling, const AdapterIds a,
                                                              int64_t C, int r, void* __restrict__ dst, int fp32,
                                                              float* __restrict__ part, int32_t* __restrict__ used) {
  pdl_entry();
  using S = OuterSmem<RP>;
  constexpr int R = S::R;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ int ids[2][kRows];
  const int th = threadIdx.x, lane = th & 31, warp = th >> 5;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kCols;
  const int id = blockIdx.y, splits = gridDim.z, split = blockIdx.z;
  const int tiles = static_cast<int>((a.T + kRows - 1) / kRows);
  const int first = static_cast<int>(static_cast<int64_t>(tiles) * split / splits);
  const int last = static_cast<int>(static_cast<int64_t>(tiles) * (split + 1) / splits);

  // the next row tile from `tile` on that holds a token of this adapter, its
  // ids in ids[b]; `last` if there is none
  auto next = [&](int tile, int b) {
    for (; tile < last; ++tile) {
      bool mine = false;
      if (th < kRows) {
        const int v = adapter_of(a, static_cast<int64_t>(tile) * kRows + th, false);
        ids[b][th] = v;
        mine = v == id;
      }
      if (__syncthreads_or(mine)) return tile;
    }
    return last;
  };
  auto load = [&](int tile, int b) {
    uint8_t* base = dyn + b * (S::ZB + 2 * S::HB);
    const int64_t row0 = static_cast<int64_t>(tile) * kRows;
#pragma unroll
    for (int i = 0; i < kRows * 16 / kOuterNT; ++i) {
      const int k = th + kOuterNT * i, row = k >> 4, ch = k & 15;
      const bool ok = ids[b][row] == id && c0 + 8 * ch < C;
      copy16(base + row * (kCols + 8) * 2 + 16 * ch, ok ? z + (row0 + row) * ldz + c0 + 8 * ch : z, ok);
    }
    cp_async_commit();
    __nv_bfloat16* hh = reinterpret_cast<__nv_bfloat16*>(base + S::ZB);
    __nv_bfloat16* hl = reinterpret_cast<__nv_bfloat16*>(base + S::ZB + S::HB);
    for (int k = th; k < kRows * R; k += kOuterNT) {
      const int row = k / R, j = k % R;
      const float v = (j < r && ids[b][row] == id) ? __ldg(w + (row0 + row) * r + j) : 0.0f;
      split_bf16(v, hh[row * (R + 8) + j], hl[row * (R + 8) + j]);
    }
  };

  float sum[RP][2][4];
#pragma unroll
  for (int m = 0; m < RP; ++m)
#pragma unroll
    for (int q = 0; q < 2; ++q) sum[m][q][0] = sum[m][q][1] = sum[m][q][2] = sum[m][q][3] = 0.0f;
  int tile = next(first, 0), b = 0;
  const bool any = tile < last;
  if (any) load(tile, 0);
  while (tile < last) {
    const int ahead = next(tile + 1, b ^ 1);   // its barriers also free the other buffer
    if (ahead < last) load(ahead, b ^ 1);
    else cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    const uint8_t* base = dyn + b * (S::ZB + 2 * S::HB);
    const __nv_bfloat16* zs = reinterpret_cast<const __nv_bfloat16*>(base);
    const __nv_bfloat16* hh = reinterpret_cast<const __nv_bfloat16*>(base + S::ZB);
    const __nv_bfloat16* hl = reinterpret_cast<const __nv_bfloat16*>(base + S::ZB + S::HB);
#pragma unroll
    for (int m = 0; m < RP; ++m) {
      float acc[2][4] = {};
#pragma unroll
      for (int kk = 0; kk < kRows; kk += 16) {
        uint32_t ah[4], al[4], bf[4];
        const int arow = kk + (lane & 7) + ((lane >> 4) << 3), acol = 16 * m + ((lane >> 3) & 1) * 8;
        ldsm4_t(ah, hh + arow * (R + 8) + acol);
        ldsm4_t(al, hl + arow * (R + 8) + acol);
        ldsm4_t(bf, zs + (kk + (lane & 7) + ((lane >> 3) & 1) * 8) * (kCols + 8) + 16 * warp + (lane >> 4) * 8);
        mma16(acc[0], al, bf);
        mma16(acc[1], al, bf + 2);
        mma16(acc[0], ah, bf);
        mma16(acc[1], ah, bf + 2);
      }
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[m][q][e] = __fadd_rn(sum[m][q][e], acc[q][e]);
    }
    __syncthreads();   // this buffer is refilled in the next round
    tile = ahead;
    b ^= 1;
  }
  cp_async_wait<0>();
  const bool direct = splits == 1;
  if (!direct) {
    if (th == 0) used[(static_cast<int64_t>(id) * splits + split) * gridDim.x + blockIdx.x] = any ? 1 : 0;
    if (!any) return;
  }
  const float s = direct ? __ldg(scaling + id) : 1.0f;   // with splits the sum is scaled once, at the end
#pragma unroll
  for (int m = 0; m < RP; ++m)
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = 16 * m + (lane >> 2) + 8 * (e >> 1);
        const int64_t c = c0 + 16 * warp + 8 * q + 2 * (lane & 3) + (e & 1);
        if (j < r && c < C) {
          const int64_t at = COLS_FIRST ? (static_cast<int64_t>(id) * C + c) * r + j : (static_cast<int64_t>(id) * r + j) * C + c;
          if (direct) store_out(dst, at, __fmul_rn(s, sum[m][q][e]), fp32);
          else part[static_cast<int64_t>(split) * a.n * r * C + at] = sum[m][q][e];
        }
      }
}

// Sum of the splits' partials, in their order, those that saw a token.
template <bool COLS_FIRST>
__global__ void __launch_bounds__(256) lora_outer_sum_kernel(const float* __restrict__ part,
                                                             const int32_t* __restrict__ used, int splits, int n,
                                                             int64_t C, int r, const float* __restrict__ scaling,
                                                             void* __restrict__ dst, int fp32) {
  pdl_entry();
  const int64_t per = r * C, total = per * n;
  const int col_tiles = static_cast<int>((C + kCols - 1) / kCols);
  for (int64_t k = blockIdx.x * 256ll + threadIdx.x; k < total; k += gridDim.x * 256ll) {
    const int id = static_cast<int>(k / per);
    const int64_t in = k - id * per, c = COLS_FIRST ? in / r : in % C;
    float v = 0.0f;
    for (int s = 0; s < splits; ++s)
      if (__ldcg(used + (static_cast<int64_t>(id) * splits + s) * col_tiles + c / kCols))
        v = __fadd_rn(v, __ldcg(part + s * total + k));
    store_out(dst, k, __fmul_rn(__ldg(scaling + id), v), fp32);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Columns per shrink split: enough CTAs for four on each SM, whole stages.
int64_t shrink_per_split(int64_t T, int64_t C) {
  const int64_t tiles = ceil_div(T, kRows);
  int64_t splits = std::max<int64_t>(1, std::min<int64_t>(kMaxSplit, ceil_div(4 * sm_count(), tiles)));
  return ceil_div(ceil_div(C, splits), kStep) * kStep;
}
int shrink_splits(int64_t T, int64_t C) { return static_cast<int>(ceil_div(C, shrink_per_split(T, C))); }

// Row ranges per outer product: with requests in a row, about (splits + n)
// of the (adapter, range) pairs hold tokens.
int outer_splits(int64_t T, int64_t C, int64_t n) {
  const int64_t col_tiles = ceil_div(C, kCols), tiles = ceil_div(T, kRows);
  const int64_t want = ceil_div(3 * sm_count(), col_tiles) - n + 1;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({want, 8, ceil_div(tiles, 4)})));
}

// Parts of the workspace, in 16-byte steps.
struct LoraWorkspace {
  size_t part, sum, outer, used, total;
};
size_t up16(size_t v) { return (v + 15) & ~static_cast<size_t>(15); }
LoraWorkspace lora_workspace(int64_t T, int64_t K, int64_t N, int64_t r, int64_t n, bool backward) {
  LoraWorkspace w{};
  const int64_t C = backward ? N : K;
  w.part = 0;
  w.sum = up16(static_cast<size_t>(shrink_splits(T, C)) * T * r * 4);
  w.total = w.sum;
  if (backward) {
    w.outer = w.sum + up16(static_cast<size_t>(T) * r * 4);
    const int sa = outer_splits(T, K, n), sb = outer_splits(T, N, n);
    const size_t pa = sa > 1 ? static_cast<size_t>(sa) * n * r * K * 4 : 0, pb = sb > 1 ? static_cast<size_t>(sb) * n * r * N * 4 : 0;
    w.used = w.outer + up16(std::max(pa, pb));
    w.total = w.used + up16(static_cast<size_t>(std::max(sa * ceil_div(K, kCols), sb * ceil_div(N, kCols))) * n * 4);
  }
  return w;
}

template <class F>
cudaError_t allow_smem(F fn, int bytes, bool* done) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  return e;
}

template <int RP, bool TRANS>
cudaError_t shrink(const __nv_bfloat16* z, int64_t ldz, const __nv_bfloat16* W, const AdapterIds& a, int64_t C, int r,
                   float* part, cudaStream_t st) {
  auto fn = lora_shrink_kernel<RP, TRANS>;
  constexpr int smem = ShrinkSmem<RP, TRANS>::BYTES;
  static bool done[64] = {false};
  cudaError_t e = allow_smem(fn, smem, done);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(ceil_div(a.T, kRows)), static_cast<unsigned>(shrink_splits(a.T, C)));
  e = launch_k(fn, grid, dim3(128), smem, st, 1u, z, ldz, W, a, C, r, shrink_per_split(a.T, C), part);
  note_launch();
  return e;
}

template <int RP, bool TRANS>
cudaError_t expand(const float* part, int splits, const __nv_bfloat16* W, const float* scaling, const AdapterIds& a,
                   int64_t C, int r, const __nv_bfloat16* in, int64_t ldi, __nv_bfloat16* out, int64_t ldo, float* w_out,
                   cudaStream_t st) {
  auto fn = lora_expand_kernel<RP, TRANS>;
  constexpr int smem = ExpandSmem<RP, TRANS>::BYTES;
  static bool done[64] = {false};
  cudaError_t e = allow_smem(fn, smem, done);
  if (e != cudaSuccess) return e;
  // up to eight column tiles share one sum of the partials, as long as the
  // grid still fills the GPU twice
  const int64_t rows = ceil_div(a.T, kRows), cols = ceil_div(C, kCols);
  const int per = out ? static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(8, rows * cols / (8 * sm_count())))) : 1;
  const dim3 grid(static_cast<unsigned>(rows), out ? static_cast<unsigned>(ceil_div(cols, per)) : 1u);
  e = launch_k(fn, grid, dim3(128), smem, st, 1u, part, splits, W, scaling, a, C, r, per, in, ldi, out, ldo, w_out);
  note_launch();
  return e;
}

template <int RP, bool COLS_FIRST>
cudaError_t outer(const float* w, const __nv_bfloat16* z, int64_t ldz, const float* scaling, const AdapterIds& a,
                  int64_t C, int r, void* dst, bool fp32, float* part, int32_t* used, cudaStream_t st) {
  auto fn = lora_outer_kernel<RP, COLS_FIRST>;
  constexpr int smem = OuterSmem<RP>::BYTES;
  static bool done[64] = {false};
  cudaError_t e = allow_smem(fn, smem, done);
  if (e != cudaSuccess) return e;
  const int splits = outer_splits(a.T, C, a.n);
  const dim3 grid(static_cast<unsigned>(ceil_div(C, kCols)), static_cast<unsigned>(a.n), static_cast<unsigned>(splits));
  e = launch_k(fn, grid, dim3(kOuterNT), smem, st, 1u, w, z, ldz, scaling, a, C, r, dst, static_cast<int>(fp32), part, used);
  note_launch();
  if (e != cudaSuccess || splits == 1) return e;
  const int64_t blocks = std::min<int64_t>(ceil_div(static_cast<int64_t>(a.n) * r * C, 256), 8 * sm_count());
  e = launch_k(lora_outer_sum_kernel<COLS_FIRST>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, 1u, part, used,
               splits, a.n, C, r, scaling, dst, static_cast<int>(fp32));
  note_launch();
  return e;
}

template <int RP>
cudaError_t forward(const LoraArgs& l, float* part, cudaStream_t st) {
  const AdapterIds a{l.ids, l.T, static_cast<int>(l.n), l.status};
  cudaError_t e = shrink<RP, false>(l.x, l.ldx, l.A, a, l.K, static_cast<int>(l.r), part, st);
  if (e != cudaSuccess) return e;
  return expand<RP, false>(part, shrink_splits(l.T, l.K), l.B, l.scaling, a, l.N, static_cast<int>(l.r), l.in, l.ldi,
                           l.out, l.ldo, l.h, st);
}

template <int RP>
cudaError_t backward(const LoraArgs& l, uint8_t* ws, const LoraWorkspace& w, cudaStream_t st) {
  const AdapterIds a{l.ids, l.T, static_cast<int>(l.n), l.status};
  const int r = static_cast<int>(l.r);
  float* part = reinterpret_cast<float*>(ws + w.part);
  float* g = reinterpret_cast<float*>(ws + w.sum);
  float* outer_part = reinterpret_cast<float*>(ws + w.outer);
  int32_t* used = reinterpret_cast<int32_t*>(ws + w.used);
  cudaError_t e = cudaSuccess;
  if (l.out || l.dA) {
    e = shrink<RP, true>(l.dy, l.lddy, l.B, a, l.N, r, part, st);
    if (e != cudaSuccess) return e;
    e = expand<RP, true>(part, shrink_splits(l.T, l.N), l.A, l.scaling, a, l.K, r, l.in, l.ldi, l.out, l.ldo, g, st);
    if (e != cudaSuccess) return e;
  }
  if (l.dA) {
    e = outer<RP, false>(g, l.x, l.ldx, l.scaling, a, l.K, r, l.dA, l.fp32, outer_part, used, st);
    if (e != cudaSuccess) return e;
  }
  if (l.dB) e = outer<RP, true>(l.h, l.dy, l.lddy, l.scaling, a, l.N, r, l.dB, l.fp32, outer_part, used, st);
  return e;
}

}  // namespace

size_t lora_workspace_bytes(int64_t T, int64_t K, int64_t N, int64_t r, int64_t n, bool backward) {
  return T == 0 ? 0 : lora_workspace(T, K, N, r, n, backward).total;
}

cudaError_t lora_forward_launch(const LoraArgs& l, void* workspace, cudaStream_t st) {
  float* part = static_cast<float*>(workspace);
  if (l.r <= 16) return forward<1>(l, part, st);
  if (l.r <= 32) return forward<2>(l, part, st);
  if (l.r <= 64) return forward<4>(l, part, st);
  return forward<8>(l, part, st);
}

cudaError_t lora_backward_launch(const LoraArgs& l, void* workspace, cudaStream_t st) {
  if (l.T == 0) {
    cudaError_t e = cudaSuccess;
    const size_t size = l.fp32 ? 4 : 2;
    if (l.dA) e = cudaMemsetAsync(l.dA, 0, static_cast<size_t>(l.n * l.r * l.K) * size, st);
    if (e == cudaSuccess && l.dB) e = cudaMemsetAsync(l.dB, 0, static_cast<size_t>(l.n * l.r * l.N) * size, st);
    return e;
  }
  const LoraWorkspace w = lora_workspace(l.T, l.K, l.N, l.r, l.n, true);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (l.r <= 16) return backward<1>(l, ws, w, st);
  if (l.r <= 32) return backward<2>(l, ws, w, st);
  if (l.r <= 64) return backward<4>(l, ws, w, st);
  return backward<8>(l, ws, w, st);
}

}  // namespace nvfp4
