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
// pass and any order is right.  The forward pass of few tokens gathers them by
// adapter instead.
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
constexpr int kNT = 256;       // threads of the tile kernels
constexpr int kCols = 256;     // columns of an expand tile (512 bytes of a row)
constexpr int kFewTokens = 256;   // up to here the tokens are gathered by adapter

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
__device__ __forceinline__ float rest_of(float v, float hi) {
  const float rest = __fsub_rn(v, hi);
  return fabsf(rest) <= 3.402823466e38f ? rest : 0.0f;
}
__device__ __forceinline__ void split_bf16(float v, __nv_bfloat16& hi, __nv_bfloat16& lo) {
  hi = __float2bfloat16_rn(v);
  lo = __float2bfloat16_rn(rest_of(v, __bfloat162float(hi)));
}
// v = hi + mid + lo, all 24 bits
__device__ __forceinline__ void split_bf16(float v, __nv_bfloat16& hi, __nv_bfloat16& mid, __nv_bfloat16& lo) {
  hi = __float2bfloat16_rn(v);
  const float r1 = rest_of(v, __bfloat162float(hi));
  mid = __float2bfloat16_rn(r1);
  lo = __float2bfloat16_rn(__fsub_rn(r1, __bfloat162float(mid)));
}
__device__ __forceinline__ uint32_t pack_bf16(__nv_bfloat16 a, __nv_bfloat16 b) {
  return static_cast<uint32_t>(__bfloat16_as_ushort(a)) | (static_cast<uint32_t>(__bfloat16_as_ushort(b)) << 16);
}

// base + d of eight columns, rounded once to bf16
__device__ __forceinline__ uint4 add_round(const uint4 y, const float* d) {
  const uint32_t yw[4] = {y.x, y.y, y.z, y.w};
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(__fadd_rn(__uint_as_float(yw[j] << 16), d[2 * j]),
                                                   __fadd_rn(__uint_as_float(yw[j] & 0xFFFF0000u), d[2 * j + 1]));
    o[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Column order of a 32-column group in the expand products: thread c of a
// quad owns columns 8c .. 8c + 7 of its rows (16 bytes of bf16) when column
// 8 (n / 2) + 2 q + n % 2 of the group is column n of the group's MMA q.
// Weights are staged in that order, 8 q + n.
__device__ __forceinline__ int mma_slot(int col) {   // column -> slot of its 32-group
  return (col & ~31) + 8 * ((col & 7) >> 1) + 2 * ((col & 31) >> 3) + (col & 1);
}
__device__ __forceinline__ int slot_col(int slot) {   // and back
  const int q = (slot & 31) >> 3, n = slot & 7;
  return (slot & ~31) + 8 * (n >> 1) + 2 * q + (n & 1);
}

// The adapters of a tile of 64 tokens: ids[64] (-1: none) and the list of the
// distinct ones.  All threads call it (at least two warps); ends with a
// barrier.
struct TileAdapters {
  int ids[kRows];
  int list[kRows];
  int head, count;   // distinct ones of the first 32 tokens, and in all
};
__device__ __forceinline__ void tile_adapters(TileAdapters& ta, const AdapterIds& a, int64_t row0, bool report) {
  const int t = threadIdx.x, lane = t & 31;
  int id = -1;
  bool first = false;
  if (t < kRows) {
    id = adapter_of(a, row0 + t, report);
    ta.ids[t] = id;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, id);   // by every lane, whatever its id
    first = id >= 0 && __ffs(same) - 1 == lane;
    if (t < 32) {
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, first);
      if (first) ta.list[__popc(m & ((1u << lane) - 1u))] = id;
      if (t == 0) ta.head = __popc(m);
    }
  }
  __syncthreads();
  if (t >= 32 && t < kRows) {
    const int head = ta.head;
    for (int i = 0; i < head; ++i) first = first && ta.list[i] != id;
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, first);
    __syncwarp();
    if (first) ta.list[head + __popc(m & ((1u << lane) - 1u))] = id;
    if (lane == 0) ta.count = head + __popc(m);
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// shrink: part[split][t][j] = sum over this split's columns of z[t, c] W[j, c]
// TRANS: W is stored [C, r] (c-major), else [r, C].
// A stage is 64 rows x 256 columns: every warp's copy is 512 contiguous bytes
// of one row.  (64 x 64 stages, 128 bytes of a row at a time, ran at 2.9 TB/s
// on 8192 x 14336: scattered short reads.)  Warp w multiplies rows 16 (w % 4)
// over half w / 4 of the stage's columns; the halves are added at the end.
// ---------------------------------------------------------------------------
template <int RP, bool TRANS>
struct ShrinkCfg {
  static constexpr int R = 16 * RP;
  static constexpr int KC = RP == 8 ? 128 : 256;   // columns of a stage (RP = 8: the weights' stage is as large)
  static constexpr int ZB = kRows * (KC + 8) * 2;
  static constexpr int WB = (TRANS ? KC * (R + 8) : R * (KC + 8)) * 2;
  static constexpr int BYTES = 2 * (ZB + WB);
};

template <int RP, bool TRANS>
__global__ void __launch_bounds__(kNT, RP <= 2 ? 2 : 1)
    lora_shrink_kernel(const __nv_bfloat16* __restrict__ z, int64_t ldz, const __nv_bfloat16* __restrict__ W,
                       const AdapterIds a, int64_t C, int r, int64_t per_split, float* __restrict__ part) {
  pdl_entry();
  using S = ShrinkCfg<RP, TRANS>;
  constexpr int R = S::R, KC = S::KC;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ TileAdapters ta;
  const int th = threadIdx.x, lane = th & 31, warp = th >> 5, rg = warp & 3, kh = warp >> 2;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kRows;
  const int64_t c_begin = blockIdx.y * per_split;
  const int64_t c_end = c_begin + per_split < C ? c_begin + per_split : C;
  const int steps = static_cast<int>((c_end - c_begin + KC - 1) / KC);
  tile_adapters(ta, a, row0, blockIdx.y == 0);
  float* mine = part + static_cast<int64_t>(blockIdx.y) * a.T * r;

  auto load = [&](int step, const __nv_bfloat16* w) {
    uint8_t* base = dyn + (step & 1) * (S::ZB + S::WB);
    const int64_t c0 = c_begin + static_cast<int64_t>(step) * KC;
#pragma unroll
    for (int i = 0; i < kRows * KC / 8 / kNT; ++i) {
      const int k = th + kNT * i, row = k / (KC / 8), ch = k % (KC / 8);
      const bool ok = c0 + 8 * ch < c_end && ta.ids[row] >= 0;
      copy16(base + row * (KC + 8) * 2 + 16 * ch, ok ? z + (row0 + row) * ldz + c0 + 8 * ch : z, ok);
    }
    uint8_t* wb = base + S::ZB;
    if constexpr (!TRANS) {
#pragma unroll
      for (int i = 0; i < (R * KC / 8 + kNT - 1) / kNT; ++i) {
        const int k = th + kNT * i, j = k / (KC / 8), ch = k % (KC / 8);
        const bool ok = j < r && c0 + 8 * ch < c_end;
        copy16(wb + j * (KC + 8) * 2 + 16 * ch, ok ? w + j * C + c0 + 8 * ch : w, ok);
      }
    } else {
#pragma unroll
      for (int i = 0; i < (KC * R / 8 + kNT - 1) / kNT; ++i) {
        const int k = th + kNT * i, c = k / (R / 8), ch = k % (R / 8);
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
    load(0, w);
    for (int s = 0; s < steps; ++s) {
      if (s + 1 < steps) load(s + 1, w);
      else cp_async_commit();
      cp_async_wait<1>();
      __syncthreads();
      const uint8_t* base = dyn + (s & 1) * (S::ZB + S::WB);
      const __nv_bfloat16* zs = reinterpret_cast<const __nv_bfloat16*>(base);
      const __nv_bfloat16* ws = reinterpret_cast<const __nv_bfloat16*>(base + S::ZB);
      // this stage's sums start from zero and are added to the running ones:
      // the tensor core truncates as it adds, so its runs are kept short
      float acc[2 * RP][4];
#pragma unroll
      for (int i = 0; i < 2 * RP; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
#pragma unroll
      for (int k8 = 0; k8 < KC / 2; k8 += 16) {
        const int kk = kh * (KC / 2) + k8;
        uint32_t af[4];
        ldsm4(af, zs + (16 * rg + (lane & 15)) * (KC + 8) + kk + (lane >> 4) * 8);
#pragma unroll
        for (int p = 0; p < RP; ++p) {
          uint32_t bf[4];
          if constexpr (!TRANS)
            ldsm4(bf, ws + (16 * p + (lane & 7) + ((lane >> 4) << 3)) * (KC + 8) + kk + ((lane >> 3) & 1) * 8);
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
      __syncthreads();   // this buffer is refilled in the next round
    }
    // add the second half's sums (the ring is free: every copy has landed)
    float* other = reinterpret_cast<float*>(dyn);
    if (kh == 1) {
#pragma unroll
      for (int i = 0; i < 2 * RP; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) other[((rg * 2 * RP + i) * 4 + e) * 32 + lane] = sum[i][e];
    }
    __syncthreads();
    if (kh == 0) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int row = 16 * rg + (lane >> 2) + 8 * half;
        if (ta.ids[row] == id) {
#pragma unroll
          for (int i = 0; i < 2 * RP; ++i) {
            const int j = 8 * i + 2 * (lane & 3);
            const float* o = other + ((rg * 2 * RP + i) * 4 + 2 * half) * 32 + lane;
            if (j < r)
              *reinterpret_cast<float2*>(mine + (row0 + row) * r + j) =
                  make_float2(__fadd_rn(sum[i][2 * half], o[0]), __fadd_rn(sum[i][2 * half + 1], o[32]));
          }
        }
      }
    }
    __syncthreads();   // before the next adapter's copies
  }
  // tokens without an adapter
  for (int k = th; k < kRows * r; k += kNT) {
    const int row = k / r;
    if (ta.ids[row] < 0 && row0 + row < a.T) mine[(row0 + row) * r + (k - row * r)] = 0.0f;
  }
}

// ---------------------------------------------------------------------------
// expand: out[t, c] = base[t, c] + s_a sum_j w[t, j] W[c, j], w = sum of the
// partials; w itself goes to w_out.  TRANS: W is stored [r, C], else [C, r].
// A CTA takes 64 tokens and `per_cta` tiles of 256 columns; warp w rows
// 16 (w % 4), columns 128 (w / 4).  A thread's products land on the 16 bytes
// of base it has loaded (see mma_slot), so neither base nor result passes
// through shared memory.
// ---------------------------------------------------------------------------
template <int RP>
struct ExpandCfg {
  static constexpr int R = 16 * RP;
  static constexpr int HB = kRows * (R + 8) * 2;
  static constexpr int WB = kCols * (R + 8) * 2;
  static constexpr int BYTES = 2 * HB + WB;
};

template <int RP, bool TRANS>
__global__ void __launch_bounds__(kNT, RP <= 4 ? 3 : 2)
    lora_expand_kernel(const float* __restrict__ part, int splits, const __nv_bfloat16* __restrict__ W,
                       const float* __restrict__ scaling, const AdapterIds a, int64_t C, int r, int per_cta,
                       const __nv_bfloat16* in, int64_t ldi, __nv_bfloat16* out, int64_t ldo,
                       float* __restrict__ w_out) {
  pdl_entry();
  using S = ExpandCfg<RP>;
  constexpr int R = S::R;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ TileAdapters ta;
  __nv_bfloat16* hh = reinterpret_cast<__nv_bfloat16*>(dyn);
  __nv_bfloat16* hl = reinterpret_cast<__nv_bfloat16*>(dyn + S::HB);
  __nv_bfloat16* ws = reinterpret_cast<__nv_bfloat16*>(dyn + 2 * S::HB);
  const int th = threadIdx.x, lane = th & 31, warp = th >> 5, rg = warp & 3, ch = warp >> 2;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kRows;
  const int64_t ta_row = row0 + 16 * rg + (lane >> 2);   // this thread's rows: ta_row and ta_row + 8
  const int piece = lane & 3;
  tile_adapters(ta, a, row0, false);
  // the sum of the partials, in their order
  for (int k = th; k < kRows * R; k += kNT) {
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
  const int id_lo = ta.ids[16 * rg + (lane >> 2)], id_hi = ta.ids[16 * rg + (lane >> 2) + 8];

  for (int i = 0; i < per_cta; ++i) {
    const int64_t c0 = (static_cast<int64_t>(blockIdx.y) * per_cta + i) * kCols;
    if (c0 >= C) break;
    const int64_t c_mine = c0 + 128 * ch + 8 * piece;   // + 32 per column group
    uint4 y[4][2];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int64_t t = ta_row + 8 * half, c = c_mine + 32 * q;
        y[q][half] = make_uint4(0u, 0u, 0u, 0u);
        if (in && c < C && t < a.T) y[q][half] = __ldcs(reinterpret_cast<const uint4*>(in + t * ldi + c));
      }
    }
    for (int u = 0; u < ta.count; ++u) {
      const int id = ta.list[u];
      const __nv_bfloat16* w = W + static_cast<int64_t>(id) * r * C;
      __syncthreads();   // the previous weights have been read
      if constexpr (!TRANS) {
        for (int k = th; k < kCols * (R / 8); k += kNT) {
          const int c = k / (R / 8), c8 = k % (R / 8);
          const bool ok = c0 + c < C && 8 * c8 < r;
          copy16(ws + mma_slot(c) * (R + 8) + 8 * c8, ok ? w + (c0 + c) * r + 8 * c8 : w, ok);
        }
        cp_async_commit();
        cp_async_wait<0>();
      } else {
        // transposed on the way: two rows j, j + 1 of eight columns give
        // eight words (j, j + 1) of those columns
        for (int k = th; k < (R / 2) * (kCols / 8); k += kNT) {
          const int j = 2 * (k / (kCols / 8)), c8 = k % (kCols / 8);
          uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
          if (j < r && c0 + 8 * c8 < C) {   // r is even
            lo = __ldg(reinterpret_cast<const uint4*>(w + j * C + c0 + 8 * c8));
            hi = __ldg(reinterpret_cast<const uint4*>(w + (j + 1) * C + c0 + 8 * c8));
          }
          const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, h[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<uint32_t*>(ws + mma_slot(8 * c8 + e) * (R + 8) + j) =
                __byte_perm(l[e >> 1], h[e >> 1], (e & 1) ? 0x7632 : 0x5410);
        }
      }
      __syncthreads();
      const bool lo_mine = id_lo == id, hi_mine = id_hi == id;
      if (!__any_sync(0xFFFFFFFFu, lo_mine || hi_mine)) continue;
      const float s = __ldg(scaling + id);
#pragma unroll
      for (int q = 0; q < 4; ++q) {   // 32 columns each
        float acc[4][4] = {};
#pragma unroll
        for (int kk = 0; kk < R; kk += 16) {
          uint32_t ah[4], al[4], b0[4], b1[4];
          ldsm4(ah, hh + (16 * rg + (lane & 15)) * (R + 8) + kk + (lane >> 4) * 8);
          ldsm4(al, hl + (16 * rg + (lane & 15)) * (R + 8) + kk + (lane >> 4) * 8);
          const __nv_bfloat16* wq = ws + (128 * ch + 32 * q + (lane & 7) + ((lane >> 4) << 3)) * (R + 8) + kk + ((lane >> 3) & 1) * 8;
          ldsm4(b0, wq);
          ldsm4(b1, wq + 16 * (R + 8));
          mma16(acc[0], al, b0);
          mma16(acc[1], al, b0 + 2);
          mma16(acc[2], al, b1);
          mma16(acc[3], al, b1 + 2);
          mma16(acc[0], ah, b0);
          mma16(acc[1], ah, b0 + 2);
          mma16(acc[2], ah, b1);
          mma16(acc[3], ah, b1 + 2);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // a token without an adapter keeps the base's bits (a NaN's payload, a zero's sign)
          if (half ? hi_mine : lo_mine) {
            float d[8];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              d[2 * m] = __fmul_rn(s, acc[m][2 * half]);
              d[2 * m + 1] = __fmul_rn(s, acc[m][2 * half + 1]);
            }
            y[q][half] = add_round(y[q][half], d);
          }
        }
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int64_t t = ta_row + 8 * half, c = c_mine + 32 * q;
        if (c < C && t < a.T) __stcs(reinterpret_cast<uint4*>(out + t * ldo + c), y[q][half]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Few tokens (a decode step): the tokens of one adapter are gathered, 16 at a
// time, wherever they stand in the batch, so that an adapter's weights are
// read once per 16 of its tokens.  The operands go from global memory straight
// into the MMA registers: with the contraction index permuted alike in both
// operands, a thread's 16 (or 8) contiguous bytes are its share of the
// fragments.
// ---------------------------------------------------------------------------
struct Unit {
  int ids[kFewTokens];
  int rank[kFewTokens];          // how many earlier tokens have the same id
  uint32_t leaders[kFewTokens / 32];
  int id, first;                 // the unit's adapter and the rank of its first token
  int member[16];                // its tokens, -1: none
};

// Unit `u` of the batch (a unit: up to 16 tokens of one adapter, or of none);
// false if there are fewer units.  All 128 threads; ends with a barrier.
__device__ __forceinline__ bool find_unit(Unit& un, const AdapterIds& a, int u, bool report) {
  const int th = threadIdx.x, lane = th & 31, T = static_cast<int>(a.T);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = th + 128 * i;
    un.ids[t] = t < T ? adapter_of(a, t, report) : -2;
  }
  if (th < 16) un.member[th] = -1;
  if (th == 0) un.id = -2;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = th + 128 * i, id = un.ids[t];
    int rank = 0;
    if (t - lane < T) {   // uniform over the warp
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, id);
      rank = __popc(same & ((1u << lane) - 1u));
      for (int j = 0; j < t - lane; j += 4) {
        const int4 v = *reinterpret_cast<const int4*>(&un.ids[j]);
        rank += (v.x == id) + (v.y == id) + (v.z == id) + (v.w == id);
      }
    }
    un.rank[t] = rank;
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, t < T && (rank & 15) == 0);
    if (lane == 0) un.leaders[t >> 5] = m;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = th + 128 * i;
    const uint32_t m = un.leaders[t >> 5];
    if (m >> lane & 1u) {
      int before = __popc(m & ((1u << lane) - 1u));
      for (int w = 0; w < (t >> 5); ++w) before += __popc(un.leaders[w]);
      if (before == u) {
        un.id = un.ids[t];
        un.first = un.rank[t];
      }
    }
  }
  __syncthreads();
  if (un.id == -2) return false;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = th + 128 * i;
    const int at = un.rank[t] - un.first;
    if (t < T && un.ids[t] == un.id && at >= 0 && at < 16) un.member[at] = t;
  }
  __syncthreads();
  return true;
}

__device__ __forceinline__ uint4 load16(const __nv_bfloat16* p, bool ok) {
  return ok ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0u, 0u, 0u, 0u);
}

// grid: split, unit.  Warp w takes the 32-column blocks w, w + 4, .. of the
// split; thread c of a quad holds columns 8c .. 8c + 7 of a block.
template <int RP>
__global__ void __launch_bounds__(128) lora_shrink_few_kernel(const __nv_bfloat16* __restrict__ z, int64_t ldz,
                                                              const __nv_bfloat16* __restrict__ W, const AdapterIds a,
                                                              int64_t C, int r, int64_t per_split,
                                                              float* __restrict__ part) {
  pdl_entry();
  constexpr int R = 16 * RP;
  __shared__ __align__(16) Unit un;
  __shared__ float sums[4][16][R + 4];
  const int th = threadIdx.x, lane = th & 31, warp = th >> 5, g = lane >> 2, c = lane & 3;
  if (!find_unit(un, a, blockIdx.y, blockIdx.x == 0)) return;
  float* mine = part + static_cast<int64_t>(blockIdx.x) * a.T * r;
  if (un.id < 0) {
    for (int k = th; k < 16 * r; k += 128)
      if (un.member[k / r] >= 0) mine[static_cast<int64_t>(un.member[k / r]) * r + k % r] = 0.0f;
    return;
  }
  const __nv_bfloat16* w = W + static_cast<int64_t>(un.id) * r * C;
  const int t0 = un.member[g], t1 = un.member[g + 8];
  const int64_t c_begin = blockIdx.x * per_split, c_end = min(c_begin + per_split, C);
  float acc[2 * RP][4] = {};
  for (int64_t c0 = c_begin + 32 * warp; c0 < c_end; c0 += 128) {
    const int64_t cc = c0 + 8 * c;
    const bool ok = cc < c_end;
    const uint4 a0 = load16(z + t0 * ldz + cc, ok && t0 >= 0), a1 = load16(z + t1 * ldz + cc, ok && t1 >= 0);
    uint4 b[2 * RP];
#pragma unroll
    for (int i = 0; i < 2 * RP; ++i) b[i] = load16(w + (8 * i + g) * C + cc, ok && 8 * i + g < r);
    const uint32_t f0[4] = {a0.x, a1.x, a0.y, a1.y}, f1[4] = {a0.z, a1.z, a0.w, a1.w};
    float run[2 * RP][4] = {};   // short runs on the tensor core, fp32 sums outside
#pragma unroll
    for (int i = 0; i < 2 * RP; ++i) {
      const uint32_t b0[2] = {b[i].x, b[i].y}, b1[2] = {b[i].z, b[i].w};
      mma16(run[i], f0, b0);
      mma16(run[i], f1, b1);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = __fadd_rn(acc[i][e], run[i][e]);
    }
  }
#pragma unroll
  for (int i = 0; i < 2 * RP; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) sums[warp][g + 8 * (e >> 1)][8 * i + 2 * c + (e & 1)] = acc[i][e];
  __syncthreads();
  for (int k = th; k < 16 * r; k += 128) {
    const int row = k / r, j = k - row * r, t = un.member[row];
    if (t >= 0)
      mine[static_cast<int64_t>(t) * r + j] = __fadd_rn(__fadd_rn(sums[0][row][j], sums[1][row][j]),
                                                        __fadd_rn(sums[2][row][j], sums[3][row][j]));
  }
}

// grid: 512 columns, unit.  Warp w takes 128 of the columns.
constexpr int kFewCols = 512;

template <int RP>
__global__ void __launch_bounds__(128) lora_expand_few_kernel(const float* __restrict__ part, int splits,
                                                              const __nv_bfloat16* __restrict__ W,
                                                              const float* __restrict__ scaling, const AdapterIds a,
                                                              int64_t C, int r, const __nv_bfloat16* in, int64_t ldi,
                                                              __nv_bfloat16* out, int64_t ldo, float* __restrict__ w_out) {
  pdl_entry();
  constexpr int R = 16 * RP;
  __shared__ __align__(16) Unit un;
  __shared__ __align__(16) float hs[16][R + 4];   // read as float4
  const int th = threadIdx.x, lane = th & 31, warp = th >> 5, g = lane >> 2, c = lane & 3;
  if (!find_unit(un, a, blockIdx.y, false)) return;
  const int64_t c_warp = static_cast<int64_t>(blockIdx.x) * kFewCols + 128 * warp;
  const int t0 = un.member[g], t1 = un.member[g + 8];
  uint4 y[4][2];
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int t = half ? t1 : t0;
      const int64_t col = c_warp + 32 * q + 8 * c;
      y[q][half] = make_uint4(0u, 0u, 0u, 0u);
      if (in && t >= 0 && col < C) y[q][half] = __ldcg(reinterpret_cast<const uint4*>(in + t * ldi + col));
    }
  for (int k = th; k < 16 * R; k += 128) {
    const int row = k / R, j = k % R, t = un.member[row];
    float v = 0.0f;
    if (t >= 0 && j < r) {
      const int64_t at = static_cast<int64_t>(t) * r + j;
      for (int s = 0; s < splits; ++s) v = __fadd_rn(v, __ldcg(part + s * a.T * r + at));
      if (w_out && blockIdx.x == 0) w_out[at] = v;
    }
    hs[row][j] = v;
  }
  __syncthreads();
  if (un.id >= 0) {
    const __nv_bfloat16* w = W + static_cast<int64_t>(un.id) * r * C;
    const float s = __ldg(scaling + un.id);
    // thread c of a quad holds ranks 4c .. 4c + 3 of each 16
    uint32_t ah[RP][4], al[RP][4];
#pragma unroll
    for (int p = 0; p < RP; ++p)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float4 v = *reinterpret_cast<const float4*>(&hs[g + 8 * half][16 * p + 4 * c]);
        const float vv[4] = {v.x, v.y, v.z, v.w};
        __nv_bfloat16 h[4], l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split_bf16(vv[e], h[e], l[e]);
        ah[p][half] = pack_bf16(h[0], h[1]);
        ah[p][2 + half] = pack_bf16(h[2], h[3]);
        al[p][half] = pack_bf16(l[0], l[1]);
        al[p][2 + half] = pack_bf16(l[2], l[3]);
      }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float acc[4][4] = {};
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int64_t col = c_warp + 32 * q + slot_col(8 * m + g);
        uint2 b[RP];
#pragma unroll
        for (int p = 0; p < RP; ++p)
          b[p] = (col < C && 16 * p + 4 * c < r) ? __ldg(reinterpret_cast<const uint2*>(w + col * r + 16 * p + 4 * c))
                                                  : make_uint2(0u, 0u);
#pragma unroll
        for (int p = 0; p < RP; ++p) {
          const uint32_t bb[2] = {b[p].x, b[p].y};
          mma16(acc[m], al[p], bb);
          mma16(acc[m], ah[p], bb);
        }
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float d[8];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          d[2 * m] = __fmul_rn(s, acc[m][2 * half]);
          d[2 * m + 1] = __fmul_rn(s, acc[m][2 * half + 1]);
        }
        y[q][half] = add_round(y[q][half], d);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int t = half ? t1 : t0;
      const int64_t col = c_warp + 32 * q + 8 * c;
      if (t >= 0 && col < C) *reinterpret_cast<uint4*>(out + t * ldo + col) = y[q][half];
    }
}

// ---------------------------------------------------------------------------
// outer: P[a][j, c] = s_a sum_{ids[t] = a} w[t, j] z[t, c] over a range of
// row tiles.  Rows of other adapters are not read (their slots are zero, so a
// NaN there reaches nothing).  Two products share a launch: dA (z = x, w = g,
// stored [r, C]) and dB (z = dy, w = h, stored [C, r]).
// grid: column tiles of both products, adapter, split of the rows.
// TERMS: bf16 numbers that w enters as: 3 (all of fp32) for fp32 gradients,
// 2 (2^-17) for bf16 ones.
// ---------------------------------------------------------------------------
struct OuterProduct {
  const float* w;
  const __nv_bfloat16* z;
  int64_t ldz, C;
  void* dst;
  float* part;
  int tiles;         // column tiles, 0: this product is not asked for
  int cols_first;    // stored [C, r]
};
struct OuterArgs {
  OuterProduct p[2];
  const float* scaling;
  AdapterIds a;
  int r, fp32;
  int32_t* used;     // [adapter][split][column tile of both]: the split saw a token
};

template <int RP, int TERMS>
struct OuterCfg {
  static constexpr int R = 16 * RP;
  static constexpr int NQ = RP <= 2 ? 2 : 1;          // 16-column groups of a warp
  static constexpr int COLS = 8 * 16 * NQ;            // columns of a tile
  static constexpr int ZB = kRows * (COLS + 8) * 2;
  static constexpr int FB = kRows * R * 4;            // w as it is in memory
  static constexpr int HB = kRows * (R + 8) * 2;
  static constexpr int STAGES = 2;
  static constexpr int BYTES = STAGES * (ZB + FB) + TERMS * HB;
};
constexpr int kWindow = 2048;   // rows whose ids a CTA looks at together

__device__ __forceinline__ void store_out(void* dst, int64_t at, float v, bool fp32) {
  if (fp32) static_cast<float*>(dst)[at] = v;
  else static_cast<__nv_bfloat16*>(dst)[at] = __float2bfloat16_rn(v);
}

template <int RP, int TERMS>
__global__ void __launch_bounds__(kNT, RP <= 2 ? 2 : 1) lora_outer_kernel(const OuterArgs o) {
  pdl_entry();
  using S = OuterCfg<RP, TERMS>;
  constexpr int R = S::R, COLS = S::COLS, NQ = S::NQ;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ __align__(16) int ids[kWindow];
  __shared__ int list[kWindow / kRows];
  __shared__ int listed;
  const int th = threadIdx.x, lane = th & 31, warp = th >> 5;
  const bool second = static_cast<int>(blockIdx.x) >= o.p[0].tiles;
  const OuterProduct& p = o.p[second ? 1 : 0];
  const int64_t c0 = static_cast<int64_t>(blockIdx.x - (second ? o.p[0].tiles : 0)) * COLS;
  const int id = blockIdx.y, splits = gridDim.z, split = blockIdx.z, r = o.r;
  const int tiles = static_cast<int>((o.a.T + kRows - 1) / kRows);
  const int first = static_cast<int>(static_cast<int64_t>(tiles) * split / splits);
  const int last = static_cast<int>(static_cast<int64_t>(tiles) * (split + 1) / splits);
  __nv_bfloat16* wb = reinterpret_cast<__nv_bfloat16*>(dyn + S::STAGES * (S::ZB + S::FB));

  float sum[RP][2 * NQ][4];
#pragma unroll
  for (int m = 0; m < RP; ++m)
#pragma unroll
    for (int q = 0; q < 2 * NQ; ++q) sum[m][q][0] = sum[m][q][1] = sum[m][q][2] = sum[m][q][3] = 0.0f;
  bool any = false;

  for (int base = first; base < last; base += kWindow / kRows) {
    const int n_tiles = min(kWindow / kRows, last - base);
    const int64_t row_base = static_cast<int64_t>(base) * kRows;
    __syncthreads();   // the previous window's ids and list have been read
    for (int k = th; k < n_tiles * kRows; k += kNT) ids[k] = adapter_of(o.a, row_base + k, false);
    __syncthreads();
    if (warp == 0) {   // the tiles that hold a token of this adapter
      bool mine = false;
      if (lane < n_tiles)
        for (int k = 0; k < kRows / 4; ++k) {
          // lanes start at different places: no bank conflicts
          const int4 v = *reinterpret_cast<const int4*>(&ids[lane * kRows + 4 * ((k + lane) % (kRows / 4))]);
          mine |= v.x == id || v.y == id || v.z == id || v.w == id;
        }
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, mine);
      if (mine) list[__popc(m & ((1u << lane) - 1u))] = lane;
      if (lane == 0) listed = __popc(m);
    }
    __syncthreads();
    const int count = listed;
    any |= count > 0;

    auto load = [&](int k) {
      const int tile = list[k];
      uint8_t* st = dyn + (k & 1) * (S::ZB + S::FB);
      const int64_t row0 = row_base + static_cast<int64_t>(tile) * kRows;
#pragma unroll
      for (int i = 0; i < kRows * COLS / 8 / kNT; ++i) {
        const int e = th + kNT * i, row = e / (COLS / 8), ch = e % (COLS / 8);
        const bool ok = ids[tile * kRows + row] == id && c0 + 8 * ch < p.C;
        copy16(st + row * (COLS + 8) * 2 + 16 * ch, ok ? p.z + (row0 + row) * p.ldz + c0 + 8 * ch : p.z, ok);
      }
      for (int e = th; e < kRows * (R / 4); e += kNT) {
        const int row = e / (R / 4), j4 = e % (R / 4);
        const bool ok = ids[tile * kRows + row] == id && 4 * j4 < r;
        copy16(st + S::ZB + row * R * 4 + 16 * j4, ok ? p.w + (row0 + row) * r + 4 * j4 : p.w, ok);
      }
      cp_async_commit();
    };
    if (count > 0) load(0);
    for (int k = 0; k < count; ++k) {
      if (k + 1 < count) load(k + 1);
      else cp_async_commit();
      cp_async_wait<1>();
      __syncthreads();
      const uint8_t* st = dyn + (k & 1) * (S::ZB + S::FB);
      const float* wf = reinterpret_cast<const float*>(st + S::ZB);
      for (int e = th; e < kRows * R / 2; e += kNT) {   // pairs of ranks
        const int row = e / (R / 2), j = 2 * (e % (R / 2));
        const float2 v = *reinterpret_cast<const float2*>(wf + row * R + j);
        __nv_bfloat16 s0[3], s1[3];
        if constexpr (TERMS == 3) {
          split_bf16(v.x, s0[0], s0[1], s0[2]);
          split_bf16(v.y, s1[0], s1[1], s1[2]);
        } else {
          split_bf16(v.x, s0[0], s0[1]);
          split_bf16(v.y, s1[0], s1[1]);
        }
#pragma unroll
        for (int x = 0; x < TERMS; ++x)
          *reinterpret_cast<uint32_t*>(wb + x * (S::HB / 2) + row * (R + 8) + j) = pack_bf16(s0[x], s1[x]);
      }
      __syncthreads();
      const __nv_bfloat16* zs = reinterpret_cast<const __nv_bfloat16*>(st);
#pragma unroll
      for (int m = 0; m < RP; ++m) {
        float acc[2 * NQ][4];
#pragma unroll
        for (int q = 0; q < 2 * NQ; ++q) acc[q][0] = acc[q][1] = acc[q][2] = acc[q][3] = 0.0f;
#pragma unroll
        for (int kk = 0; kk < kRows; kk += 16) {
          uint32_t af[TERMS][4], bf[NQ][4];
          const int arow = kk + (lane & 7) + ((lane >> 4) << 3), acol = 16 * m + ((lane >> 3) & 1) * 8;
#pragma unroll
          for (int x = 0; x < TERMS; ++x) ldsm4_t(af[x], wb + x * (S::HB / 2) + arow * (R + 8) + acol);
#pragma unroll
          for (int q = 0; q < NQ; ++q)
            ldsm4_t(bf[q], zs + (kk + (lane & 7) + ((lane >> 3) & 1) * 8) * (COLS + 8) + 16 * (NQ * warp + q) + (lane >> 4) * 8);
#pragma unroll
          for (int x = TERMS - 1; x >= 0; --x)
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
              mma16(acc[2 * q], af[x], bf[q]);
              mma16(acc[2 * q + 1], af[x], bf[q] + 2);
            }
        }
#pragma unroll
        for (int q = 0; q < 2 * NQ; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[m][q][e] = __fadd_rn(sum[m][q][e], acc[q][e]);
      }
      __syncthreads();   // this stage and wb are rewritten in the next round
    }
    cp_async_wait<0>();
  }
  const bool direct = splits == 1;
  if (!direct) {
    if (th == 0) o.used[(static_cast<int64_t>(id) * splits + split) * gridDim.x + blockIdx.x] = any ? 1 : 0;
    if (!any) return;
  }
  const float s = direct ? __ldg(o.scaling + id) : 1.0f;   // with splits the sum is scaled once, at the end
#pragma unroll
  for (int m = 0; m < RP; ++m)
#pragma unroll
    for (int q = 0; q < 2 * NQ; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = 16 * m + (lane >> 2) + 8 * (e >> 1);
        const int64_t c = c0 + 16 * NQ * warp + 8 * q + 2 * (lane & 3) + (e & 1);
        if (j < r && c < p.C) {
          const int64_t at = p.cols_first ? (static_cast<int64_t>(id) * p.C + c) * r + j : (static_cast<int64_t>(id) * r + j) * p.C + c;
          if (direct) store_out(p.dst, at, __fmul_rn(s, sum[m][q][e]), o.fp32);
          else p.part[static_cast<int64_t>(split) * o.a.n * r * p.C + at] = sum[m][q][e];
        }
      }
}

// Sum of the splits' partials, in their order, those that saw a token; four
// elements per thread.
__global__ void __launch_bounds__(256) lora_outer_sum_kernel(const OuterArgs o, int splits, int cols) {
  pdl_entry();
  const int all_tiles = o.p[0].tiles + o.p[1].tiles;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const OuterProduct& p = o.p[which];
    if (!p.tiles) continue;
    const int64_t per = o.r * p.C, total = per * o.a.n;
    for (int64_t k = 4 * (blockIdx.x * 256ll + threadIdx.x); k < total; k += 4 * (gridDim.x * 256ll)) {
      // r and C are multiples of 8: four neighbours share an adapter and a column tile
      const int id = static_cast<int>(k / per);
      const int64_t in = k - id * per, c = p.cols_first ? in / o.r : in % p.C;
      const int32_t* used = o.used + static_cast<int64_t>(id) * splits * all_tiles + (which ? o.p[0].tiles : 0) + c / cols;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int s = 0; s < splits; ++s)
        if (__ldcg(used + s * all_tiles)) {
          const float4 q = __ldcg(reinterpret_cast<const float4*>(p.part + s * total + k));
          v = make_float4(__fadd_rn(v.x, q.x), __fadd_rn(v.y, q.y), __fadd_rn(v.z, q.z), __fadd_rn(v.w, q.w));
        }
      const float sc = __ldg(o.scaling + id);
      v = make_float4(__fmul_rn(sc, v.x), __fmul_rn(sc, v.y), __fmul_rn(sc, v.z), __fmul_rn(sc, v.w));
      if (o.fp32) {
        *reinterpret_cast<float4*>(static_cast<float*>(p.dst) + k) = v;
      } else {
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.dst) + k) =
            make_uint2(pack_bf16(__float2bfloat16_rn(v.x), __float2bfloat16_rn(v.y)),
                       pack_bf16(__float2bfloat16_rn(v.z), __float2bfloat16_rn(v.w)));
      }
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Units that T tokens and n adapters (and "none") can make.
int64_t most_units(int64_t T, int64_t n) { return std::min<int64_t>(n + 1, T) + T / 16; }

// Columns per shrink split: one wave of two CTAs per SM, whole stages; with
// few tokens about eight small CTAs per SM, whole 128-column rounds.
int64_t shrink_per_split(int64_t T, int64_t C, int64_t n) {
  const bool few = T <= kFewTokens;
  const int64_t rows = few ? most_units(T, n) : ceil_div(T, kRows);
  const int64_t step = few ? 128 : 256;
  const int64_t splits = std::max<int64_t>(1, std::min<int64_t>(few ? 16 : 32, (few ? 8 : 2) * sm_count() / rows));
  return ceil_div(ceil_div(C, splits), step) * step;
}
int shrink_splits(int64_t T, int64_t C, int64_t n) { return static_cast<int>(ceil_div(C, shrink_per_split(T, C, n))); }
// The backward pass shrinks with the tile kernel for any T.
int64_t tile_per_split(int64_t T, int64_t C) {
  const int64_t splits = std::max<int64_t>(1, std::min<int64_t>(32, 2 * sm_count() / ceil_div(T, kRows)));
  return ceil_div(ceil_div(C, splits), 256) * 256;
}
int tile_splits(int64_t T, int64_t C) { return static_cast<int>(ceil_div(C, tile_per_split(T, C))); }

int outer_cols(int64_t r) { return r <= 32 ? 256 : 128; }
// Row ranges of the outer products: at most 2048 tokens each (an adapter may
// own all of them), unless that makes more than 8.
int outer_splits(int64_t T) { return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(8, ceil_div(T, kWindow)))); }

// Parts of the workspace, in 16-byte steps.
struct LoraWorkspace {
  size_t part, sum, outer_a, outer_b, used, total;
};
size_t up16(size_t v) { return (v + 15) & ~static_cast<size_t>(15); }
LoraWorkspace lora_workspace(int64_t T, int64_t K, int64_t N, int64_t r, int64_t n, bool backward) {
  LoraWorkspace w{};
  w.part = 0;
  w.sum = up16(static_cast<size_t>(backward ? tile_splits(T, N) : shrink_splits(T, K, n)) * T * r * 4);
  w.total = w.sum;
  if (backward) {
    w.outer_a = w.sum + up16(static_cast<size_t>(T) * r * 4);
    const int s = outer_splits(T);
    const size_t each = s > 1 ? static_cast<size_t>(s) * n * r * 4 : 0;
    w.outer_b = w.outer_a + up16(each * K);
    w.used = w.outer_b + up16(each * N);
    w.total = w.used + up16(static_cast<size_t>(s) * n * 4 * (ceil_div(K, outer_cols(r)) + ceil_div(N, outer_cols(r))));
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
  constexpr int smem = ShrinkCfg<RP, TRANS>::BYTES;
  static bool done[64] = {false};
  cudaError_t e = allow_smem(fn, smem, done);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(ceil_div(a.T, kRows)), static_cast<unsigned>(tile_splits(a.T, C)));
  e = launch_k(fn, grid, dim3(kNT), smem, st, 1u, z, ldz, W, a, C, r, tile_per_split(a.T, C), part);
  note_launch();
  return e;
}

template <int RP, bool TRANS>
cudaError_t expand(const float* part, int splits, const __nv_bfloat16* W, const float* scaling, const AdapterIds& a,
                   int64_t C, int r, const __nv_bfloat16* in, int64_t ldi, __nv_bfloat16* out, int64_t ldo, float* w_out,
                   cudaStream_t st) {
  auto fn = lora_expand_kernel<RP, TRANS>;
  constexpr int smem = ExpandCfg<RP>::BYTES;
  static bool done[64] = {false};
  cudaError_t e = allow_smem(fn, smem, done);
  if (e != cudaSuccess) return e;
  // up to four column tiles share one sum of the partials, as long as the
  // grid still fills the GPU a few times over
  const int64_t rows = ceil_div(a.T, kRows), cols = ceil_div(C, kCols);
  const int per = out ? static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(4, rows * cols / (12 * sm_count())))) : 1;
  const dim3 grid(static_cast<unsigned>(rows), out ? static_cast<unsigned>(ceil_div(cols, per)) : 1u);
  e = launch_k(fn, grid, dim3(kNT), smem, st, 1u, part, splits, W, scaling, a, C, r, per, in, ldi, out, ldo, w_out);
  note_launch();
  return e;
}

template <int RP, int TERMS>
cudaError_t outer(const OuterArgs& o, cudaStream_t st) {
  auto fn = lora_outer_kernel<RP, TERMS>;
  constexpr int smem = OuterCfg<RP, TERMS>::BYTES;
  static bool done[64] = {false};
  cudaError_t e = allow_smem(fn, smem, done);
  if (e != cudaSuccess) return e;
  const int splits = outer_splits(o.a.T);
  const dim3 grid(static_cast<unsigned>(o.p[0].tiles + o.p[1].tiles), static_cast<unsigned>(o.a.n), static_cast<unsigned>(splits));
  e = launch_k(fn, grid, dim3(kNT), smem, st, 1u, o);
  note_launch();
  if (e != cudaSuccess || splits == 1) return e;
  const int64_t most = static_cast<int64_t>(o.a.n) * o.r * std::max(o.p[0].tiles ? o.p[0].C : 0, o.p[1].tiles ? o.p[1].C : 0);
  const int64_t blocks = std::min<int64_t>(ceil_div(most, 1024), 8 * sm_count());
  e = launch_k(lora_outer_sum_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, 1u, o, splits, OuterCfg<RP, TERMS>::COLS);
  note_launch();
  return e;
}

template <int RP>
cudaError_t forward(const LoraArgs& l, float* part, cudaStream_t st) {
  const AdapterIds a{l.ids, l.T, static_cast<int>(l.n), l.status};
  const int r = static_cast<int>(l.r);
  if (l.T > kFewTokens) {
    const cudaError_t e = shrink<RP, false>(l.x, l.ldx, l.A, a, l.K, r, part, st);
    if (e != cudaSuccess) return e;
    return expand<RP, false>(part, tile_splits(l.T, l.K), l.B, l.scaling, a, l.N, r, l.in, l.ldi, l.out, l.ldo, l.h, st);
  }
  const unsigned units = static_cast<unsigned>(most_units(l.T, l.n));
  const int splits = shrink_splits(l.T, l.K, l.n);
  cudaError_t e = launch_k(lora_shrink_few_kernel<RP>, dim3(static_cast<unsigned>(splits), units), dim3(128), 0, st, 1u,
                           l.x, l.ldx, l.A, a, l.K, r, shrink_per_split(l.T, l.K, l.n), part);
  note_launch();
  if (e != cudaSuccess) return e;
  e = launch_k(lora_expand_few_kernel<RP>, dim3(static_cast<unsigned>(ceil_div(l.N, kFewCols)), units), dim3(128), 0, st,
               1u, part, splits, l.B, l.scaling, a, l.N, r, l.in, l.ldi, l.out, l.ldo, l.h);
  note_launch();
  return e;
}

template <int RP>
cudaError_t backward(const LoraArgs& l, uint8_t* ws, const LoraWorkspace& w, cudaStream_t st) {
  const AdapterIds a{l.ids, l.T, static_cast<int>(l.n), l.status};
  const int r = static_cast<int>(l.r);
  float* part = reinterpret_cast<float*>(ws + w.part);
  float* g = reinterpret_cast<float*>(ws + w.sum);
  if (l.out || l.dA) {
    cudaError_t e = shrink<RP, true>(l.dy, l.lddy, l.B, a, l.N, r, part, st);
    if (e != cudaSuccess) return e;
    e = expand<RP, true>(part, tile_splits(l.T, l.N), l.A, l.scaling, a, l.K, r, l.in, l.ldi, l.out, l.ldo, g, st);
    if (e != cudaSuccess) return e;
  }
  if (!l.dA && !l.dB) return cudaSuccess;
  const int cols = outer_cols(l.r);
  OuterArgs o{};
  o.p[0] = OuterProduct{g, l.x, l.ldx, l.K, l.dA, reinterpret_cast<float*>(ws + w.outer_a),
                        l.dA ? static_cast<int>(ceil_div(l.K, cols)) : 0, 0};
  o.p[1] = OuterProduct{l.h, l.dy, l.lddy, l.N, l.dB, reinterpret_cast<float*>(ws + w.outer_b),
                        l.dB ? static_cast<int>(ceil_div(l.N, cols)) : 0, 1};
  o.scaling = l.scaling;
  o.a = a;
  o.r = r;
  o.fp32 = l.fp32 ? 1 : 0;
  o.used = reinterpret_cast<int32_t*>(ws + w.used);
  return l.fp32 ? outer<RP, 3>(o, st) : outer<RP, 2>(o, st);
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
