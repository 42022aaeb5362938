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
constexpr int kCols = 128;     // columns of an expand tile
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

__device__ __forceinline__ void copy4(void* smem, const void* gmem, bool valid) {
  const int bytes = valid ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(smem_addr(smem)), "l"(gmem), "r"(bytes) : "memory");
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

// base + d of two columns, rounded once to bf16
__device__ __forceinline__ uint32_t add_round(uint32_t y, float d0, float d1) {
  const float2 v = __fadd2_rn(make_float2(__uint_as_float(y << 16), __uint_as_float(y & 0xFFFF0000u)), make_float2(d0, d1));
  const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&b);
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
// distinct ones.  All threads call it (at least two warps), thread t < 64 with
// token t's adapter; ends with a barrier.
struct TileAdapters {
  int ids[kRows];
  int list[kRows];
  int head, count;   // distinct ones of the first 32 tokens, and in all
};
__device__ __forceinline__ void tile_adapters(TileAdapters& ta, int id) {
  const int t = threadIdx.x, lane = t & 31;
  bool first = false;
  if (t < kRows) {
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

// The bf16 numbers that make up w [T, r] (TERMS of them), rows padded to R
// with zeros: operands of the outer products.  terms[x][t][j].
template <int RP>
__device__ __forceinline__ void write_terms(__nv_bfloat16* terms, int n_terms, int64_t T, int64_t t, int j, float v) {
  constexpr int R = 16 * RP;
  __nv_bfloat16 s[3];
  if (n_terms == 3) split_bf16(v, s[0], s[1], s[2]);
  else split_bf16(v, s[0], s[1]);
  for (int x = 0; x < n_terms; ++x) terms[(x * T + t) * R + j] = s[x];
}

// ---------------------------------------------------------------------------
// shrink: part[split][t][j] = sum over this split's columns of z[t, c] W[j, c]
// TRANS: W is stored [C, r] (c-major), else [r, C].
// 64 rows x 128 columns a stage; warp w multiplies rows 16 (w % 4) over half
// w / 4 of the stage's columns, the halves are added at the end.  The rows'
// traffic bounds it; what it takes is warps and copies in flight, so the ring
// is sized for three CTAs per SM.
// In the backward pass the first split also writes h's terms for dB.
// ---------------------------------------------------------------------------
template <int RP, bool TRANS>
struct ShrinkCfg {
  static constexpr int R = 16 * RP;
  static constexpr int KC = 128;   // columns of a stage
  static constexpr int ZB = kRows * (KC + 8) * 2;
  static constexpr int WB = (TRANS ? KC * (R + 8) : R * (KC + 8)) * 2;
  static constexpr int CTAS = RP == 1 ? 3 : (RP <= 4 ? 2 : 1);   // per SM
  static constexpr int STAGES = 224 * 1024 / CTAS / (ZB + WB);
  static constexpr int BYTES = STAGES * (ZB + WB);
};

template <int RP, bool TRANS>
__global__ void __launch_bounds__(kNT, ShrinkCfg<RP, TRANS>::CTAS)
    lora_shrink_kernel(const __nv_bfloat16* __restrict__ z, int64_t ldz, const __nv_bfloat16* __restrict__ W,
                       const AdapterIds a, int64_t C, int r, int64_t per_split, float* __restrict__ part,
                       const float* __restrict__ h, __nv_bfloat16* __restrict__ h_terms, int n_terms) {
  pdl_entry();
  using S = ShrinkCfg<RP, TRANS>;
  constexpr int R = S::R, KC = S::KC, ST = S::STAGES;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ TileAdapters ta;
  const int th = threadIdx.x, lane = th & 31, warp = th >> 5, rg = warp & 3, kh = warp >> 2;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kRows;
  const int64_t c_begin = blockIdx.y * per_split;
  const int64_t c_end = c_begin + per_split < C ? c_begin + per_split : C;
  const int steps = static_cast<int>((c_end - c_begin + KC - 1) / KC);
  tile_adapters(ta, th < kRows ? adapter_of(a, row0 + th, blockIdx.y == 0) : -1);
  float* mine = part + static_cast<int64_t>(blockIdx.y) * a.T * r;

  // this thread copies chunk zch of rows zrow, zrow + 16, ..
  const int zrow = th >> 4, zch = th & 15;
  const __nv_bfloat16* zsrc = z + (row0 + zrow) * ldz + c_begin + 8 * zch;
  uint32_t zok = 0;
#pragma unroll
  for (int i = 0; i < kRows / 16; ++i) zok |= (ta.ids[zrow + 16 * i] >= 0 ? 1u : 0u) << i;
  auto load = [&](int step, int slot, const __nv_bfloat16* w) {
    uint8_t* base = dyn + slot * (S::ZB + S::WB);
    const int64_t off = static_cast<int64_t>(step) * KC, c0 = c_begin + off;
    const uint32_t ok4 = c0 + 8 * zch < c_end ? zok : 0u;
#pragma unroll
    for (int i = 0; i < kRows / 16; ++i) {
      const bool ok = ok4 >> i & 1u;
      copy16(base + (zrow + 16 * i) * (KC + 8) * 2 + 16 * zch, ok ? zsrc + off + 16 * i * ldz : z, ok);
    }
    uint8_t* wb = base + S::ZB;
#pragma unroll
    for (int i = 0; i < RP; ++i) {
      if constexpr (!TRANS) {   // ranks zrow + 16 i, chunk zch
        const int j = zrow + 16 * i;
        const bool ok = j < r && c0 + 8 * zch < c_end;
        copy16(wb + j * (KC + 8) * 2 + 16 * zch, ok ? w + j * C + c0 + 8 * zch : w, ok);
      } else {
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
#pragma unroll
    for (int p = 0; p < ST - 1; ++p) {
      if (p < steps) load(p, p, w);
      else cp_async_commit();
    }
    int slot = 0, ahead = ST - 1;
    for (int s = 0; s < steps; ++s) {
      cp_async_wait<ST - 2>();   // this stage has landed
      __syncthreads();           // for every thread, and the stage before it has been read
      if (s + ST - 1 < steps) load(s + ST - 1, ahead, w);
      else cp_async_commit();
      const uint8_t* base = dyn + slot * (S::ZB + S::WB);
      if (++slot == ST) slot = 0;
      if (++ahead == ST) ahead = 0;
      const __nv_bfloat16* zs = reinterpret_cast<const __nv_bfloat16*>(base);
      const __nv_bfloat16* ws = reinterpret_cast<const __nv_bfloat16*>(base + S::ZB);
      // this stage's sums start from zero and are added to the running ones:
      // the tensor core truncates as it adds, so its runs are kept short
      float acc[2 * RP][4];
#pragma unroll
      for (int i = 0; i < 2 * RP; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
      // fragments of kBatch products of 16 columns are loaded together, so
      // their latencies overlap
      constexpr int kBatch = RP <= 2 ? 4 : 2;
#pragma unroll
      for (int k8 = 0; k8 < KC / 2; k8 += 16 * kBatch) {
        uint32_t af[kBatch][4], bf[kBatch][RP][4];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int kk = kh * (KC / 2) + k8 + 16 * b;
          ldsm4(af[b], zs + (16 * rg + (lane & 15)) * (KC + 8) + kk + (lane >> 4) * 8);
#pragma unroll
          for (int p = 0; p < RP; ++p) {
            if constexpr (!TRANS)
              ldsm4(bf[b][p], ws + (16 * p + (lane & 7) + ((lane >> 4) << 3)) * (KC + 8) + kk + ((lane >> 3) & 1) * 8);
            else
              ldsm4_t(bf[b][p], ws + (kk + (lane & 7) + ((lane >> 3) & 1) * 8) * (R + 8) + 16 * p + (lane >> 4) * 8);
          }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
#pragma unroll
          for (int p = 0; p < RP; ++p) {
            mma16(acc[2 * p], af[b], bf[b][p]);
            mma16(acc[2 * p + 1], af[b], bf[b][p] + 2);
          }
      }
#pragma unroll
      for (int i = 0; i < 2 * RP; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[i][e] = __fadd_rn(sum[i][e], acc[i][e]);
    }
    __syncthreads();   // the ring is free: every copy has landed and been read
    // add the second half's sums
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
  if (h_terms && blockIdx.y == 0) {
    for (int k = th; k < kRows * R; k += kNT) {
      const int64_t t = row0 + k / R;
      const int j = k % R;
      if (t < a.T) write_terms<RP>(h_terms, n_terms, a.T, t, j, j < r ? __ldg(h + t * r + j) : 0.0f);
    }
  }
}

// ---------------------------------------------------------------------------
// expand: out[t, c] = base[t, c] + s_a sum_j w[t, j] W[c, j], w = sum of the
// partials; w itself goes to w_out, its terms to w_terms.  TRANS: W is stored
// [r, C], else [C, r].
// A CTA takes 64 tokens and `per_cta` tiles of 128 columns; warp w rows
// 16 (w % 4), columns 64 (w / 4).  A thread's products land on the 16 bytes
// of base it has loaded (see mma_slot), so neither base nor result passes
// through shared memory.  Instructions and their latencies bound it before
// memory does: the scale is folded into w, base is added in pairs, and tiles
// are narrow so that four CTAs (32 warps) fit an SM.  Measured at 8192 x
// 14336, r = 16: 256-column tiles, three CTAs and 632 instructions per warp
// and 256 columns 105 us; a persistent form that prefetched the next tile with
// two CTAs 120 us.
// ---------------------------------------------------------------------------
template <int RP, bool TRANS>
struct ExpandCfg {
  static constexpr int R = 16 * RP;
  static constexpr int HB = kRows * (R + 8) * 2;
  static constexpr int WB = (TRANS ? R * (kCols + 8) : kCols * (R + 8)) * 2;
  static constexpr int BYTES = 2 * HB + WB;
  static constexpr int CTAS = RP <= 4 ? 4 : 2;   // per SM
};

template <int RP, bool TRANS>
__global__ void __launch_bounds__(kNT, ExpandCfg<RP, TRANS>::CTAS)
    lora_expand_kernel(const float* __restrict__ part, int splits, const __nv_bfloat16* __restrict__ W,
                       const float* __restrict__ scaling, const AdapterIds a, int64_t C, int r, int per_cta, int groups,
                       const __nv_bfloat16* in, int64_t ldi, __nv_bfloat16* out, int64_t ldo,
                       float* __restrict__ w_out, __nv_bfloat16* __restrict__ w_terms, int n_terms) {
  pdl_entry();
  using S = ExpandCfg<RP, TRANS>;
  constexpr int R = S::R;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ TileAdapters ta;
  __nv_bfloat16* hh = reinterpret_cast<__nv_bfloat16*>(dyn);
  __nv_bfloat16* hl = reinterpret_cast<__nv_bfloat16*>(dyn + S::HB);
  __nv_bfloat16* ws = reinterpret_cast<__nv_bfloat16*>(dyn + 2 * S::HB);
  const int th = threadIdx.x, lane = th & 31, warp = th >> 5, rg = warp & 3, ch = warp >> 2;
  // neighbouring CTAs take neighbouring columns of the same rows
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / groups) * kRows;
  const int group = blockIdx.x % groups;
  const int my_row = 16 * rg + (lane >> 2);        // this thread's rows of the tile: my_row and my_row + 8
  const int my_col = 64 * ch + 8 * (lane & 3);     // and its columns: 8 from here on, and 32 further
  uint4 y[2][2];
  auto load_base = [&](int64_t c0) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int64_t t = row0 + my_row + 8 * half, c = c0 + my_col + 32 * q;
        y[q][half] = make_uint4(0u, 0u, 0u, 0u);
        if (in && c < C && t < a.T) y[q][half] = __ldcs(reinterpret_cast<const uint4*>(in + t * ldi + c));
      }
    }
  };
  // loads that do not depend on the adapters first
  const int id_mine = th < kRows ? adapter_of(a, row0 + th, false) : -1;
  if (out) load_base(static_cast<int64_t>(group) * per_cta * kCols);
  tile_adapters(ta, id_mine);
  // the sum of the partials, in their order
#pragma unroll 4
  for (int k = th; k < kRows * R; k += kNT) {
    const int row = k / R, j = k % R;
    float v = 0.0f;
    if (row0 + row < a.T) {
      const int64_t at = (row0 + row) * r + j;
      if (j < r)
        for (int s = 0; s < splits; ++s) v = __fadd_rn(v, __ldcg(part + s * a.T * r + at));
      if (group == 0) {
        if (w_out && j < r) w_out[at] = v;
        if (w_terms) write_terms<RP>(w_terms, n_terms, a.T, row0 + row, j, v);
      }
    }
    const int id = ta.ids[row];
    split_bf16(id >= 0 ? __fmul_rn(__ldg(scaling + id), v) : 0.0f, hh[row * (R + 8) + j], hl[row * (R + 8) + j]);
  }
  if (!out) return;   // only the sum was asked for
  const int id_lo = ta.ids[my_row], id_hi = ta.ids[my_row + 8];

  for (int i = 0; i < per_cta; ++i) {
    const int64_t c0 = (static_cast<int64_t>(group) * per_cta + i) * kCols;
    if (c0 >= C) break;
    if (i > 0) load_base(c0);
    for (int u = 0; u < ta.count; ++u) {
      const int id = ta.list[u];
      const __nv_bfloat16* w = W + static_cast<int64_t>(id) * r * C;
      if (i > 0 || u > 0) __syncthreads();   // the previous weights have been read
      if constexpr (!TRANS) {
#pragma unroll
        for (int x = 0; x < RP; ++x) {
          const int k = th + kNT * x, c = k / (R / 8), c8 = k % (R / 8);
          const bool ok = c0 + c < C && 8 * c8 < r;
          copy16(ws + mma_slot(c) * (R + 8) + 8 * c8, ok ? w + (c0 + c) * r + 8 * c8 : w, ok);
        }
      } else {
        // pairs of columns, each to its slot
        const int c = 2 * (th & 63), slot = mma_slot(c);
        const bool col_ok = c0 + c < C;
#pragma unroll
        for (int x = 0; x < R / 4; ++x) {
          const int j = (th >> 6) + 4 * x;
          const bool ok = col_ok && j < r;
          copy4(ws + j * (kCols + 8) + slot, ok ? w + j * C + c0 + c : w, ok);
        }
      }
      cp_async_commit();
      cp_async_wait<0>();
      __syncthreads();
      const bool lo_mine = id_lo == id, hi_mine = id_hi == id;
      if (!__any_sync(0xFFFFFFFFu, lo_mine || hi_mine)) continue;
#pragma unroll
      for (int q = 0; q < 2; ++q) {   // 32 columns each
        float acc[4][4] = {};
#pragma unroll
        for (int kk = 0; kk < R; kk += 16) {
          uint32_t ah[4], al[4], b0[4], b1[4];
          ldsm4(ah, hh + (16 * rg + (lane & 15)) * (R + 8) + kk + (lane >> 4) * 8);
          ldsm4(al, hl + (16 * rg + (lane & 15)) * (R + 8) + kk + (lane >> 4) * 8);
          if constexpr (!TRANS) {
            const __nv_bfloat16* wq = ws + (64 * ch + 32 * q + (lane & 7) + ((lane >> 4) << 3)) * (R + 8) + kk + ((lane >> 3) & 1) * 8;
            ldsm4(b0, wq);
            ldsm4(b1, wq + 16 * (R + 8));
          } else {
            const __nv_bfloat16* wq = ws + (kk + (lane & 7) + ((lane >> 3) & 1) * 8) * (kCols + 8) + 64 * ch + 32 * q + (lane >> 4) * 8;
            ldsm4_t(b0, wq);
            ldsm4_t(b1, wq + 16);
          }
          mma16(acc[0], al, b0);
          mma16(acc[1], al, b0 + 2);
          mma16(acc[2], al, b1);
          mma16(acc[3], al, b1 + 2);
          mma16(acc[0], ah, b0);
          mma16(acc[1], ah, b0 + 2);
          mma16(acc[2], ah, b1);
          mma16(acc[3], ah, b1 + 2);
        }
        // a token without an adapter keeps the base's bits (a NaN's payload, a zero's sign)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (half ? hi_mine : lo_mine) {
            uint4& v = y[q][half];
            v.x = add_round(v.x, acc[0][2 * half], acc[0][2 * half + 1]);
            v.y = add_round(v.y, acc[1][2 * half], acc[1][2 * half + 1]);
            v.z = add_round(v.z, acc[2][2 * half], acc[2][2 * half + 1]);
            v.w = add_round(v.w, acc[3][2 * half], acc[3][2 * half + 1]);
          }
        }
      }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int64_t t = row0 + my_row + 8 * half, c = c0 + my_col + 32 * q;
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
        for (int e = 0; e < 4; ++e) split_bf16(__fmul_rn(s, vv[e]), h[e], l[e]);
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
        uint4& v = y[q][half];
        v.x = add_round(v.x, acc[0][2 * half], acc[0][2 * half + 1]);
        v.y = add_round(v.y, acc[1][2 * half], acc[1][2 * half + 1]);
        v.z = add_round(v.z, acc[2][2 * half], acc[2][2 * half + 1]);
        v.w = add_round(v.w, acc[3][2 * half], acc[3][2 * half + 1]);
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
// 2 (2^-17) for bf16 ones.  They were written by the kernels before this one,
// once for all column tiles.
// ---------------------------------------------------------------------------
struct OuterProduct {
  const __nv_bfloat16* w;   // [TERMS][T][16 RP]
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
  static constexpr int HB = kRows * (R + 8) * 2;
  static constexpr int STAGE = ZB + TERMS * HB;
  static constexpr int CTAS = RP <= 2 ? 2 : 1;        // per SM
  static constexpr int STAGES = (CTAS == 2 ? 104 : 208) * 1024 / STAGE;
  static constexpr int BYTES = STAGES * STAGE;
};
constexpr int kWindow = 2048;   // rows whose ids a CTA looks at together

__device__ __forceinline__ void store_out(void* dst, int64_t at, float v, bool fp32) {
  if (fp32) static_cast<float*>(dst)[at] = v;
  else static_cast<__nv_bfloat16*>(dst)[at] = __float2bfloat16_rn(v);
}

template <int RP, int TERMS>
__global__ void __launch_bounds__(kNT, OuterCfg<RP, TERMS>::CTAS) lora_outer_kernel(const OuterArgs o) {
  pdl_entry();
  using S = OuterCfg<RP, TERMS>;
  constexpr int R = S::R, COLS = S::COLS, NQ = S::NQ, ST = S::STAGES;
  static_assert(ST >= 2, "a ring");
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
  // this thread copies one 16-byte chunk of rows zrow, zrow + kRowStep, ..
  constexpr int kRowStep = kNT / (COLS / 8);
  const int zrow = th / (COLS / 8), zch = th % (COLS / 8);
  const bool zcol_ok = c0 + 8 * zch < p.C;
  const __nv_bfloat16* zbase = p.z + c0 + 8 * zch;
  const int64_t zstep = kRowStep * p.ldz;

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

    auto load = [&](int k, int slot) {
      const int tile = list[k];
      uint8_t* st = dyn + slot * S::STAGE;
      const int64_t row0 = row_base + static_cast<int64_t>(tile) * kRows;
      const __nv_bfloat16* src = zbase + (row0 + zrow) * p.ldz;
      const int* idr = ids + tile * kRows + zrow;
      uint8_t* to = st + zrow * (COLS + 8) * 2 + 16 * zch;
#pragma unroll
      for (int i = 0; i < kRows / kRowStep; ++i) {
        const bool ok = zcol_ok && idr[kRowStep * i] == id;
        copy16(to + i * kRowStep * (COLS + 8) * 2, ok ? src + i * zstep : p.z, ok);
      }
      for (int e = th; e < TERMS * kRows * (R / 8); e += kNT) {
        const int x = e / (kRows * (R / 8)), row = e / (R / 8) % kRows, ch = e % (R / 8);
        const bool ok = ids[tile * kRows + row] == id;
        copy16(st + S::ZB + x * S::HB + row * (R + 8) * 2 + 16 * ch,
               ok ? p.w + (x * o.a.T + row0 + row) * R + 8 * ch : p.w, ok);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < ST - 1; ++k) {
      if (k < count) load(k, k);
      else cp_async_commit();
    }
    int slot = 0, ahead = ST - 1;
    for (int k = 0; k < count; ++k) {
      cp_async_wait<ST - 2>();   // this tile has landed
      __syncthreads();           // for every thread, and the tile before it has been read
      if (k + ST - 1 < count) load(k + ST - 1, ahead);
      else cp_async_commit();
      const uint8_t* st = dyn + slot * S::STAGE;
      if (++slot == ST) slot = 0;
      if (++ahead == ST) ahead = 0;
      const __nv_bfloat16* zs = reinterpret_cast<const __nv_bfloat16*>(st);
      const __nv_bfloat16* wb = reinterpret_cast<const __nv_bfloat16*>(st + S::ZB);
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

// Columns per shrink split: one wave of three CTAs per SM, with few tokens
// about eight small CTAs per SM; whole 128-column stages.
int64_t shrink_per_split(int64_t T, int64_t C, int64_t n) {
  const bool few = T <= kFewTokens;
  const int64_t rows = few ? most_units(T, n) : ceil_div(T, kRows);
  const int64_t step = 128;
  const int64_t splits = std::max<int64_t>(1, std::min<int64_t>(few ? 16 : 32, (few ? 8 : 3) * sm_count() / rows));
  return ceil_div(ceil_div(C, splits), step) * step;
}
int shrink_splits(int64_t T, int64_t C, int64_t n) { return static_cast<int>(ceil_div(C, shrink_per_split(T, C, n))); }
// The backward pass shrinks with the tile kernel for any T.
int64_t tile_per_split(int64_t T, int64_t C) {
  const int64_t splits = std::max<int64_t>(1, std::min<int64_t>(32, 3 * sm_count() / ceil_div(T, kRows)));
  return ceil_div(ceil_div(C, splits), 128) * 128;
}
int tile_splits(int64_t T, int64_t C) { return static_cast<int>(ceil_div(C, tile_per_split(T, C))); }

int outer_cols(int64_t r) { return r <= 32 ? 256 : 128; }
// Row ranges of the outer products: at most 2048 tokens each (an adapter may
// own all of them), unless that makes more than 8.
int outer_splits(int64_t T) { return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(8, ceil_div(T, kWindow)))); }

// Parts of the workspace, in 16-byte steps.
struct LoraWorkspace {
  size_t part, g_terms, h_terms, outer_a, outer_b, used, total;
};
size_t up16(size_t v) { return (v + 15) & ~static_cast<size_t>(15); }
int64_t padded_rank(int64_t r) { return r <= 16 ? 16 : (r <= 32 ? 32 : (r <= 64 ? 64 : 128)); }
LoraWorkspace lora_workspace(int64_t T, int64_t K, int64_t N, int64_t r, int64_t n, bool backward) {
  LoraWorkspace w{};
  w.part = 0;
  w.total = up16(static_cast<size_t>(backward ? tile_splits(T, N) : shrink_splits(T, K, n)) * T * r * 4);
  if (backward) {
    const size_t terms = up16(static_cast<size_t>(3 * T) * padded_rank(r) * 2);
    w.g_terms = w.total;
    w.h_terms = w.g_terms + terms;
    w.outer_a = w.h_terms + terms;
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
                   float* part, const float* h, __nv_bfloat16* h_terms, int n_terms, cudaStream_t st) {
  auto fn = lora_shrink_kernel<RP, TRANS>;
  constexpr int smem = ShrinkCfg<RP, TRANS>::BYTES;
  static bool done[64] = {false};
  cudaError_t e = allow_smem(fn, smem, done);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(ceil_div(a.T, kRows)), static_cast<unsigned>(tile_splits(a.T, C)));
  e = launch_k(fn, grid, dim3(kNT), smem, st, 1u, z, ldz, W, a, C, r, tile_per_split(a.T, C), part, h,
               h_terms, n_terms);
  note_launch();
  return e;
}

template <int RP, bool TRANS>
cudaError_t expand(const float* part, int splits, const __nv_bfloat16* W, const float* scaling, const AdapterIds& a,
                   int64_t C, int r, const __nv_bfloat16* in, int64_t ldi, __nv_bfloat16* out, int64_t ldo, float* w_out,
                   __nv_bfloat16* w_terms, int n_terms, cudaStream_t st) {
  auto fn = lora_expand_kernel<RP, TRANS>;
  constexpr int smem = ExpandCfg<RP, TRANS>::BYTES;
  static bool done[64] = {false};
  cudaError_t e = allow_smem(fn, smem, done);
  if (e != cudaSuccess) return e;
  // up to eight column tiles share one sum of the partials, as long as the
  // grid still fills the GPU a few times over
  const int64_t rows = ceil_div(a.T, kRows), cols = ceil_div(C, kCols);
  const int per = out ? static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(8, rows * cols / (8 * sm_count())))) : 1;
  const int64_t groups = out ? ceil_div(cols, per) : 1;
  e = launch_k(fn, dim3(static_cast<unsigned>(rows * groups)), dim3(kNT), smem, st, 1u, part, splits, W, scaling, a, C, r, per,
               static_cast<int>(groups), in, ldi, out, ldo, w_out, w_terms, n_terms);
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
    const cudaError_t e = shrink<RP, false>(l.x, l.ldx, l.A, a, l.K, r, part, nullptr, nullptr, 0, st);
    if (e != cudaSuccess) return e;
    return expand<RP, false>(part, tile_splits(l.T, l.K), l.B, l.scaling, a, l.N, r, l.in, l.ldi, l.out, l.ldo, l.h,
                             nullptr, 0, st);
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
  const int r = static_cast<int>(l.r), n_terms = l.fp32 ? 3 : 2;
  float* part = reinterpret_cast<float*>(ws + w.part);
  __nv_bfloat16* g_terms = reinterpret_cast<__nv_bfloat16*>(ws + w.g_terms);
  __nv_bfloat16* h_terms = reinterpret_cast<__nv_bfloat16*>(ws + w.h_terms);
  // the shrink also writes h's terms, so it runs even where dB alone is asked for
  cudaError_t e = shrink<RP, true>(l.dy, l.lddy, l.B, a, l.N, r, part, l.h, l.dB ? h_terms : nullptr, n_terms, st);
  if (e != cudaSuccess) return e;
  if (l.out || l.dA) {
    e = expand<RP, true>(part, tile_splits(l.T, l.N), l.A, l.scaling, a, l.K, r, l.in, l.ldi, l.out, l.ldo, nullptr,
                         l.dA ? g_terms : nullptr, n_terms, st);
    if (e != cudaSuccess) return e;
  }
  if (!l.dA && !l.dB) return cudaSuccess;
  const int cols = outer_cols(l.r);
  OuterArgs o{};
  o.p[0] = OuterProduct{g_terms, l.x, l.ldx, l.K, l.dA, reinterpret_cast<float*>(ws + w.outer_a),
                        l.dA ? static_cast<int>(ceil_div(l.K, cols)) : 0, 0};
  o.p[1] = OuterProduct{h_terms, l.dy, l.lddy, l.N, l.dB, reinterpret_cast<float*>(ws + w.outer_b),
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
