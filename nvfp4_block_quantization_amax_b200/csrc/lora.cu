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
//           split over the CTAs of a cluster, which add their sums through
//           distributed shared memory;
//   expand  (h, B) + y -> out and (g, A) + dx0 -> dx: contraction over the
//           rank;
//   outer   (g, x) -> dA and (h, dy) -> dB: contraction over one adapter's
//           tokens.
// What bounds them are the long rows that pass through memory once (shrink,
// outer) or twice (expand).  They stream through rings of shared memory that
// one producer warp fills with TMA, so that the copies in flight do not depend
// on how many warps fit an SM: with copies issued by the computing threads
// the same products ran at 2.2 to 4.5 TB/s (a plain copy kernel needs six
// 256-thread CTAs per SM to reach 6 TB/s, and these have registers for two to
// four).
// The products are small (2 T r (K + N) flops) beside the rows that pass
// through memory, so they run on mma.sync with bf16 operands and fp32 sums.
// h and g are kept in fp32; where they are an operand of a product they enter
// as the sum of two bf16 numbers (16 bits of mantissa, error 2^-17), which
// costs one more product of the rank's size instead of bf16's 2^-8.
// Adapters are found tile by tile: a tile of 64 tokens loops over the
// adapters that occur in it, so tokens of one request (in a row) share one
// pass and any order is right.  The forward pass of few tokens gathers them by
// adapter instead.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>
#include <cstdlib>

#include "gemm_ptx.cuh"
#include "launch.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

constexpr int kRows = 64;      // tokens of a tile
// Up to here the tokens are gathered by adapter.  4096 -> 14336, gathered /
// tiles of 64 tokens, us: 256 tokens of 32 adapters in random order r = 16
// 30 / 92, r = 64 71 / 163; one adapter's after the other r = 16 30 / 36,
// r = 64 70 / 66; of one adapter r = 16 20 / 20, r = 64 45 / 25 (64 tokens
// 21 / 20).  The host does not know the ids, so the size alone decides, for
// the order that costs most.  Beyond, tiles of many adapters take their time:
// 32 adapters in random order / in runs, r = 16, 257 tokens 93 / 37, 512
// 141 / 35, 1024 246 / 39, 2048 450 / 57.
constexpr int kFewTokens = 256;

struct AdapterIds {
  const int32_t* ids;
  int64_t T;
  int n;
  int32_t* status;
  uint32_t wait_ns;   // time limit of a ring's wait
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

// The leading bf16 part of v.  Where v is neither zero nor infinite, nor is it
// (the first and the last half steps of the range would round to those), so
// that its product with an infinity, or with zero, is v's.
__device__ __forceinline__ __nv_bfloat16 lead_bf16(float v) {
  uint32_t h = __bfloat16_as_ushort(__float2bfloat16_rn(v));
  if ((__float_as_uint(v) & 0x7FFFFFFFu) - 1u < 0x7F7FFFFFu) h = (h & 0x8000u) | min(max(h & 0x7FFFu, 1u), 0x7F7Fu);
  return __ushort_as_bfloat16(static_cast<unsigned short>(h));
}
// A sum of the lower parts' products made finite (NaN: the largest number).
// Next to an infinite factor such sums are infinities of any sign, or
// 0 inf = NaN; the leading parts' sum is infinite or NaN there as the formula
// is, and a number added to it changes nothing.
__device__ __forceinline__ float clamp(float low) {
  float v;   // the sign of low, the smaller magnitude
  asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(v) : "f"(low), "f"(3.402823466e38f));
  return v;
}

// v = hi + lo up to 2^-17 |v| (an infinity or NaN is all in hi: its lo would
// be a NaN of its own)
__device__ __forceinline__ float rest_of(float v, float hi) {
  const float rest = __fsub_rn(v, hi);
  return fabsf(rest) <= 3.402823466e38f ? rest : 0.0f;
}
__device__ __forceinline__ void split_bf16(float v, __nv_bfloat16& hi, __nv_bfloat16& lo) {
  hi = lead_bf16(v);
  lo = __float2bfloat16_rn(rest_of(v, __bfloat162float(hi)));
}
// v = hi + mid + lo, all 24 bits
__device__ __forceinline__ void split_bf16(float v, __nv_bfloat16& hi, __nv_bfloat16& mid, __nv_bfloat16& lo) {
  hi = lead_bf16(v);
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

// Column order of a 32-column group in the few-token expand: thread c of a
// quad owns columns 8c .. 8c + 7 of its rows (16 bytes of bf16) when column
// 8 (n / 2) + 2 q + n % 2 of the group is column n of the group's MMA q.
__device__ __forceinline__ int slot_col(int slot) {
  const int q = (slot & 31) >> 3, n = slot & 7;
  return (slot & ~31) + 8 * (n >> 1) + 2 * q + (n & 1);
}

// ---- rings of shared memory, filled by TMA --------------------------------
// A ring's barriers: full[s] completes when a slot's bytes have landed,
// empty[s] when every consumer warp has arrived.  All waits are bounded: one
// that gives up raises the abort flag and reports NVFP4_ERR_TIMEOUT, and the
// kernel runs to its end.  The producer then issues nothing more.  The
// consumers' lanes may disagree about a wait near its limit (one gives up,
// another still sees the data), so none of them leaves its loop: the warps go
// on in step through whatever the slots hold and meet at every barrier.
constexpr int kConsumers = 8;                      // warps
constexpr int kThreads = 32 * (kConsumers + 1);    // and the producer warp

// The abort flag and the time limit of a wait (shared memory; the limit is
// looked at only by a wait that did not succeed at once).
struct Abort {
  volatile int flag;
  volatile uint32_t limit_ns;
};
__device__ __forceinline__ bool ring_wait(uint32_t bar, uint32_t parity, Abort* abort) {
  if (mbar_test_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (!abort->flag) {
    if (mbar_try_wait(bar, parity)) return true;
    if (globaltimer() - t0 > abort->limit_ns) abort->flag = 1;
  }
  return false;
}

struct Ring {
  uint64_t* full;
  uint64_t* empty;
  int slots;
  int slot = 0;
  uint32_t phase = 0;   // of the current pass over the slots
  __device__ __forceinline__ void init() const {   // one thread
    for (int i = 0; i < slots; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), kConsumers);
    }
  }
  __device__ __forceinline__ void next() {
    if (++slot == slots) {
      slot = 0;
      phase ^= 1;
    }
  }
  // By every lane of a consumer warp, which goes on together.
  __device__ __forceinline__ void wait_full(Abort* abort, int32_t* status) const {
    if (!ring_wait(smem_u32(&full[slot]), phase, abort) && status) *status = kStatusTimeout;
    __syncwarp();
  }
  // By the producer's lane; false: nothing more is to be issued (a consumer
  // that gave up raised the flag before it gave the slot back, in which a copy
  // may still be landing).
  __device__ __forceinline__ bool wait_empty(Abort* abort) const {
    return ring_wait(smem_u32(&empty[slot]), phase ^ 1, abort) && !abort->flag;
  }
  // The producer lets the copies it has issued (`issued` slots in all) land
  // before its CTA goes.
  __device__ __forceinline__ void drain(int issued) const {
    for (int i = issued > slots ? issued - slots : 0; i < issued; ++i)
      mbar_wait_bounded(smem_u32(&full[i % slots]), (i / slots) & 1);
  }
};
// A consumer warp is done with a slot.
__device__ __forceinline__ void release(uint64_t* empty) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(empty)) : "memory");
}
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kConsumers) : "memory"); }

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// Shared-memory tiles as TMA writes them: rows of ROW bytes (64 or 128) whose
// 16-byte chunks are swizzled by the row, so that eight rows of one chunk lie
// in different banks.  Wider tiles are several boxes, one behind the other.
template <int ROW>
__device__ __forceinline__ const uint8_t* chunk_at(const uint8_t* tile, int row, int chunk) {
  constexpr int kShift = ROW == 128 ? 0 : 1;
  return tile + row * ROW + ((chunk ^ ((row >> kShift) & (ROW / 16 - 1))) << 4);
}
template <int ROW>
__device__ __forceinline__ uint8_t* chunk_at(uint8_t* tile, int row, int chunk) {
  return const_cast<uint8_t*>(chunk_at<ROW>(static_cast<const uint8_t*>(tile), row, chunk));
}

// A tile of rank vectors: ROWS rows of R = 16 RP ranks (R = 128: two boxes).
// Rows of 32 bytes (R = 16) are not swizzled: a tile of them is one piece of
// memory, which a plain bulk copy brings in 128-byte lines, where a tensor copy
// takes as long for each 32-byte row as for one of 128 (eight rows then share
// two cycles of shared memory instead of one, which costs less).
template <int RP>
struct RankTile {
  static constexpr int R = 16 * RP;
  static constexpr int ROW = RP == 8 ? 128 : 2 * R;
  static constexpr int BOXES = RP == 8 ? 2 : 1;
  template <int ROWS>
  static __device__ __forceinline__ const uint8_t* at(const uint8_t* tile, int row, int chunk) {   // chunk: 8 ranks
    if constexpr (RP == 1) return tile + row * ROW + 16 * chunk;
    else if constexpr (BOXES == 1) return chunk_at<ROW>(tile, row, chunk);
    else return chunk_at<ROW>(tile + (chunk >> 3) * (ROWS * ROW), row, chunk & 7);
  }
};

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

// Rank vectors c .. c + ROWS - 1 of adapter `id` (W [n, C, r]) into a tile.
template <int RP, int ROWS>
__device__ __forceinline__ void load_ranks(uint32_t dst, const CUtensorMap* map, const __nv_bfloat16* W, int id, int c,
                                           int64_t C, int r, uint32_t bar) {
  if (RP == 1 && r == 16 && c + ROWS <= C) {
    bulk_load(dst, W + (static_cast<int64_t>(id) * C + c) * 16, ROWS * 32, bar);
    return;
  }
  tma_load_3d(dst, map, 0, c, id, bar);   // rows past the last one read as zeros
  if constexpr (RP == 8) tma_load_3d(dst + ROWS * 128, map, 64, c, id, bar);
}

// The bf16 numbers that make up w [T, r] (n_terms of them), rows padded to R
// with zeros: operands of the outer products.  terms[x][t][j].
__device__ __forceinline__ void write_terms(__nv_bfloat16* terms, int n_terms, int64_t T, int R, int64_t t, int j, float v) {
  __nv_bfloat16 s[3];
  if (n_terms == 3) split_bf16(v, s[0], s[1], s[2]);
  else split_bf16(v, s[0], s[1]);
  for (int x = 0; x < n_terms; ++x) terms[(x * T + t) * R + j] = s[x];
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Sum over the cluster's `split` <= 8 CTAs, in rank order, of the float at this
// shared-memory address in each (the loads go out together).
__device__ __forceinline__ float sum_cluster(const float* p, int split) {
  float v[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    v[q] = 0.0f;
    if (q < split)
      asm volatile("ld.shared::cluster.f32 %0, [%1];"
                   : "=f"(v[q]) : "r"(map_to_rank(smem_u32(p), static_cast<uint32_t>(q))) : "memory");
  }
#pragma unroll
  for (int q = 1; q < 8; ++q) v[0] = __fadd_rn(v[0], v[q]);
  return v[0];
}

// ---------------------------------------------------------------------------
// shrink: w[t][j] = sum over the columns of z[t, c] W[j, c], fp32.
// TRANS: W is stored [C, r] (c-major), else [r, C].
// A cluster of S CTAs takes 64 rows, each CTA a share of the columns in stages
// of 128 (16 KB of z, 4 to 32 KB of weights).  Warp w multiplies rows
// 16 (w % 4) over half w / 4 of a stage.  Sums of the cluster are added in
// rank order.  In the backward pass the terms of w and of h are written here.
// Memory bounds it: 8192 x 4096, r = 16 21 us (3.2 TB/s), 8192 x 14336 63 us
// (3.7 TB/s): 256 CTAs on 148 SMs leave 40 SMs with half the work of the rest.
// ---------------------------------------------------------------------------
template <int RP, bool TRANS>
struct ShrinkCfg {
  static constexpr int R = 16 * RP;
  static constexpr int KC = 128;                     // columns of a stage
  static constexpr int ZB = kRows * KC * 2;          // two boxes of 64 columns
  static constexpr int WB = R * KC * 2;
  static constexpr int SUM = kRows * R * 4;
  static constexpr int CTAS = RP <= 2 ? 2 : 1;       // per SM
  static constexpr int STAGES = ((CTAS == 2 ? 110 : 224) * 1024 - SUM) / (ZB + WB);
  static constexpr int BYTES = 1024 + STAGES * (ZB + WB) + SUM + 256;
};

template <int RP, bool TRANS>
__global__ void __launch_bounds__(kThreads, ShrinkCfg<RP, TRANS>::CTAS)
    lora_shrink_kernel(const __grid_constant__ CUtensorMap tmap_z, const __grid_constant__ CUtensorMap tmap_w,
                       const __nv_bfloat16* __restrict__ W, const AdapterIds a, int64_t C, int r, int split, float* __restrict__ w_out,
                       __nv_bfloat16* __restrict__ w_terms, const float* __restrict__ h,
                       __nv_bfloat16* __restrict__ h_terms, int n_terms) {
  pdl_entry();
  using S = ShrinkCfg<RP, TRANS>;
  [[maybe_unused]] constexpr int R = S::R, KC = S::KC;
  extern __shared__ uint8_t dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
  uint8_t* zs = smem;
  uint8_t* wsm = zs + S::STAGES * S::ZB;
  float* sums = reinterpret_cast<float*>(wsm + S::STAGES * S::WB);   // [64][R]
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sums) + S::SUM);
  Ring ring{bars, bars + S::STAGES, S::STAGES};
  Abort* abort = reinterpret_cast<Abort*>(bars + 2 * S::STAGES);
  __shared__ TileAdapters ta;
  const int th = threadIdx.x, lane = th & 31, warp = th >> 5;
  const int rank = static_cast<int>(blockIdx.x) % split;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / split) * kRows;
  // stages rank, rank + split, ..: the cluster reads neighbouring columns at a
  // time, which DRAM answers faster than distant ones
  const int stages = static_cast<int>((C + KC - 1) / KC);
  const int steps = (stages - rank + split - 1) / split;
  if (th == 0) {
    ring.init();
    abort->flag = 0;
    abort->limit_ns = a.wait_ns;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  for (int k = th; k < kRows * R; k += kThreads) sums[k] = 0.0f;
  tile_adapters(ta, th < kRows ? adapter_of(a, row0 + th, rank == 0) : -1);   // ends with a barrier

  if (warp == kConsumers) {
    if (lane == 0) {
      int issued = 0;
      for (int u = 0; u < ta.count && !abort->flag; ++u) {
        for (int s = 0; s < steps; ++s, ++issued, ring.next()) {
          if (!ring.wait_empty(abort)) break;
          const uint32_t bar = smem_u32(&ring.full[ring.slot]);
          const uint32_t zd = smem_u32(zs + ring.slot * S::ZB), wd = smem_u32(wsm + ring.slot * S::WB);
          const int c = (s * split + rank) * KC;
          mbar_expect_tx(bar, S::ZB + S::WB);
          tma_load_2d(zd, &tmap_z, c, static_cast<int>(row0), bar);
          tma_load_2d(zd + S::ZB / 2, &tmap_z, c + 64, static_cast<int>(row0), bar);
          if constexpr (!TRANS) {
            tma_load_3d(wd, &tmap_w, c, 0, ta.list[u], bar);
            tma_load_3d(wd + S::WB / 2, &tmap_w, c + 64, 0, ta.list[u], bar);
          } else {
            load_ranks<RP, KC>(wd, &tmap_w, W, ta.list[u], c, C, r, bar);
          }
        }
      }
      ring.drain(issued);
    }
    __syncwarp();
  } else {
    const int rg = warp & 3, kh = warp >> 2;
    for (int u = 0; u < ta.count; ++u) {
      const int id = ta.list[u];
      float sum[2 * RP][4];
#pragma unroll
      for (int i = 0; i < 2 * RP; ++i) sum[i][0] = sum[i][1] = sum[i][2] = sum[i][3] = 0.0f;
      for (int s = 0; s < steps; ++s) {
        ring.wait_full(abort, a.status);
        const uint8_t* zt = zs + ring.slot * S::ZB + kh * (S::ZB / 2);   // this half's box of 64 columns
        const uint8_t* wt = wsm + ring.slot * S::WB;
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
            const int kk = k8 + 16 * b;   // within this half
            ldsm4(af[b], chunk_at<128>(zt, 16 * rg + (lane & 15), kk / 8 + (lane >> 4)));
#pragma unroll
            for (int p = 0; p < RP; ++p) {
              if constexpr (!TRANS)
                ldsm4(bf[b][p], chunk_at<128>(wt + kh * (S::WB / 2), 16 * p + (lane & 7) + ((lane >> 4) << 3), kk / 8 + ((lane >> 3) & 1)));
              else
                ldsm4_t(bf[b][p], RankTile<RP>::template at<KC>(wt, 64 * kh + kk + (lane & 7) + ((lane >> 3) & 1) * 8, 2 * p + (lane >> 4)));
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
        release(&ring.empty[ring.slot]);
        ring.next();
#pragma unroll
        for (int i = 0; i < 2 * RP; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[i][e] = __fadd_rn(sum[i][e], acc[i][e]);
      }
      // this adapter's rows: the second half's sums, then the first's on top
#pragma unroll
      for (int turn = 1; turn >= 0; --turn) {
        if (kh == turn) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int row = 16 * rg + (lane >> 2) + 8 * half;
            if (ta.ids[row] == id) {
#pragma unroll
              for (int i = 0; i < 2 * RP; ++i) {
                float2* at = reinterpret_cast<float2*>(sums + row * R + 8 * i + 2 * (lane & 3));
                float2 v = make_float2(sum[i][2 * half], sum[i][2 * half + 1]);
                if (turn == 0) v = make_float2(__fadd_rn(v.x, at->x), __fadd_rn(v.y, at->y));
                *at = v;
              }
            }
          }
        }
        consumers_sync();
      }
    }
  }
  // the cluster's sums, in rank order; each CTA finishes a share of the rows
  if (split > 1) cluster_barrier();
  else __syncthreads();
  const int first = kRows * rank / split, rows = kRows * (rank + 1) / split - first;
  for (int k = th; k < rows * R; k += kThreads) {
    const int row = first + k / R, j = k % R;
    const int64_t t = row0 + row;
    if (t >= a.T) continue;
    const float v = split == 1 ? sums[row * R + j] : sum_cluster(sums + row * R + j, split);
    if (w_out && j < r) w_out[t * r + j] = v;
    if (w_terms) write_terms(w_terms, n_terms, a.T, R, t, j, v);
    if (h_terms) write_terms(h_terms, n_terms, a.T, R, t, j, j < r ? __ldg(h + t * r + j) : 0.0f);
  }
  if (split > 1) cluster_barrier();   // no CTA leaves while another may still read its sums
}

// ---------------------------------------------------------------------------
// expand: out[t, c] = base[t, c] + s_a sum_j w[t, j] W[c, j].
// TRANS: W is stored [r, C], else [C, r].
// A CTA takes 64 rows and every groups-th tile of 128 columns, so that the
// CTAs at work read and write neighbouring columns at a time.  One ring holds
// base tiles (TMA in, changed in place, TMA out), another the weights of the
// rows' adapters, one slot each; w stays in registers, its scale folded in.
// Warp w: rows 16 (w % 4), columns 64 (w / 4) of a tile.
// Memory bounds it: 8192 x 14336, r = 16 92 us (5.1 TB/s read and written).
// ---------------------------------------------------------------------------
template <int RP>
struct ExpandCfg {
  static constexpr int R = 16 * RP;
  static constexpr int KC = 128;                  // columns of a tile
  static constexpr int YB = kRows * KC * 2;       // two boxes of 64 columns
  static constexpr int WB = R * KC * 2;
  static constexpr int CTAS = RP <= 4 ? 2 : 1;    // per SM
  static constexpr int WSLOTS = RP <= 2 ? 3 : (RP == 4 ? 2 : 4);
  static constexpr int YSLOTS = ((CTAS == 2 ? 110 : 224) * 1024 - WSLOTS * WB) / YB;
  static constexpr int BYTES = 1024 + YSLOTS * YB + WSLOTS * WB + 512;
};

template <int RP, bool TRANS>
__global__ void __launch_bounds__(kThreads, ExpandCfg<RP>::CTAS)
    lora_expand_kernel(const __grid_constant__ CUtensorMap tmap_in, const __grid_constant__ CUtensorMap tmap_w,
                       const __grid_constant__ CUtensorMap tmap_out, const __nv_bfloat16* __restrict__ W,
                       const float* __restrict__ w,
                       const float* __restrict__ scaling, const AdapterIds a, int64_t C, int r, int has_in, int groups) {
  // launched right behind the shrink kernel: all but w is older than that, so
  // the producer and the adapters need not wait for it (see pdl_entry below)
  using S = ExpandCfg<RP>;
  [[maybe_unused]] constexpr int R = S::R, KC = S::KC;
  extern __shared__ uint8_t dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
  uint8_t* ys = smem;
  uint8_t* wsm = ys + S::YSLOTS * S::YB;
  uint64_t* bars = reinterpret_cast<uint64_t*>(wsm + S::WSLOTS * S::WB);
  Ring yr{bars, bars + S::YSLOTS, S::YSLOTS};
  Ring wr{bars + 2 * S::YSLOTS, bars + 2 * S::YSLOTS + S::WSLOTS, S::WSLOTS};
  Abort* abort = reinterpret_cast<Abort*>(bars + 2 * (S::YSLOTS + S::WSLOTS));
  __shared__ TileAdapters ta;
  const int th = threadIdx.x, lane = th & 31, warp = th >> 5;
  const int group = static_cast<int>(blockIdx.x) % groups;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / groups) * kRows;
  if (th == 0) {
    yr.init();
    wr.init();
    abort->flag = 0;
    abort->limit_ns = a.wait_ns;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tile_adapters(ta, th < kRows ? adapter_of(a, row0 + th, false) : -1);   // ends with a barrier
  const int stride = groups * KC;   // between this CTA's columns
  if (warp == kConsumers) {
    int y_issued = 0, w_issued = 0;
    if (lane == 0) {
      for (int c = group * KC; c < C && !abort->flag; c += stride) {
        if (!yr.wait_empty(abort)) break;
        const uint32_t yb = smem_u32(&yr.full[yr.slot]), yd = smem_u32(ys + yr.slot * S::YB);
        if (has_in) {
          mbar_expect_tx(yb, S::YB);
          tma_load_2d(yd, &tmap_in, c, static_cast<int>(row0), yb);
          tma_load_2d(yd + S::YB / 2, &tmap_in, c + 64, static_cast<int>(row0), yb);
        } else {
          mbar_expect_tx(yb, 0);
        }
        yr.next();
        ++y_issued;
        for (int u = 0; u < ta.count; ++u) {
          if (!wr.wait_empty(abort)) break;
          const uint32_t wb = smem_u32(&wr.full[wr.slot]), wd = smem_u32(wsm + wr.slot * S::WB);
          mbar_expect_tx(wb, S::WB);
          if constexpr (!TRANS) {
            load_ranks<RP, KC>(wd, &tmap_w, W, ta.list[u], c, C, r, wb);
          } else {
            tma_load_3d(wd, &tmap_w, c, 0, ta.list[u], wb);
            tma_load_3d(wd + S::WB / 2, &tmap_w, c + 64, 0, ta.list[u], wb);
          }
          wr.next();
          ++w_issued;
        }
      }
    }
    __syncwarp();
    pdl_entry();
    if (lane == 0) {
      yr.drain(y_issued);
      wr.drain(w_issued);
    }
  } else {
    const int rg = warp & 3, ch = warp >> 2;
    const int my_row = 16 * rg + (lane >> 2);   // this thread's rows of the tile: my_row and my_row + 8
    const int id_lo = ta.ids[my_row], id_hi = ta.ids[my_row + 8];
    pdl_entry();
    // w of this warp's rows as MMA operands: hi and lo parts of s_a w
    uint32_t ah[RP][4], al[RP][4];
    const float s_lo = id_lo >= 0 ? __ldg(scaling + id_lo) : 0.0f, s_hi = id_hi >= 0 ? __ldg(scaling + id_hi) : 0.0f;
#pragma unroll
    for (int p = 0; p < RP; ++p)
#pragma unroll
      for (int e = 0; e < 4; ++e) {   // row + 8 (e % 2), ranks 16 p + 2 (lane % 4) + 8 (e / 2), + 1
        const int id = e & 1 ? id_hi : id_lo, j = 16 * p + 2 * (lane & 3) + 8 * (e >> 1);
        float2 v = make_float2(0.0f, 0.0f);
        if (id >= 0 && j < r) v = __ldcg(reinterpret_cast<const float2*>(w + (row0 + my_row + 8 * (e & 1)) * r + j));
        const float s = e & 1 ? s_hi : s_lo;
        __nv_bfloat16 h0, l0, h1, l1;
        split_bf16(id >= 0 ? __fmul_rn(s, v.x) : 0.0f, h0, l0);
        split_bf16(id >= 0 ? __fmul_rn(s, v.y) : 0.0f, h1, l1);
        ah[p][e] = pack_bf16(h0, h1);
        al[p][e] = pack_bf16(l0, l1);
      }
    int held = -1;   // base slot whose store may still be reading it
    for (int c0 = group * KC; c0 < C; c0 += stride) {
      yr.wait_full(abort, a.status);
      uint8_t* yt = ys + yr.slot * S::YB + ch * (S::YB / 2);   // this half's box of 64 columns
      if (!has_in) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(yt + (16 * rg) * 128 + 16 * (lane + 32 * i)) = make_uint4(0u, 0u, 0u, 0u);
        __syncwarp();
      }
      for (int u = 0; u < ta.count; ++u) {
        wr.wait_full(abort, a.status);
        const int id = ta.list[u];
        const uint8_t* wt = wsm + wr.slot * S::WB;
        const bool lo_mine = id_lo == id, hi_mine = id_hi == id;
        if (__any_sync(0xFFFFFFFFu, lo_mine || hi_mine)) {
#pragma unroll(RP == 4 ? 2 : 4)   // registers (forward, r = 64: 196 us with 4)
          for (int n = 0; n < 64; n += 16) {   // columns of this half
            float acc[2][4] = {}, low[2][4] = {};   // hi and lo parts apart: two shorter chains
#pragma unroll
            for (int p = 0; p < RP; ++p) {
              uint32_t bf[4];
              if constexpr (!TRANS)
                ldsm4(bf, RankTile<RP>::template at<KC>(wt, 64 * ch + n + (lane & 7) + ((lane >> 4) << 3), 2 * p + ((lane >> 3) & 1)));
              else
                ldsm4_t(bf, chunk_at<128>(wt + ch * (S::WB / 2), 16 * p + (lane & 7) + ((lane >> 3) & 1) * 8, n / 8 + (lane >> 4)));
              mma16(low[0], al[p], bf);
              mma16(low[1], al[p], bf + 2);
              mma16(acc[0], ah[p], bf);
              mma16(acc[1], ah[p], bf + 2);
            }
            // a token without an adapter keeps the base's bits (a NaN's payload, a zero's sign)
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const float2 d = __fadd2_rn(make_float2(acc[q][2 * half], acc[q][2 * half + 1]),
                                            make_float2(clamp(low[q][2 * half]), clamp(low[q][2 * half + 1])));
                if (half ? hi_mine : lo_mine) {
                  uint32_t* at = reinterpret_cast<uint32_t*>(chunk_at<128>(yt, my_row + 8 * half, n / 8 + q)) + (lane & 3);
                  *at = add_round(*at, d.x, d.y);
                }
              }
          }
        }
        release(&wr.empty[wr.slot]);
        wr.next();
      }
      fence_proxy_async_smem();
      __syncwarp();
      // store this warp's part; the previous tile's store has read its slot by
      // now (a part that lies outside makes no store, so all are waited for)
      const bool inside = c0 + 64 * ch < C && row0 + 16 * rg < a.T;
      if (lane == 0) {
        if (inside) {
          tma_store_2d(&tmap_out, smem_u32(yt + 16 * rg * 128), c0 + 64 * ch, static_cast<int>(row0) + 16 * rg);
          bulk_commit();
          bulk_wait_read<1>();
        } else {
          bulk_wait_read<0>();
        }
      }
      if (held >= 0) release(&yr.empty[held]);
      held = yr.slot;
      yr.next();
    }
    if (lane == 0) bulk_wait_all();
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

// grid: split (a cluster), unit.  Warp w takes the 32-column blocks w, w + 4,
// .. of the split; thread c of a quad holds columns 8c .. 8c + 7 of a block.
// The cluster's sums are added in rank order.  Latency bounds it, as it does
// the expand of few tokens: 64 tokens of 32 adapters, 4096 -> 14336, r = 16:
// 10 us each, 20 us in all.
template <int RP>
__global__ void __launch_bounds__(128) lora_shrink_few_kernel(const __nv_bfloat16* __restrict__ z, int64_t ldz,
                                                              const __nv_bfloat16* __restrict__ W, const AdapterIds a,
                                                              int64_t C, int r, int64_t per_split,
                                                              float* __restrict__ h) {
  pdl_entry();
  constexpr int R = 16 * RP;
  __shared__ __align__(16) Unit un;
  __shared__ float sums[4][16][R + 4];
  __shared__ float total[16][R];
  const int th = threadIdx.x, lane = th & 31, warp = th >> 5, g = lane >> 2, c = lane & 3;
  if (!find_unit(un, a, blockIdx.y, blockIdx.x == 0)) return;
  if (un.id < 0) {   // tokens without an adapter; the whole cluster leaves
    if (blockIdx.x == 0)
      for (int k = th; k < 16 * r; k += 128)
        if (un.member[k / r] >= 0) h[static_cast<int64_t>(un.member[k / r]) * r + k % r] = 0.0f;
    return;
  }
  const __nv_bfloat16* w = W + static_cast<int64_t>(un.id) * r * C;
  const int t0 = un.member[g], t1 = un.member[g + 8];
  const int64_t c_begin = blockIdx.x * per_split, c_end = min(c_begin + per_split, C);
  float acc[2 * RP][4] = {};
  // the loads of kBlocks blocks are in flight together
  constexpr int kBlocks = RP == 1 ? 4 : (RP == 2 ? 2 : 1);
  for (int64_t c0 = c_begin + 32 * warp; c0 < c_end; c0 += 128 * kBlocks) {
    uint4 a0[kBlocks], a1[kBlocks], b[kBlocks][2 * RP];
#pragma unroll
    for (int x = 0; x < kBlocks; ++x) {
      const int64_t cc = c0 + 128 * x + 8 * c;
      const bool ok = cc < c_end;
      a0[x] = load16(z + t0 * ldz + cc, ok && t0 >= 0);
      a1[x] = load16(z + t1 * ldz + cc, ok && t1 >= 0);
#pragma unroll
      for (int i = 0; i < 2 * RP; ++i) b[x][i] = load16(w + (8 * i + g) * C + cc, ok && 8 * i + g < r);
    }
#pragma unroll
    for (int x = 0; x < kBlocks; ++x) {
      const uint32_t f0[4] = {a0[x].x, a1[x].x, a0[x].y, a1[x].y}, f1[4] = {a0[x].z, a1[x].z, a0[x].w, a1[x].w};
#pragma unroll
      for (int i = 0; i < 2 * RP; ++i) {
        float run[4] = {};   // short runs on the tensor core, fp32 sums outside
        const uint32_t b0[2] = {b[x][i].x, b[x][i].y}, b1[2] = {b[x][i].z, b[x][i].w};
        mma16(run, f0, b0);
        mma16(run, f1, b1);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = __fadd_rn(acc[i][e], run[e]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2 * RP; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) sums[warp][g + 8 * (e >> 1)][8 * i + 2 * c + (e & 1)] = acc[i][e];
  __syncthreads();
  for (int k = th; k < 16 * R; k += 128) {
    const int row = k / R, j = k % R;
    total[row][j] = __fadd_rn(__fadd_rn(sums[0][row][j], sums[1][row][j]), __fadd_rn(sums[2][row][j], sums[3][row][j]));
  }
  const int split = gridDim.x, rank = blockIdx.x;
  cluster_barrier();
  const int begin = 16 * R * rank / split, end = 16 * R * (rank + 1) / split;
  for (int k = begin + th; k < end; k += 128) {
    const int row = k / R, j = k % R, t = un.member[row];
    if (t < 0 || j >= r) continue;
    h[static_cast<int64_t>(t) * r + j] = sum_cluster(&total[row][j], split);
  }
  cluster_barrier();   // no CTA leaves while another may still read its sums
}

// grid: 512 columns, unit.  Warp w takes 128 of the columns.
constexpr int kFewCols = 512;

template <int RP>
__global__ void __launch_bounds__(128) lora_expand_few_kernel(const float* __restrict__ h,
                                                              const __nv_bfloat16* __restrict__ W,
                                                              const float* __restrict__ scaling, const AdapterIds a,
                                                              int64_t C, int r, const __nv_bfloat16* in, int64_t ldi,
                                                              __nv_bfloat16* out, int64_t ldo) {
  // launched right behind the shrink kernel: all but h is older than that
  constexpr int R = 16 * RP;
  __shared__ __align__(16) Unit un;
  __shared__ __align__(16) float hs[16][R + 4];   // read as float4
  const int th = threadIdx.x, lane = th & 31, warp = th >> 5, g = lane >> 2, c = lane & 3;
  if (!find_unit(un, a, blockIdx.y, false)) {
    pdl_entry();
    return;
  }
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
  pdl_entry();
  for (int k = th; k < 16 * R; k += 128) {
    const int row = k / R, j = k % R, t = un.member[row];
    const float v = (t >= 0 && j < r) ? __ldcg(h + static_cast<int64_t>(t) * r + j) : 0.0f;
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
        __nv_bfloat16 hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split_bf16(__fmul_rn(s, vv[e]), hi[e], lo[e]);
        ah[p][half] = pack_bf16(hi[0], hi[1]);
        ah[p][2 + half] = pack_bf16(hi[2], hi[3]);
        al[p][half] = pack_bf16(lo[0], lo[1]);
        al[p][2 + half] = pack_bf16(lo[2], lo[3]);
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
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][e] = clamp(acc[m][e]);
#pragma unroll
        for (int p = 0; p < RP; ++p) {
          const uint32_t bb[2] = {b[p].x, b[p].y};
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
// rows, in tiles of 32.  Rows of other adapters in a tile are made zero before
// it is used, w's too, so that a NaN there reaches nothing.  Two products
// share a launch: dA (z = x, w = g, stored [r, C]) and dB (z = dy, w = h,
// stored [C, r]).
// grid: column tiles of both products, adapter, split of the rows.
// TERMS: bf16 numbers that w enters as: 3 (all of fp32) for fp32 gradients,
// 2 (2^-17) for bf16 ones, as the shrink kernel wrote them.
// Where a sum is NaN, an infinite z may have met lower terms of the other sign
// or of zero: a second walk over the rows, with the leading terms alone, gives
// those elements what the formula does.
// x 8192 x 4096 and dy 8192 x 14336, r = 16, fp32: 81 us (3.8 TB/s; tensor pipe
// 43% busy with the three terms).  Neither is at its limit: a CTA takes one
// adapter's tokens of a range of rows, and the longest run sets the time.
// ---------------------------------------------------------------------------
struct OuterProduct {
  int64_t C;
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

constexpr int kRowsO = 32;                   // rows of a tile
constexpr int kWindow = 64 * kRowsO;         // rows whose ids a CTA looks at together

template <int RP, int TERMS>
struct OuterCfg {
  static constexpr int R = 16 * RP;
  static constexpr int NQ = RP <= 2 ? 2 : 1;          // 16-column groups of a warp
  static constexpr int COLS = kConsumers * 16 * NQ;   // columns of a tile
  static constexpr int ZBOX = kRowsO * 128;           // 64 columns
  static constexpr int ZB = COLS / 64 * ZBOX;
  static constexpr int HB = kRowsO * R * 2;
  static constexpr int STAGE = ZB + TERMS * HB;
  static constexpr int CTAS = RP <= 4 ? 2 : 1;        // per SM
  static constexpr int STAGES = (CTAS == 2 ? 100 : 200) * 1024 / STAGE;
  static constexpr int BYTES = 1024 + STAGES * STAGE + 256;
};

__device__ __forceinline__ void store_out(void* dst, int64_t at, float v, bool fp32) {
  if (fp32) static_cast<float*>(dst)[at] = v;
  else static_cast<__nv_bfloat16*>(dst)[at] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ bool is_nan(const void* src, int64_t at, bool fp32) {
  return fp32 ? isnan(static_cast<const float*>(src)[at]) : __hisnan(static_cast<const __nv_bfloat16*>(src)[at]);
}

// A CTA's walk over its rows: where it reads and writes, and how far its ring is.
struct OuterWalk {
  uint8_t* smem;
  int *ids, *list, *listed;   // of a window: its rows' adapters; its tiles with a token of this adapter (bit 8: all are), how many
  Abort* abort;
  const CUtensorMap *map_z, *map_w;
  int c0, id, split, splits;
  int64_t first, last;        // tiles
  Ring ring;
  int issued;
  bool any;                   // a token of this adapter was seen
};

// Sums over the rows, and their store.  Returns whether a sum is NaN.  LEAD: with
// the leading terms alone, storing where the memory holds a NaN.
template <int RP, int TERMS, bool LEAD>
__device__ __forceinline__ bool outer_walk(OuterWalk& v, const OuterArgs& o, const OuterProduct& p) {
  using S = OuterCfg<RP, TERMS>;
  using Ranks = RankTile<RP>;
  [[maybe_unused]] constexpr int R = S::R, COLS = S::COLS, NQ = S::NQ;
  constexpr int kRankBox = kRowsO * Ranks::ROW;   // one term's rows in a box
  const int th = threadIdx.x, lane = th & 31, warp = th >> 5, id = v.id, r = o.r;
  float sum[RP][2 * NQ][4];
#pragma unroll
  for (int m = 0; m < RP; ++m)
#pragma unroll
    for (int q = 0; q < 2 * NQ; ++q) sum[m][q][0] = sum[m][q][1] = sum[m][q][2] = sum[m][q][3] = 0.0f;

  for (int64_t base = v.first; base < v.last; base += kWindow / kRowsO) {
    const int n_tiles = static_cast<int>(v.last - base < kWindow / kRowsO ? v.last - base : kWindow / kRowsO);
    const int64_t row_base = base * kRowsO;
    // the previous window's ids and list have been read; after an abort all leave
    if (__syncthreads_or(v.abort->flag != 0)) break;
    for (int k = th; k < n_tiles * kRowsO; k += kThreads) v.ids[k] = adapter_of(o.a, row_base + k, false);
    __syncthreads();
    if (warp == 0) {
      int n = 0;
      for (int first_tile = 0; first_tile < n_tiles; first_tile += 32) {
        const int tile = first_tile + lane;
        bool some = false, all = true;
        if (tile < n_tiles)
          for (int k = 0; k < kRowsO / 4; ++k) {
            // lanes start at different places: fewer bank conflicts
            const int4 four = *reinterpret_cast<const int4*>(&v.ids[tile * kRowsO + 4 * ((k + lane) % (kRowsO / 4))]);
            some |= four.x == id || four.y == id || four.z == id || four.w == id;
            all &= four.x == id && four.y == id && four.z == id && four.w == id;
          }
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, some);
        if (some) v.list[n + __popc(m & ((1u << lane) - 1u))] = tile | (all ? 256 : 0);
        n += __popc(m);
      }
      if (lane == 0) *v.listed = n;
    }
    __syncthreads();
    const int count = *v.listed;
    v.any |= count > 0;

    if (warp == kConsumers) {
      if (lane == 0) {
        for (int k = 0; k < count; ++k, ++v.issued, v.ring.next()) {
          if (!v.ring.wait_empty(v.abort)) break;
          const uint32_t bar = smem_u32(&v.ring.full[v.ring.slot]), zd = smem_u32(v.smem + v.ring.slot * S::STAGE), wd = zd + S::ZB;
          const int row = static_cast<int>(row_base) + (v.list[k] & 255) * kRowsO;
          mbar_expect_tx(bar, S::STAGE);
#pragma unroll
          for (int b = 0; b < COLS / 64; ++b) tma_load_2d(zd + b * S::ZBOX, v.map_z, v.c0 + 64 * b, row, bar);
          // all terms in one copy (a tensor copy costs some 100 ns, however small)
#pragma unroll
          for (int b = 0; b < Ranks::BOXES; ++b) tma_load_3d(wd + b * TERMS * kRankBox, v.map_w, 64 * b, row, 0, bar);
        }
      }
      __syncwarp();
    } else {
      for (int k = 0; k < count; ++k) {
        v.ring.wait_full(v.abort, o.a.status);
        uint8_t* zs = v.smem + v.ring.slot * S::STAGE;
        uint8_t* wb = zs + S::ZB;
        const bool mixed = !(v.list[k] & 256);
        if (mixed) {   // zeros in the place of other adapters' rows (a row's chunks are its own, whatever their order)
          const int* row_ids = v.ids + (v.list[k] & 255) * kRowsO;
          for (int e = th; e < S::STAGE / 16; e += 32 * kConsumers) {
            const int at = 16 * e;
            const int row = at < S::ZB ? at % S::ZBOX / 128 : (at - S::ZB) % (kRowsO * Ranks::ROW) / Ranks::ROW;
            if (row_ids[row] != id) *reinterpret_cast<uint4*>(zs + at) = make_uint4(0u, 0u, 0u, 0u);
          }
          consumers_sync();
        }
        // kPair groups of 16 ranks at a time: their chains of products overlap
        constexpr int kPair = RP >= 2 ? 2 : 1;
#pragma unroll
        for (int m0 = 0; m0 < RP; m0 += kPair) {
          float acc[kPair][2 * NQ][4];
#pragma unroll
          for (int m = 0; m < kPair; ++m)
#pragma unroll
            for (int q = 0; q < 2 * NQ; ++q) acc[m][q][0] = acc[m][q][1] = acc[m][q][2] = acc[m][q][3] = 0.0f;
#pragma unroll
          for (int kk = 0; kk < kRowsO; kk += 16) {
            uint32_t af[kPair][TERMS][4], bf[NQ][4];
            const int arow = kk + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
              const int chunk = 2 * (NQ * warp + q) + (lane >> 4);   // of eight columns
              ldsm4_t(bf[q], chunk_at<128>(zs + (chunk >> 3) * S::ZBOX, kk + (lane & 7) + ((lane >> 3) & 1) * 8, chunk & 7));
            }
#pragma unroll
            for (int m = 0; m < kPair; ++m)
#pragma unroll
              for (int x = 0; x < (LEAD ? 1 : TERMS); ++x)
                ldsm4_t(af[m][x], Ranks::template at<TERMS * kRowsO>(wb, x * kRowsO + arow, 2 * (m0 + m) + ((lane >> 3) & 1)));
#pragma unroll
            for (int x = LEAD ? 0 : TERMS - 1; x >= 0; --x)
#pragma unroll
              for (int m = 0; m < kPair; ++m)
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                  mma16(acc[m][2 * q], af[m][x], bf[q]);
                  mma16(acc[m][2 * q + 1], af[m][x], bf[q] + 2);
                }
          }
#pragma unroll
          for (int m = 0; m < kPair; ++m)
#pragma unroll
            for (int q = 0; q < 2 * NQ; ++q)
#pragma unroll
              for (int e = 0; e < 4; ++e) sum[m0 + m][q][e] = __fadd_rn(sum[m0 + m][q][e], acc[m][q][e]);
        }
        if (mixed) fence_proxy_async_smem();   // the zeros were plain stores, the next copy is not
        release(&v.ring.empty[v.ring.slot]);
        v.ring.next();
      }
    }
  }
  bool nan = false;
  const bool direct = v.splits == 1;
  if (warp == kConsumers || (!direct && !v.any)) return nan;
  // with splits the sum is scaled once, at the end; the scale of an adapter
  // without tokens says nothing
  const float s = !direct ? 1.0f : v.any ? __ldg(o.scaling + id) : 0.0f;
#pragma unroll
  for (int m = 0; m < RP; ++m)
#pragma unroll
    for (int q = 0; q < 2 * NQ; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = 16 * m + (lane >> 2) + 8 * (e >> 1);
        const int64_t c = v.c0 + 16 * NQ * warp + 8 * q + 2 * (lane & 3) + (e & 1);
        if (j < r && c < p.C) {
          const int64_t at = p.cols_first ? (static_cast<int64_t>(id) * p.C + c) * r + j : (static_cast<int64_t>(id) * r + j) * p.C + c;
          float* part = p.part + static_cast<int64_t>(v.split) * o.a.n * r * p.C + at;
          if constexpr (LEAD) {
            if (!(direct ? is_nan(p.dst, at, o.fp32) : isnan(*part))) continue;
          } else {
            nan |= isnan(sum[m][q][e]);
          }
          if (direct) store_out(p.dst, at, __fmul_rn(s, sum[m][q][e]), o.fp32);
          else *part = sum[m][q][e];
        }
      }
  return nan;
}

// Apart, so that the first walk keeps its registers; returns the slots issued.
template <int RP, int TERMS>
__device__ __noinline__ int outer_again(OuterWalk v, const OuterArgs& o, const OuterProduct& p) {
  outer_walk<RP, TERMS, true>(v, o, p);
  return v.issued;
}

template <int RP, int TERMS>
__global__ void __launch_bounds__(kThreads, OuterCfg<RP, TERMS>::CTAS)
    lora_outer_kernel(const __grid_constant__ CUtensorMap tmap_z0, const __grid_constant__ CUtensorMap tmap_w0,
                      const __grid_constant__ CUtensorMap tmap_z1, const __grid_constant__ CUtensorMap tmap_w1,
                      const __grid_constant__ OuterArgs o) {
  pdl_entry();
  using S = OuterCfg<RP, TERMS>;
  extern __shared__ uint8_t dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::STAGES * S::STAGE);
  Ring ring{bars, bars + S::STAGES, S::STAGES};
  Abort* abort = reinterpret_cast<Abort*>(bars + 2 * S::STAGES);
  __shared__ __align__(16) int ids[kWindow];
  __shared__ int list[kWindow / kRowsO];
  __shared__ int listed;
  const int th = threadIdx.x;
  const bool second = static_cast<int>(blockIdx.x) >= o.p[0].tiles;
  const OuterProduct& p = o.p[second ? 1 : 0];
  const int splits = gridDim.z, split = blockIdx.z;
  const int64_t tiles = (o.a.T + kRowsO - 1) / kRowsO;
  if (th == 0) {
    ring.init();
    abort->flag = 0;
    abort->limit_ns = o.a.wait_ns;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();

  OuterWalk v{smem, ids, list, &listed, abort, second ? &tmap_z1 : &tmap_z0, second ? &tmap_w1 : &tmap_w0,
              (static_cast<int>(blockIdx.x) - (second ? o.p[0].tiles : 0)) * S::COLS, static_cast<int>(blockIdx.y), split, splits,
              tiles * split / splits, tiles * (split + 1) / splits, ring, 0, false};
  const bool nan = outer_walk<RP, TERMS, false>(v, o, p);
  if (__syncthreads_or(nan)) v.issued = outer_again<RP, TERMS>(v, o, p);
  if (th == 32 * kConsumers) v.ring.drain(v.issued);
  if (splits > 1 && th == 0) o.used[(static_cast<int64_t>(v.id) * splits + split) * gridDim.x + blockIdx.x] = v.any ? 1 : 0;
}

// Sum of the splits' partials, in their order, those that saw a token; four
// elements per thread.  Latency of dependent loads: 9 us for 2 x 4 x 16 x
// 18432 elements.
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
      bool any = false;
      for (int s = 0; s < splits; ++s)
        if (__ldcg(used + s * all_tiles)) {
          any = true;
          const float4 q = __ldcg(reinterpret_cast<const float4*>(p.part + s * total + k));
          v = make_float4(__fadd_rn(v.x, q.x), __fadd_rn(v.y, q.y), __fadd_rn(v.z, q.z), __fadd_rn(v.w, q.w));
        }
      const float sc = any ? __ldg(o.scaling + id) : 0.0f;
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

// Time limit of the rings' waits: the GEMMs' 2 s, or the nanoseconds in the
// environment variable NVFP4_WAIT_TIMEOUT_NS, read at every call (tests let
// the waits run out with it).
uint32_t wait_limit_ns() {
  if (const char* env = std::getenv("NVFP4_WAIT_TIMEOUT_NS")) {
    char* end = nullptr;
    const unsigned long long v = std::strtoull(env, &end, 10);
    if (end != env && *end == '\0') return static_cast<uint32_t>(std::min<unsigned long long>(v, kTimeoutNs));
  }
  return static_cast<uint32_t>(kTimeoutNs);
}

// A bf16 matrix [rows, cols] with row stride ld: boxes of 64 columns (128
// bytes, swizzled) x box_rows.
bool map_rows(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)}, estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// n contiguous bf16 matrices [rows, cols]: boxes of box_cols (16, or 32 or 64
// swizzled over their 64 or 128 bytes) x box_rows of box_n matrices.  What a
// box has outside a matrix reads as zeros.
bool map_stack(CUtensorMap* map, const void* base, int64_t n, int64_t rows, int64_t cols, int box_cols, int box_rows,
               int box_n = 1) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(n)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * 2, static_cast<cuuint64_t>(rows * cols) * 2};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows),
                             static_cast<cuuint32_t>(box_n)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapSwizzle swizzle =
      box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : (box_cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE);
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
int rank_box(int rp) { return rp >= 4 ? 64 : 16 * rp; }   // ranks of a RankTile's box

// Units that T tokens and n adapters (and "none") can make.
int64_t most_units(int64_t T, int64_t n) { return std::min<int64_t>(n + 1, T) + T / 16; }

// CTAs that share a row tile's columns (a cluster): enough for one on every
// SM, and beyond that 32 stages each (a CTA's start and the cluster's meeting
// cost a few stages): backward of 8192 tokens, 14336 columns, with 8, 16, 32
// stages: r = 16 223, 214, 207 us, r = 64 465, 430, 418 us.
constexpr int kShrinkStages = 32;
int shrink_split(int64_t T, int64_t C) {
  const int64_t rows = ceil_div(T, kRows), stages = ceil_div(C, 128);
  int s = 1;
  while (s < 8 && stages >= 2 * s && (rows * s < sm_count() || stages >= kShrinkStages * 2 * s)) s *= 2;
  return s;
}
int few_split(int64_t C) { return C >= 1024 ? 8 : (C >= 512 ? 4 : (C >= 256 ? 2 : 1)); }

int outer_cols(int64_t r) { return r <= 32 ? 256 : 128; }
// Row ranges of the outer products, for an adapter that owns most tokens: at
// most 4096 tokens each, unless that makes more than 8.  (Backward of 8192
// tokens, r = 16, ranges of 1024, 2048, 4096: 209, 214, 186 us.)
int outer_splits(int64_t T) { return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(8, ceil_div(T, 4096)))); }

// Parts of the workspace, in 16-byte steps: h where the caller keeps none, or
// g, the terms of both and the outer products' partial sums.
struct LoraWorkspace {
  size_t g, g_terms, h_terms, outer_a, outer_b, used, total;
};
size_t up16(size_t v) { return (v + 15) & ~static_cast<size_t>(15); }
int64_t padded_rank(int64_t r) { return r <= 16 ? 16 : (r <= 32 ? 32 : (r <= 64 ? 64 : 128)); }
LoraWorkspace lora_workspace(int64_t T, int64_t K, int64_t N, int64_t r, int64_t n, bool backward) {
  LoraWorkspace w{};
  w.g = 0;
  w.total = up16(static_cast<size_t>(T * r) * 4);
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

// W: [n, r, C], TRANS: [n, C, r]
template <int RP, bool TRANS>
cudaError_t shrink(const __nv_bfloat16* z, int64_t ldz, const __nv_bfloat16* W, const AdapterIds& a, int64_t C, int64_t r,
                   float* w_out, __nv_bfloat16* w_terms, const float* h, __nv_bfloat16* h_terms, int n_terms,
                   cudaStream_t st) {
  using S = ShrinkCfg<RP, TRANS>;
  auto fn = lora_shrink_kernel<RP, TRANS>;
  static bool done[64] = {false};
  cudaError_t e = allow_smem(fn, S::BYTES, done);
  if (e != cudaSuccess) return e;
  CUtensorMap mz, mw;
  if (!map_rows(&mz, z, a.T, C, ldz, kRows) ||
      !(TRANS ? map_stack(&mw, W, a.n, C, r, rank_box(RP), S::KC) : map_stack(&mw, W, a.n, r, C, 64, S::R)))
    return cudaErrorInvalidValue;
  const int split = shrink_split(a.T, C);
  e = launch_k(fn, dim3(static_cast<unsigned>(ceil_div(a.T, kRows) * split)), dim3(kThreads), S::BYTES, st,
               static_cast<unsigned>(split), mz, mw, W, a, C, static_cast<int>(r), split, w_out, w_terms, h, h_terms, n_terms);
  note_launch();
  return e;
}

// Column tiles of a CTA, where that leaves enough CTAs: forward of 8192 tokens
// 4096 -> 14336 with 2, 4, 7, 14: r = 16 163, 136, 124, 120 us, r = 64 275,
// 222, 191, 175 us.
constexpr int64_t kExpandTiles = 14;

// W: [n, C, r], TRANS: [n, r, C]
template <int RP, bool TRANS>
cudaError_t expand(const float* w, const __nv_bfloat16* W, const float* scaling, const AdapterIds& a, int64_t C, int64_t r,
                   const __nv_bfloat16* in, int64_t ldi, __nv_bfloat16* out, int64_t ldo, cudaStream_t st) {
  using S = ExpandCfg<RP>;
  auto fn = lora_expand_kernel<RP, TRANS>;
  static bool done[64] = {false};
  cudaError_t e = allow_smem(fn, S::BYTES, done);
  if (e != cudaSuccess) return e;
  CUtensorMap mi, mw, mo;
  if (!map_rows(&mo, out, a.T, C, ldo, 16) || !map_rows(&mi, in ? in : out, a.T, C, in ? ldi : ldo, kRows) ||
      !(TRANS ? map_stack(&mw, W, a.n, r, C, 64, S::R) : map_stack(&mw, W, a.n, C, r, rank_box(RP), S::KC)))
    return cudaErrorInvalidValue;
  const int64_t rows = ceil_div(a.T, kRows), cols = ceil_div(C, S::KC);
  const int groups = static_cast<int>(ceil_div(cols, std::max<int64_t>(1, std::min<int64_t>(kExpandTiles, rows * cols / (S::CTAS * sm_count())))));
  e = launch_k(fn, dim3(static_cast<unsigned>(rows * groups)), dim3(kThreads), S::BYTES, st, 1u, mi, mw, mo, W, w, scaling, a, C,
               static_cast<int>(r), in ? 1 : 0, groups);
  note_launch();
  return e;
}

template <int RP, int TERMS>
cudaError_t outer(const LoraArgs& l, const AdapterIds& a, uint8_t* ws, const LoraWorkspace& w, cudaStream_t st) {
  using S = OuterCfg<RP, TERMS>;
  auto fn = lora_outer_kernel<RP, TERMS>;
  static bool done[64] = {false};
  cudaError_t e = allow_smem(fn, S::BYTES, done);
  if (e != cudaSuccess) return e;
  const int64_t ka = l.dA ? ceil_div(l.K, S::COLS) : 0, kb = l.dB ? ceil_div(l.N, S::COLS) : 0;
  OuterArgs o{};
  o.p[0] = OuterProduct{l.K, l.dA, reinterpret_cast<float*>(ws + w.outer_a), static_cast<int>(ka), 0};
  o.p[1] = OuterProduct{l.N, l.dB, reinterpret_cast<float*>(ws + w.outer_b), static_cast<int>(kb), 1};
  o.scaling = l.scaling;
  o.a = a;
  o.r = static_cast<int>(l.r);
  o.fp32 = l.fp32 ? 1 : 0;
  o.used = reinterpret_cast<int32_t*>(ws + w.used);
  CUtensorMap mz[2], mw[2];
  const int R = S::R;
  // a product that is not asked for has no tiles; its maps are the other's
  const bool both = l.dA && l.dB;
  const __nv_bfloat16* z[2] = {l.dA ? l.x : l.dy, l.dB ? l.dy : l.x};
  const int64_t ld[2] = {l.dA ? l.ldx : l.lddy, l.dB ? l.lddy : l.ldx}, C[2] = {l.dA ? l.K : l.N, l.dB ? l.N : l.K};
  const uint8_t* terms[2] = {ws + (l.dA ? w.g_terms : w.h_terms), ws + (l.dB ? w.h_terms : w.g_terms)};
  for (int i = 0; i < 2; ++i) {
    if (i == 1 && !both) {
      mz[1] = mz[0];
      mw[1] = mw[0];
    } else if (!map_rows(&mz[i], z[i], a.T, C[i], ld[i], kRowsO) ||
               !map_stack(&mw[i], terms[i], TERMS, a.T, R, rank_box(RP), kRowsO, TERMS)) {
      return cudaErrorInvalidValue;
    }
  }
  const int splits = outer_splits(a.T);
  const dim3 grid(static_cast<unsigned>(ka + kb), static_cast<unsigned>(a.n), static_cast<unsigned>(splits));
  e = launch_k(fn, grid, dim3(kThreads), S::BYTES, st, 1u, mz[0], mw[0], mz[1], mw[1], o);
  note_launch();
  if (e != cudaSuccess || splits == 1) return e;
  const int64_t most = l.n * l.r * std::max(l.dA ? l.K : 0, l.dB ? l.N : 0);
  const int64_t blocks = std::min<int64_t>(ceil_div(most, 1024), 8 * sm_count());
  e = launch_k(lora_outer_sum_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, 1u, o, splits, S::COLS);
  note_launch();
  return e;
}

template <int RP>
cudaError_t forward(const LoraArgs& l, float* h, cudaStream_t st) {
  const AdapterIds a{l.ids, l.T, static_cast<int>(l.n), l.status, l.T > kFewTokens ? wait_limit_ns() : 0u};
  const int r = static_cast<int>(l.r);
  if (l.T > kFewTokens) {
    const cudaError_t e = shrink<RP, false>(l.x, l.ldx, l.A, a, l.K, r, h, nullptr, nullptr, nullptr, 0, st);
    if (e != cudaSuccess) return e;
    return expand<RP, false>(h, l.B, l.scaling, a, l.N, r, l.in, l.ldi, l.out, l.ldo, st);
  }
  const unsigned units = static_cast<unsigned>(most_units(l.T, l.n));
  const int split = few_split(l.K);
  cudaError_t e = launch_k(lora_shrink_few_kernel<RP>, dim3(static_cast<unsigned>(split), units), dim3(128), 0, st,
                           static_cast<unsigned>(split), l.x, l.ldx, l.A, a, l.K, r,
                           ceil_div(ceil_div(l.K, split), 32) * 32, h);
  note_launch();
  if (e != cudaSuccess) return e;
  e = launch_k(lora_expand_few_kernel<RP>, dim3(static_cast<unsigned>(ceil_div(l.N, kFewCols)), units), dim3(128), 0, st,
               1u, h, l.B, l.scaling, a, l.N, r, l.in, l.ldi, l.out, l.ldo);
  note_launch();
  return e;
}

template <int RP>
cudaError_t backward(const LoraArgs& l, uint8_t* ws, const LoraWorkspace& w, cudaStream_t st) {
  const AdapterIds a{l.ids, l.T, static_cast<int>(l.n), l.status, wait_limit_ns()};
  const int n_terms = l.fp32 ? 3 : 2;
  float* g = reinterpret_cast<float*>(ws + w.g);
  __nv_bfloat16* g_terms = reinterpret_cast<__nv_bfloat16*>(ws + w.g_terms);
  __nv_bfloat16* h_terms = reinterpret_cast<__nv_bfloat16*>(ws + w.h_terms);
  // the shrink also writes h's terms, so it runs even where dB alone is asked for
  cudaError_t e = shrink<RP, true>(l.dy, l.lddy, l.B, a, l.N, l.r, l.out ? g : nullptr, l.dA ? g_terms : nullptr, l.h,
                                   l.dB ? h_terms : nullptr, n_terms, st);
  if (e == cudaSuccess && l.out)
    e = expand<RP, true>(g, l.A, l.scaling, a, l.K, l.r, l.in, l.ldi, l.out, l.ldo, st);
  if (e != cudaSuccess || (!l.dA && !l.dB)) return e;
  return l.fp32 ? outer<RP, 3>(l, a, ws, w, st) : outer<RP, 2>(l, a, ws, w, st);
}

}  // namespace

size_t lora_workspace_bytes(int64_t T, int64_t K, int64_t N, int64_t r, int64_t n, bool backward) {
  return T == 0 ? 0 : lora_workspace(T, K, N, r, n, backward).total;
}

cudaError_t lora_forward_launch(const LoraArgs& l, void* workspace, cudaStream_t st) {
  float* h = l.h ? l.h : static_cast<float*>(workspace);
  if (l.r <= 16) return forward<1>(l, h, st);
  if (l.r <= 32) return forward<2>(l, h, st);
  if (l.r <= 64) return forward<4>(l, h, st);
  return forward<8>(l, h, st);
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
