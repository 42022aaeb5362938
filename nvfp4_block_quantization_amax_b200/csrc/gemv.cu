// gemv.cu -- products of a few bf16 rows with NVFP4 weights.
//
//   y[p, n] = alpha_e sum_k x[p / rep, k] q[e, n, k] Delta[e, n, k / 16],   e = ids[p]
//
// What it cannot do without is the weight, 0.5625 bytes per value, read once for
// all rows that need it.  q Delta has at most 6 significant bits (2 of E2M1, 4 of
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
// Two kernels, by the rows that share a weight.  With up to 8 (one column group
// of a product) x is small beside the weight and is read from memory; with more
// it is not, and comes once per 128 weight rows.  24 rows, 4096 x 14336: 28 us in
// the first form (with three column groups), 22 in the second.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>

#include "launch.cuh"
#include "nvfp4_internal.h"
#include "smem.cuh"

namespace cg = cooperative_groups;

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

// Two E4M3 bytes of a word, picked by a byte selector, as bf16 pairs (each in
// both halves) times 2^118: a byte's bits e e e e, m m m at a bf16's bits 10 .. 7,
// 6 .. 4 are Delta 2^-120, denormals included (0x7F, which no quantizer writes,
// would be 480, not NaN).
__device__ __forceinline__ void scale_pairs(uint32_t word, uint32_t pick, uint32_t* s) {
  constexpr uint32_t up = 0x7B007B00u;   // 2^119 twice
  const uint32_t v = mul2(mul2(__byte_perm(word, 0u, pick) << 4, up), up);
  s[0] = __byte_perm(v, v, 0x1010);
  s[1] = __byte_perm(v, v, 0x3232);
}

// The eight codes of a word times their scale: pairs (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ void decode(uint32_t w, uint32_t s, uint32_t* q) {
  const uint32_t v = w >> 8;
  q[0] = mul2(((w & 0x000F000Fu) * 0x1040u) & 0x81C081C0u, s);
  q[1] = mul2(((w & 0x00F000F0u) * 0x0104u) & 0x81C081C0u, s);
  q[2] = mul2(((v & 0x000F000Fu) * 0x1040u) & 0x81C081C0u, s);
  q[3] = mul2(((v & 0x00F000F0u) * 0x0104u) & 0x81C081C0u, s);
}

__device__ const uint4 kNothing[4] = {};

// Codes and scales of one lane and 128 values of K: four rows' 16 bytes and
// the 16 bytes with their scales.
constexpr int kPieces = 5;

__device__ __forceinline__ void copy16(uint4* to, const uint8_t* from, bool real) {
  const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(to));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(from), "r"(real ? 16 : 0) : "memory");
}

// Pairs sorted by expert and cut into slots of at most kGroup pairs of one expert.
struct Slots {
  short pairs[1024];            // in the order of their experts
  short begin[1026];            // where an expert's begin
  short expert[1024], pass[1024];   // of a slot
  int counts[1024];
  int scan[2][kWarps];
  int number;
};

// Fill the tables, with all threads; ends with a barrier.  The number of slots.
template <int kGroup>
__device__ __forceinline__ int find_slots(const GemvArgs& a, Slots& t, bool report) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, P = static_cast<int>(a.P), E = static_cast<int>(a.E);
  for (int e = tid; e < E; e += kThreads) t.counts[e] = 0;
  __syncthreads();
  for (int p = tid; p < P; p += kThreads) {
    const int id = __ldg(a.ids + p);
    if (id >= 0 && id < E) atomicAdd(&t.counts[id], 1);
    else if (id != -1 && report && a.status) *a.status = kStatusArg;
  }
  __syncthreads();
  // where an expert's pairs and slots begin: four experts a thread
  int n[4], pairs = 0, passes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = tid * 4 + i;
    n[i] = e < E ? t.counts[e] : 0;
    pairs += n[i];
    passes += (n[i] + kGroup - 1) / kGroup;
  }
  int up = pairs, us = passes;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int vp = __shfl_up_sync(0xFFFFFFFFu, up, o), vs = __shfl_up_sync(0xFFFFFFFFu, us, o);
    if (lane >= o) {
      up += vp;
      us += vs;
    }
  }
  if (lane == 31) {
    t.scan[0][warp] = up;
    t.scan[1][warp] = us;
  }
  __syncthreads();
  int p0 = up - pairs, s0 = us - passes;
  for (int i = 0; i < warp; ++i) {
    p0 += t.scan[0][i];
    s0 += t.scan[1][i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = tid * 4 + i;
    if (e >= E) break;
    t.begin[e] = static_cast<short>(p0);
    t.counts[e] = p0;   // where its next pair goes
    p0 += n[i];
    for (int m = 0; m * kGroup < n[i]; ++m, ++s0) {
      t.expert[s0] = static_cast<short>(e);
      t.pass[s0] = static_cast<short>(m);
    }
    if (e == E - 1) {
      t.begin[E] = static_cast<short>(p0);
      t.number = s0;
    }
  }
  __syncthreads();
  if (warp == 0) {
    // an expert's pairs in order: every CTA cuts them into the same slots
    for (int p = lane; p < (P + 31) / 32 * 32; p += 32) {
      const int id = p < P ? __ldg(a.ids + p) : -1;
      const bool is = id >= 0 && id < E;
      const unsigned same = __match_any_sync(0xFFFFFFFFu, is ? id : -1);
      if (is) t.pairs[t.counts[id] + __popc(same & ((1u << lane) - 1u))] = static_cast<short>(p);
      __syncwarp();
      if (is && lane == __ffs(same) - 1) t.counts[id] += __popc(same);
      __syncwarp();
    }
  }
  __syncthreads();
  return t.number;
}

// Zeros in the rows of pairs without an expert; CTA `me` of `crowd` takes its
// share of the tiles of `rows` columns.
template <int rows, typename Out>
__device__ __forceinline__ void clear_rows(const GemvArgs& a, Out* out, int me, int crowd) {
  const int lane = threadIdx.x & 31, P = static_cast<int>(a.P);
  for (int p = threadIdx.x >> 5; p < P; p += kWarps) {
    const int id = __ldg(a.ids + p);
    if (id >= 0 && id < a.E) continue;
    for (int64_t tile = me; tile < a.N / rows; tile += crowd)
      for (int i = lane; i < rows; i += 32) out[p * a.ldo + tile * rows + i] = Out(0.0f);
  }
}

// ---------------------------------------------------------------------------
// Up to 8 rows of a weight.  A CTA (a cluster of `ranks` CTAs that share out K)
// takes a run of items; an item is 32 weight rows, 8 b + g and 32, 64, 96
// further of a 128-row atom, for up to 8 pairs of one expert (a slot), and its 8
// warps share out K.  Weights stream through a ring of shared memory that every
// thread fills for itself, across the items' borders, so that no item waits for
// memory from its beginning.
// 14336 x 4096, one row: 14.2 us, 2.3 TB/s (weights from memory; 5.05 us at the
// measured rate).  8 weights of that size, 16 rows: 57 to 66 us, 4.0 to 4.7 TB/s.
// What bounds the larger: instructions (issue 70% of the active cycles), of them
// unpacking, 19 cycles of the logic and multiply pipes per 8 codes and warp (59%
// and 52% busy), and the item borders (one CTA's warps meet).  One row is bound by
// its start, its end and its balance: 448 items on 444 CTAs, an SM active 21
// thousand cycles on average, 27 at most, of 32; the logic pipe is 35% busy.  Two
// copies of the warps' sums and one barrier less: 70 us (less L1 for x); two CTAs
// per SM with a deeper ring: 15.8 and 68; four CTAs: 15.3 and 84; x a word ahead:
// 15.0 and 68.
// ---------------------------------------------------------------------------
constexpr int kDepth = 2;   // chunks of a lane on their way and in use
constexpr int kCtas = 3;    // per SM
struct Smem {
  uint4 ring[kDepth][kPieces][kThreads];   // every thread copies and reads its own pieces
  float part[kWarps][8][kTileRows + 1];
  float share[2][8][kTileRows];            // this CTA's sums, read by its cluster
  Slots slots;
};

template <typename Out>
__global__ void __launch_bounds__(kThreads, kCtas) gemv_kernel(const __grid_constant__ GemvArgs a) {
  extern __shared__ __align__(16) uint8_t gemv_smem[];
  Smem& sm = *reinterpret_cast<Smem*>(gemv_smem);
  pdl_entry();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int P = static_cast<int>(a.P);
  const int64_t N = a.N, K = a.K;
  const int tiles = static_cast<int>(N / kTileRows);
  Out* const out = static_cast<Out*>(a.out);
  int slots = (P + 7) / 8;
  if (a.ids) {
    slots = find_slots<8>(a, sm.slots, rank == 0);
    if (rank == 0) clear_rows<kTileRows>(a, out, blockIdx.x / ranks, gridDim.x / ranks);
  }

  // items are counted in 32 bits: at most 1024 slots and 2^20 tiles
  const uint32_t crowd = gridDim.x / ranks, me = blockIdx.x / ranks, items = static_cast<uint32_t>(slots) * tiles;
  const uint32_t each = items / crowd, more = items % crowd;
  const uint32_t first = me * each + min(me, more);
  uint32_t left = each + (me < more);
  const int chunks = static_cast<int>((K + 127) / 128);
  const int stride = kWarps * ranks, start = rank * kWarps + warp;
  const int mine = chunks > start ? (chunks - start + stride - 1) / stride : 0;   // chunks of this warp and an item
  const uint32_t pick = c & 1 ? 0x4342u : 0x4140u;                                // this lane's two scales of four
  const bool tail = c * 32 + (chunks - 1) * 128 < K;                              // this lane has values in the last chunk

  // the ring's filling end; an item is (slot, tile)
  uint32_t f_left = left;
  int f_slot = static_cast<int>(first / tiles), f_tile = static_cast<int>(first) - f_slot * tiles;
  int tile = f_tile, slot = f_slot;
  int f_chunk = 0, f_stage = 0;
  const uint8_t *f_codes = nullptr, *f_scales = nullptr;
  auto aim = [&]() {
    const int64_t e = a.ids ? sm.slots.expert[f_slot] : 0;
    const int64_t row = (f_tile >> 2) * 128ll + (f_tile & 3) * 8 + g;
    f_codes = a.W + (e * N + row) * (K / 2) + start * 64 + c * 16;
    f_scales = a.sW + e * N * (K / 16) + ((f_tile >> 2) * (K / 64) + start * 2 + (c >> 1)) * 512 + ((f_tile & 3) * 8 + g) * 16;
  };
  auto fill = [&]() {
    if (f_left && mine) {
      const bool real = tail || f_chunk + 1 < mine || start + f_chunk * stride + 1 < chunks;
      const uint8_t* const codes = real ? f_codes : a.W;
      const int64_t apart = real ? 16 * K : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) copy16(&sm.ring[f_stage][i][tid], codes + i * apart, real);
      copy16(&sm.ring[f_stage][4][tid], real ? f_scales : a.sW, real);
      f_codes += stride * 64;
      f_scales += stride * 1024;
      if (++f_chunk == mine) {
        f_chunk = 0;
        if (++f_tile == tiles) {
          f_tile = 0;
          ++f_slot;
        }
        if (--f_left) aim();
      }
      f_stage = f_stage + 1 == kDepth ? 0 : f_stage + 1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (left) aim();
#pragma unroll
  for (int s = 0; s < kDepth - 1; ++s) fill();

  int use = 0, turn = 0;
  for (; left; --left, turn ^= 1) {
    const int e = a.ids ? sm.slots.expert[slot] : 0;
    const int m0 = a.ids ? sm.slots.begin[e] + sm.slots.pass[slot] * 8 : slot * 8;
    const int members = min((a.ids ? sm.slots.begin[e + 1] : P) - m0, 8);
    // columns without a pair read the first one's row; their sums are dropped
    const int column = m0 + (g < members ? g : 0);
    const uint32_t pair = a.ids ? sm.slots.pairs[column] : column;
    const __nv_bfloat16* x = a.x + static_cast<int64_t>(pair / static_cast<uint32_t>(a.rep)) * a.ldx + start * 128 + c * 32;
    float acc[2][4] = {};
    for (int j = 0, kc = start; j < mine; ++j, kc += stride) {
      // nothing here: no number in x's place may meet the zero weights
      if (!tail && kc + 1 == chunks) x = reinterpret_cast<const __nv_bfloat16*>(kNothing);
      fill();
      asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
      uint32_t u[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 w = sm.ring[use][i][tid];
        u[i][0] = w.x;
        u[i][1] = w.y;
        u[i][2] = w.z;
        u[i][3] = w.w;
      }
      const uint4 sw = sm.ring[use][4][tid];
      use = use + 1 == kDepth ? 0 : use + 1;
      uint32_t sc[4][2];
      scale_pairs(sw.x, pick, sc[0]);
      scale_pairs(sw.y, pick, sc[1]);
      scale_pairs(sw.z, pick, sc[2]);
      scale_pairs(sw.w, pick, sc[3]);
#pragma unroll
      for (int word = 0; word < 4; ++word) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(x) + word);
        const uint32_t b[4] = {__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                               __byte_perm(v.y, v.w, 0x7632)};
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          uint32_t lo[4], hi[4];
          decode(u[2 * m][word], sc[2 * m][word >> 1], lo);
          decode(u[2 * m + 1][word], sc[2 * m + 1][word >> 1], hi);
          const uint32_t op0[4] = {lo[0], hi[0], lo[1], hi[1]}, op1[4] = {lo[2], hi[2], lo[3], hi[3]};
          mma16(acc[m], op0, b[0], b[1]);
          mma16(acc[m], op1, b[2], b[3]);
        }
      }
      x += stride * 128;
    }
    __syncthreads();   // part is read until here in the item before
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 4; ++h)
        // weight row: 32 (2 m + h / 2) + g; x row 2 c + h % 2
        sm.part[warp][2 * c + (h & 1)][(2 * m + (h >> 1)) * 8 + g] = acc[m][h];
    __syncthreads();
    const float alpha = __ldg(a.alphaW + e);
    const int64_t n0 = (tile >> 2) * 128ll + (tile & 3) * 8;
    for (int v = tid; v < members * kTileRows; v += kThreads) {
      const int m = v / kTileRows, r = v % kTileRows;
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) s += sm.part[i][m][r];
      if (ranks > 1) {
        sm.share[turn][m][r] = s;
      } else {
        const int64_t p = a.ids ? sm.slots.pairs[m0 + m] : m0 + m;
        out[p * a.ldo + n0 + (r >> 3) * 32 + (r & 7)] = Out(s * alpha * 256.0f);
      }
    }
    if (ranks > 1) {
      cluster.sync();   // share is complete; the other copy has been read by all
      for (int v = rank * kThreads + tid; v < members * kTileRows; v += ranks * kThreads) {
        const int m = v / kTileRows, r = v % kTileRows;
        float s = 0.0f;
        for (int i = 0; i < ranks; ++i) s += cluster.map_shared_rank(&sm.share[turn][m][r], i)[0];
        const int64_t p = a.ids ? sm.slots.pairs[m0 + m] : m0 + m;
        out[p * a.ldo + n0 + (r >> 3) * 32 + (r & 7)] = Out(s * alpha * 256.0f);
      }
    }
    if (++tile == tiles) {
      tile = 0;
      ++slot;
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (ranks > 1) cluster.sync();   // no CTA leaves while its share is read
}

// ---------------------------------------------------------------------------
// More rows.  x is as large as the weight's rows that share it, so a CTA takes a
// whole 128-row atom: warp w its quarter w % 4 and, of each 256 values of K, half
// w / 4; x comes once per CTA, through shared memory.  One item per cluster of
// `ranks` CTAs, which share out K.
// 4096 x 14336, 24 rows, fp32: 22 us (5.2 at the measured rate): 520 instructions
// per 128 values of K and 32 weight rows, 48 of them products, on 256 CTAs, one
// or two per SM, for 7 stages each between the start and the cluster's sum.
// ---------------------------------------------------------------------------
template <int NT>
struct WideCfg {
  static constexpr int kDepth = 3;   // stages of 256 values of K
  struct Stage {
    uint4 w[kPieces][kThreads];      // every thread copies and reads its own
    uint4 x[2][NT * 8][16];          // half, row: 16 bytes of word v of lane c at 4 c + (v + c + row) % 4
  };
  struct Smem {
    union {
      Stage ring[kDepth];
      float share[2][NT * 8][129];   // sums of the halves, read by the cluster
    };
    Slots slots;
  };
  // CTAs that an SM has room for: one of 32 columns.  A grid for two left half of
  // the CTAs waiting for the others: 32 rows, 4096 x 14336 45.0 us for 25.7, 4096 x
  // 4096 23.3 for 11.2, 14336 x 4096 35.0 for 28.9.
  static constexpr int kCtas = 2 * (sizeof(Smem) + 1024) <= 228 * 1024 ? 2 : 1;
};

template <int NT, typename Out>
__global__ void __launch_bounds__(kThreads, 2) gemv_wide_kernel(const __grid_constant__ GemvArgs a) {
  using Cfg = WideCfg<NT>;
  constexpr int kDepth = Cfg::kDepth, kGroup = NT * 8;
  extern __shared__ __align__(16) uint8_t gemv_smem[];
  typename Cfg::Smem& sm = *reinterpret_cast<typename Cfg::Smem*>(gemv_smem);
  pdl_entry();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3, part = warp >> 2;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int64_t N = a.N, K = a.K;
  const int atoms = static_cast<int>(N / 128);
  const int item = blockIdx.x / ranks, slot = item / atoms, atom = item - slot * atoms;
  Out* const out = static_cast<Out*>(a.out);
  int slots = (static_cast<int>(a.P) + kGroup - 1) / kGroup;
  if (a.ids) {
    slots = find_slots<kGroup>(a, sm.slots, rank == 0);
    if (rank == 0 && slot == 0) clear_rows<128>(a, out, atom, atoms);
  }
  if (slot >= slots) return;   // the whole cluster
  const int64_t e = a.ids ? sm.slots.expert[slot] : 0;
  const int m0 = a.ids ? sm.slots.begin[e] + sm.slots.pass[slot] * kGroup : slot * kGroup;
  const int members = min((a.ids ? sm.slots.begin[e + 1] : static_cast<int>(a.P)) - m0, kGroup);
  const int stages = static_cast<int>((K + 255) / 256);
  const int from = static_cast<int>(static_cast<int64_t>(stages) * rank / ranks);
  const int to = static_cast<int>(static_cast<int64_t>(stages) * (rank + 1) / ranks);

  const int row0 = (warp & 3) * 8 + g;   // of the atom; its others 32, 64, 96 further
  const uint8_t* codes = a.W + (e * N + atom * 128ll + row0) * (K / 2) + (from * 2ll + part) * 64 + c * 16;
  const uint8_t* scales = a.sW + e * N * (K / 16) + (atom * (K / 64) + (from * 2ll + part) * 2 + (c >> 1)) * 512 + row0 * 16;
  // copied by this thread: piece `lane` of rows warp, warp + 8, ..; rows behind
  // the last pair's are copies of the first, and their sums are dropped
  const __nv_bfloat16* x[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int m = m0 + (i * 8 + warp < members ? i * 8 + warp : 0);
    const uint32_t p = a.ids ? sm.slots.pairs[m] : m;
    x[i] = a.x + static_cast<int64_t>(p / static_cast<uint32_t>(a.rep)) * a.ldx + from * 256ll + lane * 8;
  }
  const int x_at = ((lane & 15) & ~3) + ((lane + ((lane & 15) >> 2) + warp) & 3);   // rows i * 8 + warp: (row) % 4 = warp % 4

  int fill = from, f_stage = 0;
  auto copy = [&]() {
    if (fill < to) {
      typename Cfg::Stage& st = sm.ring[f_stage];
      const bool real = fill * 256ll + part * 128 + c * 32 < K, x_real = fill * 256ll + lane * 8 < K;
#pragma unroll
      for (int i = 0; i < 4; ++i) copy16(&st.w[i][tid], real ? codes + i * 16 * K : a.W, real);
      copy16(&st.w[4][tid], real ? scales : a.sW, real);
#pragma unroll
      for (int i = 0; i < NT; ++i)
        copy16(&st.x[lane >> 4][i * 8 + warp][x_at], reinterpret_cast<const uint8_t*>(x_real ? x[i] : a.x), x_real);
      codes += 128;
      scales += 2048;
#pragma unroll
      for (int i = 0; i < NT; ++i) x[i] += 256;
      ++fill;
      f_stage = f_stage + 1 == kDepth ? 0 : f_stage + 1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < kDepth - 1; ++s) copy();

  const uint32_t pick = c & 1 ? 0x4342u : 0x4140u;
  float acc[NT][2][4] = {};
  int use = 0;
  for (int s = from; s < to; ++s) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
    __syncthreads();   // everyone's copies are here; the stage before is free
    copy();
    const typename Cfg::Stage& st = sm.ring[use];
    use = use + 1 == kDepth ? 0 : use + 1;
    uint32_t u[4][4], sc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 w = st.w[i][tid];
      u[i][0] = w.x;
      u[i][1] = w.y;
      u[i][2] = w.z;
      u[i][3] = w.w;
    }
    const uint4 sw = st.w[4][tid];
    scale_pairs(sw.x, pick, sc[0]);
    scale_pairs(sw.y, pick, sc[1]);
    scale_pairs(sw.z, pick, sc[2]);
    scale_pairs(sw.w, pick, sc[3]);
#pragma unroll
    for (int word = 0; word < 4; ++word) {
      uint32_t b[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const uint4 v = st.x[part][i * 8 + g][4 * c + ((word + c + g) & 3)];
        b[i][0] = __byte_perm(v.x, v.z, 0x5410);
        b[i][1] = __byte_perm(v.x, v.z, 0x7632);
        b[i][2] = __byte_perm(v.y, v.w, 0x5410);
        b[i][3] = __byte_perm(v.y, v.w, 0x7632);
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint32_t lo[4], hi[4];
        decode(u[2 * m][word], sc[2 * m][word >> 1], lo);
        decode(u[2 * m + 1][word], sc[2 * m + 1][word >> 1], hi);
        const uint32_t op0[4] = {lo[0], hi[0], lo[1], hi[1]}, op1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          mma16(acc[i][m], op0, b[i][0], b[i][1]);
          mma16(acc[i][m], op1, b[i][2], b[i][3]);
        }
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();   // the ring becomes share
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 4; ++h)
        sm.share[part][i * 8 + 2 * c + (h & 1)][(2 * m + (h >> 1)) * 32 + row0] = acc[i][m][h];
  if (ranks > 1) cluster.sync();
  else __syncthreads();
  const float alpha = __ldg(a.alphaW + e);
  for (int v = rank * kThreads + tid; v < members * 128; v += ranks * kThreads) {
    const int m = v >> 7, r = v & 127;
    float sum = 0.0f;
    for (int i = 0; i < ranks; ++i) {
      const float* const from_rank = ranks > 1 ? cluster.map_shared_rank(&sm.share[0][m][r], i) : &sm.share[0][m][r];
      sum += from_rank[0];
      sum += from_rank[NT * 8 * 129];
    }
    const int64_t p = a.ids ? sm.slots.pairs[m0 + m] : m0 + m;
    out[p * a.ldo + atom * 128ll + r] = Out(sum * alpha * 256.0f);
  }
  if (ranks > 1) cluster.sync();   // no CTA leaves while its share is read
}

template <typename Out>
cudaError_t launch_narrow(const GemvArgs& a, cudaStream_t st) {
  constexpr size_t smem = sizeof(Smem);
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(gemv_kernel<Out>, smem, done);
  if (e != cudaSuccess) return e;
  const int64_t slots = a.ids ? std::min(a.P, a.E) : (a.P + 7) / 8;
  const int64_t items = slots * (a.N / kTileRows), chunks = (a.K + 127) / 128;
  const int64_t room = static_cast<int64_t>(sm_count()) * kCtas;
  int ranks = 1;
  while (ranks < 8 && items * ranks * 2 <= room && chunks >= 2 * ranks * kWarps) ranks *= 2;
  const int64_t crowd = std::max<int64_t>(1, std::min(items, room / ranks));
  note_launch();
  return launch_k(gemv_kernel<Out>, dim3(static_cast<unsigned>(crowd * ranks)), dim3(kThreads), smem, st,
                  static_cast<unsigned>(ranks), a);
}

template <int NT, typename Out>
cudaError_t launch_wide(const GemvArgs& a, cudaStream_t st) {
  constexpr size_t smem = sizeof(typename WideCfg<NT>::Smem);
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(gemv_wide_kernel<NT, Out>, smem, done);
  if (e != cudaSuccess) return e;
  const int64_t full = (a.P + NT * 8 - 1) / (NT * 8);
  const int64_t slots = a.ids ? std::min(a.P, full + std::min(a.P, a.E) - 1) : full;
  const int64_t items = slots * (a.N / 128), stages = (a.K + 255) / 256;
  const int64_t room = static_cast<int64_t>(sm_count()) * WideCfg<NT>::kCtas;
  int ranks = 1;
  while (ranks < 8 && items * ranks * 2 <= room && stages >= 4 * ranks) ranks *= 2;
  note_launch();
  return launch_k(gemv_wide_kernel<NT, Out>, dim3(static_cast<unsigned>(items * ranks)), dim3(kThreads), smem, st,
                  static_cast<unsigned>(ranks), a);
}

// The kernel goes by the rows that a weight is likely to have: P without ids,
// else the mean of the weights that can be taken.  More than 8 are cut into as
// few passes of up to 32 as there can be, of as few columns as that takes.
// Even / uneven choices (weights proportional to exp of a normal), us:
//   rows of each                    6           8          12          16          24
//   8 experts of 14336 x 4096
//     first kernel            86 /  96    89 / 126   161 / 160   164 / 197   248 / 274
//     16 columns             116 /  92   117 / 118   119 / 139   121 / 155   220 / 226
//     24 columns             137 / 111   138 / 139   139 / 141   141 / 168   145 / 201
//     32 columns             192 / 129   195 / 195   197 / 177   199 / 198   204 / 267
//   128 experts of 1408 x 2048
//     first kernel            91 / 103    99 / 127
//     16 columns             141 / 130   163 / 160
//   32 experts of 1024 x 1024
//     first kernel          17.4 / 18.2  19.7 / 22.3 29.2 / 27.0 32.2 / 34.2
//     16 columns            15.1 / 14.8  17.0 / 17.5 23.0 / 27.7 25.4 / 31.9 42.9 / 37.6
//     24 columns            18.4 / 18.4  19.5 / 20.3 21.6 / 22.0 27.3 / 32.2 33.3 / 39.2
// Up to K = 1024 a spare column costs less than another pass, so half as many
// rows again are taken for likely.  One weight, 40 rows, 24 / 32 columns: 4096 x
// 14336 37 / 47, 14336 x 4096 43 / 62, 4096 x 4096 15 / 18.
template <typename Out>
cudaError_t launch_out(const GemvArgs& a, cudaStream_t st) {
  int64_t rows = a.P;
  if (a.ids) {
    const int64_t weights = std::min(a.P, a.E), likely = a.K > 1024 ? 2 * a.P : 3 * a.P;
    rows = (likely + 2 * weights - 1) / (2 * weights);
  }
  const int64_t passes = (rows + 31) / 32, columns = (rows + passes - 1) / passes;
  return rows <= 8       ? launch_narrow<Out>(a, st)
         : columns <= 16 ? launch_wide<2, Out>(a, st)
         : columns <= 24 ? launch_wide<3, Out>(a, st)
                         : launch_wide<4, Out>(a, st);
}

}  // namespace

cudaError_t gemv_launch(const GemvArgs& a, cudaStream_t st) {
  return a.fp32 ? launch_out<float>(a, st) : launch_out<__nv_bfloat16>(a, st);
}

}  // namespace nvfp4
