// grouped_quantize.cu -- NVFP4 quantization of rows sorted by group (the
// tokens of each expert of a mixture layer), and its inverse.
//
// Every group is a tensor of its own (Four Over Six §2.1 Eq. 1-3 per group):
// alpha_e from the group's amax, blocks of 16 along the rows' elements and /
// or down the group's rows.  Group e gets exactly the codes and scales that
// nvfp4_quantize writes for its rows alone, padded with zero rows to a
// multiple of 64, with stream id stream_id + e.
//
// Two launches, as for one tensor: an amax pass folds each tile's maximum
// into its group's word, then the tiles are encoded.  Both walk 64 x 128
// tiles of the groups' own row frames, a contiguous run per CTA, so the
// group changes rarely within a CTA.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "nvfp4_device.cuh"
#include "block_modes.cuh"
#include "grouped.cuh"
#include "launch.cuh"
#include "nvfp4_internal.h"
#include "tile.cuh"

namespace nvfp4 {
namespace {

struct GroupedArgs {
  const uint16_t* x;
  int64_t T, C, ld;
  const int32_t* offsets;
  int E;
  uint64_t seed;
  uint32_t stream_id, flags;
  uint32_t* amax_r;      // [E] float bits (or kNonFinite)
  uint32_t* amax_c;      // [E] (== amax_r when not rotated)
  uint8_t* codes_row;
  uint8_t* scales_row;
  float* alpha_row;
  uint8_t* codes_col;
  uint8_t* scales_col;
  float* alpha_col;
  float* amax_out;       // [2, E] or null
  int32_t* status;
  uint32_t tiles_c;
  int64_t kcap;          // columns of codes_col in elements (a multiple of 64)
};

__device__ __forceinline__ void cp_async16_or_zero(void* smem, const void* gmem, bool valid) {
  const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  const int bytes = valid ? 16 : 0;   // 0: nothing is read, the 16 bytes become zero
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(s), "l"(gmem), "r"(bytes) : "memory");
}

// One 64 x 128 tile of a group whose first row is x (rows x C valid): chunks
// outside it become zeros, so that a block that the group's end cuts holds
// the zero rows of its padding.
template <int NT>
__device__ __forceinline__ void load_group_tile(uint4 (*buf)[TC / 8], const uint16_t* x, int rows, int64_t C,
                                                int64_t ld, int tr, uint32_t tc) {
  constexpr int kRowStep = NT / 16, kPasses = TR / kRowStep;
  const int row0 = static_cast<int>(threadIdx.x) >> 4, cc = static_cast<int>(threadIdx.x) & 15;
  const int64_t c0 = static_cast<int64_t>(tc) * TC + 8 * cc;
  const int left = rows - tr * TR;
  const uint16_t* src = x + (static_cast<int64_t>(tr) * TR + row0) * ld + c0;
  if (left >= TR && static_cast<int64_t>(tc + 1) * TC <= C) {
    const int64_t step = kRowStep * ld;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int row = row0 + kRowStep * i;
      cp_async16(&buf[row][tile_chunk(row, cc)], src + i * step);
    }
  } else {
    const bool col_ok = c0 < C;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int row = row0 + kRowStep * i;
      const bool ok = col_ok && row < left;
      cp_async16_or_zero(&buf[row][tile_chunk(row, cc)], ok ? src + static_cast<int64_t>(kRowStep * i) * ld : x, ok);
    }
  }
  cp_async_commit();
}

// A CTA's run of tiles: [first, last) of the total, the runs differing by at
// most one tile.
struct TileRun {
  uint32_t tile, end;
  __device__ __forceinline__ TileRun(uint32_t total, uint32_t cta, uint32_t ncta) {
    tile = static_cast<uint32_t>(static_cast<uint64_t>(total) * cta / ncta);
    end = static_cast<uint32_t>(static_cast<uint64_t>(total) * (cta + 1) / ncta);
  }
};

// Tile -> (group, tile row within the group, tile column).  A group's tiles
// are walked in bands of four tile rows, down a band's rows first, then along
// its columns: four 32-byte pieces of a column's codes and, two columns on,
// two 64-byte pieces of a row's complete 128-byte lines within a few tiles of
// one CTA.  (Row by row, columns first, each column piece was a partial line
// of its own, and decoding 16301 x 14336 column codes took a third longer.)
constexpr int kBand = 4;
struct GroupTile {
  int e, tr;
  uint32_t tc;
};
__device__ __forceinline__ GroupTile group_tile(const GroupTable& g, uint32_t tile, uint32_t tiles_c) {
  const int e = find_group(g.pa, g.E, static_cast<int>(tile / tiles_c));
  const uint32_t local = tile - static_cast<uint32_t>(g.pa[e]) * tiles_c;
  const uint32_t n_tr = static_cast<uint32_t>(g.pa[e + 1] - g.pa[e]);
  const uint32_t band = local / (kBand * tiles_c), in = local - band * kBand * tiles_c;
  const uint32_t h = min(static_cast<uint32_t>(kBand), n_tr - band * kBand);
  return GroupTile{e, static_cast<int>(band * kBand + in % h), in / h};
}
__device__ __forceinline__ void next_tile(const GroupTable& g, GroupTile& t, uint32_t tiles_c) {
  const int n_tr = g.pa[t.e + 1] - g.pa[t.e];
  const int start = t.tr & ~(kBand - 1);
  if (++t.tr < min(start + kBand, n_tr)) return;
  t.tr = start;
  if (++t.tc < tiles_c) return;
  t.tc = 0;
  t.tr = start + kBand;
  while (t.e + 1 < g.E && t.tr >= g.pa[t.e + 1] - g.pa[t.e]) {   // past this group's last tile row
    ++t.e;
    t.tr = 0;
  }
}

// The two halves of pdl_entry().  The kernels that walk many tiles let the next
// kernel launch at their last tile: CTAs of the next kernel that were resident
// (waiting) from the start kept the SM in this kernel's split of L1 and shared
// memory, and ran in it to their end (decoding the columns right behind the
// encoding of 16301 x 14336 took 240 us instead of 150).
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// All threads of the cluster; what they wrote to shared memory before is
// visible to the others after.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The word at this shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t load_cluster_u32(const uint32_t* p, int rank) {
  uint32_t addr, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// ---------------------------------------------------------------------------
// amax per group.  Plain: memory bounds it (16384 x 4096 25 us, 5.4 TB/s).
// Rotated: its instructions (a butterfly per orientation, 13 thread instructions
// per value, 61% of the issue slots used; 16301 x 14336, both, 143 us, 3.3 TB/s).
// ---------------------------------------------------------------------------
// Fold the CTA's running maximum (float bits) into a group's word.
template <int NT>
__device__ __forceinline__ void flush_max(uint32_t m, uint32_t* dst, uint32_t* red, int32_t* status) {
  m = block_max_u32<NT>(m, red);
  if (threadIdx.x == 0 && m) {
    atomicMax(dst, m);   // the order of a maximum does not matter
    if (m == kNonFinite && status) *status = kStatusNonFinite;
  }
}

constexpr int kPlainNT = 256;

__global__ void __launch_bounds__(kPlainNT) grouped_amax_plain_kernel(const GroupedArgs a) {
  pdl_wait();
  extern __shared__ int table_mem[];
  __shared__ uint32_t red[kPlainNT / 32];
  const GroupTable g = build_group_table<kPlainNT>(a.offsets, a.E, a.T, TR, 128, table_mem, a.status, blockIdx.x == 0);
  TileRun run(static_cast<uint32_t>(g.pa[a.E]) * a.tiles_c, blockIdx.x, gridDim.x);
  if (run.tile >= run.end) return;
  GroupTile t = group_tile(g, run.tile, a.tiles_c);
  int e = t.e;
  uint32_t hm = 0;
  auto flush = [&]() {
    const uint32_t h = max(hm & 0xFFFFu, hm >> 16);
    flush_max<kPlainNT>(h >= 0x7F80u ? kNonFinite : (h << 16), a.amax_r + e, red, a.status);
    hm = 0;
  };
  for (; run.tile < run.end; ++run.tile, next_tile(g, t, a.tiles_c)) {
    if (run.tile + 1 == run.end) pdl_release();
    if (t.e != e) {   // uniform over the CTA
      flush();
      e = t.e;
    }
    const int left = g.rows(t.e) - t.tr * TR;
    const int row0 = static_cast<int>(threadIdx.x) >> 4, cc = static_cast<int>(threadIdx.x) & 15;
    const int64_t c0 = static_cast<int64_t>(t.tc) * TC + 8 * cc;
    const uint16_t* src = a.x + (static_cast<int64_t>(g.off[t.e]) + t.tr * TR + row0) * a.ld + c0;
    uint4 u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[i] = make_uint4(0u, 0u, 0u, 0u);
      if (c0 < a.C && row0 + 16 * i < left)
        u[i] = __ldg(reinterpret_cast<const uint4*>(src + static_cast<int64_t>(16 * i) * a.ld));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hm = __vmaxu2(hm, u[i].x & 0x7FFF7FFFu);
      hm = __vmaxu2(hm, u[i].y & 0x7FFF7FFFu);
      hm = __vmaxu2(hm, u[i].z & 0x7FFF7FFFu);
      hm = __vmaxu2(hm, u[i].w & 0x7FFF7FFFu);
    }
  }
  flush();
}

// Rotated maxima, rows and / or columns.  The transform's final 1/4 commutes
// with the maximum and is applied at the end.
constexpr int kRotNT = 128;
template <bool ROW, bool COL>
__global__ void __launch_bounds__(kRotNT) grouped_amax_rot_kernel(const GroupedArgs a) {
  pdl_wait();
  extern __shared__ int table_mem[];
  __shared__ __align__(16) uint4 tiles[2][TR][TC / 8];
  __shared__ uint32_t red[kRotNT / 32];
  const GroupTable g = build_group_table<kRotNT>(a.offsets, a.E, a.T, TR, 128, table_mem, a.status, blockIdx.x == 0);
  TileRun run(static_cast<uint32_t>(g.pa[a.E]) * a.tiles_c, blockIdx.x, gridDim.x);
  if (run.tile >= run.end) return;
  const SignMasks sm = sign_masks(sign_bits(philox_keys(a.seed)));
  GroupTile t = group_tile(g, run.tile, a.tiles_c), ahead = t;
  auto load = [&](int b) {
    load_group_tile<kRotNT>(tiles[b], a.x + static_cast<int64_t>(g.off[ahead.e]) * a.ld, g.rows(ahead.e), a.C, a.ld,
                         ahead.tr, ahead.tc);
    next_tile(g, ahead, a.tiles_c);
  };
  load(0);
  int e = t.e, buf = 0;
  float mr = 0.0f, mc = 0.0f;
  uint32_t hm = 0;
  auto flush = [&]() {
    const bool inf = max(hm & 0xFFFFu, hm >> 16) >= 0x7F80u;
    if constexpr (ROW)
      flush_max<kRotNT>(inf ? kNonFinite : __float_as_uint(__fmul_rn(mr, 0.25f)), a.amax_r + e, red, a.status);
    if constexpr (COL)
      flush_max<kRotNT>(inf ? kNonFinite : __float_as_uint(__fmul_rn(mc, 0.25f)), a.amax_c + e, red, a.status);
    mr = mc = 0.0f;
    hm = 0;
  };
  const int th = threadIdx.x;
  constexpr int kReps = 256 / kRotNT;   // row pairs and column units per thread and tile
  for (; run.tile < run.end; ++run.tile, next_tile(g, t, a.tiles_c), buf ^= 1) {
    if (run.tile + 1 == run.end) pdl_release();
    if (t.e != e) {
      flush();
      e = t.e;
    }
    if (run.tile + 1 < run.end) load(buf ^ 1);
    else cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    const uint4 (*s)[TC / 8] = tiles[buf];
    const int left = g.rows(t.e) - t.tr * TR;   // blocks of padding rows alone have nothing to add
    if constexpr (ROW) {
#pragma unroll
      for (int k = 0; k < kReps; ++k) {
      const int row = (th >> 3) + (kRotNT / 8) * k, cb = th & 7;
      if (row >= left) continue;
      const uint4 a0 = s[row][tile_chunk(row, 2 * cb)], a1 = s[row][tile_chunk(row, 2 * cb + 1)];
      const uint4 b0 = s[row + 32][tile_chunk(row + 32, 2 * cb)], b1 = s[row + 32][tile_chunk(row + 32, 2 * cb + 1)];
      const uint32_t w[16] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w,
                              b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
      for (int i = 0; i < 16; ++i) hm = __vmaxu2(hm, w[i] & 0x7FFF7FFFu);
      float2 v[16];
      unpack16x2_signed(a0, a1, b0, b1, sm, v);
      hadamard16x2(v);
      float ma, mb;
      max_abs16x2(v, ma, mb);
      mr = max3(mr, ma, mb);
      }
    }
    if constexpr (COL) {
#pragma unroll
      for (int k = 0; k < kReps; ++k) {
      const int cp = th & 63, rb = (th >> 6) + (kRotNT / 64) * k;
      if (16 * rb >= left) continue;
      const uint32_t* base = reinterpret_cast<const uint32_t*>(&s[16 * rb][0]);
      const int wofs = tile_word(16 * rb, cp);
      float2 v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t w = base[i * (TC / 2) + wofs];
        if constexpr (!ROW) hm = __vmaxu2(hm, w & 0x7FFF7FFFu);
        v[i] = make_float2(bf16lo_flip(w, sm.m[i]), bf16hi_flip(w, sm.m[i]));
      }
      hadamard16x2(v);
      float ma, mb;
      max_abs16x2(v, ma, mb);
      mc = max3(mc, ma, mb);
      }
    }
    __syncthreads();   // the buffer is refilled two iterations on
  }
  cp_async_wait<0>();
  flush();
}

// ---------------------------------------------------------------------------
// encode.  Its instructions bound it.  Rows and columns, thread instructions per
// value and issue slots used: 4/6 26, 71% (16384 x 4096 133 us; to nearest 55);
// rotated, to nearest 21, 58% (16301 x 14336 240 us), MS-EDEN 40, 60%, software
// stochastic rounding 76, 64% with the ALU pipe 62% busy.  Registers keep 16
// warps or fewer on an SM, which leave the rest of the slots to latencies.
// ---------------------------------------------------------------------------
struct GroupStaging {
  uint8_t colcodes[TC][48];        // transposed codes of one tile (32 bytes used per column)
  uint8_t colscale[TC][TR / 16];
  uint4 words[TNT / 32][32];       // scale-SR words shared by a warp (MS-EDEN, 256 threads)
  float2 tab_r[kScaleTab];
  float2 tab_c[kScaleTab];
};

__device__ __forceinline__ float group_alpha(const GroupedArgs& a, const uint32_t* amax, int e) {
  const uint32_t m = __ldcg(amax + e);
  return __fdiv_rn(m == kNonFinite ? 0.0f : __uint_as_float(m), (a.flags & kHeadroom) ? 1792.0f : 2688.0f);
}

// Threads of a CTA (128: two row pairs and two column pairs of a tile each) and
// CTAs per SM.  Times of amax and encoding, 16301 x 14336 in 64 groups, rows
// and columns: to nearest, rotated, 256 threads x 3 482 us, 128 x 5 446,
// 128 x 4 410; MS-EDEN, whose draws want 256, x 3 630, x 2 612; software
// stochastic rounding 256 x 2 971, 128 x 4 1298 (registers).  16384 x 4096 in
// 8 groups, 4/6 rows alone: 256 x 2 120, 128 x 4 109; one orientation alone of
// the 256-thread modes keeps three (2048 x 4096 in 64 groups, MS-EDEN columns:
// x 2 53 us, x 3 43).
template <int MODE>
constexpr int encode_threads() { return (MODE == kModeMsEden || MODE == kModeRhtSR) ? 256 : 128; }
template <int MODE, bool ROW, bool COL>
constexpr int encode_ctas() { return encode_threads<MODE>() == 128 ? 4 : ROW && COL ? 2 : 3; }

template <int MODE, bool ROT, bool ROW, bool COL>
__global__ void __launch_bounds__(encode_threads<MODE>(), encode_ctas<MODE, ROW, COL>()) grouped_quantize_kernel(const GroupedArgs a) {
  constexpr int NT = encode_threads<MODE>(), kReps = 256 / NT;   // row pairs and column units per thread and tile
  // Both orientations of the longer modes: the row pairs share their code,
  // which otherwise outgrows the instruction cache (4/6, 16384 x 4096, amax
  // and encoding 174 -> 158 us; to nearest, short, 391 -> 397 for 16301 x 14336).
  constexpr int kUnroll = ROW && COL && MODE != kModeRTN ? 1 : kReps;
  pdl_wait();
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ __align__(16) GroupStaging stg;
  auto tiles = reinterpret_cast<uint4(*)[TR][TC / 8]>(dyn);
  int* table_mem = reinterpret_cast<int*>(dyn + 2 * TR * TC * 2);
  const GroupTable g = build_group_table<NT>(a.offsets, a.E, a.T, TR, 128, table_mem, a.status, blockIdx.x == 0);
  const int th = threadIdx.x;
  if (blockIdx.x == 0) {
    for (int e = th; e < a.E; e += NT) {
      if constexpr (ROW) a.alpha_row[e] = group_alpha(a, a.amax_r, e);
      if constexpr (COL) a.alpha_col[e] = group_alpha(a, a.amax_c, e);
      if (a.amax_out) {
        const uint32_t r = __ldcg(a.amax_r + e), c = __ldcg(a.amax_c + e);
        if constexpr (ROW) a.amax_out[e] = r == kNonFinite ? 0.0f : __uint_as_float(r);
        if constexpr (COL) a.amax_out[a.E + e] = c == kNonFinite ? 0.0f : __uint_as_float(c);
      }
    }
  }
  TileRun run(static_cast<uint32_t>(g.pa[a.E]) * a.tiles_c, blockIdx.x, gridDim.x);
  if (run.tile >= run.end) return;

  const PhiloxKeys K = philox_keys(a.seed);
  SignMasks sm;
  if constexpr (ROT) {
    sm = sign_masks(sign_bits(K));
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) sm.m[i] = 0u;
  }
  const int64_t nbr = a.C / 16;
  const int trow = th >> 3, tcb = th & 7, tcp = th >> 2, trb = th & 3, lane = th & 31, j4 = th & 3;

  GroupTile t = group_tile(g, run.tile, a.tiles_c), ahead = t;
  auto load = [&](int b) {
    load_group_tile<NT>(tiles[b], a.x + static_cast<int64_t>(g.off[ahead.e]) * a.ld, g.rows(ahead.e), a.C, a.ld,
                         ahead.tr, ahead.tc);
    next_tile(g, ahead, a.tiles_c);
  };
  load(0);
  int e = -1, buf = 0;
  TabScales scr{}, scc{};
  for (; run.tile < run.end; ++run.tile, next_tile(g, t, a.tiles_c), buf ^= 1) {
    if (run.tile + 1 == run.end) pdl_release();
    if (run.tile + 1 < run.end) load(buf ^ 1);
    else cp_async_commit();
    if (t.e != e) {   // the scale tables of this group; the barrier below publishes them
      e = t.e;
      if constexpr (ROW) {
        const float al = group_alpha(a, a.amax_r, e);
        build_scale_tab<NT>(stg.tab_r, al);
        scr = make_scale_ctx(stg.tab_r, al);
      }
      if constexpr (COL) {
        const float al = group_alpha(a, a.amax_c, e);
        build_scale_tab<NT>(stg.tab_c, al);
        scc = make_scale_ctx(stg.tab_c, al);
      }
    }
    cp_async_wait<1>();
    __syncthreads();
    const uint4 (*s)[TC / 8] = tiles[buf];
    const int left = g.rows(e) - t.tr * TR;
    const int rows = left < TR ? left : TR;
    const int64_t c0 = static_cast<int64_t>(t.tc) * TC;
    const int cols = static_cast<int>(a.C - c0 < TC ? a.C - c0 : TC);
    const uint32_t c2r = (a.stream_id + static_cast<uint32_t>(e)) * 2u, c2c = c2r + 1u;
    // blocks down the rows, in the group's own frame padded to 64 rows
    const int64_t nbc = static_cast<int64_t>(g.pa[e + 1] - g.pa[e]) * (TR / 16);
    const int64_t rblk = (static_cast<int64_t>(t.tr) * TR + trow) * nbr + c0 / 16 + tcb;
    const int64_t cblk = (c0 + 2 * tcp) * nbc + t.tr * (TR / 16) + trb;

    // MS-EDEN: lanes 4k .. 4k + 3 hold blocks of the same two row units and
    // two column units (C and the padded rows are multiples of 64); each
    // draws one unit's four words and they are exchanged in shared memory.
    uint32_t w_ra = 0, w_rb = 0, w_ca = 0, w_cb = 0;
    if constexpr (MODE == kModeMsEden) {
      const int64_t unit_r = rblk - (tcb & 3) + (j4 & 1) * 32 * nbr;
      const int64_t unit_c = (c0 + 2 * tcp + (j4 & 1)) * nbc + t.tr * (TR / 16);
      const uint64_t unit = static_cast<uint64_t>(j4 < 2 ? unit_r : unit_c) >> 2;
      uint4* xs = stg.words[th >> 5];
      xs[lane] = philox(K, static_cast<uint32_t>(unit), static_cast<uint32_t>(unit >> 32), j4 < 2 ? c2r : c2c, kTagScaleSR);
      __syncwarp();
      const uint32_t* xw = reinterpret_cast<const uint32_t*>(xs + (lane & ~3)) + j4;
      w_ra = xw[0];
      w_rb = xw[4];
      w_ca = xw[8];
      w_cb = xw[12];
      __syncwarp();
    }

    if constexpr (ROW) {
#pragma unroll(kUnroll)
      for (int k = 0; k < kReps; ++k) {
      const int row = trow + (NT / 8) * k, cb = tcb;
      const bool va = row < rows && 16 * cb < cols, vb = row + 32 < rows && 16 * cb < cols;
      if (va || vb) {
        const uint4 a0 = s[row][tile_chunk(row, 2 * cb)], a1 = s[row][tile_chunk(row, 2 * cb + 1)];
        const uint4 b0 = s[row + 32][tile_chunk(row + 32, 2 * cb)];
        const uint4 b1 = s[row + 32][tile_chunk(row + 32, 2 * cb + 1)];
        float2 v[16];
        unpack16x2_signed(a0, a1, b0, b1, sm, v);
        if constexpr (ROT) rht16x2_presigned(v);
        Packed16 pa, pb;
        uint32_t sa, sb;
        const int64_t blk = rblk + (NT / 8) * k * nbr;
        quantize_pair<MODE>(v, scr, K, c2r, static_cast<uint64_t>(blk), static_cast<uint64_t>(blk + 32 * nbr), pa, pb,
                            sa, sb, MODE == kModeMsEden, w_ra, w_rb);
        uint8_t* crow = a.codes_row + (static_cast<int64_t>(g.off[e]) + t.tr * TR + row) * (a.C / 2) + c0 / 2 + 8 * cb;
        if (va) *reinterpret_cast<uint2*>(crow) = make_uint2(pa.lo, pa.hi);
        if (vb) *reinterpret_cast<uint2*>(crow + 32 * (a.C / 2)) = make_uint2(pb.lo, pb.hi);
        uint8_t* srow = a.scales_row + gemm_scale_tile_row(2 * static_cast<int64_t>(g.pb[e]) + t.tr, t.tc, nbr) +
                        gemm_scale_thread_row(row, cb);
        if (va) srow[0] = static_cast<uint8_t>(sa);
        if (vb) srow[4] = static_cast<uint8_t>(sb);
      }
      }
    }
    if constexpr (COL) {
#pragma unroll
      for (int k = 0; k < kReps; ++k) {
        const int cp = tcp + (NT / 4) * k;
        const int64_t blk = cblk + 2 * (NT / 4) * k * nbc;
        const uint32_t* base = reinterpret_cast<const uint32_t*>(&s[16 * trb][0]);
        const int wofs = tile_word(16 * trb, cp);
        float2 v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t w = base[i * (TC / 2) + wofs];
          v[i] = make_float2(bf16lo_flip(w, sm.m[i]), bf16hi_flip(w, sm.m[i]));
        }
        if constexpr (ROT) rht16x2_presigned(v);
        Packed16 qa, qb;
        uint32_t sa, sb;
        quantize_pair<MODE>(v, scc, K, c2c, static_cast<uint64_t>(blk), static_cast<uint64_t>(blk + nbc), qa, qb, sa,
                            sb, MODE == kModeMsEden, w_ca, w_cb);
        *reinterpret_cast<uint2*>(&stg.colcodes[2 * cp][8 * trb]) = make_uint2(qa.lo, qa.hi);
        *reinterpret_cast<uint2*>(&stg.colcodes[2 * cp + 1][8 * trb]) = make_uint2(qb.lo, qb.hi);
        stg.colscale[2 * cp][trb] = static_cast<uint8_t>(sa);
        stg.colscale[2 * cp + 1][trb] = static_cast<uint8_t>(sb);
      }
      __syncthreads();
      // 16 code bytes of column th / 2 and column th's four scales: whole
      // tiles of the padded frame (C % 128 == 0 with columns)
      const int64_t kt = g.pa[e] + t.tr;   // 64-row tile of the padded frame
#pragma unroll
      for (int k = 0; k < kReps; ++k) {
        const int c = (th >> 1) + (NT / 2) * k, h = th & 1;
        *reinterpret_cast<uint4*>(a.codes_col + (c0 + c) * (a.kcap / 2) + 32 * kt + 16 * h) =
            *reinterpret_cast<const uint4*>(&stg.colcodes[c][16 * h]);
      }
      if (th < TC)
        *reinterpret_cast<uint32_t*>(a.scales_col + gemm_scale_tile_col(kt, t.tc, a.kcap / 16) +
                                     gemm_scale_thread_col(th)) = *reinterpret_cast<const uint32_t*>(&stg.colscale[th][0]);
    }
    __syncthreads();   // the tile buffer, the staging and the tables are free again
  }
  cp_async_wait<0>();
}

// ---------------------------------------------------------------------------
// Few rows (a decode step's tokens), rowwise: one launch.  A cluster of eight
// CTAs takes a group, each CTA an eighth of its columns; the CTAs' maxima are
// exchanged through distributed shared memory and the rows, still in
// registers where they fit, are encoded at once.  What it saves are launches:
// clearing the maxima, the amax pass and the encoding pass were three of
// 2 to 7 us each for 16 rows of 4096.
// ---------------------------------------------------------------------------
constexpr int kFewRows = 64;        // rows (of all groups) up to which this path is taken
constexpr int kFewGroups = 128;     // and groups: each costs a cluster, rows or not
constexpr int kFewSplit = 8;        // CTAs of a cluster (the portable size)
constexpr int kFewNT = 256;
constexpr int kFewKept = 2;         // block pairs of a thread that stay in registers

template <int MODE, bool ROT>
__global__ void __launch_bounds__(kFewNT) grouped_quantize_few_kernel(const GroupedArgs a) {
  pdl_entry();
  extern __shared__ int table_mem[];
  __shared__ uint32_t red[kFewNT / 32];
  __shared__ uint32_t cta_max;
  const GroupTable g = build_group_table<kFewNT>(a.offsets, a.E, a.T, TR, 128, table_mem, a.status, blockIdx.x == 0);
  const int e = static_cast<int>(blockIdx.x) / kFewSplit, rank = static_cast<int>(blockIdx.x) % kFewSplit;
  const int rows = g.rows(e), th = threadIdx.x;
  if (rows == 0) {   // every CTA of the cluster leaves here
    if (rank == 0 && th == 0) {
      a.alpha_row[e] = 0.0f;
      if (a.amax_out) a.amax_out[e] = 0.0f;
    }
    return;
  }
  const PhiloxKeys K = philox_keys(a.seed);
  SignMasks sm;
  if constexpr (ROT) {
    sm = sign_masks(sign_bits(K));
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) sm.m[i] = 0u;
  }
  // pairs of neighbouring blocks (32 elements); C is a multiple of 64
  const int pairs_row = static_cast<int>(a.C / 32);
  const int first = pairs_row * rank / kFewSplit, width = pairs_row * (rank + 1) / kFewSplit - first;
  const int total = rows * width;
  const uint16_t* x = a.x + static_cast<int64_t>(g.off[e]) * a.ld;
  auto load = [&](int k, uint4* u) {
    const int r = k / width, p = first + k - r * width;
    const uint4* src = reinterpret_cast<const uint4*>(x + r * a.ld + 32 * p);
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __ldg(src + i);
  };
  auto values = [&](const uint4* u, float2* v) {
    unpack16x2_signed(u[0], u[1], u[2], u[3], sm, v);
    if constexpr (ROT) rht16x2_presigned(v);
  };
  uint4 kept[kFewKept][4];
  uint32_t m = 0;
  auto take_max = [&](const uint4* u) {
    uint32_t hm = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hm = __vmaxu2(hm, u[i].x & 0x7FFF7FFFu);
      hm = __vmaxu2(hm, u[i].y & 0x7FFF7FFFu);
      hm = __vmaxu2(hm, u[i].z & 0x7FFF7FFFu);
      hm = __vmaxu2(hm, u[i].w & 0x7FFF7FFFu);
    }
    const uint32_t h = max(hm & 0xFFFFu, hm >> 16);
    uint32_t b = h << 16;
    if constexpr (ROT) {
      float2 v[16];
      values(u, v);
      float ma, mb;
      max_abs16x2(v, ma, mb);
      b = __float_as_uint(fmaxf(ma, mb));
    }
    m = max(m, h >= 0x7F80u ? kNonFinite : b);
  };
#pragma unroll
  for (int i = 0; i < kFewKept; ++i)
    if (th + i * kFewNT < total) load(th + i * kFewNT, kept[i]);
#pragma unroll
  for (int i = 0; i < kFewKept; ++i)
    if (th + i * kFewNT < total) take_max(kept[i]);
  for (int k = th + kFewKept * kFewNT; k < total; k += kFewNT) {
    uint4 u[4];
    load(k, u);
    take_max(u);
  }
  m = block_max_u32<kFewNT>(m, red);
  if (th == 0) cta_max = m;
  cluster_barrier();
  if (th < kFewSplit) m = max(m, load_cluster_u32(&cta_max, th));
  m = block_max_u32<kFewNT>(m, red);
  cluster_barrier();   // no CTA leaves while another may still read its word
  const float amax = m == kNonFinite ? 0.0f : __uint_as_float(m);
  const float al = __fdiv_rn(amax, (a.flags & kHeadroom) ? 1792.0f : 2688.0f);
  if (rank == 0 && th == 0) {
    a.alpha_row[e] = al;
    if (a.amax_out) a.amax_out[e] = amax;
    if (m == kNonFinite && a.status) *a.status = kStatusNonFinite;
  }
  const VecScales sc = make_vec_scales(al, al);
  const uint32_t c2 = (a.stream_id + static_cast<uint32_t>(e)) * 2u;
  const int64_t nbr = a.C / 16;
  auto encode = [&](int k, const uint4* u) {
    const int r = k / width, p = first + k - r * width;
    float2 v[16];
    values(u, v);
    const int64_t blk = r * nbr + 2 * p;
    Packed16 pa, pb;
    uint32_t sa, sb;
    quantize_pair<MODE>(v, sc, K, c2, static_cast<uint64_t>(blk), static_cast<uint64_t>(blk + 1), pa, pb, sa, sb);
    *reinterpret_cast<uint4*>(a.codes_row + (static_cast<int64_t>(g.off[e]) + r) * (a.C / 2) + 16 * p) =
        make_uint4(pa.lo, pa.hi, pb.lo, pb.hi);
    // both scales lie in one 16-bit half of the four-scale word
    *reinterpret_cast<uint16_t*>(a.scales_row + gemm_scale_offset(128 * static_cast<int64_t>(g.pb[e]) + r, 2 * p, nbr)) =
        static_cast<uint16_t>(sa | (sb << 8));
  };
#pragma unroll
  for (int i = 0; i < kFewKept; ++i)
    if (th + i * kFewNT < total) encode(th + i * kFewNT, kept[i]);
  for (int k = th + kFewKept * kFewNT; k < total; k += kFewNT) {
    uint4 u[4];
    load(k, u);
    encode(k, u);
  }
}

// ---------------------------------------------------------------------------
// decode.  Memory bounds it (0.5625 bytes in, 2 or 4 out per element); what
// counts is that every warp store is whole and contiguous.  To bf16, 16301 x
// 14336: rows 115 us (5.2 TB/s), columns 124 us (4.8); 16384 x 4096 37 and 39.
// ---------------------------------------------------------------------------
template <bool BF16>
__device__ __forceinline__ void store8(void* y, int64_t at, const float* v) {   // eight values of a row
  if constexpr (BF16) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(y) + at);
    dst[0] = make_float4(v[0], v[1], v[2], v[3]);
    dst[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

__device__ __forceinline__ void scale8(float* v, float s) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 p = mul2(make_float2(v[j], v[j + 1]), make_float2(s, s));
    v[j] = p.x;
    v[j + 1] = p.y;
  }
}

// The inverse rotation of two lane-paired blocks, as irht16 does it for one:
// its final (1/4 and the sign) is one exact product.  q: +-1/4 per element.
__device__ __forceinline__ void inverse_factors(uint32_t signs, float* q) {
#pragma unroll
  for (int i = 0; i < 16; ++i) q[i] = __uint_as_float(0x3E800000u ^ (((signs >> i) & 1u) << 31));
}
__device__ __forceinline__ void irht16x2(float2* v, const float* q) {
  hadamard16x2(v);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = mul2(v[i], make_float2(q[i], q[i]));
}

// Row operands: 64 x 256 tiles, a warp takes one row at a time, lane l the
// elements 8 l .. 8 l + 7 (a 16-byte bf16 store).  With INV a lane takes
// one 16-element block of two rows instead, since the rotation mixes it.
template <bool INV, bool BF16>
__global__ void __launch_bounds__(256) grouped_dequantize_rows_kernel(const uint8_t* __restrict__ codes,
                                                                      const uint8_t* __restrict__ scales,
                                                                      const float* __restrict__ alpha, int64_t T,
                                                                      int64_t C, const int32_t* __restrict__ offsets,
                                                                      int E, uint64_t seed, void* __restrict__ y,
                                                                      int32_t* status) {
  pdl_wait();
  extern __shared__ int table_mem[];
  const GroupTable g = build_group_table<256>(offsets, E, T, TR, 128, table_mem, status, blockIdx.x == 0);
  const uint32_t tiles_c = static_cast<uint32_t>((C + 255) / 256);
  TileRun run(static_cast<uint32_t>(g.pa[E]) * tiles_c, blockIdx.x, gridDim.x);
  if (run.tile >= run.end) return;
  [[maybe_unused]] float q[16];
  if constexpr (INV) inverse_factors(sign_bits(philox_keys(seed)), q);
  GroupTile t = group_tile(g, run.tile, tiles_c);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t katoms = C / 64;
  for (; run.tile < run.end; ++run.tile, next_tile(g, t, tiles_c)) {
    if (run.tile + 1 == run.end) pdl_release();
    const int left = g.rows(t.e) - t.tr * TR;
    const int rows = left < TR ? left : TR;
    const float al = __ldg(alpha + t.e);
    const int64_t row0 = static_cast<int64_t>(g.off[t.e]) + t.tr * TR;                  // in codes and y
    const int64_t srow0 = 128 * static_cast<int64_t>(g.pb[t.e]) + t.tr * TR;            // in the scale layout
    const uint8_t* sbase = scales + (srow0 >> 7) * katoms * 512 + ((srow0 >> 5) & 3) * 4;
    if constexpr (!INV) {
      const int64_t c = static_cast<int64_t>(t.tc) * 256 + 8 * lane;
      const bool col_ok = c < C;
      uint32_t w[8], sw[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {   // rows warp + 8 i
        const int r = warp + 8 * i;
        w[i] = sw[i] = 0u;
        if (col_ok && r < rows) {
          w[i] = __ldg(reinterpret_cast<const uint32_t*>(codes + (row0 + r) * (C / 2) + c / 2));
          // the four scales of 64 elements; row r of the half atom
          sw[i] = __ldg(reinterpret_cast<const uint32_t*>(sbase + (c >> 6) * 512 + (r & 31) * 16 + (r >> 5) * 4));
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = warp + 8 * i;
        const float s = __fmul_rn(al, e4m3_value((sw[i] >> (8 * ((lane >> 1) & 3))) & 0xFFu));
        float v[8];
        e2m1x8_values(w[i], v);
        scale8(v, s);
        if (col_ok && r < rows) store8<BF16>(y, (row0 + r) * C + c, v);
      }
    } else {
      const int64_t c = static_cast<int64_t>(t.tc) * 256 + 16 * (lane & 15);
      if (c < C) {
        for (int r0 = 2 * warp + (lane >> 4); r0 < rows; r0 += 32) {   // rows r0 and r0 + 16
          float v[2][16];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int r = min(r0 + 16 * k, rows - 1);
            const uint2 p = __ldg(reinterpret_cast<const uint2*>(codes + (row0 + r) * (C / 2) + c / 2));
            const float s = __fmul_rn(al, e4m3_value(__ldg(sbase + (c >> 6) * 512 + (r & 31) * 16 + (r >> 5) * 4 + ((c >> 4) & 3))));
            e2m1x8_values(p.x, v[k]);
            e2m1x8_values(p.y, v[k] + 8);
            // scalar: a packed product could be merged into the first addition
#pragma unroll
            for (int j = 0; j < 16; ++j) v[k][j] = __fmul_rn(v[k][j], s);
          }
          float2 u[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) u[j] = make_float2(v[0][j], v[1][j]);
          irht16x2(u, q);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (r0 + 16 * k >= rows) continue;
#pragma unroll
            for (int j = 0; j < 16; ++j) v[k][j] = k ? u[j].y : u[j].x;
            store8<BF16>(y, (row0 + r0 + 16 * k) * C + c, v[k]);
            store8<BF16>(y, (row0 + r0 + 16 * k) * C + c + 8, v[k] + 8);
          }
        }
      }
    }
  }
}

// Column operands: 64 x 128 tiles of the rows' frame.  A thread decodes one
// 16-row block of two neighbouring columns, four lanes the 32 bytes (one
// sector) that a tile holds of a column, and leaves the values in shared
// memory pairwise, from where rows are written whole.  (With a block per warp
// instead, four warps shared each sector through L1, and 16301 x 14336
// columns took 150 us, or 240 where a quantizer's shared memory had left
// little of L1.)
// Pair p of the rows of block b is stored at p ^ (kSwap b): the pairs of the
// four blocks that a store writes at once are in different banks.
template <bool INV, bool BF16>
__global__ void __launch_bounds__(256) grouped_dequantize_cols_kernel(const uint8_t* __restrict__ codes,
                                                                      const uint8_t* __restrict__ scales,
                                                                      const float* __restrict__ alpha, int64_t T,
                                                                      int64_t C, const int32_t* __restrict__ offsets,
                                                                      int E, int64_t kcap, uint64_t seed,
                                                                      void* __restrict__ y, int32_t* status) {
  using Pair = typename std::conditional<BF16, uint32_t, float2>::type;
  constexpr int kSwap = BF16 ? 8 : 4;
  pdl_wait();
  extern __shared__ int table_mem[];
  __shared__ __align__(16) Pair vals[TR][TC / 2];
  const GroupTable g = build_group_table<256>(offsets, E, T, TR, 128, table_mem, status, blockIdx.x == 0);
  const uint32_t tiles_c = static_cast<uint32_t>(C / TC);
  TileRun run(static_cast<uint32_t>(g.pa[E]) * tiles_c, blockIdx.x, gridDim.x);
  if (run.tile >= run.end) return;
  [[maybe_unused]] float q[16];
  if constexpr (INV) inverse_factors(sign_bits(philox_keys(seed)), q);
  GroupTile t = group_tile(g, run.tile, tiles_c);
  const int th = threadIdx.x;
  const int pair = th >> 2, b = th & 3;   // column pair and 16-row block
  // the next tile's codes and scales are on their way while this one is
  // written (8 bytes per column and thread leave little in flight otherwise)
  struct Column {
    uint2 p;
    uint32_t s;
  } na, nb;
  auto fetch = [&](const GroupTile& f) {
    const int64_t c = static_cast<int64_t>(f.tc) * TC + 2 * pair, kt = g.pa[f.e] + f.tr;
    const uint8_t* src = codes + c * (kcap / 2) + 32 * kt + 8 * b;
    const uint8_t* sc = scales + gemm_scale_offset(c, 4 * kt + b, kcap / 16);   // column c + 1: the next 16-byte line
    na.p = __ldg(reinterpret_cast<const uint2*>(src));
    nb.p = __ldg(reinterpret_cast<const uint2*>(src + kcap / 2));
    na.s = __ldg(sc);
    nb.s = __ldg(sc + 16);
  };
  fetch(t);
  GroupTile ahead = t;
  for (; run.tile < run.end; ++run.tile, t = ahead) {
    if (run.tile + 1 == run.end) pdl_release();
    const int left = g.rows(t.e) - t.tr * TR;
    const int rows = left < TR ? left : TR;
    const int64_t c0 = static_cast<int64_t>(t.tc) * TC;
    const float al = __ldg(alpha + t.e);
    const uint2 pa = na.p, pb = nb.p;
    const float sa = __fmul_rn(al, e4m3_value(na.s)), sb = __fmul_rn(al, e4m3_value(nb.s));
    next_tile(g, ahead, tiles_c);
    if (run.tile + 1 < run.end) fetch(ahead);
    float va[16], vb[16];
    e2m1x8_values(pa.x, va);
    e2m1x8_values(pa.y, va + 8);
    e2m1x8_values(pb.x, vb);
    e2m1x8_values(pb.y, vb + 8);
    float2 u[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      // with INV scalar: a packed product could be merged into the first addition
      u[j] = INV ? make_float2(__fmul_rn(va[j], sa), __fmul_rn(vb[j], sb)) : mul2(make_float2(va[j], vb[j]), make_float2(sa, sb));
    }
    if constexpr (INV) irht16x2(u, q);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      if constexpr (BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(u[j].x, u[j].y);
        vals[16 * b + j][pair ^ (kSwap * b)] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        vals[16 * b + j][pair ^ (kSwap * b)] = u[j];
      }
    }
    __syncthreads();
    constexpr int kPieces = TC * (BF16 ? 2 : 4) / 16;   // 16-byte pieces of a row
    constexpr int kEach = 16 / (BF16 ? 2 : 4);          // their elements
    const int64_t row0 = static_cast<int64_t>(g.off[t.e]) + t.tr * TR;
#pragma unroll
    for (int i = 0; i < TR * kPieces / 256; ++i) {
      const int k = th + 256 * i, r = k / kPieces, piece = k % kPieces;
      if (r < rows) {
        const int64_t at = (row0 + r) * C + c0 + kEach * piece;
        uint4* dst = BF16 ? reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + at)
                          : reinterpret_cast<uint4*>(static_cast<float*>(y) + at);
        *dst = *reinterpret_cast<const uint4*>(&vals[r][(kEach / 2 * piece) ^ (kSwap * (r >> 4))]);
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// CTAs for the tiles that T rows in E groups can make: `per_sm` on each SM
// where there are as many tiles, and up to `most` times as many while each
// keeps a run of six (whole multiples: 3.6 times as many took 182 us where
// 4 times took 172).  Shorter runs keep the CTAs of a moment closer together
// in memory; below six the group table of each CTA costs more.  16301 x
// 14336 in 64 groups, per_sm alone / this / runs of two: column decode 148 /
// 124 / 142 us, row decode 123 / 115 / 130; rotated amax and encoding (both
// orientations, to nearest) 411 us with per_sm CTAs, 391 with 4 times as many
// for the encoding, 403 with 8 times.  16384 x 4096 in 8 groups: column decode
// 38.6 us, with runs of one or two 50.
int grid_for(int64_t T, int64_t E, int64_t tiles_c, int per_sm, int most) {
  const int64_t tiles = grouped_capacity(T, E, TR) / TR * tiles_c, one = static_cast<int64_t>(sm_count()) * per_sm;
  const int64_t times = std::max<int64_t>(1, std::min<int64_t>(most, tiles / (6 * one)));
  return static_cast<int>(std::max<int64_t>(1, std::min(tiles, times * one)));
}

// Once per kernel and device: raise the dynamic shared memory limit.
template <class F>
cudaError_t allow_smem(F fn, int bytes, bool* done) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  return e;
}

template <int MODE, bool ROT, bool ROW, bool COL>
cudaError_t launch_encode(const GroupedArgs& a, cudaStream_t st) {
  auto fn = grouped_quantize_kernel<MODE, ROT, ROW, COL>;
  static bool done[64] = {false};
  constexpr int ring = 2 * TR * TC * 2;
  cudaError_t e = allow_smem(fn, ring + static_cast<int>(group_table_bytes(kMaxGroups)), done);
  if (e != cudaSuccess) return e;
  e = launch_k(fn, dim3(grid_for(a.T, a.E, a.tiles_c, encode_ctas<MODE, ROW, COL>(), 4)), dim3(encode_threads<MODE>()), ring + group_table_bytes(a.E), st, 1u, a);
  note_launch();
  return e;
}

template <int MODE, bool ROT>
cudaError_t dispatch_encode(const GroupedArgs& a, bool row, bool col, cudaStream_t st) {
  if (row && col) return launch_encode<MODE, ROT, true, true>(a, st);
  return row ? launch_encode<MODE, ROT, true, false>(a, st) : launch_encode<MODE, ROT, false, true>(a, st);
}

cudaError_t launch_group_amax(const GroupedArgs& a, bool row, bool col, bool rot, cudaStream_t st) {
  const size_t tab = group_table_bytes(a.E);
  cudaError_t e;
  if (!rot) e = launch_k(grouped_amax_plain_kernel, dim3(grid_for(a.T, a.E, a.tiles_c, 6, 1)), dim3(kPlainNT), tab, st, 1u, a);
  else {
    const dim3 grid(grid_for(a.T, a.E, a.tiles_c, 6, 1));
    if (row && col) e = launch_k(grouped_amax_rot_kernel<true, true>, grid, dim3(kRotNT), tab, st, 1u, a);
    else if (row) e = launch_k(grouped_amax_rot_kernel<true, false>, grid, dim3(kRotNT), tab, st, 1u, a);
    else e = launch_k(grouped_amax_rot_kernel<false, true>, grid, dim3(kRotNT), tab, st, 1u, a);
  }
  note_launch();
  return e;
}

template <int MODE, bool ROT>
cudaError_t launch_few(const GroupedArgs& a, cudaStream_t st) {
  const cudaError_t e = launch_k(grouped_quantize_few_kernel<MODE, ROT>, dim3(static_cast<unsigned>(kFewSplit * a.E)),
                                 dim3(kFewNT), group_table_bytes(a.E), st, kFewSplit, a);
  note_launch();
  return e;
}

template <bool INV, bool BF16>
cudaError_t launch_decode(const uint8_t* codes, const uint8_t* scales, const float* alpha, int64_t T, int64_t C,
                          const int32_t* offsets, int E, bool col, uint64_t seed, void* y, int32_t* status,
                          cudaStream_t st) {
  const size_t tab = group_table_bytes(E);
  cudaError_t e;
  if (col) {
    static bool done[64] = {false};
    auto fn = grouped_dequantize_cols_kernel<INV, BF16>;
    if ((e = allow_smem(fn, static_cast<int>(group_table_bytes(kMaxGroups)), done)) != cudaSuccess) return e;
    e = launch_k(fn, dim3(grid_for(T, E, C / TC, 8, 3)), dim3(256), tab, st, 1u, codes, scales, alpha, T, C, offsets, E,
                 grouped_capacity(T, E, 64), seed, y, status);
  } else {
    e = launch_k(grouped_dequantize_rows_kernel<INV, BF16>, dim3(grid_for(T, E, (C + 255) / 256, 8, 3)), dim3(256), tab, st, 1u,
                 codes, scales, alpha, T, C, offsets, E, seed, y, status);
  }
  note_launch();
  return e;
}

}  // namespace

size_t grouped_workspace_bytes(int64_t E) { return static_cast<size_t>(2 * E) * sizeof(uint32_t); }

cudaError_t grouped_quantize_launch(const void* x, int64_t T, int64_t C, int64_t ld, const int32_t* offsets, int64_t E,
                                    int mode, uint32_t flags, uint64_t seed, uint32_t stream_id, const QuantOutputs& o,
                                    void* workspace, cudaStream_t st) {
  const bool row = flags & kRowwise, col = flags & kColwise;
  const bool rot = mode == kModeRhtSR || mode == kModeMsEden || mode == kModeRhtSRHw || (flags & kRht);
  GroupedArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.T = T;
  a.C = C;
  a.ld = ld;
  a.offsets = offsets;
  a.E = static_cast<int>(E);
  a.seed = seed;
  a.stream_id = stream_id;
  a.flags = flags;
  a.amax_r = static_cast<uint32_t*>(workspace);
  a.amax_c = rot ? a.amax_r + E : a.amax_r;
  a.codes_row = o.codes_row;
  a.scales_row = o.scales_row;
  a.alpha_row = o.alpha_row;
  a.codes_col = o.codes_col;
  a.scales_col = o.scales_col;
  a.alpha_col = o.alpha_col;
  a.amax_out = o.amax_out;
  a.status = o.status;
  a.tiles_c = static_cast<uint32_t>((C + TC - 1) / TC);
  a.kcap = grouped_capacity(T, E, 64);
  if (row && !col && T <= kFewRows && E <= kFewGroups) {
    switch (mode) {
      case kModeRTN: return rot ? launch_few<kModeRTN, true>(a, st) : launch_few<kModeRTN, false>(a, st);
      case kModeFourSix: return rot ? launch_few<kModeFourSix, true>(a, st) : launch_few<kModeFourSix, false>(a, st);
      case kModeRhtSR: return launch_few<kModeRhtSR, true>(a, st);
      case kModeRhtSRHw: return launch_few<kModeRhtSRHw, true>(a, st);
      default: return launch_few<kModeMsEden, true>(a, st);
    }
  }
  cudaError_t e = cudaMemsetAsync(workspace, 0, grouped_workspace_bytes(E), st);
  if (e != cudaSuccess) return e;
  if ((e = launch_group_amax(a, row, col, rot, st)) != cudaSuccess) return e;
  switch (mode) {
    case kModeRTN: return rot ? dispatch_encode<kModeRTN, true>(a, row, col, st) : dispatch_encode<kModeRTN, false>(a, row, col, st);
    case kModeFourSix:
      return rot ? dispatch_encode<kModeFourSix, true>(a, row, col, st) : dispatch_encode<kModeFourSix, false>(a, row, col, st);
    case kModeRhtSR: return dispatch_encode<kModeRhtSR, true>(a, row, col, st);
    case kModeRhtSRHw: return dispatch_encode<kModeRhtSRHw, true>(a, row, col, st);
    default: return dispatch_encode<kModeMsEden, true>(a, row, col, st);
  }
}

cudaError_t grouped_dequantize_launch(const uint8_t* codes, const uint8_t* scales, const float* alpha, int64_t T,
                                      int64_t C, const int32_t* offsets, int64_t E, uint32_t flags, uint64_t seed,
                                      void* y, int32_t* status, cudaStream_t st) {
  const bool col = flags & kColwise, inv = flags & kInverseRht, bf = flags & kOutBf16;
  const int e = static_cast<int>(E);
  if (inv)
    return bf ? launch_decode<true, true>(codes, scales, alpha, T, C, offsets, e, col, seed, y, status, st)
              : launch_decode<true, false>(codes, scales, alpha, T, C, offsets, e, col, seed, y, status, st);
  return bf ? launch_decode<false, true>(codes, scales, alpha, T, C, offsets, e, col, seed, y, status, st)
            : launch_decode<false, false>(codes, scales, alpha, T, C, offsets, e, col, seed, y, status, st);
}

}  // namespace nvfp4
