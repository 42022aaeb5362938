// grouped_gemm.cu -- block-scaled NVFP4 products of ragged groups on the
// sm_100a tensor cores (the expert layers of a mixture model).
//
//   rows grouped (forward, data gradient):
//     D[m, n] = alphaA[e] alphaB[e] sum_k (qA DeltaA)[m, k] (qB DeltaB)[e, n, k],  m in group e
//   contraction grouped (weight gradient):
//     D[e, m, n] = alphaA[e] alphaB[e] sum_{t in group e} (qA DeltaA)[m, t] (qB DeltaB)[n, t]
//
// One persistent launch covers every group: a CTA pair (cluster of 2)
// computes 256 x 256 tiles with tcgen05.mma.cta_group::2 as the plain GEMM
// does, and maps a running tile index to (group, m tile, n tile) with prefix
// sums of the device-side offsets, so the host never waits for them.
//   * rows grouped: A's codes are dense, so a group's last tile also loads
//     rows of the next group; the products of those rows are computed and not
//     stored.  A's scales sit in 128-row atoms, each group starting a new one.
//   * contraction grouped: a group's tokens are padded with zero codes to 64
//     (one MMA's K), and only its own K blocks are multiplied.
// 16384 tokens of 8 groups x 14336 x 4096 take 374 us in a short run (5.1
// PFLOP/s, bf16 results) and about 465 in long ones, under the power cap; the
// tensor pipe is busy 67% of the time (the plain GEMM's 70%), the operands
// come from L2 at 11 TB/s, a third of what that way carries.  The fp32 weight
// gradient of the same sizes takes 595 to 615 us, 705 to 715 in long runs: the
// tensor pipe is busy 40% of the time (54% with bf16 results), operands come at
// 7 TB/s, DRAM is at 37%.  None of them is at its limit; it is the results'
// way out that costs: a tile has eight stages of products (2048 tokens of a
// group), then 256 KB of results leave the one accumulator through one small
// box per warp (GroupedCfg).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>
#include <cstring>

#include "nvfp4_device.cuh"
#include "gemm_ptx.cuh"
#include "grouped.cuh"
#include "launch.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

constexpr int G_STAGE_AB = 128 * BK_BYTES;          // own 128 rows of one operand, 256 K
constexpr int G_SF = KB_PER_STAGE * 512;            // scales of 128 rows, 256 K
constexpr int G_STAGE = 2 * G_STAGE_AB + 3 * G_SF;  // A, B, own A scales, all 256 B rows' scales
constexpr int G_EPI_WARPS = 8;
constexpr int G_THREADS = 64 + 32 * G_EPI_WARPS;
constexpr int G_TABLE = static_cast<int>(group_table_bytes(kMaxGroups));
// Output staging: a 16-row x 128-byte box per epilogue warp, or (WIDE) two of
// 32 rows, for which the operand ring gives up one of its five stages.
// Measured, narrow against wide, 14336 x 4096 outputs per group: weight
// gradient of 8 x 2048 tokens fp32 614 / 707 us, bf16 475 / 551; of 8 x 256
// tokens fp32 385 / 410, bf16 236 / 214; 64 groups of 62 tokens, 1408 x 2048,
// fp32 171 / 164, bf16 111 / 88.  So the wide form is for bf16 weight
// gradients of few tokens per group.  (Plain stores of whole 128-byte lines
// by the threads were slower than the narrow boxes nearly everywhere.)
template <bool WIDE>
struct GroupedCfg {
  static constexpr int BOX = WIDE ? 4096 : 2048;
  static constexpr int OUT = G_EPI_WARPS * BOX * (WIDE ? 2 : 1);
  static constexpr int STAGES = (232448 - OUT - 1024 - 512 - 1024 - G_TABLE) / G_STAGE;
  static constexpr int SMEM = STAGES * G_STAGE + OUT + 1024 + 512 + G_TABLE;
};
constexpr int64_t kWideTokens = 512;   // tokens per group, on average, up to which bf16 weight gradients are wide
constexpr uint32_t G_SF_W = 12, G_SF_COL = 256, G_TMEM_COLS = 512;
// M = 256, N = 256, E2M1 x E2M1, E4M3 scales
constexpr uint32_t G_IDESC = (1u << 7) | (1u << 10) | ((256u >> 3) << 17) | ((256u >> 4) << 24);

struct GroupedGemm {
  const float* alpha_a;
  const float* alpha_b;
  const int32_t* offsets;
  int E;
  int64_t T;
  int M, N, K;        // WGRAD: M x N outputs per group; else N x K weights, M unused
  int katoms_a;       // scale atoms along K of A (and of B)
  int group_m;        // m tiles per raster group
  void* D;
  int64_t ldd;        // rows grouped: row stride of D; WGRAD: N
  int32_t* status;
};

// Where a tile's operands and outputs are.
struct TileAt {
  int e;
  int a_row, b_row;     // first operand row (TMA y)
  int x0;               // first byte along K (TMA x)
  int sfa, sfb;         // first scale atom of A's and of B's 128 rows
  int kblocks;          // K / 64
  int row0, rows;       // first output row of D, rows that are stored
  int col0, cols;       // first output column, columns that are stored
};

template <bool WGRAD>
__device__ __forceinline__ TileAt locate(const GroupTable& g, const GroupedGemm& p, int tile, int n_tiles) {
  TileAt t;
  int tm, tn;
  if constexpr (!WGRAD) {
    // prefix pa counts 256-row tiles, pb 128-row scale atoms
    t.e = find_group(g.pa, g.E, tile / n_tiles);
    const int m_tiles = g.pa[t.e + 1] - g.pa[t.e];
    pair_tile_coords(tile - g.pa[t.e] * n_tiles, m_tiles, n_tiles, min(p.group_m, m_tiles), tm, tn);
    t.a_row = g.off[t.e] + 256 * tm;
    t.b_row = t.e * p.N + 256 * tn;
    t.x0 = 0;
    t.sfa = (g.pb[t.e] + 2 * tm) * p.katoms_a;
    t.sfb = (t.e * (p.N / 128) + 2 * tn) * p.katoms_a;
    t.kblocks = p.K / 64;
    t.row0 = t.a_row;
    t.rows = min(256, g.rows(t.e) - 256 * tm);
  } else {
    // prefix pb counts 64-token K blocks
    const int m_tiles = (p.M + 255) / 256, per = m_tiles * n_tiles;
    t.e = tile / per;
    pair_tile_coords(tile - t.e * per, m_tiles, n_tiles, min(p.group_m, m_tiles), tm, tn);
    const int k0 = g.pb[t.e];
    t.a_row = 256 * tm;
    t.b_row = 256 * tn;
    t.x0 = 32 * k0;
    t.sfa = 2 * tm * p.katoms_a + k0;
    t.sfb = 2 * tn * p.katoms_a + k0;
    t.kblocks = g.pb[t.e + 1] - k0;
    t.row0 = t.e * p.M + 256 * tm;
    t.rows = min(256, p.M - 256 * tm);
  }
  t.col0 = 256 * tn;
  t.cols = min(256, p.N - 256 * tn);
  return t;
}

template <bool WGRAD, bool FP32, bool WIDE>
__global__ void __launch_bounds__(G_THREADS, 1)
    nvfp4_grouped_gemm_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                              const __grid_constant__ CUtensorMap tmap_d, const __grid_constant__ CUtensorMap tmap_sfa,
                              const __grid_constant__ CUtensorMap tmap_sfb, const GroupedGemm p) {
  pdl_entry();
  using GC = GroupedCfg<WIDE>;
  constexpr int G_STAGES = GC::STAGES;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + G_STAGES * G_STAGE_AB;
  uint8_t* sSFA = sB + G_STAGES * G_STAGE_AB;
  uint8_t* sSFB = sSFA + G_STAGES * G_SF;
  uint8_t* sOut = sSFB + G_STAGES * 2 * G_SF;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sOut + GC::OUT);
  uint64_t* full = bars;
  uint64_t* empty = bars + G_STAGES;
  uint64_t* acc_full = bars + 2 * G_STAGES;
  uint64_t* acc_empty = bars + 2 * G_STAGES + 1;
  uint64_t* drain = bars + 2 * G_STAGES + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * G_STAGES + 3);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* table_mem = reinterpret_cast<int*>(sOut + GC::OUT + 512);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = static_cast<int>(blockIdx.x) >> 1, num_pairs = static_cast<int>(gridDim.x) >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < G_STAGES; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(acc_full), 1);
    mbar_init(smem_u32(acc_empty), 2 * G_EPI_WARPS);
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(G_TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  const GroupTable g = build_group_table<G_THREADS>(p.offsets, p.E, p.T, WGRAD ? 64 : 256, WGRAD ? 64 : 128, table_mem,
                                                    p.status, blockIdx.x == 0);
  fence_before();
  __syncwarp();
  cluster_sync();   // barriers of both CTAs initialised, TMEM allocated
  fence_after();
  const uint32_t tmem = *tmem_slot;
  const int n_tiles = (p.N + 255) / 256;
  const int num_tiles = WGRAD ? p.E * ((p.M + 255) / 256) * n_tiles : g.pa[p.E] * n_tiles;

  if (warp == 0) {
    // ---------------- producer (both CTAs, one elected lane) ----------------
    if (elect_one()) {
      int it = 0, s = 0;
      uint32_t ph = 0;
      bool stop = false;
      for (int tile = pair; tile < num_tiles && !stop; tile += num_pairs) {
        const TileAt t = locate<WGRAD>(g, p, tile, n_tiles);
        const int kstages = (t.kblocks + KB_PER_STAGE - 1) / KB_PER_STAGE;
        const int r = static_cast<int>(rank);
        for (int kt = 0; kt < kstages; ++kt, ++it) {
          if (!mbar_wait(smem_u32(&empty[s]), ph ^ 1, abort_flag)) {
            stop = true;
            break;
          }
          const uint32_t fb = map_to_rank(smem_u32(&full[s]), 0);
          const uint32_t dSB = smem_u32(sSFB + s * 2 * G_SF);
          // scale atoms viewed as rows of 256 bytes (two per atom)
          const int ysa = (t.sfa + r * p.katoms_a + KB_PER_STAGE * kt) * 2;
          const int ysb = (t.sfb + KB_PER_STAGE * kt) * 2;
          if (leader) mbar_expect_tx(smem_u32(&full[s]), 2 * G_STAGE);
          tma_load_2d_pair(smem_u32(sA + s * G_STAGE_AB), &tmap_a, t.x0 + kt * BK_BYTES, t.a_row + 128 * r, fb);
          tma_load_2d_pair(smem_u32(sB + s * G_STAGE_AB), &tmap_b, t.x0 + kt * BK_BYTES, t.b_row + 128 * r, fb);
          tma_load_2d_pair(smem_u32(sSFA + s * G_SF), &tmap_sfa, 0, ysa, fb);
          tma_load_2d_pair(dSB, &tmap_sfb, 0, ysb, fb);
          tma_load_2d_pair(dSB + G_SF, &tmap_sfb, 0, ysb + 2 * p.katoms_a, fb);
          if (++s == G_STAGES) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (leader) {
        // the copies issued, the peer's among them, land before the pair exits
        for (int i = (it > G_STAGES ? it - G_STAGES : 0); i < it; ++i)
          mbar_wait_bounded(smem_u32(&full[i % G_STAGES]), (i / G_STAGES) & 1);
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (leader CTA, one elected lane) ----------------
    if (leader && elect_one()) {
      int s = 0;
      uint32_t full_ph = 0, acc_ph = 0, set = 0;
      bool stop = false;
      for (int tile = pair; tile < num_tiles && !stop; tile += num_pairs) {
        const TileAt t = locate<WGRAD>(g, p, tile, n_tiles);
        if (t.kblocks == 0) continue;   // a group without tokens: the epilogue writes zeros
        // the epilogue must have drained the previous accumulator
        if (!mbar_wait(smem_u32(acc_empty), acc_ph ^ 1, abort_flag)) break;
        acc_ph ^= 1;
        fence_after();
        for (int kb = 0; kb < t.kblocks; kb += KB_PER_STAGE) {
          if (!mbar_wait(smem_u32(&full[s]), full_ph, abort_flag)) {
            stop = true;
            break;
          }
          fence_after();
          const uint32_t sfa_s = smem_u32(sSFA + s * G_SF), sfb_s = smem_u32(sSFB + s * 2 * G_SF);
          const int nk = min(KB_PER_STAGE, t.kblocks - kb);
          const uint64_t adesc = desc_sw128(smem_u32(sA + s * G_STAGE_AB));
          const uint64_t bdesc = desc_sw128(smem_u32(sB + s * G_STAGE_AB));
          for (int kk = 0; kk < nk; ++kk) {
            // this K block's scales right before its MMA, in the slot set the
            // previous stage did not use
            const uint32_t col = tmem + G_SF_COL + (set + kk) * G_SF_W;
            tmem_cp_sf_pair(col, desc_sf(sfa_s + 512 * kk));
            tmem_cp_sf_pair(col + 4, desc_sf(sfb_s + 512 * kk));
            tmem_cp_sf_pair(col + 8, desc_sf(sfb_s + G_SF + 512 * kk));
            mma_mxf4nvf4_pair(tmem, adesc + 2 * kk, bdesc + 2 * kk, G_IDESC, (kb > 0 || kk > 0) ? 1u : 0u, col, col + 4);
          }
          set ^= KB_PER_STAGE;
          umma_commit_pair(smem_u32(&empty[s]));
          if (kb + KB_PER_STAGE >= t.kblocks) umma_commit_pair(smem_u32(acc_full));
          if (++s == G_STAGES) {
            s = 0;
            full_ph ^= 1;
          }
        }
      }
      // the MMAs issued finish before TMEM is freed
      umma_commit_pair_own(smem_u32(drain));
      mbar_wait_bounded(smem_u32(drain), 0);
    }
  } else {
    // ---------------- epilogue (warps 2..9 of both CTAs) ----------------
    const int q = warp & 3, h = (warp - 2) >> 2;
    uint8_t* buf = sOut + (warp - 2) * (GC::OUT / G_EPI_WARPS);
    uint32_t box = 0;   // WIDE: the staging box used next
    const uint32_t acc_empty_leader = map_to_rank(smem_u32(acc_empty), 0);
    const int64_t row_bytes = p.ldd * (FP32 ? 4 : 2);
    uint32_t acc_ph = 0;
    for (int tile = pair; tile < num_tiles; tile += num_pairs) {
      const TileAt t = locate<WGRAD>(g, p, tile, n_tiles);
      const bool zero = t.kblocks == 0;
      if (!zero) {
        if (!mbar_wait_warp(smem_u32(acc_full), acc_ph, abort_flag)) break;
        acc_ph ^= 1;
        fence_after();
      }
      const float ab = zero ? 0.0f : __fmul_rn(__ldg(p.alpha_a + t.e), __ldg(p.alpha_b + t.e));
      const int lrow = 128 * static_cast<int>(rank) + 32 * q;   // this warp's first row within the tile
      const int row0 = t.row0 + lrow, left = t.rows - lrow;     // rows of this warp that are stored
      const int col0 = t.col0 + 128 * h;
      const bool store = 128 * h < t.cols && left > 0;
      const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * q) << 16) + 128 * h;
      // 128 bytes of each of the warp's rows (w: this lane's row)
      auto put = [&](const uint32_t* w, int col) {
        auto stage = [&](uint8_t* rowp) {   // this lane's row into a box, 16-byte chunks swizzled by the row
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(rowp + ((j ^ (lane & 7)) << 4)) =
                make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        };
        uint8_t* out = static_cast<uint8_t*>(p.D) + static_cast<int64_t>(row0) * row_bytes + (FP32 ? 4 : 2) * static_cast<int64_t>(col);
        int boxed = 0;   // rows that left as whole boxes
        if constexpr (WIDE) {
          if (left >= 32) {
            if (lane == 0) bulk_wait_read<1>();   // the box before the previous one has been read
            __syncwarp();
            stage(buf + box * GC::BOX + lane * 128);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&tmap_d, smem_u32(buf + box * GC::BOX), col, row0);
              bulk_commit();
            }
            box ^= 1;
            boxed = 32;
          }
        } else {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (left >= 16 * half + 16) {
              if (lane == 0) bulk_wait_read<0>();   // the previous box has been read
              __syncwarp();
              if ((lane >> 4) == half) stage(buf + (lane & 15) * 128);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_2d(&tmap_d, smem_u32(buf), col, row0 + 16 * half);
                bulk_commit();
              }
              boxed = 16 * half + 16;
            }
          }
        }
        if (lane >= boxed && lane < left) {   // the rows of a box that is not whole, lane by lane
#pragma unroll
          for (int j = 0; j < 8; ++j)
            reinterpret_cast<uint4*>(out + lane * row_bytes)[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        }
      };
      if constexpr (!FP32) {
        uint32_t packed[64];
        if (zero) {
#pragma unroll
          for (int j = 0; j < 64; ++j) packed[j] = 0u;
        } else {
#pragma unroll
          for (int c = 0; c < 128; c += 64) {
            uint32_t r[64];
            tmem_ld32_nowait(taddr + c, r);
            tmem_ld32_nowait(taddr + c + 32, r + 32);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float2 v = __fmul2_rn(make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])),
                                          make_float2(ab, ab));
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(v.x, v.y);
              packed[c / 2 + j] = *reinterpret_cast<const uint32_t*>(&b2);
            }
          }
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(acc_empty_leader);
        }
        if (store) {
          put(packed, col0);
          put(packed + 32, col0 + 64);
        }
      } else {
        // the whole row goes to registers, so the accumulator is handed back
        // before anything is stored
        uint32_t r[128];
        if (zero) {
#pragma unroll
          for (int j = 0; j < 128; ++j) r[j] = 0u;
        } else {
#pragma unroll
          for (int c = 0; c < 128; c += 32) tmem_ld32_nowait(taddr + c, r + c);
          tmem_ld_wait();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(acc_empty_leader);
#pragma unroll
          for (int j = 0; j < 128; ++j) r[j] = __float_as_uint(__fmul_rn(__uint_as_float(r[j]), ab));
        }
        if (store) {
#pragma unroll
          for (int c = 0; c < 128; c += 32) put(r + c, col0 + c);
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  fence_before();
  __syncwarp();
  // neither CTA may leave (or free TMEM) while its peer can still touch its
  // shared memory or its TMEM
  cluster_sync();
  if (threadIdx.x == 0 && *abort_flag && p.status) *p.status = kStatusTimeout;
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(G_TMEM_COLS) : "memory");
  }
}

// ===========================================================================
// Few rows per group (decode, small experts): the roles are swapped.  128 rows
// of the weight are the MMA's M and up to 128 tokens of a group its N, so no
// tensor-core row and no load is spent on tokens that are not there: N is
// rounded up to 16 tile by tile, and a tile of up to 32 tokens loads 32 rows.
// One CTA per SM; what bounds it is the weights' stream from memory, so the
// ring holds as many stages as fit, and two accumulators let the next tile
// start while the epilogue drains this one.
// D^T comes out of the MMA: lane n of the accumulator is a weight row, column
// j a token; a warp stores 64 (bf16) or 128 (fp32) contiguous bytes per token.
// 16 tokens, 6 of 8 groups, 14336 x 4096: 38 us, the weights at 5.2 TB/s; 5003
// tokens of 64 groups, 1408 x 2112: 39 us, five rounds of tiles of 128 weight
// rows over 148 SMs, the last one half empty.
// ===========================================================================
constexpr int F_STAGE_W = 128 * BK_BYTES, F_STAGE_X = 128 * BK_BYTES;   // weight rows, token rows
constexpr int F_STAGE = F_STAGE_W + F_STAGE_X + 2 * G_SF;
constexpr int F_STAGES = (232448 - 1024 - 512 - 1024 - G_TABLE) / F_STAGE;
constexpr int F_SMEM = F_STAGES * F_STAGE + 1024 + 512 + G_TABLE;
constexpr int F_THREADS = 192;      // producer, MMA, four epilogue warps
constexpr int F_SMALL = 32;         // tokens up to which a tile loads F_SMALL rows
constexpr uint32_t F_ACC = 128;     // columns of an accumulator
constexpr uint32_t F_SF_COL = 2 * F_ACC, F_SF_W = 8, F_TMEM_COLS = 512;
constexpr uint32_t F_IDESC = (1u << 7) | (1u << 10) | ((128u >> 4) << 24);   // M = 128; N >> 3 at bit 17

struct FewAt {
  int e, tn, tokens;    // group, weight tile, tokens of this tile
  int w_row, x_row;     // first rows of the operands
  int sfw, sfx;         // first scale atoms
};

__device__ __forceinline__ FewAt locate_few(const GroupTable& g, const GroupedGemm& p, int tile, int n_tiles) {
  FewAt t;
  t.e = find_group(g.pb, g.E, tile / n_tiles);
  const int m_tiles = g.pb[t.e + 1] - g.pb[t.e], local = tile - g.pb[t.e] * n_tiles;
  t.tn = local / m_tiles;
  const int tm = local - t.tn * m_tiles;   // token tiles of one weight tile follow one another: it stays in L2
  t.tokens = min(128, g.rows(t.e) - 128 * tm);
  t.w_row = t.e * p.N + 128 * t.tn;
  t.x_row = g.off[t.e] + 128 * tm;
  t.sfw = (t.e * n_tiles + t.tn) * p.katoms_a;
  t.sfx = (g.pb[t.e] + tm) * p.katoms_a;
  return t;
}

template <bool FP32>
__global__ void __launch_bounds__(F_THREADS, 1)
    nvfp4_grouped_gemm_few_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                                  const __grid_constant__ CUtensorMap tmap_x_small,
                                  const __grid_constant__ CUtensorMap tmap_sfw,
                                  const __grid_constant__ CUtensorMap tmap_sfx, const GroupedGemm p) {
  pdl_entry();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sW = smem;
  uint8_t* sX = sW + F_STAGES * F_STAGE_W;
  uint8_t* sSFW = sX + F_STAGES * F_STAGE_X;
  uint8_t* sSFX = sSFW + F_STAGES * G_SF;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sSFX + F_STAGES * G_SF);
  uint64_t* full = bars;
  uint64_t* empty = bars + F_STAGES;
  uint64_t* acc_full = bars + 2 * F_STAGES;        // [2]
  uint64_t* acc_empty = bars + 2 * F_STAGES + 2;   // [2]
  uint64_t* drain = bars + 2 * F_STAGES + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * F_STAGES + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* table_mem = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + 512);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < F_STAGES; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&acc_full[i]), 1);
      mbar_init(smem_u32(&acc_empty[i]), 4);   // one arrival per epilogue warp
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(F_TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  const GroupTable g =
      build_group_table<F_THREADS>(p.offsets, p.E, p.T, 128, 128, table_mem, p.status, blockIdx.x == 0);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  const int n_tiles = p.N / 128, num_tiles = g.pb[p.E] * n_tiles;
  const int kblocks = p.K / 64, kstages = (kblocks + KB_PER_STAGE - 1) / KB_PER_STAGE;

  if (warp == 0) {
    // ---------------- producer ----------------
    if (elect_one()) {
      int it = 0, s = 0;
      uint32_t ph = 0;
      bool stop = false;
      for (int tile = blockIdx.x; tile < num_tiles && !stop; tile += gridDim.x) {
        const FewAt t = locate_few(g, p, tile, n_tiles);
        const bool small = t.tokens <= F_SMALL;
        const uint32_t bytes = F_STAGE_W + 2 * G_SF + (small ? F_SMALL : 128) * BK_BYTES;
        for (int kt = 0; kt < kstages; ++kt, ++it) {
          if (!mbar_wait(smem_u32(&empty[s]), ph ^ 1, abort_flag)) {
            stop = true;
            break;
          }
          const uint32_t fb = smem_u32(&full[s]);
          mbar_expect_tx(fb, bytes);
          tma_load_2d(smem_u32(sW + s * F_STAGE_W), &tmap_w, kt * BK_BYTES, t.w_row, fb);
          tma_load_2d(smem_u32(sX + s * F_STAGE_X), small ? &tmap_x_small : &tmap_x, kt * BK_BYTES, t.x_row, fb);
          tma_load_2d(smem_u32(sSFW + s * G_SF), &tmap_sfw, 0, (t.sfw + KB_PER_STAGE * kt) * 2, fb);
          tma_load_2d(smem_u32(sSFX + s * G_SF), &tmap_sfx, 0, (t.sfx + KB_PER_STAGE * kt) * 2, fb);
          if (++s == F_STAGES) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      // the copies issued land before the CTA exits
      for (int i = (it > F_STAGES ? it - F_STAGES : 0); i < it; ++i)
        mbar_wait_bounded(smem_u32(&full[i % F_STAGES]), (i / F_STAGES) & 1);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (elect_one()) {
      int s = 0, buf = 0;
      uint32_t full_ph = 0, acc_ph = 0, set = 0;
      bool stop = false;
      for (int tile = blockIdx.x; tile < num_tiles && !stop; tile += gridDim.x) {
        const FewAt t = locate_few(g, p, tile, n_tiles);
        const uint32_t idesc = F_IDESC | ((static_cast<uint32_t>((t.tokens + 15) & ~15) >> 3) << 17);
        // the epilogue must have drained this accumulator's previous tile
        if (!mbar_wait(smem_u32(&acc_empty[buf]), acc_ph ^ 1, abort_flag)) break;
        fence_after();
        const uint32_t acc = tmem + buf * F_ACC;
        for (int kt = 0; kt < kstages; ++kt) {
          if (!mbar_wait(smem_u32(&full[s]), full_ph, abort_flag)) {
            stop = true;
            break;
          }
          fence_after();
          const uint32_t sfw = smem_u32(sSFW + s * G_SF), sfx = smem_u32(sSFX + s * G_SF);
          const uint64_t wdesc = desc_sw128(smem_u32(sW + s * F_STAGE_W));
          const uint64_t xdesc = desc_sw128(smem_u32(sX + s * F_STAGE_X));
          const int nk = min(KB_PER_STAGE, kblocks - KB_PER_STAGE * kt);
          for (int kk = 0; kk < nk; ++kk) {
            const uint32_t col = tmem + F_SF_COL + (set + kk) * F_SF_W;
            tmem_cp_sf(col, desc_sf(sfw + 512 * kk));
            tmem_cp_sf(col + 4, desc_sf(sfx + 512 * kk));
            mma_mxf4nvf4(acc, wdesc + 2 * kk, xdesc + 2 * kk, idesc, (kt > 0 || kk > 0) ? 1u : 0u, col, col + 4);
          }
          set ^= KB_PER_STAGE;
          umma_commit(smem_u32(&empty[s]));
          if (kt == kstages - 1) umma_commit(smem_u32(&acc_full[buf]));
          if (++s == F_STAGES) {
            s = 0;
            full_ph ^= 1;
          }
        }
        buf ^= 1;
        if (buf == 0) acc_ph ^= 1;
      }
      // the MMAs issued finish before TMEM is freed
      umma_commit(smem_u32(drain));
      mbar_wait_bounded(smem_u32(drain), 0);
    }
  } else {
    // ---------------- epilogue (warps 2..5) ----------------
    const int q = warp & 3;
    int buf = 0;
    uint32_t acc_ph = 0;
    for (int tile = blockIdx.x; tile < num_tiles; tile += gridDim.x) {
      const FewAt t = locate_few(g, p, tile, n_tiles);
      const float ab = __fmul_rn(__ldg(p.alpha_a + t.e), __ldg(p.alpha_b + t.e));
      if (!mbar_wait_warp(smem_u32(&acc_full[buf]), acc_ph, abort_flag)) break;
      fence_after();
      const uint32_t taddr = tmem + buf * F_ACC + (static_cast<uint32_t>(32 * q) << 16);
      const int64_t n = 128 * static_cast<int64_t>(t.tn) + 32 * q + lane;   // this lane's output column
      for (int c = 0; c < t.tokens; c += 32) {
        uint32_t r[32];
        tmem_ld32_nowait(taddr + c, r);
        tmem_ld_wait();
        if (c + 32 >= t.tokens) {
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&acc_empty[buf]));
        }
        const int64_t row = t.x_row + c;
        if constexpr (FP32) {
          float* out = static_cast<float*>(p.D) + row * p.ldd + n;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c + j < t.tokens) out[j * p.ldd] = __fmul_rn(__uint_as_float(r[j]), ab);
        } else {
          // neighbouring lanes exchange, so that an even lane holds two
          // columns of token j and an odd one of token j + 1
          const bool odd = lane & 1;
          uint16_t* out = static_cast<uint16_t*>(p.D) + row * p.ldd + (n & ~int64_t(1));
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float v0 = __fmul_rn(__uint_as_float(r[j]), ab), v1 = __fmul_rn(__uint_as_float(r[j + 1]), ab);
            const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? v0 : v1, 1);
            const __nv_bfloat162 b2 = odd ? __floats2bfloat162_rn(got, v1) : __floats2bfloat162_rn(v0, got);
            const int tok = j + (odd ? 1 : 0);
            if (c + tok < t.tokens) *reinterpret_cast<uint32_t*>(out + tok * p.ldd) = *reinterpret_cast<const uint32_t*>(&b2);
          }
        }
      }
      buf ^= 1;
      if (buf == 0) acc_ph ^= 1;
    }
  }
  fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag && p.status) *p.status = kStatusTimeout;
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(F_TMEM_COLS) : "memory");
  }
}

// Tokens per group, on average, up to which the swapped form is taken.  Timed
// by themselves, pair form against swapped, bf16 results: 64 groups, 1408 x
// 2112: 44 / 40 us at 4 tokens each, 52 / 49 at 64, 53 / 57 at 96; 8 groups,
// 14336 x 4096: 81 / 66, 75 / 72, 77 / 74, and 79 / 84 at 128.
constexpr int64_t kFewTokensPerGroup = 80;

template <bool FP32>
cudaError_t launch_few(const CUtensorMap& mw, const CUtensorMap& mx, const CUtensorMap& mxs, const CUtensorMap& msw,
                       const CUtensorMap& msx, const GroupedGemm& p, int64_t most_tiles, cudaStream_t st) {
  auto fn = nvfp4_grouped_gemm_few_kernel<FP32>;
  static bool done[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !done[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, F_SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev] = true;
  }
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(most_tiles, sm_count()));
  const cudaError_t e =
      launch_k(fn, dim3(static_cast<unsigned>(grid)), dim3(F_THREADS), F_SMEM, st, 1u, mw, mx, mxs, msw, msx, p);
  note_launch();
  return e;
}

template <bool WGRAD, bool FP32, bool WIDE>
cudaError_t launch_grouped(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& md, const CUtensorMap& msa,
                           const CUtensorMap& msb, const GroupedGemm& p, int64_t most_tiles, cudaStream_t st) {
  auto fn = nvfp4_grouped_gemm_kernel<WGRAD, FP32, WIDE>;
  static bool done[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !done[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, GroupedCfg<WIDE>::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev] = true;
  }
  const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(most_tiles, sm_count() / 2));
  const cudaError_t e = launch_k(fn, dim3(static_cast<unsigned>(2 * pairs)), dim3(G_THREADS), GroupedCfg<WIDE>::SMEM, st, 2u, ma,
                                 mb, md, msa, msb, p);
  note_launch();
  return e;
}

// m tiles per raster group, as the plain GEMM chooses them: the group's A
// panels and all of B within about 64 MB of L2 (k: the contraction's length)
int raster_group(int64_t k, int64_t n_tiles) {
  const int64_t panel = 256 * (k / 2 + k / 16);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(1 << 20, (int64_t(64) << 20) / panel - n_tiles)));
}

}  // namespace

cudaError_t grouped_gemm_launch(const uint8_t* A, const uint8_t* sA, const float* alphaA, const uint8_t* B,
                                const uint8_t* sB, const float* alphaB, const int32_t* offsets, int64_t E, int64_t T,
                                int64_t N, int64_t K, void* D, int out_dtype, int64_t ldd, int32_t* status,
                                cudaStream_t st) {
  const bool fp32 = out_dtype == NVFP4_OUT_DTYPE_FP32;
  if (T <= kFewTokensPerGroup * E) {
    CUtensorMap mw, mx, mxs, msw, msx;
    if (!make_map(&mw, B, E * N, K / 2, 128) || !make_map(&mx, A, T, K / 2, 128) || !make_map(&mxs, A, T, K / 2, F_SMALL) ||
        !make_sf_map(&msw, sB, E * N, K) || !make_sf_map(&msx, sA, grouped_capacity(T, E, 128), K))
      return cudaErrorInvalidValue;
    const GroupedGemm p{alphaA, alphaB, offsets, static_cast<int>(E), T, 0, static_cast<int>(N), static_cast<int>(K),
                        static_cast<int>(K / 64), 0, D, ldd, status};
    const int64_t most = grouped_capacity(T, E, 128) / 128 * (N / 128);
    return fp32 ? launch_few<true>(mw, mx, mxs, msw, msx, p, most, st) : launch_few<false>(mw, mx, mxs, msw, msx, p, most, st);
  }
  CUtensorMap ma, mb, md, msa, msb;
  if (!make_map(&ma, A, T, K / 2, 128) || !make_map(&mb, B, E * N, K / 2, 128) ||
      !make_sf_map(&msa, sA, grouped_capacity(T, E, 128), K) || !make_sf_map(&msb, sB, E * N, K) ||
      !make_out_map(&md, D, T, N, ldd, fp32))
    return cudaErrorInvalidValue;
  const int64_t n_tiles = (N + 255) / 256;
  GroupedGemm p{alphaA, alphaB, offsets, static_cast<int>(E), T, 0, static_cast<int>(N), static_cast<int>(K),
                static_cast<int>(K / 64), raster_group(K, n_tiles), D, ldd, status};
  const int64_t most = grouped_capacity(T, E, 256) / 256 * n_tiles;
  return fp32 ? launch_grouped<false, true, false>(ma, mb, md, msa, msb, p, most, st)
              : launch_grouped<false, false, false>(ma, mb, md, msa, msb, p, most, st);
}

cudaError_t grouped_wgrad_launch(const uint8_t* A, const uint8_t* sA, const float* alphaA, const uint8_t* B,
                                 const uint8_t* sB, const float* alphaB, const int32_t* offsets, int64_t E, int64_t T,
                                 int64_t M, int64_t N, void* D, int out_dtype, int32_t* status, cudaStream_t st) {
  const bool fp32 = out_dtype == NVFP4_OUT_DTYPE_FP32;
  const int64_t kcap = grouped_capacity(T, E, 64);
  if (kcap == 0) return cudaMemsetAsync(D, 0, static_cast<size_t>(E * M * N) * (fp32 ? 4 : 2), st);   // no token at all
  const bool wide = !fp32 && T <= kWideTokens * E;
  CUtensorMap ma, mb, md, msa, msb;
  if (!make_map(&ma, A, M, kcap / 2, 128) || !make_map(&mb, B, N, kcap / 2, 128) || !make_sf_map(&msa, sA, M, kcap) ||
      !make_sf_map(&msb, sB, N, kcap) ||
      !make_out_map(&md, D, E * M, N, N, fp32, wide ? 32 : 16))
    return cudaErrorInvalidValue;
  const int64_t n_tiles = (N + 255) / 256, m_tiles = (M + 255) / 256;
  GroupedGemm p{alphaA, alphaB, offsets, static_cast<int>(E), T, static_cast<int>(M), static_cast<int>(N), 0,
                static_cast<int>(kcap / 64), raster_group(std::max<int64_t>(64, T / E), n_tiles), D, N, status};
  const int64_t most = E * m_tiles * n_tiles;
  if (fp32) return launch_grouped<true, true, false>(ma, mb, md, msa, msb, p, most, st);
  return wide ? launch_grouped<true, false, true>(ma, mb, md, msa, msb, p, most, st)
              : launch_grouped<true, false, false>(ma, mb, md, msa, msb, p, most, st);
}

}  // namespace nvfp4
