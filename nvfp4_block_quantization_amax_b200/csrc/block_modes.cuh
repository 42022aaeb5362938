// block_modes.cuh -- one 16-element block pair in each quantization mode, and
// the amax helpers, shared by the single-tensor and the grouped quantizer.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "nvfp4_device.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {

constexpr uint32_t kNonFinite = 0xFFFFFFFFu;   // partial marker: a NaN / Inf was read

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Block-wide max of a uint32 (all threads get the result).
template <int NT>
__device__ __forceinline__ uint32_t block_max_u32(uint32_t v, uint32_t* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  __syncthreads();
  if (l == 0) red[w] = v;
  __syncthreads();
  v = (l < NT / 32) ? red[l] : 0u;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

__device__ __forceinline__ uint32_t sign_bits(const PhiloxKeys& K) {
  return philox(K, 0u, 0u, 0u, kTagSigns).x & 0xFFFFu;
}

// ---------------------------------------------------------------------------
// One mode's quantization of two lane-paired 16-element blocks (x: block a,
// y: block b), the element-wise steps done two blocks at a time.  v holds the
// (rotated) values; a block's random streams are keyed by (seed,
// c2 = 2 stream_id + orientation, block index).
// ---------------------------------------------------------------------------
// MS-EDEN scale of one block from its sums and its random word.
__device__ __forceinline__ uint32_t eden_scale(float num, float den, uint32_t word) {
  const uint32_t sc = e4m3_sr(__fdiv_rn(num, den), word >> 8);   // a select, not a branch, on den == 0
  return (den == 0.0f) ? 0u : sc;
}

// have_words: MS-EDEN only - wa / wb already hold the blocks' scale-SR words.
// c: the tensor scale's table (s and 1 / s per scale byte) and the Eq. 2
// denominators.
template <int MODE, class S>
__device__ __forceinline__ void quantize_pair(const float2* v, const S& c, const PhiloxKeys& K, uint32_t c2,
                                              uint64_t blka, uint64_t blkb, Packed16& pa, Packed16& pb,
                                              uint32_t& sba, uint32_t& sbb, bool have_words = false,
                                              uint32_t wa = 0u, uint32_t wb = 0u) {
  if constexpr (MODE == kModeRTN || MODE == kModeFourSix) {
    quantize_pair_tab<MODE == kModeFourSix>(v, c, pa, pb, sba, sbb);
  } else if constexpr (MODE == kModeMsEden) {
    // RTN codes under the provisional scale (M = 6), then the unbiasing
    // scale sum(r^2) / (alpha sum(r q)), stochastically rounded to E4M3
    float ma, mb;
    max_abs16x2(v, ma, mb);
    const float2 d6 = c.d6();
    const uint32_t prov = e4m3x2_rne(scale_quot(ma, d6.x), scale_quot(mb, d6.y));
    const float2 ta = c.ent_a(prov & 0xFFu), tb = c.ent_b(prov >> 8);
    float2 q[16], rr[16], rq[16];
    encode_decode_x2(v, make_float2(ta.y, tb.y), pa, pb, q);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      rr[i] = mul2(v[i], v[i]);
      rq[i] = mul2(v[i], q[i]);
    }
    const float2 num = sum16x2<true>(rr);
    const float2 den = mul2(c.alpha2(), sum16x2<true>(rq));
    if (!have_words) {
      const uint64_t ua = blka >> 2, ub = blkb >> 2;
      const uint4 da = philox(K, static_cast<uint32_t>(ua), static_cast<uint32_t>(ua >> 32), c2, kTagScaleSR);
      const uint4 db =
          (ua == ub) ? da : philox(K, static_cast<uint32_t>(ub), static_cast<uint32_t>(ub >> 32), c2, kTagScaleSR);
      const uint32_t sa = static_cast<uint32_t>(blka & 3), sbw = static_cast<uint32_t>(blkb & 3);
      wa = sa == 0 ? da.x : (sa == 1 ? da.y : (sa == 2 ? da.z : da.w));
      wb = sbw == 0 ? db.x : (sbw == 1 ? db.y : (sbw == 2 ? db.z : db.w));
    }
    sba = eden_scale(num.x, den.x, wa);
    sbb = eden_scale(num.y, den.y, wb);
  } else if constexpr (MODE == kModeRhtSRHw) {
    // RHT + stochastic rounding by the convert instruction: ceil scales as
    // below; one draw per block (unit blk), word g rounds elements 4g..4g+3,
    // handed over last element first so that nibble j holds element 4g + j.
    float ma, mb;
    max_abs16x2(v, ma, mb);
    const float2 d6 = c.d6();
    e4m3x2_ceil(scale_quot(ma, d6.x), scale_quot(mb, d6.y), sba, sbb);
    const float2 r2 = make_float2(c.ent_a(sba).y, c.ent_b(sbb).y);
    const uint4 da = philox(K, static_cast<uint32_t>(blka), static_cast<uint32_t>(blka >> 32), c2, kTagValueSRHw);
    const uint4 db = philox(K, static_cast<uint32_t>(blkb), static_cast<uint32_t>(blkb >> 32), c2, kTagValueSRHw);
    const uint32_t wa4[4] = {da.x, da.y, da.z, da.w}, wb4[4] = {db.x, db.y, db.z, db.w};
    float2 y[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = mul2(v[i], r2);
    uint32_t ca[4], cb[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      ca[g] = e2m1x4_sr_hw(y[4 * g + 3].x, y[4 * g + 2].x, y[4 * g + 1].x, y[4 * g].x, wa4[g]);
      cb[g] = e2m1x4_sr_hw(y[4 * g + 3].y, y[4 * g + 2].y, y[4 * g + 1].y, y[4 * g].y, wb4[g]);
    }
    // the sign nibble follows the input's sign bit, zeros included (a zero
    // reciprocal leaves magnitude 0 and the sign alone)
    const Packed16 sa = sign_codes16<false>(v), sb = sign_codes16<true>(v);
    pa.lo = (ca[0] | (ca[1] << 16)) | sa.lo;
    pa.hi = (ca[2] | (ca[3] << 16)) | sa.hi;
    pb.lo = (cb[0] | (cb[1] << 16)) | sb.lo;
    pb.hi = (cb[2] | (cb[3] << 16)) | sb.hi;
  } else {  // RHT + stochastic rounding of the values
    float ma, mb;
    max_abs16x2(v, ma, mb);
    const float2 d6 = c.d6();
    e4m3x2_ceil(scale_quot(ma, d6.x), scale_quot(mb, d6.y), sba, sbb);
    const float2 r2 = make_float2(c.ent_a(sba).y, c.ent_b(sbb).y);
    // element i uses half (i & 1) of word (i >> 1) & 3 of draw i >> 3 (unit 2 blk + draw)
    uint32_t wa8[8], wb8[8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint64_t ua = 2 * blka + j, ub = 2 * blkb + j;
      const uint4 da = philox(K, static_cast<uint32_t>(ua), static_cast<uint32_t>(ua >> 32), c2, kTagValueSR);
      const uint4 db = philox(K, static_cast<uint32_t>(ub), static_cast<uint32_t>(ub >> 32), c2, kTagValueSR);
      wa8[4 * j] = da.x; wa8[4 * j + 1] = da.y; wa8[4 * j + 2] = da.z; wa8[4 * j + 3] = da.w;
      wb8[4 * j] = db.x; wb8[4 * j + 1] = db.y; wb8[4 * j + 2] = db.z; wb8[4 * j + 3] = db.w;
    }
    float qa[16], qb[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 y = mul2(v[i], r2);
      const int w = ((i >> 3) << 2) | ((i >> 1) & 3), sh = 16 * (i & 1);
      qa[i] = e2m1_sr_value_nb(y.x, (wa8[w] >> sh) & 0xFFFFu);
      qb[i] = e2m1_sr_value_nb(y.y, (wb8[w] >> sh) & 0xFFFFu);
    }
    // the rounded values lie on the grid, so their encoding is exact (a zero
    // reciprocal gives signed zeros)
    pa.lo = e2m1x8_rne(qa[0], qa[1], qa[2], qa[3], qa[4], qa[5], qa[6], qa[7]);
    pa.hi = e2m1x8_rne(qa[8], qa[9], qa[10], qa[11], qa[12], qa[13], qa[14], qa[15]);
    pb.lo = e2m1x8_rne(qb[0], qb[1], qb[2], qb[3], qb[4], qb[5], qb[6], qb[7]);
    pb.hi = e2m1x8_rne(qb[8], qb[9], qb[10], qb[11], qb[12], qb[13], qb[14], qb[15]);
  }
}

}  // namespace nvfp4
