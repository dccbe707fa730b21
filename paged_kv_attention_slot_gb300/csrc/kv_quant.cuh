// What the KV writes share: quantisation of bf16 rows to a pool's type.
#pragma once

#include "ptx.cuh"

namespace pkv {

// 8 bf16 -> 8 E4M3 codes: code = E4M3_RNE_satfinite(float(x) * inv_scale), product in fp32
__device__ __forceinline__ uint2 quant_e4m3x8(const uint4 x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float lo = __uint_as_float(w[j] << 16) * inv;
    const float hi = __uint_as_float(w[j] & 0xffff0000u) * inv;
    b[j] = f32x2_to_e4m3x2(lo, hi);
  }
  return make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
}

// Quotients t / s rounded to nearest without a division: q = t r with r = 1 / s rounded, then one Newton step on
// the quotient (Markstein's correction), two quotients at a time.  It takes u = -t and -r: the step is then
// q - r (q s - t), whose sums keep the sign of t = -0 where t - q s would be +0.  The caller keeps t / s away
// from over- and underflow.
__device__ __forceinline__ uint64_t div2_rn(uint64_t u2, uint64_t s2, uint64_t minus_r2) {
  const uint64_t q2 = fmul2(u2, minus_r2);
  return ffma2(ffma2(q2, s2, u2), minus_r2, q2);
}

// The 16 codes of a block of bf16 pairs w under the block scale s (r = 1 / s rounded).  CLAMP: values may be
// beyond 2688 = 6 * 448, where the scale is 448 and the code 6, infinities included.
template <bool CLAMP>
__device__ __forceinline__ uint2 quant_codes(const uint32_t (&w)[8], float inv, float s, float r) {
  const uint64_t minus_inv2 = f2pack(-inv, -inv), minus_r2 = f2pack(-r, -r), s2 = f2pack(s, s);
  uint32_t c[2];
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    float q[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x = w[4 * v + j];
      uint64_t u2 = fmul2(f2pack(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)), minus_inv2);
      if constexpr (CLAMP) {
        float lo, hi;
        f2unpack(u2, lo, hi);
        u2 = f2pack(fminf(fmaxf(lo, -2688.f), 2688.f), fminf(fmaxf(hi, -2688.f), 2688.f));
      }
      f2unpack(div2_rn(u2, s2, minus_r2), q[2 * j], q[2 * j + 1]);
    }
    c[v] = f32x8_to_e2m1x8(q);
  }
  return make_uint2(c[0], c[1]);
}

// One block of 16 bf16 values (two 16-byte vectors) to its E4M3 scale code and 8 bytes of E2M1 codes.
// The largest magnitude is found on the bf16 bits (scaling is monotonic), two at a time; a NaN's are
// above infinity's.
__device__ __forceinline__ uint2 quant_block(const uint4 a, const uint4 b, float inv, uint32_t& sf) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t top = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = __vmaxu2(top, w[j] & 0x7fff7fffu);
  top = max(top & 0xffffu, top >> 16);
  const float amax = fminf(__uint_as_float(top << 16) * inv, 1e30f);  // (above 2688 the scale is 448 in any case)
  const float sixth = 1.f / 6.f, q6 = amax * sixth;
  sf = f32x2_to_e4m3x2(fmaf(fmaf(-q6, 6.f, amax), sixth, q6), 0.f) & 0xffu;
  if (top > 0x7f80u) sf = 0x7fu;  // a NaN
  if (sf == 0 || sf == 0x7fu) return make_uint2(0u, 0u);
  // an E4M3 value's reciprocal is never near the middle of two floats, so one Newton step rounds it
  const float s = e4m3_to_f32(sf), r0 = rcp_approx(s), r = fmaf(fmaf(-s, r0, 1.f), r0, r0);
  if (amax > 1e6f) return quant_codes<true>(w, inv, s, r);
  return quant_codes<false>(w, inv, s, r);
}

}  // namespace pkv
