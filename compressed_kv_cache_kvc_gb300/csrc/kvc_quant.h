// Quantisation helpers of the append kernels: integer and FP8 E4M3 codes of
// x / scale with the IEEE fp32 quotient, mostly without the division.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kvc_tc.h"

namespace kvc {
namespace quant {

// Four fp32 values -> four FP8 E4M3 codes (byte i = value i), rounded to
// nearest even and saturated to +-448 by the conversion instruction (which
// packs its first source into the upper byte).
__device__ __forceinline__ uint32_t e4m3x4(float y0, float y1, float y2, float y3) {
  uint32_t w;
  asm("{\n .reg .b16 l, h;\n"
      " cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n"
      " cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n"
      " mov.b32 %0, {l, h};\n}"
      : "=r"(w)
      : "f"(y0), "f"(y1), "f"(y2), "f"(y3));
  return w;
}

// Integer codes of 8 values of a row, as words whose low byte is the
// two's-complement 8-bit code and whose low nibble is the 4-bit one
// (0x4B400000 + code: the fp32 bit pattern of 1.5 * 2^23 + code).
//
// code = round-half-even(x / scale) with x / scale the IEEE fp32 quotient,
// clamped, as in quantize_row.  Here the code comes, where that decides it,
// from the exact product P = x * inv, inv an approximate reciprocal of the
// scale (relative error at most 2^-23, one ulp): P differs from the rounded
// quotient by at most 2^-23 |x / scale| + 2^-24 |x / scale| < 2^-14.4,
// because |x| <= amax gives |x / scale| <= qmax (1 + 2^-23) < 128 (the scale
// is a normal number here; a subnormal one has an infinite reciprocal under
// ftz).  One fused multiply-add rounds P + 1.5 * 2^23 to the integer r
// nearest P (round to nearest even in the binade of unit spacing); a second
// gives P - r.  Where |P - r| < 1/2 - 2^-12 the quotient lies in the same
// unit interval around r and rounds to r, and |r| <= qmax needs no clamp.
// Elsewhere (P within about 2^-12 of a half-integer, or not finite) the
// division decides.  About one value in 2^11 takes that path.
__device__ __forceinline__ float rcp_approx_ftz(float a) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
  return r;
}

template <int BITS>
__device__ __forceinline__ void int_codes8(const float* x, float scale, float inv, uint32_t (&w)[8]) {
  constexpr float kM = 12582912.0f;  // 1.5 * 2^23
  constexpr float kNear = 0.5f - 0x1p-12f;
  constexpr int kLo = BITS == 8 ? -127 : -8;
  constexpr int kHi = BITS == 8 ? 127 : 7;
  bool slow = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float sm = __fmaf_rn(x[e], inv, kM);
    w[e] = __float_as_uint(sm);
    slow |= !(fabsf(__fmaf_rn(x[e], inv, -__fadd_rn(sm, -kM))) < kNear);
  }
  if (slow) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float r = __fadd_rn(__fmaf_rn(x[e], inv, kM), -kM);
      if (!(fabsf(__fmaf_rn(x[e], inv, -r)) < kNear)) {
        const int q = scale > 0.0f ? min(max(__float2int_rn(__fdiv_rn(x[e], scale)), kLo), kHi) : 0;
        w[e] = 0x4B400000u + (uint32_t)q;
      }
    }
  }
}

// the low bytes of four words, in order
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Codes of 8 bf16 values (four words) of a block whose largest magnitude is at
// most qmax scale: byte i of the result holds value i's code of x / scale, the
// IEEE fp32 quotient.  A NaN gets code 0, and so does every value of a block
// whose scale is 0 or infinite, but for E4M3's signed zeros.
//
// The division, for the values of bit mask m: one value a turn, each lane its
// own.  A quotient near a border is no rare thing among bf16 values (x = amax /
// 2 lies at 63.5 steps): one group of 32 lanes x 8 normal values in three has
// one, so that eight divisions for it would cost more than all the rest.
template <bool FP8>
__device__ __noinline__ uint2 block_codes8_div(uint4 w, uint2 o, uint32_t m, float scale) {
  while (m) {
    const int e = __ffs(m) - 1;
    m &= m - 1;
    const uint32_t wd = e < 4 ? (e < 2 ? w.x : w.y) : (e < 6 ? w.z : w.w);
    const float x = __uint_as_float(e & 1 ? wd & 0xFFFF0000u : wd << 16);
    float y = scale > 0.0f ? __fdiv_rn(x, scale) : 0.0f;
    y = y == y ? y : 0.0f;
    const uint32_t code = FP8 ? e4m3x4(y, 0.0f, 0.0f, 0.0f) : (uint32_t)min(max(__float2int_rn(y), -127), 127);
    const int sh = 8 * (e & 3);
    const uint32_t keep = ~(0xFFu << sh), put = (code & 0xFFu) << sh;
    if (e < 4)
      o.x = (o.x & keep) | put;
    else
      o.y = (o.y & keep) | put;
  }
  return o;
}

// Two values an instruction.  INT8: as int_codes8, with the border at 1/2 -
// 2^-14 (the two quotients differ by less than 2^-14.4, the residual's own
// rounding is below 2^-25), so that about one value in 2^13 divides.  E4M3:
// with y = x * inv rounded (inv within one ulp of 1 / scale), |x / scale - y| <
// 2^-22 |x / scale|, so the quotient lies between y (1 - 2^-21) and
// y (1 + 2^-21); the conversion is monotone, so where both ends give one code
// the quotient gives it too (elsewhere, about one value in 2^15, the division
// decides).  `exact`: a scale without a normal reciprocal divides throughout.
template <bool FP8>
__device__ __forceinline__ uint2 block_codes8(uint4 w, float scale, float inv, bool exact) {
  const uint32_t wd[4] = {w.x, w.y, w.z, w.w};
  const tc::f32x2 inv2 = tc::pack2(inv, inv);
  float top = 0.0f;  // NaN if any value is
  uint2 o;
  uint32_t m = 0;
  if (FP8) {
    constexpr float kLo = 1.0f - 0x1p-21f, kHi = 1.0f + 0x1p-21f;
    const tc::f32x2 lo2 = tc::pack2(kLo, kLo), hi2 = tc::pack2(kHi, kHi);
    float a[8], b[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const tc::f32x2 y =
          tc::mul2(tc::pack2(__uint_as_float(wd[e] << 16), __uint_as_float(wd[e] & 0xFFFF0000u)), inv2);
      tc::unpack2(tc::mul2(y, lo2), a[2 * e], a[2 * e + 1]);
      tc::unpack2(tc::mul2(y, hi2), b[2 * e], b[2 * e + 1]);
      top = tc::max3_abs_nan(a[2 * e], a[2 * e + 1], top);
    }
    o = make_uint2(e4m3x4(a[0], a[1], a[2], a[3]), e4m3x4(a[4], a[5], a[6], a[7]));
    const uint2 u = make_uint2(e4m3x4(b[0], b[1], b[2], b[3]), e4m3x4(b[4], b[5], b[6], b[7]));
    if (o.x == u.x && o.y == u.y && top < INFINITY && !exact) return o;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t d = e < 4 ? (o.x ^ u.x) >> (8 * e) : (o.y ^ u.y) >> (8 * (e - 4));
      m |= (uint32_t)((d & 0xFFu) != 0u || !(fabsf(a[e]) < INFINITY)) << e;
    }
  } else {
    constexpr float kM = 12582912.0f;  // 1.5 * 2^23
    constexpr float kNear = 0.5f - 0x1p-14f;
    float d[8];
    const tc::f32x2 m2 = tc::pack2(kM, kM), neg = tc::pack2(-1.0f, -1.0f);
    uint32_t q[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const tc::f32x2 x = tc::pack2(__uint_as_float(wd[e] << 16), __uint_as_float(wd[e] & 0xFFFF0000u));
      const tc::f32x2 r = tc::fma2(x, inv2, m2);  // kM + the nearest integer
      float r0, r1;
      tc::unpack2(r, r0, r1);
      tc::unpack2(tc::fma2(x, inv2, tc::fma2(r, neg, m2)), d[2 * e], d[2 * e + 1]);
      q[2 * e] = __float_as_uint(r0);
      q[2 * e + 1] = __float_as_uint(r1);
      top = tc::max3_abs_nan(d[2 * e], d[2 * e + 1], top);
    }
    o = make_uint2(low_bytes(q[0], q[1], q[2], q[3]), low_bytes(q[4], q[5], q[6], q[7]));
    if (top < kNear && !exact) return o;
#pragma unroll
    for (int e = 0; e < 8; ++e) m |= (uint32_t)!(fabsf(d[e]) < kNear) << e;
  }
  return block_codes8_div<FP8>(w, o, exact ? 0xFFu : m, scale);
}

}  // namespace quant
}  // namespace kvc
