// Quantisation helpers of the append kernels: integer and FP8 E4M3 codes of
// x / scale with the IEEE fp32 quotient, mostly without the division.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

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

// FP8 E4M3 codes of 4 values of a block or row whose largest magnitude is at
// most 448 scale: byte i holds value i's.  code = E4M3(x / scale), x / scale
// the IEEE fp32 quotient.  With y = x * inv rounded (inv within one ulp of 1 /
// scale), |x / scale - y| < 2^-22 |x / scale|, so the quotient lies between
// y (1 - 2^-21) and y (1 + 2^-21); the conversion is monotone, so where both
// ends give one code the quotient gives it too.  Elsewhere (near a rounding
// border: about one value in 2^15; `exact` for a scale without a normal
// reciprocal) the division decides.  A NaN gets code 0.
__device__ __forceinline__ uint32_t e4m3_codes4(const float* x, float scale, float inv, bool exact) {
  float a[4], b[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float y = x[e] * inv;
    a[e] = y * (1.0f - 0x1p-21f);
    b[e] = y * (1.0f + 0x1p-21f);
  }
  const uint32_t lo = e4m3x4(a[0], a[1], a[2], a[3]), hi = e4m3x4(b[0], b[1], b[2], b[3]);
  if (lo == hi && !exact) return lo;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float y = scale > 0.0f ? __fdiv_rn(x[e], scale) : 0.0f;
    a[e] = y == y ? y : 0.0f;
  }
  return e4m3x4(a[0], a[1], a[2], a[3]);
}

}  // namespace quant
}  // namespace kvc
