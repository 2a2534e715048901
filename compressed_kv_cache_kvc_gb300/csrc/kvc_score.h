// Score transforms of the attention kernels: the cap by a tanh and the bias
// that depends on the distance between query and key.
//
// With x = sm_scale * q . k, the transformed score is
//   z = cap * tanh(x / cap) - slope_h * |p_q - p_k|      (cap > 0; x alone without a cap)
// and the softmax runs over z.  Kernels work in the log2 domain, so they hold
// z * log2(e): the cap is stored as c2 = cap * log2(e), the slopes are
// multiplied by log2(e) as they are read.
//
// tanh(y), y = x / cap:
//   |y| <= 0.6   y * (1 + u * P(u)), u = y^2, P of degree 4 fitted here to
//                (tanh(y) / y - 1) / u by iterated weighted least squares:
//                relative error 2.6e-9, 7.5e-8 as evaluated in fp32.  c2 is
//                multiplied into the coefficients, so z costs seven
//                multiply-adds and no MUFU instruction.
//   else         (1 - e) / (1 + e), e = 2^(-2 log2(e) |y|): 1 from |y| = 9 on;
//                ex2 is off by at most 2^-22 e, rcp by 2^-23 of its value, so
//                tanh is off by at most 2 * 2^-22 + 2^-23 + 2 * 2^-24 < 7.2e-7
//                for every y, also where a group of scores takes this form
//                because one of them left the first interval.
// A score is so accurate to 7.2e-7 of the cap.  Scores rarely leave the first
// interval with the caps that models use (30 to 50); the second form costs two
// MUFU instructions a score.
#pragma once

#include <cuda_runtime.h>
#include <math.h>

namespace kvc {

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kCapPolyMax = 0.6f;  // |x / cap| up to which the polynomial serves

// By value in kernel arguments.
struct ScoreMod {
  float c2;             // cap * log2(e); 0: no cap
  float y_scale;        // sm_scale / cap: q . k -> y
  float poly[6];        // c2 * (1, P's coefficients)
  const float* slopes;  // [hq] (natural-log units) or null: no bias
};

// sm_scale and cap as the caller gave them (cap 0: none).
inline ScoreMod make_score_mod(float sm_scale, float cap, const float* slopes) {
  constexpr double kP[5] = {-0.33333298563957214, 0.13331958651542664, -0.053786683827638626, 0.02080538310110569,
                            -0.005905867554247379};
  ScoreMod m{};
  m.slopes = slopes;
  if (cap > 0.0f) {
    const double c2 = (double)cap * 1.4426950408889634;
    m.c2 = (float)c2;
    m.y_scale = (float)((double)sm_scale / (double)cap);
    m.poly[0] = (float)c2;
    for (int i = 0; i < 5; ++i) m.poly[i + 1] = (float)(c2 * kP[i]);
  }
  return m;
}

#ifdef __CUDACC__
namespace dev {

__device__ __forceinline__ float cap_poly(const ScoreMod& m, float y) {
  const float u = y * y;
  float h = fmaf(m.poly[5], u, m.poly[4]);
  h = fmaf(h, u, m.poly[3]);
  h = fmaf(h, u, m.poly[2]);
  h = fmaf(h, u, m.poly[1]);
  h = fmaf(h, u, m.poly[0]);
  return y * h;
}

__device__ __forceinline__ float cap_far(const ScoreMod& m, float y) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-2.0f * kLog2E * fabsf(y)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return copysignf(m.c2 * ((1.0f - e) * r), y);
}

// z (log2 units) of y = x / cap; NaN stays NaN, infinities give +-c2.
__device__ __forceinline__ float cap_score(const ScoreMod& m, float y) {
  return fabsf(y) <= kCapPolyMax ? cap_poly(m, y) : cap_far(m, y);
}

// N scores in place: the polynomial when all are within its interval.
template <int N>
__device__ __forceinline__ void cap_scores(const ScoreMod& m, float (&y)[N]) {
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, fabsf(y[i]));
  if (top <= kCapPolyMax) {  // (a NaN alone stays NaN in the polynomial)
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = cap_poly(m, y[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = cap_far(m, y[i]);
  }
}

// A dot product q . k (already times sm_scale * log2(e) without a cap, times
// y_scale with one) of head slope `slope2` (log2 units) at `dist` positions.
__device__ __forceinline__ float transform_score(const ScoreMod& m, float x, float slope2, int dist) {
  if (m.c2 > 0.0f) x = cap_score(m, x);
  return fmaf(-slope2, (float)dist, x);
}

__device__ __forceinline__ float slope_log2(const ScoreMod& m, int head) {
  return m.slopes != nullptr ? m.slopes[head] * kLog2E : 0.0f;
}

}  // namespace dev
#endif

}  // namespace kvc
