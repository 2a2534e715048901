// Score transforms of the attention kernels: the cap by a tanh and the bias
// that depends on the distance between query and key.
//
// With x = sm_scale * q . k, the transformed score is
//   z = cap * tanh(x / cap) - slope_h * |p_q - p_k|      (cap > 0; x alone without a cap)
// and the softmax runs over z.  Kernels work in the log2 domain, so they hold
// z * log2(e): the cap is stored as c2 = cap * log2(e), the slopes are
// multiplied by log2(e) as they are read.
//
// tanh(y), y = x / cap, with P fitted here to (tanh(y) / y - 1) / u, u = y^2,
// by iterated weighted least squares:
//   |y| <= 0.6   y * (1 + u * P(u)), P of degree 3: relative error 1.6e-7 as
//                evaluated in fp32.  The cap is multiplied into the
//                coefficients: six multiply-adds a score and no MUFU.
//   |y| <= 0.4   (prompts, which form scores by the thousand per thread) the
//                same with P of degree 2, 1.8e-7;
//   |y| <= 1.5   (prompts) with P of degree 8, 2.0e-7.
//   else         (1 - e) / (1 + e), e = 2^(-2 log2(e) |y|): 1 from |y| = 9 on;
//                ex2 is off by at most 2^-22 e, rcp by 2^-23 of its value, so
//                tanh is off by at most 2 * 2^-22 + 2^-23 + 2 * 2^-24 < 7.2e-7
//                for every y, also where a group of scores takes this form
//                because one of them left the intervals above.  Two MUFU
//                instructions a score.
// A score is so accurate to 7.2e-7 of the cap.  With the caps that models use
// (30 to 50) scores rarely leave the first interval.
#pragma once

#include <cuda_runtime.h>
#include <math.h>

namespace kvc {

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kCapNear = 0.6f;  // |x / cap| up to which the polynomial of degree 3 serves
constexpr float kCapClose = 0.4f;  // the one of degree 2
constexpr float kCapMid = 1.5f;    // and the one of degree 8
constexpr double kCapP2[3] = {-0.3333190183144874, 0.13278022829794303, -0.047811859768676745};
constexpr double kCapP3[4] = {-0.3333262160369896, 0.13313520721608138, -0.052231106454585126, 0.01564048021294071};
constexpr double kCapP8[9] = {-0.3333324241639356, 0.13331582011696386, -0.053850984564149926,
                              0.021477584226268928, -0.008099126689853861, 0.002642995882885061,
                              -0.000656591311100134, 0.00010466406356551689, -7.770424672509535e-06};

// By value in kernel arguments.
struct ScoreMod {
  float c2;             // cap * log2(e); 0: no cap
  float y_scale;        // sm_scale / cap: q . k -> y
  float poly[5];        // c2 * (1, the coefficients of P of degree 3)
  const float* slopes;  // [hq] (natural-log units) or null: no bias
};

// sm_scale and cap as the caller gave them (cap 0: none).
inline ScoreMod make_score_mod(float sm_scale, float cap, const float* slopes) {
  ScoreMod m{};
  m.slopes = slopes;
  if (cap > 0.0f) {
    const double c2 = (double)cap * 1.4426950408889634;
    // (finite for every cap, with room for the kernels' powers of two beside it:
    // an infinite factor would make NaN of a product of 0)
    constexpr double kMost = 3.4028234663852886e38, kMostY = 1152921504606846976.0;  // 2^60
    m.c2 = (float)(c2 < kMost ? c2 : kMost);
    const double ys = (double)sm_scale / (double)cap;
    m.y_scale = (float)(ys < kMostY ? ys : kMostY);
    m.poly[0] = m.c2;
    for (int i = 0; i < 4; ++i) m.poly[i + 1] = (float)(c2 * kCapP3[i]);
  }
  return m;
}

#ifdef __CUDACC__
namespace dev {

__device__ __forceinline__ float cap_poly(const ScoreMod& m, float y) {
  const float u = y * y;
  float h = fmaf(m.poly[4], u, m.poly[3]);
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
  return fabsf(y) <= kCapNear ? cap_poly(m, y) : cap_far(m, y);
}

// N scores in place: the polynomial when all are within its interval.
template <int N>
__device__ __forceinline__ void cap_scores(const ScoreMod& m, float (&y)[N]) {
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, fabsf(y[i]));
  if (top <= kCapNear) {  // (a NaN alone stays NaN in the polynomial)
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
