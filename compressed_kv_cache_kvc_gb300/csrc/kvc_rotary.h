// Rotary positions: what the stand-alone rotation (kvc_rotary.cu) and the
// block-scaled cache's append (kvc_block_rotary.cu) share.  Not part of the ABI.
//
// Pair i of a row, (x, y), at the position p of the pair's axis:
//   t = p freq[i],  x' = x cos t - y sin t,  y' = y cos t + x sin t
// in fp32, rounded once to bf16.  Positions run to 2^31, where an fp32 angle
// has lost every digit and an fp64 product costs 16 cycles a warp, so the angle is
// kept as a fraction of a turn: freq[i] / 2 pi mod 1 as a 64-bit fixed-point
// number F (made on the host, off by at most 2^-65), p F mod 2^64 by one integer
// product that wraps as turns do, off by 2^-34 of a turn at most.  Its upper word
// (another 2^-32) splits into the nearest quarter turn and a rest of at most pi / 4,
// whose sine and cosine are polynomials fitted here by iterated weighted least
// squares: sin x = x + x u S(u) with relative error 3.6e-9, cos x = 1 - u / 2 +
// u^2 C(u) with 9.5e-11, u = x^2 (both S and C of degree 2).  x is held in two
// parts, so that cos and sin are off by little more than their own rounding: 2^-25
// and, of terms below 0.31, three roundings of 2^-24: 9e-8.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kvc_internal.h"

namespace kvc {

constexpr int kRotPairs = kHeadDim / 2;
constexpr int kRotAxes = 4;

// By value in kernel arguments.
struct RotaryTable {
  uint64_t turns[kRotPairs];  // freq / 2 pi mod 1, times 2^64
  uint8_t axis[kRotPairs];
  int32_t rot, adjacent, axes;
  int32_t first;       // position of a sequence's token 0 where pos is null
  const int32_t* pos;  // [axes][batch][n], or null
};

// bf16 rows of 128: element (b, h, i) at in + b sb + h sh + i st.
struct RowsIn {
  const uint16_t* in;
  int64_t sb, sh, st;
};

// q (and k): rows in, packed rows out.
struct RotaryArgs {
  RotaryTable table;
  RowsIn q, k;
  uint16_t *q_out, *k_out;  // [batch][heads][n][128]
  int32_t batch, n, hq, hk;  // hk 0: no k
};
cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t st);

// Warps that share a token's heads: enough of them for every SM to have 16.
inline int rotary_splits(long long rows, int heads) {
  const long long groups = (rows + 3) / 4, want = (152 * 16 + groups - 1) / groups;
  return (int)(want < 1 ? 1 : want < heads ? want : heads);
}

#ifdef __CUDACC__
namespace rotary {

// Eight lanes have a row: lane c two chunks of 8 values, pairs 8 c .. 8 c + 7 when
// c < rot / 16; the others have two chunks that pass.
__device__ __forceinline__ bool turns_here(const RotaryTable& t, int c) { return 16 * c < t.rot; }
__device__ __forceinline__ int chunk_a(const RotaryTable& t, int c) {
  if (t.adjacent) return 2 * c;
  return 16 * c < t.rot ? c : 2 * c;  // (the passing chunks rot / 8 .. 15, two by two)
}
__device__ __forceinline__ int chunk_b(const RotaryTable& t, int c) {
  if (t.adjacent) return 2 * c + 1;
  return 16 * c < t.rot ? c + t.rot / 16 : 2 * c + 1;
}

// cos and sin of 2 pi w / 2^32
__device__ __forceinline__ void cos_sin(uint32_t w, float& c, float& s) {
  // 2 pi / 2^32 = kUnit + kUnitLo
  constexpr float kUnit = 1.462918119976564e-9f, kUnitLo = (float)(1.4629180792671596e-9 - 1.462918119976564e-9);
  const uint32_t q = w + 0x20000000u;  // its top bits: the nearest quarter turn
  // the rest in units, in two parts that fp32 holds: x + xl is right to 2^-30
  const int32_t r = (int32_t)(w - (q & 0xC0000000u));
  const float rh = (float)(r & ~0xFF), rl = (float)(r & 0xFF);
  const float x0 = rh * kUnit;
  const float e = fmaf(rh, kUnit, -x0) + fmaf(rh, kUnitLo, rl * kUnit);
  const float x = x0 + e, xl = e - (x - x0);
  const float u = x * x;
  float ps = fmaf(-1.9517296e-4f, u, 8.3321781e-3f);
  ps = fmaf(ps, u, -1.6666655e-1f);
  const float sx = x + fmaf(x * u, ps, xl);
  float pc = fmaf(2.4438446e-5f, u, -1.3887367e-3f);
  pc = fmaf(pc, u, 4.1666647e-2f);
  const float cx = 1.0f + (fmaf(u * u, pc, -0.5f * u) - x * xl);
  const bool odd = (q >> 30) & 1u;
  c = odd ? sx : cx;
  s = odd ? cx : sx;
  // quarter 1: (-sin, cos), 2: (-cos, -sin), 3: (sin, -cos)
  if (((q >> 30) + 1u) & 2u) c = -c;
  if (q & 0x80000000u) s = -s;
}

// The positions of a row on every axis.
struct RowPos {
  int p[kRotAxes];
};
// index: (sequence of the call) * n + new token; token: its index in the sequence
__device__ __forceinline__ RowPos row_pos(const RotaryTable& t, size_t index, size_t rows, int token) {
  RowPos r;
  if (t.pos == nullptr) {
    r.p[0] = r.p[1] = r.p[2] = r.p[3] = t.first + token;
  } else {
#pragma unroll
    for (int a = 0; a < kRotAxes; ++a) r.p[a] = t.pos[index + (a < t.axes ? a : 0) * rows];
  }
  return r;
}

// cos and sin of a lane's eight pairs
__device__ __forceinline__ void angles(const uint64_t* turns, const uint8_t* axis, const RowPos& r, int c,
                                       float (&cs)[8], float (&sn)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int a = axis[8 * c + j];
    const int p = a == 0 ? r.p[0] : a == 1 ? r.p[1] : a == 2 ? r.p[2] : r.p[3];
    cos_sin((uint32_t)(((uint64_t)(int64_t)p * turns[8 * c + j]) >> 32), cs[j], sn[j]);
  }
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t round2(float lo, float hi) {
  uint32_t w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}
__device__ __forceinline__ void turn(float& x, float& y, float c, float s) {
  const float a = fmaf(x, c, -(y * s));
  y = fmaf(y, c, x * s);
  x = a;
}

// A lane's two chunks turned.
__device__ __forceinline__ void turn16(bool adjacent, uint4& a, uint4& b, const float (&cs)[8], const float (&sn)[8]) {
  uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
  if (adjacent) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x = lo_f(wa[j]), y = hi_f(wa[j]);
      turn(x, y, cs[j], sn[j]);
      wa[j] = round2(x, y);
      x = lo_f(wb[j]), y = hi_f(wb[j]);
      turn(x, y, cs[4 + j], sn[4 + j]);
      wb[j] = round2(x, y);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x0 = lo_f(wa[j]), y0 = lo_f(wb[j]), x1 = hi_f(wa[j]), y1 = hi_f(wb[j]);
      turn(x0, y0, cs[2 * j], sn[2 * j]);
      turn(x1, y1, cs[2 * j + 1], sn[2 * j + 1]);
      wa[j] = round2(x0, x1);
      wb[j] = round2(y0, y1);
    }
  }
  a = make_uint4(wa[0], wa[1], wa[2], wa[3]);
  b = make_uint4(wb[0], wb[1], wb[2], wb[3]);
}

// One warp: four tokens (8 lanes a row) and their share of the heads, kAtOnce rows
// of each lane in flight.  token0(b): index of sequence b's first row.
template <int kAtOnce, class Token0>
__device__ __forceinline__ void rotate_unit(const RotaryArgs& a, const uint64_t* turns, const uint8_t* axis,
                                            long long unit, int splits, Token0 token0) {
  const int lane = threadIdx.x & 31, c = lane & 7;
  const long long rows = (long long)a.batch * a.n;
  const long long row = unit / splits * 4 + (lane >> 3);
  const int split = (int)(unit % splits), heads = a.hq + a.hk;
  const int h0 = (int)((long long)heads * split / splits), h1 = (int)((long long)heads * (split + 1) / splits);
  if (row >= rows) return;
  const int b = (int)(row / a.n), i = (int)(row % a.n);
  const bool turned = turns_here(a.table, c), adjacent = a.table.adjacent != 0;
  const int ca = 8 * chunk_a(a.table, c), cb = 8 * chunk_b(a.table, c);
  float cs[8], sn[8];
  if (turned) angles(turns, axis, row_pos(a.table, row, rows, token0(b) + i), c, cs, sn);
#pragma unroll 1
  for (int h = h0; h < h1; h += kAtOnce) {
    uint4 x[kAtOnce], y[kAtOnce];
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e)
      if (h + e < h1) {
        const bool key = h + e >= a.hq;
        const RowsIn& r = key ? a.k : a.q;
        const uint16_t* in = r.in + b * r.sb + (h + e - (key ? a.hq : 0)) * r.sh + i * r.st;
        x[e] = *reinterpret_cast<const uint4*>(in + ca);
        y[e] = *reinterpret_cast<const uint4*>(in + cb);
      }
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e)
      if (h + e < h1) {
        const bool key = h + e >= a.hq;
        if (turned) turn16(adjacent, x[e], y[e], cs, sn);
        uint16_t* out = key ? a.k_out + (((size_t)b * a.hk + (h + e - a.hq)) * a.n + i) * kHeadDim
                            : a.q_out + (((size_t)b * a.hq + (h + e)) * a.n + i) * kHeadDim;
        *reinterpret_cast<uint4*>(out + ca) = x[e];
        *reinterpret_cast<uint4*>(out + cb) = y[e];
      }
  }
}

}  // namespace rotary
#endif

}  // namespace kvc
