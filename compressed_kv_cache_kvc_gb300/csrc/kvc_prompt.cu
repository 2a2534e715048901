// Attention of a prompt over itself with capped scores, a distance bias and
// per-query runs of keys, on the fifth-generation tensor cores.
//
// Query i of a sequence sees the keys [begin_i, end_i) (causal when no runs
// are given); with s = sm_scale * q_i . k_j, z = cap * tanh(s / cap) - slope_h
// |i - j| (kvc_score.h), the output is softmax(z) . v over the keys it sees (0
// when it sees none) and, on request, every key's column sum of the
// probabilities over the queries and the query heads of its KV head.
//
// Three kernels:
//   prompt_prep_kernel   V from bf16 to fp16 in the workspace, times a power of
//                        two where a (sequence, KV head) holds nothing from 2^-6
//                        on, the keys whose V row is not finite as bit masks, the
//                        runs' bounds per 128-query tile;
//   prompt_fwd_kernel    outputs and (for the sums) row statistics;
//   prompt_sums_kernel   column sums from the row statistics.
//
// prompt_fwd_kernel.  4 * 128 flops per visible pair.  Bound by issue and latency,
// not by one pipe (32 capped heads of 8,192 causal tokens in 506 us, 1.09 PFLOP/s:
// issue 52 %, tensor pipe 47 %, FMA pipe 39 %), and for short runs of keys by the
// softmax's own chain, about 9 us a block whatever it holds.  One 576-thread CTA per
// (256 queries, query head, sequence), the longest blocks of all heads first (head
// by head 598 us for that prompt, 271 against 228 us for two-way prefixes with
// sums).  Launched while the prep
// kernel runs: only V and the masks of its rows are waited for.  Q is loaded
// while the runs are read; the output goes through Q's shared memory and
// leaves by TMA (stores of a row a thread and a later Q: 185 against 172 us for
// packed documents):
//   * warps 0-7 and 8-15 own one 128-query tile each ("A", "B"), two threads a
//     query row: of each eight the first four warps take the even key tiles,
//     the others the odd ones, so that four warps per scheduler hide each
//     other's latencies (eight warps, a thread a row, took 729 us where this then
//     took 597, 32 capped heads of 8,192 causal tokens);
//   * warp 16 issues the products, warp 17 the TMA loads: K and V tiles of 64
//     keys into four slots each.  K is read K-major and V in its own layout
//     (MN-major), both with the 128-byte swizzle, so nothing is transposed.
// TMEM columns: S_x of key tile t at 128 x + 64 (t % 2), O_x at 256 + 128 x; the
// first 32 columns of an S become its P in fp16.  In round r the MMA warp issues
// P V_A(r - 2), S_A(r), P V_B(r - 2), S_B(r): the pipe runs them in order, so
// S(r) may overwrite P(r - 2) without a wait, and with two S per query tile its
// softmax has the next scores ready.  The other form, one S of 128 keys per
// query tile, halves the products' issue (N = 64 products cost 48 cycles, not
// 32) but every tile waits for its own products and runs are rounded to 128
// keys: 4 % slower over prompts of 1 to 8000 tokens and all masks (packed biased
// documents 213 against 199 us, capped and biased prefixes 167 against 157 us),
// faster for long causal prompts without a cap (32 heads of 8192 tokens: 454
// against 561 us plain, 582 against 594 us capped; all before blocks went longest
// first).
// Key tiles go from the last to the first: with a distance bias the nearest
// keys, which set the maximum, come first.  The running maximum is lazy (O is
// rescaled when a row's maximum grows by more than 8 in log2 units, after a
// wait for the P V before), P is rounded to fp16 (11 significant bits; p <=
// 2^8), the sums add the unrounded p in fp32.  The two threads of a row pass
// the running maximum on from tile to tile through shared memory (an mbarrier
// per warp); each sums its own tiles' p.  A tile's scores are read from TMEM
// twice, for the maximum and for P: 96 registers a thread is what 18 warps
// leave.
// Key tiles no query of a 128-query tile sees are skipped; tiles every row of
// a warp sees whole take no mask.  Masked scores are replaced before the
// maximum, and P is exactly 0 there; V rows that are not finite enter the
// product as 0 and give NaN only to the rows that see them.
// V in fp16 is exact from 2^-14 (bf16 has 8 bits) to 2^16 and off by at most 2^-25
// below.  Where the largest |v| of a (sequence, KV head) lies below 2^-6 all of its
// V enter times the power of two that brings it to [2^14, 2^15), and O leaves
// divided by it: a value is off by at most 2^-19 of that largest one.
//
// Synchronisation: mbarriers, every wait bounded as in the prefill kernels (a
// wait that runs out sets KVC_DEV_WAIT_TIMEOUT, all roles leave, the TMEM is
// freed).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kvc_device.h"
#include "kvc_internal.h"
#include "kvc_tc.h"

namespace kvc {
namespace {

using namespace dev;
using namespace tc;

constexpr int kTile = 128;                        // queries per tile; keys per tile of the column sums
constexpr int kKeys = 64;                         // keys per tile of the forward
constexpr int kFwdThreads = 576;
constexpr int kFwdBlock = 2 * kTile;
constexpr float kLazyMax = 8.0f;
constexpr int kTileB = kTile * kHeadDim * 2;      // 32 KB: a 128-row tile, two boxes of 64 dims
constexpr int kBoxB = kTileB / 2;
constexpr int kKeyB = kKeys * kHeadDim * 2;       // 16 KB: a K or V tile, two boxes of 64 dims
constexpr int kKeyBox = kKeyB / 2;
constexpr int kSlots = 4;
constexpr int kFOffQ = 0;                         // 2 tiles
constexpr int kFOffK = kFOffQ + 2 * kTileB;
constexpr int kFOffV = kFOffK + kSlots * kKeyB;
constexpr int kFOffBar = kFOffV + kSlots * kKeyB;
// mbarriers: Q landed (per query tile); a round's K and V landed, its slots
// free (per round % 4); S complete, P written, P V complete (per query tile and
// tile parity); all products complete; the running maximum passed on (per warp)
constexpr int kFBarQ = 0, kFBarKv = 2, kFBarFree = 6, kFBarS = 10, kFBarP = 14, kFBarO = 18, kFBarDone = 22,
              kFBarM = 23, kFNumBars = 39;
constexpr int kFOffMisc = kFOffBar + 8 * kFNumBars;  // TMEM base, abort flag, [8][2] run bounds per 32 rows
constexpr int kFOffMax = kFOffMisc + 8 + 64;         // [2 query tiles][2 parities][128] row maxima, then sums
constexpr int kFwdSmem = kFOffMax + 2 * 2 * kTile * 4;
constexpr int kNbTile = 1;                           // named barriers of a query tile's warps: 1, 2
constexpr uint32_t kFwdCols = 512;

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

__device__ __forceinline__ void set_abort(int* status, volatile int* abort) {
  if (!*abort) {
    *abort = 1;
    atomicOr(status, kDevWaitTimeout);
  }
}

// The keys [lo, hi) query `i` of sequence `bl` sees; an empty run is (0, 0).
__device__ __forceinline__ int2 run_of(const PromptArgs& a, int bl, int i) {
  int lo = 0, hi = i + 1;
  if (a.key_begin != nullptr) lo = max(a.key_begin[(size_t)bl * a.n + i], 0);
  if (a.key_end != nullptr) hi = min(a.key_end[(size_t)bl * a.n + i], a.n);
  return lo < hi ? make_int2(lo, hi) : make_int2(0, 0);
}

// ---------------------------------------------------------------------------
constexpr int kPrepThreads = 256;
constexpr float kSmallV = 0x1p-6f;
// what the forward has to know of a tile of V: whether a row is not finite, and (from
// bit kInfoShift on) the exponent of its power of two
constexpr uint32_t kInfoBad = 1;
constexpr int kInfoShift = 1;

__global__ void __launch_bounds__(kPrepThreads) prompt_prep_kernel(PromptArgs a, const uint16_t* __restrict__ v) {
  __shared__ uint32_t sh_bad[4], sh_top;
  __shared__ int sh_run[4];
  launch_dependents();
  const int tiles = (a.n + kTile - 1) / kTile;
  const int tile = blockIdx.x % tiles, plane = blockIdx.x / tiles, tid = threadIdx.x, lane = tid & 31;
  const int k0 = tile * kTile, rows = min(kTile, a.n - k0);
  if (tid < 4) sh_bad[tid] = 0;
  if (tid == 0) {
    sh_run[0] = INT_MAX;
    sh_run[1] = 0;
    sh_run[2] = 0;
    sh_run[3] = INT_MAX;
    sh_top = 0;
  }
  __syncthreads();
  // 16 bytes a lane, 16 lanes a row, 16 rows a pass
  const int r0 = tid >> 4, ch = tid & 15;
  const uint4* src = reinterpret_cast<const uint4*>(v + ((size_t)plane * a.n + k0) * kHeadDim) + ch;
  uint4* dst = reinterpret_cast<uint4*>(a.v16 + ((size_t)plane * a.n + k0) * kHeadDim) + ch;
  uint4 w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (r0 + 16 * i < rows) w[i] = src[(size_t)(r0 + 16 * i) * 16];
  bool range = false;
  float most = 0.0f;  // the largest finite magnitude
  auto convert = [&](float scale) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + 16 * i;
      bool bad = false;
      if (r < rows) {
        uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float lo = bf16f(x[e] & 0xFFFFu), hi = bf16f(x[e] >> 16);
          range |= !(fabsf(lo) < 65536.0f) || !(fabsf(hi) < 65536.0f);
          if ((x[e] & 0x7F80u) == 0x7F80u) bad = true, lo = 0.0f;
          if ((x[e] & 0x7F800000u) == 0x7F800000u) bad = true, hi = 0.0f;
          most = max3_abs(lo, hi, most);
          asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(x[e]) : "f"(hi * scale), "f"(lo * scale));
        }
        dst[(size_t)r * 16] = make_uint4(x[0], x[1], x[2], x[3]);
      }
      const uint32_t vote = __ballot_sync(0xffffffffu, bad);
      if (vote != 0 && (lane & 15) == 0 && ((vote >> lane) & 0xFFFFu) != 0) atomicOr(&sh_bad[r >> 5], 1u << (r & 31));
    }
  };
  convert(1.0f);
  uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
  if (lane == 0) atomicMax(&sh_top, top);
  if (range) atomicOr(a.status, kDevPrefillRange);
  // bounds of the runs of query tile `tile`, once per sequence
  if (a.runs != nullptr && plane % a.hkv == 0 && tid < kTile && tid < rows) {
    const int2 run = run_of(a, plane / a.hkv, k0 + tid);
    const bool any = run.x < run.y;
    if (any) {
      atomicMin(&sh_run[0], run.x);
      atomicMax(&sh_run[1], run.y);
    }
    atomicMax(&sh_run[2], any ? run.x : INT_MAX);
    atomicMin(&sh_run[3], any ? run.y : 0);
  }
  __syncthreads();
  int shift = 0;
  if (sh_top != 0 && sh_top < __float_as_uint(kSmallV)) {
    // nothing from 2^-6 on in this tile (rare): is there anywhere in the plane?  The
    // CTA looks from the next tile on until it finds some; where there is none every
    // CTA of the plane with other values than zeros comes to the same power
    const uint4* all = reinterpret_cast<const uint4*>(v + (size_t)plane * a.n * kHeadDim);
    for (int t = 1; t < tiles && sh_top < __float_as_uint(kSmallV); ++t) {
      const int other = (tile + t) % tiles;
      const size_t end = min((size_t)(other + 1) * kTile, (size_t)a.n) * 16;
      for (size_t i = (size_t)other * kTile * 16 + tid; i < end; i += kPrepThreads) {
        const uint4 y = all[i];
        const uint32_t x[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t lo = (x[e] << 16) & 0x7FFF0000u, hi = x[e] & 0x7FFF0000u;
          top = max(top, max(lo < 0x7F800000u ? lo : 0u, hi < 0x7F800000u ? hi : 0u));
        }
      }
      top = __reduce_max_sync(0xffffffffu, top);
      __syncthreads();  // (every thread has read sh_top)
      if (lane == 0) atomicMax(&sh_top, top);
      __syncthreads();
    }
    if (sh_top < __float_as_uint(kSmallV)) {
      shift = min(14 - ((int)(sh_top >> 23) - 127), 126);
      convert(pow2(shift));
    }
  }
  if (tid < 4) a.bad[((size_t)plane * tiles + tile) * 4 + tid] = sh_bad[tid];
  if (tid == 0)
    a.info[(size_t)plane * tiles + tile] =
        (sh_bad[0] | sh_bad[1] | sh_bad[2] | sh_bad[3] ? kInfoBad : 0) | (uint32_t)shift << kInfoShift;
  if (tid == 0 && a.sum_parts > 1) a.sum_tickets[(size_t)plane * tiles + tile] = 0;
  if (a.runs != nullptr && plane % a.hkv == 0 && tid == 0)
    a.runs[(size_t)(plane / a.hkv) * tiles + tile] = make_int4(sh_run[0], sh_run[1], sh_run[2], sh_run[3]);
}

// ---------------------------------------------------------------------------
__device__ __forceinline__ float chunk_most(const float (&z)[32], float most) {
  float t0 = most, t1 = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    t0 = max3_abs(t0, z[i], z[i + 1]);
    t1 = max3_abs(t1, z[i + 2], z[i + 3]);
  }
  return fmaxf(t0, t1);
}

// Capped scores (log2 units) plus nm(i) of 32 raw products of a row, none larger
// in magnitude than `most`; nm(i) is the packed pair for products i and i + 1.
template <typename NM>
__device__ __forceinline__ void chunk_cap_plus(const PromptArgs& a, float (&z)[32], float most, NM nm) {
  if (!(most > a.close_max)) {  // (a NaN stays NaN in the polynomials)
    f32x2 c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = pack2(a.close[i], a.close[i]);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const f32x2 x = pack2(z[i], z[i + 1]);
      const f32x2 u = mul2(x, x);
      f32x2 h = fma2(c[3], u, c[2]);
      h = fma2(h, u, c[1]);
      h = fma2(h, u, c[0]);
      unpack2(fma2(x, h, nm(i)), z[i], z[i + 1]);
    }
  } else if (most <= a.mid_max) {
    const f32x2 ys = pack2(a.mod.y_scale, a.mod.y_scale);
    f32x2 c[10];
#pragma unroll
    for (int i = 0; i < 10; ++i) c[i] = pack2(a.mid[i], a.mid[i]);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const f32x2 y = mul2(pack2(z[i], z[i + 1]), ys);
      const f32x2 u = mul2(y, y);
      f32x2 h = c[9];
#pragma unroll
      for (int e = 8; e >= 0; --e) h = fma2(h, u, c[e]);
      unpack2(fma2(y, h, nm(i)), z[i], z[i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float x = cap_far(a.mod, z[i] * a.mod.y_scale), y = cap_far(a.mod, z[i + 1] * a.mod.y_scale);
      unpack2(add2(pack2(x, y), nm(i)), z[i], z[i + 1]);
    }
  }
}

__device__ __forceinline__ void chunk_cap(const PromptArgs& a, float (&z)[32], float most, float m) {
  const f32x2 nm = pack2(-m, -m);
  chunk_cap_plus(a, z, most, [&](int) { return nm; });
}

// The distance bias of 32 scores: z scale - slope2 |d|, d = d0, d0 + 1, ..., all
// of the sign of `toward` (slope2 or -slope2 with it) unless `both`.
__device__ __forceinline__ void chunk_bias(float (&z)[32], float scale, float slope2, float toward, float d0,
                                           bool both) {
  const f32x2 sl = pack2(toward, toward), sc = pack2(scale, scale), two = pack2(2.0f, 2.0f);
  if (!both) {
    f32x2 d = pack2(d0, d0 + 1.0f);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      unpack2(fma2(d, sl, mul2(pack2(z[i], z[i + 1]), sc)), z[i], z[i + 1]);
      d = add2(d, two);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) z[i] = fmaf(-slope2, fabsf(d0 + (float)i), z[i] * scale);
  }
}

// -inf outside [b, e) (key indices relative to the chunk).
__device__ __forceinline__ void chunk_mask(float (&z)[32], int b, int e) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (!(i >= b && i < e)) z[i] = -INFINITY;
}

__device__ __forceinline__ float chunk_max(const float (&z)[32], float m) {
  float t0 = m, t1 = -INFINITY;
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    t0 = max3(t0, z[i], z[i + 1]);
    t1 = max3(t1, z[i + 2], z[i + 3]);
  }
  return fmaxf(t0, t1);
}

// 32 scores less m -> probabilities in fp16 pairs; their unrounded sum is added
// to ls.
__device__ __forceinline__ void chunk_probs(const float (&z)[32], uint32_t (&pw)[16], f32x2 (&ls)[2]) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float x = fast_exp2(z[2 * e]), y = fast_exp2(z[2 * e + 1]);
    ls[e & 1] = add2(ls[e & 1], pack2(x, y));
    const __half2 hh = __floats2half2_rn(x, y);
    pw[e] = *reinterpret_cast<const uint32_t*>(&hh);
  }
}

// z scale - m
__device__ __forceinline__ void chunk_shift(float (&z)[32], float scale, float m) {
  const f32x2 nm = pack2(-m, -m), sc = pack2(scale, scale);
#pragma unroll
  for (int i = 0; i < 32; i += 2) unpack2(fma2(pack2(z[i], z[i + 1]), sc, nm), z[i], z[i + 1]);
}

template <bool CAP, bool BIAS>
__global__ void __launch_bounds__(kFwdThreads, 1)
    prompt_fwd_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CUtensorMap tm_o) {
  extern __shared__ __align__(1024) uint8_t fsm[];
  const uint32_t base = saddr(fsm);
  uint32_t* tbase = reinterpret_cast<uint32_t*>(fsm + kFOffMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(fsm + kFOffMisc + 4);
  int* sh_run = reinterpret_cast<int*>(fsm + kFOffMisc + 8);
  auto bar = [&](int i) { return base + kFOffBar + 8 * i; };

  const int n = a.n;
  // the longest blocks of all heads first (head by head, the last heads' blocks
  // left the SMs idle at the end)
  const int planes = a.hq * a.batch, plane_q = blockIdx.x % planes;
  const int qb = (n + kFwdBlock - 1) / kFwdBlock - 1 - blockIdx.x / planes;
  const int bl = plane_q / a.hq, hqi = plane_q % a.hq;
  const int plane_kv = bl * a.hkv + hqi / a.group;
  // (what steers a whole warp goes through a shuffle: the compiler then keeps it,
  // and the operands of the products that hang on it, in uniform registers)
  auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const int qblk = qb * kFwdBlock;
  // (softmax threads) query tile, parity of the key tiles, query row
  const int x = warp >> 3, odd = (warp >> 2) & 1, row = tid & (kTile - 1);
  const int qi = qblk + kTile * x + row;

  if (warp == 16) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tbase)), "r"(kFwdCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 17 * 32) {
    for (int i = 0; i < kFNumBars; ++i)
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar(i)),
                   "r"(i >= kFBarP && i < kFBarP + 4 ? 4u : 1u));
    *abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async();
    // Q comes while the runs are read
    tma_prefetch_map(&tm_k);
    tma_prefetch_map(&tm_v);
#pragma unroll
    for (int y = 1; y >= 0; --y) {
      const uint32_t dst = base + kFOffQ + y * kTileB;
      bar_expect_tx(bar(kFBarQ + y), kTileB);
      tma_load_3d(dst, &tm_q, 0, qblk + y * kTile, plane_q, bar(kFBarQ + y));
      tma_load_3d(dst + kBoxB, &tm_q, 64, qblk + y * kTile, plane_q, bar(kFBarQ + y));
    }
    tma_prefetch_map(&tm_o);
  }
  // the rows' runs; per warp the keys some row sees and those every row sees
  int2 run = make_int2(0, 0);
  int all_lo = 0, all_hi = INT_MAX;
  if (warp < 16) {
    int lo = INT_MAX, hi = 0;
    if (qi < n) {
      run = run_of(a, bl, qi);
      const bool any = run.x < run.y;
      lo = any ? run.x : INT_MAX;
      hi = run.y;
      all_lo = lo;
      all_hi = hi;
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    all_lo = __reduce_max_sync(0xffffffffu, all_lo);
    all_hi = __reduce_min_sync(0xffffffffu, all_hi);
    if (lane == 0 && !odd) {
      sh_run[2 * (4 * x + (warp & 3))] = lo;
      sh_run[2 * (4 * x + (warp & 3)) + 1] = hi;
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = (uint32_t)uniform((int)*tbase);
  // key tiles [x_lo, x_hi) of query tile x; [t_lo, t_hi) of both
  int x_lo[2], x_hi[2];
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    int lo = INT_MAX, hi = 0;
#pragma unroll
    for (int w = 4 * y; w < 4 * y + 4; ++w) {
      lo = min(lo, sh_run[2 * w]);
      hi = max(hi, sh_run[2 * w + 1]);
    }
    x_lo[y] = uniform(lo < hi ? lo / kKeys : 0);
    x_hi[y] = uniform(lo < hi ? (hi + kKeys - 1) / kKeys : 0);
  }
  const bool on0 = x_lo[0] < x_hi[0], on1 = x_lo[1] < x_hi[1];
  const int t_lo = on0 && on1 ? min(x_lo[0], x_lo[1]) : on0 ? x_lo[0] : x_lo[1];
  const int t_hi = max(x_hi[0], x_hi[1]);
  const int n_t = t_hi - t_lo;  // key tiles; the one of round r is t_hi - 1 - r

  if (warp == 17) {
    // ------------------------------------------------------------- TMA loads
    // Round r brings K of its tile and V of the tile two rounds before, on one
    // barrier; both are consumed by the products of round r.
    if (lane == 0) {
      int rounds = 0;
      for (int r = 0; n_t > 0 && r < n_t + 2; ++r) {
        const int j = t_hi - 1 - r;
        const uint32_t b = bar(kFBarKv + (r & 3));
        if (r >= kSlots && !bar_wait(bar(kFBarFree + (r & 3)), (uint32_t)((r >> 2) & 1) ^ 1u, abort)) {
          set_abort(a.status, abort);
          break;
        }
        bar_expect_tx(b, (r < n_t ? kKeyB : 0) + (r >= 2 ? kKeyB : 0));
        if (r < n_t) {
          const uint32_t dst = base + kFOffK + (r & 3) * kKeyB;
          tma_load_3d(dst, &tm_k, 0, j * kKeys, plane_kv, b);
          tma_load_3d(dst + kKeyBox, &tm_k, 64, j * kKeys, plane_kv, b);
        }
        if (r == 2) wait_for_previous();  // V in fp16
        if (r >= 2) {
          const uint32_t dst = base + kFOffV + ((r - 2) & 3) * kKeyB;
          tma_load_3d(dst, &tm_v, 0, (j + 2) * kKeys, plane_kv, b);
          tma_load_3d(dst + kKeyBox, &tm_v, 64, (j + 2) * kKeys, plane_kv, b);
        }
        rounds = r + 1;
      }
      // the last copies land before the CTA goes away (they may not have been
      // waited for when another role gave up)
      for (int y = 0; y < 2; ++y) bar_wait(bar(kFBarQ + y), 0, nullptr);
      for (int e = max(0, rounds - kSlots); e < rounds; ++e)
        bar_wait(bar(kFBarKv + (e & 3)), (uint32_t)((e >> 2) & 1), nullptr);
    }
    __syncwarp();
  } else if (warp == 16) {
    // -------------------------------------------------------------- products
    const bool el = elect_one();
    const uint32_t id_s = instr_desc(kTile, kKeys, true);
    const uint32_t id_o = instr_desc(kTile, kHeadDim, false) | kInstrTransB;
    bool ok = true;
    auto wait = [&](int b, uint32_t par) {
      if (!__all_sync(0xffffffffu, bar_try(bar(b), par)) && !__all_sync(0xffffffffu, bar_wait(bar(b), par, abort))) {
        ok = false;
        set_abort(a.status, abort);
      }
    };
    const uint64_t dq = op_desc_sw128(base + kFOffQ), dk = op_desc_sw128(base + kFOffK),
                   dv = op_desc_mn_sw128(base + kFOffV, kKeyBox);
    for (int r = 0; n_t > 0 && r < n_t + 2; ++r) {
      wait(kFBarKv + (r & 3), (uint32_t)((r >> 2) & 1));
      if (!ok) break;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint32_t t_o = tmem + 256 + kTile * y;
        const int i = r - (t_hi - x_hi[y]), n_y = x_hi[y] - x_lo[y];  // this round's tile of y, y's tiles
        const uint32_t t_s = tmem + kTile * y + kKeys * (i & 1);
        if (i >= 2 && i - 2 < n_y) {
          wait(kFBarP + 2 * y + (i & 1), (uint32_t)(((i - 2) >> 1) & 1));
          if (!ok) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          if (el) {
            const uint64_t d = dv + (uint64_t)((((r - 2) & 3) * kKeyB) >> 4);
#pragma unroll
            for (int ks = 0; ks < kKeys / 16; ++ks)
              mma_f16_ts(t_o, t_s + 8 * ks, d + (uint64_t)((ks * 2048) >> 4), id_o, i > 2 || ks > 0);
            mma_commit(bar(kFBarO + 2 * y + (i & 1)));
          }
        }
        // (a query tile's first two S come together: else the second waits for the
        // other tile's P V of this round; capped 8,192-token prompt 521 -> 504 us,
        // packed documents 172 -> 168)
        if (i >= 0 && i < n_y && i != 1) {
          if (i == 0) wait(kFBarQ + y, 0);
          if (!ok) break;
          const int count = i == 0 && n_y > 1 ? 2 : 1;
#pragma unroll 1
          for (int e = 0; e < count; ++e) {
            const int q = (r + e) & 3;
            if (e > 0) wait(kFBarKv + q, (uint32_t)(((r + e) >> 2) & 1));
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            if (el) {
              const uint64_t d = dk + (uint64_t)((q * kKeyB) >> 4);
#pragma unroll
              for (int ks = 0; ks < kHeadDim / 16; ++ks)
                mma_f16(t_s + kKeys * e, dq + (uint64_t)((y * kTileB + (ks >> 2) * kBoxB + (ks & 3) * 32) >> 4),
                        d + (uint64_t)(((ks >> 2) * kKeyBox + (ks & 3) * 32) >> 4), id_s, ks > 0);
              mma_commit(bar(kFBarS + 2 * y + ((i + e) & 1)));
            }
          }
        }
      }
      if (!ok) break;
      if (el) mma_commit(bar(kFBarFree + (r & 3)));
      __syncwarp();
    }
    if (n_t > 0) {
      // every product complete before the tensor memory goes back
      if (el) mma_commit(bar(kFBarDone));
      bar_wait(bar(kFBarDone), 0, nullptr);
    }
    __syncwarp();
  } else {
    // ----------------------------------------------------------- query rows
    const int lo = x == 0 ? x_lo[0] : x_lo[1], hi = x == 0 ? x_hi[0] : x_hi[1];
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_s = trow + kTile * x + kKeys * odd, t_o = trow + 256 + kTile * x;
    const float slope2 = BIAS ? slope_log2(a.mod, hqi) : 0.0f;
    const size_t info_row = (size_t)plane_kv * ((n + kTile - 1) / kTile);
    float* sh_m = reinterpret_cast<float*>(fsm + kFOffMax) + x * 2 * kTile + row;
    const int bar_m = kFBarM + 8 * x + (warp & 3);  // + 4 * parity
    const int n_x = hi - lo;
    bool ok = true, poison = false;
    // what is rare about the tiles of V ahead (under the first loads: a word read
    // in the loop would put a global load's latency into every tile); tiles of a
    // plane have one power of two, or none where they hold nothing but zeros
    wait_for_previous();
    uint32_t rare = 0;
    for (int j = lo / 2 + lane; j < (hi + 1) / 2; j += 32) rare |= a.info[info_row + j];
    rare = __reduce_or_sync(0xffffffffu, rare);
    auto wait = [&](int b, uint32_t par) {
      if (!__all_sync(0xffffffffu, bar_try(bar(b), par)) && !__all_sync(0xffffffffu, bar_wait(bar(b), par, abort))) {
        ok = false;
        set_abort(a.status, abort);
      }
    };
    float m = kNegBig, l = 0.0f;
#pragma unroll 1
    for (int i = odd; i < n_x; i += 2) {
      const int k0 = (hi - 1 - i) * kKeys;
      const uint32_t par = (uint32_t)((i >> 1) & 1);
      wait(kFBarS + 2 * x + odd, par);
      if (!ok) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      float z[32];
      const bool masked = k0 < all_lo || k0 + kKeys > all_hi;  // (the same for the warp)
      const bool beyond = k0 + kKeys - 1 > qi - lane;
      const float dist0 = (float)(k0 - qi);
      // the maximum: with a bias, over the scores, which then take the products'
      // place; else over the products (a cap and the scale keep their order).
      // With a cap alone the largest magnitude, which the choice of the
      // polynomial needs anyway, bounds it: where that bound would not move the
      // running maximum, the maximum itself is not looked for.
      float mx = -INFINITY, most = 0.0f;
      if (CAP && !BIAS) {
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          ld32(t_s + 32 * c, z);
          most = chunk_most(z, most);
        }
        mx = cap_score(a.mod, most * a.mod.y_scale);
      } else {
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          ld32(t_s + 32 * c, z);
          if (CAP && BIAS && !beyond) {  // (the cap ends in the bias's addition)
            const f32x2 sl = pack2(slope2, slope2), two = pack2(2.0f, 2.0f);
            f32x2 d = pack2(dist0 + 32.0f * c, dist0 + 32.0f * c + 1.0f);
            chunk_cap_plus(a, z, chunk_most(z, 0.0f), [&](int) {
              const f32x2 add = mul2(d, sl);
              d = add2(d, two);
              return add;
            });
          } else {
            if (CAP) chunk_cap(a, z, chunk_most(z, 0.0f), 0.0f);
            if (BIAS) chunk_bias(z, CAP ? 1.0f : a.qk_scale_log2, slope2, slope2, dist0 + 32.0f * c, beyond);
          }
          if (masked) chunk_mask(z, run.x - k0 - 32 * c, run.y - k0 - 32 * c);
          if (BIAS) tmem_st32(t_s + 32 * c, z);
          mx = chunk_max(z, mx);
        }
        if (!BIAS) mx *= a.qk_scale_log2;  // scale > 0; -inf stays
      }
      // the running maximum as the tile before left it
      const float m_old = m;
      if (i > 0) {
        wait(bar_m + 4 * (odd ^ 1), (uint32_t)(((i - 1) >> 1) & 1));
        if (!ok) break;
        m = sh_m[(odd ^ 1) * kTile];
      }
      float top = m + kLazyMax;
      if (CAP && !BIAS) {
        const bool ask = !(mx <= top);
        if (__any_sync(0xffffffffu, ask)) {
          float exact = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            ld32(t_s + 32 * c, z);
            if (masked) chunk_mask(z, run.x - k0 - 32 * c, run.y - k0 - 32 * c);
            exact = chunk_max(z, exact);
          }
          // (a row asks for itself: the others' results do not depend on it)
          if (ask) {
            mx = exact > -INFINITY ? cap_score(a.mod, exact * a.mod.y_scale) : exact;
            top = m;  // so that the bound will not ask again soon
          }
        }
      }
      const float m_prev = m;
      const bool grow = mx > top;
      if (grow) m = mx;
      sh_m[odd * kTile] = m;
      __syncwarp();
      if (lane == 0) bar_arrive(bar(bar_m + 4 * odd));
      if (__any_sync(0xffffffffu, m != m_old)) l *= fast_exp2(m_old - m);
      if (i > 0 && __any_sync(0xffffffffu, grow)) {
        const float alpha = fast_exp2(m_prev - m);
        wait(kFBarO + 2 * x + (odd ^ 1), (uint32_t)(((i - 1) >> 1) & 1));  // the P V before
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll 1
        for (int c0 = 0; c0 < kHeadDim; c0 += 16) {
          float t[16];
          ld16(t_o + c0, t);
#pragma unroll
          for (int e = 0; e < 16; ++e) t[e] *= alpha;
          st16(t_o + c0, t);
        }
      }
      if (rare & kInfoBad) {  // V rows that are not finite
#pragma unroll 1
        for (int e = 0; e < kKeys && k0 + e < n; ++e)
          if ((a.bad[info_row * 4 + (k0 + e) / 32] >> (e & 31)) & 1u) poison |= k0 + e >= run.x && k0 + e < run.y;
      }
      // P (fp16) over the front of the products: chunk c's 16 columns lie before
      // the products of chunk c + 1
      f32x2 ls[2] = {0, 0};
      if (BIAS) tmem_st_wait();
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t pw[16];
        ld32(t_s + 32 * c, z);
        if (CAP && !BIAS)
          chunk_cap(a, z, most, m);
        else
          chunk_shift(z, BIAS ? 1.0f : a.qk_scale_log2, m);
        if (!BIAS && masked) chunk_mask(z, run.x - k0 - 32 * c, run.y - k0 - 32 * c);
        chunk_probs(z, pw, ls);
        tmem_st16(t_s + 16 * c, pw);
      }
      float lx, ly;
      unpack2(add2(ls[0], ls[1]), lx, ly);
      l += lx + ly;
      tmem_st_wait();
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) bar_arrive(bar(kFBarP + 2 * x + odd));
    }
    // the final maximum, the sum and poison of both threads of the row
    const int last = n_x - 1;
    if (ok && last >= 0) {
      if (odd != (last & 1)) {
        wait(bar_m + 4 * (odd ^ 1), (uint32_t)((last >> 1) & 1));
        const float m_last = sh_m[(odd ^ 1) * kTile];
        l *= fast_exp2(m - m_last);
        m = m_last;
      }
      wait(kFBarO + 2 * x + (last & 1), (uint32_t)((last >> 1) & 1));
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    }
    asm volatile("bar.sync %0, 256;" ::"r"(kNbTile + x) : "memory");  // every maximum is read
    sh_m[odd * kTile] = l;
    asm volatile("bar.sync %0, 256;" ::"r"(kNbTile + x) : "memory");
    const float total = sh_m[0] + sh_m[kTile];
    asm volatile("bar.sync %0, 256;" ::"r"(kNbTile + x) : "memory");
    sh_m[odd * kTile] = poison ? 1.0f : 0.0f;
    asm volatile("bar.sync %0, 256;" ::"r"(kNbTile + x) : "memory");
    poison = sh_m[0] + sh_m[kTile] != 0.0f;
    // (where the tile has no keys nothing above has waited for its Q)
    if (last < 0) wait(kFBarQ + x, 0);
    if (ok && !*abort) {
      // the output takes Q's place in shared memory (every S of the tile is
      // complete) and leaves by TMA, 32 rows of 64 dims a warp: stores of a row
      // a thread took 2800 cycles of the load-store unit a block
      float inv = total != 0.0f ? 1.0f / total : 0.0f;  // a row that sees nothing is 0
      // V's power of two comes out, in two steps where 1 / l over it would be subnormal
      const int shift = (int)(rare >> kInfoShift), down = max(shift - 60, 0);
      if (shift != 0) inv *= pow2(down - shift);
      uint8_t* orow = fsm + kFOffQ + x * kTileB + odd * kBoxB + row * 128;
#pragma unroll 1
      for (int c0 = 0; c0 < 64; c0 += 32) {
        float t[32];
        if (last >= 0) {
          ld32(t_o + 64 * odd + c0, t);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) t[e] = 0.0f;
        }
        if (down != 0) {
#pragma unroll
          for (int e = 0; e < 32; ++e) t[e] *= pow2(-down);
        }
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const __nv_bfloat162 pr = __floats2bfloat162_rn(t[2 * e] * inv, t[2 * e + 1] * inv);
          w[e] = poison ? 0x7FFF7FFFu : *reinterpret_cast<const uint32_t*>(&pr);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)  // (chunks of 16 bytes in the 128-byte swizzle)
          *reinterpret_cast<uint4*>(orow + (((c0 >> 3) + e) ^ (row & 7)) * 16) =
              make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
      }
      fence_async();
      __syncwarp();
      if (lane == 0 && qi < n) {
        tma_store_3d(&tm_o, base + kFOffQ + x * kTileB + odd * kBoxB + row * 128, 64 * odd, qi, plane_q);
        tma_stores_read();
      }
      const bool row_ok = qi < n;
      if (row_ok && !odd && a.stats != nullptr)
        *reinterpret_cast<float2*>(a.stats + ((size_t)plane_q * n + qi) * 2) = make_float2(m, total);
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 16) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kFwdCols));
}

// ---------------------------------------------------------------------------
// Column sums: key j's sum over the queries that see it and the query heads of
// its KV head of exp2(z - m_i) / l_i, with the forward's row statistics.
//
// One 320-thread CTA per (128-key tile, KV head, sequence), two per SM, keys
// on the TMEM lanes: S^T = K Q^T (M 128, N 128), so thread t of a warpgroup
// owns key t and adds in registers; a fixed order.  With few key tiles several
// CTAs share one, each with some of the query heads; the last of them (a ticket)
// adds their sums in order.  (64 heads of
// 2,100 tokens, capped and biased: about 88 us, bound by the FMA pipe and the
// unevenness of the blocks.)  A block's statistics have places of their own, and
// its products' place is free once they are read, so that the next Q and S come
// under a block's sums (40 heads on 8 of 2 x 4,000 tokens: 526 us with the
// attention, 551 with Q's place held to the block's end).  Warpgroups 0
// and 1 take alternate (query head, query tile) blocks, warp 8 loads the query
// tiles and stages -m, 1 / l and the run per query, warp 9 issues the products.
// Two queries go through each instruction (their -m and 1 / l are pairs in
// shared memory; the cap ends in an addition, which takes -m along).
// Query tiles none of whose queries sees the key tile are skipped; tiles seen
// whole take no mask.
constexpr int kSumThreads = 320;
constexpr int kSOffK = 0;
constexpr int kSOffQ = kSOffK + kTileB;                    // 2 slots
constexpr int kSStats = 4;                                 // places of a block's statistics and runs
constexpr int kSOffStat = kSOffQ + 2 * kTileB;             // 4 x (128 x -m, 128 x 1 / l)
constexpr int kSOffRun = kSOffStat + kSStats * kTile * 8;  // 4 x 128 x (begin, end)
constexpr int kSOffRed = kSOffRun + kSStats * kTile * 8;   // 128 sums
constexpr int kSOffBar = kSOffRed + kTile * 4;
// mbarriers: K landed; a block's Q landed, its place free (per block % 2); S
// complete, read (% 2); statistics there, read (% 4); all products complete
constexpr int kSBarK = 0, kSBarFull = 1, kSBarEmpty = 3, kSBarS = 5, kSBarSfree = 7, kSBarStat = 9, kSBarStatfree = 13,
              kSBarDone = 17, kSNumBars = 18;
constexpr int kSumSmem = kSOffBar + 8 * kSNumBars + 16;
constexpr uint32_t kSumCols = 256;
constexpr size_t kSumCtas = 608;  // two waves of two a SM on 152 SMs

// The (query head, query tile) blocks some of whose queries see the keys [k0,
// k1), in order, for a warp: 32 tiles' bounds are read at a time, one a lane (a
// load per tile would put its latency into every block).
struct SeenBlocks {
  const int4* runs;
  int tiles, heads, k0, k1, lane;
  int g, qt, base;
  uint32_t left, whole;
  bool all;  // every query of the block sees every key
  __device__ SeenBlocks(const int4* r, int t, int first, int end, int a, int b, int l)
      : runs(r), tiles(t), heads(end), k0(a), k1(b), lane(l), g(first), qt(0), base(-32), left(0), whole(0), all(false) {}
  __device__ bool next() {
    while (left == 0) {
      base += 32;
      if (base >= tiles) {
        base = -32;
        if (++g >= heads) return false;
        continue;
      }
      const int4 r = base + lane < tiles ? runs[base + lane] : make_int4(INT_MAX, 0, 0, 0);
      const bool sees = r.x < k1 && r.y > k0;
      left = __ballot_sync(0xffffffffu, sees);
      whole = __ballot_sync(0xffffffffu, r.z <= k0 && r.w >= k1);
    }
    const int b = __ffs(left) - 1;
    left &= left - 1;
    qt = base + b;
    all = (whole >> b) & 1u;
    return true;
  }
};

template <bool CAP, bool BIAS>
__global__ void __launch_bounds__(kSumThreads, 2)
    prompt_sums_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k) {
  extern __shared__ __align__(1024) uint8_t ssm[];
  __shared__ int sh_last;
  const uint32_t base = saddr(ssm);
  uint32_t* tbase = reinterpret_cast<uint32_t*>(ssm + kSOffBar + 8 * kSNumBars);
  volatile int* abort = reinterpret_cast<volatile int*>(ssm + kSOffBar + 8 * kSNumBars + 4);
  auto bar = [&](int i) { return base + kSOffBar + 8 * i; };
  const int n = a.n, G = a.group;
  const int planes = a.hkv * a.batch, parts = a.sum_parts, rest = blockIdx.x % (planes * parts);
  const int kt = blockIdx.x / (planes * parts), plane_kv = rest / parts, part = rest % parts;
  const int h = plane_kv % a.hkv, bl = plane_kv / a.hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int k0 = kt * kTile, k1 = min(k0 + kTile, n);
  const int tiles = (n + kTile - 1) / kTile;
  SeenBlocks blk(a.runs + (size_t)bl * tiles, tiles, G * part / parts, G * (part + 1) / parts, k0, k1, lane);

  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tbase)), "r"(kSumCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int i = 0; i < kSNumBars; ++i) {
      const uint32_t cnt = (i >= kSBarSfree && i < kSBarSfree + 2) || (i >= kSBarStatfree && i < kSBarStatfree + 4) ? 4 : 1;
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar(i)), "r"(cnt));
    }
    *abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tbase, 0);
  float sum = 0.0f;

  if (warp == 8) {
    // ------------------------------------------ K, query tiles, row statistics
    if (lane == 0) {
      bar_expect_tx(bar(kSBarK), kTileB);
      tma_load_3d(base + kSOffK, &tm_k, 0, k0, bl * a.hkv + h, bar(kSBarK));
      tma_load_3d(base + kSOffK + kBoxB, &tm_k, 64, k0, bl * a.hkv + h, bar(kSBarK));
    }
    int it = 0;
    // the statistics and runs of a block, read while the one before is waited for
    float2 s[kTile / 32];
    int2 r[kTile / 32];
    auto read = [&]() {
      const int plane = bl * a.hq + h * G + blk.g;
#pragma unroll
      for (int e = 0; e < kTile / 32; ++e) {
        const int qi = blk.qt * kTile + lane + 32 * e;
        s[e] = make_float2(INFINITY, 0.0f);  // past the prompt: p = 2^-inf
        r[e] = make_int2(0, 0);
        if (qi < n) {
          s[e] = *reinterpret_cast<const float2*>(a.stats + ((size_t)plane * n + qi) * 2);
          r[e] = run_of(a, bl, qi);
        }
      }
    };
    bool more = blk.next();
    if (more) read();
    while (more) {
      const int x = it & 1;
      if (it >= 2 && !__all_sync(0xffffffffu, bar_wait(bar(kSBarEmpty + x), (uint32_t)(((it - 2) >> 1) & 1), abort))) {
        set_abort(a.status, abort);
        break;
      }
      if (lane == 0) {
        const int plane = bl * a.hq + h * G + blk.g;
        const uint32_t dst = base + kSOffQ + x * kTileB, b = bar(kSBarFull + x);
        bar_expect_tx(b, kTileB);
        tma_load_3d(dst, &tm_q, 0, blk.qt * kTile, plane, b);
        tma_load_3d(dst + kBoxB, &tm_q, 64, blk.qt * kTile, plane, b);
      }
      const int y = it % kSStats;
      if (it >= kSStats && !__all_sync(0xffffffffu, bar_wait(bar(kSBarStatfree + y),
                                                             (uint32_t)(((it - kSStats) / kSStats) & 1), abort))) {
        set_abort(a.status, abort);
        ++it;  // (its Q is on the way)
        break;
      }
      float* st = reinterpret_cast<float*>(ssm + kSOffStat) + y * 2 * kTile;
      int2* rn = reinterpret_cast<int2*>(ssm + kSOffRun) + y * kTile;
#pragma unroll
      for (int e = 0; e < kTile / 32; ++e) {
        const int i = lane + 32 * e;
        const bool some = s[e].y != 0.0f;
        st[i] = some ? -s[e].x : -INFINITY;
        st[kTile + i] = some ? 1.0f / s[e].y : 0.0f;
        rn[i] = r[e];
      }
      __syncwarp();
      if (lane == 0) bar_arrive(bar(kSBarStat + y));
      ++it;
      more = blk.next();
      if (more) read();
    }
    if (lane == 0) {
      // the last copies land before the CTA goes away
      bar_wait(bar(kSBarK), 0, nullptr);
      for (int e = max(0, it - 2); e < it; ++e) bar_wait(bar(kSBarFull + (e & 1)), (uint32_t)((e >> 1) & 1), nullptr);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ----------------------------------------------------------------- products
    const bool el = elect_one();
    const uint32_t id_s = instr_desc(kTile, kTile, true);
    bool ok = __all_sync(0xffffffffu, bar_wait(bar(kSBarK), 0, abort));
    if (!ok) set_abort(a.status, abort);
    for (int it = 0; ok && blk.next(); ++it) {
      const int x = it & 1;
      if (!__all_sync(0xffffffffu, bar_wait(bar(kSBarFull + x), (uint32_t)((it >> 1) & 1), abort) &&
                                       (it < 2 || bar_wait(bar(kSBarSfree + x), (uint32_t)(((it - 2) >> 1) & 1), abort)))) {
        set_abort(a.status, abort);
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      if (el) {
        const uint32_t ka = base + kSOffK, qa = base + kSOffQ + x * kTileB;
#pragma unroll
        for (int ks = 0; ks < kHeadDim / 16; ++ks) {
          const uint32_t off = (ks >> 2) * kBoxB + (ks & 3) * 32;
          mma_f16(tmem + kTile * x, op_desc_sw128(ka + off), op_desc_sw128(qa + off), id_s, ks > 0);
        }
        mma_commit(bar(kSBarS + x));
        mma_commit(bar(kSBarEmpty + x));
      }
      __syncwarp();
    }
    if (el) mma_commit(bar(kSBarDone));
    bar_wait(bar(kSBarDone), 0, nullptr);
    __syncwarp();
  } else {
    // ------------------------------------------------------ sums over the queries
    const int x = warp >> 2, t = tid & (kTile - 1);
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kTile * x;
    const int key = k0 + t;
    int g = -1;
    float slope2 = 0.0f;
    for (int it = 0; blk.next(); ++it) {
      if ((it & 1) != x) continue;
      if (BIAS && blk.g != g) {
        g = blk.g;
        slope2 = slope_log2(a.mod, h * G + g);
      }
      const uint32_t par = (uint32_t)((it >> 1) & 1);
      const int y = it % kSStats;
      const float* st = reinterpret_cast<const float*>(ssm + kSOffStat) + y * 2 * kTile;
      const int2* rn = reinterpret_cast<const int2*>(ssm + kSOffRun) + y * kTile;
      if (!__all_sync(0xffffffffu, bar_wait(bar(kSBarS + x), par, abort) &&
                                       bar_wait(bar(kSBarStat + y), (uint32_t)((it / kSStats) & 1), abort))) {
        set_abort(a.status, abort);
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const bool whole = blk.all;
      const int q0 = blk.qt * kTile;
      f32x2 acc[2] = {0, 0};
#pragma unroll 1
      for (int c0 = 0; c0 < kTile; c0 += 32) {
        float z[32];
        ld32(trow + c0, z);
        if (c0 == kTile - 32) {  // the products may come over these
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();
          if (lane == 0) bar_arrive(bar(kSBarSfree + x));
        }
        auto nm = [&](int i) { return *reinterpret_cast<const f32x2*>(st + c0 + i); };
        const float d0 = (float)(q0 + c0 - key);
        const bool both = q0 + c0 < key - lane + 31;  // some key of the warp lies after the query
        if (BIAS && both) {
          if (CAP) chunk_cap(a, z, chunk_most(z, 0.0f), 0.0f);
          chunk_bias(z, CAP ? 1.0f : a.qk_scale_log2, slope2, -slope2, d0, true);
#pragma unroll
          for (int i = 0; i < 32; i += 2) unpack2(add2(pack2(z[i], z[i + 1]), nm(i)), z[i], z[i + 1]);
        } else {
          // what is added to a pair of scores: -m, less the bias
          const f32x2 sl = pack2(-slope2, -slope2), two = pack2(2.0f, 2.0f);
          f32x2 d = pack2(d0, d0 + 1.0f);
          auto plus = [&](int i) {
            if (!BIAS) return nm(i);
            const f32x2 add = fma2(d, sl, nm(i));
            d = add2(d, two);
            return add;
          };
          if (CAP) {
            chunk_cap_plus(a, z, chunk_most(z, 0.0f), plus);
          } else {
            const f32x2 sc = pack2(a.qk_scale_log2, a.qk_scale_log2);
#pragma unroll
            for (int i = 0; i < 32; i += 2) unpack2(fma2(pack2(z[i], z[i + 1]), sc, plus(i)), z[i], z[i + 1]);
          }
        }
        if (whole) {
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const f32x2 p = pack2(fast_exp2(z[i]), fast_exp2(z[i + 1]));
            acc[(i >> 1) & 1] = fma2(p, *reinterpret_cast<const f32x2*>(st + kTile + c0 + i), acc[(i >> 1) & 1]);
          }
        } else {
          // (statistics of a row that does not see the key may be anything)
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const int4 b = *reinterpret_cast<const int4*>(rn + c0 + i);
            float x0, x1;
            unpack2(mul2(pack2(fast_exp2(z[i]), fast_exp2(z[i + 1])),
                         *reinterpret_cast<const f32x2*>(st + kTile + c0 + i)),
                    x0, x1);
            x0 = key >= b.x && key < b.y ? x0 : 0.0f;
            x1 = key >= b.z && key < b.w ? x1 : 0.0f;
            acc[(i >> 1) & 1] = add2(acc[(i >> 1) & 1], pack2(x0, x1));
          }
        }
      }
      float ax, ay;
      unpack2(add2(acc[0], acc[1]), ax, ay);
      sum += ax + ay;
      __syncwarp();
      if (lane == 0) bar_arrive(bar(kSBarStatfree + y));
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  float* red = reinterpret_cast<float*>(ssm + kSOffRed);
  if (tid < kTile) red[tid] = sum;
  __syncthreads();
  const bool mine = tid >= kTile && tid < 2 * kTile && k0 + tid - kTile < n && !*abort;
  const size_t at = (size_t)plane_kv * n + k0 + tid - kTile;
  if (parts == 1) {
    if (mine) a.sums[at] = sum + red[tid - kTile];
  } else {
    // the last part of the key tile adds them up, in order
    if (mine) a.sum_part[(size_t)part * planes * n + at] = sum + red[tid - kTile];
    __syncthreads();
    if (tid == 0) {
      __threadfence();
      sh_last = atomicAdd(&a.sum_tickets[(size_t)plane_kv * tiles + kt], 1) == parts - 1;
      __threadfence();
    }
    __syncthreads();
    if (sh_last && mine) {
      float total = 0.0f;
      for (int e = 0; e < parts; ++e) total += __ldcg(a.sum_part + (size_t)e * planes * n + at);
      a.sums[at] = total;
    }
  }
  if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kSumCols));
}

// Column sums of a fresh prompt into the score slots of a cache's tokens.
__global__ void prompt_scores_kernel(DevState s, int seq_begin, int n, const float* __restrict__ sums) {
  const int p = blockIdx.x * blockDim.x + threadIdx.x, h = blockIdx.y, bl = blockIdx.z;
  if (p >= n) return;
  const int b = seq_begin + bl;
  const float v = sums[((size_t)bl * s.hkv + h) * n + p];
  int lo, hi;
  pool_range(0, n, s.ring, &lo, &hi);
  if (p < kSinks) {
    s.sink_score[((size_t)b * s.hkv + h) * kSinks + p] = v;
  } else if (p < hi) {
    const int slot = p - lo;
    const int blk = s.block_table[(size_t)b * s.max_bps + slot / kPage];
    if ((unsigned)blk < (unsigned)s.num_blocks)
      s.score[((size_t)blk * s.hkv + h) * kPage + slot % kPage] = v;
    else
      atomicOr(&s.counters[kCtrStatus], kDevBadBlockId);
  } else {
    s.ring_score[((size_t)b * s.hkv + h) * s.ring + (p - kSinks) % s.ring] = v;
  }
}

template <bool CAP, bool BIAS>
cudaError_t launch_fwd(const PromptArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                       const CUtensorMap& o, cudaStream_t st) {
  static int done[64] = {0};
  const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(prompt_fwd_kernel<CAP, BIAS>), kFwdSmem, done);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((a.n + kFwdBlock - 1) / kFwdBlock * (a.hq * a.batch)));
  // may start while the prep kernel's last CTAs run (wait_for_previous)
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kFwdThreads);
  cfg.dynamicSmemBytes = kFwdSmem;
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prompt_fwd_kernel<CAP, BIAS>, a, q, k, v, o);
}

template <bool CAP, bool BIAS>
cudaError_t launch_sums(const PromptArgs& a, const CUtensorMap& q, const CUtensorMap& k, cudaStream_t st) {
  static int done[64] = {0};
  const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(prompt_sums_kernel<CAP, BIAS>), kSumSmem, done);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((a.n + kTile - 1) / kTile * (a.hkv * a.batch * a.sum_parts)));
  prompt_sums_kernel<CAP, BIAS><<<grid, kSumThreads, kSumSmem, st>>>(a, q, k);
  return cudaGetLastError();
}

}  // namespace

PromptWs prompt_ws(int batch, int hq, int hkv, int n, bool sums) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t tiles = ((size_t)n + kTile - 1) / kTile, planes = (size_t)batch * hkv;
  PromptWs w{};
  w.v16 = 0;
  w.bad = up(planes * n * kHeadDim * 2);
  w.info = w.bad + up(planes * tiles * 16);
  w.runs = w.info + up(planes * tiles * 4);
  w.stats = w.runs + up(sums ? batch * tiles * 16 : 0);
  w.sums = w.stats + up(sums ? (size_t)batch * hq * n * 8 : 0);
  // column sums with few key tiles and KV heads: several CTAs for each, with some
  // of its query heads, so that there are about kSumCtas, two full waves (32 heads
  // on 8 of 8,192 tokens then 910 us with the attention, 984 with one CTA each, 981
  // at 304, 925 at 1,216; 2 x 14 heads on 2 of 1,529 tokens 68 against 155; every
  // parts-th block instead of some heads: 926 and 74)
  const size_t group = (size_t)(hq / hkv), each = planes * tiles;
  w.sum_parts = sums ? (int)std::min(group, (kSumCtas + each - 1) / each) : 1;
  const bool split = w.sum_parts > 1;
  w.part = w.sums + up(sums ? planes * n * 4 : 0);
  w.tickets = w.part + up(split ? w.sum_parts * planes * n * 4 : 0);
  w.total = w.tickets + up(split ? each * 4 : 0);
  return w;
}

cudaError_t launch_prompt_scores(const DevState& s, int seq_begin, int batch, int n, const float* sums,
                                 cudaStream_t st) {
  prompt_scores_kernel<<<dim3((n + 255) / 256, s.hkv, batch), 256, 0, st>>>(s, seq_begin, n, sums);
  return cudaGetLastError();
}

// The degree-2 polynomial takes q . k itself: x (c0 + u (c1 + ...)), u = x^2, so
// its coefficients carry powers of y_scale up to the seventh times the cap: a
// y_scale far from 1, or coefficients beyond fp32's normal range (caps no model
// uses), go without it.
void prompt_polynomials(PromptArgs* a) {
  a->close_max = a->mid_max = -1.0f;
  const double ys = a->mod.y_scale, c2 = a->mod.c2;
  if (!(c2 > 0.0) || !(ys > 0.0)) return;
  a->mid_max = (float)(kCapMid / ys);
  a->mid[0] = (float)c2;
  for (int i = 0; i < 9; ++i) a->mid[i + 1] = (float)(c2 * kCapP8[i]);
  if (ys < 5e-4 || ys > 1e3) return;
  double pw = ys, c[4] = {c2 * pw};
  for (int i = 0; i < 3; ++i) {
    pw *= ys * ys;
    c[i + 1] = c2 * kCapP2[i] * pw;
  }
  for (int i = 0; i < 4; ++i) {
    if (!(std::abs(c[i]) >= 1e-37 && std::abs(c[i]) <= 1e37)) return;
    a->close[i] = (float)c[i];
  }
  a->close_max = (float)(kCapClose / ys);
}

cudaError_t launch_prompt(const PromptArgs& args, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                          cudaStream_t st) {
  PromptArgs a = args;
  prompt_polynomials(&a);
  CUtensorMap tm_q, tm_k, tm_v, tm_o, tm_ks;
  if (!encode_rows_map(&tm_q, q, a.n, a.batch * a.hq, kTile) || !encode_rows_map(&tm_k, k, a.n, a.batch * a.hkv, kKeys) ||
      !encode_rows_map(&tm_v, a.v16, a.n, a.batch * a.hkv, kKeys, CU_TENSOR_MAP_DATA_TYPE_FLOAT16) ||
      !encode_rows_map(&tm_o, a.out, a.n, a.batch * a.hq, 32) ||
      (a.sums != nullptr && !encode_rows_map(&tm_ks, k, a.n, a.batch * a.hkv, kTile)))
    return cudaErrorInvalidValue;
  prompt_prep_kernel<<<(a.n + kTile - 1) / kTile * (a.batch * a.hkv), kPrepThreads, 0, st>>>(a, v);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const bool cap = a.mod.c2 > 0.0f, bias = a.mod.slopes != nullptr;
  e = cap ? (bias ? launch_fwd<true, true>(a, tm_q, tm_k, tm_v, tm_o, st) : launch_fwd<true, false>(a, tm_q, tm_k, tm_v, tm_o, st))
          : (bias ? launch_fwd<false, true>(a, tm_q, tm_k, tm_v, tm_o, st)
                  : launch_fwd<false, false>(a, tm_q, tm_k, tm_v, tm_o, st));
  if (e != cudaSuccess || a.sums == nullptr) return e;
  return cap ? (bias ? launch_sums<true, true>(a, tm_q, tm_ks, st) : launch_sums<true, false>(a, tm_q, tm_ks, st))
             : (bias ? launch_sums<false, true>(a, tm_q, tm_ks, st) : launch_sums<false, false>(a, tm_q, tm_ks, st));
}

}  // namespace kvc
