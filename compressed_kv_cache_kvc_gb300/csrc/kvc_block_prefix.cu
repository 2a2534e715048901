// Attention of sequences that share a prefix: softmax over the prefix's tokens,
// held once, and each sequence's own.
//
// Two forms.  Few or short: block_attn_kernel goes through the prefix's pages for
// every sequence (they come from L2 after the first).  Else the prefix's closed
// blocks are a matrix product, 4 * 128 flops per query row and token:
// prefix_tc_kernel takes all rows of a KV head (batch x query heads of the group)
// against a run of the blocks on the fifth-generation tensor cores, and
// block_attn_kernel, which has the sequences' own tokens and everything held
// exactly, joins its partial results.
//
// prefix_tc_kernel.  One 640-thread CTA per (up to 256 rows, KV head, run of
// 128-token tiles), in two streams: the two 128-row query tiles, or (up to 128 rows)
// every other tile of tokens for the same rows, joined in the end.
//   * warps 4-7 and 8-11: the softmax of one stream each, a thread a row;
//   * warps 12-19: codes from global memory (the next tile's on their way in
//     registers) to fp16 in shared memory, K and V alike [128 tokens][128 dims] in
//     two boxes of 64 dims with the 128-byte swizzle; every code is exact in fp16;
//   * warp 1: the scales, and the codes of the tiles ahead into L2;
//   * warps 0 and 2 issue the products of a query tile each (one warp for both spent
//     half of its time between them): S = Q K^T (Q fp16 times a power of two per
//     row, which is exact for everything within 2^-28 of the row's largest value),
//     O += P V with P from tensor memory.
// A step is 64 tokens.  TMEM columns: S_x of step j at 128 x + 64 (j % 2), O_x at
// 256 + 128 x; P (fp16) takes the back half of its S.  In step j the MMA warp of query
// tile x issues PV_x(j - 2), S_x(j): the pipe runs one thread's products in order, so
// S(j) may overwrite P(j - 2), and a softmax finds the scores of its next step ready.
// A block's K scale multiplies its scores, its V scale over a power of two its
// probabilities (P, fp16).  That power is the row's own and follows the largest product
// of p and V scale that the row has met, so that P keeps 11 bits down to 2^-14 of it
// and is off by 2^-25 of it below, whatever the V of tokens without weight; O leaves
// times that power.  Maximum and power are lazy: P is formed with those so far, and only
// where 32 p, or they times their V scales, sum to more than 2^15 are they looked for
// and O rescaled, so that P fits fp16 and most steps read their scores once and compare
// nothing (with the maximum of every step first 43 us where this takes 37, 64 x 32
// heads after 32,768 tokens).  The sums add the unrounded p in fp32.
// Tiles, and the steps and chunks inside, go from the last to the first: with a
// distance bias the nearest come first, and the maximum hardly ever rises again.
// Synchronisation: mbarriers, every wait bounded, as in the prompt kernels.
//
// 64 x 32 heads on 8 after 32,768 tokens 38 us, 0.91 PFLOP/s (47 % of a library product's
// rate, which counts the conversion of the codes, exp2 and the first and last 4 us of a
// CTA); 24 x 40 heads, capped, biased E4M3, after 16,001 25 us: the softmax of 120 rows.
// The sequences' own tokens and the join after them 24 and 21 us: one and a half and
// one wave of CTAs, each a chain of round trips (lengths, ids, scales and pages, the
// parts), 11 to 14 us without any page.
#include "kvc_block_attn.h"
#include "kvc_tc.h"

namespace kvc {
namespace {

using namespace tc;

constexpr int kTile = 128;  // query rows and tokens per tile
constexpr int kStep = 64;   // tokens per step of the softmax
constexpr int kRows = 2 * kTile;
constexpr int kSoftWarps = 8, kLoadWarps = 8;
// (the first warps are the ones the schedulers prefer: what the others wait for goes first)
constexpr int kMmaWarp = 0, kScoutWarp = 1, kMmaWarp2 = 2, kSoft0 = 4, kLoad0 = kSoft0 + kSoftWarps;
constexpr int kThreads = 32 * (kLoad0 + kLoadWarps);
constexpr int kTileB = kTile * kHeadDim * 2;  // 32 KB, two boxes of 64 dims
constexpr int kBoxB = kTileB / 2;
constexpr int kOffQ = 0, kOffK = kOffQ + 2 * kTileB, kOffV = kOffK + 2 * kTileB;
// a tile's K and V scales and which of its eight 16-token pages count, four tiles deep
// (a slot is written again when the softmax of the tile four before has read it: the
// scout has a barrier of its own for that, since one that also completes without its
// scales could complete twice before it looks)
constexpr int kOffScale = kOffV + 2 * kTileB;  // [4][2][8] f32
constexpr int kOffMask = kOffScale + 4 * 2 * 8 * 4;
constexpr int kOffBar = kOffMask + 4 * 4;
constexpr int kBarQ = 0, kBarK = 1, kBarV = 3, kBarKFree = 5, kBarVFree = 7, kBarS = 9, kBarP = 13, kBarO = 17,
              kBarScale = 21, kBarDone = 25, kBarScaleFree = 27, kNumBars = 31;  // (S, P, O: 2 x + step parity)
constexpr int kOffMisc = kOffBar + 8 * kNumBars;  // TMEM base, abort flag
constexpr int kOffMl = kOffMisc + 32;  // [2][128][2] the rows' maxima and sums
constexpr int kSmem = kOffMl + 2 * kTile * 8;
constexpr float kMostSum = 32768.0f;
constexpr int kAhead = 1;  // (before the scout's own up to four) tiles whose codes are on their way to L2
constexpr uint32_t kCols = 512;

__device__ __forceinline__ float group_max(const float* z, float m) {
  float t0 = m, t1 = -INFINITY;
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    t0 = max3(t0, z[i], z[i + 1]);
    t1 = max3(t1, z[i + 2], z[i + 3]);
  }
  return fmaxf(t0, t1);
}
__device__ __forceinline__ float group_most(const float* z, float m) {
  float t0 = m, t1 = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    t0 = max3_abs(t0, z[i], z[i + 1]);
    t1 = max3_abs(t1, z[i + 2], z[i + 3]);
  }
  return fmaxf(t0, t1);
}

// 16 raw products times f, capped, plus `add` (the magnitudes of the scaled ones are
// at most `most`)
__device__ __forceinline__ void group_cap(const ScoreMod& mod, float* z, float f, float most, float add) {
  if (most <= kCapNear) {
    const f32x2 f2 = pack2(f, f), a2 = pack2(add, add);
    f32x2 c[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) c[i] = pack2(mod.poly[i], mod.poly[i]);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const f32x2 y = mul2(pack2(z[i], z[i + 1]), f2), u = mul2(y, y);
      f32x2 h = fma2(c[4], u, c[3]);
      h = fma2(h, u, c[2]);
      h = fma2(h, u, c[1]);
      h = fma2(h, u, c[0]);
      unpack2(fma2(y, h, a2), z[i], z[i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = cap_far(mod, z[i] * f) + add;
  }
}

template <bool FP8, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_tc_kernel(BlockState s, int seq_begin, const uint16_t* __restrict__ q, const __grid_constant__ PrefixTc a) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t base = saddr(sm);
  uint32_t* tbase = reinterpret_cast<uint32_t*>(sm + kOffMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(sm + kOffMisc + 4);
  auto bar = [&](int i) { return base + kOffBar + 8 * i; };
  auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  int* status = s.counters + kCtrStatus;

  launch_dependents();
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tbase)), "r"(kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  const int G = s.group, hkv = s.hkv, bt = s.bt, sh = __ffs(bt) - 1;
  const int rows_all = a.batch * G, row_blocks = (rows_all + kRows - 1) / kRows;
  const int rb = blockIdx.x % row_blocks, split = blockIdx.x / row_blocks % a.splits;
  const int h = blockIdx.x / row_blocks / a.splits;
  // up to 128 rows: both streams have them, every other tile each
  const int rows = min(rows_all - rb * kRows, kRows), nq = rows > kTile ? 2 : 1;
  const bool single = nq == 1;
  if (tid == 32) {
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t count = 1;
      if (i == kBarQ) count = 4 * nq;
      if (i >= kBarK && i < kBarKFree) count = kLoadWarps / 2;
      if (i >= kBarKFree && i < kBarS) count = nq;
      if (i >= kBarP && i < kBarO) count = 4;  // (warps of a query tile)
      if (i >= kBarScaleFree) count = 4 * nq;
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar(i)), "r"(count));
    }
    *abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async();
  }
  const int pre_len = s.seq_pos[a.prefix];
  const int n_tok = block_closed(pre_len, bt) << sh;
  const int tiles = (n_tok + kTile - 1) / kTile;
  const int t0 = (int)((long long)tiles * split / a.splits), t1 = (int)((long long)tiles * (split + 1) / a.splits);
  const int n_t = t1 - t0;  // tile i of the loops is t1 - 1 - i (none: a graph replayed with a shorter prefix)
  const int32_t* table = s.table + (size_t)a.prefix * s.max_bps;
  // this thread's row (softmax warps)
  const bool soft = warp >= kSoft0 && warp < kLoad0;
  const int x = (warp - kSoft0) >> 2, row = tid & (kTile - 1);
  const int in_block = (single ? 0 : x * kTile) + row, rr = rb * kRows + in_block;  // among the rows of the KV head
  const bool on = soft && in_block < rows;
  const int bl = on ? rr / G : 0, g = on ? rr % G : 0;
  const size_t part = (((size_t)split * hkv + h) * a.batch + bl) * G + g;
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = (uint32_t)uniform((int)*tbase);

  bool ok = true;
  auto wait = [&](int b, uint32_t par) {
    if (!__all_sync(0xffffffffu, bar_try(bar(b), par)) && !__all_sync(0xffffffffu, bar_wait(bar(b), par, abort))) {
      ok = false;
      if (!*abort) {
        *abort = 1;
        atomicOr(status, kDevWaitTimeout);
      }
    }
  };

  // stream x's tiles, the one of its index i, its slot of K and V and the slot's use
  auto tiles_of = [&](int x) { return single ? (n_t + 1 - x) >> 1 : n_t; };
  auto tile_of = [&](int x, int i) { return single ? 2 * i + x : i; };

  if (n_t == 0) {
    if (on && (x == 0 || !single)) {
      for (int e = 0; e < kHeadDim / 4; ++e)
        reinterpret_cast<float4*>(a.more_o + part * kHeadDim)[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      *reinterpret_cast<float2*>(a.more_ml + part * 2) = make_float2(kNegBig, 0.0f);
    }
  } else if (warp == kMmaWarp || warp == kMmaWarp2) {
    // ------------------------------------- products of one stream
    const bool el = elect_one();
    const int y = warp == kMmaWarp2;
    const uint32_t id_s = instr_desc(kTile, kStep, false), id_o = instr_desc(kTile, kHeadDim, false) | kInstrTransB;
    const uint64_t dq = op_desc_sw128(base + kOffQ), dk = op_desc_sw128(base + kOffK),
                   dv = op_desc_mn_sw128(base + kOffV, kBoxB);
    const int n_y = tiles_of(y);
    auto slot = [&](int i) { return tile_of(y, i) & 1; };
    auto use = [&](int i) { return (uint32_t)(tile_of(y, i) >> 1 & 1); };
    wait(kBarQ, 0);
    for (int j = 0; ok && j < 2 * n_y + 2; ++j) {
      const int i = j >> 1, e = i - 1;  // the tiles of this step's S and P V
      if (!(j & 1)) {
        if (i < n_y) wait(kBarK + slot(i), use(i));
        if (ok && e >= 0) wait(kBarV + slot(e), use(e));
        if (!ok) break;
      }
      if (e >= 0) {
        wait(kBarP + 2 * y + (j & 1), (uint32_t)(e & 1));
        if (!ok) break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t t_s = tmem + kTile * y + kStep * (j & 1), t_o = tmem + 256 + kTile * y;
      if (e >= 0 && el) {
        const uint64_t d = dv + (uint64_t)((slot(e) * kTileB + (~j & 1) * (kStep * 128)) >> 4);
#pragma unroll
        for (int ks = 0; ks < kStep / 16; ++ks)
          mma_f16_ts(t_o, t_s + kStep / 2 + 8 * ks, d + (uint64_t)((ks * 2048) >> 4), id_o, j > 2 || ks > 0);
        mma_commit(bar(kBarO + 2 * y + (j & 1)));
      }
      if (i < n_y && el) {
        const uint64_t d = dk + (uint64_t)((slot(i) * kTileB + (~j & 1) * (kStep * 128)) >> 4);
#pragma unroll
        for (int ks = 0; ks < kHeadDim / 16; ++ks)
          mma_f16(t_s, dq + (uint64_t)(((single ? 0 : y * kTileB) + (ks >> 2) * kBoxB + (ks & 3) * 32) >> 4),
                  d + (uint64_t)(((ks >> 2) * kBoxB + (ks & 3) * 32) >> 4), id_s, ks > 0);
        mma_commit(bar(kBarS + 2 * y + (j & 1)));
      }
      if (el && (j & 1)) {
        if (e >= 0) mma_commit(bar(kBarVFree + slot(e)));
        if (i < n_y) mma_commit(bar(kBarKFree + slot(i)));
      }
      __syncwarp();
    }
    // every product complete before the tensor memory goes back
    if (el) mma_commit(bar(kBarDone + y));
    bar_wait(bar(kBarDone + y), 0, nullptr);
    __syncwarp();
  } else if (warp == kScoutWarp) {
    // ------------------------- scales, and the codes of the tiles ahead into L2
    // lanes 0 .. 7 have the K, 8 .. 15 the V of a 16-token page
    const int page = lane & 7;
    const bool v = lane & 8;
    const uint8_t* codes = (v ? s.v_codes : s.k_codes) + (size_t)h * bt * kHeadDim;
    const float* scales = v ? s.v_scale : s.k_scale;
    auto id_of = [&](int i) {
      const int tok = (t1 - 1 - i) * kTile + 16 * page;
      if (lane >= 16 || i >= n_t || tok >= n_tok) return -1;
      const int id = table[tok >> sh];
      return (unsigned)id < (unsigned)s.num_blocks ? id : -2;
    };
    auto scale_of = [&](int id) { return id >= 0 ? scales[(size_t)id * hkv + h] : 0.0f; };
    auto fetch = [&](int i, int id) {
      if (id < 0) return;
      const int tok = (t1 - 1 - i) * kTile + 16 * page;
      const uint8_t* at = codes + (size_t)id * hkv * bt * kHeadDim + (size_t)(tok & (bt - 1)) * kHeadDim;
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"(16 * kHeadDim) : "memory");
    };
    int ids[kAhead + 1];  // of tiles i .. i + kAhead
#pragma unroll
    for (int e = 0; e <= kAhead; ++e) ids[e] = id_of(e);
#pragma unroll
    for (int e = 1; e < kAhead; ++e) fetch(e, ids[e]);
    float sc = scale_of(ids[0]);
#pragma unroll 1
    for (int i = 0; i < n_t; ++i) {
      const int id = ids[0], next = id_of(i + kAhead + 1);
      fetch(i + kAhead, ids[kAhead]);
      const float sc_next = scale_of(ids[1]);
      if (i >= 4) wait(kBarScaleFree + (i & 3), (uint32_t)((i >> 2) & 1) ^ 1u);
      if (!ok) break;
      float* to = reinterpret_cast<float*>(sm + kOffScale) + (i & 3) * 16;
      if (lane < 16) to[lane] = sc;
      if (id == -2 && lane < 8) atomicOr(status, kDevBadBlockId);
      const uint32_t pages = __ballot_sync(0xffffffffu, id >= 0) & 0xFFu;
      if (lane == 0) reinterpret_cast<uint32_t*>(sm + kOffMask)[i & 3] = pages;
      __syncwarp();
      if (lane == 0) bar_arrive(bar(kBarScale + (i & 3)));
      sc = sc_next;
#pragma unroll
      for (int e = 0; e < kAhead; ++e) ids[e] = ids[e + 1];
      ids[kAhead] = next;
    }
  } else if (warp >= kLoad0) {
    // ----------------------------------------------------- codes -> fp16 tiles
    // four warps have K, four V (so that neither waits for the other's slot); a thread
    // has 16 codes (column ch) of the rows r0, r0 + 16, ..
    const bool v = warp >= kLoad0 + kLoadWarps / 2;
    const int pt = tid - 32 * (kLoad0 + (v ? kLoadWarps / 2 : 0)), r0 = pt >> 3, ch = pt & 7;
    const size_t stride = (size_t)hkv * bt * kHeadDim;
    // (a row's place in its block: blocks do not cross tiles)
    const uint8_t* from = (v ? s.v_codes : s.k_codes) + (size_t)(h * bt + r0) * kHeadDim + 16 * ch;
    auto load_ids = [&](int i, int (&id)[8]) {
      const int tok = (t1 - 1 - i) * kTile;
#pragma unroll
      for (int e = 0; e < 8; ++e) id[e] = i < n_t && tok + 16 * e < n_tok ? table[(tok + 16 * e) >> sh] : -1;
    };
    auto load_codes = [&](const int (&id)[8], uint4 (&w)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        w[e] = make_uint4(0u, 0u, 0u, 0u);  // (the code 0 in both formats)
        if ((unsigned)id[e] < (unsigned)s.num_blocks)
          w[e] = *reinterpret_cast<const uint4*>(from + (uint32_t)id[e] * stride + (16 * e & (bt - 1)) * kHeadDim);
      }
    };
    auto to_halves = [&](uint32_t c, uint32_t& lo, uint32_t& hi) {
      if (FP8) {
        e4m3x4_to_h2(c, lo, hi);
      } else {  // 1024 + (code + 128) as fp16 patterns, minus 1152: exact
        const uint32_t u = c ^ 0x80808080u, k = 0x64806480u;
        const uint32_t a0 = __byte_perm(u, 0x64646464u, 0x4140), a1 = __byte_perm(u, 0x64646464u, 0x4342);
        __half2 x0 = __hsub2(*reinterpret_cast<const __half2*>(&a0), *reinterpret_cast<const __half2*>(&k));
        __half2 x1 = __hsub2(*reinterpret_cast<const __half2*>(&a1), *reinterpret_cast<const __half2*>(&k));
        lo = *reinterpret_cast<const uint32_t*>(&x0);
        hi = *reinterpret_cast<const uint32_t*>(&x1);
      }
    };
    // 16-byte chunks 2 (ch & 3) and the next of a row; the second box's lanes write
    // them in the other order (each bank once per 8 lanes)
    const int c0 = 2 * (ch & 3) + (ch >> 2);
    uint8_t* to0 = sm + (v ? kOffV : kOffK) + (ch >> 2) * kBoxB + r0 * 128 + ((c0 ^ (r0 & 7)) << 4);
    uint8_t* to1 = sm + (v ? kOffV : kOffK) + (ch >> 2) * kBoxB + r0 * 128 + ((c0 ^ 1 ^ (r0 & 7)) << 4);
    int id[8];
    uint4 w[8];
    load_ids(0, id);
    load_codes(id, w);
    load_ids(1, id);
    for (int i = 0; i < n_t; ++i) {
      if (i >= 2) wait((v ? kBarVFree : kBarKFree) + (i & 1), (uint32_t)((i >> 1) & 1) ^ 1u);
      if (!ok) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint4 y0, y1;
        to_halves(w[e].x, y0.x, y0.y);
        to_halves(w[e].y, y0.z, y0.w);
        to_halves(w[e].z, y1.x, y1.y);
        to_halves(w[e].w, y1.z, y1.w);
        *reinterpret_cast<uint4*>(to0 + (i & 1) * kTileB + e * 2048) = ch >> 2 ? y1 : y0;
        *reinterpret_cast<uint4*>(to1 + (i & 1) * kTileB + e * 2048) = ch >> 2 ? y0 : y1;
      }
      fence_async();
      __syncwarp();
      if (lane == 0) bar_arrive(bar((v ? kBarV : kBarK) + (i & 1)));
      load_codes(id, w);
      load_ids(i + 2, id);
    }
  } else if (soft) {
    // ----------------------------------------------------------- query rows
    float cq;
    int dist = 0;  // (BIAS) from the query to position 4 of the prefix
    if (BIAS && on) dist = pre_len + s.seq_pos[seq_begin + bl] - 1 - kSinks;
    {
      // the warp's rows as they are into their places (whole rows a copy), then each
      // thread its own, times a power of two, in fp16
      const uint32_t mine = (uint32_t)(bl * s.hq + h * G + g);
      const uint32_t to = base + kOffQ + (single ? 0 : x * kTileB);
      if (x < nq) {
#pragma unroll 8
        for (int i = 0; i < 16; ++i) {
          const int src_lane = 2 * i + (lane >> 4), r = (row & ~31) + src_lane, c = lane & 15;
          const uint32_t from = __shfl_sync(0xffffffffu, mine, src_lane);
          const uint32_t dst = to + (c >> 3) * kBoxB + r * 128 + (((c & 7) ^ (r & 7)) << 4);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst),
                       "l"(q + (size_t)from * kHeadDim + 8 * c), "r"((in_block & ~31) + src_lane < rows ? 16 : 0)
                       : "memory");
        }
        cp_async_commit();
        cp_async_wait<0>();
      }
      if (single) {  // (both streams' warps read the rows)
        asm volatile("bar.sync 1, %0;" ::"r"(32 * kSoftWarps) : "memory");
      } else {
        __syncwarp();
      }
      uint8_t* own = sm + kOffQ + (single ? 0 : x * kTileB) + row * 128;
      auto chunk = [&](int c) {
        return reinterpret_cast<uint4*>(own + (c >> 3) * kBoxB + (((c & 7) ^ (row & 7)) << 4));
      };
      float amax = 0.0f;
#pragma unroll 4
      for (int c = 0; c < 16; ++c) {
        const uint4 w = *chunk(c);
        const uint32_t y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = max3_abs(amax, bf16f(y[e] & 0xFFFFu), bf16f(y[e] >> 16));
      }
      int e2 = 0;
      if (amax > 0.0f) e2 = min(max(14 - exponent_of(amax), -100), 100);
      const float up = pow2i(e2);
      cq = (CAP ? a.mod.y_scale : a.qk_scale_log2) * pow2i(-e2);
      if (single) asm volatile("bar.sync 1, %0;" ::"r"(32 * kSoftWarps) : "memory");
      if (x < nq) {
#pragma unroll 4
        for (int c = 0; c < 16; ++c) {
          const uint4 w = *chunk(c);
          const uint32_t y[4] = {w.x, w.y, w.z, w.w};
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = pack_half2(bf16f(y[e] & 0xFFFFu) * up, bf16f(y[e] >> 16) * up);
          *chunk(c) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        fence_async();
        __syncwarp();
        if (lane == 0) bar_arrive(bar(kBarQ));
      }
    }
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_x = trow + kTile * x, t_o = trow + 256 + kTile * x;
    const float slope2 = BIAS && on ? slope_log2(a.mod, h * G + g) : 0.0f;
    const int n_x = tiles_of(x);
    float m = kNegBig, l = 0.0f, per_unit = 1.0f;  // O is in units of 1 / per_unit, a power of two
#pragma unroll 1
    for (int j = 0; j < 2 * n_x; ++j) {
      const int i = tile_of(x, j >> 1), first = kStep * (~j & 1);  // the tile, the step's first token in it
      const uint32_t t_s = t_x + kStep * (j & 1);
      if (!(j & 1)) wait(kBarScale + (i & 3), (uint32_t)((i >> 2) & 1));
      if (ok) wait(kBarS + 2 * x + (j & 1), (uint32_t)(j >> 1 & 1));
      if (!ok) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const float* scales = reinterpret_cast<const float*>(sm + kOffScale) + (i & 3) * 16 + (first >> 4);
      const float4 sk = *reinterpret_cast<const float4*>(scales), sv = *reinterpret_cast<const float4*>(scales + 8);
      const uint32_t pages = reinterpret_cast<const uint32_t*>(sm + kOffMask)[i & 3] >> (first >> 4) & 15u;
      // (a page that does not count has scores of -inf)
      const float f[4] = {pages & 1u ? sk.x * cq : 1.0f, pages & 2u ? sk.y * cq : 1.0f, pages & 4u ? sk.z * cq : 1.0f,
                          pages & 8u ? sk.w * cq : 1.0f};
      const float v[4] = {sv.x, sv.y, sv.z, sv.w};
      // P (fp16) over the back half of the products, 32 of which have been read when the
      // first 16 columns of P come there.  P is formed with the maximum and the unit so
      // far; only where the sums say that a p or an element of P may exceed 2^9 are these
      // themselves looked for
#pragma unroll
      for (int c = 1; c >= 0; --c) {
        float z[32];
        uint32_t pw[16];
        f32x2 sum;
        float vu[2];
        unpack2(mul2(pack2(v[2 * c], v[2 * c + 1]), pack2(per_unit, per_unit)), vu[0], vu[1]);
        // scores less the maximum -> P, and the unrounded sum
        auto probabilities = [&]() {
          f32x2 ls[2] = {0, 0};
          const f32x2 nm = pack2(-m, -m);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float* zz = z + 16 * e;
            const float fe = f[2 * c + e];
            const f32x2 f2 = pack2(fe, fe), v2 = pack2(vu[e], vu[e]);
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              const f32x2 zp = pack2(zz[k], zz[k + 1]);
              float y0, y1;
              unpack2(CAP || BIAS ? add2(zp, nm) : fma2(zp, f2, nm), y0, y1);
              const f32x2 p = pack2(fast_exp2(y0), fast_exp2(y1));
              ls[(k >> 1) & 1] = add2(ls[(k >> 1) & 1], p);
              unpack2(mul2(p, v2), y0, y1);
              pw[8 * e + (k >> 1)] = pack_half2(y0, y1);
            }
          }
          sum = add2(ls[0], ls[1]);
        };
        // products -> capped and biased scores (without either they stay products);
        // pages that do not count become -inf
        auto scores = [&]() {
          ld32(t_s + 32 * c, z);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float* zz = z + 16 * e;
            const float fe = f[2 * c + e];
            if (CAP) group_cap(a.mod, zz, fe, group_most(zz, 0.0f) * fe, 0.0f);
            if (BIAS) {
              const float d0 = (float)(dist - (t1 - 1 - i) * kTile - first - 32 * c - 16 * e);
              const f32x2 fz = CAP ? pack2(1.0f, 1.0f) : pack2(fe, fe), ns = pack2(-slope2, -slope2);
              f32x2 d = pack2(d0, d0 - 1.0f);
              const f32x2 two = pack2(-2.0f, -2.0f);
#pragma unroll
              for (int k = 0; k < 16; k += 2) {
                const f32x2 zp = pack2(zz[k], zz[k + 1]);
                unpack2(fma2(ns, d, CAP ? zp : mul2(zp, fz)), zz[k], zz[k + 1]);
                d = add2(d, two);
              }
            }
            if (pages != 15u && !((pages >> (2 * c + e)) & 1u)) {
#pragma unroll
              for (int k = 0; k < 16; ++k) zz[k] = -INFINITY;
            }
          }
        };
        scores();
        float lx, ly;
        bool ask = true;
        if (j > 0 || c == 0) {
          probabilities();
          unpack2(sum, lx, ly);
          // (a row's results do not depend on the others'; a unit that takes the V scale
          // beyond fp32 asks too)
          ask = !((lx + ly) * max3(vu[0], vu[1], 1.0f) <= kMostSum);
        }
        if (__any_sync(0xffffffffu, ask)) {
          if (j > 0 || c == 0) scores();  // (P has taken none of this chunk's products yet)
          float mx = -INFINITY, top = -INFINITY;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float y = group_max(z + 16 * e, -INFINITY) * (CAP || BIAS ? 1.0f : f[2 * c + e]);
            mx = fmaxf(mx, y);
            top = fmaxf(top, y + (float)exponent_of(v[2 * c + e]));
          }
          // the maximum rises by a whole number, so that what has been rounded is
          // scaled without a second rounding while it stays in fp16's normal range
          float alpha = 1.0f;
          if (ask && mx > -INFINITY) {
            const bool none = m <= kNegBig;
            const int unit = -exponent_of(per_unit), up = none || mx - m > 4096.0f ? 4096 : max((int)ceilf(mx - m), 0);
            m = up < 4096 ? m + (float)up : mx;
            const int to = min(max(none ? -126 : unit - up, (int)ceilf(fmaxf(top - m, -126.0f))), 126);
            const int by = none ? -4096 : unit - up - to;
            alpha = by >= -126 ? pow2i(by) : 0.0f;
            l *= up <= 126 ? pow2i(-up) : 0.0f;
            per_unit = pow2i(-to);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) vu[e] = fminf(v[2 * c + e] * per_unit, 0x1p127f);  // (beyond it p is 0)
          if (c == 0) {  // the other chunk's P
            uint32_t w[16];
            tmem_st_wait();
            ld16u(t_s + kStep * 3 / 4, w);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 y = unpack_half2(w[e]);
              w[e] = pack_half2(y.x * alpha, y.y * alpha);
            }
            tmem_st16(t_s + kStep * 3 / 4, w);
          }
          if (j > 0) {
            wait(kBarO + 2 * x + ((j - 1) & 1), (uint32_t)((j - 1) >> 1 & 1));  // the product before
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
          probabilities();
          unpack2(sum, lx, ly);
        }
        l += lx + ly;
        tmem_st16(t_s + kStep / 2 + 16 * c, pw);
      }
      if (!ok) break;
      tmem_st_wait();
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        bar_arrive(bar(kBarP + 2 * x + (j & 1)));
        if (j & 1) bar_arrive(bar(kBarScaleFree + (i & 3)));
      }
    }
    if (ok && n_x > 0) wait(kBarO + 2 * x + 1, (uint32_t)((n_x - 1) & 1));
    // through shared memory (32 rows of 512 bytes a warp, over the Q and K tiles; 16-byte
    // chunk e of row i at e ^ i), so that a warp stores whole rows.  Both streams read
    // the K tiles, and of up to 128 rows the Q tile: both must be through
    if (ok) wait(kBarDone + (x ^ 1), 0);
    uint8_t* box = sm + (row < kTile / 2 ? kOffQ : kOffK) + (row >> 5 & 1) * kBoxB;
    if (ok) {
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const float inv = l != 0.0f ? 1.0f / l : 0.0f;
      const float up = pow2i(-exponent_of(per_unit));
#pragma unroll 1
      for (int c0 = 0; c0 < kHeadDim; c0 += 32) {
        float o[32];
        if (n_x > 0) {
          ld32(t_o + c0, o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          *reinterpret_cast<float4*>(box + x * kTileB + lane * 512 + (((c0 + e) >> 2 ^ lane) << 4)) =
              make_float4(o[e] * inv * up, o[e + 1] * inv * up, o[e + 2] * inv * up, o[e + 3] * inv * up);
      }
    }
    float2* sh_ml = reinterpret_cast<float2*>(sm + kOffMl);  // [2 streams][128]
    sh_ml[x * kTile + row] = make_float2(m, l);
    if (single)
      asm volatile("bar.sync 1, %0;" ::"r"(32 * kSoftWarps) : "memory");
    else
      __syncwarp();
    if (ok && !*abort) {
      const int first = in_block & ~31;  // the warp's first row; the rows' places follow one another
      float* to = a.more_o + (((size_t)split * hkv + h) * rows_all + rb * kRows + first) * kHeadDim;
      float* to_ml = a.more_ml + (((size_t)split * hkv + h) * rows_all + rb * kRows + first) * 2;
      if (!single) {
#pragma unroll
        for (int i0 = 0; i0 < 32; i0 += 8) {
          float4 y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            y[i] = *reinterpret_cast<const float4*>(box + x * kTileB + (i0 + i) * 512 + ((lane ^ (i0 + i)) << 4));
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (first + i0 + i < rows) reinterpret_cast<float4*>(to + (size_t)(i0 + i) * kHeadDim)[lane] = y[i];
        }
        if (on) reinterpret_cast<float2*>(to_ml)[lane] = make_float2(m, l);
      } else {  // each stream stores every other row, joined
        const float2 ml = sh_ml[row], o = sh_ml[kTile + row];
        const float top = fmaxf(ml.x, o.x);
        float wy = fast_exp2(ml.x - top) * ml.y, wz = fast_exp2(o.x - top) * o.y;
        const float sum = wy + wz, inv = sum != 0.0f ? 1.0f / sum : 0.0f;
        if (on && x == 0) reinterpret_cast<float2*>(to_ml)[lane] = make_float2(top, sum);
        wy *= inv;
        wz *= inv;
#pragma unroll
        for (int i0 = x; i0 < 32; i0 += 8) {
          float4 y[4], z[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = i0 + 2 * i;
            y[i] = *reinterpret_cast<const float4*>(box + r * 512 + ((lane ^ r) << 4));
            z[i] = *reinterpret_cast<const float4*>(box + kTileB + r * 512 + ((lane ^ r) << 4));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float u = __shfl_sync(0xffffffffu, wy, i0 + 2 * i), w = __shfl_sync(0xffffffffu, wz, i0 + 2 * i);
            if (first + i0 + 2 * i < rows)
              reinterpret_cast<float4*>(to + (size_t)(i0 + 2 * i) * kHeadDim)[lane] =
                  make_float4(u * y[i].x + w * z[i].x, u * y[i].y + w * z[i].y, u * y[i].z + w * z[i].z,
                              u * y[i].w + w * z[i].w);
          }
        }
      }
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols));
}

template <bool FP8, bool CAP, bool BIAS>
cudaError_t launch_tc(const BlockState& s, int seq_begin, const uint16_t* q, const PrefixTc& a, cudaStream_t st) {
  static int done[64] = {0};
  const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(prefix_tc_kernel<FP8, CAP, BIAS>), kSmem, done);
  if (e != cudaSuccess) return e;
  const int row_blocks = (a.batch * s.group + kRows - 1) / kRows;
  prefix_tc_kernel<FP8, CAP, BIAS><<<row_blocks * a.splits * s.hkv, kThreads, kSmem, st>>>(s, seq_begin, q, a);
  return cudaGetLastError();
}

template <bool FP8>
cudaError_t launch_tc_mod(const BlockState& s, int seq_begin, const uint16_t* q, const PrefixTc& a, cudaStream_t st) {
  switch (block_mod(a.mod)) {
    case 0: return launch_tc<FP8, false, false>(s, seq_begin, q, a, st);
    case 1: return launch_tc<FP8, true, false>(s, seq_begin, q, a, st);
    case 2: return launch_tc<FP8, false, true>(s, seq_begin, q, a, st);
    default: return launch_tc<FP8, true, true>(s, seq_begin, q, a, st);
  }
}

}  // namespace

cudaError_t launch_prefix_tc(const BlockState& s, int seq_begin, const uint16_t* q, const PrefixTc& a,
                             cudaStream_t st) {
  return s.fp8 ? launch_tc_mod<true>(s, seq_begin, q, a, st) : launch_tc_mod<false>(s, seq_begin, q, a, st);
}

cudaError_t launch_block_prefix(const BlockState& s, int seq_begin, int batch, const uint16_t* q, uint16_t* out,
                                const BlockAttn& w, cudaStream_t st) {
  return attn_launch<kPrefix>(s, seq_begin, batch, q, out, w, st);
}

}  // namespace kvc
