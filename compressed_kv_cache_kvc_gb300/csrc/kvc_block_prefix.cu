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
// prefix_tc_kernel.  One 544-thread CTA per (up to 256 rows, KV head, run of
// 128-token tiles):
//   * warps 0-3 and 4-7: the softmax of one 128-row query tile each, a thread a row;
//   * warps 8-15: codes from global memory (the next tile's on their way in
//     registers) to fp16 in shared memory, K and V alike [128 tokens][128 dims] in
//     two boxes of 64 dims with the 128-byte swizzle; every code is exact in fp16;
//   * warp 16 issues the products: S = Q K^T (Q fp16 times a power of two per
//     row, which is exact for everything within 2^-28 of the row's largest value),
//     O += P V with P from tensor memory.
// TMEM columns: S_x at 128 x, O_x at 256 + 128 x; P (fp16) takes the front half of
// its S.  Per tile PV_0(i - 1), S_0(i), PV_1(i - 1), S_1(i): the pipe runs them in
// order, so S(i) may overwrite P(i - 1), and each query tile's softmax runs under the
// other's products.
// A block's K scale multiplies its scores, its V scale over the largest of the
// run (times 2^7) its probabilities, which so keep 11 bits down to 2^-21 of what
// the largest value would contribute at p = 1; O leaves times that scale.  The
// running maximum is lazy (O is rescaled when it grows by more than 8 in log2
// units: p <= 2^8, so P stays below 2^15), the sums add the unrounded p in fp32.
// Tiles go from the last to the first: with a distance bias the nearest come first.
// Synchronisation: mbarriers, every wait bounded, as in the prompt kernels.
#include "kvc_block_attn.h"
#include "kvc_tc.h"

namespace kvc {
namespace {

using namespace tc;

constexpr int kTile = 128;  // query rows and tokens per tile
constexpr int kRows = 2 * kTile;
constexpr int kSoftWarps = 16, kLoadWarps = 8;
constexpr int kMmaWarp = kSoftWarps + kLoadWarps, kScoutWarp = kMmaWarp + 1;
constexpr int kThreads = 32 * (kScoutWarp + 1);
constexpr int kTileB = kTile * kHeadDim * 2;  // 32 KB, two boxes of 64 dims
constexpr int kBoxB = kTileB / 2;
constexpr int kOffQ = 0, kOffK = kOffQ + 2 * kTileB, kOffV = kOffK + 2 * kTileB;
// a tile's K and V scales and which of its eight 16-token pages count, four tiles deep
// (a slot is written again when the tile four before is through its softmax)
constexpr int kOffScale = kOffV + 2 * kTileB;  // [4][2][8] f32
constexpr int kOffMask = kOffScale + 4 * 2 * 8 * 4;
constexpr int kOffBar = kOffMask + 4 * 4;
constexpr int kBarQ = 0, kBarK = 1, kBarV = 3, kBarKFree = 5, kBarVFree = 7, kBarS = 9, kBarP = 11, kBarO = 13,
              kBarScale = 15, kBarRead = 19, kBarDone = 27, kNumBars = 28;
constexpr int kOffMisc = kOffBar + 8 * kNumBars;  // TMEM base, abort flag, largest V scale
constexpr int kOffMax = kOffMisc + 16;            // [2][2 halves][256] what a row's two threads exchange
constexpr int kSmem = kOffMax + 4 * kRows * 4;
constexpr int kNbPair = 1;  // named barriers 1 .. 8 of the two warps that share 32 rows
constexpr float kLazyMax = 8.0f;
constexpr int kAhead = 4;  // tiles whose codes are on their way to L2
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
  uint32_t* sh_vmax = reinterpret_cast<uint32_t*>(sm + kOffMisc + 8);
  auto bar = [&](int i) { return base + kOffBar + 8 * i; };
  auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  int* status = s.counters + kCtrStatus;

  const int G = s.group, hkv = s.hkv, bt = s.bt, sh = __ffs(bt) - 1;
  const int rows_all = a.batch * G, row_blocks = (rows_all + kRows - 1) / kRows;
  const int rb = blockIdx.x % row_blocks, split = blockIdx.x / row_blocks % a.splits, h = blockIdx.x / row_blocks / a.splits;
  const int pre_len = s.seq_pos[a.prefix];
  const int n_tok = block_closed(pre_len, bt) << sh;
  const int tiles = (n_tok + kTile - 1) / kTile;
  const int t0 = (int)((long long)tiles * split / a.splits), t1 = (int)((long long)tiles * (split + 1) / a.splits);
  const int n_t = t1 - t0;  // tile i of the loops is t1 - 1 - i
  const int rows = min(rows_all - rb * kRows, kRows), nq = rows > kTile ? 2 : 1;
  const int32_t* table = s.table + (size_t)a.prefix * s.max_bps;
  launch_dependents();

  // this thread's row (softmax warps), and which half of a tile's tokens it has
  const int x = warp >> 3, half = (warp >> 2) & 1, row = tid & (kTile - 1);
  const int rr = rb * kRows + x * kTile + row;  // among the rows of the KV head
  const bool on = warp < kSoftWarps && x * kTile + row < rows;
  const int bl = on ? rr / G : 0, g = on ? rr % G : 0;
  const size_t part = (((size_t)split * hkv + h) * a.batch + bl) * G + g;
  if (n_t == 0) {  // (a graph replayed with a shorter prefix: nothing to add)
    if (on && half == 0) {
      for (int e = 0; e < kHeadDim / 4; ++e)
        reinterpret_cast<float4*>(a.more_o + part * kHeadDim)[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      *reinterpret_cast<float2*>(a.more_ml + part * 2) = make_float2(kNegBig, 0.0f);
    }
    return;
  }

  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tbase)), "r"(kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t count = 1;
      if (i == kBarQ) count = 8 * nq;
      if (i >= kBarK && i < kBarKFree) count = kLoadWarps;
      if (i >= kBarP && i < kBarO) count = 8;
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar(i)), "r"(count));
    }
    *abort = 0;
    *sh_vmax = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async();
  }
  __syncthreads();
  {  // the largest V scale of the run's blocks
    const int b0 = (t0 * kTile) >> sh, b1 = min(n_tok, t1 * kTile) >> sh;
    uint32_t most = 0;
    for (int i = b0 + tid; i < b1; i += kThreads) {
      const int id = table[i];
      if ((unsigned)id < (unsigned)s.num_blocks) most = max(most, __float_as_uint(s.v_scale[(size_t)id * hkv + h]));
    }
    most = __reduce_max_sync(0xffffffffu, most);  // (scales are not negative: their order is their bits')
    if (lane == 0 && most != 0) atomicMax(sh_vmax, most);
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = (uint32_t)uniform((int)*tbase);
  const float vmax = __uint_as_float(*sh_vmax);

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

  if (warp == kMmaWarp) {
    // -------------------------------------------------------------- products
    const bool el = elect_one();
    const uint32_t id_s = instr_desc(kTile, kTile, false), id_o = instr_desc(kTile, kHeadDim, false) | kInstrTransB;
    const uint64_t dq = op_desc_sw128(base + kOffQ), dk = op_desc_sw128(base + kOffK),
                   dv = op_desc_mn_sw128(base + kOffV, kBoxB);
    wait(kBarQ, 0);
    for (int i = 0; ok && i <= n_t; ++i) {
      if (i < n_t) wait(kBarK + (i & 1), (uint32_t)((i >> 1) & 1));
      if (ok && i > 0) wait(kBarV + ((i - 1) & 1), (uint32_t)(((i - 1) >> 1) & 1));
      if (!ok) break;
      for (int y = 0; y < nq; ++y) {
        const uint32_t t_s = tmem + kTile * y, t_o = tmem + 256 + kTile * y;
        if (i > 0) {
          wait(kBarP + y, (uint32_t)((i - 1) & 1));
          if (!ok) break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if (i > 0 && el) {
          const uint64_t d = dv + (uint64_t)((((i - 1) & 1) * kTileB) >> 4);
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks)
            mma_f16_ts(t_o, t_s + 8 * ks, d + (uint64_t)((ks * 2048) >> 4), id_o, i > 1 || ks > 0);
          mma_commit(bar(kBarO + y));
        }
        if (i < n_t && el) {
          const uint64_t d = dk + (uint64_t)(((i & 1) * kTileB) >> 4);
#pragma unroll
          for (int ks = 0; ks < kHeadDim / 16; ++ks)
            mma_f16(t_s, dq + (uint64_t)((y * kTileB + (ks >> 2) * kBoxB + (ks & 3) * 32) >> 4),
                    d + (uint64_t)(((ks >> 2) * kBoxB + (ks & 3) * 32) >> 4), id_s, ks > 0);
          mma_commit(bar(kBarS + y));
        }
        __syncwarp();
      }
      if (!ok) break;
      if (el) {
        if (i > 0) mma_commit(bar(kBarVFree + ((i - 1) & 1)));
        if (i < n_t) mma_commit(bar(kBarKFree + (i & 1)));
      }
      __syncwarp();
    }
    // every product complete before the tensor memory goes back
    if (el) mma_commit(bar(kBarDone));
    bar_wait(bar(kBarDone), 0, nullptr);
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
    float sc = scale_of(ids[0]);
#pragma unroll
    for (int e = 1; e < kAhead; ++e) fetch(e, ids[e]);
#pragma unroll 1
    for (int i = 0; i < n_t; ++i) {
      const int id = ids[0], next = id_of(i + kAhead + 1);
      fetch(i + kAhead, ids[kAhead]);
      const float sc_next = scale_of(ids[1]);
      if (i >= 2) wait(kBarKFree + (i & 1), (uint32_t)((i >> 1) & 1) ^ 1u);
      if (!ok) break;
      float* to = reinterpret_cast<float*>(sm + kOffScale) + (i & 3) * 16;
      if (lane < 8) to[lane] = sc;
      if (lane >= 8 && lane < 16) to[lane] = vmax > 0.0f ? __fdiv_rn(sc, vmax) * 128.0f : 0.0f;
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
  } else if (warp >= kSoftWarps) {
    // ----------------------------------------------------- codes -> fp16 tiles
    // a thread has 16 codes (column ch) of rows r0, r0 + 32, .. of K and of V
    const int pt = tid - 32 * kSoftWarps, r0 = pt >> 3, ch = pt & 7;
    const size_t head = (size_t)h * bt * kHeadDim + 16 * ch;
    const size_t stride = (size_t)hkv * bt * kHeadDim;
    auto load_ids = [&](int i, int (&id)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int tok = (t1 - 1 - i) * kTile + r0 + 32 * e;
        id[e] = i < n_t && tok < n_tok ? table[tok >> sh] : -1;
      }
    };
    auto load_codes = [&](const uint8_t* from, int i, const int (&id)[4], uint4 (&w)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int tok = (t1 - 1 - i) * kTile + r0 + 32 * e;
        w[e] = make_uint4(0u, 0u, 0u, 0u);  // (the code 0 in both formats)
        if ((unsigned)id[e] < (unsigned)s.num_blocks)
          w[e] = *reinterpret_cast<const uint4*>(from + id[e] * stride + head + (size_t)(tok & (bt - 1)) * kHeadDim);
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
    auto store = [&](uint8_t* tile, const uint4 (&w)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = r0 + 32 * e;
        uint4 y0, y1;
        to_halves(w[e].x, y0.x, y0.y);
        to_halves(w[e].y, y0.z, y0.w);
        to_halves(w[e].z, y1.x, y1.y);
        to_halves(w[e].w, y1.z, y1.w);
        // 16-byte chunks 2 (ch & 3) and the next of the row; the second box's lanes
        // write them in the other order (each bank once per 8 lanes)
        uint8_t* dst = tile + (ch >> 2) * kBoxB + r * 128;
        const int c0 = 2 * (ch & 3) + (ch >> 2), c1 = c0 ^ 1;
        *reinterpret_cast<uint4*>(dst + ((c0 ^ (r & 7)) << 4)) = ch >> 2 ? y1 : y0;
        *reinterpret_cast<uint4*>(dst + ((c1 ^ (r & 7)) << 4)) = ch >> 2 ? y0 : y1;
      }
      fence_async();
      __syncwarp();
    };
    int id[4], id_next[4];
    uint4 wk[4], wv[4];
    load_ids(0, id);
    load_codes(s.k_codes, 0, id, wk);
    load_codes(s.v_codes, 0, id, wv);
    load_ids(1, id_next);
    for (int i = 0; i < n_t; ++i) {
      if (i >= 2) wait(kBarKFree + (i & 1), (uint32_t)((i >> 1) & 1) ^ 1u);
      if (!ok) break;
      store(sm + kOffK + (i & 1) * kTileB, wk);
      if (lane == 0) bar_arrive(bar(kBarK + (i & 1)));
      load_codes(s.k_codes, i + 1, id_next, wk);
      if (i >= 2) wait(kBarVFree + (i & 1), (uint32_t)((i >> 1) & 1) ^ 1u);
      if (!ok) break;
      store(sm + kOffV + (i & 1) * kTileB, wv);
      if (lane == 0) bar_arrive(bar(kBarV + (i & 1)));
      load_codes(s.v_codes, i + 1, id_next, wv);
      load_ids(i + 2, id_next);
    }
  } else if (x < nq) {
    // ----------------------------------------------------------- query rows
    // the value of the row's other thread (two places in turn, so that one barrier
    // of the two warps is enough)
    float* sh_x = reinterpret_cast<float*>(sm + kOffMax) + x * kTile + row;
    const int pair = 4 * x + (warp & 3);
    int turn = 0;
    auto exchange = [&](float v) {
      sh_x[turn * 2 * kRows + half * kRows] = v;
      asm volatile("bar.sync %0, 64;" ::"r"(kNbPair + pair) : "memory");
      const float o = sh_x[turn * 2 * kRows + (half ^ 1) * kRows];
      turn ^= 1;
      return o;
    };
    float cq;
    int dist = 0;  // (BIAS) from the query to position 4 of the prefix
    {
      const uint16_t* src = q + ((size_t)bl * s.hq + h * G + g) * kHeadDim;
      if (BIAS && on) dist = pre_len + s.seq_pos[seq_begin + bl] - 1 - kSinks;
      float amax = 0.0f;
      uint4 mine[8];  // (the thread's half of the row)
#pragma unroll
      for (int c = 0; c < 8; ++c)
        mine[c] = on ? reinterpret_cast<const uint4*>(src)[8 * half + c] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint32_t y[4] = {mine[c].x, mine[c].y, mine[c].z, mine[c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = max3_abs(amax, bf16f(y[e] & 0xFFFFu), bf16f(y[e] >> 16));
      }
      amax = fmaxf(amax, exchange(amax));
      int e2 = 0;
      if (amax > 0.0f) e2 = min(max(14 - exponent_of(amax), -100), 100);
      const float up = pow2i(e2);
      cq = (CAP ? a.mod.y_scale : a.qk_scale_log2) * pow2i(-e2);
      uint8_t* dst = sm + kOffQ + x * kTileB + half * kBoxB + row * 128;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint32_t y[4] = {mine[c].x, mine[c].y, mine[c].z, mine[c].w};
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = pack_half2(bf16f(y[e] & 0xFFFFu) * up, bf16f(y[e] >> 16) * up);
        *reinterpret_cast<uint4*>(dst + ((c ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
      fence_async();
      __syncwarp();
      if (lane == 0) bar_arrive(bar(kBarQ));
    }
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_s = trow + kTile * x, t_o = trow + 256 + kTile * x + 64 * half;
    const float slope2 = BIAS && on ? slope_log2(a.mod, h * G + g) : 0.0f;
    float m = kNegBig, l = 0.0f;
#pragma unroll 1
    for (int i = 0; i < n_t; ++i) {
      wait(kBarScale + (i & 3), (uint32_t)((i >> 2) & 1));
      if (ok) wait(kBarS + x, (uint32_t)(i & 1));
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const float* sk = reinterpret_cast<const float*>(sm + kOffScale) + (i & 3) * 16 + 4 * half;
      const uint32_t pages = reinterpret_cast<const uint32_t*>(sm + kOffMask)[i & 3] >> (4 * half) & 15u;
      const int d0 = dist - (t1 - 1 - i) * kTile - 64 * half;  // distance to the half's first token
      float z[32];
      // the maximum: over the products (scales and a cap keep their order), with a
      // bias over the scores, which then take the products' place
      float mx = -INFINITY, most = 0.0f;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        ld32(t_s + 64 * half + 32 * c, z);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float* zz = z + 16 * e;
          const float f = sk[2 * c + e] * cq;
          const bool counts = (pages >> (2 * c + e)) & 1u;
          if (!BIAS) {
            if (counts) {
              mx = fmaxf(mx, group_max(zz, -INFINITY) * f);
              if (CAP) most = fmaxf(most, group_most(zz, 0.0f) * f);
            }
          } else {
            if (CAP) group_cap(a.mod, zz, f, group_most(zz, 0.0f) * f, 0.0f);
            const float fz = CAP ? 1.0f : f, first = (float)(d0 - 32 * c - 16 * e);
#pragma unroll
            for (int j = 0; j < 16; ++j) zz[j] = counts ? fmaf(-slope2, first - (float)j, zz[j] * fz) : -INFINITY;
            mx = group_max(zz, mx);
          }
        }
        if (BIAS) tmem_st32(t_s + 64 * half + 32 * c, z);
      }
      // (no maximum is a NaN: it says that a wait ran out, and both warps leave here)
      const float mine = ok ? mx : __int_as_float(0x7FFFFFFF), other = exchange(mine);
      ok = __all_sync(0xffffffffu, mine == mine && other == other);
      if (!ok) break;
      mx = fmaxf(mx, other);
      if (CAP && !BIAS && mx > -INFINITY) mx = cap_score(a.mod, mx);
      const bool grow = mx > m + kLazyMax;
      if (__any_sync(0xffffffffu, grow)) {
        const float m_old = m;
        if (grow) m = mx;
        const float alpha = fast_exp2(m_old - m);
        l *= alpha;
        if (i > 0) {
          wait(kBarO + x, (uint32_t)((i - 1) & 1));  // the product before
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll 1
          for (int c0 = 0; c0 < 64; c0 += 16) {
            float t[16];
            ld16(t_o + c0, t);
#pragma unroll
            for (int e = 0; e < 16; ++e) t[e] *= alpha;
            st16(t_o + c0, t);
          }
        }
      }
      // P (fp16) over the front of the products: the second half's goes where the
      // first half's products 32 .. 63 were, once these are read
      f32x2 ls[2] = {0, 0};
      if (BIAS) tmem_st_wait();
      const f32x2 nm = pack2(-m, -m);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t pw[16];
        ld32(t_s + 64 * half + 32 * c, z);
        if (half == 0 && c == 1) {
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();
          if (lane == 0) bar_arrive(bar(kBarRead + pair));
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float* zz = z + 16 * e;
          const float f = BIAS ? 1.0f : sk[2 * c + e] * cq, v = sk[8 + 2 * c + e];
          const f32x2 f2 = pack2(f, f), v2 = pack2(v, v);
          if (CAP && !BIAS) {
            group_cap(a.mod, zz, f, most, -m);
          } else {
#pragma unroll
            for (int j = 0; j < 16; j += 2) unpack2(fma2(pack2(zz[j], zz[j + 1]), f2, nm), zz[j], zz[j + 1]);
          }
          if (!BIAS && !((pages >> (2 * c + e)) & 1u)) {
#pragma unroll
            for (int j = 0; j < 16; ++j) zz[j] = -INFINITY;
          }
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            const f32x2 p = pack2(fast_exp2(zz[j]), fast_exp2(zz[j + 1]));
            ls[(j >> 1) & 1] = add2(ls[(j >> 1) & 1], p);
            float lo, hi;
            unpack2(mul2(p, v2), lo, hi);
            pw[8 * e + (j >> 1)] = pack_half2(lo, hi);
          }
        }
        if (half == 1 && c == 0) {
          wait(kBarRead + pair, (uint32_t)(i & 1));
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        }
        tmem_st16(t_s + 32 * half + 16 * c, pw);
      }
      float lx, ly;
      unpack2(add2(ls[0], ls[1]), lx, ly);
      l += lx + ly;
      tmem_st_wait();
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) bar_arrive(bar(kBarP + x));
    }
    if (ok) wait(kBarO + x, (uint32_t)((n_t - 1) & 1));
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const float l_other = exchange(l);
    l = half == 0 ? l + l_other : l_other + l;
    if (ok) {
      const float inv = l != 0.0f ? 1.0f / l : 0.0f, unit = vmax * 0x1p-7f;
      float* to = a.more_o + part * kHeadDim + 64 * half;
#pragma unroll 1
      for (int c0 = 0; c0 < 64; c0 += 32) {
        float o[32];
        ld32(t_o + c0, o);
        if (on) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(to + c0 + e) =
                make_float4(o[e] * inv * unit, o[e + 1] * inv * unit, o[e + 2] * inv * unit, o[e + 3] * inv * unit);
        }
      }
      if (on && half == 0) *reinterpret_cast<float2*>(a.more_ml + part * 2) = make_float2(m, l);
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
