// The single-query attention kernel over the block-scaled cache, instantiated by
// the translation units of its forms: a sequence whole (kvc_block.cu), its selected
// blocks (kvc_block_select.cu), a shared prefix and the sequence's own tokens
// (kvc_block_prefix.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "kvc_block.h"
#include "kvc_device.h"
#include "kvc_mma.h"

namespace kvc {
namespace {

using namespace dev;
using namespace codes;

__host__ __device__ constexpr int kExactRows(int bt) { return kSinks + bt; }

enum { kPlain = 0, kSelected = 1, kPrefix = 2 };  // forms

// ---------------------------------------------------------------- attention
// out = softmax(z) . v over everything a sequence holds, z as kvc_score.h says.
//
// Bound by DRAM: 256 bytes a token and KV head (16 sequences x 32 heads x 4,111
// INT8 tokens, capped: 91 us a call, 5.9 TB/s; one of 8 heads x 517: 8.6 us, latency).
// As in the per-token cache's kernel, one wave of CTAs shares the units of all
// (sequence, KV head) pairs end to end (each CTA an equal run, which may span
// pairs), the four warps of a CTA take a run's units in turn, and each warp streams
// 16-token pages
// through its own ring of four shared-memory stages with cp.async (a block of
// one head is one contiguous run, so a page is 2 KB of K and 2 KB of V).  The
// codes enter mma.sync m16n8k16 as fp16 (INT8 offset subnormals, E4M3 by the
// conversion instruction), 16 tokens on M and the G <= 8 query heads on N.
// What the scale per block changes: every page is full and has ONE K scale and
// ONE V scale, so a logit is acc * (k_scale * cq), the P V operand p *
// (v_scale 2^-E), the pages need no scale rows, and positions follow from the
// page index, so the distance bias reads nothing.
// The exact rows (sinks and open block, up to 3 + bt) are the pair's last
// units: tiles of 16 bf16 rows read straight into the MMA fragments, P as two
// bf16 parts (16 significant bits).
// V may be any finite value, also where blocks and exact rows differ by all of
// bf16's range: a head's accumulators are in units of 2^E, which follows the largest
// p V scale (of exact rows p |v| / 128) as the maxima follow the scores: V of
// any size and no weight costs the others no bits.  Partial results are divided by
// their sum before they leave units of 2^E, since the sum over a long sequence of
// values near the top of the range is beyond fp32.
// The CTA that finishes a pair last (an atomic ticket, no CTA waits) joins the
// pair's partials in CTA order, so the result does not depend on the order of
// completion.  (A warp per query head, eight rows of 16 bytes a lane in flight:
// joining a row at a time took 28.7 against 19.4 us for one sequence of 32,000
// tokens.)
//
// PARTS, for few sequences of unequal lengths: a CTA takes a part of one pair,
// the parts of a sequence in proportion to its length, so that no CTA ends
// inside a part.  Two CTAs per SM then, with the registers of two; the equal
// runs take a full wave of three (168 registers; at 216 and two per SM 16 x 32
// heads of 4,111 capped tokens 94 against 88 us).
//
// The forms of selected blocks and of a prefix always take parts, one CTA each: the
// pair follows from the CTA's number, nothing is summed over the sequences, and the
// exact rows go first, under the first pages' copies or the choice of the blocks (with
// the launches overlapped and the merge without bank conflicts 64 x 32 heads after a
// prefix of 32,768 tokens 119 -> 73 us, 16 x 32 heads of selected blocks 71 -> 60).
// 16 x 32 heads with 128 of 2,048 blocks of 32 tokens each: 31 us, 4.4 TB/s: blocks of
// 4 KB in no order, the round trips and joins that one sequence's 11 us are made of,
// and uneven CTAs (the busiest SM has 258 units, the mean is 217).  Two or three CTAs per
// SM and four or six pages of ring took the same, with that busiest SM in each.
// kPrefix joins the partials of the prefix's product with the pair's own.  Where the
// pair has one CTA a warp has up to 20 rows of them on their way under the merge of the
// warps, and nothing goes through memory (64 x 32 heads: 65.6 -> 61.4 us a call).
constexpr int kBWarps = 4;
constexpr int kBThreads = kBWarps * 32;
constexpr int kBStages = 4;
constexpr int kBStage = 4096;  // K page, V page
constexpr int kBSmem = kBWarps * kBStages * kBStage;
constexpr float kBLazy = 4.0f;
constexpr int kMergeRow = kHeadDim + 4;  // one warp's row of a head before the merge
constexpr int kJoinRow = kHeadDim + 4;  // one warp's joined row: 128 means, the maximum, the sum

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
constexpr int kBCap = 1, kBBias = 2;

// chunk j (16 bytes) of row t of a page: every copy and read instruction of
// the kernel touches each bank at most once per 128 bytes
__host__ __device__ constexpr int bchunk(int t, int j) {
  return 128 * t + 16 * (j ^ ((2 * ((t >> 2) & 3)) ^ (4 * ((t >> 1) & 1))));
}

template <int FORM, bool FP8, int MOD, bool PARTS>
__global__ void __launch_bounds__(kBThreads, PARTS ? 2 : 3) block_attn_kernel(BlockState s, int seq_begin, int batch,
                                                               const uint16_t* __restrict__ q,
                                                               uint16_t* __restrict__ out, BlockAttn a) {
  constexpr bool kCap = (MOD & kBCap) != 0, kBias = (MOD & kBBias) != 0;
  constexpr bool kOffset = !FP8;
  constexpr bool kDirect = FORM != kPlain;  // a CTA has one part of one pair
  constexpr float kOffK = 128.0f * 0x1p-24f, kOffV = 128.0f;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int cum[kDirect ? 1 : kMaxCallBatch + 1], len[kDirect ? 1 : kMaxCallBatch];
  // (split pairs) parts of a head of the sequences before
  __shared__ int parts[PARTS && !kDirect ? kMaxSplitBatch + 1 : 1];
  __shared__ int sh_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int bt = s.bt, ppb = bt / kPage;  // pages per block
  const int G = s.group, hkv = s.hkv;
  int bl = 0, h = 0, P = 0, part = 0;  // the pair, its sequence's length, the part
  if (kDirect) {
    part = blockIdx.x % a.parts;
    h = blockIdx.x / a.parts % hkv;
    bl = blockIdx.x / a.parts / hkv;
    P = s.seq_pos[seq_begin + bl];
  }
  // (kPrefix) tokens of the prefix; its pages and tiles of exact rows among the units
  const int pre_len = FORM == kPrefix ? s.seq_pos[a.prefix] : 0;
  const int pre_npg = FORM == kPrefix && a.prefix_pages ? block_closed(pre_len, bt) * ppb : 0;
  const int pre_tiles = FORM == kPrefix ? (block_exact_rows(pre_len, bt) + kPage - 1) / kPage : 0;
  // closed blocks among the units, and all units, of a sequence that holds n tokens
  auto blocks_of = [&](int n) { return FORM == kSelected ? min(block_closed(n, bt), a.most) : block_closed(n, bt); };
  auto units_of = [&](int n) {
    return pre_npg + pre_tiles + blocks_of(n) * ppb + (block_exact_rows(n, bt) + kPage - 1) / kPage;
  };
  if (!kDirect && warp == 0) {
    int carry = 0;
    if (lane == 0) cum[0] = 0;
    for (int base = 0; base < batch; base += 32) {
      const int i = base + lane;
      const int held = i < batch ? s.seq_pos[seq_begin + i] : 0;
      int v = i < batch ? units_of(held) : 0;
      if (i < batch) len[i] = held;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
      }
      if (i < batch) cum[i + 1] = carry + v;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
    if (PARTS) {
      // every sequence's share of the parts of a head, rounded down (but one at least)
      const long long per_head = a.parts, total = max(carry, 1);
      int before = 0;
      if (lane == 0) parts[0] = 0;
      for (int base = 0; base < batch; base += 32) {
        const int i = base + lane;
        const int nu = i < batch ? units_of(len[i]) : 0;
        int v = nu > 0 ? (int)max(1LL, min((long long)nu, nu * per_head / total)) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += y;
        }
        if (i < batch) parts[i + 1] = before + v;
        before += __shfl_sync(0xffffffffu, v, 31);
      }
    }
  }
  if (!kDirect) __syncthreads();

  const int r = lane >> 2, c = lane & 3;
  const int N = gridDim.x, cta = blockIdx.x;
  // this CTA's run of units [F, F1), or its parts F, F + N, .. of F1
  long long T = 0, F = 0, F1 = 1;
  int direct_nu = 0, direct_parts = 0;  // units of the pair and the parts they make
  const int* first = PARTS ? parts : cum;
  if (kDirect) {
    direct_nu = units_of(P);
    direct_parts = max(1, min(a.parts, direct_nu / a.part_units));
    if (direct_nu == 0 && part == 0) {  // (a replayed graph may find a sequence empty)
      uint4* rows = reinterpret_cast<uint4*>(out + ((size_t)bl * s.hq + h * G) * kHeadDim);
      if (threadIdx.x < G * (kHeadDim / 8)) rows[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
      wait_for_previous();  // (this kernel does not end before the one under which it runs)
    }
    if (direct_nu == 0 || part >= direct_parts) return;
  } else {
    T = (long long)hkv * cum[batch];
    for (int i = cta; i < batch; i += N)
      if (cum[i + 1] == cum[i])
        for (int e = threadIdx.x; e < s.hq * (kHeadDim / 8); e += kBThreads)
          reinterpret_cast<uint4*>(out + (size_t)i * s.hq * kHeadDim)[e] = make_uint4(0u, 0u, 0u, 0u);
    const PageRun run = PARTS ? PageRun{cta, (long long)hkv * parts[batch]} : cta_pages(cta, T, N);
    F = run.first;
    F1 = run.end;
  }
  const uint32_t ring_s = smem_u32(smem) + warp * kBStages * kBStage;
  const uint8_t* ring = smem + warp * kBStages * kBStage;
  uint32_t cp_d[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) cp_d[i] = bchunk((lane + 32 * i) >> 3, (lane + 32 * i) & 7);
  const int k_off[4] = {bchunk(2 * r, c), bchunk(2 * r, c + 4), bchunk(2 * r + 1, c), bchunk(2 * r + 1, c + 4)};
  int v_off[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) v_off[k] = 2048 + bchunk(4 * c + k, r);
  const uint64_t pol = l2_evict_first();
  const float qk = kCap ? a.mod.y_scale : a.qk_scale_log2;

  while (F < F1) {
    // ---- the pair of unit (or part) F and the units of it that are this CTA's
    int nu = direct_nu, per_pair = direct_parts;
    long long Pf = 0;
    if (!kDirect) {
      int lo = 0, hi = batch - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((long long)hkv * first[mid] <= F) lo = mid; else hi = mid - 1;
      }
      bl = lo;
      nu = cum[bl + 1] - cum[bl];
      const long long pbase = (long long)hkv * first[bl];
      per_pair = first[bl + 1] - first[bl];
      h = (int)((F - pbase) / per_pair);
      Pf = pbase + (long long)h * per_pair;
      part = (int)(F - Pf);
      P = len[bl];
    }
    const int b = seq_begin + bl;
    int u_a, u_e;  // units [u_a, u_e)
    if (PARTS || kDirect) {
      u_a = (int)((long long)nu * part / per_pair);
      u_e = (int)((long long)nu * (part + 1) / per_pair);
    } else {
      u_a = (int)(F - Pf);
      u_e = (int)((F1 < Pf + nu ? F1 : Pf + nu) - Pf);
    }
    const int closed = block_closed(P, bt), npg = pre_npg + blocks_of(P) * ppb;

    // ---- this warp's units u_a + warp, + kBWarps, ...: n_my, the first n_pg of them pages
    const int n_my = u_e - u_a > warp ? (u_e - u_a - warp + kBWarps - 1) / kBWarps : 0;
    const int n_pg = min(u_e, npg) - u_a > warp ? (min(u_e, npg) - u_a - warp + kBWarps - 1) / kBWarps : 0;
    const int32_t* table = s.table + (size_t)b * s.max_bps;
    const int32_t* list = FORM == kSelected ? a.list + ((size_t)bl * hkv + h) * a.list_row : nullptr;
    // block ids and scales of this warp's pages, 32 at a time across the lanes
    auto tab_load = [&](int chunk) -> int {
      const int k = chunk * 32 + lane, u = u_a + warp + kBWarps * k;
      if (k >= n_pg) return -1;
      if (FORM == kSelected) return a.ids[((size_t)bl * hkv + h) * a.ids_row + u / ppb];
      if (FORM == kPrefix)
        return u < pre_npg ? s.table[(size_t)a.prefix * s.max_bps + u / ppb] : table[(u - pre_npg) / ppb];
      return table[u / ppb];
    };
    // (selected, biased) the pages' blocks in the sequence
    constexpr bool kBlocks = FORM == kSelected && kBias;
    auto block_load = [&](int chunk) -> int {
      const int k = chunk * 32 + lane;
      return kBlocks && k < n_pg ? list[(u_a + warp + kBWarps * k) / ppb] : 0;
    };
    int blk_use = 0, blk_nxt = 0, id_cur = -1, id_nxt = -1;
    auto scale_of = [&](const float* sc, int id) {
      return (unsigned)id < (unsigned)s.num_blocks ? sc[(size_t)id * hkv + h] : 0.0f;
    };
    float ks_use = 0.0f, vs_use = 0.0f, ks_nxt = 0.0f, vs_nxt = 0.0f;
    uint32_t stage_ok = 0;
    const uint8_t* kb = s.k_codes + (size_t)h * bt * kHeadDim + 16 * lane;
    const uint8_t* vb = s.v_codes + (size_t)h * bt * kHeadDim + 16 * lane;
    const uint32_t stride = (uint32_t)hkv * bt * kHeadDim;
    auto issue = [&](int k) {
      if ((k & 31) == 0 && k > 0) {
        id_cur = id_nxt;
        id_nxt = tab_load((k >> 5) + 1);
      }
      const int id = __shfl_sync(0xffffffffu, id_cur, k & 31);
      const bool ok = k < n_pg && (unsigned)id < (unsigned)s.num_blocks;
      const int st = k & (kBStages - 1);
      stage_ok = (stage_ok & ~(1u << st)) | ((uint32_t)ok << st);
      if (ok) {
        const int sub = (u_a + warp + kBWarps * k) % ppb;
        const size_t off = (size_t)id * stride + (size_t)sub * (kPage * kHeadDim);
        const uint32_t sb = ring_s + st * kBStage;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;\n" ::"r"(sb + cp_d[i]),
                       "l"(kb + off + 512 * i), "l"(pol));
          asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;\n" ::"r"(sb + 2048 + cp_d[i]),
                       "l"(vb + off + 512 * i), "l"(pol));
        }
      }
      cp_async_commit();
    };
    auto first_pages = [&] {
      blk_use = block_load(0);
      id_cur = tab_load(0);
      if (n_pg > 32) {
        blk_nxt = block_load(1);
        id_nxt = tab_load(1);
      }
      ks_use = scale_of(s.k_scale, id_cur);
      vs_use = scale_of(s.v_scale, id_cur);
      ks_nxt = scale_of(s.k_scale, id_nxt);
      vs_nxt = scale_of(s.v_scale, id_nxt);
      issue(0);
      issue(1);
    };
    if (FORM != kSelected) first_pages();

    // ---- query fragments (B operand), scaled by 2^e into fp16 range
    uint32_t bq[8][2];
    float cq0, cq1, ch0 = 0.0f, ch1 = 0.0f;
    const uint16_t* qrow = q + ((size_t)bl * s.hq + h * G + (r < G ? r : 0)) * kHeadDim;
    {
      float qv[32];
      const uint4* src_a = reinterpret_cast<const uint4*>(qrow + 16 * c);
      const uint4* src_b = reinterpret_cast<const uint4*>(qrow + 64 + 16 * c);
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 u = i < 2 ? src_a[i] : src_b[i - 2];
        const uint32_t ws[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          qv[8 * i + 2 * j] = r < G ? bf16f(ws[j] & 0xFFFFu) : 0.0f;
          qv[8 * i + 2 * j + 1] = r < G ? bf16f(ws[j] >> 16) : 0.0f;
        }
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(qv[i]));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      int e = 0;
      if (amax > 0.0f) e = min(max(14 - exponent_of(amax), -100), 100);
      const float f2e = pow2i(e);
#pragma unroll
      for (int i = 0; i < 32; ++i) qv[i] *= f2e;
      float qs = 0.0f;
#pragma unroll
      for (int st = 0; st < 8; ++st) {
        // INT8 offset codes pair bytes (0, 2) and (1, 3) of a word, E4M3 (0, 1) and (2, 3)
        bq[st][0] = FP8 ? pack_half2(qv[4 * st], qv[4 * st + 1]) : pack_half2(qv[4 * st], qv[4 * st + 2]);
        bq[st][1] = FP8 ? pack_half2(qv[4 * st + 2], qv[4 * st + 3]) : pack_half2(qv[4 * st + 1], qv[4 * st + 3]);
        if (kOffset) {
          const float2 x = unpack_half2(bq[st][0]), y = unpack_half2(bq[st][1]);
          qs += (x.x + x.y) + (y.x + y.y);
        }
      }
      if (kOffset) {
        qs += __shfl_xor_sync(0xffffffffu, qs, 1);
        qs += __shfl_xor_sync(0xffffffffu, qs, 2);
        ch0 = kOffK * __shfl_sync(0xffffffffu, qs, 8 * c);
        ch1 = kOffK * __shfl_sync(0xffffffffu, qs, 8 * c + 4);
      }
      cq0 = qk * pow2i((kOffset ? 24 : 0) - __shfl_sync(0xffffffffu, e, 8 * c));
      cq1 = qk * pow2i((kOffset ? 24 : 0) - __shfl_sync(0xffffffffu, e, 8 * c + 4));
    }
    const float sl0 = kBias && 2 * c < G ? slope_log2(a.mod, h * G + 2 * c) : 0.0f;
    const float sl1 = kBias && 2 * c + 1 < G ? slope_log2(a.mod, h * G + 2 * c + 1) : 0.0f;

    float oacc[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) oacc[j][0] = oacc[j][1] = oacc[j][2] = oacc[j][3] = 0.0f;
    float osum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    float m0 = kNegBig, m1 = kNegBig, l0 = 0.0f, l1 = 0.0f;
    // the two heads' E (kNegBig: not set yet) and 2^-E, the largest V scale that leaves
    // the units as they are
    float E0 = kNegBig, E1 = kNegBig, inv2E0 = 1.0f, inv2E1 = 1.0f, sv_hi = 0.0f;

    // slots (2r, 2r + 1) x heads (2c, 2c + 1): cap and bias; slot 2r is at
    // distance d0 from the query
    auto transform = [&](float (&lg)[4], int d0) {
      if (kCap) cap_scores(a.mod, lg);
      if (kBias) {
        const float da = (float)d0, db = (float)(d0 - 1);
        lg[0] = fmaf(-sl0, da, lg[0]);
        lg[1] = fmaf(-sl1, da, lg[1]);
        lg[2] = fmaf(-sl0, db, lg[2]);
        lg[3] = fmaf(-sl1, db, lg[3]);
      }
    };
    // A head's E once its maximum has risen from m to nm, of V scales below 2^(ex + 1)
    // and products of exp2(score) and V scale below 2^(tw + 1): it stays while that fits
    // both the scales and the largest product so far, to 2^4; scales of no weight do not
    // raise it, and where the maximum leaves what set it behind it falls.
    auto next_unit = [&](float m, float nm, float tw, float ex, float E) {
      const float e = ex < E + 4.0f ? E : ex, top = fmaxf(m - nm + E, tw - nm);
      return fminf(fmaxf(top < e - 4.0f ? ceilf(top) : e, -126.0f), 126.0f);
    };
    // Exact rows' accumulators are in units of 2^E within 2^+-40: P carries the power
    // alone, V enters as it is, and neither leaves bf16's range, nor the products fp32's,
    // for any V.
    auto exact_unit = [](float E) { return fminf(fmaxf(E, -40.0f), 40.0f); };
    auto exact_power = [](float x) { return fminf(fmaxf(x, 0x1p-40f), 0x1p40f); };
    // the running maxima rise to cover tm0, tm1 and, if `units`, the units follow V
    // scales and products as in next_unit; O, the sums and l are rescaled
    auto rescale = [&](auto exact_tag, float tm0, float tm1, bool units, float tw0, float tw1, float ex) {
      constexpr bool kExact = decltype(exact_tag)::value;
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        tm0 = fmaxf(tm0, __shfl_xor_sync(0xffffffffu, tm0, o));
        tm1 = fmaxf(tm1, __shfl_xor_sync(0xffffffffu, tm1, o));
        if (units) {
          tw0 = fmaxf(tw0, __shfl_xor_sync(0xffffffffu, tw0, o));
          tw1 = fmaxf(tw1, __shfl_xor_sync(0xffffffffu, tw1, o));
        }
      }
      const float nm0 = fmaxf(m0, tm0), nm1 = fmaxf(m1, tm1);
      const float al0 = fast_exp2(m0 - nm0), al1 = fast_exp2(m1 - nm1);
      float f0 = al0, f1 = al1;
      if (units) {
        const float n0 = next_unit(m0, nm0, tw0, ex, E0), n1 = next_unit(m1, nm1, tw1, ex, E1);
        f0 = fast_exp2(m0 - nm0 + (kExact ? exact_unit(E0) - exact_unit(n0) : E0 - n0));
        f1 = fast_exp2(m1 - nm1 + (kExact ? exact_unit(E1) - exact_unit(n1) : E1 - n1));
        const int i0 = (int)n0, i1 = (int)n1;
        sv_hi = pow2i(min(min(i0, i1) + 4, 127));
        inv2E0 = pow2i(-i0);
        inv2E1 = pow2i(-i1);
        E0 = n0;
        E1 = n1;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        oacc[j][0] *= f0;
        oacc[j][2] *= f0;
        oacc[j][1] *= f1;
        oacc[j][3] *= f1;
      }
      osum[0] *= f0;
      osum[2] *= f0;
      osum[1] *= f1;
      osum[3] *= f1;
      l0 *= al0;
      l1 *= al1;
      m0 = nm0;
      m1 = nm1;
    };
    // the accumulators from the pages' units (2^24 more for offset codes) to the exact
    // rows' or back
    auto to_units = [&](bool exact) {
      constexpr float kCodes = kOffset ? 0x1p24f : 1.0f;
      // (2^E from 2^-E by their exponent fields)
      const float p0 = __int_as_float(0x7F000000 - __float_as_int(inv2E0));
      const float p1 = __int_as_float(0x7F000000 - __float_as_int(inv2E1));
      const float a0 = exact ? exact_power(inv2E0) * p0 : exact_power(p0) * inv2E0;
      const float a1 = exact ? exact_power(inv2E1) * p1 : exact_power(p1) * inv2E1;
      const float f0 = a0 * (exact ? kCodes : 1.0f / kCodes), f1 = a1 * (exact ? kCodes : 1.0f / kCodes);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        oacc[j][0] *= f0;
        oacc[j][2] *= f0;
        oacc[j][1] *= f1;
        oacc[j][3] *= f1;
      }
      if (kOffset && exact) {
        osum[0] *= a0;
        osum[1] *= a1;
      }
    };

    // the position of page k's first slot
    auto page_pos = [&](int k) {
      const int u = u_a + warp + kBWarps * k;
      if (kBlocks) return kSinks + __shfl_sync(0xffffffffu, blk_use, k & 31) * bt + u % ppb * kPage;
      if (FORM == kPrefix) return kSinks + (u < pre_npg ? u * kPage : pre_len + (u - pre_npg) * kPage);
      return kSinks + u * kPage;
    };
    // K and V scale of page k (called once per page, in order)
    auto scales_at = [&](int k, float& ks, float& vs) {
      if ((k & 31) == 0 && k > 0) {
        if (kBlocks) {
          blk_use = blk_nxt;
          blk_nxt = block_load((k >> 5) + 1);
        }
        ks_use = ks_nxt;
        vs_use = vs_nxt;
        const int id = tab_load((k >> 5) + 1);
        ks_nxt = scale_of(s.k_scale, id);
        vs_nxt = scale_of(s.v_scale, id);
      }
      ks = __shfl_sync(0xffffffffu, ks_use, k & 31);
      vs = __shfl_sync(0xffffffffu, vs_use, k & 31);
    };

    // NP consecutive pages of this warp, their instructions interleaved
    auto pages = [&](auto np_tag, int k) {
      constexpr int NP = decltype(np_tag)::value;
      const uint8_t* st[NP];
      float ks[NP], vs[NP];
#pragma unroll
      for (int pp = 0; pp < NP; ++pp) {
        st[pp] = ring + ((k + pp) & (kBStages - 1)) * kBStage;
        scales_at(k + pp, ks[pp], vs[pp]);
      }
      float acc[NP][4];
#pragma unroll
      for (int pp = 0; pp < NP; ++pp) {
        acc[pp][0] = acc[pp][2] = -ch0;
        acc[pp][1] = acc[pp][3] = -ch1;
      }
      {
        uint32_t w0[NP][8], w1[NP][8];
#pragma unroll
        for (int pp = 0; pp < NP; ++pp) {
          const uint4 x0 = *reinterpret_cast<const uint4*>(st[pp] + k_off[0]);
          const uint4 x1 = *reinterpret_cast<const uint4*>(st[pp] + k_off[1]);
          const uint4 x2 = *reinterpret_cast<const uint4*>(st[pp] + k_off[2]);
          const uint4 x3 = *reinterpret_cast<const uint4*>(st[pp] + k_off[3]);
          w0[pp][0] = x0.x; w0[pp][1] = x0.y; w0[pp][2] = x0.z; w0[pp][3] = x0.w;
          w0[pp][4] = x1.x; w0[pp][5] = x1.y; w0[pp][6] = x1.z; w0[pp][7] = x1.w;
          w1[pp][0] = x2.x; w1[pp][1] = x2.y; w1[pp][2] = x2.z; w1[pp][3] = x2.w;
          w1[pp][4] = x3.x; w1[pp][5] = x3.y; w1[pp][6] = x3.z; w1[pp][7] = x3.w;
        }
#pragma unroll
        for (int stp = 0; stp < 8; ++stp) {
#pragma unroll
          for (int pp = 0; pp < NP; ++pp) {
            uint32_t a0, a1, a2, a3;
            if (FP8) {
              e4m3x4_to_h2(w0[pp][stp], a0, a2);
              e4m3x4_to_h2(w1[pp][stp], a1, a3);
            } else {
              a0 = u8_even(w0[pp][stp]);
              a1 = u8_even(w1[pp][stp]);
              a2 = u8_even(w0[pp][stp] >> 8);
              a3 = u8_even(w1[pp][stp] >> 8);
            }
            mma16816(acc[pp], a0, a1, a2, a3, bq[stp][0], bq[stp][1]);
          }
        }
      }
      float tm0 = -INFINITY, tm1 = -INFINITY, svm = 0.0f;
#pragma unroll
      for (int pp = 0; pp < NP; ++pp) {
        const float f0 = ks[pp] * cq0, f1 = ks[pp] * cq1;
        acc[pp][0] *= f0;
        acc[pp][1] *= f1;
        acc[pp][2] *= f0;
        acc[pp][3] *= f1;
        transform(acc[pp], pre_len + P - 1 - (page_pos(k + pp) + 2 * r));
        tm0 = fmaxf(tm0, fmaxf(acc[pp][0], acc[pp][2]));
        tm1 = fmaxf(tm1, fmaxf(acc[pp][1], acc[pp][3]));
        svm = fmaxf(svm, vs[pp]);
      }
      if (__any_sync(0xffffffffu, tm0 > m0 + kBLazy || tm1 > m1 + kBLazy || svm > sv_hi)) {
        float tw0 = -INFINITY, tw1 = -INFINITY, least = INFINITY, ex = -INFINITY;
#pragma unroll
        for (int pp = 0; pp < NP; ++pp) {
          const float e = (float)exponent_of(vs[pp]);
          tw0 = fmaxf(tw0, fmaxf(acc[pp][0], acc[pp][2]) + e);
          tw1 = fmaxf(tw1, fmaxf(acc[pp][1], acc[pp][3]) + e);
          least = fminf(least, e);
          ex = fmaxf(ex, e);
        }
        // (whatever raises a maximum has a scale that keeps the unit, else)
        const bool units = __any_sync(0xffffffffu, svm > sv_hi || least < fmaxf(E0, E1) - 4.0f);
        rescale(std::false_type{}, tm0, tm1, units, tw0, tw1, ex);
      }
      uint32_t pb0[NP], pb1[NP];
#pragma unroll
      for (int pp = 0; pp < NP; ++pp) {
        // (beyond fp32 only where every p is 0)
        const float sn0 = fminf(vs[pp] * inv2E0, 0x1p127f), sn1 = fminf(vs[pp] * inv2E1, 0x1p127f);
        const float p0 = fast_exp2(acc[pp][0] - m0), p1 = fast_exp2(acc[pp][1] - m1);
        const float p2 = fast_exp2(acc[pp][2] - m0), p3 = fast_exp2(acc[pp][3] - m1);
        l0 += p0 + p2;
        l1 += p1 + p3;
        pb0[pp] = movmatrix_t(pack_half2(p0 * sn0, p1 * sn1));
        pb1[pp] = movmatrix_t(pack_half2(p2 * sn0, p3 * sn1));
      }
      // O^T += V_codes^T . P^T (rows: head dims 16r + 2j (+1), columns: query heads)
#pragma unroll
      for (int pp = 0; pp < NP; ++pp) {
        const uint4 r0 = *reinterpret_cast<const uint4*>(st[pp] + v_off[0]);
        const uint4 r1 = *reinterpret_cast<const uint4*>(st[pp] + v_off[1]);
        const uint4 r2 = *reinterpret_cast<const uint4*>(st[pp] + v_off[2]);
        const uint4 r3 = *reinterpret_cast<const uint4*>(st[pp] + v_off[3]);
        const uint32_t x0[4] = {r0.x, r0.y, r0.z, r0.w};
        const uint32_t x1[4] = {r1.x, r1.y, r1.z, r1.w};
        const uint32_t x2[4] = {r2.x, r2.y, r2.z, r2.w};
        const uint32_t x3[4] = {r3.x, r3.y, r3.z, r3.w};
#pragma unroll
        for (int wd = 0; wd < 4; ++wd) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t sa = (2 * half) | ((4 + 2 * half) << 8);
            const uint32_t sb = (2 * half + 1) | ((5 + 2 * half) << 8);
            uint32_t a0, a1, a2, a3;
            if (FP8) {
              a0 = e4m3_pair_to_h2(x0[wd], x2[wd], 2 * half);
              a1 = e4m3_pair_to_h2(x0[wd], x2[wd], 2 * half + 1);
              a2 = e4m3_pair_to_h2(x1[wd], x3[wd], 2 * half);
              a3 = e4m3_pair_to_h2(x1[wd], x3[wd], 2 * half + 1);
            } else {
              a0 = u8_even(prmt(x0[wd], x2[wd], sa));
              a1 = u8_even(prmt(x0[wd], x2[wd], sb));
              a2 = u8_even(prmt(x1[wd], x3[wd], sa));
              a3 = u8_even(prmt(x1[wd], x3[wd], sb));
            }
            mma16816(oacc[2 * wd + half], a0, a1, a2, a3, pb0[pp], pb1[pp]);
          }
        }
        if (kOffset) {
          constexpr uint32_t kOne = 0x3C003C00u;  // fp16 (1, 1)
          mma16816(osum, kOne, kOne, kOne, kOne, pb0[pp], pb1[pp]);
        }
      }
    };

    // ---- exact rows: tiles of 16 (mma.sync bf16; the lane's dims are 32c ..
    // 32c + 31 of its rows, in the order of Q and K alike)
    auto exact_tile = [&](int k) {
      // first exact row of the tile; (kPrefix) the prefix's tiles come before the sequence's
      const int tile = u_a + warp + kBWarps * k - npg;
      const bool shared = FORM == kPrefix && tile < pre_tiles;
      const int e0 = (FORM == kPrefix && !shared ? tile - pre_tiles : tile) * kPage;
      const int rows = block_exact_rows(shared ? pre_len : P, bt) - e0;
      const size_t eb = ((size_t)(shared ? a.prefix : b) * hkv + h) * kExactRows(bt) + e0;
      float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      // MMA rows r and r + 8 hold exact rows 2r and 2r + 1 (as the pages' slots)
      const bool on0 = 2 * r < rows, on1 = 2 * r + 1 < rows;
      const uint4* ka = reinterpret_cast<const uint4*>(s.k_exact + (eb + (on0 ? 2 * r : 0)) * kHeadDim + 32 * c);
      const uint4* kc = reinterpret_cast<const uint4*>(s.k_exact + (eb + (on1 ? 2 * r + 1 : 0)) * kHeadDim + 32 * c);
      // V rows 2r (first K half) and 2r + 1 (second) of the tile, dims 32c ..:
      // head dims 16r' + 2j and 16r' + 2j + 1 on the MMA's rows
      const uint4* va = reinterpret_cast<const uint4*>(s.v_exact + (eb + (on0 ? 2 * r : 0)) * kHeadDim + 32 * c);
      const uint4* vc = reinterpret_cast<const uint4*>(s.v_exact + (eb + (on1 ? 2 * r + 1 : 0)) * kHeadDim + 32 * c);
      uint32_t wa[16], wc[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4 x = va[i], y = vc[i];
        if (!on0) x = make_uint4(0u, 0u, 0u, 0u);
        if (!on1) y = make_uint4(0u, 0u, 0u, 0u);
        wa[4 * i] = x.x; wa[4 * i + 1] = x.y; wa[4 * i + 2] = x.z; wa[4 * i + 3] = x.w;
        wc[4 * i] = y.x; wc[4 * i + 1] = y.y; wc[4 * i + 2] = y.z; wc[4 * i + 3] = y.w;
      }
      const uint4* qp = reinterpret_cast<const uint4*>(qrow + 32 * c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 x = ka[i], y = kc[i];
        uint4 z = qp[i];
        if (r >= G) z = make_uint4(0u, 0u, 0u, 0u);
        mma16816_bf16(acc, x.x, y.x, x.y, y.y, z.x, z.y);
        mma16816_bf16(acc, x.z, y.z, x.w, y.w, z.z, z.w);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] *= qk;
      // position of exact row e: e itself (sinks), then the open block's
      if (kCap) cap_scores(a.mod, acc);
      if (kBias) {
        const int ea = e0 + 2 * r, ec = ea + 1;
        const int open = (shared ? block_closed(pre_len, bt) : closed) * bt;
        const int last = pre_len + P - 1 - (FORM == kPrefix && !shared ? pre_len : 0);
        const float da = (float)(last - (ea < kSinks ? ea : ea + open));
        const float dc = (float)(last - (ec < kSinks ? ec : ec + open));
        acc[0] = fmaf(-sl0, da, acc[0]);
        acc[1] = fmaf(-sl1, da, acc[1]);
        acc[2] = fmaf(-sl0, dc, acc[2]);
        acc[3] = fmaf(-sl1, dc, acc[3]);
      }
      if (!on0) acc[0] = acc[1] = -INFINITY;
      if (!on1) acc[2] = acc[3] = -INFINITY;
      // the largest magnitudes of the lane's two V rows
      __nv_bfloat162 va2 = __floats2bfloat162_rn(0.0f, 0.0f), vc2 = va2;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        va2 = __hmax2(va2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&wa[i])));
        vc2 = __hmax2(vc2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&wc[i])));
      }
      float sva = fmaxf(__low2float(va2), __high2float(va2)) * 0x1p-7f;
      float svc = fmaxf(__low2float(vc2), __high2float(vc2)) * 0x1p-7f;
      const float tm0 = fmaxf(acc[0], acc[2]), tm1 = fmaxf(acc[1], acc[3]);
      if (__any_sync(0xffffffffu, tm0 > m0 + kBLazy || tm1 > m1 + kBLazy || fmaxf(sva, svc) > sv_hi)) {
        // (four lanes have a row: a quarter of it is enough to say that it may not be small)
        int xa = exponent_of(sva), xc = exponent_of(svc);
        float ea = (float)xa, ec = (float)xc;
        const float lo = fmaxf(E0, E1) - 4.0f;
        const bool units =
            __any_sync(0xffffffffu, fmaxf(sva, svc) > sv_hi || (on0 && ea < lo) || (on1 && ec < lo));
        float ex = 0.0f;
        if (units) {
          ex = (float)__reduce_max_sync(0xffffffffu, max(xa, xc));
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) {
            ea = fmaxf(ea, __shfl_xor_sync(0xffffffffu, ea, o));
            ec = fmaxf(ec, __shfl_xor_sync(0xffffffffu, ec, o));
          }
        }
        rescale(std::true_type{}, tm0, tm1, units, fmaxf(acc[0] + ea, acc[2] + ec), fmaxf(acc[1] + ea, acc[3] + ec), ex);
      }
      const float p0 = fast_exp2(acc[0] - m0), p1 = fast_exp2(acc[1] - m1);
      const float p2 = fast_exp2(acc[2] - m0), p3 = fast_exp2(acc[3] - m1);
      l0 += p0 + p2;
      l1 += p1 + p3;
      const float unit0 = exact_power(inv2E0), unit1 = exact_power(inv2E1);
      uint32_t h0, h1, q0, q1;
      split_bf16x2(p0 * unit0, p1 * unit1, h0, q0);
      split_bf16x2(p2 * unit0, p3 * unit1, h1, q1);
      h0 = movmatrix_t(h0);
      h1 = movmatrix_t(h1);
      q0 = movmatrix_t(q0);
      q1 = movmatrix_t(q1);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t a0 = movmatrix_t(prmt(wa[j], wa[8 + j], 0x5410u)), a1 = movmatrix_t(prmt(wa[j], wa[8 + j], 0x7632u));
        const uint32_t a2 = movmatrix_t(prmt(wc[j], wc[8 + j], 0x5410u)), a3 = movmatrix_t(prmt(wc[j], wc[8 + j], 0x7632u));
        mma16816_bf16(oacc[j], a0, a1, a2, a3, h0, h1);
        mma16816_bf16(oacc[j], a0, a1, a2, a3, q0, q1);
      }
    };

    // the other forms' come before them, while the first pages are on their way
    // (kSelected: while they are chosen)
    if (kDirect) {
#pragma unroll 1
      for (int k = n_pg; k < n_my; ++k) exact_tile(k);
      if (0 < n_pg && n_pg < n_my) to_units(false);
    }
    if (FORM == kSelected) {
      wait_for_previous();
      first_pages();
    }

    int k = 0;
    // two pages an iteration, the copies of the next two in flight
#pragma unroll 1
    for (; k + 1 < n_pg; k += 2) {
      if (((stage_ok >> (k & (kBStages - 1))) & 3u) != 3u) break;  // a bad block id
      issue(k + 2);
      issue(k + 3);
      cp_async_wait<2>();
      __syncwarp();
      pages(std::integral_constant<int, 2>{}, k);
      __syncwarp();
    }
#pragma unroll 1
    for (; k < n_pg; ++k) {
      // pages k and k + 1 were issued; the rest one at a time
      cp_async_wait<1>();
      __syncwarp();
      if ((stage_ok >> (k & (kBStages - 1))) & 1u) {
        pages(std::integral_constant<int, 1>{}, k);
      } else {  // a bad block id: flagged and left out
        float ks, vs;
        scales_at(k, ks, vs);
        if (lane == 0) atomicOr(&s.counters[kCtrStatus], kDevBadBlockId);
      }
      __syncwarp();
      issue(k + 2);
    }
    cp_async_wait<0>();

    // the plain form's exact rows come after its pages
    if (!kDirect) {
      if (0 < n_pg && n_pg < n_my) to_units(true);
#pragma unroll 1
      for (; k < n_my; ++k) exact_tile(k);
    }

    // ---- per-warp totals, CTA merge of the warps
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
    __syncthreads();  // every warp is done with its ring: reuse shared memory
    float* sm_m = reinterpret_cast<float*>(smem);
    float* sm_l = sm_m + kBWarps * kMaxGroup;
    float* sm_o = sm_l + kBWarps * kMaxGroup;  // [kBWarps][8][kMergeRow]
    float* sm_e = sm_o + kBWarps * kMaxGroup * kMergeRow;
    const bool page_units = kDirect ? n_pg > 0 : n_pg == n_my;
    if (r == 0) {
      sm_e[warp * kMaxGroup + 2 * c] = page_units ? E0 : exact_unit(E0);
      sm_e[warp * kMaxGroup + 2 * c + 1] = page_units ? E1 : exact_unit(E1);
      sm_m[warp * kMaxGroup + 2 * c] = m0;
      sm_m[warp * kMaxGroup + 2 * c + 1] = m1;
      sm_l[warp * kMaxGroup + 2 * c] = l0;
      sm_l[warp * kMaxGroup + 2 * c + 1] = l1;
    }
    {
      const float sA = kOffset && page_units ? 0x1p24f : 1.0f;
      const float b0 = kOffset ? kOffV * osum[0] : 0.0f;
      const float b1 = kOffset ? kOffV * osum[1] : 0.0f;
      // dim 16 r + i of a head at 8 i + r, rows of 132: each bank once a store
      float* o0 = sm_o + ((size_t)warp * kMaxGroup + 2 * c) * kMergeRow + r;
      float* o1 = o0 + kMergeRow;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        o0[16 * j] = oacc[j][0] * sA - b0;
        o0[16 * j + 8] = oacc[j][2] * sA - b0;
        o1[16 * j] = oacc[j][1] * sA - b1;
        o1[16 * j + 8] = oacc[j][3] * sA - b1;
      }
    }
    // (kPrefix) partials of the prefix's blocks, joined with the pair's own.  Where the
    // pair has one CTA, a warp's first rows of them come under the merge of the warps
    const int more = FORM == kPrefix ? a.more : 0;
    constexpr int kFirstRows = FORM == kPrefix ? 20 : 1;
    const bool quick = FORM == kPrefix && more > 0 && more <= 32 && per_pair == 1;
    const size_t more_step = FORM == kPrefix ? (size_t)hkv * batch * G : 0;
    float2 more_ml = make_float2(kNegBig, 0.0f);
    float4 more_rows[kFirstRows];
    auto more_at = [&](int g) { return ((size_t)h * batch + bl) * G + g; };
    auto load_more = [&](int g, int i0) {
#pragma unroll
      for (int i = 0; i < kFirstRows; ++i) {  // past the end: the last part again, weight 0
        const float* from = a.more_o + (more_at(g) + min(i0 + i, more - 1) * more_step) * kHeadDim;
        more_rows[i] = __ldcg(reinterpret_cast<const float4*>(from) + lane);
      }
    };
    auto load_more_ml = [&](int g) {
      if (lane < more) more_ml = __ldcg(reinterpret_cast<const float2*>(a.more_ml) + more_at(g) + lane * more_step);
    };
    if (FORM == kPrefix && quick) {
      wait_for_previous();
      if (warp < G) {
        load_more_ml(warp);
        load_more(warp, 0);
      }
    }
    __syncthreads();
    // the pair's partials, the slot of this one and of the first (here, not above:
    // alive across the loops they cost 1 us of 90 for 16 x 32 heads of 4,111 tokens)
    const int i_first = PARTS || kDirect ? 0 : cta_of_page(Pf, T, N);
    const int cnt = PARTS || kDirect ? per_pair : cta_of_page(Pf + nu - 1, T, N) - i_first + 1;
    const long long pair = (long long)bl * hkv + h;
    const long long slot0 = kDirect ? pair * a.parts : PARTS ? Pf : pair + i_first;
    const long long slot = kDirect ? slot0 + part : PARTS ? F : pair + cta;
    const int d = threadIdx.x;  // 128 threads = head_dim
    uint16_t* orow = out + ((size_t)bl * s.hq + h * G) * kHeadDim + d;
    float* sm_own = sm_o + kBWarps * kMaxGroup * kMergeRow + kBWarps * kMaxGroup;  // (quick) [8][kMergeRow]: o, M, l
    // lane 4 g + w has warp w's weights of head g: exp2(m_w - M) for the sums, for O the
    // same times 2^(E_w - e), e the unit of the largest
    static_assert(kBWarps == 4 && kMaxGroup == 8, "a lane per warp and head");
    const int at_w = (lane & 3) * kMaxGroup + (lane >> 2);
    float M_g = sm_m[at_w], top_g = M_g + sm_e[at_w], l_g = 0.0f;
#pragma unroll
    for (int o = 1; o < kBWarps; o <<= 1) {
      M_g = fmaxf(M_g, __shfl_xor_sync(0xffffffffu, M_g, o));
      top_g = fmaxf(top_g, __shfl_xor_sync(0xffffffffu, top_g, o));
    }
    const float e_g = fminf(fmaxf(floorf(top_g - M_g), -126.0f), 126.0f), de = sm_e[at_w] - e_g;
    const float less = sm_m[at_w] - M_g, wt_l = fast_exp2(less), o_g = pow2i((int)e_g);
    const float wt_o = fabsf(de) < 64.0f ? wt_l * pow2i((int)de) : fast_exp2(less + de);
#pragma unroll
    for (int ww = 0; ww < kBWarps; ++ww)
      l_g = fmaf(__shfl_sync(0xffffffffu, wt_l, (lane & ~3) + ww), sm_l[ww * kMaxGroup + (lane >> 2)], l_g);
    for (int g = 0; g < G; ++g) {
      const float M = __shfl_sync(0xffffffffu, M_g, 4 * g), l = __shfl_sync(0xffffffffu, l_g, 4 * g);
      float o = 0.0f;
#pragma unroll
      for (int ww = 0; ww < kBWarps; ++ww)
        o = fmaf(__shfl_sync(0xffffffffu, wt_o, 4 * g + ww),
                 sm_o[((size_t)ww * kMaxGroup + g) * kMergeRow + 8 * (d & 15) + (d >> 4)], o);
      o = l != 0.0f ? o * (1.0f / l) * __shfl_sync(0xffffffffu, o_g, 4 * g) : 0.0f;
      if (FORM == kPrefix && quick) {
        sm_own[g * kMergeRow + d] = o;
        if (d == 0) {
          sm_own[g * kMergeRow + kHeadDim] = M;
          sm_own[g * kMergeRow + kHeadDim + 1] = l;
        }
      } else if (cnt + more == 1) {
        orow[(size_t)g * kHeadDim] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
      } else {
        const size_t ps = (size_t)slot * G + g;
        a.part_o[ps * kHeadDim + d] = o;
        if (d == 0) {
          a.part_ml[ps * 2] = M;
          a.part_ml[ps * 2 + 1] = l;
        }
      }
    }
    if (FORM == kPrefix && quick) {
      __syncthreads();
      for (int g = warp; g < G; g += kBWarps) {
        if (g != warp) {
          load_more_ml(g);
          load_more(g, 0);
        }
        const float* own = sm_own + g * kMergeRow;
        const float M = own[kHeadDim], top = fmaxf(M, warp_max(more_ml.x));
        float wt = lane < more ? fast_exp2(more_ml.x - top) * more_ml.y : 0.0f;
        float wo = fast_exp2(M - top) * own[kHeadDim + 1];
        const float sum = warp_sum(wt) + wo, inv = sum != 0.0f ? 1.0f / sum : 0.0f;
        wt *= inv;
        wo *= inv;
        float4 o = *reinterpret_cast<const float4*>(own + 4 * lane);
        o = make_float4(wo * o.x, wo * o.y, wo * o.z, wo * o.w);
        for (int i0 = 0; i0 < more; i0 += kFirstRows) {
          if (i0 > 0) load_more(g, i0);
#pragma unroll
          for (int i = 0; i < kFirstRows; ++i) {
            const float w = __shfl_sync(0xffffffffu, wt, (i0 + i) & 31);
            if (i0 + i < more) {
              o.x += w * more_rows[i].x; o.y += w * more_rows[i].y; o.z += w * more_rows[i].z; o.w += w * more_rows[i].w;
            }
          }
        }
        uint2 w;
        w.x = pack_bf16x2(o.x, o.y);
        w.y = pack_bf16x2(o.z, o.w);
        *reinterpret_cast<uint2*>(out + ((size_t)bl * s.hq + h * G + g) * kHeadDim + 4 * lane) = w;
      }
    } else if (cnt + more > 1) {
      // the pair's last CTA joins the partials, in CTA order
      __syncthreads();
      if (!kDirect || cnt > 1) {
        if (threadIdx.x == 0) {
          __threadfence();
          sh_last = atomicAdd(&s.tickets[b * hkv + h], 1) == cnt - 1;
          __threadfence();
        }
        __syncthreads();
      }
      if ((kDirect && cnt == 1) || sh_last) {
        if (FORM == kPrefix && more > 0) wait_for_previous();  // the prefix's partials
        // a warp per head (several when there are fewer heads than warps, each
        // with every wph-th part): 32 parts' maxima and sums across the lanes,
        // then their rows, eight of 16 bytes a lane in flight
        const int wph = G >= kBWarps ? 1 : kBWarps / G, share = warp % wph;
        const size_t base = (size_t)slot0 * G;
        float* sm_j = reinterpret_cast<float*>(smem);  // [kBWarps][kHeadDim + 2]
        for (int g = warp / wph; g < G; g += kBWarps / wph) {
          float M = kNegBig, l = 0.0f;
          float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + base + g;
          const float4* po = reinterpret_cast<const float4*>(a.part_o + (base + g) * kHeadDim) + lane;
          const int mine = (cnt + more - share + wph - 1) / wph;  // parts share + wph j
          // part i: the pair's own, then (kPrefix) those of the prefix
          const size_t more0 = more_at(g);
          auto part_ml = [&](int i) {
            if (FORM == kPrefix && i >= cnt)
              return __ldcg(reinterpret_cast<const float2*>(a.more_ml) + more0 + (i - cnt) * more_step);
            return __ldcg(ml + (size_t)i * G);
          };
          auto part_o = [&](int i) {
            if (FORM == kPrefix && i >= cnt)
              return __ldcg(reinterpret_cast<const float4*>(a.more_o + (more0 + (i - cnt) * more_step) * kHeadDim) +
                            lane);
            return __ldcg(po + (size_t)i * G * (kHeadDim / 4));
          };
          for (int j0 = 0; j0 < mine; j0 += 32) {
            const bool on = j0 + lane < mine;
            const float2 x = on ? part_ml(share + wph * (j0 + lane)) : make_float2(kNegBig, 0.0f);
            const float top = fmaxf(M, warp_max(x.x));
            // the mean so far and the parts' shares of the new one
            float al = l * fast_exp2(M - top), wt = on ? fast_exp2(x.x - top) * x.y : 0.0f;
            M = top;
            l = al + warp_sum(wt);
            const float inv = l != 0.0f ? 1.0f / l : 0.0f;
            al *= inv;
            wt *= inv;
            o.x *= al; o.y *= al; o.z *= al; o.w *= al;
            constexpr int kAtOnce = FORM == kPrefix ? 16 : 8;
            for (int i0 = 0; i0 < min(32, mine - j0); i0 += kAtOnce) {
              float4 y[kAtOnce];
#pragma unroll
              for (int i = 0; i < kAtOnce; ++i)  // past the end: the last part again, weight 0
                y[i] = part_o(share + wph * min(j0 + i0 + i, mine - 1));
#pragma unroll
              for (int i = 0; i < kAtOnce; ++i) {
                const float w = __shfl_sync(0xffffffffu, wt, i0 + i);
                if (j0 + i0 + i < mine) {
                  o.x += w * y[i].x; o.y += w * y[i].y; o.z += w * y[i].z; o.w += w * y[i].w;
                }
              }
            }
          }
          if (wph > 1) {  // (kBWarps >= wph G: every warp with a head comes here once)
            *reinterpret_cast<float4*>(sm_j + warp * kJoinRow + 4 * lane) = o;
            if (lane == 0) {
              sm_j[warp * kJoinRow + kHeadDim] = M;
              sm_j[warp * kJoinRow + kHeadDim + 1] = l;
            }
          } else {
            uint2 w;
            w.x = pack_bf16x2(o.x, o.y);
            w.y = pack_bf16x2(o.z, o.w);
            *reinterpret_cast<uint2*>(out + ((size_t)bl * s.hq + h * G + g) * kHeadDim + 4 * lane) = w;
          }
        }
        if (wph > 1) {
          __syncthreads();
          for (int g = 0; g < G; ++g) {
            const float* row = sm_j + g * wph * kJoinRow;
            float M = kNegBig, o = 0.0f, l = 0.0f;
            for (int i = 0; i < wph; ++i) M = fmaxf(M, row[i * kJoinRow + kHeadDim]);
            for (int i = 0; i < wph; ++i)
              l += fast_exp2(row[i * kJoinRow + kHeadDim] - M) * row[i * kJoinRow + kHeadDim + 1];
            const float inv = l != 0.0f ? 1.0f / l : 0.0f;
            for (int i = 0; i < wph; ++i)
              o += fast_exp2(row[i * kJoinRow + kHeadDim] - M) * row[i * kJoinRow + kHeadDim + 1] * inv *
                   row[i * kJoinRow + d];
            orow[(size_t)g * kHeadDim] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
          }
        }
        if (threadIdx.x == 0 && (!kDirect || cnt > 1)) s.tickets[b * hkv + h] = 0;
      }
    }
    __syncthreads();  // shared memory is reused by the next pair
    F = kDirect ? F1 : PARTS ? F + N : Pf + u_e;
  }
}

template <int FORM, bool FP8, int MOD, bool PARTS>
cudaError_t block_attn_smem() {
  static int done[64] = {0};
  return opt_in_smem(reinterpret_cast<const void*>(block_attn_kernel<FORM, FP8, MOD, PARTS>), kBSmem, done);
}

template <int FORM, bool FP8, int MOD>
int block_attn_ctas() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (dev < 64 && cached[dev] > 0) return cached[dev];
  int n = 0;
  if (block_attn_smem<FORM, FP8, MOD, false>() != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, block_attn_kernel<FORM, FP8, MOD, false>, kBThreads, kBSmem) !=
          cudaSuccess ||
      n < 1)
    n = 1;
  if (dev < 64) cached[dev] = n;
  return n;
}

int block_mod(const ScoreMod& m) { return (m.c2 > 0.0f ? kBCap : 0) | (m.slopes != nullptr ? kBBias : 0); }

template <int FORM, bool FP8, int MOD>
cudaError_t launch_block_attn_t(const BlockState& s, int seq_begin, int batch, const uint16_t* q, uint16_t* out,
                                const BlockAttn& w, cudaStream_t st) {
  if constexpr (FORM != kPlain) {
    const cudaError_t e = block_attn_smem<FORM, FP8, MOD, true>();
    if (e != cudaSuccess) return e;
    // may start under the kernel before it (wait_for_previous)
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(w.ncta);
    cfg.blockDim = dim3(kBThreads);
    cfg.dynamicSmemBytes = kBSmem;
    cfg.stream = st;
    cfg.attrs = &early;
    cfg.numAttrs = w.early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, block_attn_kernel<FORM, FP8, MOD, true>, s, seq_begin, batch, q, out, w);
  } else {
    const cudaError_t e = w.parts ? block_attn_smem<FORM, FP8, MOD, true>() : block_attn_smem<FORM, FP8, MOD, false>();
    if (e != cudaSuccess) return e;
    if (w.parts)
      block_attn_kernel<FORM, FP8, MOD, true><<<w.ncta, kBThreads, kBSmem, st>>>(s, seq_begin, batch, q, out, w);
    else
      block_attn_kernel<FORM, FP8, MOD, false><<<w.ncta, kBThreads, kBSmem, st>>>(s, seq_begin, batch, q, out, w);
    return cudaGetLastError();
  }
}

template <int FORM, bool FP8>
cudaError_t launch_block_attn_mod(const BlockState& s, int seq_begin, int batch, const uint16_t* q, uint16_t* out,
                                  const BlockAttn& w, cudaStream_t st) {
  switch (block_mod(w.mod)) {
    case 0: return launch_block_attn_t<FORM, FP8, 0>(s, seq_begin, batch, q, out, w, st);
    case 1: return launch_block_attn_t<FORM, FP8, 1>(s, seq_begin, batch, q, out, w, st);
    case 2: return launch_block_attn_t<FORM, FP8, 2>(s, seq_begin, batch, q, out, w, st);
    default: return launch_block_attn_t<FORM, FP8, 3>(s, seq_begin, batch, q, out, w, st);
  }
}

template <int FORM, bool FP8>
int block_attn_ctas_mod(int mod) {
  switch (mod) {
    case 0: return block_attn_ctas<FORM, FP8, 0>();
    case 1: return block_attn_ctas<FORM, FP8, 1>();
    case 2: return block_attn_ctas<FORM, FP8, 2>();
    default: return block_attn_ctas<FORM, FP8, 3>();
  }
}


template <int FORM>
int attn_ctas(const BlockState& s, const ScoreMod& mod) {
  return s.fp8 ? block_attn_ctas_mod<FORM, true>(block_mod(mod)) : block_attn_ctas_mod<FORM, false>(block_mod(mod));
}

template <int FORM>
cudaError_t attn_launch(const BlockState& s, int seq_begin, int batch, const uint16_t* q, uint16_t* out,
                        const BlockAttn& w, cudaStream_t st) {
  return s.fp8 ? launch_block_attn_mod<FORM, true>(s, seq_begin, batch, q, out, w, st)
               : launch_block_attn_mod<FORM, false>(s, seq_begin, batch, q, out, w, st);
}

}  // namespace
}  // namespace kvc
