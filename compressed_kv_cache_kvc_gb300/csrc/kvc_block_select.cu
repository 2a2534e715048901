// Attention to selected blocks of the block-scaled cache: a cheap score of every
// closed block, the choice of the best, the attention over them.
//
// The score estimates the largest dot product of the block's keys.  With q8 the INT8 codes
// of a query row (s = amax / 127, code = round-half-even(q / s), IEEE fp32), lo and
// hi the least and the largest INT8 code of a channel of the block's keys (scale
// t) and
//   I = sum over the channels of max(q8 lo, q8 hi)
//     = sum of min(q8, 0) lo + max(q8, 0) hi,
// the score is (I s) t, both products rounded to fp32, and a KV head's the largest
// of its query heads'.  I is at least the product of the query's codes with those of any
// key of the block; values, which the codes round, may have a larger product than the
// score.  |I| <= 127^2 128 < 2^24: I is exact, and so the scores are the same bits
// wherever they are computed, and the choice (ties to the lower block) is too.
//
// block_score_kernel: 260 bytes of bounds per block and KV head: 16 x 8 KV heads of up to
// 65,536 tokens in blocks of 32, 48 MB: 11.5 us, 4.2 TB/s, the integer matrix pipe 46 %
// busy (a group of 4 fills half of N).  Integer matrix instructions, 16 blocks on M, the group's query rows on N, 256 codes on K,
// fed from registers: four lanes a block, so that a load instruction takes 64 bytes of
// each of eight blocks (with dot products of four codes and the query rows in shared
// memory 17 us; all KV heads of a block in one CTA, 2 KB in a run, 22).
// block_choose_kernel: one CTA per (sequence, KV head): the top_blocks-th key, then the
// blocks in ascending order, and their places in the pool beside (128 pairs 6.3 us, 8
// pairs 5: barriers).  The attention over them runs block_attn_kernel's form kSelected.
// The second and the third are launched under the one before.
#include "kvc_block_attn.h"

namespace kvc {
namespace {

constexpr int kScoreThreads = 128, kScoreCtas = 6 * 152;
constexpr int kScoreStep = kScoreThreads / 32 * 16;  // blocks a CTA takes at once

// c += A (16 rows of 32 codes) x B (32 x 8): of lane l, a holds four codes of the
// rows l / 4 and l / 4 + 8 at two places, b of column l / 4 at the same two.
__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t order_key(float z) {  // NaN (never of finite inputs) lowest
  const uint32_t u = __float_as_uint(z + 0.0f);           // (-0 is 0)
  return z == z ? (u & 0x80000000u ? ~u : u | 0x80000000u) : 0u;
}

__global__ void __launch_bounds__(kScoreThreads) block_score_kernel(BlockState s, KeyBounds bounds, BlockChoice ch,
                                                                    int seq_begin, int chunks,
                                                                    const uint16_t* __restrict__ q) {
  __shared__ __align__(16) uint32_t sh_q[kMaxGroup][2][32];  // four codes a word: min(q8, 0), max(q8, 0)
  __shared__ float sh_s[kMaxGroup];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = s.group, hkv = s.hkv;
  const int pair = blockIdx.x / chunks, bl = pair / hkv, h = pair % hkv, b = seq_begin + bl;
  const int closed = block_closed(s.seq_pos[b], s.bt);
  const int n = closed - ch.recent;
  launch_dependents();
  if (closed <= ch.top + ch.recent) return;  // all are chosen
  // a warp's 16 blocks are the rows of A, the group's query rows the columns of B;
  // block ids are loaded two steps ahead, bounds one
  const int j = lane & 3, row = lane >> 2, step = chunks * kScoreStep;
  const int32_t* table = s.table + (size_t)b * s.max_bps;
  uint32_t* keys = ch.keys + (size_t)pair * s.max_bps;
  int c = (int)(blockIdx.x % chunks) * kScoreStep + warp * 16 + row;
  int blk[2], next[2];
  uint4 w[2][4];
  float t[2] = {0.0f, 0.0f};
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) w[r][i] = make_uint4(0u, 0u, 0u, 0u);
  auto ids = [&](int (&to)[2], int c) {
#pragma unroll
    for (int r = 0; r < 2; ++r) to[r] = c + 8 * r < n ? table[c + 8 * r] : -1;
  };
  auto load = [&] {
#pragma unroll
    for (int r = 0; r < 2; ++r)
      if ((unsigned)blk[r] < (unsigned)s.num_blocks) {
        const size_t at = (size_t)blk[r] * hkv + h;
        const uint4* src = reinterpret_cast<const uint4*>(bounds.codes + at * (2 * kHeadDim)) + j;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[r][i] = src[4 * i];
        t[r] = bounds.scale[at];
      }
  };
  ids(blk, c);
  ids(next, c + step);
  load();
  for (int g = warp; g < G; g += kScoreThreads / 32) {
    const uint2 v = reinterpret_cast<const uint2*>(q + ((size_t)bl * s.hq + h * G + g) * kHeadDim)[lane];
    const float x[4] = {bf16f(v.x & 0xFFFFu), bf16f(v.x >> 16), bf16f(v.y & 0xFFFFu), bf16f(v.y >> 16)};
    const float amax = warp_max(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))));
    const float scale = __fdiv_rn(amax, 127.0f);
    uint32_t neg = 0, pos = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int code = scale > 0.0f ? min(max(__float2int_rn(__fdiv_rn(x[e], scale)), -127), 127) : 0;
      neg |= (uint32_t)(min(code, 0) & 0xFF) << (8 * e);
      pos |= (uint32_t)max(code, 0) << (8 * e);
    }
    sh_q[g][0][lane] = neg;
    sh_q[g][1][lane] = pos;
    if (lane == 0) sh_s[g] = scale;
  }
  __syncthreads();
  uint4 y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    y[i] = row < G ? *reinterpret_cast<const uint4*>(&sh_q[row][i >> 1][4 * (j + 4 * (i & 1))])
                   : make_uint4(0u, 0u, 0u, 0u);
  const bool has[2] = {2 * j < G, 2 * j + 1 < G};
  const float scale[2] = {has[0] ? sh_s[2 * j] : 0.0f, has[1] ? sh_s[2 * j + 1] : 0.0f};
#pragma unroll 1
  for (; c - row < n; c += step) {  // (a warp's blocks all or none)
    int dot[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      mma_s8(dot, w[0][i].x, w[1][i].x, w[0][i].y, w[1][i].y, y[i].x, y[i].y);
      mma_s8(dot, w[0][i].z, w[1][i].z, w[0][i].w, w[1][i].w, y[i].z, y[i].w);
    }
    float best[2];
    bool ok[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      best[r] = -INFINITY;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (has[e]) best[r] = fmaxf(best[r], __fmul_rn(__fmul_rn((float)dot[2 * r + e], scale[e]), t[r]));
      ok[r] = (unsigned)blk[r] < (unsigned)s.num_blocks;
      blk[r] = next[r];
    }
    ids(next, c + 2 * step);
    load();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 1));
      best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 2));
      // (a bad block id is flagged by the attention)
      if (j == r && c + 8 * r < n) keys[c + 8 * r] = ok[r] ? order_key(best[r]) : 0u;
    }
  }
}

constexpr int kChooseThreads = 512;
constexpr int kChooseWarps = kChooseThreads / 32;
constexpr int kKeysHeld = 8;  // keys a thread holds
constexpr int kKeysStaged = kKeysHeld * kChooseThreads;
constexpr int kDigit = 9;  // bits of a digit: a bin per thread

struct ChooseShared {
  uint2 ends[kChooseWarps];
  int hist[2][kChooseThreads], sums[2][kChooseWarps], found[2][3];
};

// A limit for the `want` largest of n keys (0 < want < n), a thread's own
// (threadIdx.x + 512 k) in `own`: all keys above it are taken, and of those at it the
// *same first.  Radix select from the highest bit in which the keys differ (a head's
// scores are of one size: their first digits would all meet in a few bins), until the
// rest of the want is all of a bin.
__device__ uint32_t choose_limit(const uint32_t (&own)[kKeysHeld], int n, int want, ChooseShared& sh, int* same) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t lo = 0xffffffffu, hi = 0;
#pragma unroll
  for (int k = 0; k < kKeysHeld; ++k)
    if (tid + k * kChooseThreads < n) {
      lo = min(lo, own[k]);
      hi = max(hi, own[k]);
    }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) sh.ends[warp] = make_uint2(lo, hi);
  sh.hist[0][tid] = 0;
  __syncthreads();
  const uint2 e = sh.ends[lane & (kChooseWarps - 1)];
  lo = __reduce_min_sync(0xffffffffu, e.x);
  hi = __reduce_max_sync(0xffffffffu, e.y);
  int bits = 32 - __clz(lo ^ hi);  // below these all keys are as v
  uint32_t v = bits < 32 ? lo >> bits << bits : 0u;
  for (int round = 0; bits > 0; round ^= 1) {
    const int shift = max(bits - kDigit, 0);
    const uint32_t digit = (1u << (bits - shift)) - 1u, rest = bits < 32 ? 0xffffffffu << bits : 0u;
#pragma unroll
    for (int k = 0; k < kKeysHeld; ++k)
      if (tid + k * kChooseThreads < n && ((own[k] ^ v) & rest) == 0)
        atomicAdd(&sh.hist[round][own[k] >> shift & digit], 1);
    sh.hist[round ^ 1][tid] = 0;
    __syncthreads();
    const int bin = kChooseThreads - 1 - tid, count = sh.hist[round][bin];  // (from the largest on)
    int upto = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) sh.sums[round][warp] = upto;
    __syncthreads();
    upto += __reduce_add_sync(0xffffffffu, lane < warp ? sh.sums[round][lane] : 0);
    if (upto >= want && upto - count < want) {
      sh.found[round][0] = bin;
      sh.found[round][1] = want - (upto - count);
      sh.found[round][2] = count;
    }
    __syncthreads();
    v |= (uint32_t)sh.found[round][0] << shift;
    want = sh.found[round][1];
    bits = shift;
    if (want == sh.found[round][2] && v > 0) {
      *same = 0;
      return v - 1;
    }
  }
  *same = want;
  return v;
}

__global__ void __launch_bounds__(kChooseThreads) block_choose_kernel(BlockState s, BlockChoice ch, int seq_begin) {
  __shared__ uint32_t sh_keys[kKeysStaged];
  __shared__ int32_t sh_table[kKeysStaged];
  __shared__ ChooseShared sh;
  __shared__ int hist[kRadixBins], sh_warp[32], sh_sel[3], sh_more[kChooseWarps], sh_same[kChooseWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int pair = blockIdx.x, b = seq_begin + pair / s.hkv, most = ch.top + ch.recent;
  const int closed = block_closed(s.seq_pos[b], s.bt);
  int32_t* list = ch.list + (size_t)pair * ch.list_row;
  int32_t* ids = ch.ids + (size_t)pair * ch.ids_row;
  const int32_t* table = s.table + (size_t)b * s.max_bps;
  launch_dependents();
  for (int i = threadIdx.x; i < min(closed, kKeysStaged); i += kChooseThreads) sh_table[i] = table[i];
  wait_for_previous();  // the keys (and, for a list that stays, the call before)
  if (closed <= most) {
    for (int i = threadIdx.x; i < ch.list_row; i += kChooseThreads) {
      list[i] = i < closed ? i : -1;
      if (i < closed) ids[i] = table[i];
    }
    return;
  }
  const int n = closed - ch.recent;
  const uint32_t* keys = ch.keys + (size_t)pair * s.max_bps;
  const bool staged = n <= kKeysStaged;
  auto key = [&](int i) { return staged ? sh_keys[i] : __ldcg(keys + i); };
  int same_left;
  uint32_t limit;
  if (staged) {
    uint32_t own[kKeysHeld];
#pragma unroll
    for (int k = 0; k < kKeysHeld; ++k) {
      const int i = threadIdx.x + k * kChooseThreads;
      own[k] = i < n ? __ldcg(keys + i) : 0u;
      if (i < n) sh_keys[i] = own[k];
    }
    limit = choose_limit(own, n, ch.top, sh, &same_left);
  } else {
    int ties;
    limit = radix_select<kChooseThreads>(n, ch.top, true, [](int) { return true; }, key, hist, sh_warp, sh_sel,
                                         &same_left, &ties);
  }
  // a warp has a run of blocks: those above the limit, and at it
  const int run = ((n + kChooseWarps - 1) / kChooseWarps + 31) / 32 * 32;
  const int lo = min(warp * run, n), hi = min(lo + run, n);
  int more = 0, same = 0;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const uint32_t k = i0 + lane < hi ? key(i0 + lane) : 0u;
    more += __popc(__ballot_sync(0xffffffffu, i0 + lane < hi && k > limit));
    same += __popc(__ballot_sync(0xffffffffu, i0 + lane < hi && k == limit));
  }
  if (lane == 0) {
    sh_more[warp] = more;
    sh_same[warp] = same;
  }
  __syncthreads();
  more = same = 0;
  for (int i = 0; i < warp; ++i) {
    more += sh_more[i];
    same += sh_same[i];
  }
  const uint32_t below = (1u << lane) - 1u;
  auto put = [&](int at, int block) {
    list[at] = block;
    ids[at] = block < kKeysStaged ? sh_table[block] : table[block];
  };
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const uint32_t k = i0 + lane < hi ? key(i0 + lane) : 0u;
    const uint32_t up = __ballot_sync(0xffffffffu, i0 + lane < hi && k > limit);
    const uint32_t at = __ballot_sync(0xffffffffu, i0 + lane < hi && k == limit);
    // blocks at the limit are taken from the lowest on
    const int same_before = same + __popc(at & below);
    const bool take = ((up >> lane) & 1u) || (((at >> lane) & 1u) && same_before < same_left);
    if (take) put(more + __popc(up & below) + min(same_before, same_left), i0 + lane);
    more += __popc(up);
    same += __popc(at);
  }
  for (int i = threadIdx.x; i < ch.recent; i += kChooseThreads) put(ch.top + i, n + i);
}

}  // namespace

cudaError_t launch_block_choice(const BlockState& s, const KeyBounds& bounds, const BlockChoice& ch, int seq_begin,
                                int batch, int longest, const uint16_t* q, cudaStream_t st) {
  const int pairs = batch * s.hkv, n = block_closed(longest, s.bt) - ch.recent;
  const int steps = (n + kScoreStep - 1) / kScoreStep;
  // one wave of CTAs (a graph replayed at longer sequences takes more steps a CTA)
  const int chunks = std::max(1, std::min(steps, kScoreCtas / pairs));
  block_score_kernel<<<pairs * chunks, kScoreThreads, 0, st>>>(s, bounds, ch, seq_begin, chunks, q);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // may start under the scores (wait_for_previous)
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(pairs);
  cfg.blockDim = dim3(kChooseThreads);
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_choose_kernel, s, ch, seq_begin);
}

cudaError_t launch_block_selected(const BlockState& s, int seq_begin, int batch, const uint16_t* q, uint16_t* out,
                                  const BlockAttn& w, cudaStream_t st) {
  return attn_launch<kSelected>(s, seq_begin, batch, q, out, w, st);
}

}  // namespace kvc
