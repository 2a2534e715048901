// Attention to selected blocks of the block-scaled cache: a cheap score of every
// closed block, the choice of the best, the attention over them.
//
// The score bounds the block's dot products from above.  With q8 the INT8 codes
// of a query row (s = amax / 127, code = round-half-even(q / s), IEEE fp32), lo and
// hi the least and the largest INT8 code of a channel of the block's keys (scale
// t) and
//   I = sum over the channels of max(q8 lo, q8 hi)
//     = sum of min(q8, 0) lo + max(q8, 0) hi,
// the score is (I s) t, both products rounded to fp32, and a KV head's the largest
// of its query heads'.  |I| <= 127^2 128 < 2^24: I is exact, and so the scores are
// the same bits wherever they are computed, and the choice (ties to the lower
// block) is too.
//
// block_score_kernel: 256 bytes of bounds per block and KV head, integer dot
// products of four (dp4a); four lanes a block, so that a load instruction takes
// 64 bytes of each of eight blocks.  block_choose_kernel: one CTA per (sequence, KV
// head): radix select of the top_blocks-th key, then the blocks in ascending order.
#include "kvc_block_attn.h"

namespace kvc {
namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreStep = kScoreThreads / 4;  // blocks a CTA takes at once

__device__ __forceinline__ uint32_t order_key(float z) {  // NaN (never of finite inputs) lowest
  const uint32_t u = __float_as_uint(z + 0.0f);           // (-0 is 0)
  return z == z ? (u & 0x80000000u ? ~u : u | 0x80000000u) : 0u;
}

__global__ void __launch_bounds__(kScoreThreads) block_score_kernel(BlockState s, KeyBounds bounds, BlockChoice ch,
                                                                    int seq_begin, int chunks,
                                                                    const uint16_t* __restrict__ q) {
  __shared__ uint32_t sh_q[kMaxGroup][2][32];  // four codes a word: min(q8, 0), max(q8, 0)
  __shared__ float sh_s[kMaxGroup];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = s.group, hkv = s.hkv;
  const int pair = blockIdx.x / chunks, bl = pair / hkv, h = pair % hkv, b = seq_begin + bl;
  const int closed = block_closed(s.seq_pos[b], s.bt);
  const int n = closed - ch.recent;
  launch_dependents();
  if (closed <= ch.top + ch.recent) return;  // all are chosen
  if (warp < G) {
    const uint2 w = reinterpret_cast<const uint2*>(q + ((size_t)bl * s.hq + h * G + warp) * kHeadDim)[lane];
    const float x[4] = {bf16f(w.x & 0xFFFFu), bf16f(w.x >> 16), bf16f(w.y & 0xFFFFu), bf16f(w.y >> 16)};
    const float amax = warp_max(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))));
    const float scale = __fdiv_rn(amax, 127.0f);
    uint32_t neg = 0, pos = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = scale > 0.0f ? min(max(__float2int_rn(__fdiv_rn(x[e], scale)), -127), 127) : 0;
      neg |= (uint32_t)(min(c, 0) & 0xFF) << (8 * e);
      pos |= (uint32_t)max(c, 0) << (8 * e);
    }
    sh_q[warp][0][lane] = neg;
    sh_q[warp][1][lane] = pos;
    if (lane == 0) sh_s[warp] = scale;
  }
  __syncthreads();
  const int j = threadIdx.x & 3;
  const int32_t* table = s.table + (size_t)b * s.max_bps;
  uint32_t* keys = ch.keys + (size_t)pair * s.max_bps;
  for (int c0 = (int)(blockIdx.x % chunks) * kScoreStep; c0 < n; c0 += chunks * kScoreStep) {
    const int c = c0 + (threadIdx.x >> 2);
    const int blk = c < n ? table[c] : -1;
    uint4 w[4];
    float t = 0.0f;
    const bool ok = (unsigned)blk < (unsigned)s.num_blocks;
    if (ok) {
      const uint4* src = reinterpret_cast<const uint4*>(bounds.codes + ((size_t)blk * hkv + h) * (2 * kHeadDim)) + j;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = src[4 * i];
      t = bounds.scale[(size_t)blk * hkv + h];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    float best = -INFINITY;
    for (int g = 0; g < G; ++g) {
      int dot = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(&sh_q[g][i >> 1][4 * (j + 4 * (i & 1))]);
        dot = __dp4a((int)x.x, (int)w[i].x, dot);
        dot = __dp4a((int)x.y, (int)w[i].y, dot);
        dot = __dp4a((int)x.z, (int)w[i].z, dot);
        dot = __dp4a((int)x.w, (int)w[i].w, dot);
      }
      dot += __shfl_xor_sync(0xffffffffu, dot, 1);
      dot += __shfl_xor_sync(0xffffffffu, dot, 2);
      best = fmaxf(best, __fmul_rn(__fmul_rn((float)dot, sh_s[g]), t));
    }
    if (j == 0 && c < n) keys[c] = ok ? order_key(best) : 0u;  // (a bad block id is flagged by the attention)
  }
}

constexpr int kChooseThreads = 512;
constexpr int kChooseWarps = kChooseThreads / 32;
constexpr int kKeysStaged = 4096;

__global__ void __launch_bounds__(kChooseThreads) block_choose_kernel(BlockState s, BlockChoice ch, int seq_begin) {
  __shared__ uint32_t sh_keys[kKeysStaged];
  __shared__ int hist[kRadixBins], sh_warp[32], sh_sel[3], sh_more[kChooseWarps], sh_same[kChooseWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int pair = blockIdx.x, b = seq_begin + pair / s.hkv, most = ch.top + ch.recent;
  const int closed = block_closed(s.seq_pos[b], s.bt);
  int32_t* list = ch.list + (size_t)pair * most;
  launch_dependents();
  wait_for_previous();  // the keys (and, for a list that stays, the call before)
  if (closed <= most) {
    for (int i = threadIdx.x; i < most; i += kChooseThreads) list[i] = i < closed ? i : -1;
    return;
  }
  const int n = closed - ch.recent;
  const uint32_t* keys = ch.keys + (size_t)pair * s.max_bps;
  const bool staged = n <= kKeysStaged;
  if (staged) {
    for (int i = threadIdx.x; i < n; i += kChooseThreads) sh_keys[i] = __ldcg(keys + i);
    __syncthreads();
  }
  auto key = [&](int i) { return staged ? sh_keys[i] : __ldcg(keys + i); };
  int same_left, ties;
  const uint32_t limit = radix_select<kChooseThreads>(n, ch.top, true, [](int) { return true; }, key, hist, sh_warp, sh_sel,
                                                      &same_left, &ties);
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
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const uint32_t k = i0 + lane < hi ? key(i0 + lane) : 0u;
    const uint32_t up = __ballot_sync(0xffffffffu, i0 + lane < hi && k > limit);
    const uint32_t at = __ballot_sync(0xffffffffu, i0 + lane < hi && k == limit);
    // blocks at the limit are taken from the lowest on
    const int same_before = same + __popc(at & below);
    const bool take = ((up >> lane) & 1u) || (((at >> lane) & 1u) && same_before < same_left);
    if (take) list[more + __popc(up & below) + min(same_before, same_left)] = i0 + lane;
    more += __popc(up);
    same += __popc(at);
  }
  for (int i = threadIdx.x; i < ch.recent; i += kChooseThreads) list[ch.top + i] = n + i;
}

}  // namespace

cudaError_t launch_block_choice(const BlockState& s, const KeyBounds& bounds, const BlockChoice& ch, int seq_begin,
                                int batch, int longest, const uint16_t* q, cudaStream_t st) {
  const int pairs = batch * s.hkv, n = block_closed(longest, s.bt) - ch.recent;
  const int steps = (n + kScoreStep - 1) / kScoreStep;
  // (a graph replayed at longer sequences takes more steps a CTA)
  const int chunks = std::max(1, std::min(steps, (8 * 152 + pairs - 1) / pairs));
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
