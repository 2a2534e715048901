// The block-scaled cache: quantise-on-write by blocks, read-back, release, and
// the single-query attention over it.
//
// A block is `bt` (16 to 128) consecutive tokens of a sequence; per KV head its
// 128 bt K values share one scale, its V values another:
//   scale = max |x| / qmax, code = round-half-even(x / scale)  (IEEE fp32),
//   qmax 127 (INT8) or 448 (E4M3).
// Positions 0..3 and the open block stay in bf16 until the block's last token
// arrives, so no value is ever quantised twice.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "kvc_block_attn.h"
#include "kvc_quant.h"

namespace kvc {
namespace {

using namespace quant;

// ------------------------------------------------------------------- append
// One launch.  The work is tiles of 128 body rows (128 / bt blocks) of one
// (sequence, KV head, K or V), of which every resident CTA takes an equal run.
// A warp has 16 rows of a tile; its rows of the next tiles are on their way to
// shared memory (cp.async, each lane reads back what it copied itself), so the
// loads do not wait for the quantisation: first the block's maximum (bt / 16
// warps share one through a named barrier), then the codes.  Bound by DRAM: 2
// bytes read and 1 written a value; 16 sequences x 32 heads x 4,096 INT8 tokens
// in 276 us (5.8 TB/s; 411 us with a tile per CTA, its rows in registers, a
// division for eight values where one is near a border and the block geometry
// by integer division), E4M3 in 303.
//
// Every CTA derives the blocks its sequences take from the lengths alone (the
// free stack's top and an exclusive prefix of the blocks that the slice's
// earlier sequences complete), so no CTA waits for an allocation; the CTA that
// finishes last (an atomic ticket) advances the lengths and the stack.  A
// block's first rows may lie in the open block's buffer, which the rows left
// over after the last completed block overwrite: the CTA of a pair's first
// tile, the only one with rows of that buffer, writes the rows left over once
// the tile is in shared memory.
constexpr int kAppThreads = 256;
constexpr int kAppWarps = kAppThreads / 32;
constexpr int kAppRows = 16 * kAppWarps;
constexpr int kAppStages = 2;
constexpr int kAppCtas = 3;  // per SM; with three stages and two CTAs 299 us where this takes 276
constexpr int kAppStage = 16 * kHeadDim * 2 + 128;  // a warp's rows, and a lane's copy of the block's id
constexpr int kAppSmem = kAppWarps * kAppStages * kAppStage;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}

// What a form of the append has beside the plain one: the bounds of every block's keys.
struct AppendPlain {
  static constexpr bool kBounds = false;
};
struct AppendBounds {
  static constexpr bool kBounds = true;
  KeyBounds bounds;
};
template <bool FP8, class Form>
__global__ void __launch_bounds__(kAppThreads, kAppCtas) block_append_kernel(BlockState s, int seq_begin, int batch, int n_new,
                                                                      int tiles_per_pair,
                                                                      const uint16_t* __restrict__ kin,
                                                                      const uint16_t* __restrict__ vin,
                                                                      const __grid_constant__ Form f) {
  constexpr bool kBounds = Form::kBounds;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int before[kMaxCallBatch], held[kMaxCallBatch];  // blocks completed before it; its length
  __shared__ int sh_total, sh_bad, sh_last;
  __shared__ float sh_amax[2][kAppWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hkv = s.hkv, bt = s.bt;
  const int top = s.counters[kCtrFreeTop];
  if (warp == 0) {
    int total = 0, bad = 0;
    for (int base = 0; base < batch; base += 32) {
      const int i = base + lane;
      const int P = i < batch ? s.seq_pos[seq_begin + i] : 0;
      const int c1 = i < batch ? block_closed(P + n_new, bt) : 0, nb = i < batch ? c1 - block_closed(P, bt) : 0;
      bad |= c1 > s.max_bps;
      int v = nb;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
      }
      if (i < batch) {
        before[i] = total + v - nb;
        held[i] = P;
      }
      total += __shfl_sync(0xffffffffu, v, 31);
    }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      sh_total = total;
      sh_bad = (bad ? kDevTableOverflow : 0) | (total > top || top > s.num_blocks ? kDevOutOfBlocks : 0);
    }
  }
  __syncthreads();
  const bool ok = sh_bad == 0;  // the same for every CTA
  if (ok) {
    const long long T = 2LL * batch * hkv * tiles_per_pair;
    const long long t0 = (long long)blockIdx.x * T / gridDim.x;
    const int n_my = (int)((long long)(blockIdx.x + 1) * T / gridDim.x - t0);
    const int wpb = bt / 16, w0 = warp & ~(wpb - 1);  // warps per block, the block's first
    uint8_t* ring = smem + warp * kAppStages * kAppStage + 16 * lane;
    const uint8_t* ring_id = smem + warp * kAppStages * kAppStage + 16 * kHeadDim * 2 + 4 * lane;
    const uint32_t ring_s = smem_u32(ring), ring_id_s = smem_u32(ring_id);
    const size_t exact_rows = kExactRows(bt);

    const int sh = __ffs(bt) - 1;  // (bt is a power of two)
    auto closed_at = [&](int P) { return P > kSinks ? (P - kSinks) >> sh : 0; };

    // a tile: the x-th of sequence bl's K (kv = 0) or V of KV head h
    struct Tile {
      int bl, h, kv, x;
    };
    auto advance = [&](Tile& t) {
      if (++t.x == tiles_per_pair) {
        t.x = 0;
        t.kv ^= 1;
        if (t.kv == 0 && ++t.h == hkv) {
          t.h = 0;
          ++t.bl;
        }
      }
    };
    Tile cur;
    {
      const long long pair = t0 / tiles_per_pair;
      cur.x = (int)(t0 % tiles_per_pair);
      cur.kv = (int)(pair & 1);
      cur.h = (int)(pair / 2 % hkv);
      cur.bl = (int)(pair / 2 / hkv);
    }

    // the new rows of a (sequence, KV head)
    auto rows_in = [&](int kv, int bl, int h) { return (kv ? vin : kin) + ((size_t)bl * hkv + h) * n_new * kHeadDim; };

    // the copies of the CTA's next tile
    int i_next = 0, st_next = 0;
    Tile nxt = cur;
    auto issue = [&]() {
      if (i_next < n_my) {
        const int P = held[nxt.bl];
        const int c0 = closed_at(P), nb = closed_at(P + n_new) - c0;
        const long long row0 = (long long)nxt.x * kAppRows + warp * 16;
        if (row0 < (long long)nb << sh) {
          const size_t pair = (size_t)nxt.bl * hkv + nxt.h;
          const int p0 = kSinks + (c0 << sh) + (int)row0 + (lane >> 4);  // the lane's first row
          const uint16_t* in = rows_in(nxt.kv, nxt.bl, nxt.h) + (p0 - P) * (ptrdiff_t)kHeadDim + 8 * (lane & 15);
          if (nxt.x == 0) {  // may begin in the open block's rows
            const uint16_t* exact = (nxt.kv ? s.v_exact : s.k_exact) +
                                    (((size_t)seq_begin * hkv + pair) * exact_rows + kSinks) * kHeadDim + 8 * (lane & 15);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int p = p0 + 2 * i;
              cp_async16(ring_s + st_next * kAppStage + 512 * i,
                         p < P ? exact + (size_t)((p - kSinks) & (bt - 1)) * kHeadDim : in + 2 * i * kHeadDim);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) cp_async16(ring_s + st_next * kAppStage + 512 * i, in + 2 * i * kHeadDim);
          }
          cp_async4(ring_id_s + st_next * kAppStage, s.free_stack + (top - 1 - (before[nxt.bl] + ((int)row0 >> sh))));
        }
        ++i_next;
        st_next = st_next + 1 == kAppStages ? 0 : st_next + 1;
        advance(nxt);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kAppStages - 1; ++i) issue();

    int st = 0, flip = 0;
#pragma unroll 1
    for (int j = 0; j < n_my; ++j) {
      issue();
      cp_async_wait<kAppStages - 1>();
      __syncwarp();
      const int bl = cur.bl, h = cur.h, kv = cur.kv, b = seq_begin + bl, P = held[bl];
      const int c0 = closed_at(P), nb = closed_at(P + n_new) - c0;
      const long long row0 = (long long)cur.x * kAppRows + warp * 16;
      const bool live = row0 < (long long)nb << sh;
      const int c = live ? (int)row0 >> sh : 0;
      const uint8_t* rows = ring + st * kAppStage;
      float amax = 0.0f;
      // (a lane's eight channels, kBounds: the least of them in lanes 0 .. 15, the largest
      // in the others)
      uint4 ends = make_uint4(0u, 0u, 0u, 0u);
      if (live) {
        __nv_bfloat162 mx = __floats2bfloat162_rn(0.0f, 0.0f);
        if (kBounds && kv == 0) {
          __nv_bfloat162 least[4], most[4];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 w = *reinterpret_cast<const uint4*>(rows + 512 * i);
            const uint32_t y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&y[e]);
              least[e] = i == 0 ? x : __hmin2(least[e], x);
              most[e] = i == 0 ? x : __hmax2(most[e], x);
            }
          }
          uint32_t z[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 a = __shfl_xor_sync(0xffffffffu, least[e], 16);
            const __nv_bfloat162 b = __shfl_xor_sync(0xffffffffu, most[e], 16);
            const __nv_bfloat162 x = lane < 16 ? __hmin2(least[e], a) : __hmax2(most[e], b);
            mx = __hmax2(mx, __habs2(x));
            z[e] = *reinterpret_cast<const uint32_t*>(&x);
          }
          ends = make_uint4(z[0], z[1], z[2], z[3]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 w = *reinterpret_cast<const uint4*>(rows + 512 * i);
            const uint32_t y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) mx = __hmax2(mx, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&y[e])));
          }
        }
        amax = fmaxf(__low2float(mx), __high2float(mx));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (wpb > 1) {  // (a block's warps are all live or none)
          if (lane == 0) sh_amax[flip][warp] = amax;
          named_sync(1 + w0, 32 * wpb);
          for (int i = w0; i < w0 + wpb; ++i) amax = fmaxf(amax, sh_amax[flip][i]);
          flip ^= 1;  // the next maxima go beside these, which a slower warp may still read
        }
      }
      if (cur.x == 0) {
        // sinks, and the rows of the block that stays open, now that the first
        // block's rows are in shared memory
        __syncthreads();
        const uint16_t* in = rows_in(kv, bl, h);
        uint16_t* exact = (kv ? s.v_exact : s.k_exact) + ((size_t)b * hkv + h) * exact_rows * kHeadDim;
        const int open0 = kSinks + ((c0 + nb) << sh);
        const int n_sink = max(0, min(kSinks - P, n_new));
        const int first = min(max(open0 - P, n_sink), n_new);  // first new token of the open block
#pragma unroll 4
        for (int r = threadIdx.x >> 4; r < n_sink + (n_new - first); r += kAppThreads / 16) {
          const int i = r < n_sink ? r : first + (r - n_sink);
          const int p = P + i;
          const int row = p < kSinks ? p : kSinks + ((p - kSinks) & (bt - 1));
          reinterpret_cast<uint4*>(exact + (size_t)row * kHeadDim)[threadIdx.x & 15] =
              reinterpret_cast<const uint4*>(in + (size_t)i * kHeadDim)[threadIdx.x & 15];
        }
      }
      if (live) {
        const float scale = __fdiv_rn(amax, FP8 ? 448.0f : 127.0f);
        const float inv = rcp_approx_ftz(scale);
        const bool exact_div = !(scale >= 0x1p-126f && scale < INFINITY);
        const int blk = *reinterpret_cast<const int*>(ring_id + st * kAppStage);
        if ((unsigned)blk < (unsigned)s.num_blocks) {
          const size_t hblk = (size_t)blk * hkv + h;
          const int in_block = (int)row0 & (bt - 1);
          uint8_t* dst = (kv ? s.v_codes : s.k_codes) + ((hblk << sh) + in_block + (lane >> 4)) * kHeadDim +
                         8 * (lane & 15);
#pragma unroll 4
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint2*>(dst + 2 * i * kHeadDim) =
                block_codes8<FP8>(*reinterpret_cast<const uint4*>(rows + 512 * i), scale, inv, exact_div);
          if (in_block == 0 && lane == 0) {
            (kv ? s.v_scale : s.k_scale)[hblk] = scale;
            if (h == 0 && kv == 0) s.table[(size_t)b * s.max_bps + c0 + c] = blk;
          }
          if constexpr (kBounds) {
            if (kv == 0) {
              // the block's warps meet in the places of their rows, which they have read
              if (wpb > 1) {
                uint8_t* met = smem + st * kAppStage + 16 * lane;
                __syncwarp();
                *reinterpret_cast<uint4*>(met + warp * kAppStages * kAppStage) = ends;
                named_sync(1 + w0, 32 * wpb);
                if (warp == w0) {
                  uint32_t z[4] = {ends.x, ends.y, ends.z, ends.w};
                  for (int i = w0 + 1; i < w0 + wpb; ++i) {
                    const uint4 o = *reinterpret_cast<const uint4*>(met + i * kAppStages * kAppStage);
                    const uint32_t y[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                      const __nv_bfloat162 a = *reinterpret_cast<const __nv_bfloat162*>(&z[e]);
                      const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162*>(&y[e]);
                      const __nv_bfloat162 x = lane < 16 ? __hmin2(a, b) : __hmax2(a, b);
                      z[e] = *reinterpret_cast<const uint32_t*>(&x);
                    }
                  }
                  ends = make_uint4(z[0], z[1], z[2], z[3]);
                }
                named_sync(1 + w0, 32 * wpb);
              }
              if (warp == w0) {
                const float t = FP8 ? __fdiv_rn(amax, 127.0f) : scale;
                *reinterpret_cast<uint2*>(f.bounds.codes + hblk * (2 * kHeadDim) + 8 * lane) = block_codes8<false>(
                    ends, t, FP8 ? rcp_approx_ftz(t) : inv, !(t >= 0x1p-126f && t < INFINITY));
                if (lane == 0) f.bounds.scale[hblk] = t;
              }
            }
          }
        } else if (lane == 0) {
          atomicOr(&s.counters[kCtrStatus], kDevBadBlockId);
        }
      }
      st = st + 1 == kAppStages ? 0 : st + 1;
      advance(cur);
    }
    cp_async_wait<0>();
  }
  // the last CTA advances the lengths and the stack (every CTA has read them)
  __syncthreads();
  int32_t* ticket = s.tickets + s.max_batch * hkv;
  if (threadIdx.x == 0) {
    __threadfence();
    sh_last = atomicAdd(ticket, 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!sh_last) return;
  if (ok)
    for (int i = threadIdx.x; i < batch; i += kAppThreads) s.seq_pos[seq_begin + i] += n_new;
  if (threadIdx.x == 0) {
    *ticket = 0;
    if (ok)
      s.counters[kCtrFreeTop] = top - sh_total;
    else
      atomicOr(&s.counters[kCtrStatus], sh_bad);
  }
}

// ------------------------------------------------------------------ release
// One CTA per sequence; the places on the stack and the last step as in append.
__global__ void __launch_bounds__(128) block_release_kernel(BlockState s, int seq_begin, int batch) {
  __shared__ int sh_before, sh_total, sh_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int bl = blockIdx.x, b = seq_begin + bl;
  const int top = s.counters[kCtrFreeTop];
  if (warp == 0) {
    int before = 0, total = 0;
    for (int i = lane; i < batch; i += 32) {
      const int nb = min(block_closed(s.seq_pos[seq_begin + i], s.bt), s.max_bps);
      if (i < bl) before += nb;
      total += nb;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    total = __reduce_add_sync(0xffffffffu, total);
    if (lane == 0) {
      sh_before = before;
      sh_total = total;
    }
  }
  const int nb = min(block_closed(s.seq_pos[b], s.bt), s.max_bps);
  __syncthreads();
  const bool fits = top >= 0 && sh_total <= s.num_blocks - top;  // the same for every CTA
  const int32_t* row = s.table + (size_t)b * s.max_bps;
  if (fits)
    for (int j = threadIdx.x; j < nb; j += blockDim.x) s.free_stack[top + sh_before + j] = row[nb - 1 - j];
  int32_t* ticket = s.tickets + s.max_batch * s.hkv;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    sh_last = atomicAdd(ticket, 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!sh_last) return;
  for (int i = threadIdx.x; i < batch; i += blockDim.x) s.seq_pos[seq_begin + i] = 0;
  if (threadIdx.x == 0) {
    *ticket = 0;
    if (fits)
      s.counters[kCtrFreeTop] = top + sh_total;
    else
      atomicOr(&s.counters[kCtrStatus], kDevStackOverflow);
  }
}

__global__ void block_fill_kernel(int32_t* stack, int n) {
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) stack[i] = n - 1 - i;
}

// --------------------------------------------------------------------- read
// 8 lanes a row, 16 values a lane; a warp has 16 rows in flight.  Bound by
// DRAM: 1 byte read and 2 written a value; 16 x 32 x 4,096 tokens in 246 us
// (6.5 TB/s).
constexpr int kReadThreads = 256;
constexpr int kReadRows = 4;  // row groups of 4 per warp

template <bool FP8>
__device__ __forceinline__ uint32_t dequant2(uint32_t pair_src, int k, float scale) {
  // values 2k, 2k + 1 of the four codes in pair_src (k = 0, 1) as a bf16 pair
  float lo, hi;
  if (FP8) {
    uint32_t a, b2;
    e4m3x4_to_h2(pair_src, a, b2);
    const float2 f = unpack_half2(k == 0 ? a : b2);
    lo = f.x;
    hi = f.y;
  } else {
    // 2^23 + (code + 128) as an fp32 pattern, minus 2^23 + 128: exact
    const uint32_t u = pair_src ^ 0x80808080u;
    lo = __uint_as_float(__byte_perm(u, 0x4B000000u, k == 0 ? 0x7440 : 0x7442)) - 8388736.0f;
    hi = __uint_as_float(__byte_perm(u, 0x4B000000u, k == 0 ? 0x7441 : 0x7443)) - 8388736.0f;
  }
  return pack_bf16x2(lo * scale, hi * scale);
}

template <bool FP8>
__global__ void __launch_bounds__(kReadThreads) block_read_kernel(BlockState s, int seq_begin, int pos_begin, int n,
                                                                  uint16_t* __restrict__ ko,
                                                                  uint16_t* __restrict__ vo) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hkv = s.hkv, bt = s.bt;
  const int h = blockIdx.y >> 1, kv = blockIdx.y & 1, bl = blockIdx.z;
  const int b = seq_begin + bl;
  const int P = s.seq_pos[b], closed_end = kSinks + block_closed(P, bt) * bt;
  const uint16_t* exact = (kv ? s.v_exact : s.k_exact) + ((size_t)b * hkv + h) * kExactRows(bt) * kHeadDim;
  const uint8_t* codes8 = kv ? s.v_codes : s.k_codes;
  const float* scales = kv ? s.v_scale : s.k_scale;
  uint16_t* out = (kv ? vo : ko) + ((size_t)bl * hkv + h) * n * kHeadDim;
  const int r0 = (blockIdx.x * (kReadThreads / 32) + warp) * 4 * kReadRows + (lane >> 3);
  const int ch = lane & 7;
  uint4 w[kReadRows], w2[kReadRows];
  float sc[kReadRows];
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    const int r = r0 + 4 * i, p = pos_begin + r;
    sc[i] = -1.0f;  // nothing to write
    if (r >= n || p >= P) continue;
    if (p < kSinks || p >= closed_end) {
      const int row = p < kSinks ? p : kSinks + (p - kSinks) % bt;
      const uint4* src = reinterpret_cast<const uint4*>(exact + (size_t)row * kHeadDim) + 2 * ch;
      w[i] = src[0];
      w2[i] = src[1];
      sc[i] = -2.0f;  // exact
    } else {
      const int blk = s.table[(size_t)b * s.max_bps + (p - kSinks) / bt];
      if ((unsigned)blk < (unsigned)s.num_blocks) {
        const size_t hb = (size_t)blk * hkv + h;
        w[i] = reinterpret_cast<const uint4*>(codes8 + (hb * bt + (p - kSinks) % bt) * kHeadDim)[ch];
        sc[i] = scales[hb];
      } else if (ch == 0) {
        atomicOr(&s.counters[kCtrStatus], kDevBadBlockId);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    if (sc[i] == -1.0f) continue;
    uint4 a, c;
    if (sc[i] == -2.0f) {
      a = w[i];
      c = w2[i];
    } else {
      a = make_uint4(dequant2<FP8>(w[i].x, 0, sc[i]), dequant2<FP8>(w[i].x, 1, sc[i]), dequant2<FP8>(w[i].y, 0, sc[i]),
                     dequant2<FP8>(w[i].y, 1, sc[i]));
      c = make_uint4(dequant2<FP8>(w[i].z, 0, sc[i]), dequant2<FP8>(w[i].z, 1, sc[i]), dequant2<FP8>(w[i].w, 0, sc[i]),
                     dequant2<FP8>(w[i].w, 1, sc[i]));
    }
    uint4* dst = reinterpret_cast<uint4*>(out + (size_t)(r0 + 4 * i) * kHeadDim) + 2 * ch;
    dst[0] = a;
    dst[1] = c;
  }
}

template <bool FP8, class Form>
cudaError_t append_launch(const BlockState& s, int seq_begin, int batch, int n_new, const uint16_t* k,
                          const uint16_t* v, const Form& f, cudaStream_t st) {
  // rows of the most blocks an append of n_new tokens completes (at any state)
  const long long rows = ((long long)n_new + s.bt - 1) / s.bt * s.bt;
  const int tpp = (int)((rows + kAppRows - 1) / kAppRows);
  const long long tiles = 2LL * batch * s.hkv * tpp;
  static int done[64] = {0};
  const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(block_append_kernel<FP8, Form>), kAppSmem, done);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
    sms = 152;
  const int grid = (int)std::min(tiles, (long long)kAppCtas * sms);
  block_append_kernel<FP8, Form><<<grid, kAppThreads, kAppSmem, st>>>(s, seq_begin, batch, n_new, tpp, k, v, f);
  return cudaGetLastError();
}

template <class Form>
cudaError_t append_launch(const BlockState& s, int seq_begin, int batch, int n_new, const uint16_t* k,
                          const uint16_t* v, const Form& f, cudaStream_t st) {
  return s.fp8 ? append_launch<true>(s, seq_begin, batch, n_new, k, v, f, st)
               : append_launch<false>(s, seq_begin, batch, n_new, k, v, f, st);
}

}  // namespace

int block_attention_ctas_per_sm(const BlockState& s, const ScoreMod& mod) { return attn_ctas<kPlain>(s, mod); }

cudaError_t launch_block_attention(const BlockState& s, int seq_begin, int batch, const uint16_t* q, uint16_t* out,
                                   const BlockAttn& w, cudaStream_t st) {
  return attn_launch<kPlain>(s, seq_begin, batch, q, out, w, st);
}

cudaError_t launch_block_append(const BlockState& s, const KeyBounds& bounds, int seq_begin, int batch, int n_new,
                                const uint16_t* k, const uint16_t* v, cudaStream_t st) {
  return bounds.codes ? append_launch(s, seq_begin, batch, n_new, k, v, AppendBounds{bounds}, st)
                      : append_launch(s, seq_begin, batch, n_new, k, v, AppendPlain{}, st);
}

cudaError_t launch_block_release(const BlockState& s, int seq_begin, int batch, cudaStream_t st) {
  block_release_kernel<<<batch, 128, 0, st>>>(s, seq_begin, batch);
  return cudaGetLastError();
}

cudaError_t launch_block_read(const BlockState& s, int seq_begin, int batch, int pos_begin, int n, uint16_t* k,
                              uint16_t* v, cudaStream_t st) {
  constexpr int rows = kReadThreads / 32 * 4 * kReadRows;
  const dim3 grid((unsigned)(((long long)n + rows - 1) / rows), 2 * s.hkv, batch);
  if (s.fp8)
    block_read_kernel<true><<<grid, kReadThreads, 0, st>>>(s, seq_begin, pos_begin, n, k, v);
  else
    block_read_kernel<false><<<grid, kReadThreads, 0, st>>>(s, seq_begin, pos_begin, n, k, v);
  return cudaGetLastError();
}

cudaError_t launch_block_fill(const BlockState& s, cudaStream_t st) {
  block_fill_kernel<<<64, 256, 0, st>>>(s.free_stack, s.num_blocks);
  return cudaGetLastError();
}

}  // namespace kvc
