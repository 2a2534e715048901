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

#include "kvc_block.h"
#include "kvc_device.h"
#include "kvc_mma.h"
#include "kvc_quant.h"

namespace kvc {
namespace {

using namespace dev;
using namespace codes;
using namespace quant;

__host__ __device__ constexpr int kExactRows(int bt) { return kSinks + bt; }

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

// What a form of the append has beside the plain one: keys (and queries) rotated
// on the way, rows at strides; the bounds of every block's keys.
struct AppendPlain {
  static constexpr bool kRot = false, kBounds = false;
};
struct AppendBounds {
  static constexpr bool kRot = false, kBounds = true;
  KeyBounds bounds;
};
struct AppendRotary {
  static constexpr bool kRot = true, kBounds = false;
  RotaryArgs rot;  // q's rows, k's input; hk 0
  RowsIn v;
  int splits;
};
struct AppendRotaryBounds {
  static constexpr bool kRot = true, kBounds = true;
  RotaryArgs rot;
  RowsIn v;
  int splits;
  KeyBounds bounds;
};

template <bool FP8, class Form>
__global__ void __launch_bounds__(kAppThreads, kAppCtas) block_append_kernel(BlockState s, int seq_begin, int batch, int n_new,
                                                                      int tiles_per_pair,
                                                                      const uint16_t* __restrict__ kin,
                                                                      const uint16_t* __restrict__ vin,
                                                                      const __grid_constant__ Form f) {
  constexpr bool kRot = Form::kRot, kBounds = Form::kBounds;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int before[kMaxCallBatch], held[kMaxCallBatch];  // blocks completed before it; its length
  __shared__ int sh_total, sh_bad, sh_last;
  __shared__ float sh_amax[2][kAppWarps];
  __shared__ uint64_t sh_turns[kRot ? kRotPairs : 1];
  __shared__ uint8_t sh_axis[kRot ? kRotPairs : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hkv = s.hkv, bt = s.bt;
  const int top = s.counters[kCtrFreeTop];
  if constexpr (kRot) {
    if (threadIdx.x < kRotPairs) {
      sh_turns[threadIdx.x] = f.rot.table.turns[threadIdx.x];
      sh_axis[threadIdx.x] = f.rot.table.axis[threadIdx.x];
    }
  }
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

    // row i of the new tokens of a (sequence, KV head), values from one row to the next
    auto rows_in = [&](int kv, int bl, int h) -> const uint16_t* {
      if constexpr (kRot) {
        const RowsIn& r = kv ? f.v : f.rot.k;
        return r.in + bl * r.sb + h * r.sh;
      } else {
        return (kv ? vin : kin) + ((size_t)bl * hkv + h) * n_new * kHeadDim;
      }
    };
    auto step_in = [&](int kv) -> ptrdiff_t {
      if constexpr (kRot) return kv ? f.v.st : f.rot.k.st;
      return kHeadDim;
    };

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
          const ptrdiff_t step = step_in(nxt.kv);
          const uint16_t* in = rows_in(nxt.kv, nxt.bl, nxt.h) + (p0 - P) * step + 8 * (lane & 15);
          if (nxt.x == 0) {  // may begin in the open block's rows
            const uint16_t* exact = (nxt.kv ? s.v_exact : s.k_exact) +
                                    (((size_t)seq_begin * hkv + pair) * exact_rows + kSinks) * kHeadDim + 8 * (lane & 15);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int p = p0 + 2 * i;
              cp_async16(ring_s + st_next * kAppStage + 512 * i,
                         p < P ? exact + (size_t)((p - kSinks) & (bt - 1)) * kHeadDim : in + 2 * i * step);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) cp_async16(ring_s + st_next * kAppStage + 512 * i, in + 2 * i * step);
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
      if constexpr (kRot) {
        // new keys are turned where they lie (a row of the open block was when it came)
        if (kv == 0 && live) {
          const int cl = lane & 7;
          if (rotary::turns_here(f.rot.table, cl)) {
            const int p0 = kSinks + (c0 << sh) + (int)row0;
            uint8_t* mine = smem + warp * kAppStages * kAppStage + st * kAppStage;
            const int ca = 16 * rotary::chunk_a(f.rot.table, cl), cb = 16 * rotary::chunk_b(f.rot.table, cl);
#pragma unroll 1
            for (int r = lane >> 3; r < 16; r += 4) {
              const int p = p0 + r;
              if (p < P) continue;
              float cs[8], sn[8];
              rotary::angles(sh_turns, sh_axis,
                             rotary::row_pos(f.rot.table, (size_t)bl * n_new + (p - P), (size_t)batch * n_new, p), cl, cs,
                             sn);
              uint4* xa = reinterpret_cast<uint4*>(mine + 256 * r + ca);
              uint4* xb = reinterpret_cast<uint4*>(mine + 256 * r + cb);
              uint4 x = *xa, y = *xb;
              rotary::turn16(f.rot.table.adjacent != 0, x, y, cs, sn);
              *xa = x;
              *xb = y;
            }
          }
          __syncwarp();
        }
      }
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
        const ptrdiff_t step = step_in(kv);
        uint16_t* exact = (kv ? s.v_exact : s.k_exact) + ((size_t)b * hkv + h) * exact_rows * kHeadDim;
        const int open0 = kSinks + ((c0 + nb) << sh);
        const int n_sink = max(0, min(kSinks - P, n_new));
        const int first = min(max(open0 - P, n_sink), n_new);  // first new token of the open block
        auto new_token = [&](int r) { return r < n_sink ? r : first + (r - n_sink); };
        auto place = [&](int p) {
          return exact + (size_t)(p < kSinks ? p : kSinks + ((p - kSinks) & (bt - 1))) * kHeadDim;
        };
        if (kRot && kv == 0) {
          if constexpr (kRot) {
            const int cl = lane & 7;
            const int ca = 8 * rotary::chunk_a(f.rot.table, cl), cb = 8 * rotary::chunk_b(f.rot.table, cl);
#pragma unroll 1
            for (int r = threadIdx.x >> 3; r < n_sink + (n_new - first); r += kAppThreads / 8) {
              const int i = new_token(r);
              uint4 x = *reinterpret_cast<const uint4*>(in + i * step + ca);
              uint4 y = *reinterpret_cast<const uint4*>(in + i * step + cb);
              if (rotary::turns_here(f.rot.table, cl)) {
                float cs[8], sn[8];
                rotary::angles(
                    sh_turns, sh_axis,
                    rotary::row_pos(f.rot.table, (size_t)bl * n_new + i, (size_t)batch * n_new, P + i), cl, cs, sn);
                rotary::turn16(f.rot.table.adjacent != 0, x, y, cs, sn);
              }
              *reinterpret_cast<uint4*>(place(P + i) + ca) = x;
              *reinterpret_cast<uint4*>(place(P + i) + cb) = y;
            }
          }
        } else {
#pragma unroll 4
          for (int r = threadIdx.x >> 4; r < n_sink + (n_new - first); r += kAppThreads / 16) {
            const int i = new_token(r);
            reinterpret_cast<uint4*>(place(P + i))[threadIdx.x & 15] =
                reinterpret_cast<const uint4*>(in + i * step)[threadIdx.x & 15];
          }
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
    if constexpr (kRot) {
      if (f.rot.hq > 0) {
        const long long units = ((long long)batch * n_new + 3) / 4 * f.splits;
        for (long long u = (long long)blockIdx.x * kAppWarps + warp; u < units; u += (long long)gridDim.x * kAppWarps)
          rotary::rotate_unit(f.rot, sh_turns, sh_axis, u, f.splits, [&](int b) { return held[b]; });
      }
    }
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
// bf16's range: the accumulators are in units of 2^E, which follows the largest V
// scale (of exact rows 1/128 of the largest |v|) as the maxima follow the scores,
// and partial results are divided by their sum before they leave units of 2^E,
// since the sum over a long sequence of values near the top of the range is
// beyond fp32.
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
constexpr int kBWarps = 4;
constexpr int kBThreads = kBWarps * 32;
constexpr int kBStages = 4;
constexpr int kBStage = 4096;  // K page, V page
constexpr int kBSmem = kBWarps * kBStages * kBStage;
constexpr float kBLazy = 4.0f;
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

template <bool FP8, int MOD, bool PARTS>
__global__ void __launch_bounds__(kBThreads, PARTS ? 2 : 3) block_attn_kernel(BlockState s, int seq_begin, int batch,
                                                               const uint16_t* __restrict__ q,
                                                               uint16_t* __restrict__ out, BlockAttn a) {
  constexpr bool kCap = (MOD & kBCap) != 0, kBias = (MOD & kBBias) != 0;
  constexpr bool kOffset = !FP8;
  constexpr float kOffK = 128.0f * 0x1p-24f, kOffV = 128.0f;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int cum[kMaxCallBatch + 1], len[kMaxCallBatch];
  __shared__ int parts[PARTS ? kMaxSplitBatch + 1 : 1];  // (split pairs) parts of a head of the sequences before
  __shared__ int sh_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int bt = s.bt, ppb = bt / kPage;  // pages per block
  if (warp == 0) {
    int carry = 0;
    if (lane == 0) cum[0] = 0;
    for (int base = 0; base < batch; base += 32) {
      const int i = base + lane;
      const int held = i < batch ? s.seq_pos[seq_begin + i] : 0;
      int v = block_units(held, bt);
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
        const int nu = i < batch ? block_units(len[i], bt) : 0;
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
  __syncthreads();

  const int G = s.group, hkv = s.hkv;
  const int r = lane >> 2, c = lane & 3;
  const long long T = (long long)hkv * cum[batch];
  const int N = gridDim.x, cta = blockIdx.x;
  // (a replayed graph may find a sequence empty)
  for (int i = cta; i < batch; i += N)
    if (len[i] <= 0)
      for (int e = threadIdx.x; e < s.hq * (kHeadDim / 8); e += kBThreads)
        reinterpret_cast<uint4*>(out + (size_t)i * s.hq * kHeadDim)[e] = make_uint4(0u, 0u, 0u, 0u);
  // this CTA's run of units [F, F1), or its parts F, F + N, .. of F1
  const PageRun run = PARTS ? PageRun{cta, (long long)hkv * parts[batch]} : cta_pages(cta, T, N);
  long long F = run.first;
  const long long F1 = run.end;
  const int* first = PARTS ? parts : cum;
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
    int lo = 0, hi = batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((long long)hkv * first[mid] <= F) lo = mid; else hi = mid - 1;
    }
    const int bl = lo, b = seq_begin + bl;
    const int nu = cum[bl + 1] - cum[bl];
    const long long pbase = (long long)hkv * first[bl];
    const int per_pair = first[bl + 1] - first[bl];
    const int h = (int)((F - pbase) / per_pair);
    const long long Pf = pbase + (long long)h * per_pair;
    int u_a, u_e;  // units [u_a, u_e)
    if (PARTS) {
      const int part = (int)(F - Pf);
      u_a = (int)((long long)nu * part / per_pair);
      u_e = (int)((long long)nu * (part + 1) / per_pair);
    } else {
      u_a = (int)(F - Pf);
      u_e = (int)((F1 < Pf + nu ? F1 : Pf + nu) - Pf);
    }
    const int P = len[bl];
    const int closed = block_closed(P, bt), npg = closed * ppb;

    // ---- this warp's units u_a + warp, + kBWarps, ...: n_my, the first n_pg of them pages
    const int n_my = u_e - u_a > warp ? (u_e - u_a - warp + kBWarps - 1) / kBWarps : 0;
    const int n_pg = min(u_e, npg) - u_a > warp ? (min(u_e, npg) - u_a - warp + kBWarps - 1) / kBWarps : 0;
    const int32_t* table = s.table + (size_t)b * s.max_bps;
    // block ids and scales of this warp's pages, 32 at a time across the lanes
    auto tab_load = [&](int chunk) -> int {
      const int k = chunk * 32 + lane;
      return k < n_pg ? table[(u_a + warp + kBWarps * k) / ppb] : -1;
    };
    int id_cur = tab_load(0), id_nxt = n_pg > 32 ? tab_load(1) : -1;
    auto scale_of = [&](const float* sc, int id) {
      return (unsigned)id < (unsigned)s.num_blocks ? sc[(size_t)id * hkv + h] : 0.0f;
    };
    float ks_use = scale_of(s.k_scale, id_cur), vs_use = scale_of(s.v_scale, id_cur);
    float ks_nxt = scale_of(s.k_scale, id_nxt), vs_nxt = scale_of(s.v_scale, id_nxt);
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
    issue(0);
    issue(1);

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
    int E = 0;
    float sv_hi = 0.0f, inv2E = 1.0f;  // (0: E not set yet)

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
    // the running maxima rise to cover tm0, tm1 and the P V scale to cover a V
    // scale svm > 0 (0: unchanged); O, the sums and l are rescaled
    auto rescale = [&](float tm0, float tm1, float svm) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        tm0 = fmaxf(tm0, __shfl_xor_sync(0xffffffffu, tm0, o));
        tm1 = fmaxf(tm1, __shfl_xor_sync(0xffffffffu, tm1, o));
      }
      const float nm0 = fmaxf(m0, tm0), nm1 = fmaxf(m1, tm1);
      const float al0 = fast_exp2(m0 - nm0), al1 = fast_exp2(m1 - nm1);
      const bool rescale_e = svm > sv_hi;
      const int nE = rescale_e ? min(max(exponent_of(svm), -126), 126) : E;
      const int dE = E - nE;
      const float f = dE >= -126 ? pow2i(min(dE, 127)) : 0.0f;
      const float f0 = al0 * f, f1 = al1 * f;
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
      if (rescale_e) {
        E = nE;
        sv_hi = pow2i(min(E + 4, 127));
        inv2E = pow2i(-E);
      }
    };

    // K and V scale of page k (called once per page, in order)
    auto scales_at = [&](int k, float& ks, float& vs) {
      if ((k & 31) == 0 && k > 0) {
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
        transform(acc[pp], P - 1 - (kSinks + (u_a + warp + kBWarps * (k + pp)) * kPage + 2 * r));
        tm0 = fmaxf(tm0, fmaxf(acc[pp][0], acc[pp][2]));
        tm1 = fmaxf(tm1, fmaxf(acc[pp][1], acc[pp][3]));
        svm = fmaxf(svm, vs[pp]);
      }
      if (__any_sync(0xffffffffu, tm0 > m0 + kBLazy || tm1 > m1 + kBLazy || svm > sv_hi))
        rescale(tm0, tm1, svm);
      uint32_t pb0[NP], pb1[NP];
#pragma unroll
      for (int pp = 0; pp < NP; ++pp) {
        const float sn = vs[pp] * inv2E;
        const float p0 = fast_exp2(acc[pp][0] - m0), p1 = fast_exp2(acc[pp][1] - m1);
        const float p2 = fast_exp2(acc[pp][2] - m0), p3 = fast_exp2(acc[pp][3] - m1);
        l0 += p0 + p2;
        l1 += p1 + p3;
        pb0[pp] = movmatrix_t(pack_half2(p0 * sn, p1 * sn));
        pb1[pp] = movmatrix_t(pack_half2(p2 * sn, p3 * sn));
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

    // ---- exact rows: tiles of 16 (mma.sync bf16; the lane's dims are 32c ..
    // 32c + 31 of its rows, in the order of Q and K alike)
#pragma unroll 1
    for (; k < n_my; ++k) {
      const int e0 = (u_a + warp + kBWarps * k - npg) * kPage;  // first exact row of the tile
      const int rows = block_exact_rows(P, bt) - e0;
      const size_t eb = ((size_t)b * hkv + h) * kExactRows(bt) + e0;
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
        const float da = (float)(P - 1 - (ea < kSinks ? ea : ea + closed * bt));
        const float dc = (float)(P - 1 - (ec < kSinks ? ec : ec + closed * bt));
        acc[0] = fmaf(-sl0, da, acc[0]);
        acc[1] = fmaf(-sl1, da, acc[1]);
        acc[2] = fmaf(-sl0, dc, acc[2]);
        acc[3] = fmaf(-sl1, dc, acc[3]);
      }
      if (!on0) acc[0] = acc[1] = -INFINITY;
      if (!on1) acc[2] = acc[3] = -INFINITY;
      __nv_bfloat162 vm2 = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        vm2 = __hmax2(vm2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&wa[i])));
        vm2 = __hmax2(vm2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&wc[i])));
      }
      float svm = fmaxf(__low2float(vm2), __high2float(vm2)) * 0x1p-7f;
      const float tm0 = fmaxf(acc[0], acc[2]), tm1 = fmaxf(acc[1], acc[3]);
      if (__any_sync(0xffffffffu, tm0 > m0 + kBLazy || tm1 > m1 + kBLazy || svm > sv_hi)) {
        svm = warp_max(svm);
        rescale(tm0, tm1, svm);
      }
      const float p0 = fast_exp2(acc[0] - m0), p1 = fast_exp2(acc[1] - m1);
      const float p2 = fast_exp2(acc[2] - m0), p3 = fast_exp2(acc[3] - m1);
      l0 += p0 + p2;
      l1 += p1 + p3;
      // the P V operands in the accumulators' units (2^24 for offset codes, 2^E),
      // the power on both where it is large (V that leaves bf16's range by it is
      // nothing beside 2^E)
      const int eu = (kOffset ? 24 : 0) + E, ev = eu > 64 ? -64 : eu < -64 ? 64 : 0;
      if (ev != 0) {
        const __nv_bfloat162 f = __float2bfloat162_rn(pow2i(ev));
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&wa[i]), f);
          __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&wc[i]), f);
          wa[i] = *reinterpret_cast<const uint32_t*>(&x);
          wc[i] = *reinterpret_cast<const uint32_t*>(&y);
        }
      }
      const float unit = pow2i(-eu - ev);
      uint32_t h0, h1, q0, q1;
      split_bf16x2(p0 * unit, p1 * unit, h0, q0);
      split_bf16x2(p2 * unit, p3 * unit, h1, q1);
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
    float* sm_o = sm_l + kBWarps * kMaxGroup;  // [kBWarps][8][128]
    int* sm_e = reinterpret_cast<int*>(sm_o + kBWarps * kMaxGroup * kHeadDim);
    if (lane == 0) sm_e[warp] = E;
    if (r == 0) {
      sm_m[warp * kMaxGroup + 2 * c] = m0;
      sm_m[warp * kMaxGroup + 2 * c + 1] = m1;
      sm_l[warp * kMaxGroup + 2 * c] = l0;
      sm_l[warp * kMaxGroup + 2 * c + 1] = l1;
    }
    {
      const float sA = kOffset ? 0x1p24f : 1.0f;
      const float b0 = kOffset ? kOffV * osum[0] : 0.0f;
      const float b1 = kOffset ? kOffV * osum[1] : 0.0f;
      float* o0 = sm_o + ((size_t)warp * kMaxGroup + 2 * c) * kHeadDim + 16 * r;
      float* o1 = o0 + kHeadDim;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        o0[2 * j] = oacc[j][0] * sA - b0;
        o0[2 * j + 1] = oacc[j][2] * sA - b0;
        o1[2 * j] = oacc[j][1] * sA - b1;
        o1[2 * j + 1] = oacc[j][3] * sA - b1;
      }
    }
    __syncthreads();
    // the pair's partials, the slot of this one and of the first (here, not above:
    // alive across the loops they cost 1 us of 90 for 16 x 32 heads of 4,111 tokens)
    const int i_first = PARTS ? 0 : cta_of_page(Pf, T, N);
    const int cnt = PARTS ? per_pair : cta_of_page(Pf + nu - 1, T, N) - i_first + 1;
    const long long slot0 = PARTS ? Pf : (long long)bl * hkv + h + i_first;
    const long long slot = PARTS ? F : (long long)bl * hkv + h + cta;
    const int d = threadIdx.x;  // 128 threads = head_dim
    uint16_t* orow = out + ((size_t)bl * s.hq + h * G) * kHeadDim + d;
    int e_most = sm_e[0];
#pragma unroll
    for (int ww = 1; ww < kBWarps; ++ww) e_most = max(e_most, sm_e[ww]);
    for (int g = 0; g < G; ++g) {
      float M = kNegBig;
#pragma unroll
      for (int ww = 0; ww < kBWarps; ++ww) M = fmaxf(M, sm_m[ww * kMaxGroup + g]);
      float o = 0.0f, l = 0.0f;
#pragma unroll
      for (int ww = 0; ww < kBWarps; ++ww) {
        const float wt = fast_exp2(sm_m[ww * kMaxGroup + g] - M);
        o += wt * pow2i(max(sm_e[ww] - e_most, -126)) * sm_o[((size_t)ww * kMaxGroup + g) * kHeadDim + d];
        l += wt * sm_l[ww * kMaxGroup + g];
      }
      o = l != 0.0f ? o * (1.0f / l) * pow2i(e_most) : 0.0f;
      if (cnt == 1) {
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
    if (cnt > 1) {
      // the pair's last CTA joins the partials, in CTA order
      __syncthreads();
      if (threadIdx.x == 0) {
        __threadfence();
        sh_last = atomicAdd(&s.tickets[b * hkv + h], 1) == cnt - 1;
        __threadfence();
      }
      __syncthreads();
      if (sh_last) {
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
          const int mine = (cnt - share + wph - 1) / wph;  // parts share + wph j
          for (int j0 = 0; j0 < mine; j0 += 32) {
            const bool on = j0 + lane < mine;
            const float2 x = on ? __ldcg(ml + (size_t)(share + wph * (j0 + lane)) * G) : make_float2(kNegBig, 0.0f);
            const float top = fmaxf(M, warp_max(x.x));
            // the mean so far and the parts' shares of the new one
            float al = l * fast_exp2(M - top), wt = on ? fast_exp2(x.x - top) * x.y : 0.0f;
            M = top;
            l = al + warp_sum(wt);
            const float inv = l != 0.0f ? 1.0f / l : 0.0f;
            al *= inv;
            wt *= inv;
            o.x *= al; o.y *= al; o.z *= al; o.w *= al;
            for (int i0 = 0; i0 < min(32, mine - j0); i0 += 8) {
              float4 y[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)  // past the end: the last part again, weight 0
                y[i] = __ldcg(po + (size_t)(share + wph * min(j0 + i0 + i, mine - 1)) * G * (kHeadDim / 4));
#pragma unroll
              for (int i = 0; i < 8; ++i) {
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
        if (threadIdx.x == 0) s.tickets[b * hkv + h] = 0;
      }
    }
    __syncthreads();  // shared memory is reused by the next pair
    F = PARTS ? F + N : Pf + u_e;
  }
}

template <bool FP8, int MOD, bool PARTS>
cudaError_t block_attn_smem() {
  static int done[64] = {0};
  return opt_in_smem(reinterpret_cast<const void*>(block_attn_kernel<FP8, MOD, PARTS>), kBSmem, done);
}

template <bool FP8, int MOD>
int block_attn_ctas() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (dev < 64 && cached[dev] > 0) return cached[dev];
  int n = 0;
  if (block_attn_smem<FP8, MOD, false>() != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, block_attn_kernel<FP8, MOD, false>, kBThreads, kBSmem) !=
          cudaSuccess ||
      n < 1)
    n = 1;
  if (dev < 64) cached[dev] = n;
  return n;
}

int block_mod(const ScoreMod& m) { return (m.c2 > 0.0f ? kBCap : 0) | (m.slopes != nullptr ? kBBias : 0); }

template <bool FP8, int MOD>
cudaError_t launch_block_attn_t(const BlockState& s, int seq_begin, int batch, const uint16_t* q, uint16_t* out,
                                const BlockAttn& w, cudaStream_t st) {
  const cudaError_t e = w.parts ? block_attn_smem<FP8, MOD, true>() : block_attn_smem<FP8, MOD, false>();
  if (e != cudaSuccess) return e;
  if (w.parts)
    block_attn_kernel<FP8, MOD, true><<<w.ncta, kBThreads, kBSmem, st>>>(s, seq_begin, batch, q, out, w);
  else
    block_attn_kernel<FP8, MOD, false><<<w.ncta, kBThreads, kBSmem, st>>>(s, seq_begin, batch, q, out, w);
  return cudaGetLastError();
}

template <bool FP8>
cudaError_t launch_block_attn_mod(const BlockState& s, int seq_begin, int batch, const uint16_t* q, uint16_t* out,
                                  const BlockAttn& w, cudaStream_t st) {
  switch (block_mod(w.mod)) {
    case 0: return launch_block_attn_t<FP8, 0>(s, seq_begin, batch, q, out, w, st);
    case 1: return launch_block_attn_t<FP8, 1>(s, seq_begin, batch, q, out, w, st);
    case 2: return launch_block_attn_t<FP8, 2>(s, seq_begin, batch, q, out, w, st);
    default: return launch_block_attn_t<FP8, 3>(s, seq_begin, batch, q, out, w, st);
  }
}

template <bool FP8>
int block_attn_ctas_mod(int mod) {
  switch (mod) {
    case 0: return block_attn_ctas<FP8, 0>();
    case 1: return block_attn_ctas<FP8, 1>();
    case 2: return block_attn_ctas<FP8, 2>();
    default: return block_attn_ctas<FP8, 3>();
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

int block_attention_ctas_per_sm(const BlockState& s, const ScoreMod& mod) {
  return s.fp8 ? block_attn_ctas_mod<true>(block_mod(mod)) : block_attn_ctas_mod<false>(block_mod(mod));
}

cudaError_t launch_block_attention(const BlockState& s, int seq_begin, int batch, const uint16_t* q, uint16_t* out,
                                   const BlockAttn& w, cudaStream_t st) {
  return s.fp8 ? launch_block_attn_mod<true>(s, seq_begin, batch, q, out, w, st)
               : launch_block_attn_mod<false>(s, seq_begin, batch, q, out, w, st);
}

cudaError_t launch_block_append(const BlockState& s, const KeyBounds& bounds, int seq_begin, int batch, int n_new,
                                const uint16_t* k, const uint16_t* v, cudaStream_t st) {
  return bounds.codes ? append_launch(s, seq_begin, batch, n_new, k, v, AppendBounds{bounds}, st)
                      : append_launch(s, seq_begin, batch, n_new, k, v, AppendPlain{}, st);
}

cudaError_t launch_block_append_rotary(const BlockState& s, const KeyBounds& bounds, int seq_begin,
                                       const RotaryArgs& rot, const RowsIn& v, cudaStream_t st) {
  const int splits = rotary_splits((long long)rot.batch * rot.n, rot.hq);
  return bounds.codes ? append_launch(s, seq_begin, rot.batch, rot.n, nullptr, nullptr,
                                      AppendRotaryBounds{rot, v, splits, bounds}, st)
                      : append_launch(s, seq_begin, rot.batch, rot.n, nullptr, nullptr, AppendRotary{rot, v, splits}, st);
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
