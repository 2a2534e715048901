// Appends to the block-scaled cache with the rotation on the way: keys turned by
// their positions and rounded to bf16, then keys and values quantised by blocks as
// block_append_kernel does, to the same codes; the queries turned beside.
//
// A (token, KV head) needs the same cosines and sines as the token's other heads, and
// they cost more than all the rest of a key: with the angles of every key computed where
// it is quantised, 8 x 8 heads x 8,192 tokens took 203 us where the plain append takes
// 78.  So the work is units of 128 body rows (128 / bt blocks) of one sequence for
// some of its KV heads: the CTA (one per SM) makes a table of the rows' cosines and
// sines in shared memory, 512 bytes a row, and two groups of eight warps (more of fewer,
// where an append has few rows) go through the unit's (head, K or V) pairs with it, a
// warp 16 rows of each, the rows of the next ones on their way (cp.async, two stages).  The rows that stay exact (sinks, the
// block that stays open) follow at the end of the sequence's first unit, once its
// tiles, which may hold rows of the open block so far, are in shared memory.
//
// Places of blocks and the last CTA's step as in block_append_kernel.
//
// K and V of 8 x 8 heads x 8,192 tokens (INT8) 147 us, of 4 x 32 x 4,001 (E4M3) 172,
// where the plain append, bound by DRAM, takes 80 and 97.  Bound by latency: 88
// instructions a row (16 of them its share of the table), issue 57 %, four warps a
// scheduler (ring and table leave no shared memory for more), one fifth of their time at
// barriers.  Tried and slower: the rows in registers without the ring, at three CTAs of
// eight warps (80 registers, spilled) and at two (391 and 328 us where the two calls with
// queries and read-back took 380 and 290).
#include <cuda_bf16.h>

#include <algorithm>

#include "kvc_block.h"
#include "kvc_device.h"
#include "kvc_mma.h"
#include "kvc_quant.h"

namespace kvc {
namespace {

using namespace dev;
using namespace codes;
using namespace quant;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kUnitRows = 128;  // of a unit at most
constexpr int kStages = 2;
constexpr int kStage = 16 * kHeadDim * 2 + 128;  // a warp's rows, and a lane's copy of the block's id
constexpr int kTableRows = kUnitRows + kSinks;   // (the exact rows: at most 4 + 127)
constexpr int kTableRow = kRotPairs * 8;
constexpr int kOffTable = kWarps * kStages * kStage;
constexpr int kSmem = kOffTable + kTableRows * kTableRow;
// rows of queries from which they are turned by a launch of their own, under the append.
// With the release, in a graph, in the append's CTAs / apart: 1 x 32 heads on 8 x 1,024 /
// 2,048 / 8,192 tokens 29 / 31 / 56, 21 / 22 / 49 us; 64 x 32 on 8 x 16 / 41 16.4 / 30, 17.1 /
// 26; 8 x 32 on 8 x 8,192 328, 299.  Fewer rows are left to one launch, which the host issues
// 1.3 to 2.3 us sooner, although the GPU would gain by two there too: 1 x 32 on 8 x 64 /
// 512 17 / 25, 15 / 21; 64 x 8 x 41 28, 23; 64 x 32 on 8 x 1 12.0, 9.9, but eager 14.9, 16.0.
constexpr long long kManyQueryRows = 1 << 15;

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}

struct RotaryAppend {
  RotaryArgs rot;  // q's rows, k's input; hk 0
  RowsIn v;
  KeyBounds bounds;
  int splits;      // warps that share a query row's heads
  int tiles;       // units of a sequence and share of its heads
  int shares;      // shares of the KV heads
  int group;       // warps that have a (head, K or V) together, 16 rows each
  int advance;     // the lengths and the stack too (else the queries' launch does)
};

// The last CTA's step, by one warp: the lengths and the stack of free blocks.
__device__ void advance(const BlockState& s, int seq_begin, int batch, int n_new) {
  const int lane = threadIdx.x & 31, top = s.counters[kCtrFreeTop];
  int total = 0, bad = 0;
  for (int i = lane; i < batch; i += 32) {
    const int P = s.seq_pos[seq_begin + i], c1 = block_closed(P + n_new, s.bt);
    total += c1 - block_closed(P, s.bt);
    bad |= c1 > s.max_bps;
  }
  total = __reduce_add_sync(0xffffffffu, total);
  bad = __any_sync(0xffffffffu, bad);
  const int flags = (bad ? kDevTableOverflow : 0) | (total > top || top > s.num_blocks ? kDevOutOfBlocks : 0);
  if (flags == 0)
    for (int i = lane; i < batch; i += 32) s.seq_pos[seq_begin + i] += n_new;
  if (lane == 0) {
    s.tickets[s.max_batch * s.hkv] = 0;
    if (flags == 0)
      s.counters[kCtrFreeTop] = top - total;
    else
      atomicOr(&s.counters[kCtrStatus], flags);
  }
}

// FULL: groups of eight warps
template <bool FP8, bool BOUNDS, bool FULL>
__global__ void __launch_bounds__(kThreads, 1)
    append_rotary_kernel(BlockState s, int seq_begin, const __grid_constant__ RotaryAppend a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int before[kMaxCallBatch], held[kMaxCallBatch];  // blocks completed before it; its length
  __shared__ int sh_bad, sh_last;
  __shared__ float sh_amax[2][kWarps];
  __shared__ uint64_t sh_turns[kRotPairs];
  __shared__ uint8_t sh_axis[kRotPairs];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hkv = s.hkv, bt = s.bt, sh = __ffs(bt) - 1, batch = a.rot.batch, n_new = a.rot.n;
  const int top = s.counters[kCtrFreeTop];
  launch_dependents();
  if (tid < kRotPairs) {
    sh_turns[tid] = a.rot.table.turns[tid];
    sh_axis[tid] = a.rot.table.axis[tid];
  }
  if (warp == kWarps - 1) {
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
      sh_bad = (bad ? kDevTableOverflow : 0) | (total > top || top > s.num_blocks ? kDevOutOfBlocks : 0);
    }
  }
  __syncthreads();
  const bool ok = sh_bad == 0;  // the same for every CTA
  if (ok) {
    const int gsz = FULL ? kUnitRows / 16 : a.group, groups = kWarps / gsz, group = warp / gsz, gw = warp % gsz, unit_rows = 16 * gsz;
    const int wpb = bt / 16, w0 = gw & ~(wpb - 1);     // warps per block, the block's first of the group
    const int block_bar = 1 + (group * gsz + w0) / 2;  // (blocks of one warp need none)
    const size_t exact_rows = kSinks + bt;
    const bool adjacent = a.rot.table.adjacent != 0;
    const int cl = lane & 7, ca = rotary::chunk_a(a.rot.table, cl), cb = rotary::chunk_b(a.rot.table, cl);
    const bool turned = rotary::turns_here(a.rot.table, cl);
    auto closed_at = [&](int P) { return P > kSinks ? (P - kSinks) >> sh : 0; };
    auto place = [&](int p) { return p < kSinks ? p : kSinks + ((p - kSinks) & (bt - 1)); };
    auto rows_in = [&](int kv, int bl, int h) -> const uint16_t* {
      const RowsIn& r = kv ? a.v : a.rot.k;
      return r.in + bl * r.sb + h * r.sh;
    };
    auto step_in = [&](int kv) -> ptrdiff_t { return kv ? a.v.st : a.rot.k.st; };
    auto exact_of = [&](int kv, int bl, int h) {
      return (kv ? s.v_exact : s.k_exact) + ((size_t)(seq_begin + bl) * hkv + h) * exact_rows * kHeadDim;
    };

    // unit u: share u % shares of the heads, tile x of sequence bl
    struct Unit {
      int u, bl, x, h0, h1;
    };
    const int units = batch * a.tiles * a.shares;
    auto unit_of = [&](int u) {
      Unit t;
      t.u = u;
      const int share = u % a.shares;
      t.x = u / a.shares % a.tiles;
      t.bl = u / a.shares / a.tiles;
      t.h0 = (int)((long long)hkv * share / a.shares);
      t.h1 = (int)((long long)hkv * (share + 1) / a.shares);
      return t;
    };
    auto live_rows = [&](const Unit& t) {  // body rows of the unit's tile
      const int P = held[t.bl];
      const long long rows = (long long)(closed_at(P + n_new) - closed_at(P)) << sh;
      return (int)max(0LL, min(rows - (long long)t.x * unit_rows, (long long)unit_rows));
    };
    // item q of a unit: (h0 + q / 2, K or V); the groups take heads in turn, of fewer
    // heads than groups K and V
    auto items = [&](const Unit& t) { return 2 * (t.h1 - t.h0); };
    auto mine = [&](const Unit& t, int q) {
      return (t.h1 - t.h0 < groups ? q : q >> 1) % groups == group;
    };

    // the copies of the group's next item
    uint8_t* ring = smem + warp * kStages * kStage;
    const uint32_t ring_s = smem_u32(ring);
    Unit nu = unit_of(blockIdx.x);
    int nq = -1, st_next = 0;
    auto next_item = [&]() {  // the cursor goes to the group's next item, over units without rows
      while (nu.u < units) {
        if (live_rows(nu) > 0)
          for (++nq; nq < items(nu); ++nq)
            if (mine(nu, nq)) return;
        nq = -1;
        nu.u += gridDim.x;
        if (nu.u < units) nu = unit_of(nu.u);
      }
    };
    auto issue = [&]() {
      if (nu.u < units) {
        const int P = held[nu.bl], c0 = closed_at(P), h = nu.h0 + (nq >> 1), kv = nq & 1;
        const int row0 = nu.x * unit_rows + gw * 16;
        if (16 * gw < live_rows(nu)) {
          const int p0 = kSinks + (c0 << sh) + row0 + (lane >> 4);  // the lane's first row
          const ptrdiff_t step = step_in(kv);
          const uint16_t* in = rows_in(kv, nu.bl, h) + (p0 - P) * step + 8 * (lane & 15);
          const uint16_t* exact = exact_of(kv, nu.bl, h) + kSinks * kHeadDim + 8 * (lane & 15);
          const uint32_t dst = ring_s + st_next * kStage + 16 * lane;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int p = p0 + 2 * i;  // (a first tile may begin in the open block's rows)
            cp16(dst + 512 * i, p < P ? exact + (size_t)((p - kSinks) & (bt - 1)) * kHeadDim : in + 2 * i * step);
          }
          cp4(ring_s + st_next * kStage + 16 * kHeadDim * 2 + 4 * lane,
              s.free_stack + (top - 1 - (before[nu.bl] + (row0 >> sh))));
        }
        st_next = st_next + 1 == kStages ? 0 : st_next + 1;
        next_item();
      }
      cp_async_commit();
    };
    next_item();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue();

    // the table: 16-byte chunk 8 k + c of a row has the cosines and sines of pairs
    // 8 c + 2 k and the next (eight lanes read 128 bytes)
    auto make_table = [&](int bl, int rows, auto token_of) {  // token_of(row): index among the new tokens, or -1
      const int P = held[bl];
      for (int e = tid; e < rows * 8; e += kThreads) {
        const int r = e >> 3, c = e & 7, i = token_of(r);
        if (i < 0 || !rotary::turns_here(a.rot.table, c)) continue;
        float cs[8], sn[8];
        rotary::angles(sh_turns, sh_axis,
                       rotary::row_pos(a.rot.table, (size_t)bl * n_new + i, (size_t)batch * n_new, P + i), c, cs, sn);
        float4* to = reinterpret_cast<float4*>(smem + kOffTable + r * kTableRow) + c;
#pragma unroll
        for (int k = 0; k < 4; ++k) to[8 * k] = make_float4(cs[2 * k], sn[2 * k], cs[2 * k + 1], sn[2 * k + 1]);
      }
    };
    auto turn_row = [&](int r, uint4& x, uint4& y) {  // by the table's row r
      const float4* from = reinterpret_cast<const float4*>(smem + kOffTable + r * kTableRow) + cl;
      float cs[8], sn[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 t = from[8 * k];
        cs[2 * k] = t.x; sn[2 * k] = t.y; cs[2 * k + 1] = t.z; sn[2 * k + 1] = t.w;
      }
      rotary::turn16(adjacent, x, y, cs, sn);
    };

    int st = 0, flip = 0;
#pragma unroll 1
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
      const Unit t = unit_of(u);
      const int bl = t.bl, P = held[bl], c0 = closed_at(P), nb = closed_at(P + n_new) - c0, live = live_rows(t);
      const int p_tile = kSinks + (c0 << sh) + t.x * unit_rows;
      if (live > 0) {
        make_table(bl, live, [&](int r) { return p_tile + r >= P ? p_tile + r - P : -1; });
        __syncthreads();
        const bool on = 16 * gw < live;
#pragma unroll 1
        for (int q = 0; q < items(t); ++q) {
          if (!mine(t, q)) continue;
          const int h = t.h0 + (q >> 1), kv = q & 1;
          issue();
          cp_async_wait<kStages - 1>();
          __syncwarp();
          uint8_t* stage = ring + st * kStage;
          st = st + 1 == kStages ? 0 : st + 1;
          if (!on) continue;  // (a block's warps are all on or none)
          // new keys are turned where they lie (a row of the open block was when it came)
          if (kv == 0) {
            if (turned)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int r = 4 * k + (lane >> 3);
                if (p_tile + 16 * gw + r < P) continue;
                uint4* xa = reinterpret_cast<uint4*>(stage + 256 * r + 16 * ca);
                uint4* xb = reinterpret_cast<uint4*>(stage + 256 * r + 16 * cb);
                uint4 x = *xa, y = *xb;
                turn_row(16 * gw + r, x, y);
                *xa = x;
                *xb = y;
              }
            __syncwarp();
          }
          const uint8_t* rows = stage + 16 * lane;
          // the block's maximum; (BOUNDS) a lane's eight channels, the least of them in
          // lanes 0 .. 15, the largest in the others
          uint4 ends = make_uint4(0u, 0u, 0u, 0u);
          __nv_bfloat162 mx = __floats2bfloat162_rn(0.0f, 0.0f);
          if (BOUNDS && kv == 0) {
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
              const __nv_bfloat162 lo = __shfl_xor_sync(0xffffffffu, least[e], 16);
              const __nv_bfloat162 hi = __shfl_xor_sync(0xffffffffu, most[e], 16);
              const __nv_bfloat162 x = lane < 16 ? __hmin2(least[e], lo) : __hmax2(most[e], hi);
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
          float amax = fmaxf(__low2float(mx), __high2float(mx));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          if (wpb > 1) {
            if (lane == 0) sh_amax[flip][warp] = amax;
            bar_sync(block_bar, 32 * wpb);
            for (int i = w0; i < w0 + wpb; ++i) amax = fmaxf(amax, sh_amax[flip][group * gsz + i]);
            flip ^= 1;  // the next maxima go beside these, which a slower warp may still read
          }
          const float scale = __fdiv_rn(amax, FP8 ? 448.0f : 127.0f);
          const float inv = rcp_approx_ftz(scale);
          const bool exact_div = !(scale >= 0x1p-126f && scale < INFINITY);
          const int blk = *reinterpret_cast<const int*>(stage + 16 * kHeadDim * 2 + 4 * lane);
          if ((unsigned)blk >= (unsigned)s.num_blocks) {  // (the same for the block's warps)
            if (lane == 0) atomicOr(&s.counters[kCtrStatus], kDevBadBlockId);
            continue;
          }
          const size_t hblk = (size_t)blk * hkv + h;
          const int in_block = (16 * gw) & (bt - 1);
          uint8_t* dst =
              (kv ? s.v_codes : s.k_codes) + ((hblk << sh) + in_block + (lane >> 4)) * kHeadDim + 8 * (lane & 15);
#pragma unroll 4
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint2*>(dst + 2 * i * kHeadDim) =
                block_codes8<FP8>(*reinterpret_cast<const uint4*>(rows + 512 * i), scale, inv, exact_div);
          if (in_block == 0 && lane == 0) {
            (kv ? s.v_scale : s.k_scale)[hblk] = scale;
            if (h == 0 && kv == 0)
              s.table[(size_t)(seq_begin + bl) * s.max_bps + c0 + ((t.x * unit_rows + 16 * gw) >> sh)] = blk;
          }
          if (BOUNDS && kv == 0) {
            if (wpb > 1) {  // the block's warps meet in the places of their rows, which they have read
              __syncwarp();
              *reinterpret_cast<uint4*>(stage + 16 * lane) = ends;
              bar_sync(block_bar, 32 * wpb);
              if (gw == w0) {
                uint32_t z[4] = {ends.x, ends.y, ends.z, ends.w};
                for (int i = 1; i < wpb; ++i) {
                  const uint4 o = *reinterpret_cast<const uint4*>(stage + i * kStages * kStage + 16 * lane);
                  const uint32_t y[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const __nv_bfloat162 p = *reinterpret_cast<const __nv_bfloat162*>(&z[e]);
                    const __nv_bfloat162 r = *reinterpret_cast<const __nv_bfloat162*>(&y[e]);
                    const __nv_bfloat162 x = lane < 16 ? __hmin2(p, r) : __hmax2(p, r);
                    z[e] = *reinterpret_cast<const uint32_t*>(&x);
                  }
                }
                ends = make_uint4(z[0], z[1], z[2], z[3]);
              }
              bar_sync(block_bar, 32 * wpb);
            }
            if (gw == w0) {
              const float b = FP8 ? __fdiv_rn(amax, 127.0f) : scale;
              *reinterpret_cast<uint2*>(a.bounds.codes + hblk * (2 * kHeadDim) + 8 * lane) = block_codes8<false>(
                  ends, b, FP8 ? rcp_approx_ftz(b) : inv, !(b >= 0x1p-126f && b < INFINITY));
              if (lane == 0) a.bounds.scale[hblk] = b;
            }
          }
        }
        __syncthreads();  // (the table, and the open block's rows, have been read)
      }
      if (t.x == 0) {
        // sinks, and the rows of the block that stays open
        const int open0 = kSinks + ((c0 + nb) << sh);
        const int n_sink = max(0, min(kSinks - P, n_new));
        const int first = min(max(open0 - P, n_sink), n_new);  // first new token of the open block
        const int rows = n_sink + (n_new - first), heads = t.h1 - t.h0;
        auto token = [&](int r) { return r < n_sink ? r : first + (r - n_sink); };
        make_table(bl, rows, token);
        __syncthreads();
        // keys: eight lanes a row, values: sixteen
        for (int e = tid >> 3; e < rows * heads; e += kThreads / 8) {
          const int r = e % rows, h = t.h0 + e / rows, i = token(r);
          const uint16_t* in = rows_in(0, bl, h) + i * step_in(0);
          uint4 x = *reinterpret_cast<const uint4*>(in + 8 * ca), y = *reinterpret_cast<const uint4*>(in + 8 * cb);
          if (turned) turn_row(r, x, y);
          uint16_t* to = exact_of(0, bl, h) + (size_t)place(P + i) * kHeadDim;
          *reinterpret_cast<uint4*>(to + 8 * ca) = x;
          *reinterpret_cast<uint4*>(to + 8 * cb) = y;
        }
#pragma unroll 2
        for (int e = tid >> 4; e < rows * heads; e += kThreads / 16) {
          const int r = e % rows, h = t.h0 + e / rows, i = token(r);
          reinterpret_cast<uint4*>(exact_of(1, bl, h) + (size_t)place(P + i) * kHeadDim)[tid & 15] =
              reinterpret_cast<const uint4*>(rows_in(1, bl, h) + i * step_in(1))[tid & 15];
        }
        __syncthreads();
      }
    }
    cp_async_wait<0>();
    if (a.rot.hq > 0) {
      const long long n_q = ((long long)batch * n_new + 3) / 4 * a.splits;
      for (long long k = (long long)blockIdx.x * kWarps + warp; k < n_q; k += (long long)gridDim.x * kWarps)
        rotary::rotate_unit<4>(a.rot, sh_turns, sh_axis, k, a.splits, [&](int b) { return held[b]; });
    }
  }
  if (!a.advance) return;
  // the last CTA advances the lengths and the stack (every CTA has read them)
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    sh_last = atomicAdd(s.tickets + s.max_batch * hkv, 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (sh_last && warp == 0) advance(s, seq_begin, batch, n_new);
}

// The queries of a long append (positions counted from what the sequences hold), started
// under the append, which is bound by issue where they are by DRAM: a CTA of four warps
// with 64 registers, three rows of a lane in flight, fits beside the append's, more of
// them come as those end (before the append, with all of an SM, and the append under
// their end: 8 x 32 heads on 8 x 8,192 tokens with release and read-back 380 us, 4 x 32
// x 4,001 E4M3 287; so 378 and 258.  Room for two or three such CTAs, the append's
// threads kept to 104 or 80 registers, 366 and 273, 361 and 275).  The last one of them
// advances the lengths.
constexpr int kQueryThreads = 128;
__global__ void __launch_bounds__(kQueryThreads, 8)
    append_queries_kernel(BlockState s, int seq_begin, const __grid_constant__ RotaryArgs a, int splits) {
  __shared__ uint64_t turns[kRotPairs];
  __shared__ uint8_t axis[kRotPairs];
  __shared__ int sh_last;
  if (threadIdx.x < kRotPairs) {
    turns[threadIdx.x] = a.table.turns[threadIdx.x];
    axis[threadIdx.x] = a.table.axis[threadIdx.x];
  }
  __syncthreads();
  rotary::rotate_unit<3>(a, turns, axis, (long long)blockIdx.x * (kQueryThreads / 32) + (threadIdx.x >> 5), splits,
                      [&](int b) { return s.seq_pos[seq_begin + b]; });
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    sh_last = atomicAdd(s.tickets + s.max_batch * s.hkv, 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!sh_last || threadIdx.x >= 32) return;
  wait_for_previous();  // the append
  advance(s, seq_begin, a.batch, a.n);
}

template <bool FP8, bool BOUNDS, bool FULL>
cudaError_t launch_t(const BlockState& s, int seq_begin, const RotaryAppend& a, cudaStream_t st) {
  static int done[64] = {0};
  const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(append_rotary_kernel<FP8, BOUNDS, FULL>), kSmem, done);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
    sms = 152;
  const long long units = (long long)a.rot.batch * a.tiles * a.shares;
  const unsigned grid = (unsigned)(a.rot.hq > 0 ? sms : std::min<long long>(units, sms));
  append_rotary_kernel<FP8, BOUNDS, FULL><<<grid, kThreads, kSmem, st>>>(s, seq_begin, a);
  return cudaGetLastError();
}

template <bool FP8, bool BOUNDS>
cudaError_t launch(const BlockState& s, int seq_begin, const RotaryAppend& a, cudaStream_t st) {
  return a.group == kUnitRows / 16 ? launch_t<FP8, BOUNDS, true>(s, seq_begin, a, st)
                                   : launch_t<FP8, BOUNDS, false>(s, seq_begin, a, st);
}

}  // namespace

// Shares of the KV heads, of two heads at least: the number that takes the least time
// in rounds of a unit per SM, a unit's table costing 0.6 of a head's keys and values.
// (Four units per SM instead: 4 x 32 heads x 4,001 FP8 tokens, 128 tiles, in 5 shares
// 182 us where 7 take 172.)
static int head_shares(long long tiles, int hkv) {
  int best = 1;
  double least = 0.0;
  for (int k = 1; k <= std::max(1, hkv / 2); ++k) {
    const double cost = (double)((tiles * k + 151) / 152) * ((double)hkv / k + 0.6);
    if (k == 1 || cost < least) {
      best = k;
      least = cost;
    }
  }
  return best;
}

int block_append_rotary_launches(const RotaryArgs& rot) {
  return (long long)rot.batch * rot.n * rot.hq >= kManyQueryRows ? 2 : 1;
}

cudaError_t launch_block_append_rotary(const BlockState& s, const KeyBounds& bounds, int seq_begin,
                                       const RotaryArgs& rot, const RowsIn& v, cudaStream_t st) {
  const bool apart = block_append_rotary_launches(rot) > 1;
  RotaryAppend a{rot, v, bounds, 1, 1, 1, 1, !apart};
  const long long rows = (long long)rot.batch * rot.n;
  if (rot.hq > 0) a.splits = rotary_splits(rows, rot.hq);
  if (apart) a.splits = std::max(a.splits, (rot.hq + 7) / 8);  // (eight heads a warp, as without a cache)
  if (apart) a.rot.hq = 0;
  // rows of the most blocks an append of n tokens completes (at any state)
  const long long body = ((long long)rot.n + s.bt - 1) / s.bt * s.bt;
  // few rows: more groups of fewer warps (64 x 41 tokens of 8 heads 24.6 us with eight
  // warps, 22.5)
  a.group = kUnitRows / 16;
  while (a.group > s.bt / 16 && 8 * a.group >= body) a.group /= 2;
  a.tiles = (int)((body + 16 * a.group - 1) / (16 * a.group));
  a.shares = head_shares((long long)rot.batch * a.tiles, s.hkv);
  const bool kept = bounds.codes != nullptr;
  const cudaError_t e = s.fp8 ? kept ? launch<true, true>(s, seq_begin, a, st) : launch<true, false>(s, seq_begin, a, st)
                        : kept ? launch<false, true>(s, seq_begin, a, st)
                               : launch<false, false>(s, seq_begin, a, st);
  if (e != cudaSuccess || !apart) return e;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  constexpr int kWarpsQ = kQueryThreads / 32;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(((rows + 3) / 4 * a.splits + kWarpsQ - 1) / kWarpsQ));
  cfg.blockDim = dim3(kQueryThreads);
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, append_queries_kernel, s, seq_begin, rot, a.splits);
}

}  // namespace kvc
