// Queries and keys rotated by their positions, outside any cache.
//
// Per row 256 bytes in, 256 out and 128 values turned: bound by DRAM (4 x 40 heads x
// 4,099 tokens 60.4 us a call, 5.6 TB/s, 82 % of a copy's rate; one token of 16 heads
// 4.5 us, the host's 16 before it).  The angles of a token serve all of its heads,
// so a warp takes four tokens (eight lanes a row) and goes through heads with them in
// registers, four rows of each lane in flight.
#include "kvc_rotary.h"

#include <algorithm>

namespace kvc {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a, int splits) {
  __shared__ uint64_t turns[kRotPairs];
  __shared__ uint8_t axis[kRotPairs];
  if (threadIdx.x < kRotPairs) {
    turns[threadIdx.x] = a.table.turns[threadIdx.x];
    axis[threadIdx.x] = a.table.axis[threadIdx.x];
  }
  __syncthreads();
  rotary::rotate_unit<4>(a, turns, axis, (long long)blockIdx.x * kWarps + (threadIdx.x >> 5), splits,
                      [](int) { return 0; });
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t st) {
  const long long rows = (long long)a.batch * a.n;
  // eight heads a warp at most: longer ones make for an uneven last wave (4 x 40 heads
  // x 4,099 tokens: 67.3 us with all of a token's heads in a warp, 60.4 with eight,
  // 67.7 with six, four being loaded at once)
  const int splits = std::max(rotary_splits(rows, a.hq + a.hk), (a.hq + a.hk + 7) / 8);
  const long long warps = (rows + 3) / 4 * splits;
  rotary_kernel<<<(unsigned)((warps + kWarps - 1) / kWarps), kThreads, 0, st>>>(a, splits);
  return cudaGetLastError();
}

}  // namespace kvc
