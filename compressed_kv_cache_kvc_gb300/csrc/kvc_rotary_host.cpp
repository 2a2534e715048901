// Host side of the rotary positions: argument checks, the frequencies as fractions
// of a turn, the launch.
#include "kvc_rotary_host.h"

#include <algorithm>
#include <cmath>
#include <cstring>

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// f / 2 pi mod 1, times 2^64, of |f| <= 2^16: f is m 2^e with m below 2^24 and e
// at most -7, 1 / 2 pi the first 128 bits behind the point, so that the product
// (kept from its 64th bit behind the point on, the lower ones added in) is off by
// less than one unit of the last place before it is rounded.
uint64_t turns_of(float f) {
  uint32_t bits;
  std::memcpy(&bits, &f, 4);
  const int field = bits >> 23 & 0xFF, e = std::max(field, 1) - 150;
  const uint64_t mi = (bits & 0x7FFFFF) | (field ? 0x800000u : 0u);
  constexpr uint64_t hi = 0x28BE60DB9391054Aull, lo = 0x7F09D5F47D4D3770ull;
  unsigned __int128 t = (unsigned __int128)mi * hi + (((unsigned __int128)mi * lo) >> 64);
  if (mi == 0 || -e >= 120) return 0;
  t = (t + ((unsigned __int128)1 << (-e - 1))) >> -e;
  return f < 0.0f ? 0 - (uint64_t)t : (uint64_t)t;
}

}  // namespace

namespace kvc {

kvc_status rotary_table(const kvc_rotary* r, const int32_t* d_pos, int32_t first, RotaryTable* t) {
  if (!r || !aligned(d_pos, 4)) return KVC_ERR_INVALID_ARG;
  if (r->rotary_dim < 16 || r->rotary_dim > kHeadDim || r->rotary_dim % 16 != 0) return KVC_ERR_UNSUPPORTED;
  if (r->adjacent < 0 || r->adjacent > 1 || r->axes < 1 || r->axes > kRotAxes) return KVC_ERR_INVALID_ARG;
  *t = RotaryTable{};
  for (int i = 0; i < r->rotary_dim / 2; ++i) {
    if (!(std::fabs(r->freq[i]) <= 65536.0f) || r->axis[i] >= r->axes) return KVC_ERR_INVALID_ARG;
    t->turns[i] = turns_of(r->freq[i]);
    t->axis[i] = r->axis[i];
  }
  t->rot = r->rotary_dim;
  t->adjacent = r->adjacent;
  t->axes = r->axes;
  t->first = first;
  t->pos = d_pos;
  return KVC_OK;
}

kvc_status rows_in(const kvc_rows* r, int32_t batch, int32_t n, bool out, RowsIn* in) {
  if (!r || r->heads <= 0 || !r->d_in || !aligned(r->d_in, 16)) return KVC_ERR_INVALID_ARG;
  const int64_t packed_h = (int64_t)n * kHeadDim, packed_b = packed_h * r->heads;
  const int64_t sb = batch > 1 ? r->stride_batch : packed_b, sh = r->heads > 1 ? r->stride_head : packed_h,
                st = n > 1 ? r->stride_token : kHeadDim;
  if (sb % 8 != 0 || sh % 8 != 0 || st % 8 != 0) return KVC_ERR_INVALID_ARG;
  if (out && (!r->d_out || !aligned(r->d_out, 16) ||
              (r->d_out == r->d_in && (sb != packed_b || sh != packed_h || st != kHeadDim))))
    return KVC_ERR_INVALID_ARG;
  *in = RowsIn{static_cast<const uint16_t*>(r->d_in), sb, sh, st};
  return KVC_OK;
}

}  // namespace kvc

extern "C" kvc_status kvc_rotary_rotate(const kvc_rotary* rotary, int32_t batch, int32_t n, const kvc_rows* q,
                                        const kvc_rows* k, const int32_t* d_positions, int32_t first, void* stream) {
  if (batch <= 0 || n <= 0 || (!d_positions && (int64_t)first + n - 1 > INT32_MAX)) return KVC_ERR_INVALID_ARG;
  kvc::RotaryArgs a{};
  kvc_status st = kvc::rotary_table(rotary, d_positions, first, &a.table);
  if (st == KVC_OK) st = kvc::rows_in(q, batch, n, true, &a.q);
  if (st == KVC_OK && k) st = kvc::rows_in(k, batch, n, true, &a.k);
  if (st != KVC_OK) return st;
  a.batch = batch;
  a.n = n;
  a.hq = q->heads;
  a.hk = k ? k->heads : 0;
  a.q_out = static_cast<uint16_t*>(q->d_out);
  a.k_out = k ? static_cast<uint16_t*>(k->d_out) : nullptr;
  return kvc::launch_rotary(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KVC_OK : KVC_ERR_CUDA;
}
