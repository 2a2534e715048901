// Host side of the block-scaled cache's C ABI: argument checks, the host mirror
// of the lengths (capacity errors are found before anything is enqueued), the
// buffers and the launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "../../include/kvc.h"
#include "kvc_block.h"

namespace {

constexpr size_t kAlign = 256;
constexpr int kMinUnitsPerCta = 16;  // 16-token units: a CTA's share of a pair
// Sequences of unequal lengths with at least this many CTAs per pair: each CTA
// takes a part of one pair instead of an equal run across pairs, whose ends cut
// every pair once more (4 x 8 KV heads of 32,768 tokens and less 35.1 against
// 38.4 us, 8 x 8 of 10 to 4,000 14.0 against 33.0, 16 x 8 of 500 to 8,000 39.6
// against 42.7; of equal lengths the runs end with the pairs by themselves and
// need no spare CTAs: 3 x 8 of 8,000 15.8 against 16.4).
constexpr int kPartsPerPair = 2;
constexpr int kWholePairUnits = 64;  // pairs up to this long are not cut to even out a wave

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

kvc_status config_check(const kvc_block_config* c) {
  if (!c || c->num_q_heads <= 0 || c->num_kv_heads <= 0 || c->num_blocks <= 0 || c->max_batch <= 0 ||
      c->max_blocks_per_seq <= 0 || c->num_q_heads % c->num_kv_heads != 0)
    return KVC_ERR_INVALID_ARG;
  if (c->codes != KVC_CODES_INT && c->codes != KVC_CODES_E4M3) return KVC_ERR_INVALID_ARG;
  const int bt = c->block_tokens;
  if (c->head_dim != kvc::kHeadDim || (bt != 16 && bt != 32 && bt != 64 && bt != 128) ||
      c->num_q_heads / c->num_kv_heads > kvc::kMaxGroup || c->max_batch > kvc::kMaxCallBatch ||
      c->num_kv_heads > 32767)
    return KVC_ERR_UNSUPPORTED;
  // 32-bit index arithmetic inside the kernels: positions, and the 16-token
  // units of one sequence; a block's bytes over all heads in 32 bits
  if ((double)c->max_blocks_per_seq * bt > 2.0e9 || (double)c->num_kv_heads * bt * kvc::kHeadDim > 4.0e9 ||
      (double)c->max_batch * c->max_blocks_per_seq * (bt / 16) > 2.0e9 ||
      (double)c->num_blocks * bt > 2.0e9)
    return KVC_ERR_UNSUPPORTED;
  return KVC_OK;
}

struct Layout {
  size_t off[KVC_BLOCK_BUF_COUNT], size[KVC_BLOCK_BUF_COUNT], total;
};

Layout make_layout(const kvc_block_config* c) {
  Layout L{};
  const size_t hb = (size_t)c->num_blocks * c->num_kv_heads, sh = (size_t)c->max_batch * c->num_kv_heads;
  L.size[KVC_BLOCK_BUF_K_CODES] = L.size[KVC_BLOCK_BUF_V_CODES] = hb * c->block_tokens * kvc::kHeadDim;
  L.size[KVC_BLOCK_BUF_K_SCALE] = L.size[KVC_BLOCK_BUF_V_SCALE] = hb * 4;
  L.size[KVC_BLOCK_BUF_K_EXACT] = L.size[KVC_BLOCK_BUF_V_EXACT] =
      sh * (kvc::kSinks + c->block_tokens) * kvc::kHeadDim * 2;
  L.size[KVC_BLOCK_BUF_TABLE] = (size_t)c->max_batch * c->max_blocks_per_seq * 4;
  L.size[KVC_BLOCK_BUF_SEQ_POS] = (size_t)c->max_batch * 4;
  L.size[KVC_BLOCK_BUF_FREE] = (size_t)c->num_blocks * 4;
  L.size[KVC_BLOCK_BUF_COUNTERS] = (size_t)kvc::kCounters * 4;
  L.size[KVC_BLOCK_BUF_TICKETS] = (sh + 1) * 4;
  size_t o = 0;
  for (int i = 0; i < KVC_BLOCK_BUF_COUNT; ++i) {
    L.off[i] = o;
    o = align_up(o + L.size[i]);
  }
  L.total = o;
  return L;
}

}  // namespace

struct kvc_block_cache {
  kvc_block_config cfg;
  Layout layout;
  uint8_t* base;
  kvc::BlockState dev;
  std::vector<int32_t> pos;  // host mirror: tokens held per sequence
  int32_t last_launches = 0;
  int sm_count = 0;
};

namespace {

bool range_ok(const kvc_block_cache* c, int32_t seq_begin, int32_t batch) {
  return seq_begin >= 0 && batch > 0 && (long long)seq_begin + batch <= c->cfg.max_batch;
}

struct WsLayout {
  size_t part_o, part_ml, total;
};
WsLayout ws_layout(const kvc_block_cache* c, int batch) {
  const size_t G = c->dev.group, slots = (size_t)batch * c->cfg.num_kv_heads + kvc::kMaxSplitCtas;
  WsLayout w{};
  w.part_ml = align_up(slots * G * kvc::kHeadDim * 4);
  w.total = w.part_ml + align_up(slots * G * 2 * 4);
  return w;
}

// CTAs of an attention over `units` 16-token units of `pairs` (sequence, KV
// head) pairs; any number is right for any lengths, so that a graph replayed at
// other lengths stays right.  A CTA that ends inside a pair leaves a partial to
// be joined (a store, a ticket and the last CTA's reads: about 5 us), so where
// sequences are alike CTAs end with pairs:
// - up to two CTAs per SM, k per pair of at least kMinUnitsPerCta units each
//   (batch 8 x 8 KV heads, 1,000 tokens: 11.1 us at k = 4, 16.1 at 152 CTAs;
//   1 x 8, 32,000: 18.9 at k = 38, 19.4 at 456 CTAs; 32 x 8, 8,192: 82.8 at one
//   per pair, 90.5 at 456 CTAs);
// - more pairs than that, and short: whole pairs per CTA (64 x 8, 352: 18.1 with
//   two, 26.0 at 352 CTAs);
// - more pairs, and long: one full wave, whatever it cuts (64 x 8, 4,000: 85.2;
//   89.6 with two pairs per CTA, 107.6 with one).
int grid_of(long long sms, long long per_sm, long long pairs, long long units) {
  const long long wave = std::min(sms * per_sm, (long long)kvc::kMaxSplitCtas);
  const long long per_pair = (units + pairs - 1) / pairs;
  if (pairs <= std::min(2 * sms, wave)) {
    const long long k = std::min(std::min(2 * sms, wave) / pairs, (per_pair + kMinUnitsPerCta - 1) / kMinUnitsPerCta);
    return (int)(k * pairs);
  }
  if (per_pair <= kWholePairUnits) {
    const long long m = (pairs + wave - 1) / wave;
    return (int)((pairs + m - 1) / m);
  }
  return (int)wave;
}

int sm_count(kvc_block_cache* c) {
  if (c->sm_count <= 0) {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) == cudaSuccess &&
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && n > 0)
      c->sm_count = n;
    else
      c->sm_count = 152;
  }
  return c->sm_count;
}

}  // namespace

extern "C" {

size_t kvc_block_state_bytes(const kvc_block_config* cfg) {
  return config_check(cfg) == KVC_OK ? make_layout(cfg).total : 0;
}

kvc_status kvc_block_cache_create(const kvc_block_config* cfg, void* d_state, size_t state_bytes,
                                  kvc_block_cache** out) {
  if (!out) return KVC_ERR_INVALID_ARG;
  *out = nullptr;
  const kvc_status st = config_check(cfg);
  if (st != KVC_OK) return st;
  const Layout L = make_layout(cfg);
  if (!d_state || !aligned(d_state, kAlign) || state_bytes < L.total) return KVC_ERR_INVALID_ARG;
  kvc_block_cache* c = new (std::nothrow) kvc_block_cache();
  if (!c) return KVC_ERR_INVALID_ARG;
  try {
    c->pos.assign(cfg->max_batch, 0);
  } catch (...) {
    delete c;
    return KVC_ERR_INVALID_ARG;
  }
  c->cfg = *cfg;
  c->layout = L;
  c->base = static_cast<uint8_t*>(d_state);
  uint8_t* b = c->base;
  kvc::BlockState& d = c->dev;
  d.k_codes = b + L.off[KVC_BLOCK_BUF_K_CODES];
  d.v_codes = b + L.off[KVC_BLOCK_BUF_V_CODES];
  d.k_scale = reinterpret_cast<float*>(b + L.off[KVC_BLOCK_BUF_K_SCALE]);
  d.v_scale = reinterpret_cast<float*>(b + L.off[KVC_BLOCK_BUF_V_SCALE]);
  d.k_exact = reinterpret_cast<uint16_t*>(b + L.off[KVC_BLOCK_BUF_K_EXACT]);
  d.v_exact = reinterpret_cast<uint16_t*>(b + L.off[KVC_BLOCK_BUF_V_EXACT]);
  d.table = reinterpret_cast<int32_t*>(b + L.off[KVC_BLOCK_BUF_TABLE]);
  d.seq_pos = reinterpret_cast<int32_t*>(b + L.off[KVC_BLOCK_BUF_SEQ_POS]);
  d.free_stack = reinterpret_cast<int32_t*>(b + L.off[KVC_BLOCK_BUF_FREE]);
  d.counters = reinterpret_cast<int32_t*>(b + L.off[KVC_BLOCK_BUF_COUNTERS]);
  d.tickets = reinterpret_cast<int32_t*>(b + L.off[KVC_BLOCK_BUF_TICKETS]);
  d.hq = cfg->num_q_heads;
  d.hkv = cfg->num_kv_heads;
  d.group = cfg->num_q_heads / cfg->num_kv_heads;
  d.bt = cfg->block_tokens;
  d.num_blocks = cfg->num_blocks;
  d.max_batch = cfg->max_batch;
  d.max_bps = cfg->max_blocks_per_seq;
  d.fp8 = cfg->codes == KVC_CODES_E4M3 ? 1 : 0;
  *out = c;
  return KVC_OK;
}

void kvc_block_cache_destroy(kvc_block_cache* c) { delete c; }

kvc_status kvc_block_cache_reset(kvc_block_cache* c, void* stream) {
  if (!c) return KVC_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  c->last_launches = 0;
  const int32_t top = c->cfg.num_blocks;
  if (cudaMemsetAsync(c->base, 0, c->layout.total, st) != cudaSuccess) return KVC_ERR_CUDA;
  if (kvc::launch_block_fill(c->dev, st) != cudaSuccess) return KVC_ERR_CUDA;
  c->last_launches = 1;
  if (cudaMemcpyAsync(c->dev.counters + kvc::kCtrFreeTop, &top, 4, cudaMemcpyHostToDevice, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return KVC_ERR_CUDA;
  std::fill(c->pos.begin(), c->pos.end(), 0);
  return KVC_OK;
}

kvc_status kvc_block_buffer(const kvc_block_cache* c, int32_t which, void** d_ptr, size_t* bytes) {
  if (!c || which < 0 || which >= KVC_BLOCK_BUF_COUNT) return KVC_ERR_INVALID_ARG;
  if (d_ptr) *d_ptr = c->base + c->layout.off[which];
  if (bytes) *bytes = c->layout.size[which];
  return KVC_OK;
}

kvc_status kvc_block_lengths(const kvc_block_cache* c, int32_t seq_begin, int32_t batch, int32_t* shortest,
                             int32_t* longest) {
  if (!c || !range_ok(c, seq_begin, batch)) return KVC_ERR_INVALID_ARG;
  const auto mm = std::minmax_element(c->pos.begin() + seq_begin, c->pos.begin() + seq_begin + batch);
  if (shortest) *shortest = *mm.first;
  if (longest) *longest = *mm.second;
  return KVC_OK;
}

kvc_status kvc_block_sync_host(kvc_block_cache* c, void* stream) {
  if (!c) return KVC_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(c->pos.data(), c->dev.seq_pos, c->pos.size() * 4, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return KVC_ERR_CUDA;
  return KVC_OK;
}

kvc_status kvc_block_read_status(kvc_block_cache* c, int32_t* h_status, void* stream) {
  if (!c || !h_status) return KVC_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t v = 0;
  int32_t* word = c->dev.counters + kvc::kCtrStatus;
  if (cudaMemcpyAsync(&v, word, 4, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return KVC_ERR_CUDA;
  *h_status = v;
  if (v == 0) return KVC_OK;
  if (cudaMemsetAsync(word, 0, 4, st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess) return KVC_ERR_CUDA;
  return KVC_ERR_DEVICE;
}

int32_t kvc_block_last_launch_count(const kvc_block_cache* c) { return c ? c->last_launches : 0; }

kvc_status kvc_block_release(kvc_block_cache* c, int32_t seq_begin, int32_t batch, void* stream) {
  if (!c) return KVC_ERR_INVALID_ARG;
  c->last_launches = 0;
  if (!range_ok(c, seq_begin, batch)) return KVC_ERR_INVALID_ARG;
  bool any = false;
  for (int i = 0; i < batch; ++i) any |= c->pos[seq_begin + i] != 0;
  if (!any) return KVC_OK;
  if (kvc::launch_block_release(c->dev, seq_begin, batch, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return KVC_ERR_CUDA;
  c->last_launches = 1;
  std::fill_n(c->pos.begin() + seq_begin, batch, 0);
  return KVC_OK;
}

kvc_status kvc_block_append(kvc_block_cache* c, int32_t seq_begin, int32_t batch, int32_t n_new, const void* d_k,
                            const void* d_v, void* stream) {
  if (!c) return KVC_ERR_INVALID_ARG;
  c->last_launches = 0;
  if (!range_ok(c, seq_begin, batch) || n_new < 0) return KVC_ERR_INVALID_ARG;
  if (n_new == 0) return KVC_OK;
  if (!d_k || !d_v || !aligned(d_k, 16) || !aligned(d_v, 16)) return KVC_ERR_INVALID_ARG;
  const int bt = c->cfg.block_tokens;
  long long used = 0, need = 0;
  for (int b = 0; b < c->cfg.max_batch; ++b) used += kvc::block_closed(c->pos[b], bt);
  for (int i = 0; i < batch; ++i) {
    const int P = c->pos[seq_begin + i];
    if ((long long)P + n_new > 2000000000LL) return KVC_ERR_CAPACITY;
    const int after = kvc::block_closed(P + n_new, bt);
    if (after > c->cfg.max_blocks_per_seq) return KVC_ERR_CAPACITY;
    need += after - kvc::block_closed(P, bt);
  }
  if (need > c->cfg.num_blocks - used) return KVC_ERR_CAPACITY;
  if (kvc::launch_block_append(c->dev, seq_begin, batch, n_new, static_cast<const uint16_t*>(d_k),
                               static_cast<const uint16_t*>(d_v), static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return KVC_ERR_CUDA;
  c->last_launches = 1;
  for (int i = 0; i < batch; ++i) c->pos[seq_begin + i] += n_new;
  return KVC_OK;
}

size_t kvc_block_workspace_bytes(const kvc_block_cache* c, int32_t batch) {
  if (!c || batch <= 0 || batch > c->cfg.max_batch) return 0;
  return ws_layout(c, batch).total;
}

kvc_status kvc_block_attention(kvc_block_cache* c, int32_t seq_begin, int32_t batch, const void* d_q, void* d_out,
                               float sm_scale, float softcap, const float* d_slopes, void* d_workspace,
                               size_t workspace_bytes, void* stream) {
  if (!c) return KVC_ERR_INVALID_ARG;
  c->last_launches = 0;
  if (!range_ok(c, seq_begin, batch)) return KVC_ERR_INVALID_ARG;
  if (!d_q || !d_out || !aligned(d_q, 16) || !aligned(d_out, 16) || !aligned(d_slopes, 4)) return KVC_ERR_INVALID_ARG;
  if (!(sm_scale > 0.0f) || !std::isfinite(sm_scale) || !(softcap >= 0.0f) || !std::isfinite(softcap))
    return KVC_ERR_INVALID_ARG;
  const WsLayout wl = ws_layout(c, batch);
  if (!d_workspace || !aligned(d_workspace, kAlign) || workspace_bytes < wl.total) return KVC_ERR_INVALID_ARG;
  long long units = 0;
  bool ragged = false;
  for (int i = 0; i < batch; ++i) {
    const int P = c->pos[seq_begin + i];
    if (P <= 0) return KVC_ERR_INVALID_ARG;  // nothing to attend to
    units += (long long)kvc::block_units(P, c->cfg.block_tokens) * c->cfg.num_kv_heads;
    ragged |= P != c->pos[seq_begin];
  }
  kvc::BlockAttn a{};
  a.part_o = static_cast<float*>(d_workspace);
  a.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(d_workspace) + wl.part_ml);
  a.mod = kvc::make_score_mod(sm_scale, softcap, d_slopes);
  a.qk_scale_log2 = sm_scale * kvc::kLog2E;
  a.ncta = grid_of(sm_count(c), kvc::block_attention_ctas_per_sm(c->dev, a.mod), batch * c->cfg.num_kv_heads, units);
  const int hkv = c->cfg.num_kv_heads;
  if (ragged && batch <= kvc::kMaxSplitBatch && a.ncta >= batch * hkv * kPartsPerPair) {
    // (a sequence has one part at least; a CTA without a part ends)
    a.parts = a.ncta / hkv;
    a.ncta = std::min((a.parts + batch) * hkv, kvc::kMaxSplitCtas);
  }
  if (kvc::launch_block_attention(c->dev, seq_begin, batch, static_cast<const uint16_t*>(d_q),
                                  static_cast<uint16_t*>(d_out), a, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return KVC_ERR_CUDA;
  c->last_launches = 1;
  return KVC_OK;
}

kvc_status kvc_block_read(kvc_block_cache* c, int32_t seq_begin, int32_t batch, int32_t pos_begin, int32_t n,
                          void* d_k, void* d_v, void* stream) {
  if (!c) return KVC_ERR_INVALID_ARG;
  c->last_launches = 0;
  if (!range_ok(c, seq_begin, batch) || pos_begin < 0 || n <= 0 || (long long)pos_begin + n > 2000000000LL)
    return KVC_ERR_INVALID_ARG;
  if (!d_k || !d_v || !aligned(d_k, 16) || !aligned(d_v, 16)) return KVC_ERR_INVALID_ARG;
  if (kvc::launch_block_read(c->dev, seq_begin, batch, pos_begin, n, static_cast<uint16_t*>(d_k),
                             static_cast<uint16_t*>(d_v), static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return KVC_ERR_CUDA;
  c->last_launches = 1;
  return KVC_OK;
}

}  // extern "C"
