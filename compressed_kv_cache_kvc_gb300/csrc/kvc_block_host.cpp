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
#include "kvc_rotary_host.h"

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
  kvc::KeyBounds bounds{};
  std::vector<int32_t> pos;  // host mirror: tokens held per sequence
  int32_t last_launches = 0;
  int sm_count = 0;
};

namespace {

bool range_ok(const kvc_block_cache* c, int32_t seq_begin, int32_t batch) {
  return seq_begin >= 0 && batch > 0 && (long long)seq_begin + batch <= c->cfg.max_batch;
}

// Whether n_new more tokens fit into every sequence's table row and the pool.
bool has_room(const kvc_block_cache* c, int32_t seq_begin, int32_t batch, int32_t n_new) {
  const int bt = c->cfg.block_tokens;
  long long used = 0, need = 0;
  for (int b = 0; b < c->cfg.max_batch; ++b) used += kvc::block_closed(c->pos[b], bt);
  for (int i = 0; i < batch; ++i) {
    const int P = c->pos[seq_begin + i];
    if ((long long)P + n_new > 2000000000LL) return false;
    const int after = kvc::block_closed(P + n_new, bt);
    if (after > c->cfg.max_blocks_per_seq) return false;
    need += after - kvc::block_closed(P, bt);
  }
  return need <= c->cfg.num_blocks - used;
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

bool attention_args_ok(const void* d_q, const void* d_out, float sm_scale, float softcap, const float* d_slopes) {
  return d_q && d_out && aligned(d_q, 16) && aligned(d_out, 16) && aligned(d_slopes, 4) && sm_scale > 0.0f &&
         std::isfinite(sm_scale) && softcap >= 0.0f && std::isfinite(softcap);
}

kvc::BlockAttn attention_of(const WsLayout& wl, void* d_workspace, float sm_scale, float softcap,
                            const float* d_slopes) {
  kvc::BlockAttn a{};
  a.part_o = static_cast<float*>(d_workspace);
  a.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(d_workspace) + wl.part_ml);
  a.mod = kvc::make_score_mod(sm_scale, softcap, d_slopes);
  a.qk_scale_log2 = sm_scale * kvc::kLog2E;
  return a;
}

// The CTAs of an attention, and whether they take parts of pairs.
void split_attention(kvc_block_cache* c, kvc::BlockAttn* a, int per_sm, int batch, long long units, bool ragged) {
  const int hkv = c->cfg.num_kv_heads;
  a->ncta = grid_of(sm_count(c), per_sm, batch * hkv, units);
  if (ragged && batch <= kvc::kMaxSplitBatch && a->ncta >= batch * hkv * kPartsPerPair) {
    // (a sequence has one part at least; a CTA without a part ends)
    a->parts = a->ncta / hkv;
    a->ncta = std::min((a->parts + batch) * hkv, kvc::kMaxSplitCtas);
  }
}

// The parts of pairs of the selected and the prefix form: up to `parts` CTAs for every
// pair, of at least part_units units each, so that the parts of all pairs make about
// one wave (two CTAs per SM with all their registers; three with 168 measured 51.2
// against 50.9 us for 16 x 32 heads of 65,536 selected tokens, where the busiest SM has as
// many units either way, 73.4 against 73.7 for a prefix's 64 x 32).
constexpr int kCtasPerSm = 2;
void split_pairs(kvc_block_cache* c, kvc::BlockAttn* a, int batch, long long units) {
  const long long pairs = (long long)batch * c->cfg.num_kv_heads, slots = kCtasPerSm * sm_count(c);
  a->part_units = (int)std::max<long long>(kMinUnitsPerCta, (units + slots - 1) / slots);
  a->parts = (int)std::max<long long>(1, std::min<long long>(kvc::kMaxSplitCtas / pairs, 2 * slots / pairs));
  a->ncta = (int)(pairs * a->parts);
}

bool choice_ok(int top, int recent) { return top > 0 && recent >= 0 && (long long)top + recent <= 1 << 20; }

struct SelectedLayout {
  WsLayout ws;
  size_t keys, list, ids, total;
  int places;  // of a pair's list: the blocks it may hold at most
};
SelectedLayout selected_layout(const kvc_block_cache* c, int batch, int top, int recent) {
  const size_t pairs = (size_t)batch * c->cfg.num_kv_heads;
  SelectedLayout l{};
  l.ws = ws_layout(c, batch);
  l.places = std::min(top + recent, c->cfg.max_blocks_per_seq);
  l.keys = align_up(l.ws.total);
  l.list = l.keys + align_up(pairs * c->cfg.max_blocks_per_seq * 4);
  l.ids = l.list + align_up(pairs * l.places * 4);
  l.total = l.ids + align_up(pairs * l.places * 4);
  return l;
}

// Runs of the prefix's tiles per KV head: the number that takes the fewest tiles one
// after another, over all waves of CTAs, and of those the smallest.
constexpr int kPrefixCtas = 152;
int prefix_splits(long long ctas, long long tiles) {
  const long long most = std::max(1LL, std::min(tiles, kPrefixCtas / std::min<long long>(ctas, kPrefixCtas)));
  long long best = 1, cost = 0;
  for (long long k = 1; k <= most; ++k) {
    const long long c = (ctas * k + kPrefixCtas - 1) / kPrefixCtas * ((tiles + k - 1) / k);
    if (k == 1 || c < cost) {
      best = k;
      cost = c;
    }
  }
  return (int)best;
}

struct PrefixLayout {
  WsLayout ws;
  size_t more_o, more_ml, total;
};
PrefixLayout prefix_layout(const kvc_block_cache* c, int batch) {
  const size_t rows = (size_t)batch * c->dev.group;
  const size_t ctas = (rows + kvc::kPrefixRows - 1) / kvc::kPrefixRows * c->cfg.num_kv_heads;
  const size_t parts = std::max<size_t>(1, kPrefixCtas / std::min<size_t>(ctas, kPrefixCtas)) * rows *
                       c->cfg.num_kv_heads;
  PrefixLayout l{};
  l.ws = ws_layout(c, batch);
  l.more_o = align_up(l.ws.total);
  l.more_ml = l.more_o + align_up(parts * kvc::kHeadDim * 4);
  l.total = l.more_ml + align_up(parts * 2 * 4);
  return l;
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
  if (!has_room(c, seq_begin, batch, n_new)) return KVC_ERR_CAPACITY;
  if (kvc::launch_block_append(c->dev, c->bounds, seq_begin, batch, n_new, static_cast<const uint16_t*>(d_k),
                               static_cast<const uint16_t*>(d_v), static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return KVC_ERR_CUDA;
  c->last_launches = 1;
  for (int i = 0; i < batch; ++i) c->pos[seq_begin + i] += n_new;
  return KVC_OK;
}

kvc_status kvc_block_append_rotary(kvc_block_cache* c, int32_t seq_begin, int32_t batch, int32_t n_new,
                                   const kvc_rotary* rotary, const kvc_rows* q, const kvc_rows* k, const kvc_rows* v,
                                   const int32_t* d_positions, int32_t first, void* stream) {
  if (!c) return KVC_ERR_INVALID_ARG;
  c->last_launches = 0;
  if (!range_ok(c, seq_begin, batch) || n_new < 0) return KVC_ERR_INVALID_ARG;
  if (n_new == 0) return KVC_OK;
  kvc::RotaryArgs a{};
  kvc::RowsIn rows_v{};
  kvc_status st = kvc::rotary_table(rotary, d_positions, first, &a.table);
  if (st == KVC_OK) st = kvc::rows_in(k, batch, n_new, false, &a.k);
  if (st == KVC_OK) st = kvc::rows_in(v, batch, n_new, false, &rows_v);
  if (st == KVC_OK && q) st = kvc::rows_in(q, batch, n_new, true, &a.q);
  if (st != KVC_OK) return st;
  if (k->heads != c->cfg.num_kv_heads || v->heads != c->cfg.num_kv_heads || (q && q->heads != c->cfg.num_q_heads))
    return KVC_ERR_INVALID_ARG;
  if (!d_positions)
    for (int i = 0; i < batch; ++i)
      if ((int64_t)first + c->pos[seq_begin + i] + n_new - 1 > INT32_MAX) return KVC_ERR_INVALID_ARG;
  if (!has_room(c, seq_begin, batch, n_new)) return KVC_ERR_CAPACITY;
  a.batch = batch;
  a.n = n_new;
  a.hq = q ? q->heads : 0;
  a.q_out = q ? static_cast<uint16_t*>(q->d_out) : nullptr;
  if (kvc::launch_block_append_rotary(c->dev, c->bounds, seq_begin, a, rows_v, static_cast<cudaStream_t>(stream)) !=
      cudaSuccess)
    return KVC_ERR_CUDA;
  c->last_launches = kvc::block_append_rotary_launches(a);
  for (int i = 0; i < batch; ++i) c->pos[seq_begin + i] += n_new;
  return KVC_OK;
}

size_t kvc_block_key_bounds_bytes(const kvc_block_cache* c) {
  if (!c) return 0;
  const size_t hb = (size_t)c->cfg.num_blocks * c->cfg.num_kv_heads;
  return align_up(hb * 2 * kvc::kHeadDim) + align_up(hb * 4);
}

kvc_status kvc_block_set_key_bounds(kvc_block_cache* c, void* d_bounds, size_t bytes) {
  if (!c) return KVC_ERR_INVALID_ARG;
  c->last_launches = 0;
  if (d_bounds && (!aligned(d_bounds, kAlign) || bytes < kvc_block_key_bounds_bytes(c))) return KVC_ERR_INVALID_ARG;
  for (const int32_t p : c->pos)
    if (p != 0) return KVC_ERR_STATE;
  c->bounds = kvc::KeyBounds{};
  if (d_bounds) {
    const size_t hb = (size_t)c->cfg.num_blocks * c->cfg.num_kv_heads;
    c->bounds.codes = static_cast<uint8_t*>(d_bounds);
    c->bounds.scale = reinterpret_cast<float*>(c->bounds.codes + align_up(hb * 2 * kvc::kHeadDim));
  }
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
  if (!attention_args_ok(d_q, d_out, sm_scale, softcap, d_slopes)) return KVC_ERR_INVALID_ARG;
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
  kvc::BlockAttn a = attention_of(wl, d_workspace, sm_scale, softcap, d_slopes);
  split_attention(c, &a, kvc::block_attention_ctas_per_sm(c->dev, a.mod), batch, units, ragged);
  if (kvc::launch_block_attention(c->dev, seq_begin, batch, static_cast<const uint16_t*>(d_q),
                                  static_cast<uint16_t*>(d_out), a, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return KVC_ERR_CUDA;
  c->last_launches = 1;
  return KVC_OK;
}

size_t kvc_block_selected_workspace_bytes(const kvc_block_cache* c, int32_t batch, int32_t top_blocks,
                                          int32_t recent_blocks) {
  if (!c || batch <= 0 || batch > c->cfg.max_batch || !choice_ok(top_blocks, recent_blocks)) return 0;
  return selected_layout(c, batch, top_blocks, recent_blocks).total;
}

kvc_status kvc_block_selected_attention(kvc_block_cache* c, int32_t seq_begin, int32_t batch, int32_t top_blocks,
                                        int32_t recent_blocks, const void* d_q, void* d_out, int32_t* d_blocks,
                                        float sm_scale, float softcap, const float* d_slopes, void* d_workspace,
                                        size_t workspace_bytes, void* stream) {
  if (!c) return KVC_ERR_INVALID_ARG;
  c->last_launches = 0;
  if (!range_ok(c, seq_begin, batch) || !choice_ok(top_blocks, recent_blocks)) return KVC_ERR_INVALID_ARG;
  if (!attention_args_ok(d_q, d_out, sm_scale, softcap, d_slopes) || !aligned(d_blocks, 4)) return KVC_ERR_INVALID_ARG;
  const SelectedLayout sl = selected_layout(c, batch, top_blocks, recent_blocks);
  if (!d_workspace || !aligned(d_workspace, kAlign) || workspace_bytes < sl.total) return KVC_ERR_INVALID_ARG;
  if (!c->bounds.codes) return KVC_ERR_STATE;
  const int bt = c->cfg.block_tokens, most = top_blocks + recent_blocks;
  long long units = 0;
  int longest = 0;
  for (int i = 0; i < batch; ++i) {
    const int P = c->pos[seq_begin + i];
    if (P <= 0) return KVC_ERR_INVALID_ARG;  // nothing to attend to
    const int u = std::min(kvc::block_closed(P, bt), most) * (bt / kvc::kPage) +
                  (kvc::block_exact_rows(P, bt) + kvc::kPage - 1) / kvc::kPage;
    units += (long long)u * c->cfg.num_kv_heads;
    longest = std::max(longest, P);
  }
  uint8_t* ws = static_cast<uint8_t*>(d_workspace);
  kvc::BlockChoice ch{};
  ch.keys = reinterpret_cast<uint32_t*>(ws + sl.keys);
  ch.list = d_blocks ? d_blocks : reinterpret_cast<int32_t*>(ws + sl.list);
  ch.ids = reinterpret_cast<int32_t*>(ws + sl.ids);
  ch.top = top_blocks;
  ch.recent = recent_blocks;
  ch.list_row = d_blocks ? most : sl.places;
  ch.ids_row = sl.places;
  kvc::BlockAttn a = attention_of(sl.ws, d_workspace, sm_scale, softcap, d_slopes);
  a.list = ch.list;
  a.ids = ch.ids;
  a.most = most;
  a.list_row = ch.list_row;
  a.ids_row = ch.ids_row;
  split_pairs(c, &a, batch, units);
  a.early = 1;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const uint16_t* q = static_cast<const uint16_t*>(d_q);
  if (kvc::launch_block_choice(c->dev, c->bounds, ch, seq_begin, batch, longest, q, st) != cudaSuccess ||
      kvc::launch_block_selected(c->dev, seq_begin, batch, q, static_cast<uint16_t*>(d_out), a, st) != cudaSuccess)
    return KVC_ERR_CUDA;
  c->last_launches = 3;
  return KVC_OK;
}

size_t kvc_block_prefix_workspace_bytes(const kvc_block_cache* c, int32_t batch) {
  if (!c || batch <= 0 || batch > c->cfg.max_batch) return 0;
  return prefix_layout(c, batch).total;
}

kvc_status kvc_block_prefix_attention(kvc_block_cache* c, int32_t prefix, int32_t seq_begin, int32_t batch,
                                      const void* d_q, void* d_out, float sm_scale, float softcap,
                                      const float* d_slopes, void* d_workspace, size_t workspace_bytes, void* stream) {
  if (!c) return KVC_ERR_INVALID_ARG;
  c->last_launches = 0;
  if (!range_ok(c, seq_begin, batch) || !range_ok(c, prefix, 1) || (prefix >= seq_begin && prefix < seq_begin + batch))
    return KVC_ERR_INVALID_ARG;
  if (!attention_args_ok(d_q, d_out, sm_scale, softcap, d_slopes)) return KVC_ERR_INVALID_ARG;
  const PrefixLayout pl = prefix_layout(c, batch);
  if (!d_workspace || !aligned(d_workspace, kAlign) || workspace_bytes < pl.total) return KVC_ERR_INVALID_ARG;
  const int bt = c->cfg.block_tokens, hkv = c->cfg.num_kv_heads, shared = c->pos[prefix];
  const int tiles = (kvc::block_closed(shared, bt) * bt + kvc::kPrefixTile - 1) / kvc::kPrefixTile;
  // The product costs a launch and the join of its parts, the other form takes the
  // prefix's codes from L2 once per sequence (6.9 TB/s).  200 own tokens a sequence:
  // 8 x 32 heads after 260 / 2,050 / 8,200 tokens direct 10.1 / 15.8 / 29.9, product
  // 13.8 / 18.5 / 21.5 us; 64 x 32 after 520 / 1,030 direct 22.2 / 31.5, product 23.2 /
  // 26.0; 4 x 32 of 32 KV heads after 2,050 / 4,100 direct 20.3 / 29.7, product 21.2 /
  // 25.3.  Two sequences read it faster than it is converted: 2 x 32 of 32 KV heads
  // after 16,400 direct 49, product 60.
  const bool product = batch > 2 && (long long)batch * tiles * hkv > 2048;
  const long long front = (kvc::block_exact_rows(shared, bt) + kvc::kPage - 1) / kvc::kPage +
                          (product ? 0LL : (long long)kvc::block_closed(shared, bt) * (bt / kvc::kPage));
  long long units = 0;
  for (int i = 0; i < batch; ++i) {
    const int P = c->pos[seq_begin + i];
    if (P + (long long)shared <= 0 || P + (long long)shared > 2000000000LL) return KVC_ERR_INVALID_ARG;
    units += (kvc::block_units(P, bt) + front) * hkv;
  }
  kvc::BlockAttn a = attention_of(pl.ws, d_workspace, sm_scale, softcap, d_slopes);
  a.prefix = prefix;
  a.prefix_pages = product ? 0 : 1;
  split_pairs(c, &a, batch, units);
  a.early = product ? 1 : 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const uint16_t* q = static_cast<const uint16_t*>(d_q);
  if (product) {
    uint8_t* ws = static_cast<uint8_t*>(d_workspace);
    kvc::PrefixTc t{};
    t.more_o = reinterpret_cast<float*>(ws + pl.more_o);
    t.more_ml = reinterpret_cast<float*>(ws + pl.more_ml);
    t.mod = a.mod;
    t.qk_scale_log2 = a.qk_scale_log2;
    t.prefix = prefix;
    t.batch = batch;
    t.splits = prefix_splits((long long)(batch * c->dev.group + kvc::kPrefixRows - 1) / kvc::kPrefixRows * hkv, tiles);
    a.more = t.splits;
    a.more_o = t.more_o;
    a.more_ml = t.more_ml;
    if (kvc::launch_prefix_tc(c->dev, seq_begin, q, t, st) != cudaSuccess) return KVC_ERR_CUDA;
    c->last_launches = 1;
  }
  if (kvc::launch_block_prefix(c->dev, seq_begin, batch, q, static_cast<uint16_t*>(d_out), a, st) != cudaSuccess)
    return KVC_ERR_CUDA;
  ++c->last_launches;
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
