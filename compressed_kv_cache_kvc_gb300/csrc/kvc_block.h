// Internal declarations of the block-scaled cache (kvc_block.cu,
// kvc_block_host.cpp).  Not part of the ABI.
#pragma once

#include "kvc_internal.h"
#include "kvc_rotary.h"

namespace kvc {

// Device view of one layer's block-scaled cache (by value in kernel arguments).
struct BlockState {
  uint8_t* k_codes;   // [num_blocks][hkv][bt][128]
  uint8_t* v_codes;
  float* k_scale;     // [num_blocks][hkv]
  float* v_scale;
  uint16_t* k_exact;  // [max_batch][hkv][4 + bt][128] bf16: sinks, then the open block
  uint16_t* v_exact;
  int32_t* table;     // [max_batch][max_bps]
  int32_t* seq_pos;   // [max_batch]
  int32_t* free_stack;
  int32_t* counters;  // [0] free top, [1] status
  int32_t* tickets;   // [max_batch * hkv] attention, one append; zero between calls
  int32_t hq, hkv, group, bt, num_blocks, max_batch, max_bps, fp8;
};

// Bounds of every block's keys (the caller's memory; codes null: none are kept):
// per channel the least and the largest INT8 code of the block's keys.
struct KeyBounds {
  uint8_t* codes;  // [num_blocks][hkv][2][128]
  float* scale;    // [num_blocks][hkv], amax / 127
};

// A sequence of P tokens: closed (quantised) blocks, rows held exactly (the
// sinks, then the open block's tokens).
__host__ __device__ inline int block_closed(int P, int bt) { return P > kSinks ? (P - kSinks) / bt : 0; }
__host__ __device__ inline int block_exact_rows(int P, int bt) {
  return P <= kSinks ? P : kSinks + (P - kSinks) % bt;
}
// 16-token units of the attention: the closed blocks' pages, then the exact rows.
__host__ __device__ inline int block_units(int P, int bt) {
  return block_closed(P, bt) * (bt / kPage) + (block_exact_rows(P, bt) + kPage - 1) / kPage;
}

// Sequences of a call that cuts its CTAs to the pairs (their table shares the
// shared memory with three CTAs' rings).
constexpr int kMaxSplitBatch = 255;

struct BlockAttn {
  // (at most ncta + pairs parts, however they are cut)
  float* part_o;   // [pairs + ncta][group][128], divided by their sums
  float* part_ml;  // [pairs + ncta][group][2]: maximum, sum
  ScoreMod mod;
  float qk_scale_log2;
  int ncta;
  // the selected form: up to `most` blocks of every pair in ascending order and where they
  // lie in the pool, list_row and ids_row places a pair
  const int32_t *list, *ids;
  int most, list_row, ids_row;
  // the prefix form: the sequence that holds it, whether its pages are among the
  // units; partials of its blocks from elsewhere, `more` of [hkv][batch][group]
  int prefix, prefix_pages, more;
  const float *more_o, *more_ml;
  int early;       // (those two) launched under the kernel before them
  int part_units;  // (those two) units of a part at least; `parts` of them at most per pair
  // 0: equal runs across pairs; else a CTA takes a part of one pair, and the sequences of
  // a head have about this many parts together
  int parts;
};

// The choice of blocks: the top_blocks best of the closed ones but the `recent`
// newest, and these.
struct BlockChoice {
  uint32_t* keys;  // [pairs][max_bps], ordered as the scores
  int32_t* list;   // [pairs][list_row], ascending, -1 behind the last
  int32_t* ids;    // [pairs][ids_row] their blocks in the pool
  int top, recent, list_row, ids_row;
};

cudaError_t launch_block_append(const BlockState& s, const KeyBounds& bounds, int seq_begin, int batch, int n_new,
                                const uint16_t* k, const uint16_t* v, cudaStream_t st);
int block_append_rotary_launches(const RotaryArgs& rot);
cudaError_t launch_block_append_rotary(const BlockState& s, const KeyBounds& bounds, int seq_begin,
                                       const RotaryArgs& rot, const RowsIn& v, cudaStream_t st);
cudaError_t launch_block_release(const BlockState& s, int seq_begin, int batch, cudaStream_t st);
cudaError_t launch_block_read(const BlockState& s, int seq_begin, int batch, int pos_begin, int n, uint16_t* k,
                              uint16_t* v, cudaStream_t st);
cudaError_t launch_block_fill(const BlockState& s, cudaStream_t st);
int block_attention_ctas_per_sm(const BlockState& s, const ScoreMod& mod);
cudaError_t launch_block_attention(const BlockState& s, int seq_begin, int batch, const uint16_t* q, uint16_t* out,
                                   const BlockAttn& w, cudaStream_t st);

// longest: the most tokens a sequence of the slice holds
cudaError_t launch_block_choice(const BlockState& s, const KeyBounds& bounds, const BlockChoice& ch, int seq_begin,
                                int batch, int longest, const uint16_t* q, cudaStream_t st);
cudaError_t launch_block_selected(const BlockState& s, int seq_begin, int batch, const uint16_t* q, uint16_t* out,
                                  const BlockAttn& w, cudaStream_t st);
// The products of all query rows with a prefix's closed blocks: `splits` runs of
// them per KV head, a partial result of every row each.
struct PrefixTc {
  float *more_o, *more_ml;  // [splits][hkv][batch][group][128], [..][2]
  ScoreMod mod;
  float qk_scale_log2;
  int prefix, batch, splits;
};
constexpr int kPrefixRows = 256, kPrefixTile = 128;  // query rows of a CTA, tokens of a tile
cudaError_t launch_prefix_tc(const BlockState& s, int seq_begin, const uint16_t* q, const PrefixTc& a,
                             cudaStream_t st);
cudaError_t launch_block_prefix(const BlockState& s, int seq_begin, int batch, const uint16_t* q, uint16_t* out,
                                const BlockAttn& w, cudaStream_t st);

}  // namespace kvc
