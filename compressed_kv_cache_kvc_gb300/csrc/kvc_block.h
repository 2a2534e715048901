// Internal declarations of the block-scaled cache (kvc_block.cu,
// kvc_block_host.cpp).  Not part of the ABI.
#pragma once

#include "kvc_internal.h"

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
  int parts;  // 0: equal runs across pairs; else a CTA takes a part of one pair, and the sequences of a head
                    // have about this many parts together
};

cudaError_t launch_block_append(const BlockState& s, int seq_begin, int batch, int n_new, const uint16_t* k,
                                const uint16_t* v, cudaStream_t st);
cudaError_t launch_block_release(const BlockState& s, int seq_begin, int batch, cudaStream_t st);
cudaError_t launch_block_read(const BlockState& s, int seq_begin, int batch, int pos_begin, int n, uint16_t* k,
                              uint16_t* v, cudaStream_t st);
cudaError_t launch_block_fill(const BlockState& s, cudaStream_t st);
int block_attention_ctas_per_sm(const BlockState& s, const ScoreMod& mod);
cudaError_t launch_block_attention(const BlockState& s, int seq_begin, int batch, const uint16_t* q, uint16_t* out,
                                   const BlockAttn& w, cudaStream_t st);

}  // namespace kvc
