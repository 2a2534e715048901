// Attention of sequences that share a prefix: softmax over the prefix's tokens,
// held once, and each sequence's own.
#include "kvc_block_attn.h"

namespace kvc {

int block_prefix_ctas_per_sm(const BlockState& s, const ScoreMod& mod) { return attn_ctas<kPrefix>(s, mod); }

cudaError_t launch_block_prefix(const BlockState& s, int seq_begin, int batch, const uint16_t* q, uint16_t* out,
                                const BlockAttn& w, cudaStream_t st) {
  return attn_launch<kPrefix>(s, seq_begin, batch, q, out, w, st);
}

}  // namespace kvc
