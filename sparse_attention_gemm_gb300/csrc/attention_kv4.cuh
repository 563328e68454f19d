// attention_kv4.cuh -- what the two forms of the attention over the 4-bit cache share.
#pragma once

#include "attention_kv8.cuh"
#include "kv4.cuh"

namespace dsa {

// The attention over bf16 rows (attention.cu) of a call whose arguments are checked.  t_end: NULL, or rows from
// *t_end on are left alone; their topk_length is 0 (asked in the loops of all rows the end cost the bf16 call 2%).
int sparse_attn_launch(const void* q, const void* kv, const void* v, const int32_t* idx, const int32_t* topk_length,
                       const float* sink, int T, int Tkv, int H, int Dqk, int Dv, int K, float scale, void* out, float* lse,
                       float* lse_kv, float* max_logits, int indexer_topk, float* lse_indexer, const int32_t* t_end, int sms,
                       cudaStream_t stream);

namespace kv4_attn {

// Attention in groups of 16 heads (attention_kv4_narrow.cu): the splits of a row's slots in a call that it
// takes, 0 in others, and the launch.
int narrow_splits(int T, int H, int Hc, int Dqk, int K);
int launch_narrow(const kv8_attn::Params& p, int T, int Dqk, cudaStream_t stream);

}  // namespace kv4_attn
}  // namespace dsa
