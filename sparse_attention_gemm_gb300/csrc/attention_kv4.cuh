// attention_kv4.cuh -- what the two forms of the attention over the 4-bit cache share.
#pragma once

#include "attention_kv8.cuh"
#include "kv4.cuh"

namespace dsa {
namespace kv4_attn {

// Attention in groups of 16 or 32 heads (attention_kv4_narrow.cu): whether it takes a
// call, the heads of a group, the splits of a row's slots, and the launch.
bool narrow_takes(int T, int H, int Hc, int K);
int narrow_heads(int T, int H, int Hc);
int narrow_splits(int64_t units, int heads, int K);
int launch_narrow(const kv8_attn::Params& p, int T, int heads, int Dqk, bool separate, cudaStream_t stream);

}  // namespace kv4_attn
}  // namespace dsa
