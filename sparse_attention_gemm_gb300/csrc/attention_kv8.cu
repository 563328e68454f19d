// attention_kv8.cu -- sparse attention over the 8-bit block cache: the call.
// Groups of 64 query heads run attention_cache.cuh on a gather of E4M3 codes;
// calls with few heads per KV head or few rows go to attention_kv8_narrow.cu.
#include "attention_cache.cuh"

using namespace dsa::kv8_attn;

extern "C" size_t dsa_sparse_attn_fwd_kv8_workspace_size(int T, int H, int Hc, int Dqk, int Dv, int K) {
  if (!known_shape(T, H, Hc, Dqk, Dv, K) || narrow_takes(T, H, Hc, K)) return 0;
  const int s = plan_splits(units_of(T, H, Hc, kHG), K);
  return s == 1 ? 0 : part_bytes(T, H, s) + static_cast<size_t>(T) * H * s * Dv * sizeof(float);
}

extern "C" int dsa_sparse_attn_fwd_kv8(const void* q, const void* kv8, const float* kv_scale, const void* v8,
                                       const float* v_scale, const int32_t* idx, const int32_t* topk_length,
                                       const float* sink, const int32_t* cu_seqlens, const int32_t* block_table,
                                       int n_seqs, int T, int H, int Hc, int Dqk, int Dv, int K, int block,
                                       int n_blocks, int max_blocks, float scale, void* out, float* lse,
                                       float* lse_kv, float* max_logits, void* workspace, size_t ws_bytes,
                                       cudaStream_t stream) {
  dsa::clear_error();
  const size_t need = dsa_sparse_attn_fwd_kv8_workspace_size(T, H, Hc, Dqk, Dv, K);
  Params p;
  const int rc = fill(Call{"dsa_sparse_attn_fwd_kv8", "kv8", "v8", q, kv8, kv_scale, v8, v_scale, idx, topk_length,
                           sink, cu_seqlens, block_table, n_seqs, T, H, Hc, Dqk, Dv, K, block, n_blocks, max_blocks,
                           scale, out, lse, lse_kv, max_logits, workspace, ws_bytes, need, kHG, need > 0 ? plan_splits(units_of(T, H, Hc, kHG), K) : 1},
                      &p);
  if (rc != DSA_OK || T == 0) return rc;
  p.k8 = static_cast<const uint8_t*>(kv8);
  p.k_scale = kv_scale;
  p.v8 = static_cast<const uint8_t*>(v8 ? v8 : kv8);
  p.v_scale = v8 ? v_scale : kv_scale;
  if (narrow_takes(T, H, Hc, K)) return launch_narrow(p, T, Dqk, stream);
  if (need > 0) take_workspace(p, T, workspace);
  if (v8) return launch<Gather<256, 256, true>, 256, 256, true>(p, T, stream);
  return Dqk == 576 ? launch<Gather<576, 512, false>, 576, 512, false>(p, T, stream)
                    : launch<Gather<512, 512, false>, 512, 512, false>(p, T, stream);
}
