// attention_kv4.cu -- sparse attention over the 4-bit block cache.
//
// As over the 8-bit cache, with values e2m1(code) * 2^(byte - 127), a byte per 32
// elements of a row.  Such a value is a bf16 one, so a tile is widened on its
// way into shared memory, scales and all, and the products and the softmax of
// attention_cache.cuh run on it as on a bf16 cache: the roundings are those of the bf16
// call.  A row of 576 comes as 306 bytes.
#include "attention_cache.cuh"
#include "kv4.cuh"

namespace {

using namespace dsa::kv8_attn;

// Sixteen codes (piece `piece` of 128 dims) to two units of 16 bytes of row `key`
// of a chunk of 64 dims (lanes of the upper pieces store the second unit first,
// as in dsa::kv8_attn::widen).
__device__ __forceinline__ void widen4(uint2 c, uint32_t byte, uint8_t* chunk, int key, int piece) {
  const bool up = (piece & 4) != 0;
  const uint32_t f = dsa::bf2_of_scale(byte);
  uint32_t a[4], b[4];
  dsa::bf8_of_e2m1(up ? c.y : c.x, f, a);
  dsa::bf8_of_e2m1(up ? c.x : c.y, f, b);
  const int unit = (piece & 3) * 2 + (up ? 1 : 0);
  *reinterpret_cast<uint4*>(chunk + dsa::sw128_offset(key, unit * 16)) = make_uint4(a[0], a[1], a[2], a[3]);
  *reinterpret_cast<uint4*>(chunk + dsa::sw128_offset(key, (unit ^ 1) * 16)) = make_uint4(b[0], b[1], b[2], b[3]);
}

// The gather of a tile of 64 keys, as that of the 8-bit codes: thread gt takes
// piece (gt & 7) (16 codes, 8 bytes) of keys (gt >> 3) and (gt >> 3) + 32 of every 128 dims.
template <int DQK, int DV, bool SEP>
struct Gather4 {
  static constexpr int kWarps = 8, kThreads = kWarps * 32, kStep = kThreads / 8;
  static constexpr int kFull = DQK / 128, kNv = SEP ? DV / 128 : 0;
  static constexpr bool kTail = DQK % 128 != 0;
  static_assert(2 * kStep == kKeys, "a thread gathers two keys of a tile");
  uint2 k[kFull][2], v[SEP ? kNv : 1][2], tail;
  uint8_t ke[kFull][2], ve[SEP ? kNv : 1][2], tail_e;
  float have_any[2];

  __device__ __forceinline__ void load_keys(const Params& p, const int (&r)[2], int kvh, int piece) {
    const int rows = p.g.n_blocks << p.g.lb;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const bool have = r[s] >= 0 && dsa::check(r[s] < rows, p.status);
      const int64_t at = static_cast<int64_t>(have ? r[s] : 0) * p.Hc + kvh;
      const uint8_t* src = p.k8 + at * (DQK / 2) + piece * 8;
      const uint8_t* exp = p.k_exp + at * (DQK / 32) + (piece >> 1);
#pragma unroll
      for (int c = 0; c < kFull; ++c) {
        k[c][s] = have ? __ldcg(reinterpret_cast<const uint2*>(src + c * 64)) : make_uint2(0, 0);
        ke[c][s] = have ? __ldg(exp + c * 4) : 127;
      }
      have_any[s] = have ? 1.f : 0.f;
    }
    if (kTail) {  // its four pieces: threads with piece 0..3 take the first key's, the others the second's
      const int x = piece >= 4 ? r[1] : r[0];
      const bool have = x >= 0 && dsa::check(x < rows, p.status);
      const int64_t at = static_cast<int64_t>(have ? x : 0) * p.Hc + kvh;
      tail = have ? __ldcg(reinterpret_cast<const uint2*>(p.k8 + at * (DQK / 2) + kFull * 64 + (piece & 3) * 8))
                  : make_uint2(0, 0);
      tail_e = have ? __ldg(p.k_exp + at * (DQK / 32) + kFull * 4 + ((piece & 3) >> 1)) : 127;
    }
  }
  __device__ __forceinline__ void load_values(const Params& p, const int (&r)[2], int kvh, int piece) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const bool have = r[s] >= 0 && dsa::check(r[s] < (p.g.n_blocks << p.g.lb), p.status);
      const int64_t at = static_cast<int64_t>(have ? r[s] : 0) * p.Hc + kvh;
#pragma unroll
      for (int c = 0; c < kNv; ++c) {
        v[c][s] = have ? __ldcg(reinterpret_cast<const uint2*>(p.v8 + at * (DV / 2) + c * 64 + piece * 8))
                       : make_uint2(0, 0);
        ve[c][s] = have ? __ldg(p.v_exp + at * (DV / 32) + c * 4 + (piece >> 1)) : 127;
      }
    }
  }
  // meta: 1 for each slot's key and, behind them, value; 0: no slot.
  __device__ __forceinline__ void store_keys(uint8_t* buf, float* meta, int key0, int piece) const {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int c = 0; c < kFull; ++c)
        widen4(k[c][s], ke[c][s], buf + (2 * c + (piece >> 2)) * kChunkBytes, key0 + s * kStep, piece);
    if (kTail) widen4(tail, tail_e, buf + 2 * kFull * kChunkBytes, key0 + (piece >> 2) * kStep, piece);
    if (piece < (SEP ? 4 : 2)) meta[(piece >> 1) * kKeys + (piece & 1) * kStep + key0] = have_any[piece & 1];
  }
  __device__ __forceinline__ void store_values(uint8_t* buf, int key0, int piece) const {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int c = 0; c < kNv; ++c)
        widen4(v[c][s], ve[c][s], buf + (2 * c + (piece >> 2)) * kChunkBytes, key0 + s * kStep, piece);
  }
};

}  // namespace

extern "C" size_t dsa_sparse_attn_fwd_kv4_workspace_size(int T, int H, int Hc, int Dqk, int Dv, int K) {
  if (!known_shape(T, H, Hc, Dqk, Dv, K)) return 0;
  const int s = plan_splits(units_of(T, H, Hc), K);
  return s == 1 ? 0 : part_bytes(T, H, s) + static_cast<size_t>(T) * H * s * Dv * sizeof(float);
}

extern "C" int dsa_sparse_attn_fwd_kv4(const void* q, const void* kv4, const uint8_t* kv_scale, const void* v4,
                                       const uint8_t* v_scale, const int32_t* idx, const int32_t* topk_length,
                                       const float* sink, const int32_t* cu_seqlens, const int32_t* block_table,
                                       int n_seqs, int T, int H, int Hc, int Dqk, int Dv, int K, int block,
                                       int n_blocks, int max_blocks, float scale, void* out, float* lse,
                                       float* lse_kv, float* max_logits, void* workspace, size_t ws_bytes,
                                       cudaStream_t stream) {
  dsa::clear_error();
  const size_t need = dsa_sparse_attn_fwd_kv4_workspace_size(T, H, Hc, Dqk, Dv, K);
  Params p;
  const int rc = fill(Call{"dsa_sparse_attn_fwd_kv4", "kv4", "v4", q, kv4, kv_scale, v4, v_scale, idx, topk_length,
                           sink, cu_seqlens, block_table, n_seqs, T, H, Hc, Dqk, Dv, K, block, n_blocks, max_blocks,
                           scale, out, lse, lse_kv, max_logits, workspace, ws_bytes, need},
                      &p);
  if (rc != DSA_OK || T == 0) return rc;
  p.k8 = static_cast<const uint8_t*>(kv4);
  p.k_exp = kv_scale;
  p.v8 = static_cast<const uint8_t*>(v4);
  p.v_exp = v_scale;
  if (v4) return launch<Gather4<256, 256, true>, 256, 256, true>(p, T, stream);
  return Dqk == 576 ? launch<Gather4<576, 512, false>, 576, 512, false>(p, T, stream)
                    : launch<Gather4<512, 512, false>, 512, 512, false>(p, T, stream);
}
