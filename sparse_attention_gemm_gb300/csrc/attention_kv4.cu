// attention_kv4.cu -- sparse attention over the 4-bit block cache.
//
// As over the 8-bit cache, with values e2m1(code) * 2^(byte - 127), a byte per 32
// elements of a row.  Such a value is a bf16 one, so a tile is widened on its
// way into shared memory, scales and all, and the products and the softmax of
// attention_cache.cuh run on it as on a bf16 cache: the roundings are those of the bf16
// call.  A row of 576 comes as 306 bytes.
//
// Three forms, by rules on the call's sizes (narrow_splits, widens):
// * tiles: groups of 64 heads, each row's codes widened on their way (attention_cache.cuh).
//   2048 rows of 64 heads, 2048 slots, 576 dims: 889 us, 657 TFLOP/s.  The gather bounds it: a
//   warp's conversion of its part of a tile takes 1.5K cycles and its loads' issue 1.8K, where the products take 2.2K.
//   Slower: two hand-overs a tile (977 where 938), the loads two tiles ahead (1042), scale bytes by
//   shuffles (987 where 890), loads past L1 (900 to 926).
// * narrow: groups of 16 heads, warp products (attention_kv4_narrow.cu).
// * widened: a cache whose rows are read often is written out in bf16 once and the call is the
//   bf16 one (attention.cu), which such a call comes close to: the same 2048 rows over 16,384 cache rows
//   681 us, 857 TFLOP/s, of which widening takes 4 and the positions' rows 10.
#include "attention_cache.cuh"
#include "attention_kv4.cuh"

namespace {

using namespace dsa::kv8_attn;

// 32 codes with their scale byte, dims 32 * piece to 32 * piece + 31 of four chunks of 64 dims, to row `key` of the
// piece's chunk.  Eight lanes (a key) hold two pieces of each chunk: a lane begins with the unit of 16 bytes that its chunk's
// number says, so that they touch all banks once.  Of each eight dims, element i stands at place 2i and
// element i + 4 behind it, as they come out of a word: neighbours would cost a third of the instructions more, and
// integer ones, which an SM issues half as many of, are what a tile's conversion takes its time with.  The query's
// elements lie in the same order (kPlaced), and results are put back as they are written.
// direct: no byte of the warp's is above kMxDirect.
__device__ __forceinline__ void widen8(uint32_t w, uint32_t f, uint32_t f2, bool direct, uint8_t* to) {
  uint32_t x[4];
  dsa::e2m1_raw(w, x);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = dsa::mul_bf16x2(x[i], f);
  if (!direct) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = dsa::mul_bf16x2(x[i], f2);
  }
  *reinterpret_cast<uint4*>(to) = make_uint4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void widen32(uint4 c, uint32_t byte, bool direct, uint8_t* chunks, int key, int piece) {
  const int turn = piece >> 1;
  const bool t1 = turn & 1, t2 = turn & 2;
  const uint32_t a[4] = {t1 ? c.y : c.x, t1 ? c.z : c.y, t1 ? c.w : c.z, t1 ? c.x : c.w};
  const uint32_t w[4] = {t2 ? a[2] : a[0], t2 ? a[3] : a[1], t2 ? a[0] : a[2], t2 ? a[1] : a[3]};
  const uint32_t f = dsa::mx_factor(byte), f2 = direct ? 0 : dsa::mx_second(byte);
  uint8_t* chunk = chunks + turn * kChunkBytes;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    widen8(w[j], f, f2, direct, chunk + dsa::sw128_offset(key, ((piece & 1) * 4 + ((j + turn) & 3)) * 16));
}

// The gather of a tile of 64 keys by eight warps: thread gt takes piece (gt & 7) (32 codes, 16
// bytes, one scale) of keys (gt >> 3) and (gt >> 3) + 32 of every 256 dims; of the last 64 of 576 the
// threads with piece 0..3 take 16 codes each of the first key, the others of the second.
template <int DQK, int DV, bool SEP>
struct Gather4 {
  static constexpr int kWarps = 8, kThreads = kWarps * 32, kStep = kThreads / 8;
  static constexpr bool kScaled = false, kPlaced = true;
  static constexpr int kM = DQK / 256;
  static constexpr bool kTail = DQK % 256 != 0;
  static_assert(2 * kStep == kKeys, "a thread gathers two keys of a tile");
  static_assert(SEP ? kM == 1 && DV == 256 : kM == 2 && DV == 512, "pieces");
  uint4 k[kM][2], v[2];
  uint2 tail;
  uint32_t ke[kM][2], ve[2], tail_e;
  bool have[2];

  __device__ __forceinline__ void load_keys(const Params& p, const int (&r)[2], int kvh, int piece) {
    const int rows = p.g.n_blocks << p.g.lb;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      have[s] = r[s] >= 0 && dsa::check(r[s] < rows, p.status);
      const int64_t at = static_cast<int64_t>(have[s] ? r[s] : 0) * p.Hc + kvh;
      const uint8_t* src = p.k8 + at * (DQK / 2) + piece * 16;
      const uint8_t* exp = p.k_exp + at * (DQK / 32) + piece;
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        k[m][s] = have[s] ? __ldcg(reinterpret_cast<const uint4*>(src + m * 128)) : make_uint4(0, 0, 0, 0);
        ke[m][s] = have[s] ? __ldg(exp + m * 8) : 0;
      }
    }
    if (kTail) {
      const bool any = piece >= 4 ? have[1] : have[0];
      const int64_t at = static_cast<int64_t>(any ? (piece >= 4 ? r[1] : r[0]) : 0) * p.Hc + kvh;
      tail = any ? __ldcg(reinterpret_cast<const uint2*>(p.k8 + at * (DQK / 2) + kM * 128 + (piece & 3) * 8))
                 : make_uint2(0, 0);
      tail_e = any ? __ldg(p.k_exp + at * (DQK / 32) + kM * 8 + ((piece & 3) >> 1)) : 0;
    }
  }
  __device__ __forceinline__ void load_values(const Params& p, const int (&r)[2], int kvh, int piece) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int64_t at = static_cast<int64_t>(have[s] ? r[s] : 0) * p.Hc + kvh;
      v[s] = have[s] ? __ldcg(reinterpret_cast<const uint4*>(p.v8 + at * (DV / 2) + piece * 16)) : make_uint4(0, 0, 0, 0);
      ve[s] = have[s] ? __ldg(p.v_exp + at * (DV / 32) + piece) : 0;
    }
  }

  // Whether no byte of the warp's tile is above kMxDirect (values up to 12: the usual case).
  __device__ __forceinline__ bool direct() const {
    uint32_t m = kTail ? tail_e : 0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int i = 0; i < kM; ++i) m = max(m, ke[i][s]);
      if (SEP) m = max(m, ve[s]);
    }
    return !__any_sync(0xffffffffu, m > dsa::kMxDirect);
  }
  // meta: 1 for each slot, 0: no slot.
  __device__ __forceinline__ void store_keys(uint8_t* tile, float* meta, int key0, int piece) const {
    const bool d = direct();
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int m = 0; m < kM; ++m) widen32(k[m][s], ke[m][s], d, tile + m * 4 * kChunkBytes, key0 + s * kStep, piece);
    if (kTail) {  // eight lanes hold four units of two keys' rows: upper ones store their second unit first
      const bool up = (piece & 2) != 0;
      const uint32_t f = dsa::mx_factor(tail_e), f2 = d ? 0 : dsa::mx_second(tail_e);
      const int key = key0 + (piece >> 2) * kStep, unit = (piece & 3) * 2 + (up ? 1 : 0);
      uint8_t* chunk = tile + 4 * kM * kChunkBytes;
      widen8(up ? tail.y : tail.x, f, f2, d, chunk + dsa::sw128_offset(key, unit * 16));
      widen8(up ? tail.x : tail.y, f, f2, d, chunk + dsa::sw128_offset(key, (unit ^ 1) * 16));
    }
    if (piece < 2) meta[piece * kStep + key0] = have[piece] ? 1.f : 0.f;
  }
  __device__ __forceinline__ void store_values(uint8_t* values, int key0, int piece) const {
    const bool d = direct();
#pragma unroll
    for (int s = 0; s < 2; ++s) widen32(v[s], ve[s], d, values, key0 + s * kStep, piece);
  }
};

// ---- the cache widened once, and the attention over bf16 rows on that
constexpr int kWideThreads = 256, kWidePieces = 4;

// Codes of 8 values a piece, with their scale bytes, to bf16 in the order in which they lie.
__global__ void __launch_bounds__(kWideThreads) kv4_widen_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scale,
                                                                 int64_t n, uint4* __restrict__ out) {
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kWideThreads * kWidePieces) + threadIdx.x;
  uint32_t w[kWidePieces], e[kWidePieces];
#pragma unroll
  for (int j = 0; j < kWidePieces; ++j) {
    const int64_t i = i0 + j * kWideThreads;
    w[j] = i < n ? __ldcs(codes + i) : 0;
    e[j] = i < n ? __ldg(scale + (i >> 2)) : 0;
  }
#pragma unroll
  for (int j = 0; j < kWidePieces; ++j) {
    uint32_t o[4];
    dsa::bf8_of_e2m1(w[j], e[j], o);
    const int64_t i = i0 + j * kWideThreads;
    if (i < n) out[i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// Cache rows of positions and the rows' lengths, 0 for padding: one CTA a query row, whose sequence each warp looks up.  Eight ids of a
// thread are under way at a time: their pages are loads that wait for loads.
__global__ void __launch_bounds__(kWideThreads) kv4_rows_kernel(const int32_t* __restrict__ idx, const dsa::Kv8Geom g, int K,
                                                                const int32_t* __restrict__ topk_length,
                                                                int32_t* __restrict__ rows, int32_t* __restrict__ length,
                                                                uint32_t* status) {
  const int t = blockIdx.x;
  const bool padding = t >= __ldg(g.cu + g.n_seqs);
  if (threadIdx.x == 0) length[t] = padding ? 0 : topk_length ? __ldg(topk_length + t) : K;
  if (padding) return;
  const int b = dsa::kv8_seq_warp(g.cu, g.n_seqs, t);
  const int64_t at = static_cast<int64_t>(t) * K;
  constexpr int kAhead = 8;
  for (int j0 = threadIdx.x; j0 < K; j0 += kWideThreads * kAhead) {
    int id[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int j = j0 + k * kWideThreads;
      id[k] = j < K ? __ldcs(idx + at + j) : -1;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      id[k] = id[k] < 0 ? -1 : dsa::kv8_row(g, b, id[k]);
      if (!dsa::check(id[k] < (g.n_blocks << g.lb), status)) id[k] = -1;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int j = j0 + k * kWideThreads;
      if (j < K) rows[at + j] = id[k];
    }
  }
}

struct WideSizes {
  size_t k, v, rows, length;  // bytes of the widened keys, the values, the ids and the rows' lengths
};
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
WideSizes widened_sizes(int T, int Dqk, int Dv, int K, int64_t cache_rows, bool paged) {
  return WideSizes{up256(static_cast<size_t>(cache_rows) * Dqk * 2), Dqk == 256 ? up256(static_cast<size_t>(cache_rows) * Dv * 2) : 0,
                   paged ? up256(static_cast<size_t>(T) * K * 4) : 0, paged ? up256(static_cast<size_t>(T) * 4) : 0};
}

// Whether the cache is widened once for the call.  Measured (576 dims, 64 heads): the tiles' own
// conversion costs 0.05 ns a slot and group of 64 heads over the bf16 kernel (2048 rows of 2048 slots 889 us
// against 681), widening 0.27 ns a cache row and the launches 8 us; taken where the first is
// twice the second, for a widened cache of at most 2^30 bytes.  (The cache is all of its blocks: which of them the batch's table
// names is device data.  2048 rows of 2048 slots: 682 us with up to some 359,000 cache rows, 884 beyond them.)
bool widens(int T, int H, int Hc, int Dqk, int Dv, int K, int64_t cache_rows) {
  const double slots = static_cast<double>(T) * K * ((H + kHG - 1) / kHG);
  return Hc == 1 && slots >= 10.8 * cache_rows + 320e3 && cache_rows * (Dqk == 256 ? Dqk + Dv : Dqk) <= (int64_t{1} << 29);
}

int launch_widened(const Params& p, const void* q, int T, int Dqk, int Dv, float scale, int sms, void* workspace, cudaStream_t stream) {
  const int64_t cache_rows = static_cast<int64_t>(p.g.n_blocks) << p.g.lb;
  const bool separate = Dqk == 256, paged = p.g.table != nullptr;
  const WideSizes size = widened_sizes(T, Dqk, Dv, p.K, cache_rows, paged);
  auto* ws = static_cast<uint8_t*>(workspace);
  auto widen = [&](const uint8_t* codes, const uint8_t* exp, int dim, uint8_t* to) {
    const int64_t n = cache_rows * (dim / 8);
    const unsigned grid = static_cast<unsigned>((n + kWideThreads * kWidePieces - 1) / (kWideThreads * kWidePieces));
    kv4_widen_kernel<<<grid, kWideThreads, 0, stream>>>(reinterpret_cast<const uint32_t*>(codes), exp, n, reinterpret_cast<uint4*>(to));
    return dsa::launch_error("kv4_widen_kernel");
  };
  int rc = widen(p.k8, p.k_exp, Dqk, ws);
  if (rc == DSA_OK && separate) rc = widen(p.v8, p.v_exp, Dv, ws + size.k);
  const int32_t *rows = p.idx, *length = p.topk_length;
  if (rc == DSA_OK && paged) {
    auto* to = reinterpret_cast<int32_t*>(ws + size.k + size.v);
    auto* len = reinterpret_cast<int32_t*>(ws + size.k + size.v + size.rows);
    kv4_rows_kernel<<<T, kWideThreads, 0, stream>>>(p.idx, p.g, p.K, p.topk_length, to, len, p.status);
    rc = dsa::launch_error("kv4_rows_kernel");
    rows = to, length = len;
  }
  if (rc != DSA_OK) return rc;
  return dsa::sparse_attn_launch(q, ws, separate ? ws + size.k : nullptr, rows, length, p.sink, T, static_cast<int>(cache_rows),
                                 p.H, Dqk, Dv, p.K, scale, p.out, p.lse, p.lse_kv, p.max_logits, 0, nullptr,
                                 paged ? p.g.cu + p.g.n_seqs : nullptr, sms, stream);
}

// Joining as tiles: fewer than over 8-bit codes, whose tiles take 1 us where these take 1.75 (26 rows of 64 heads, 350
// slots: 20.1 us in one CTA a row, 17.3 in five).
constexpr int kJoinTiles4 = 2;

// How a call of a known shape is worked: heads of a group, splits of a row's slots and the workspace's bytes.
struct Plan {
  enum { kTiles, kNarrow, kWidened } form;
  int heads, splits;
  size_t bytes;
};
Plan plan_of(int T, int H, int Hc, int Dqk, int Dv, int K, int64_t cache_rows, bool paged) {
  if (const int n = dsa::kv4_attn::narrow_splits(T, H, Hc, Dqk, K)) return Plan{Plan::kNarrow, 16, n, 0};
  if (widens(T, H, Hc, Dqk, Dv, K, cache_rows)) {
    const WideSizes s = widened_sizes(T, Dqk, Dv, K, cache_rows, paged);
    return Plan{Plan::kWidened, kHG, 1, s.k + s.v + s.rows + s.length};
  }
  const int s = plan_splits(units_of(T, H, Hc, kHG), K, kJoinTiles4);
  return Plan{Plan::kTiles, kHG, s, s == 1 ? 0 : part_bytes(T, H, s) + static_cast<size_t>(T) * H * s * Dv * sizeof(float)};
}

}  // namespace

extern "C" size_t dsa_sparse_attn_fwd_kv4_workspace_size(int T, int H, int Hc, int Dqk, int Dv, int K, int block,
                                                         int n_blocks, int paged) {
  if (!known_shape(T, H, Hc, Dqk, Dv, K) || block < 1 || n_blocks < 1) return 0;
  return plan_of(T, H, Hc, Dqk, Dv, K, static_cast<int64_t>(n_blocks) * block, paged != 0).bytes;
}

extern "C" int dsa_sparse_attn_fwd_kv4(const void* q, const void* kv4, const uint8_t* kv_scale, const void* v4,
                                       const uint8_t* v_scale, const int32_t* idx, const int32_t* topk_length,
                                       const float* sink, const int32_t* cu_seqlens, const int32_t* block_table,
                                       int n_seqs, int T, int H, int Hc, int Dqk, int Dv, int K, int block,
                                       int n_blocks, int max_blocks, float scale, void* out, float* lse,
                                       float* lse_kv, float* max_logits, void* workspace, size_t ws_bytes,
                                       cudaStream_t stream) {
  dsa::clear_error();
  const Plan plan = known_shape(T, H, Hc, Dqk, Dv, K) && block >= 1 && n_blocks >= 1
                        ? plan_of(T, H, Hc, Dqk, Dv, K, static_cast<int64_t>(n_blocks) * block, block_table != nullptr)
                        : Plan{Plan::kTiles, kHG, 1, 0};
  // (the scales of a row are copied in words)
  if (!dsa::aligned(kv_scale, 16) || !dsa::aligned(v_scale, 16))
    return dsa::set_error(DSA_ERR_VALUE, "dsa_sparse_attn_fwd_kv4: kv_scale and v_scale must be 16-byte aligned");
  Params p;
  int sms = 0;
  const int rc = fill(Call{"dsa_sparse_attn_fwd_kv4", "kv4", "v4", q, kv4, kv_scale, v4, v_scale, idx, topk_length,
                           sink, cu_seqlens, block_table, n_seqs, T, H, Hc, Dqk, Dv, K, block, n_blocks, max_blocks,
                           scale, out, lse, lse_kv, max_logits, workspace, ws_bytes, plan.bytes, plan.heads, plan.splits},
                      &p, &sms);
  if (rc != DSA_OK || T == 0) return rc;
  p.k8 = static_cast<const uint8_t*>(kv4);
  p.k_exp = kv_scale;
  p.v8 = static_cast<const uint8_t*>(v4);
  p.v_exp = v_scale;
  if (plan.form == Plan::kNarrow) return dsa::kv4_attn::launch_narrow(p, T, Dqk, stream);
  if (plan.form == Plan::kWidened) return launch_widened(p, q, T, Dqk, Dv, scale, sms, workspace, stream);
  if (plan.bytes > 0) take_workspace(p, T, workspace);
  if (v4) return launch<Gather4<256, 256, true>, 256, 256, true>(p, T, stream);
  return Dqk == 576 ? launch<Gather4<576, 512, false>, 576, 512, false>(p, T, stream)
                    : launch<Gather4<512, 512, false>, 512, 512, false>(p, T, stream);
}
