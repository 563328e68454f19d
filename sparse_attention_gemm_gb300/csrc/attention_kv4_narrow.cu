// attention_kv4_narrow.cu -- sparse attention over the 4-bit block cache for few
// query heads per KV head, or few rows.
//
// For row t, the heads of a group and valid slot j (see attention_kv4.cu): s_j = scale * q . k_j,
// out = sum_j exp(s_j) v_j / (sum_j exp(s_j) + exp(sink)).
//
// Here a tile's conversion is most of the work, and its way through shared memory into a
// tcgen05 product would be the rest: 64 bytes stored and read again for every 32 of codes.  So codes are
// widened straight into the operands of warp-level products (m16n8k16, bf16 in, fp32 sums):
// * scores: a lane takes 32 codes of a key, which share a scale, as its part of eight steps of 16 dims.  Which dims
//   meet in a step does not matter as long as the query lies in the same order, and it is laid out so.
// * values: a lane takes eight dims of the four keys of a step; its codes of two keys are paired by a byte permute.
// A CTA of eight warps goes through tiles of 64 keys: a warp scores eight of them, the softmax's reference (the
// running maximum of each head) is agreed on through shared memory, and a warp adds up 64 value dims
// (of 256 dims: of one half of the keys).  Raw codes arrive by cp.async, a tile ahead; three barriers a
// tile (with one for the stage's end besides, 37.6 us where 36.8).
//
// Why warp products: 16 heads fill a quarter of the tcgen05 tile's columns (N = 64), whose operands
// have to be stored and read all the same.  What bounds it is the issue of instructions (58 to 65%, the
// tensor pipe 16 to 25%): eight codes take 17 to become bf16 values.  96 rows of 2 x 12 heads, 1027 slots,
// 256 dims: 37 us, 1.3 TB/s of codes, of which SMs with three CTAs work all the time and those with two 4/5
// of it; on the tiles of 64 heads 59.  One row of 16 heads, 2048 slots, 576 dims: 12.8 us; on the tiles 15.8.
// Slower: tiles of 128 keys (73 us where 46), two CTAs an SM (51 where 41), loops that are not unrolled, pairing
// values instead of codes (39.8 where 38.9); groups of 32 heads were never ahead of the tiles.
//
// Work item = (token, KV head, group of 16 heads, split of its slots); a row's splits are the CTAs of a
// cluster and are joined there: no workspace, no second launch, nothing that waits on another cluster.
#include <algorithm>

#include "attention_kv4.cuh"

namespace {

using namespace dsa::kv8_attn;

constexpr int kTile = 64;  // keys
constexpr int kWarps = 8, kBlock = kWarps * 32;
static_assert(kTile == 8 * kWarps, "a warp scores eight keys");
constexpr int kRowRing = 4;
constexpr int kMaxCluster = 16;  // splits of a row's slots are the CTAs of a cluster

template <int DQK, int DV, bool SEP>
struct Narrow {
  static constexpr int kHeads = 16;
  static constexpr uint32_t kQPitch = DQK * 2 + 16;  // an odd number of 16-byte units: ldmatrix without conflicts
  // a key's codes, 32 bytes on from a multiple of 128: scores read 64 bytes of keys two apart at a time, values 32 of four in a
  // row, and neither meet in a bank
  static constexpr uint32_t kKPitch = DQK / 2 + (DQK == 576 ? 0 : 32), kVPitch = SEP ? DV / 2 + 32 : kKPitch;
  static_assert(kKPitch % 128 == 32 && kVPitch % 128 == 32, "banks");
  static constexpr uint32_t kVAt = SEP ? kTile * kKPitch : 0;
  static constexpr uint32_t kScaleAt = kTile * kKPitch + (SEP ? kTile * kVPitch : 0);  // 32 bytes a key
  static constexpr uint32_t kMetaAt = kScaleAt + kTile * 32;  // a byte a key: 1 there, + 2: its scales begin two bytes on
  static constexpr uint32_t kStage = kMetaAt + kTile;
  static constexpr uint32_t kStages = kHeads * kQPitch;                 // [2], behind the query
  static constexpr int kBlocksV = DV / 32;
  static constexpr uint32_t kFPitch = kTile * 2 + 16;                   // factors of a value block's keys (bf16), in
  static constexpr uint32_t kFactors = kStages + 2 * kStage;            // the order of the weights
  static constexpr uint32_t kPPitch = kTile * 2 + 16;
  static constexpr uint32_t kP = (kFactors + kBlocksV * kFPitch + 15) / 16 * 16;  // weights [heads][keys]
  static constexpr uint32_t kRows = kP + kHeads * kPPitch;              // int [kRowRing][kTile]
  // float [heads][warps], of which eight lanes at a time read 16 bytes each, of eight heads: kWPitch floats a
  // head, and no two of them in a bank
  static constexpr uint32_t kWmax = kRows + kRowRing * kTile * 4;
  static constexpr int kWPitch = 12;
  // what a CTA of a cluster leaves for the others: mean values [heads][DV] over the query and the stages, and
  // float4 [heads]: reference, sum, maximum
  static constexpr uint32_t kStats = kWmax + kHeads * kWPitch * 4;
  static constexpr uint32_t kShares = kStats + kHeads * 16;  // float [heads][kMaxCluster]
  static constexpr uint32_t kTotal = kShares + kHeads * kMaxCluster * 4;
  static_assert(kHeads * DV * 4 <= kFactors, "mean values");
  // CTAs of an SM, by their shared memory (228 KB of it, 1 KB of each the system's)
  static constexpr int kPerSm = kTotal <= 75 * 1024 ? 3 : kTotal <= 113 * 1024 ? 2 : 1;
  static_assert(kTotal <= 227 * 1024 && kStage % 16 == 0 && kStages % 16 == 0 && kP % 16 == 0 && kWmax % 16 == 0, "shared memory");
  // value dims: 64 a warp; with 256, two halves of the keys
  static constexpr int kSlices = DV / 64, kHalves = kWarps / kSlices;
  static_assert(kHalves == 1 || kHeads * DV * 4 <= 2 * kStage, "the halves' sums meet in the stages");
};

// Every thread of every CTA of the cluster arrives, on every path.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster(uint32_t smem_addr, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr), "r"(rank));
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Eight codes times the factor(s) of their scale byte: x[i] = elements i and i + 4.
template <bool DIRECT>
__device__ __forceinline__ void widen_word(uint32_t w, uint32_t f, uint32_t f2, uint32_t (&x)[4]) {
  dsa::e2m1_raw(w, x);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = dsa::mul_bf16x2(x[i], f);
  if (!DIRECT) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = dsa::mul_bf16x2(x[i], f2);
  }
}
// Whether every scale byte that a loop meets is at most kMxDirect (values up to 12: the usual case) is
// asked once: a branch at each word would keep the words from overlapping.
template <class F>
__device__ __forceinline__ void with_direct(bool direct, F f) {
  if (direct) f(std::true_type{});
  else f(std::false_type{});
}

// A tile whose scores pass a head's reference by more than this (in powers of two) moves it.
constexpr float kMove = 8.0f;

// The key (of eight) of a score's column, and the place of a key's weight: see kKPitch.
__device__ __forceinline__ constexpr int key_of(int col) { return (col & 4) + ((col >> 1) & 1) + 2 * (col & 1); }
__device__ __forceinline__ constexpr int place_of(int key) { return 2 * (key & 3) + (key >> 2); }

template <int DQK, int DV, bool SEP>
__global__ void __launch_bounds__(kBlock, (Narrow<DQK, DV, SEP>::kPerSm)) attn_kv4_narrow_kernel(const Params p) {
  using N = Narrow<DQK, DV, SEP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const uint32_t base = dsa::smem_u32(smem);

  // ---- the item
  const int per = p.Hc * p.G, group = p.H / p.Hc;
  int u = blockIdx.x;
  const int split = u % p.splits;
  u /= p.splits;
  const int t = u / per, kvh = (u - t * per) / p.G;
  const int h_in = (u - t * per - kvh * p.G) * N::kHeads;  // first head within the KV head's
  const int h0 = kvh * group + h_in, hv = min(N::kHeads, group - h_in);
  // a split's tiles go by K, so that ids are on their way before the row's length is there
  const int nt_all = (p.K + kTile - 1) / kTile;
  const int i0 = static_cast<int>(static_cast<int64_t>(nt_all) * split / p.splits);
  const int i_end = static_cast<int>(static_cast<int64_t>(nt_all) * (split + 1) / p.splits);
  const int32_t* irow = p.idx + static_cast<int64_t>(t) * p.K;
  auto peek_id = [&](int i) {
    const int j = i * kTile + tid;
    return tid < kTile && i < i_end && j < p.K ? __ldg(irow + j) : -1;
  };
  int x[5];
#pragma unroll
  for (int d = 0; d < 5; ++d) x[d] = peek_id(i0 + d);
  const int t_end = p.g.table ? __ldg(p.g.cu + p.g.n_seqs) : INT_MAX;
  int len = p.topk_length ? __ldg(p.topk_length + t) : p.K;
  // the query's words (eight dims) of this thread
  constexpr int kWords = N::kHeads * (DQK / 8) / kBlock + (N::kHeads * (DQK / 8) % kBlock != 0);
  uint4 q[kWords];
#pragma unroll
  for (int k = 0; k < kWords; ++k) {
    const int y = tid + k * kBlock, head = y / (DQK / 8);
    q[k] = head < hv ? __ldg(reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(t) * p.H + h0 + head) * DQK) + y - head * (DQK / 8))
                     : make_uint4(0, 0, 0, 0);
  }
  const int b = p.g.table ? dsa::kv8_seq_warp(p.g.cu, p.g.n_seqs, t) : 0;
  const int32_t* trow = p.g.table ? p.g.table + static_cast<int64_t>(b) * p.g.max_blocks : nullptr;
  if (t >= t_end) return;  // a padding row
  len = len < 0 ? 0 : (len > p.K ? p.K : len);
  const int i1 = min(i_end, (len + kTile - 1) / kTile);
  const int64_t orow = static_cast<int64_t>(t) * p.H + h0;
  // ---- rows of keys: thread k < kTile looks up key k of each tile, table entries two tiles and ids three ahead
  auto load_id = [&](int i) { return i * kTile + tid < len ? peek_id(i) : -1; };
  auto load_block = [&](int id) {  // as the table holds it; -1 beyond the table
    const int page = id >> p.g.lb;
    return !trow || id < 0 ? page : page < p.g.max_blocks ? __ldg(trow + page) : -1;
  };
  int* row_ring = reinterpret_cast<int*>(smem + N::kRows);
  auto put_row = [&](int i, int id, int blk) {
    const int row = id >= 0 && blk >= 0 && blk < p.g.n_blocks ? (blk << p.g.lb) + (id & ((1 << p.g.lb) - 1)) : -1;
    if (tid < kTile) row_ring[(i & (kRowRing - 1)) * kTile + tid] = row;
  };
#pragma unroll
  for (int d = 0; d < 5; ++d)
    if ((i0 + d) * kTile + tid >= len) x[d] = -1;
  int id_a = x[3], id_b = x[4], blk_a;  // of tile i + 3: id and table entry; of tile i + 4: id
  {
    const int y0 = load_block(x[0]), y1 = load_block(x[1]), y2 = load_block(x[2]);
    blk_a = load_block(id_a);
    put_row(i0, x[0], y0);
    put_row(i0 + 1, x[1], y1);
    put_row(i0 + 2, x[2], y2);
  }
  __syncthreads();

  // where a key's scales begin in its 32 bytes
  auto shift_of = [](const uint8_t* st, int key) { return DQK == 576 ? st[N::kMetaAt + key] & 2 : 0; };
  // ---- copies of a tile: eight lanes a key, so that they cover 128 bytes of its row
  const int rows = p.g.n_blocks << p.g.lb;
  const int piece = tid & 7;
  const uint8_t* const k_from = p.k8 + kvh * (DQK / 2) + piece * 16;
  const uint8_t* const v_from = SEP ? p.v8 + kvh * (DV / 2) + piece * 16 : nullptr;
  auto copy_tile = [&](int i, int stage) {
    const uint32_t st = base + N::kStages + stage * N::kStage;
    const int* ring = row_ring + (i & (kRowRing - 1)) * kTile;
#pragma unroll
    for (int s = 0; s < kTile / (kBlock / 8); ++s) {
      const int key = (tid >> 3) + s * (kBlock / 8);
      const int row = i < i1 ? ring[key] : -1;
      const bool any = row >= 0 && dsa::check(row < rows, p.status);
      const int64_t r = any ? row : 0;
      const uint32_t n = any ? 16u : 0u, to = st + key * N::kKPitch + piece * 16, sc = st + N::kScaleAt + key * 32;
      const uint8_t* src = k_from + r * (p.Hc * (DQK / 2));
#pragma unroll
      for (int m = 0; m < DQK / 256; ++m) cp_async16(to + m * 128, src + m * 128, n);
      if (SEP) cp_async16(st + N::kVAt + key * N::kVPitch + piece * 16, v_from + r * (p.Hc * (DV / 2)), n);
      uint32_t meta = any ? 1u : 0u;
      if (DQK == 576) {
        if (piece < 2) cp_async16(to + 256, src + 256, n);
        // 18 bytes from an even place on: the words that hold them, of the last one only what belongs to the row
        const int64_t first = (r * p.Hc + kvh) * 18;
        if (first & 2) meta |= 2u;
        const int need = (first & 2 ? 20 : 18) - (piece - 3) * 4;
        if (piece >= 3) cp_async4(sc + (piece - 3) * 4, p.k_exp + (first & ~int64_t{3}) + (piece - 3) * 4, any ? min(need, 4) : 0);
      } else if (DQK == 512) {
        if (piece == 0) cp_async16(sc, p.k_exp + (r * p.Hc + kvh) * 16, n);
      } else {
        if (piece < 2) cp_async8(sc + piece * 8, (piece ? p.v_exp : p.k_exp) + (r * p.Hc + kvh) * 8, n / 2);
      }
      if (piece == 0) smem[N::kStages + stage * N::kStage + N::kMetaAt + key] = static_cast<uint8_t>(meta);
    }
    cp_async_commit();
  };
  copy_tile(i0, 0);
  copy_tile(i0 + 1, 1);

  // ---- the query, in the order in which the lanes' codes meet: a super-step is four blocks of 32 dims, one a lane's c;
  // its step j and half h hold elements i and i + 4, i = 2 (j & 1) + h, of word j / 2 of each block.  The last
  // 64 of 576 dims are two blocks of which a lane has half: four steps.
#pragma unroll
  for (int k = 0; k < kWords; ++k) {
    const int y = tid + k * kBlock, head = y / (DQK / 8), w = y - head * (DQK / 8);
    if (head >= N::kHeads) break;
    const uint32_t pair[4] = {__byte_perm(q[k].x, q[k].z, 0x5410), __byte_perm(q[k].x, q[k].z, 0x7632),
                              __byte_perm(q[k].y, q[k].w, 0x5410), __byte_perm(q[k].y, q[k].w, 0x7632)};
    const bool last = w >= DQK / 256 * 32;  // of the last 64 of 576
    const int r = w & 15;
    // 32 dims are 4 words: super-step w / 16, lane (w / 4) % 4, word w % 4; the last ones: lane r / 2, word r % 2
    const int cc = last ? r >> 1 : r >> 2, step0 = (w >> 4) * 8 + 2 * (last ? r & 1 : r & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint32_t*>(smem + head * N::kQPitch + ((step0 + (i >> 1)) * 2 + (i & 1)) * 16 + cc * 4) = pair[i];
  }

  // ---- state of the softmax: heads 16 m + g and 16 m + g + 8, the same in every warp
  float m_run[2] = {-INFINITY, -INFINITY}, m_max[2] = {-INFINITY, -INFINITY}, l_part[2] = {0.f, 0.f};
  float acc[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
  float* wmax = reinterpret_cast<float*>(smem + N::kWmax);
  const int slice = warp % N::kSlices, half = warp / N::kSlices;  // value dims 64 slice .., keys of this half
  const uint32_t q_addr = base + ((lane & 7) + 8 * ((lane >> 3) & 1)) * N::kQPitch + (lane >> 4) * 16;

  for (int i = i0; i < i1; ++i) {
    const int stage = (i - i0) & 1;
    // this thread's copies of tile i, and everybody's (the first time: the query too); everybody is through with
    // tile i - 1, whose stage takes tile i + 1
    if (i == i0) cp_async_wait<1>();
    else cp_async_wait<0>();
    __syncthreads();
    if (i > i0) copy_tile(i + 1, stage ^ 1);
    const uint8_t* st = smem + N::kStages + stage * N::kStage;
    if (DQK != 256 || tid < kTile) {  // rows of tile i + 3 (at more dims registers are short for the branch)
      put_row(i + 3, id_a, blk_a);
      id_a = id_b;
      blk_a = load_block(id_b);
      id_b = load_id(i + 5);
    }

    // ---- scores of the warp's eight keys (column n of the products is key key_of(n))
    const int key0 = warp * 8;
    const uint8_t* key_at = st + (key0 + key_of(g)) * N::kKPitch;
    const uint8_t* exp_at = st + N::kScaleAt + (key0 + key_of(g)) * 32 + shift_of(st, key0 + key_of(g));
    // of this lane's columns 2 c and 2 c + 1
    const bool valid[2] = {static_cast<bool>(st[N::kMetaAt + key0 + key_of(2 * c)] & 1),
                           static_cast<bool>(st[N::kMetaAt + key0 + key_of(2 * c + 1)] & 1)};
    // factors of the values' blocks, and whether a key or value of the warp has a byte above kMxDirect
    uint32_t top_byte = 0;
#pragma unroll
    for (int y = lane; y < 8 * N::kBlocksV; y += 32) {
      const int key = key0 + y / N::kBlocksV, blk = y % N::kBlocksV;
      const uint32_t byte = st[N::kScaleAt + key * 32 + shift_of(st, key) + (SEP ? 8 : 0) + blk];
      top_byte = max(top_byte, byte);
      *reinterpret_cast<uint16_t*>(smem + N::kFactors + blk * N::kFPitch + (key0 + place_of(y / N::kBlocksV)) * 2) =
          static_cast<uint16_t>(dsa::mx_factor(byte));
    }
    constexpr int kSuper = DQK / 128;  // whole super-steps
    uint32_t byte[kSuper + 1];
#pragma unroll
    for (int s = 0; s < kSuper; ++s) byte[s] = exp_at[4 * s + c], top_byte = max(top_byte, byte[s]);
    byte[kSuper] = DQK == 576 ? exp_at[16 + (c >> 1)] : 0;
    const bool direct = !__any_sync(0xffffffffu, max(top_byte, byte[kSuper]) > dsa::kMxDirect);
    // (two sums each, of alternating steps: a product does not wait for the one before)
    float s_acc[4] = {0.f, 0.f, 0.f, 0.f}, s_two[4] = {0.f, 0.f, 0.f, 0.f};
    with_direct(direct, [&](auto d) {
      // NW words, two steps each
      auto words = [&](auto nw, const uint32_t* w, uint32_t f, uint32_t f2, int step) {
        constexpr int NW = decltype(nw)::value;
        uint32_t x[NW][4];
#pragma unroll
        for (int k = 0; k < NW; ++k) widen_word<decltype(d)::value>(w[k], f, f2, x[k]);
        uint32_t a[2 * NW][4];
#pragma unroll
        for (int k = 0; k < 2 * NW; ++k) ldmatrix4(a[k], q_addr + (step + k) * 32);
#pragma unroll
        for (int k = 0; k < NW; ++k) {
          mma16816(s_acc, a[2 * k], x[k][0], x[k][1]);
          mma16816(s_two, a[2 * k + 1], x[k][2], x[k][3]);
        }
      };
#pragma unroll
      for (int s = 0; s < kSuper; ++s) {
        const uint4 w4 = *reinterpret_cast<const uint4*>(key_at + (4 * s + c) * 16);
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
        words(std::integral_constant<int, 4>{}, w, dsa::mx_factor(byte[s]), dsa::mx_second(byte[s]), s * 8);
      }
      if (DQK == 576) {
        const uint2 w2 = *reinterpret_cast<const uint2*>(key_at + 256 + c * 8);
        const uint32_t w[2] = {w2.x, w2.y};
        words(std::integral_constant<int, 2>{}, w, dsa::mx_factor(byte[kSuper]), dsa::mx_second(byte[kSuper]), kSuper * 8);
      }
    });

    // ---- softmax: in powers of two, against a running reference of each head
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float mx = -INFINITY;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float& s = s_acc[2 * e + k];
        s = valid[k] ? (s + s_two[2 * e + k]) * p.scale_log2 : -INFINITY;
        mx = fmaxf(mx, s);
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      if (c == 0) wmax[(e * 8 + g) * N::kWPitch + warp] = mx;
    }
    const bool all_direct = !__syncthreads_or(!direct);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float4 w0 = *reinterpret_cast<const float4*>(wmax + (e * 8 + g) * N::kWPitch);
      const float4 w1 = *reinterpret_cast<const float4*>(wmax + (e * 8 + g) * N::kWPitch + 4);
      m_max[e] = fmaxf(m_max[e], fmaxf(fmaxf(fmaxf(w0.x, w0.y), fmaxf(w0.z, w0.w)), fmaxf(fmaxf(w1.x, w1.y), fmaxf(w1.z, w1.w))));
    }
    if (__any_sync(0xffffffffu, m_max[0] > m_run[0] + kMove || m_max[1] > m_run[1] + kMove)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (m_max[e] > m_run[e] + kMove) {
          const float alpha = ex2(m_run[e] - m_max[e]);
          m_run[e] = m_max[e];
          l_part[e] *= alpha;
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j][2 * e] *= alpha, acc[j][2 * e + 1] *= alpha;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float ref = m_run[e] == -INFINITY ? 0.f : m_run[e];  // (no valid slot so far)
      const float p0 = ex2(s_acc[2 * e] - ref), p1 = ex2(s_acc[2 * e + 1] - ref);
      __nv_bfloat16* to = reinterpret_cast<__nv_bfloat16*>(smem + N::kP + (e * 8 + g) * N::kPPitch) + key0;
      to[place_of(key_of(2 * c))] = __float2bfloat16_rn(p0);
      to[place_of(key_of(2 * c + 1))] = __float2bfloat16_rn(p1);
      l_part[e] += p0 + p1;
    }
    __syncthreads();

    // ---- values: 64 dims of this warp's keys; of eight weights, place 2 i is key i's and place 2 i + 1 key i + 4's
    constexpr int kSteps = kTile / 16 / N::kHalves;
    const int first = half * kSteps * 16 + c;
    const uint8_t* v0 = st + N::kVAt + first * N::kVPitch + slice * 32 + g * 4;
    const uint8_t* f0 = smem + N::kFactors + (slice * 2 + (g >> 2)) * N::kFPitch + (half * kSteps * 16 + 2 * c) * 2;
    const uint32_t p_addr = base + N::kP + ((lane & 7) + 8 * ((lane >> 3) & 1)) * N::kPPitch + (half * kSteps * 16 + (lane >> 4) * 8) * 2;
    with_direct(all_direct, [&](auto d) {
      uint32_t w[4], f[2];  // of the next step: keys c, c + 4, c + 8, c + 12 of its sixteen
      auto load = [&](int k) {
#pragma unroll
        for (int y = 0; y < 4; ++y) w[y] = *reinterpret_cast<const uint32_t*>(v0 + (k * 16 + 4 * y) * N::kVPitch);
#pragma unroll
        for (int y = 0; y < 2; ++y) f[y] = *reinterpret_cast<const uint32_t*>(f0 + (k * 16 + 8 * y) * 2);
      };
      load(0);
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        uint32_t a[4], x[2][2][4];  // of two keys: dims 0..3 and 4..7, the first key's in the low half
        ldmatrix4(a, p_addr + k * 32);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          uint32_t f2 = 0;
          if (!decltype(d)::value) {
            auto second = [&](int key) {
              return dsa::mx_second(st[N::kScaleAt + key * 32 + shift_of(st, key) + (SEP ? 8 : 0) + slice * 2 + (g >> 2)]);
            };
            const int key = first + k * 16 + 8 * y;
            f2 = __byte_perm(second(key), second(key + 4), 0x5410);
          }
          widen_word<decltype(d)::value>(__byte_perm(w[2 * y], w[2 * y + 1], 0x5410), f[y], f2, x[y][0]);
          widen_word<decltype(d)::value>(__byte_perm(w[2 * y], w[2 * y + 1], 0x7632), f[y], f2, x[y][1]);
        }
        if (k + 1 < kSteps) load(k + 1);
#pragma unroll
        for (int j = 0; j < 8; ++j) mma16816(acc[j], a, x[0][j >> 2][j & 3], x[1][j >> 2][j & 3]);
      }
    });
  }
  cp_async_wait_all();  // nothing of this thread is in flight when it leaves (or reuses the stages)

  // ---- the sums' norm, over lanes and warps, and the two halves' values
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float l = l_part[e];
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (c == 0) wmax[(e * 8 + g) * N::kWPitch + warp] = l;
  }
  __syncthreads();  // (and every thread's copies have ended)
  if constexpr (N::kHalves == 2) {
    float* other = reinterpret_cast<float*>(smem + N::kStages);
    if (half == 1) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) other[(slice * 32 + j * 4 + e) * 32 + lane] = acc[j][e];
    }
    __syncthreads();
    if (half == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] += other[(slice * 32 + j * 4 + e) * 32 + lane];
    }
    __syncthreads();
  }
  const bool split_up = p.splits > 1;
  if (half == 0) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int h = e * 8 + g;
      float l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) l += wmax[h * N::kWPitch + w];
      if (h >= hv) continue;
      const float mc = m_run[e] == -INFINITY ? 0.f : m_run[e];
      const bool any = l != 0.f;  // true for NaN too
      const bool first = slice == 0 && c == 0;
      float f = 0.f;
      if (split_up) {
        if (any) f = 1.f / l;  // a split's mean value, which stays in range where the sum might not
        if (first) *reinterpret_cast<float4*>(smem + N::kStats + h * 16) = make_float4(mc, l, m_max[e], 0.f);
      } else {
        const float sink = p.sink ? __ldg(p.sink + h0 + h) : -INFINITY, sk = sink * kLog2e;
        float lse_v = sink, lkv = INFINITY;
        if (any) {
          const float M = fmaxf(mc, sk);
          const float a = exp2f(mc - M);
          const float z = l * a + exp2f(sk - M);
          f = a / z;
          lse_v = (M + log2f(z)) * kLn2;
          lkv = (mc + log2f(l)) * kLn2;
        }
        if (first) {
          p.lse[orow + h] = lse_v;
          if (p.lse_kv) p.lse_kv[orow + h] = lkv;
          if (p.max_logits) p.max_logits[orow + h] = any ? max_logit(l, m_max[e]) : -INFINITY;
        }
      }
      // this lane's dims: 64 slice + 8 (2c + k) + j
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int d = slice * 64 + (2 * c + k) * 8;
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = any ? acc[j][2 * e + k] * f : 0.f;
        if (split_up) {
          float4* to = reinterpret_cast<float4*>(smem) + (h * DV + d) / 4;
          to[0] = make_float4(o[0], o[1], o[2], o[3]), to[1] = make_float4(o[4], o[5], o[6], o[7]);
        } else {
          __stcs(reinterpret_cast<uint4*>(p.out + (orow + h) * DV + d),
                 make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7])));
        }
      }
    }
  }
  if (!split_up) return;

  // ---- joined: with M the largest of the references and the sink, a_s = 2^(m_s - M) l_s and z = sum_s a_s + 2^(sink - M),
  // out = sum_s a_s O_s / z of the splits' means O_s.  Each CTA takes its part of the values.  lse_kv is the slots' alone, whose
  // sum against a sink far above them is nothing: under a sink it is taken again against the largest reference.
  cluster_sync();
  float* shares = reinterpret_cast<float*>(smem + N::kShares);
  for (int y = tid; y < N::kHeads * kMaxCluster; y += kBlock) {
    const int h = y / kMaxCluster, s = y % kMaxCluster;  // sixteen lanes a head
    const float4 v = s < p.splits && h < hv ? ld_cluster(base + N::kStats + h * 16, s) : make_float4(0.f, 0.f, 0.f, 0.f);
    const bool have = v.y != 0.f;
    float mm = have ? v.x : -INFINITY, mx = have ? v.z : -INFINITY;
    bool any = have;
#pragma unroll
    for (int o = 1; o < kMaxCluster; o <<= 1) {
      mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      any |= static_cast<bool>(__shfl_xor_sync(0xffffffffu, static_cast<int>(any), o));
    }
    const float sink = p.sink && h < hv ? __ldg(p.sink + h0 + h) : -INFINITY, sk = sink * kLog2e;
    const float M = fmaxf(mm, sk);
    const float a = have ? v.y * exp2f(v.x - M) : 0.f;
    float l = a;
#pragma unroll
    for (int o = 1; o < kMaxCluster; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const float z = any ? l + exp2f(sk - M) : 1.f;
    shares[y] = a / z;  // at most 1: a mean of means stays in range
    float l_kv = l;
    if (p.lse_kv && __any_sync(0xffffffffu, sk > mm)) {
      l_kv = have ? v.y * exp2f(v.x - mm) : 0.f;
#pragma unroll
      for (int o = 1; o < kMaxCluster; o <<= 1) l_kv += __shfl_xor_sync(0xffffffffu, l_kv, o);
    }
    if (split == 0 && s == 0 && h < hv) {
      p.lse[orow + h] = any ? (M + log2f(z)) * kLn2 : sink;
      if (p.lse_kv) p.lse_kv[orow + h] = any ? (mm + log2f(l_kv)) * kLn2 : INFINITY;
      if (p.max_logits) p.max_logits[orow + h] = any ? max_logit(l, mx) : -INFINITY;
    }
  }
  __syncthreads();
  for (int y = split * kBlock + tid; y < hv * (DV / 4); y += p.splits * kBlock) {
    const float* share = shares + y / (DV / 4) * kMaxCluster;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int s = 0; s < p.splits; ++s) {
      const float4 v = ld_cluster(base + y * 16, s);
      const float a = share[s];
      o.x = fmaf(a, v.x, o.x), o.y = fmaf(a, v.y, o.y), o.z = fmaf(a, v.z, o.z), o.w = fmaf(a, v.w, o.w);
    }
    reinterpret_cast<uint2*>(p.out + orow * DV)[y] = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
  }
  cluster_sync();  // the others have read this CTA's values
}

template <int DQK, int DV, bool SEP>
int launch_form(const Params& p, cudaStream_t stream) {
  using N = Narrow<DQK, DV, SEP>;
  auto kernel = attn_kv4_narrow_kernel<DQK, DV, SEP>;
  static std::atomic<uint64_t> ready{0};  // devices where the kernel's shared memory is allowed
  int dev = 0;
  cudaGetDevice(&dev);  // below 64: check_device
  if (!(ready.load(std::memory_order_acquire) >> dev & 1)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, N::kTotal) != cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
      return dsa::launch_error("attn_kv4_narrow_kernel smem attribute");
    ready.fetch_or(uint64_t{1} << dev, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.n_items);
  cfg.blockDim = dim3(kBlock);
  cfg.dynamicSmemBytes = N::kTotal;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = p.splits;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = p.splits > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) return dsa::launch_error("attn_kv4_narrow_kernel");
  return DSA_OK;
}

}  // namespace

namespace dsa {
namespace kv4_attn {

// Clusters of 1 to 16 CTAs that are resident at once, with three CTAs an SM, as the runtime's occupancy query
// says (a cluster stays within a group of SMs).
constexpr int kResident[kMaxCluster] = {456, 228, 148, 110, 87, 74, 59, 51, 46, 43, 36, 36, 28, 26, 26, 21};

// A call's time with s splits a row, in tenths of what a tile takes on a busy SM (1.65 us at 576 dims, 1.0 at 256).  Items of
// one SM take their tiles more or less one after the other, so layers of one CTA an SM count; a tile takes 1.45 times as
// long where there is one and 1.15 where there are two, and items that are not resident at once cost a
// tenth more (96 rows of 2 x 12 heads with shorter and longer contexts: 37.6 us with two splits, 44.8 with three).  An item is its tiles and 1.1 for the query and
// the results, 0.3 for its part of a join, whose latency is 2.1.  Measured, 576 dims (1.7 us beside it): one to three
// tiles 6.8, 9.4, 11.8 us in one layer, 9.7, 13.4, 17.3 in two; sixteen splits of two tiles 12.8, 17.6, 23.5 in one to
// three; 100 rows of 22 tiles 57.6 us in one layer, 43.7 with four splits.
int64_t cost_of(int units, int nt, int s) {
  const int64_t layers = (3 * units + kResident[s - 1] - 1) / kResident[s - 1];
  const int item = 10 * ((nt + s - 1) / s) + (s > 1 ? 14 : 11);
  return layers * item * (layers == 1 ? 29 : layers == 2 ? 23 : layers == 3 ? 20 : 22) / 20 + (s > 1 ? 21 : 0);
}

// The splits of a row's slots where groups of 16 heads take less time than the tiles of 64, else 0.  Measured, in us, here / there, 576 dims:
//   slots                  64          180          350          700         1400         2048
//   1 row of 64 heads   6.8 / 11.3   9.7 / 14.8  10.5 / 14.6  10.3 / 15.6  12.5 / 17.1  13.0 / 17.2 (*)
//   10 rows             6.8 / 11.3  10.1 / 14.8  12.6 / 15.2  17.5 / 16.7  25.0 / 18.4  33.1 / 20.1
//   40 rows             9.5 / 11.5  17.1 / 14.8  27.3 / 19.0  44.2 / 22.8  72.1 / 29.8  89.2 / 35.1
//   16 rows of 16 heads 7.0 / 10.5   9.9 / 14.0  10.7 / 14.2  13.2 / 16.0  20.3 / 17.7  23.9 / 19.7
//   100 rows            7.0 / 10.9  11.9 / 14.4  19.1 / 19.9  27.3 / 28.7  43.7 / 48.8  55.0 / 62.1
// (* 12.5 to 13.4 by where the ids lie, and 13.9 in a decode step with lengths and a sink over 65,536 positions.)
// (a key is widened once for 16 heads here, there for 64; tiles a quarter full cost what full ones do).  300 rows
// of 16 heads x 2048 slots 160 / 132; one of 8192 slots 27.5 / 21.4, of 65,536 165 / 72: sixteen CTAs a unit are all there
// are.  256 dims: 96 rows of 2 x 12 heads x 1027 slots 37 / 59, 1000 of 12 135 / 193, 16 of 64 heads x 700 14.6 / 14.0.
int narrow_splits(int T, int H, int Hc, int Dqk, int K) {
  const int64_t units = static_cast<int64_t>(T) * Hc * ((H / Hc + 15) / 16);
  if (units * kMaxCluster < kv8_attn::kPlanSms && K > 6144) return 0;
  const int nt = (K + kTile - 1) / kTile;
  const bool few = H / Hc <= 16 && (Dqk == 256 || K <= 1024 || (units >= 24 && units <= 100));
  if (units > 10 * kv8_attn::kPlanSms) return few ? 1 : 0;  // (many layers: splits only add to an item)
  int best = 1;
  int64_t cost = INT64_MAX;
  for (int s = 1; s <= kMaxCluster && s <= nt; ++s) {
    const int64_t c = cost_of(static_cast<int>(units), nt, s);
    if (c < cost) cost = c, best = s;
  }
  return few || cost <= 50 + 10 * std::min(nt, 3) + std::min(std::max(nt - 3, 0), 12) * 5 / 4 ? best : 0;
}

int launch_narrow(const kv8_attn::Params& p, int T, int Dqk, cudaStream_t stream) {
  if (Dqk == 256) return launch_form<256, 256, true>(p, stream);
  return Dqk == 576 ? launch_form<576, 512, false>(p, stream) : launch_form<512, 512, false>(p, stream);
}

}  // namespace kv4_attn
}  // namespace dsa
