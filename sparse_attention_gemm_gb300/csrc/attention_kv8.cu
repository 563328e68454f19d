// attention_kv8.cu -- sparse attention over the 8-bit block cache, on tcgen05.
//
// For row t, head h (of KV head kvh = h / (H / Hc)) and valid slot j, with
// cache row r_j in block b_j:
//   s_j = scale * k_scale[b_j] * (q . e4m3(kv8[r_j])),
//   out = sum_j exp(s_j) v_scale[b_j] e4m3(v8[r_j]) / (sum_j exp(s_j) + exp(sink)).
//
// Both products run on the codes as they lie in the cache (kind::f8f6f4): a
// block's scale is one number per key, so it multiplies the key's scores and
// weights afterwards and no code is ever widened in shared memory.  The other
// operand of each product is split into two E4M3 terms:
//   query:   q / s = hi + lo / 16, s the power of two that brings the head's
//            largest element to (224, 448].  A bf16 significand has 8 bits, two
//            E4M3 terms hold 4 each: exact down to 2^-14 of the scaled units.
//   weights: w = C * exp(s_j - m) * v_scale / 2^E as hi + lo: relative error
//            2^-8, what rounding to bf16 costs, and never less than 2^-10 / C
//            (half the smaller term's smallest step).
//
// Work item = (token, KV head, group of 64 query heads, split of its slots);
// calls with few heads per KV head or few rows go to attention_kv8_narrow.cu.
// Products ("swap AB"), tiles of 128 keys:
//   MMA1  S^T[key, hi|lo head] = K[key, :] . Q[hi|lo head, :]^T   (M = 128 keys, N = 128)
//   MMA2  O^T[dim, head] += V^T[dim, key] . (Phi + Plo)^T[key, head] (M = 128 dims, N = 64),
//         a half of the tile at a time: its buffer goes back that much sooner
// S^T (two buffers) and O^T fill TMEM.  Tiles are gathered with cp.async into
// 128-byte-swizzled rows, in two buffers of two halves; a copy's landing is its
// own arrival at the half's barrier, so the gather never waits for one.
// Softmax: as in the bf16 kernel, one reference maximum per head that moves
// when a tile passes it by 2^kTheta, and a reference exponent E of the value
// scales that moves when a block's scale passes 2^E; both move the running sums.
//
// What bounds it.  An M = 64 product takes the tensor core as long as an M =
// 128 one (64 cycles a K step at N = 128), so tiles of 128 keys take 18 x 64 + 32 x 53 =
// 2.85K cycles against 2 x 2.0K of tiles of 64.  The query's two terms take
// 72 KB of shared memory, which leaves two buffers of 128 keys: a tile's way
// through them (copies 2K cycles, scores 1.5-2K, softmax 3-4K, value product 2K)
// is two tiles' time, 5.2K cycles a tile at 576 dims: latency, with the tensor
// cores at 55%.  A row's end and the next one's start cost 10K more (query
// 1.7K + 4.8K, results 4K).  2048 rows of 64 heads, 2048 slots, 576 dims: 596 us, 970
// TFLOP/s of the formula's operations (half of the bf16 rate measured; 578 GFLOP).
// A CTA that has finished takes over the item of one that has not started: SMs
// differ by up to 8% in speed, and with every 152nd item a CTA's own the slowest
// ones' 14 items of 13.5 set the time (615 us).
// Tried and slower: a look at the next query's largest element during this
// item's tiles (its loads held the gather back, 2%), tiles of 64 keys in four
// buffers (677 us), results from registers two bytes a lane (+25 us), the vote on
// moving references through a flag and a plain barrier (+25 us) or an mbarrier
// (+18 us) instead of the reducing barrier, weights formed before the vote is in (+40 us).
//
// Warps: 0..7 gather and query conversion, 8..15 softmax and epilogue, 16
// MMA1, 17 MMA2.
#include "attention_kv8.cuh"

namespace {

using namespace dsa::kv8_attn;

constexpr int kHG = 64;    // query heads per group
constexpr int kGatherWarps = 8;
constexpr int kGatherThreads = kGatherWarps * 32;
constexpr int kGatherKeys = kGatherThreads / 8;   // keys one gather step covers
constexpr int kGatherSteps = kKeys / kGatherKeys;
static_assert(kGatherSteps == 2, "a thread gathers two keys of a tile");
constexpr int kSoftWarp0 = kGatherWarps;
constexpr int kSoftWarps = 8;
constexpr int kSoftThreads = kSoftWarps * 32;
constexpr int kMmaWarp = kSoftWarp0 + kSoftWarps;
constexpr int kMma2Warp = kMmaWarp + 1;
constexpr int kThreads = (kMma2Warp + 1) * 32;
// 18 warps: 96 registers a thread.  The softmax warps hold 32 scores, and keep
// some values that an item needs once in local memory.
constexpr uint32_t kQChunkBytes = 2 * kHG * 128;  // hi and lo of 64 heads x 128 codes
constexpr uint32_t kPPart = kKeys * kHG;          // one E4M3 term of P^T, 64 keys
constexpr int kTile = 2 * kKeys;                  // keys per tile: M of the score product
constexpr uint32_t kTmemCols = 512;
constexpr int kSCol = 0;    // S^T buffers at columns 0 and 128 (hi 64, lo 64)
constexpr int kOCol = 256;  // O^T blocks at 256 + 64 m
constexpr int kMaxSplits = 32;

// A key row is kFull chunks of 128 codes (128-byte swizzle) and, at 576 dims,
// a tail of 64 (64-byte swizzle).  MMA2 does not read the tail, so once a
// tile's scores are done its space takes the first term of the tile's P^T; that is
// what makes two buffers of 128 keys fit beside the query's 72 KB.
template <int DQK, int DV, bool SEP>
struct Shape {
  static constexpr int kFull = DQK / 128;
  static constexpr bool kTail = DQK % 128 != 0;
  static_assert(DQK % 128 == 0 || DQK % 128 == 64, "tail of 64 codes");
  static constexpr int kNv = DV / 128;
  static constexpr uint32_t kVOff = SEP ? kFull * 2 * kChunkBytes : 0;  // V inside a tile buffer
  static constexpr uint32_t kTailOff = kFull * 2 * kChunkBytes;
  static constexpr uint32_t kBuf = 2 * ((kFull + (SEP ? kNv : 0)) * kChunkBytes + (kTail ? kKeys * 64 : 0));
  static constexpr uint32_t kQTail = kFull * kQChunkBytes;
  static constexpr uint32_t kQBytes = kQTail + (kTail ? 2 * kHG * 64 : 0);
  static constexpr uint32_t kKv = kQBytes;                          // [2] tiles
  static constexpr uint32_t kPLo = kKv + 2 * kBuf;                  // [2] halves of a tile
  static constexpr uint32_t kPHi = kTail ? kKv + kTailOff : kPLo + 2 * kPPart;  // [2] halves; of each tile buffer, or
  static constexpr uint32_t kPHiStep = kTail ? kBuf : 0;                        // of the one in turn
  // scale of each slot's key and, behind them, value (one number where they are one), per half of a tile; 0: no slot
  static constexpr uint32_t kMeta = kPLo + (kTail ? 2 : 4) * kPPart;
  static constexpr uint32_t kMetaStep = kKeys * (SEP ? 8 : 4);
  static constexpr uint32_t kWmax = kMeta + 4 * kMetaStep;             // float [4][64]
  static constexpr uint32_t kAlpha = kWmax + 1024;                     // float [64]
  static constexpr uint32_t kFac = kAlpha + 256;                       // float [64]
  static constexpr uint32_t kQexp = kFac + 256;                        // uint8 [3][64]
  static constexpr uint32_t kSvm = kQexp + 192;                        // float [4]
  static constexpr uint32_t kBars = kSvm + 16;
  static constexpr uint32_t kSlots = kBars + 24 * 8;                   // 16 bytes [2]: answers to requests for items
  static constexpr uint32_t kMisc = kSlots + 32;
  static constexpr uint32_t kTotal = kMisc + 16;
  static_assert(kTotal <= 227 * 1024, "shared memory");
  static_assert(kKv % 1024 == 0 && kBuf % 1024 == 0 && kPLo % 1024 == 0, "alignment");
};

// The softmax warps' barrier, plain and with an OR over the group.  The
// instructions want converged warps (.aligned), and lanes part at waits and
// at `if (lane == 0)` or `if (!valid)` before them: each warp is brought
// together first.  The same goes for tcgen05.ld / st: __syncwarp before each.
__device__ __forceinline__ void group_sync() {
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(kSoftThreads) : "memory");
}
__device__ __forceinline__ bool group_any(bool x) {
  __syncwarp();
  return dsa::named_bar_any(1, kSoftThreads, x);
}

// Asks for the block index of a CTA of this grid that has not started and no
// longer will; the answer (16 bytes) arrives at the barrier.
__device__ __forceinline__ void take_cta(const void* slot, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   dsa::smem_u32(slot)),
               "r"(dsa::smem_u32(bar))
               : "memory");
}
// The answer: a block index, or -1 when all have started.
__device__ __forceinline__ int taken_cta(const void* slot) {
  const ulonglong2 r = *reinterpret_cast<const ulonglong2*>(slot);
  int x = -1;
  asm volatile(
      "{\n .reg .b128 h;\n .reg .pred p;\n mov.b128 h, {%1, %2};\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, h;\n}"
      : "+r"(x)
      : "l"(r.x), "l"(r.y)
      : "memory");
  return x;
}

// Combines v[0..7] (one value per head hb + i) over the 8 lanes that share
// lane & 3, halving the values at each step: lane keeps head hb + own_head(lane).
__device__ __forceinline__ int own_head(int lane) { return ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1); }
template <class F>
__device__ __forceinline__ float fold8(float (&v)[8], int lane, F f) {
#pragma unroll
  for (int n = 4, bit = 16; n > 0; n >>= 1, bit >>= 1) {
    const bool up = (lane & bit) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = up ? v[i + n] : v[i], send = up ? v[i] : v[i + n];
      v[i] = f(keep, __shfl_xor_sync(0xffffffffu, send, bit));
    }
  }
  return v[0];
}

// Index of a thread's score of its key k (0..3) and head h (0..7), and the largest of a head's.
__device__ __forceinline__ constexpr int at(int k, int h) { return 16 * (k >> 1) + 4 * (h >> 1) + 2 * (k & 1) + (h & 1); }
__device__ __forceinline__ float most_of(const float (&x)[32], int h) {
  return fmaxf(fmaxf(x[at(0, h)], x[at(1, h)]), fmaxf(x[at(2, h)], x[at(3, h)]));
}

// One work item: the tiles [i0, i1) of row t.
struct Item {
  int t, kvh, h0, hv;  // first query head and how many of the group's are real
  int split, i0, i1, len;
  bool dead;           // a padding row of a batch with a block table
};

__device__ __forceinline__ Item get_item(const Params& p, int it, int t_end) {
  Item w;
  int u = p.n_items - 1 - it;  // longest rows first (they are the last of a packed prompt)
  w.split = u % p.splits;
  u /= p.splits;
  const int per = p.Hc * p.G, group = p.H / p.Hc;
  w.t = u / per;
  const int r = u - w.t * per;
  w.kvh = r / p.G;
  const int g = r - w.kvh * p.G;
  w.h0 = w.kvh * group + g * kHG;
  w.hv = min(kHG, group - g * kHG);
  w.dead = w.t >= t_end;
  int len = p.K;
  if (p.topk_length) {
    len = __ldg(p.topk_length + w.t);
    len = len < 0 ? 0 : (len > p.K ? p.K : len);
  }
  if (w.dead) len = 0;
  const int nt = (len + kTile - 1) / kTile;
  w.len = len;
  // (nt <= 2^24 and at most 32 splits: the products fit)
  w.i0 = static_cast<int>(static_cast<uint32_t>(nt) * static_cast<uint32_t>(w.split) / static_cast<uint32_t>(p.splits));
  w.i1 = static_cast<int>(static_cast<uint32_t>(nt) * static_cast<uint32_t>(w.split + 1) / static_cast<uint32_t>(p.splits));
  return w;
}

// kMax: max_logits is asked for (eight registers a softmax thread).
template <int DQK, int DV, bool SEP, bool kMax>
__global__ void __launch_bounds__(kThreads, 1) attn_kv8_kernel(const Params p) {
  using S = Shape<DQK, DV, SEP>;
  extern __shared__ __align__(1024) uint8_t smem[];  // the kernel has no other shared memory
  if (dsa::smem_u32(smem) & 1023u) {                 // would break every swizzle
    if (threadIdx.x == 0) atomicOr(p.status, DSA_STATUS_CHECK_FAILED);
    return;
  }
  float* wmax = reinterpret_cast<float*>(smem + S::kWmax);  // [4 quarters][64 heads]
  // Exponents of the query scales (biased; 255: not finite) of three items in turn: the gather
  // warps convert item n + 3's query after MMA1 of item n + 2 has run, which
  // needed the S buffer of item n, which the softmax hands back after reading these.
  uint8_t* qexp = smem + S::kQexp;                        // [3][64]
  float* svm = reinterpret_cast<float*>(smem + S::kSvm);  // [4]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBars);
  uint64_t* kv_full = bars;        // [4]: halves of the two tile buffers
  uint64_t* kv_empty = bars + 4;   // [4]
  uint64_t* s_full = bars + 8;     // [2]
  uint64_t* s_empty = bars + 10;   // [2]
  uint64_t* p_empty = bars + 12;   // [2]: MMA2 of the half of a tile has run
  uint64_t* drain = bars + 14;     // [2]: the MMA issuers' exit commits
  uint64_t* p_full = bars + 16;    // of the whole tile: its first half's products already meet rescaled sums
  uint64_t* q_full = bars + 17;
  uint64_t* q_empty = bars + 18;
  uint64_t* q_read = bars + 19;    // the query's rows have been converted
  uint64_t* sched_full = bars + 20;   // [2]: the answer to a request for an item is there
  uint64_t* sched_empty = bars + 22;  // [2]: every warp has read it
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kMisc + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int b = 0; b < 4; ++b) {
      dsa::mbar_init(&kv_full[b], kGatherThreads);
      dsa::mbar_init(&kv_empty[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      dsa::mbar_init(&s_full[b], 1);
      dsa::mbar_init(&s_empty[b], kSoftWarps);
      dsa::mbar_init(&p_empty[b], 1);
      dsa::mbar_init(&drain[b], 1);
      dsa::mbar_init(&sched_full[b], 1);
      dsa::mbar_init(&sched_empty[b], kThreads / 32);
    }
    dsa::mbar_init(p_full, kSoftWarps);
    dsa::mbar_init(q_full, kGatherWarps);
    dsa::mbar_init(q_empty, 1);
    dsa::mbar_init(q_read, kGatherWarps);
    *abort_flag = 0;
    dsa::fence_barrier_init();
  }
  if (warp == kMmaWarp) dsa::tmem_alloc(tmem_slot, kTmemCols);
  dsa::tc_fence_before();
  __syncthreads();
  dsa::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const dsa::Waiter wt = dsa::make_waiter(abort_flag, p.status);
  const int t_end = p.g.table ? __ldg(p.g.cu + p.g.n_seqs) : INT_MAX;
  // The item after this CTA's n-th, -1 if there is none: that of a CTA that has
  // not started, which the request of the n-th item took over.  Taken in turn
  // like this, slower SMs work fewer rows.  Every warp asks once per item;
  // *heard = false if the wait gave up.
  auto next_item = [&](int n, bool* heard) {
    if (!p.steal) return -1;
    *heard = dsa::mbar_wait_warp(&sched_full[n & 1], (n >> 1) & 1, wt);
    if (!*heard) return -1;
    const int got = taken_cta(smem + S::kSlots + (n & 1) * 16);
    __syncwarp();
    if (lane == 0) dsa::mbar_arrive(&sched_empty[n & 1]);
    __syncwarp();
    return got;
  };

  if (warp < kGatherWarps) {
    // ------------------------------------------------------------ gather
    // Thread gt covers piece (gt & 7) (16 codes) of keys (gt >> 3) + 32 kg of
    // every chunk.  A row's place depends on its id and the block table: ids
    // are read two tiles ahead, the table one tile ahead.
    const int gt = threadIdx.x, piece = gt & 7;
    const uint32_t kv_addr = dsa::smem_u32(smem) + S::kKv, meta_addr = dsa::smem_u32(smem) + S::kMeta;
    int half_ctr = 0, item_ctr = 0;  // (here a unit of work is half a tile)
    bool ok = true;
    // The query: its bf16 rows pass through a tile's buffer (ahead of the
    // item's tiles, so that they are there when the item before leaves the
    // operand); a warp copies and converts eight heads, four threads a head,
    // units (16 values) sub, sub + 4, ...  Odd heads take the halves of a
    // 128-byte row in the other order, and a head's 16-byte pieces lie in
    // eights XOR-ed with it: eight lanes touch all banks once.
    const int hq = gt >> 2, sub = gt & 3;
    constexpr int kUnits = DQK / 64, kPieces = DQK / 8;
    static_assert(kHG * DQK * 2 <= S::kBuf, "a query fits a tile's buffer");
    // head 32 a + 8 c + 2 j + e is row 32 a + 8 j + 2 c + e of the operand,
    // which gives each softmax thread eight consecutive heads
    const int qrow = (hq & 32) + ((hq & 6) << 2) + ((hq >> 2) & 6) + (hq & 1);
    auto raw_at = [&](int h, int c) { return h * (DQK * 2) + ((c & ~7) | ((c ^ h) & 7)) * 16; };
    auto unit_of = [&](int k) { return (sub + 4 * k) ^ (k < S::kFull * 2 ? (hq & 1) * 4 : 0); };
    auto send_query = [&](const Item& w) {
      const int b = (half_ctr >> 1) & 1;
      const uint32_t ph = ((half_ctr >> 2) & 1) ^ 1, buf = kv_addr + b * S::kBuf;
      if (!dsa::mbar_wait_warp(&kv_empty[2 * b], ph, wt) || !dsa::mbar_wait_warp(&kv_empty[2 * b + 1], ph, wt)) return false;
      const __nv_bfloat16* src = p.q + (static_cast<int64_t>(w.t) * p.H + w.h0) * DQK;
#pragma unroll 3
      for (int k = 0; k < 8 * kPieces / 32; ++k) {
        const int y = k * 32 + lane, h = warp * 8 + y / kPieces, c = y % kPieces;
        const bool real = h < w.hv;
        cp_async16(buf + raw_at(h, c), src + (real ? h * DQK + c * 8 : 0), real ? 16u : 0u);
      }
      cp_async_arrive(&kv_full[2 * b]);
      cp_async_arrive(&kv_full[2 * b + 1]);
      half_ctr += 2;
      return true;
    };
    auto convert_query = [&](int query_half, int n_item) {  // query_half: half_ctr of its buffer
      const int b = (query_half >> 1) & 1;
      const uint8_t* raw = smem + S::kKv + b * S::kBuf;
      cp_async_wait_all();
      __syncwarp();  // (the warp's own copies)
      uint32_t m = 0;
#pragma unroll 2
      for (int k = 0; k < kUnits; ++k) {
        const int u = unit_of(k);
        m = dsa::amax_bf16x8(*reinterpret_cast<const uint4*>(raw + raw_at(hq, 2 * u)), m);
        m = dsa::amax_bf16x8(*reinterpret_cast<const uint4*>(raw + raw_at(hq, 2 * u + 1)), m);
      }
      m = dsa::max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = dsa::larger_half(dsa::max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 2)));
      // a head with infinity or NaN: its scores are NaN
      const bool finite = m < 0x7F80u;
      const float s = finite ? dsa::kv8_scale_of(__uint_as_float(m << 16)) : 1.f;
      const float inv = dsa::pow2_inverse(s);
      if (!dsa::mbar_wait_warp(q_empty, (n_item & 1) ^ 1, wt)) return false;
      if (sub == 0) qexp[(n_item % 3) * 64 + hq] = finite ? static_cast<uint8_t>(__float_as_uint(s) >> 23) : 255;
#pragma unroll 3
      for (int k = 0; k < kUnits; ++k) {
        const int u = unit_of(k);
        const uint4 v0 = *reinterpret_cast<const uint4*>(raw + raw_at(hq, 2 * u));
        const uint4 v1 = *reinterpret_cast<const uint4*>(raw + raw_at(hq, 2 * u + 1));
        const uint32_t wd[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint16_t h2[2], l2[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) split_query(wd[2 * j + e], inv, h2[e], l2[e]);
          hi[j] = h2[0] | (static_cast<uint32_t>(h2[1]) << 16);
          lo[j] = l2[0] | (static_cast<uint32_t>(l2[1]) << 16);
        }
        const bool tail = k >= S::kFull * 2;
        const uint32_t to = tail ? S::kQTail + sw64_offset(qrow, u - S::kFull * 8)
                                 : (u >> 3) * kQChunkBytes + dsa::sw128_offset(qrow, (u & 7) * 16);
        // (64 rows on leaves either swizzle's phase as it is)
        *reinterpret_cast<uint4*>(smem + to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(smem + to + kHG * (tail ? 64 : 128)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      dsa::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        dsa::mbar_arrive(q_full);
        dsa::mbar_arrive(q_read);
      }
      if (warp == 0) {  // everybody has read the rows: the buffer goes back
        if (!dsa::mbar_wait_warp(q_read, n_item & 1, wt)) return false;
        if (lane == 0) {
          dsa::mbar_arrive(&kv_empty[2 * b]);
          dsa::mbar_arrive(&kv_empty[2 * b + 1]);
        }
        __syncwarp();
      }
      return true;
    };
    // L2 prefetch of a later item's query and ids
    auto prefetch_item = [&](int it) {
      const Item w = get_item(p, it, t_end);
      if (w.i0 >= w.i1) return;
      const uint8_t* q0 = reinterpret_cast<const uint8_t*>(p.q + (static_cast<int64_t>(w.t) * p.H + w.h0) * DQK);
      for (int o = gt * 128; o < w.hv * DQK * 2; o += kGatherThreads * 128) l2_prefetch(q0 + o);
      const int j = w.i0 * kTile + gt * 32;
      if (j < min(w.i1 * kTile, w.len)) l2_prefetch(p.idx + static_cast<int64_t>(w.t) * p.K + j);
    };
    // The request for the item after the n-th goes out as that one begins (not
    // again after the answer that there is none).
    int requests = 0;
    auto request = [&](int n) {
      if (!p.steal) return true;
      if (n >= 2 && !dsa::mbar_wait_warp(&sched_empty[n & 1], ((n >> 1) & 1) ^ 1, wt)) return false;
      if (lane == 0) {
        dsa::mbar_expect_tx(&sched_full[n & 1], 16);
        take_cta(smem + S::kSlots + (n & 1) * 16, &sched_full[n & 1]);
      }
      __syncwarp();
      ++requests;
      return true;
    };
    int it = blockIdx.x;
    for (int n = 0; it >= 0 && ok; ++n) {
      if (warp == 0 && !request(n)) break;
      const Item w = get_item(p, it, t_end);
      if (w.i0 >= w.i1) {
        it = next_item(n, &ok);
        continue;
      }
      const int b = p.g.table ? dsa::kv8_seq_warp(p.g.cu, p.g.n_seqs, w.t) : 0;
      const int32_t* irow = p.idx + static_cast<int64_t>(w.t) * p.K;
      auto load_id = [&](int i, int kg) {
        const int j = i * kKeys + kg * kGatherKeys + (gt >> 3);
        return j < w.len ? __ldg(irow + j) : -1;
      };
      const int32_t* trow = p.g.table ? p.g.table + static_cast<int64_t>(b) * p.g.max_blocks : nullptr;
      auto load_block = [&](int id) {  // as the table holds it; -1 beyond the table
        const int page = id >> p.g.lb;
        return !trow || id < 0 ? page : page < p.g.max_blocks ? __ldg(trow + page) : -1;
      };
      // id of this tile's and the next tile's keys, table entry of this tile's:
      // loaded one tile before they are looked at
      int id[kGatherSteps], nid[kGatherSteps], blk[kGatherSteps];
#pragma unroll
      for (int kg = 0; kg < kGatherSteps; ++kg) {
        nid[kg] = load_id(2 * w.i0 + 1, kg);
        id[kg] = load_id(2 * w.i0, kg);
        blk[kg] = load_block(id[kg]);
      }
      // The query comes before the first tile, and is converted before that is
      // copied, whose buffer is not free sooner; a CTA's first query behind it.
      const int query_half = half_ctr;
      ok = send_query(w) && (item_ctr == 0 || convert_query(query_half, item_ctr));
      if (!ok) break;
      for (int i = 2 * w.i0; i < 2 * w.i1; ++i, ++half_ctr) {
        const int stage = half_ctr & 3;
        int cur[kGatherSteps];
#pragma unroll
        for (int kg = 0; kg < kGatherSteps; ++kg) {
          cur[kg] = id[kg] >= 0 && blk[kg] >= 0 && blk[kg] < p.g.n_blocks
                        ? (blk[kg] << p.g.lb) + (id[kg] & ((1 << p.g.lb) - 1))
                        : -1;
          id[kg] = nid[kg];
          blk[kg] = load_block(nid[kg]);
          nid[kg] = i + 2 < 2 * w.i1 ? load_id(i + 2, kg) : -1;
        }
        if (!dsa::mbar_wait_warp(&kv_empty[stage], ((half_ctr >> 2) & 1) ^ 1, wt)) {
          ok = false;
          break;
        }
        const uint32_t buf = kv_addr + (stage >> 1) * S::kBuf, half = stage & 1;
        {
          // the scales: lanes of even and odd pieces take the two keys' (with V, those of pieces 2, 3, 6, 7 the value's)
          const int r = piece & 1 ? cur[1] : cur[0];
          const int64_t at = static_cast<int64_t>((r >= 0 ? r : 0) >> p.g.lb) * p.Hc + w.kvh;
          const bool value = SEP && (piece & 2);
          if (dsa::check(r < (p.g.n_blocks << p.g.lb), p.status))
            cp_async4(meta_addr + stage * S::kMetaStep + (value ? kKeys * 4 : 0) + ((piece & 1) * kGatherKeys + (gt >> 3)) * 4,
                      (value ? p.v_scale : p.k_scale) + at, r >= 0 ? 4u : 0u);
        }
#pragma unroll
        for (int kg = 0; kg < kGatherSteps; ++kg) {
          const int key = kg * kGatherKeys + (gt >> 3);
          const uint32_t nbytes = cur[kg] >= 0 ? 16u : 0u;
          const int64_t rh = static_cast<int64_t>(cur[kg] >= 0 ? cur[kg] : 0) * p.Hc + w.kvh;
          // checked build: the row is inside the cache
          if (!dsa::check(cur[kg] < (p.g.n_blocks << p.g.lb), p.status)) continue;
          const uint8_t* krow = p.k8 + rh * DQK + piece * 16;
          const uint32_t dst = buf + half * kChunkBytes + dsa::sw128_offset(key, piece * 16);
#pragma unroll
          for (int c = 0; c < S::kFull; ++c) cp_async16(dst + c * 2 * kChunkBytes, krow + c * 128, nbytes);
          if (SEP) {
            const uint8_t* vrow = p.v8 + rh * DV + piece * 16;
#pragma unroll
            for (int c = 0; c < S::kNv; ++c)
              cp_async16(dst + S::kVOff + c * 2 * kChunkBytes, vrow + c * 128, nbytes);
          }
        }
        if (S::kTail) {
          // the tail's four pieces: lanes with piece 0..3 take the first key's, the others the second's
          const bool second = piece >= 4;
          const int key = (second ? kGatherKeys : 0) + (gt >> 3), r = second ? cur[1] : cur[0];
          const int64_t rh = static_cast<int64_t>(r >= 0 ? r : 0) * p.Hc + w.kvh;
          if (dsa::check(r < (p.g.n_blocks << p.g.lb), p.status))
            cp_async16(buf + S::kTailOff + half * (kKeys * 64) + sw64_offset(key, piece & 3), p.k8 + rh * DQK + S::kFull * 128 + (piece & 3) * 16,
                       r >= 0 ? 16u : 0u);
        }
        cp_async_arrive(&kv_full[stage]);
        if (i == 2 * w.i0 + 1) {
          if (item_ctr == 0 && !convert_query(query_half, 0)) {
            ok = false;
            break;
          }
          ++item_ctr;
          it = next_item(n, &ok);
          if (!ok) break;
          if (it >= 0) prefetch_item(it);
        }
      }
    }
    cp_async_wait_all();  // nothing of this thread is in flight when it leaves
    if (requests > 0 && lane == 0) dsa::mbar_drain(&sched_full[(requests - 1) & 1], ((requests - 1) >> 1) & 1, p.status);
    __syncwarp();
  } else if (warp >= kMmaWarp) {
    // ------------------------------------------------------------ MMA issue
    // Two warps, one per product, each converged with one elected issuer.
    const bool leader = elect_sync();
    const uint32_t base = dsa::smem_u32(smem);
    bool ok = true;
    if (warp == kMmaWarp) {
      constexpr uint32_t idesc1 = dsa::idesc_e4m3(kTile, 2 * kHG);
      const uint64_t q_desc = dsa::smem_desc(base, 16, 1024, dsa::kSwizzle128B);
      const uint64_t kv_desc = dsa::smem_desc(base + S::kKv, 16, 1024, dsa::kSwizzle128B);
      const uint64_t qt_desc = dsa::smem_desc(base + S::kQTail, 16, 512, dsa::kSwizzle64B);
      const uint64_t kt_desc = dsa::smem_desc(base + S::kKv + S::kTailOff, 16, 512, dsa::kSwizzle64B);
      int tile_ctr = 0, item_ctr = 0;
      int it = blockIdx.x;
      for (int n = 0; it >= 0 && ok; ++n) {
        const Item w = get_item(p, it, t_end);
        it = next_item(n, &ok);
        if (!ok) break;
        if (w.i0 >= w.i1) continue;
        if (!dsa::mbar_wait_warp(q_full, item_ctr & 1, wt)) break;
        for (int i = w.i0; i < w.i1; ++i, ++tile_ctr) {
          const int sb = tile_ctr & 1, use = tile_ctr + item_ctr + 1, b = use & 1;  // use of the tile buffers
          const uint32_t par = (use >> 1) & 1;
          const bool got = dsa::mbar_wait(&s_empty[sb], ((tile_ctr >> 1) & 1) ^ 1, wt) &&
                           dsa::mbar_wait(&kv_full[2 * b], par, wt) && dsa::mbar_wait(&kv_full[2 * b + 1], par, wt);
          // the gathered codes, before the tensor core reads them (MMA2's come
          // with the softmax warps' arrival, behind a fence of theirs)
          dsa::fence_proxy_async_smem();
          __syncwarp();
          dsa::tc_fence_after();
          const uint64_t a0 = kv_desc + b * (S::kBuf >> 4);
          const uint32_t d = tmem_base + kSCol + sb * 128;
#pragma unroll
          for (int c = 0; c < S::kFull; ++c) {
            const uint64_t ac = a0 + c * (2 * kChunkBytes >> 4), bc = q_desc + c * (kQChunkBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              dsa::umma_f8_if(leader && got, d, ac + kk * 2, bc + kk * 2, idesc1, (c | kk) != 0);
          }
          if (S::kTail) {
            const uint64_t at = kt_desc + b * (S::kBuf >> 4);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) dsa::umma_f8_if(leader && got, d, at + kk * 2, qt_desc + kk * 2, idesc1, 1u);
          }
          if (leader && got) dsa::umma_commit(&s_full[sb]);
          if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            break;
          }
        }
        if (!ok) break;
        if (leader) dsa::umma_commit(q_empty);
        __syncwarp();
        ++item_ctr;
      }
      if (leader) dsa::umma_drain(&drain[0], p.status);
      __syncwarp();
    } else {
      constexpr uint32_t idesc2 = dsa::idesc_e4m3(128, kHG) | (1u << 15) | (1u << 16);  // both MN-major
      int half_ctr = 0, tile_ctr = 0;
      const uint64_t v_desc = dsa::smem_desc(base + S::kKv + S::kVOff, 2 * kChunkBytes, 1024, dsa::kSwizzle128B);
      // P^T rows are 64 bytes (64 heads): 64-byte swizzle, groups of 8 keys 512 bytes apart
      const uint64_t ph_desc = dsa::smem_desc(base + S::kPHi, kPPart, 512, dsa::kSwizzle64B);
      const uint64_t pl_desc = dsa::smem_desc(base + S::kPLo, kPPart, 512, dsa::kSwizzle64B);
      int it = blockIdx.x;
      for (int n = 0; it >= 0 && ok; ++n) {
        const Item w = get_item(p, it, t_end);
        it = next_item(n, &ok);
        if (!ok) break;
        if (w.i0 < w.i1) half_ctr += 2;  // the query's use of a buffer
        for (int i = 2 * w.i0; i < 2 * w.i1; ++i, ++half_ctr) {
          const int half = half_ctr & 1, b = (half_ctr >> 1) & 1;
          const bool got = half == 1 || dsa::mbar_wait(p_full, tile_ctr++ & 1, wt);
          __syncwarp();
          dsa::tc_fence_after();
          const uint64_t a0 = v_desc + b * (S::kBuf >> 4) + half * (kChunkBytes >> 4);
          const uint64_t bh = ph_desc + b * (S::kPHiStep >> 4) + half * (kPPart >> 4), bl = pl_desc + half * (kPPart >> 4);
#pragma unroll
          for (int mb = 0; mb < S::kNv; ++mb) {
            const uint32_t d = tmem_base + kOCol + mb * kHG;
#pragma unroll
            for (int kk = 0; kk < kKeys / 32; ++kk) {
              const uint64_t a = a0 + mb * (2 * kChunkBytes >> 4) + kk * (32 * 128 >> 4);
              dsa::umma_f8_if(leader && got, d, a, bh + kk * (32 * kHG >> 4), idesc2, (i > 2 * w.i0 || kk > 0) ? 1u : 0u);
              dsa::umma_f8_if(leader && got, d, a, bl + kk * (32 * kHG >> 4), idesc2, 1u);
            }
          }
          if (leader && got) {
            dsa::umma_commit(&p_empty[half]);
            dsa::umma_commit(&kv_empty[half_ctr & 3]);
          }
          if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            break;
          }
        }
      }
      if (leader) dsa::umma_drain(&drain[1], p.status);
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    const int sw = warp - kSoftWarp0;
    const int st = threadIdx.x - kSoftWarp0 * 32;
    const int quarter = warp & 3;  // TMEM lane quarter
    const int hh = sw >> 2;        // head half
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    // Of S^T a thread holds four keys' scores of eight heads: key k of them is
    // row key0 + 8 k of its half of the tile, head hb + 2j + e of it is x[16 (k / 2) + 4j + 2 (k % 2) + e]
    const int half = quarter >> 1, key0 = (quarter & 1) * 32 + (lane >> 2);
    const int hb = hh * 32 + 8 * (lane & 3);
    // factors of O^T per head (the four warps of a head half write the same ones)
    float* alpha = reinterpret_cast<float*>(smem + S::kAlpha);
    float* fac = reinterpret_cast<float*>(smem + S::kFac);  // [64]: references, then the factors of the result
    uint8_t* rows = smem + S::kPLo + sw * 1024;             // this warp's, of the result: 16 heads x 32 dims, 64-byte swizzle
    int tile_ctr = 0, n_item = 0;
    bool ok = true;
    // A wait of this thread gave up: the eight warps leave together, at a
    // point that reduces the flag (see the bf16 kernel).
    bool failed = false;
    Item next = get_item(p, blockIdx.x, t_end);
    int it = blockIdx.x;
    for (int n = 0; it >= 0 && ok; ++n) {
      const Item w = next;
      const bool empty = w.dead || w.i0 >= w.i1;
      if (empty) {
        bool heard = true;
        it = next_item(n, &heard);
        failed |= !heard;
        if (p.steal && group_any(failed)) {  // the group leaves together
          ok = false;
          break;
        }
        if (it >= 0) next = get_item(p, it, t_end);
      }
      if (w.dead) continue;
      const int64_t orow = static_cast<int64_t>(w.t) * p.H + w.h0;
      if (empty) {
        if (p.splits > 1) {
          if (st < w.hv) p.part_s[(orow + st) * p.splits + w.split] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
        } else {
          for (int h = 0; h < w.hv; ++h)
            for (int d = st; d < DV; d += kSoftThreads) p.out[(orow + h) * DV + d] = __float2bfloat16_rn(0.f);
          if (st < w.hv) {
            p.lse[orow + st] = p.sink ? __ldg(p.sink + w.h0 + st) : -INFINITY;
            if (p.lse_kv) p.lse_kv[orow + st] = INFINITY;
            if (p.max_logits) p.max_logits[orow + st] = -INFINITY;
          }
        }
        continue;
      }
      ++n_item;  // (with this one: each query used a tile's buffer)
      // Per head hb + h: the reference, this thread's keys' sum and (for max_logits) maximum.
      float nm[8], l_part[8];  // (nm: the reference, negative)
      [[maybe_unused]] float top[8];
      bool unset = true;                        // no valid slot so far
      float ref = __uint_as_float(1u << 23);    // 2^E of the value scales so far
      float inv = __uint_as_float(253u << 23);  // 2^-E
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        l_part[h] = 0.f, nm[h] = 0.f;
        if (kMax) top[h] = -INFINITY;
      }
      for (int i = w.i0; i < w.i1; ++i, ++tile_ctr) {
        const int sb = tile_ctr & 1, use = tile_ctr + n_item, b = use & 1, stage = 2 * b + half;
        // the slots' scales come with the gathered tile
        if (!failed) failed = !dsa::mbar_wait(&kv_full[stage], (use >> 1) & 1, wt);
        const float* meta = reinterpret_cast<const float*>(smem + S::kMeta + stage * S::kMetaStep) + key0;
        float sk[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) sk[k] = meta[8 * k] > 0.f ? meta[8 * k] : 0.f;
        if (!failed) failed = !dsa::mbar_wait(&s_full[sb], (tile_ctr >> 1) & 1, wt);
        __syncwarp();
        dsa::tc_fence_after();
        float x[32];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint32_t v[16], lo[16];
          const uint32_t ta = tmem_base + lane_off + (static_cast<uint32_t>(g * 16) << 16) + kSCol + sb * 128 + hh * 32;
          dsa::tmem_ld16x256b_x4(ta, v);
          dsa::tmem_ld16x256b_x4(ta + 64, lo);
          dsa::tmem_wait_ld();
#pragma unroll
          for (int r = 0; r < 16; r += 2) {
            const float2 y = fma2(make_float2(__uint_as_float(lo[r]), __uint_as_float(lo[r + 1])), make_float2(0.0625f, 0.0625f),
                                  make_float2(__uint_as_float(v[r]), __uint_as_float(v[r + 1])));
            x[16 * g + r] = y.x, x[16 * g + r + 1] = y.y;
          }
        }
        const uint2 qe = *reinterpret_cast<const uint2*>(qexp + ((n_item - 1) % 3) * 64 + hb);
        dsa::tc_fence_before();
        __syncwarp();
        if (lane == 0) dsa::mbar_arrive(&s_empty[sb]);
        // scores in powers of two against the references; -inf where there is no slot
#pragma unroll
        for (int h = 0; h < 8; h += 2) {
          float2 q2;  // the query's scales times the softmax's (held as exponents: eight registers less)
          q2.x = __uint_as_float(((h < 4 ? qe.x : qe.y) >> (8 * (h & 3)) & 255u) << 23);
          q2.y = __uint_as_float(((h < 4 ? qe.x : qe.y) >> (8 * (h & 3) + 8) & 255u) << 23);
          // (255: a head with infinity or NaN)
          q2 = fma2(q2, make_float2(p.scale_log2, p.scale_log2), make_float2(q2.x - q2.x, q2.y - q2.y));
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 c = mul2(q2, make_float2(sk[k], sk[k]));
            const float2 y = fma2(make_float2(x[at(k, h)], x[at(k, h + 1)]), c, make_float2(nm[h], nm[h + 1]));
            x[at(k, h)] = y.x, x[at(k, h + 1)] = y.y;
          }
        }
        if (__any_sync(0xffffffffu, fminf(fminf(sk[0], sk[1]), fminf(sk[2], sk[3])) == 0.f)) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
#pragma unroll
            for (int h = 0; h < 8; ++h) x[at(k, h)] = sk[k] > 0.f ? x[at(k, h)] : -INFINITY;
          }
        }
        float most = x[0], sv_most = 0.f;
#pragma unroll
        for (int r = 1; r < 32; ++r) most = fmaxf(most, x[r]);
        if (SEP) {
#pragma unroll
          for (int k = 0; k < 4; ++k) sk[k] = sk[k] > 0.f ? meta[kKeys + 8 * k] : 0.f;  // from here on the values' scales
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) sv_most = fmaxf(sv_most, sk[k]);
        const bool ex = unset || most > kTheta || sv_most > ref;
        if constexpr (kMax) {
#pragma unroll
          for (int h = 0; h < 8; ++h) top[h] = fmaxf(top[h], most_of(x, h) - nm[h]);
        }
        const bool first = i == w.i0;
        bool need_rescale = false;
        float ratio = 1.f;  // of the old to the new 2^E
        if (first || group_any(ex || failed)) {
          // move the references: the tile's maximum per head over its 64 keys
          float v[8];
#pragma unroll
          for (int h = 0; h < 8; ++h) v[h] = most_of(x, h);
          const float mx = fold8(v, lane, [](float a, float c) { return fmaxf(a, c); });
          wmax[quarter * 64 + hb + own_head(lane)] = mx;
          float sv = fmaxf(sv_most, __shfl_xor_sync(0xffffffffu, sv_most, 4));
          sv = fmaxf(sv, __shfl_xor_sync(0xffffffffu, sv, 8));
          sv = fmaxf(sv, __shfl_xor_sync(0xffffffffu, sv, 16));
          if (lane == 0 && hh == 0) svm[quarter] = sv;
          if (group_any(failed)) {  // the group leaves together
            ok = false;
            break;
          }
          const float sv_max = fmaxf(fmaxf(svm[0], svm[1]), fmaxf(svm[2], svm[3]));
          const float rn = fmaxf(ref, pow2_ceil(sv_max));
          inv = dsa::pow2_inverse(rn);
          ratio = ref * inv;
          ref = rn;
          bool moved = ratio != 1.f;
#pragma unroll
          for (int g4 = 0; g4 < 2; ++g4) {
            float4 t4 = *reinterpret_cast<const float4*>(wmax + hb + 4 * g4);
#pragma unroll
            for (int q4 = 1; q4 < 4; ++q4) {
              const float4 o = *reinterpret_cast<const float4*>(wmax + q4 * 64 + hb + 4 * g4);
              t4.x = fmaxf(t4.x, o.x), t4.y = fmaxf(t4.y, o.y), t4.z = fmaxf(t4.z, o.z), t4.w = fmaxf(t4.w, o.w);
            }
            const float tm[4] = {t4.x, t4.y, t4.z, t4.w};
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const int h = 4 * g4 + n;
              // by how much the reference moves: to the tile's maximum, if that
              // passes it by kTheta or is the first
              const float up = (unset ? tm[n] > -INFINITY : tm[n] > kTheta) ? tm[n] : 0.f;
              const float a = unset ? 1.f : ex2(-up);
              moved |= up != 0.f;
              l_part[h] *= a;
              nm[h] -= up;
#pragma unroll
              for (int k = 0; k < 4; ++k) x[at(k, h)] -= up;
              if (lane < 4) alpha[hb + h] = a * ratio;
            }
          }
          unset = unset && !(sv_max > 0.f);
          need_rescale = __any_sync(0xffffffffu, moved) && !first;
        }
        // P^T rows key0 + 8 k, both terms: the thread's eight heads are bytes hb .. hb + 7 of the 64-byte rows
        if (!failed) failed = !dsa::mbar_wait(&p_empty[half], (tile_ctr & 1) ^ 1, wt);  // MMA2 of the tile before has read it
        {
          uint8_t* ph = smem + S::kPHi + b * S::kPHiStep + half * kPPart;
          uint8_t* pl = smem + S::kPLo + half * kPPart;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float wk = sk[k] * inv * kWeight;  // (2^-E alone stays in range)
            uint16_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float p0 = ex2(x[at(k, 2 * j)]), p1 = ex2(x[at(k, 2 * j + 1)]);
              const float2 l2 = add2(make_float2(l_part[2 * j], l_part[2 * j + 1]), make_float2(p0, p1));
              l_part[2 * j] = l2.x, l_part[2 * j + 1] = l2.y;
              const float2 p2 = mul2(make_float2(p0, p1), make_float2(wk, wk));
              split_weights(p2.x, p2.y, hi[j], lo[j]);
            }
            const uint32_t to = sw64_offset(key0 + 8 * k, hb >> 4) + (hb & 8);
            *reinterpret_cast<uint2*>(ph + to) = pack4(hi);
            *reinterpret_cast<uint2*>(pl + to) = pack4(lo);
          }
        }
        if (need_rescale) {
          // MMA2 of the previous tile must have landed before O^T is scaled
          if (!failed) failed = !dsa::mbar_wait(&p_empty[half ^ 1], (tile_ctr & 1) ^ 1, wt);
          __syncwarp();
          dsa::tc_fence_after();
          __syncwarp();  // alpha, written by four lanes of this warp
          const float* a32 = alpha + hh * 32;
#pragma unroll 1
          for (int mb = 0; mb < S::kNv; ++mb) {
            const uint32_t ta = tmem_base + lane_off + kOCol + mb * kHG + hh * 32;
            uint32_t v[32];
            __syncwarp();
            dsa::tmem_ld32(ta, v);
            dsa::tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * a32[c]);
            dsa::tmem_st32(ta, v);
          }
          dsa::tmem_wait_st();
        }
        dsa::fence_proxy_async_smem();
        dsa::tc_fence_before();
        __syncwarp();
        if (lane == 0) dsa::mbar_arrive(p_full);
      }
      if (!ok) break;

      // ---------------------------------------------------------- epilogue
      bool heard = true;
      it = next_item(n, &heard);
      failed |= !heard;
      if (it >= 0) next = get_item(p, it, t_end);
      const float sink = p.sink && st < w.hv ? __ldg(p.sink + w.h0 + st) : -INFINITY;
      // The sums' norm, while the last tile's MMA2 runs: over the four quarters
      // in wmax, once everybody has read the last references there.
      group_sync();
      if (quarter == 0 && lane < 4) {
#pragma unroll
        for (int h = 0; h < 8; ++h) fac[hb + h] = -nm[h];
      }
      wmax[quarter * 64 + hb + own_head(lane)] = fold8(l_part, lane, [](float a, float c) { return a + c; });
      group_sync();
      const float l = st < 64 ? wmax[st] + wmax[64 + st] + wmax[128 + st] + wmax[192 + st] : 0.f;
      float m_max = 0.f;
      if constexpr (kMax) {
        group_sync();
        wmax[quarter * 64 + hb + own_head(lane)] = fold8(top, lane, [](float a, float c) { return fmaxf(a, c); });
        group_sync();
        if (st < 64) m_max = fmaxf(fmaxf(wmax[st], wmax[64 + st]), fmaxf(wmax[128 + st], wmax[192 + st]));
      }
      const float unscale = ref * (1.f / kWeight);
      if (st < 64) {
        const float mc = fac[st];
        const bool any = l != 0.f;  // true for NaN too
        float f = unscale;
        if (p.splits > 1) {
          if (st < w.hv) p.part_s[(orow + st) * p.splits + w.split] = make_float4(mc, l, m_max, 0.f);
        } else {
          const float sk = sink * kLog2e;
          float lse_v = sink, lkv = INFINITY;
          f = 0.f;
          if (any) {
            const float M = fmaxf(mc, sk);
            const float a = exp2f(mc - M);
            const float z = l * a + exp2f(sk - M);
            f = a / z * unscale;
            lse_v = (M + log2f(z)) * kLn2;
            lkv = (mc + log2f(l)) * kLn2;
          }
          if (st < w.hv) {
            p.lse[orow + st] = lse_v;
            if (p.lse_kv) p.lse_kv[orow + st] = lkv;
            if (kMax) p.max_logits[orow + st] = any ? m_max * kLn2 : -INFINITY;
          }
        }
        fac[st] = f;
      }
      // O^T is complete with the last tile's MMA2 (each phase of p_empty has
      // been waited for in turn, so the parity names that tile)
      if (!failed) failed = !dsa::mbar_wait(&p_empty[half], (tile_ctr - 1) & 1, wt);
      if (!failed) failed = !dsa::mbar_wait(&p_empty[half ^ 1], (tile_ctr - 1) & 1, wt);
      group_sync();
      dsa::tc_fence_after();
      const int hcount = min(32, w.hv - hh * 32);
      const uint32_t tm_o = tmem_base + lane_off + kOCol + hh * 32;
      if (hcount <= 0) {
        // (no head of this half is real)
      } else if (p.splits > 1) {
        const float* f32 = fac + hh * 32;
#pragma unroll 1
        for (int mb = 0; mb < S::kNv; ++mb) {
          uint32_t v[32];
          __syncwarp();
          dsa::tmem_ld32(tm_o + mb * kHG, v);
          dsa::tmem_wait_ld();
          float* o = p.part_o + ((orow + hh * 32) * p.splits + w.split) * DV + mb * 128 + quarter * 32 + lane;
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            if (c < hcount) *o = __uint_as_float(v[c]) * f32[c];
            o += static_cast<int64_t>(p.splits) * DV;
          }
        }
      } else {
        // 16 heads x 32 dims at a time through shared memory, transposed by
        // the store of 8 x 8 matrices: 64 consecutive bytes a head.  (Two
        // bytes a lane straight to memory: 7K cycles an item, two bytes a
        // lane to shared memory 5K.)
        float f[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float2 f2 = *reinterpret_cast<const float2*>(fac + hh * 32 + 8 * c + 2 * (lane & 3));
          f[2 * c] = f2.x, f[2 * c + 1] = f2.y;
        }
        const uint32_t rows_at = dsa::smem_u32(rows);
        const int mrow = 8 * (lane >> 4) + (lane & 7), munit = (lane >> 3) & 1;  // matrices: 8 heads x 8 dims
        __nv_bfloat16* o0 = p.out + (orow + hh * 32 + (lane >> 2)) * DV + quarter * 32 + (lane & 3) * 8;
#pragma unroll 2
        for (int mb = 0; mb < S::kNv; ++mb) {
#pragma unroll
          for (int c0 = 0; c0 < 32; c0 += 16) {
            uint32_t v[2][8];
            __syncwarp();
            dsa::tmem_ld16x256b_x2(tm_o + mb * kHG + c0, v[0]);
            dsa::tmem_ld16x256b_x2(tm_o + mb * kHG + c0 + (16u << 16), v[1]);
            dsa::tmem_wait_ld();
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              uint32_t r[4];
#pragma unroll
              for (int n = 0; n < 4; ++n) {  // 8 heads n / 2, 8 dims n % 2
                const float* fn = f + (c0 >> 2) + 2 * (n >> 1);
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(v[g][2 * n]) * fn[0],
                                                                __uint_as_float(v[g][2 * n + 1]) * fn[1]);
                r[n] = *reinterpret_cast<const uint32_t*>(&b2);
              }
              dsa::stmatrix_x4_trans(rows_at + sw64_offset(mrow, 2 * g + munit), r[0], r[1], r[2], r[3]);
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int h = k * 8 + (lane >> 2);
              if (c0 + h < hcount)
                __stcs(reinterpret_cast<uint4*>(o0 + mb * 128 + (c0 + k * 8) * DV),
                       *reinterpret_cast<const uint4*>(rows + sw64_offset(h, lane & 3)));
            }
          }
        }
      }
      dsa::tc_fence_before();
      if (group_any(failed)) {  // the item's last barrier: the group leaves together
        ok = false;
        break;
      }
    }
  }

  __syncwarp();
  __syncthreads();
  if (warp == kMmaWarp) {
    dsa::tc_fence_after();
    dsa::tmem_dealloc(tmem_base, kTmemCols);
  }
}

// Joins the splits of one (token, head) per CTA: with M the largest reference,
// z = sum_s 2^(m_s - M) l_s + 2^(sink - M), out = sum_s 2^(m_s - M) O_s / z.
template <int DV>
__global__ void __launch_bounds__(DV / 4) attn_kv8_join_kernel(const Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the splits' kernel has finished
  const int64_t row = blockIdx.x;
  const int t = static_cast<int>(row / p.H), h = static_cast<int>(row - static_cast<int64_t>(t) * p.H);
  if (p.g.table && t >= __ldg(p.g.cu + p.g.n_seqs)) return;
  const int lane = threadIdx.x & 31;
  float4 s = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
  if (lane < p.splits) s = p.part_s[row * p.splits + lane];
  const bool have = s.y != 0.f;  // a split without a valid slot wrote no O
  float m = have ? s.x : -INFINITY, mx = have ? s.z : -INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  const float sink = p.sink ? __ldg(p.sink + h) : -INFINITY, sk = sink * kLog2e;
  const bool any = __any_sync(0xffffffffu, have);
  const float M = fmaxf(m, sk);
  const float a = have ? exp2f(s.x - M) : 0.f;
  float l = have ? s.y * a : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float z = any ? l + exp2f(sk - M) : 1.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4* o = reinterpret_cast<const float4*>(p.part_o + row * p.splits * DV) + threadIdx.x;
  for (int k = 0; k < p.splits; ++k) {
    const float ak = __shfl_sync(0xffffffffu, a, k);
    if (__shfl_sync(0xffffffffu, have, k)) {
      const float4 v = __ldcs(o + k * (DV / 4));
      acc.x = fmaf(ak, v.x, acc.x);
      acc.y = fmaf(ak, v.y, acc.y);
      acc.z = fmaf(ak, v.z, acc.z);
      acc.w = fmaf(ak, v.w, acc.w);
    }
  }
  const float f = 1.f / z;
  const __nv_bfloat162 r0 = __floats2bfloat162_rn(acc.x * f, acc.y * f), r1 = __floats2bfloat162_rn(acc.z * f, acc.w * f);
  reinterpret_cast<uint2*>(p.out + row * DV)[threadIdx.x] =
      make_uint2(*reinterpret_cast<const uint32_t*>(&r0), *reinterpret_cast<const uint32_t*>(&r1));
  if (threadIdx.x == 0) {
    p.lse[row] = any ? (M + log2f(z)) * kLn2 : sink;
    if (p.lse_kv) p.lse_kv[row] = any ? (M + log2f(l)) * kLn2 : INFINITY;
    if (p.max_logits) p.max_logits[row] = any ? mx * kLn2 : -INFINITY;
  }
}

// Splits of each row's slots: the number that makes the longest CTA shortest,
// counting a wave of CTAs as its tiles plus kItemTiles tiles for the query's
// conversion, the first gather and the epilogue, and joining as kJoinTiles
// tiles plus one per 16 splits.  Measured (rows of 576, 2048 slots, 128 heads;
// microseconds with 1, 2, 4, 8, 16 splits): 16 rows 49, 34, 25, 31, 49; 32 rows 50,
// 37, 42, 58, 85; 100 rows 96, 98, 118, 160, 248.
constexpr int kItemTiles = 5, kJoinTiles = 3;

int plan_splits(int64_t units, int K) {
  const int nt = (K + kTile - 1) / kTile;
  int best = 1;
  int64_t cost = INT64_MAX;
  for (int s = 1; s <= kMaxSplits && s <= nt; ++s) {
    const int64_t waves = (units * s + kPlanSms - 1) / kPlanSms;
    const int64_t c = 16 * (waves * ((nt + s - 1) / s + kItemTiles) + (s > 1 ? kJoinTiles : 0)) + (s > 1 ? s : 0);
    if (c < cost) cost = c, best = s;
  }
  return best;
}

bool known_shape(int T, int H, int Hc, int Dqk, int Dv, int K) {
  const bool form = ((Dqk == 576 || Dqk == 512) && Dv == 512) || (Dqk == 256 && Dv == 256);
  return form && T >= 1 && H >= 1 && Hc >= 1 && H % Hc == 0 && K >= 1 && K <= DSA_KV8_MAX_SLOTS;
}

int64_t units_of(int T, int H, int Hc) { return static_cast<int64_t>(T) * Hc * ((H / Hc + kHG - 1) / kHG); }

size_t part_bytes(int T, int H, int splits) {
  return (static_cast<size_t>(T) * H * splits * sizeof(float4) + 255) / 256 * 256;
}

template <int DQK, int DV, bool SEP, bool kMax>
int launch_form(const Params& p, int T, int sms, cudaStream_t stream) {
  using S = Shape<DQK, DV, SEP>;
  constexpr int smem = S::kTotal;
  auto kernel = attn_kv8_kernel<DQK, DV, SEP, kMax>;
  static std::atomic<uint64_t> ready{0};  // devices where the kernel's shared memory is allowed
  int dev = 0;
  cudaGetDevice(&dev);  // below 64: check_device
  if (!(ready.load(std::memory_order_acquire) >> dev & 1)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return dsa::launch_error("attn_kv8_kernel smem attribute");
    ready.fetch_or(uint64_t{1} << dev, std::memory_order_release);
  }
  kernel<<<p.n_items, kThreads, smem, stream>>>(p);
  int rc = dsa::launch_error("attn_kv8_kernel");
  if (rc != DSA_OK || p.splits == 1) return rc;
  // launched while the splits' kernel drains, so that its start-up hides behind it
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(T) * p.H);
  cfg.blockDim = dim3(DV / 4);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, attn_kv8_join_kernel<DV>, p) != cudaSuccess) return dsa::launch_error("attn_kv8_join_kernel");
  return DSA_OK;
}

template <int DQK, int DV, bool SEP>
int launch(const Params& p, int T, int sms, cudaStream_t stream) {
  return p.max_logits ? launch_form<DQK, DV, SEP, true>(p, T, sms, stream)
                      : launch_form<DQK, DV, SEP, false>(p, T, sms, stream);
}

}  // namespace

extern "C" size_t dsa_sparse_attn_fwd_kv8_workspace_size(int T, int H, int Hc, int Dqk, int Dv, int K) {
  if (!known_shape(T, H, Hc, Dqk, Dv, K) || narrow_takes(T, H, Hc, K)) return 0;
  const int s = plan_splits(units_of(T, H, Hc), K);
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
  const char* fn = "dsa_sparse_attn_fwd_kv8";
  const bool latent = (Dqk == 576 || Dqk == 512) && Dv == 512 && v8 == nullptr && v_scale == nullptr;
  const bool separate = Dqk == 256 && Dv == 256 && v8 != nullptr && v_scale != nullptr;
  if (!latent && !separate)
    return dsa::set_error(
        DSA_ERR_VALUE, "%s: (Dqk, Dv) must be (576|512, 512) without v8 and v_scale or (256, 256) with both", fn);
  if (T < 0 || H < 1 || Hc < 1 || Hc > DSA_KV8_MAX_HEADS || H % Hc != 0 || H / Hc > 128 || K < 0 ||
      K > DSA_KV8_MAX_SLOTS)
    return dsa::set_error(DSA_ERR_VALUE, "%s: need T >= 0, 0 <= K <= %d, 1 <= Hc <= %d, H a multiple of Hc, H / Hc <= 128",
                          fn, DSA_KV8_MAX_SLOTS, DSA_KV8_MAX_HEADS);
  const int64_t units = T > 0 ? units_of(T, H, Hc) : 0;
  if (units * kMaxSplits > INT_MAX || static_cast<int64_t>(T) * H > INT_MAX)
    return dsa::set_error(DSA_ERR_VALUE, "%s: T * H exceeds the int32 range of work items", fn);
  if (n_blocks < 1 || block < 1 || block > DSA_KV8_MAX_BLOCK || (block & (block - 1)) != 0)
    return dsa::set_error(DSA_ERR_VALUE, "%s: need n_blocks >= 1 and block a power of two in [1, %d]", fn, DSA_KV8_MAX_BLOCK);
  if (static_cast<int64_t>(n_blocks) * block > INT_MAX)
    return dsa::set_error(DSA_ERR_VALUE, "%s: n_blocks * block exceeds the int32 row range", fn);
  if (block_table && (n_seqs < 1 || max_blocks < 1 || !cu_seqlens))
    return dsa::set_error(DSA_ERR_VALUE, "%s: a block table needs cu_seqlens, n_seqs >= 1 and max_blocks >= 1", fn);
  if (!(scale > 0.f) || !(scale < INFINITY)) return dsa::set_error(DSA_ERR_VALUE, "%s: scale must be finite and > 0", fn);
  if (!kv8 || !kv_scale || (T > 0 && (!q || !out || !lse || (K > 0 && !idx))))
    return dsa::set_error(DSA_ERR_VALUE, "%s: NULL pointer", fn);
  if (!dsa::aligned(q, 16) || !dsa::aligned(kv8, 16) || !dsa::aligned(v8, 16) || !dsa::aligned(out, 16))
    return dsa::set_error(DSA_ERR_VALUE, "%s: q, kv8, v8 and out must be 16-byte aligned", fn);
  const size_t need = dsa_sparse_attn_fwd_kv8_workspace_size(T, H, Hc, Dqk, Dv, K);
  if (need > 0 && (!workspace || ws_bytes < need || !dsa::aligned(workspace, 256)))
    return dsa::set_error(DSA_ERR_WORKSPACE, "%s: needs a 256-byte aligned workspace of %zu bytes, got %zu", fn, need,
                          workspace ? ws_bytes : static_cast<size_t>(0));
  int sms = 0;
  int rc = dsa::check_device(&sms);
  if (rc != DSA_OK) return rc;
  if (T == 0) return DSA_OK;
  int lb = 0;
  while ((1 << lb) < block) ++lb;
  Params p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k8 = static_cast<const uint8_t*>(kv8);
  p.k_scale = kv_scale;
  p.v8 = static_cast<const uint8_t*>(separate ? v8 : kv8);
  p.v_scale = separate ? v_scale : kv_scale;
  p.idx = idx;
  p.topk_length = topk_length;
  p.sink = sink;
  p.g = dsa::Kv8Geom{cu_seqlens, nullptr, block_table, n_seqs, T, lb, n_blocks, max_blocks};
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.lse_kv = lse_kv;
  p.max_logits = max_logits;
  p.H = H;
  p.Hc = Hc;
  p.K = K;
  p.G = (H / Hc + kHG - 1) / kHG;
  p.splits = need > 0 ? plan_splits(units, K) : 1;
  p.n_items = static_cast<int>(units * p.splits);
  p.status = dsa::device_status_ptr();
  p.steal = p.n_items > sms;
  p.scale_log2 = scale * kLog2e;
  if (narrow_takes(T, H, Hc, K)) return launch_narrow(p, T, Dqk, stream);
  if (need > 0) {
    p.part_s = static_cast<float4*>(workspace);
    p.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + part_bytes(T, H, p.splits));
  }
  if (separate) return launch<256, 256, true>(p, T, sms, stream);
  return Dqk == 576 ? launch<576, 512, false>(p, T, sms, stream) : launch<512, 512, false>(p, T, sms, stream);
}
