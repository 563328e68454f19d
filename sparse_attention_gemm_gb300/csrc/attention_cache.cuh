// attention_cache.cuh -- sparse attention over the block caches in groups of 64
// query heads, on tcgen05.
//
// For row t, head h (of KV head kvh = h / (H / Hc)) and valid slot j, with
// cache row r_j of scale k_scale_j and v_scale_j (1 where codes carry theirs themselves):
//   s_j = scale * k_scale_j * (q . k_j),
//   out = sum_j exp(s_j) v_scale_j v_j / (sum_j exp(s_j) + exp(sink)).
// How a tile of codes becomes bf16 values in shared memory is the business of a Gather
// (attention_kv8.cuh, attention_kv4.cu); the rest is here.
//
// A code is a bf16 value exactly.  An 8-bit block's scale is one number per key: it
// multiplies the key's scores and weights, and no code is rounded.  A 4-bit code
// times its scale is a bf16 value again (kScaled = false).  Codes are widened to bf16 on their way into shared memory, and both products run in bf16
// (kind::f16) with fp32 sums.  The one rounding before out's is that of
// the weights exp(s_j - m) * v_scale / 2^E to bf16, as in the bf16 call; bf16
// has fp32's exponents, so small weights keep their relative precision.
//
// Work item = (token, KV head, group of 64 query heads, split of its slots);
// calls with few heads per KV head or few rows go to attention_kv8_narrow.cu and
// attention_kv4_narrow.cu.
// Products ("swap AB"), tiles of 64 keys:
//   MMA1  S^T[key, head]  = K[key, :] . Q[head, :]^T           (M = 64 keys, N = 64)
//   MMA2  O^T[dim, head] += V^T[dim, key] . P^T[key, head]     (M = 128 dims, N = 64)
// S^T (two buffers) and O^T live in TMEM.  Two tile buffers; eight warps load a tile's
// codes into registers while the tile before it is worked on.
// Softmax: as in the bf16 kernel, one reference maximum per head that moves
// when a tile passes it by 2^kMove, and a reference exponent E of the value
// scales that moves when a block's scale passes 2^E; both move the running sums.
//
// What bounds it, over E4M3 codes: shared memory.  A tile's products read 240 KB of operands (an
// M = 64, N = 64 step takes its 4 KB at the memory's whole rate), its codes
// arrive as 36 KB and are stored as 72: 350 KB, 2.7K of the 3.4K cycles
// that a tile takes; the rest is the chain of two buffers (stores 1.3K, scores 2K, softmax 1K,
// values 1.5K).  A row's end and the next one's start cost 8K more.  2048 rows
// of 64 heads, 2048 slots, 576 dims: 800 us, 723 TFLOP/s (578 GFLOP); with the stores left
// out 650 us, the loads 750 us; the bf16 call on the values read back: 676 us.
// Both products on the codes as they lie in the cache (kind::f8f6f4, query and weights as
// two E4M3 terms each) read half as much, 596 us, but E4M3 has a smallest step:
// weights below 2^-13.8 of the largest weight times the largest value scale were lost, and
// with them the output of rows whose largest weight meets a small value.
// Tried and slower: 16 gather warps of one key a thread (925 us) or in two groups of a buffer
// each (902 us), four of four keys (1157 us), each piece's next load behind its store (1105 us).
// A CTA that has finished takes over the item of one that has not started: SMs
// differ by up to 8% in speed, and with every 152nd item a CTA's own the slowest
// ones set the time.
//
// Warps: 0..7 gather and query, 8..15 softmax and epilogue, 16 MMA1, 17 MMA2.
#pragma once

#include "attention_kv8.cuh"

namespace dsa {
namespace kv8_attn {

constexpr int kHG = 64;    // query heads per group
constexpr int kGatherThreads = 256;
constexpr int kSoftWarp0 = 8;
constexpr int kSoftWarps = 8;
constexpr int kSoftThreads = kSoftWarps * 32;
constexpr int kMmaWarp = kSoftWarp0 + kSoftWarps;
constexpr int kMma2Warp = kMmaWarp + 1;
constexpr int kThreads = (kMma2Warp + 1) * 32;
constexpr uint32_t kQChunkBytes = kHG * 128;      // 64 heads x 64 dims
constexpr uint32_t kTmemCols = 512;
constexpr int kSCol = 0;    // S^T buffers at columns 0 and 64
constexpr int kOCol = 128;  // O^T blocks at 128 + 64 m
constexpr int kMaxSplits = 32;
// A tile whose scores pass a head's reference by more than this (in powers of two) moves it.
constexpr float kMove = 8.0f;

// A tile: key rows in chunks of 64 dims, then value rows where they are
// separate.  MMA2 does not read the key's last chunk at 576 dims, so once
// a tile's scores are done its space takes the tile's P^T.
template <int DQK, int DV, bool SEP>
struct Shape {
  static constexpr int kNk = DQK / 64;
  static constexpr int kNv = DV / 128;  // blocks of O^T
  static constexpr bool kTail = DQK % 128 != 0;
  static constexpr uint32_t kVOff = SEP ? kNk * kChunkBytes : 0;  // V inside a tile buffer
  static constexpr uint32_t kBuf = (kNk + (SEP ? 2 * kNv : 0)) * kChunkBytes;
  static constexpr uint32_t kKv = kNk * kQChunkBytes;                              // [2] tiles, behind the query
  static constexpr uint32_t kP = kTail ? kKv + DV / 64 * kChunkBytes : kKv + 2 * kBuf;  // [2] P^T
  static constexpr uint32_t kPStep = kTail ? kBuf : kChunkBytes;
  static constexpr uint32_t kRows = kKv + 2 * kBuf + (kTail ? 0 : 2 * kChunkBytes);  // results, 1 KB a softmax warp
  // scale of each slot's key and, behind them, value (one number where they are one, 1 where codes carry
  // theirs); 0: no slot
  static constexpr uint32_t kMeta = kRows + kSoftWarps * 1024;         // [2]
  static constexpr uint32_t kMetaStep = kKeys * (SEP ? 8 : 4);
  static constexpr uint32_t kWmax = kMeta + 2 * kMetaStep;             // float [4][64]
  static constexpr uint32_t kAlpha = kWmax + 1024;                     // float [64]
  static constexpr uint32_t kFac = kAlpha + 256;                       // float [64]
  static constexpr uint32_t kSvm = kFac + 256;                         // float [4]
  static constexpr uint32_t kBars = kSvm + 16;
  static constexpr uint32_t kSlots = kBars + 20 * 8;                   // 16 bytes [2]: answers to requests for items
  static constexpr uint32_t kMisc = kSlots + 32;
  static constexpr uint32_t kTotal = kMisc + 16;
  static_assert(kTotal <= 227 * 1024, "shared memory");
  static_assert(kKv % 1024 == 0 && kBuf % 1024 == 0 && kP % 1024 == 0 && kSlots % 16 == 0, "alignment");
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
// longer will; the answer (16 bytes) arrives at the barrier.  It is written
// through the async proxy into a place whose last answer was read with ordinary
// loads, so a proxy fence stands between those reads and the barrier that hands the
// place back, and between that barrier and the request.
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

// Index of a thread's score of its key k (0, 1) and head h (0..7), and the larger of a head's.
__device__ __forceinline__ constexpr int at(int k, int h) { return 4 * (h >> 1) + 2 * k + (h & 1); }
__device__ __forceinline__ float most_of(const float (&x)[16], int h) { return fmaxf(x[at(0, h)], x[at(1, h)]); }

// Eight bf16 values between their own order and 0, 4, 1, 5, 2, 6, 3, 7.
__device__ __forceinline__ uint4 to_places(uint4 u) {
  return make_uint4(__byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632), __byte_perm(u.y, u.w, 0x5410),
                    __byte_perm(u.y, u.w, 0x7632));
}
__device__ __forceinline__ uint4 from_places(uint4 u) {
  return make_uint4(__byte_perm(u.x, u.y, 0x5410), __byte_perm(u.z, u.w, 0x5410), __byte_perm(u.x, u.y, 0x7632),
                    __byte_perm(u.z, u.w, 0x7632));
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
  const int nt = (len + kKeys - 1) / kKeys;
  w.len = len;
  // (nt <= 2^24 and at most 32 splits: the products fit)
  w.i0 = static_cast<int>(static_cast<uint32_t>(nt) * static_cast<uint32_t>(w.split) / static_cast<uint32_t>(p.splits));
  w.i1 = static_cast<int>(static_cast<uint32_t>(nt) * static_cast<uint32_t>(w.split + 1) / static_cast<uint32_t>(p.splits));
  return w;
}

// G: how a tile comes into shared memory.  kMax: max_logits is asked for (eight registers a softmax thread).
template <class G, int DQK, int DV, bool SEP, bool kMax>
__global__ void __launch_bounds__(kThreads, 1) attn_cache_kernel(const Params p) {
  using S = Shape<DQK, DV, SEP>;
  static_assert(G::kThreads == kGatherThreads, "gather warps");
  extern __shared__ __align__(1024) uint8_t smem[];  // the kernel has no other shared memory
  if (dsa::smem_u32(smem) & 1023u) {                 // would break every swizzle
    if (threadIdx.x == 0) atomicOr(p.status, DSA_STATUS_CHECK_FAILED);
    return;
  }
  float* wmax = reinterpret_cast<float*>(smem + S::kWmax);  // [4 quarters][64 heads]
  float* svm = reinterpret_cast<float*>(smem + S::kSvm);    // [4]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBars);
  uint64_t* kv_full = bars;        // [2]
  uint64_t* kv_empty = bars + 2;   // [2]: MMA2 of the tile has run
  uint64_t* s_full = bars + 4;     // [2]
  uint64_t* s_empty = bars + 6;    // [2]
  uint64_t* p_full = bars + 8;     // [2]
  uint64_t* drain = bars + 10;     // [2]: the MMA issuers' exit commits
  uint64_t* sched_full = bars + 12;   // [2]: the answer to a request for an item is there
  uint64_t* sched_empty = bars + 14;  // [2]: every warp has read it
  uint64_t* q_full = bars + 16;
  uint64_t* q_empty = bars + 17;
  // Of each tile's MMA2, and of each item's last one: a wait for the last tile's
  // phase of o_tile would also pass while the tile before it still runs.  For the
  // rescale, which waits for tile i - 1 while working on tile i, MMA2 of tile i - 2
  // has run: it released the buffer that tile i came into.
  uint64_t* o_tile = bars + 18;
  uint64_t* o_item = bars + 19;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kMisc + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      dsa::mbar_init(&kv_full[b], G::kWarps);
      dsa::mbar_init(&kv_empty[b], 1);
      dsa::mbar_init(&s_full[b], 1);
      dsa::mbar_init(&s_empty[b], kSoftWarps);
      dsa::mbar_init(&p_full[b], kSoftWarps);
      dsa::mbar_init(&drain[b], 1);
      dsa::mbar_init(&sched_full[b], 1);
      dsa::mbar_init(&sched_empty[b], kThreads / 32);
    }
    dsa::mbar_init(q_full, G::kWarps);
    dsa::mbar_init(q_empty, 1);
    dsa::mbar_init(o_tile, 1);
    dsa::mbar_init(o_item, 1);
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
    dsa::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) dsa::mbar_arrive(&sched_empty[n & 1]);
    __syncwarp();
    return got;
  };

  if (warp < G::kWarps) {
    // ------------------------------------------------------------ gather
    // A row's place depends on its id and the block table, its codes on both:
    // ids are read three tiles ahead, the table two, the codes one.
    const int gt = threadIdx.x, piece = gt & 7, key0 = gt >> 3;
    int tile_ctr = 0, item_ctr = 0;
    bool ok = true;
    // The query's rows, without a stop on the way: head 32 a + 8 c + 2 j + e is
    // row 32 a + 8 j + 2 c + e of the operand, which gives each softmax thread
    // eight consecutive heads.
    auto query_unit = [&](int c) {  // four threads a head, units of 16 bytes sub, sub + 4, ...
      const int h = gt >> 2;
      return (c >> 3) * kQChunkBytes + dsa::sw128_offset((h & 32) + ((h & 6) << 2) + ((h >> 2) & 6) + (h & 1), (c & 7) * 16);
    };
    auto send_query = [&](const Item& w) {
      const __nv_bfloat16* src = p.q + (static_cast<int64_t>(w.t) * p.H + w.h0) * DQK;
      const uint32_t q_addr = dsa::smem_u32(smem);
      const int h = gt >> 2;
      const bool real = h < w.hv;
#pragma unroll 3
      for (int k = 0; k < DQK / 32; ++k) {
        const int c = (gt & 3) + 4 * k;
        cp_async16(q_addr + query_unit(c), src + (real ? h * DQK + c * 8 : 0), real ? 16u : 0u);
      }
    };
    // A thread's part of the query has landed; its elements go where the gather puts those of the keys.
    auto query_landed = [&]() {
      cp_async_wait_all();
      if constexpr (G::kPlaced) {
#pragma unroll 3
        for (int k = 0; k < DQK / 32; ++k) {
          uint4* u = reinterpret_cast<uint4*>(smem + query_unit((gt & 3) + 4 * k));
          *u = to_places(*u);
        }
      }
    };
    // L2 prefetch of a later item's query and ids
    auto prefetch_item = [&](int it) {
      const Item w = get_item(p, it, t_end);
      if (w.i0 >= w.i1) return;
      const uint8_t* q0 = reinterpret_cast<const uint8_t*>(p.q + (static_cast<int64_t>(w.t) * p.H + w.h0) * DQK);
      for (int o = gt * 128; o < w.hv * DQK * 2; o += kGatherThreads * 128) l2_prefetch(q0 + o);
      const int j = w.i0 * kKeys + gt * 32;
      if (j < min(w.i1 * kKeys, w.len)) l2_prefetch(p.idx + static_cast<int64_t>(w.t) * p.K + j);
    };
    // The request for the item after the n-th goes out as that one begins (not
    // again after the answer that there is none).
    int requests = 0;
    auto request = [&](int n) {
      if (!p.steal) return true;
      if (n >= 2 && !dsa::mbar_wait_warp(&sched_empty[n & 1], ((n >> 1) & 1) ^ 1, wt)) return false;
      dsa::fence_proxy_async_smem();
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
      auto load_id = [&](int i, int s) {
        const int j = i * kKeys + s * G::kStep + key0;
        return i < w.i1 && j < w.len ? __ldg(irow + j) : -1;
      };
      const int32_t* trow = p.g.table ? p.g.table + static_cast<int64_t>(b) * p.g.max_blocks : nullptr;
      auto load_block = [&](int id) {  // as the table holds it; -1 beyond the table
        const int page = id >> p.g.lb;
        return !trow || id < 0 ? page : page < p.g.max_blocks ? __ldg(trow + page) : -1;
      };
      auto row_of = [&](int id, int blk) {
        return id >= 0 && blk >= 0 && blk < p.g.n_blocks ? (blk << p.g.lb) + (id & ((1 << p.g.lb) - 1)) : -1;
      };
      // codes of tile i, id and table entry of tile i + 1's keys, id of tile i + 2's
      G codes;
      int id[2], nid[2], blk[2], r[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        r[s] = load_id(w.i0, s);
        id[s] = load_id(w.i0 + 1, s);
        nid[s] = load_id(w.i0 + 2, s);
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) blk[s] = load_block(r[s]);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        r[s] = row_of(r[s], blk[s]);
        blk[s] = load_block(id[s]);
      }
      codes.load_keys(p, r, w.kvh, piece);
      if (SEP) codes.load_values(p, r, w.kvh, piece);
      // MMA1 of the item before has read its query
      if (!dsa::mbar_wait_warp(q_empty, (item_ctr & 1) ^ 1, wt)) break;
      send_query(w);
      for (int i = w.i0; i < w.i1; ++i, ++tile_ctr) {
        const int buf = tile_ctr & 1;
        if (!dsa::mbar_wait_warp(&kv_empty[buf], ((tile_ctr >> 1) & 1) ^ 1, wt)) {
          ok = false;
          break;
        }
        uint8_t* tile = smem + S::kKv + buf * S::kBuf;
        codes.store_keys(tile, reinterpret_cast<float*>(smem + S::kMeta + buf * S::kMetaStep), key0, piece);
        if (SEP) codes.store_values(tile + S::kVOff, key0, piece);
        const bool first = i == w.i0;
        if (first) query_landed();
        dsa::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          dsa::mbar_arrive(&kv_full[buf]);
          if (first) dsa::mbar_arrive(q_full);
        }
        __syncwarp();
        if (i + 1 < w.i1) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            r[s] = row_of(id[s], blk[s]);
            id[s] = nid[s];
            blk[s] = load_block(nid[s]);
            nid[s] = load_id(i + 3, s);
          }
          codes.load_keys(p, r, w.kvh, piece);
          if (SEP) codes.load_values(p, r, w.kvh, piece);
        }
        if (first) {
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
      constexpr uint32_t idesc1 = dsa::idesc_bf16(kKeys, kHG, 0, 0);
      const uint64_t q_desc = dsa::smem_desc(base, 16, 1024, dsa::kSwizzle128B);
      const uint64_t kv_desc = dsa::smem_desc(base + S::kKv, 16, 1024, dsa::kSwizzle128B);
      int tile_ctr = 0, item_ctr = 0;
      int it = blockIdx.x;
      for (int n = 0; it >= 0 && ok; ++n) {
        const Item w = get_item(p, it, t_end);
        it = next_item(n, &ok);
        if (!ok) break;
        if (w.i0 >= w.i1) continue;
        if (!dsa::mbar_wait_warp(q_full, item_ctr & 1, wt)) break;
        for (int i = w.i0; i < w.i1; ++i, ++tile_ctr) {
          const int b = tile_ctr & 1;
          const uint32_t par = (tile_ctr >> 1) & 1;
          const bool got = dsa::mbar_wait(&s_empty[b], par ^ 1, wt) && dsa::mbar_wait(&kv_full[b], par, wt);
          __syncwarp();
          dsa::tc_fence_after();
          const uint64_t a0 = kv_desc + b * (S::kBuf >> 4);
          const uint32_t d = tmem_base + kSCol + b * kHG;
#pragma unroll
          for (int c = 0; c < S::kNk; ++c) {
            const uint64_t ac = a0 + c * (kChunkBytes >> 4), bc = q_desc + c * (kQChunkBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              dsa::umma_bf16_if(leader && got, d, ac + kk * 2, bc + kk * 2, idesc1, (c | kk) != 0);
          }
          if (leader && got) dsa::umma_commit(&s_full[b]);
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
      constexpr uint32_t idesc2 = dsa::idesc_bf16(128, kHG, 1, 1);  // both MN-major
      int tile_ctr = 0;
      const uint64_t v_desc = dsa::smem_desc(base + S::kKv + S::kVOff, kChunkBytes, 1024, dsa::kSwizzle128B);
      const uint64_t p_desc = dsa::smem_desc(base + S::kP, kChunkBytes, 1024, dsa::kSwizzle128B);
      int it = blockIdx.x;
      for (int n = 0; it >= 0 && ok; ++n) {
        const Item w = get_item(p, it, t_end);
        it = next_item(n, &ok);
        if (!ok) break;
        for (int i = w.i0; i < w.i1; ++i, ++tile_ctr) {
          const int b = tile_ctr & 1;
          const bool got = dsa::mbar_wait(&p_full[b], (tile_ctr >> 1) & 1, wt);
          __syncwarp();
          dsa::tc_fence_after();
          const uint64_t a0 = v_desc + b * (S::kBuf >> 4), b0 = p_desc + b * (S::kPStep >> 4);
#pragma unroll
          for (int mb = 0; mb < S::kNv; ++mb) {
            const uint32_t d = tmem_base + kOCol + mb * kHG;
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              dsa::umma_bf16_if(leader && got, d, a0 + mb * (2 * kChunkBytes >> 4) + kk * (16 * 128 >> 4),
                                b0 + kk * (16 * 128 >> 4), idesc2, (i > w.i0 || kk > 0) ? 1u : 0u);
          }
          if (leader && got) {
            dsa::umma_commit(o_tile);
            dsa::umma_commit(&kv_empty[b]);
            if (i + 1 == w.i1) dsa::umma_commit(o_item);
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
    // S^T of 64 keys lies in the first 16 lanes of each quarter.  Of it a thread holds two keys'
    // scores of eight heads: key0 + 8 k (k = 0, 1), and head hb + 2j + e of it is x[4j + 2k + e].
    const int key0 = quarter * 16 + (lane >> 2);
    const int hb = hh * 32 + 8 * (lane & 3);
    // factors of O^T per head (the four warps of a head half write the same ones)
    float* alpha = reinterpret_cast<float*>(smem + S::kAlpha);
    float* fac = reinterpret_cast<float*>(smem + S::kFac);  // [64]: references, then the factors of the result
    uint8_t* rows = smem + S::kRows + sw * 1024;            // this warp's, of the result: 16 heads x 32 dims, 64-byte swizzle
    int tile_ctr = 0, item_ctr = 0;
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
        const int b = tile_ctr & 1;
        const uint32_t par = (tile_ctr >> 1) & 1;
        // the slots' scales come with the gathered tile
        if (!failed) failed = !dsa::mbar_wait(&kv_full[b], par, wt);
        const float* meta = reinterpret_cast<const float*>(smem + S::kMeta + b * S::kMetaStep) + key0;
        float sk[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) sk[k] = meta[8 * k] > 0.f ? meta[8 * k] : 0.f;
        if (!failed) failed = !dsa::mbar_wait(&s_full[b], par, wt);
        __syncwarp();
        dsa::tc_fence_after();
        float x[16];
        {
          uint32_t v[16];
          dsa::tmem_ld16x256b_x4(tmem_base + lane_off + kSCol + b * kHG + hh * 32, v);
          dsa::tmem_wait_ld();
#pragma unroll
          for (int r = 0; r < 16; ++r) x[r] = __uint_as_float(v[r]);
        }
        dsa::tc_fence_before();
        __syncwarp();
        if (lane == 0) dsa::mbar_arrive(&s_empty[b]);
        // scores in powers of two against the references; -inf where there is no slot
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float c = p.scale_log2 * sk[k];
#pragma unroll
          for (int h = 0; h < 8; h += 2) {
            const float2 y = fma2(make_float2(x[at(k, h)], x[at(k, h + 1)]), make_float2(c, c), make_float2(nm[h], nm[h + 1]));
            x[at(k, h)] = sk[k] > 0.f ? y.x : -INFINITY, x[at(k, h + 1)] = sk[k] > 0.f ? y.y : -INFINITY;
          }
        }
        float most = x[0], sv_most = 0.f;
#pragma unroll
        for (int r = 1; r < 16; ++r) most = fmaxf(most, x[r]);
        if (SEP && G::kScaled) {
#pragma unroll
          for (int k = 0; k < 2; ++k) sk[k] = sk[k] > 0.f ? meta[kKeys + 8 * k] : 0.f;  // from here on the values' scales
        }
        sv_most = fmaxf(sk[0], sk[1]);
        const bool ex = unset || most > kMove || sv_most > ref;
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
            for (int m = 0; m < 4; ++m) {
              const int h = 4 * g4 + m;
              // by how much the reference moves: to the tile's maximum, if that
              // passes it by kMove or is the first
              const float up = (unset ? tm[m] > -INFINITY : tm[m] > kMove) ? tm[m] : 0.f;
              const float a = unset ? 1.f : ex2(-up);
              moved |= up != 0.f;
              l_part[h] *= a;
              nm[h] -= up;
#pragma unroll
              for (int k = 0; k < 2; ++k) x[at(k, h)] -= up;
              if (lane < 4) alpha[hb + h] = a * ratio;
            }
          }
          unset = unset && !(sv_max > 0.f);
          need_rescale = __any_sync(0xffffffffu, moved) && !first;
        }
        // P^T rows key0 + 8 k: the thread's eight heads are one 16-byte unit of a row of 64.  MMA2 of
        // the buffer's last tile has read it: this tile came into the buffer.
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float wk = sk[k] * inv;  // (2^-E alone stays in range)
          uint32_t u[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float p0 = ex2(x[at(k, 2 * j)]), p1 = ex2(x[at(k, 2 * j + 1)]);
            const float2 l2 = add2(make_float2(l_part[2 * j], l_part[2 * j + 1]), make_float2(p0, p1));
            l_part[2 * j] = l2.x, l_part[2 * j + 1] = l2.y;
            const float2 p2 = mul2(make_float2(p0, p1), make_float2(wk, wk));
            u[j] = pack_bf16x2(p2.x, p2.y);
          }
          *reinterpret_cast<uint4*>(smem + S::kP + b * S::kPStep + dsa::sw128_offset(key0 + 8 * k, hb * 2)) =
              make_uint4(u[0], u[1], u[2], u[3]);
        }
        if (need_rescale) {
          // MMA2 of the previous tile must have landed before O^T is scaled
          if (!failed) failed = !dsa::mbar_wait(o_tile, (tile_ctr - 1) & 1, wt);
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
        if (lane == 0) dsa::mbar_arrive(&p_full[b]);
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
      if (st < 64) {
        const float mc = fac[st];
        const bool any = l != 0.f;  // true for NaN too
        float f = 0.f;
        if (p.splits > 1) {
          // a split's mean value, which stays in range where the sum might not
          if (any) f = ref / l;
          if (st < w.hv) p.part_s[(orow + st) * p.splits + w.split] = make_float4(mc, l, m_max, 0.f);
        } else {
          const float sk = sink * kLog2e;
          float lse_v = sink, lkv = INFINITY;
          if (any) {
            const float M = fmaxf(mc, sk);
            const float a = exp2f(mc - M);
            const float z = l * a + exp2f(sk - M);
            f = a / z * ref;
            lse_v = (M + log2f(z)) * kLn2;
            lkv = (mc + log2f(l)) * kLn2;
          }
          if (st < w.hv) {
            p.lse[orow + st] = lse_v;
            if (p.lse_kv) p.lse_kv[orow + st] = lkv;
            if (kMax) p.max_logits[orow + st] = any ? max_logit(l, m_max) : -INFINITY;
          }
        }
        fac[st] = f;
      }
      // O^T is complete with the last tile's MMA2
      if (!failed) failed = !dsa::mbar_wait(o_item, item_ctr & 1, wt);
      ++item_ctr;
      group_sync();
      dsa::tc_fence_after();
      const int hcount = min(32, w.hv - hh * 32);
      const uint32_t tm_o = tmem_base + lane_off + kOCol + hh * 32;
      if (hcount <= 0) {
        // (no head of this half is real)
      } else if (p.splits > 1) {
        const float* f32 = fac + hh * 32;
        const int dim = G::kPlaced ? (lane & 24) + ((lane & 7) >> 1) + 4 * (lane & 1) : lane;
#pragma unroll 1
        for (int mb = 0; mb < S::kNv; ++mb) {
          uint32_t v[32];
          __syncwarp();
          dsa::tmem_ld32(tm_o + mb * kHG, v);
          dsa::tmem_wait_ld();
          float* o = p.part_o + ((orow + hh * 32) * p.splits + w.split) * DV + mb * 128 + quarter * 32 + dim;
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
                __stcs(reinterpret_cast<uint4*>(o0 + mb * 128 + (c0 + k * 8) * DV), [&] {
                  const uint4 u = *reinterpret_cast<const uint4*>(rows + sw64_offset(h, lane & 3));
                  return G::kPlaced ? from_places(u) : u;
                }());
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

// Joins the splits of one (token, head) per CTA: with M the largest of the references and the sink, a_s = 2^(m_s - M) l_s
// and z = sum_s a_s + 2^(sink - M), out = sum_s a_s O_s / z of the splits' means O_s.  lse_kv is the slots' alone, whose
// sum against a sink far above them is nothing: under a sink it is taken again against the largest reference.
template <int DV>
__global__ void __launch_bounds__(DV / 4) attn_cache_join_kernel(const Params p) {
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
  const float a = have ? s.y * exp2f(s.x - M) : 0.f;
  float l = a;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float z = any ? l + exp2f(sk - M) : 1.f;
  const float share = a / z;  // at most 1: a mean of means stays in range
  const bool under = p.lse_kv && any && sk > m;  // (the same in all lanes)
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4* o = reinterpret_cast<const float4*>(p.part_o + row * p.splits * DV) + threadIdx.x;
  for (int k = 0; k < p.splits; ++k) {
    const float ak = __shfl_sync(0xffffffffu, share, k);
    if (__shfl_sync(0xffffffffu, have, k)) {
      const float4 v = __ldcs(o + k * (DV / 4));
      acc.x = fmaf(ak, v.x, acc.x);
      acc.y = fmaf(ak, v.y, acc.y);
      acc.z = fmaf(ak, v.z, acc.z);
      acc.w = fmaf(ak, v.w, acc.w);
    }
  }
  reinterpret_cast<uint2*>(p.out + row * DV)[threadIdx.x] = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
  if (threadIdx.x == 0) {
    p.lse[row] = any ? (M + log2f(z)) * kLn2 : sink;
    if (p.lse_kv && !under) p.lse_kv[row] = any ? (M + log2f(l)) * kLn2 : INFINITY;
    if (p.max_logits) p.max_logits[row] = any ? max_logit(l, mx) : -INFINITY;
  }
  // (read again: kept beside the values, the sums would cost eight registers and with those a quarter of the CTAs)
  if (under && threadIdx.x < 32) {
    const float4 r = lane < p.splits ? p.part_s[row * p.splits + lane] : make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
    float top = r.y != 0.f ? r.x : -INFINITY;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float l_kv = r.y != 0.f ? r.y * exp2f(r.x - top) : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l_kv += __shfl_xor_sync(0xffffffffu, l_kv, o);
    if (lane == 0) p.lse_kv[row] = (top + log2f(l_kv)) * kLn2;
  }
}

// Splits of each row's slots: the number that makes the longest CTA shortest,
// counting a wave of CTAs as its tiles plus kItemTiles tiles for the first loads,
// the query and the epilogue, and joining as kJoinTiles tiles plus one per 16
// splits.  Measured (rows of 576, 2048 slots, 128 heads; microseconds with 1, 2, 4, 8, 16 splits):
// 16 rows 64, 41, 28, 35, 49; 32 rows 74, 48, 52, 66; 100 rows 142, 133, 135 (the last with 3).
// One row of 64 heads, 65536 slots: 1696, 854, 432, 221, 117, and 66 with 32.
constexpr int kItemTiles = 6, kJoinTiles = 5;

inline int plan_splits(int64_t units, int K, int join_tiles = kJoinTiles) {
  const int nt = (K + kKeys - 1) / kKeys;
  int best = 1;
  int64_t cost = INT64_MAX;
  for (int s = 1; s <= kMaxSplits && s <= nt; ++s) {
    const int64_t waves = (units * s + kPlanSms - 1) / kPlanSms;
    const int64_t c = 16 * (waves * ((nt + s - 1) / s + kItemTiles) + (s > 1 ? join_tiles : 0)) + (s > 1 ? s : 0);
    if (c < cost) cost = c, best = s;
  }
  return best;
}

inline bool known_shape(int T, int H, int Hc, int Dqk, int Dv, int K) {
  const bool form = ((Dqk == 576 || Dqk == 512) && Dv == 512) || (Dqk == 256 && Dv == 256);
  return form && T >= 1 && H >= 1 && Hc >= 1 && H % Hc == 0 && K >= 1 && K <= DSA_KV8_MAX_SLOTS;
}

// Work items before splitting, with groups of hg heads.
inline int64_t units_of(int T, int H, int Hc, int hg) { return static_cast<int64_t>(T) * Hc * ((H / Hc + hg - 1) / hg); }

inline size_t part_bytes(int T, int H, int splits) {
  return (static_cast<size_t>(T) * H * splits * sizeof(float4) + 255) / 256 * 256;
}

template <int DV>
int launch_join(const Params& p, int T, cudaStream_t stream) {
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
  if (cudaLaunchKernelEx(&cfg, attn_cache_join_kernel<DV>, p) != cudaSuccess) return dsa::launch_error("attn_cache_join_kernel");
  return DSA_OK;
}

template <class G, int DQK, int DV, bool SEP, bool kMax>
int launch_form(const Params& p, int T, cudaStream_t stream) {
  using S = Shape<DQK, DV, SEP>;
  constexpr int smem = S::kTotal;
  auto kernel = attn_cache_kernel<G, DQK, DV, SEP, kMax>;
  static std::atomic<uint64_t> ready{0};  // devices where the kernel's shared memory is allowed
  int dev = 0;
  cudaGetDevice(&dev);  // below 64: check_device
  if (!(ready.load(std::memory_order_acquire) >> dev & 1)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return dsa::launch_error("attn_cache_kernel smem attribute");
    ready.fetch_or(uint64_t{1} << dev, std::memory_order_release);
  }
  kernel<<<p.n_items, kThreads, smem, stream>>>(p);
  int rc = dsa::launch_error("attn_cache_kernel");
  if (rc != DSA_OK || p.splits == 1) return rc;
  return launch_join<DV>(p, T, stream);
}

template <class G, int DQK, int DV, bool SEP>
int launch(const Params& p, int T, cudaStream_t stream) {
  return p.max_logits ? launch_form<G, DQK, DV, SEP, true>(p, T, stream)
                      : launch_form<G, DQK, DV, SEP, false>(p, T, stream);
}

// The workspace of rows in several splits.
inline void take_workspace(Params& p, int T, void* workspace) {
  p.part_s = static_cast<float4*>(workspace);
  p.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + part_bytes(T, p.H, p.splits));
}

// What a call hands over, under the names of its own entry point.
struct Call {
  const char *fn, *codes, *values;  // names of the entry point and of its code arguments
  const void* q;
  const void* k;
  const void* k_scale;
  const void* v;
  const void* v_scale;
  const int32_t* idx;
  const int32_t* topk_length;
  const float* sink;
  const int32_t* cu_seqlens;
  const int32_t* block_table;
  int n_seqs, T, H, Hc, Dqk, Dv, K, block, n_blocks, max_blocks;
  float scale;
  void* out;
  float *lse, *lse_kv, *max_logits;
  void* workspace;
  size_t ws_bytes, need;
  int hg, splits;  // heads of a group, splits of a row's slots
};

// Checks a call and fills the kernels' arguments, but for the codes and scales.
inline int fill(const Call& c, Params* out, int* sm_count = nullptr) {
  const char* fn = c.fn;
  const bool separate = c.Dqk == 256 && c.Dv == 256 && c.v && c.v_scale;
  const bool latent = (c.Dqk == 576 || c.Dqk == 512) && c.Dv == 512 && !c.v && !c.v_scale;
  if (!latent && !separate)
    return set_error(DSA_ERR_VALUE,
                     "%s: (Dqk, Dv) must be (576|512, 512) without %s and v_scale or (256, 256) with both", fn, c.values);
  if (c.T < 0 || c.H < 1 || c.Hc < 1 || c.Hc > DSA_KV8_MAX_HEADS || c.H % c.Hc != 0 || c.H / c.Hc > 128 || c.K < 0 ||
      c.K > DSA_KV8_MAX_SLOTS)
    return set_error(DSA_ERR_VALUE, "%s: need T >= 0, 0 <= K <= %d, 1 <= Hc <= %d, H a multiple of Hc, H / Hc <= 128",
                     fn, DSA_KV8_MAX_SLOTS, DSA_KV8_MAX_HEADS);
  const int64_t units = c.T > 0 ? units_of(c.T, c.H, c.Hc, c.hg) : 0;
  if (units * kMaxSplits > INT_MAX || static_cast<int64_t>(c.T) * c.H > INT_MAX)
    return set_error(DSA_ERR_VALUE, "%s: T * H exceeds the int32 range of work items", fn);
  if (c.n_blocks < 1 || c.block < 1 || c.block > DSA_KV8_MAX_BLOCK || (c.block & (c.block - 1)) != 0)
    return set_error(DSA_ERR_VALUE, "%s: need n_blocks >= 1 and block a power of two in [1, %d]", fn, DSA_KV8_MAX_BLOCK);
  if (static_cast<int64_t>(c.n_blocks) * c.block > INT_MAX)
    return set_error(DSA_ERR_VALUE, "%s: n_blocks * block exceeds the int32 row range", fn);
  if (c.block_table && (c.n_seqs < 1 || c.max_blocks < 1 || !c.cu_seqlens))
    return set_error(DSA_ERR_VALUE, "%s: a block table needs cu_seqlens, n_seqs >= 1 and max_blocks >= 1", fn);
  if (!(c.scale > 0.f) || !(c.scale < INFINITY))
    return set_error(DSA_ERR_VALUE, "%s: scale must be finite and > 0", fn);
  if (!c.k || !c.k_scale || (c.T > 0 && (!c.q || !c.out || !c.lse || (c.K > 0 && !c.idx))))
    return set_error(DSA_ERR_VALUE, "%s: NULL pointer", fn);
  if (!aligned(c.q, 16) || !aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.out, 16))
    return set_error(DSA_ERR_VALUE, "%s: q, %s, %s and out must be 16-byte aligned", fn, c.codes, c.values);
  if (c.need > 0 && (!c.workspace || c.ws_bytes < c.need || !aligned(c.workspace, 256)))
    return set_error(DSA_ERR_WORKSPACE, "%s: needs a 256-byte aligned workspace of %zu bytes, got %zu", fn, c.need,
                     c.workspace ? c.ws_bytes : static_cast<size_t>(0));
  int sms = 0;
  const int rc = check_device(&sms);
  if (sm_count) *sm_count = sms;
  if (rc != DSA_OK || c.T == 0) return rc;
  int lb = 0;
  while ((1 << lb) < c.block) ++lb;
  Params p{};
  p.q = static_cast<const __nv_bfloat16*>(c.q);
  p.idx = c.idx;
  p.topk_length = c.topk_length;
  p.sink = c.sink;
  p.g = Kv8Geom{c.cu_seqlens, nullptr, c.block_table, c.n_seqs, c.T, lb, c.n_blocks, c.max_blocks};
  p.out = static_cast<__nv_bfloat16*>(c.out);
  p.lse = c.lse;
  p.lse_kv = c.lse_kv;
  p.max_logits = c.max_logits;
  p.H = c.H;
  p.Hc = c.Hc;
  p.K = c.K;
  p.G = (c.H / c.Hc + c.hg - 1) / c.hg;
  p.splits = c.splits;
  p.n_items = static_cast<int>(units * p.splits);
  p.status = device_status_ptr();
  p.steal = p.n_items > sms;
  p.scale_log2 = c.scale * kLog2e;
  *out = p;
  return DSA_OK;
}

}  // namespace kv8_attn
}  // namespace dsa

