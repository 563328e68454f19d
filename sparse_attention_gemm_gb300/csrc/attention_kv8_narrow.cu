// attention_kv8_narrow.cu -- sparse attention over the 8-bit block cache in
// groups of 16 query heads, for calls whose KV heads serve at most 16 query
// heads and for calls of few rows.
//
// Both products run on the codes as they lie in the cache (kind::f8f6f4): with
// 16 heads, what counts is that two CTAs of two or three tiles each fit an
// SM, and widened codes would not.  The other operands are sums of 8-bit terms.
//   query:   q / s = hi + lo / 16 in E4M3, s the power of two that brings the head's
//            largest element to (224, 448].  Exact (8 bits) down to 2^-14 of
//            that, off by at most 2^-22 of it below.
//   weights: w = 14 * 2^(x - R), x the score and the value's scale together in powers of two
//            and R a reference of the head's x, one of two places: itself where it is
//            2^-6 or more, else 2^14 times itself, each with an accumulator of its own.
//            There it is an E4M3 term and, for what that leaves, one in E5M2: off by at
//            most 2^-8 of itself, as bf16 would be, for 29 powers of two from the
//            largest 448 down; below by at most 2^-31 of 14, which the largest is
//            within a factor of four of (two where scales are powers of two).
//            (One place of two E4M3 terms ended at 2^-13.8 of the largest weight times the largest scale:
//            rows whose largest weight meets a small value lost their output.)
// The sum of exp(s_j) has a reference m of its own, since scales do not enter it.
// Both are whole numbers: 2^(R - m), which joins them at the end, is exact.
//
// One work item (token, KV head, 16 heads, split of its slots) per CTA, two
// CTAs on an SM: an item is a chain of latencies (ids,
// table, gather, scores, weights, sums), and what hides one CTA's is the other.
//   MMA1  S^T[key, hi|lo head] = K[key, :] . Q[hi|lo head, :]^T  (M = 64 keys, N = 32)
//   MMA2  O^T[dim, place|place head] += V^T[dim, key] . P^T[key, place|place head]
//         (M = 128 dims, N = 32), once for each term
// Splits of a row are the CTAs of a cluster: each leaves its mean value in its own
// shared memory, and each joins the dims of its rank from everyone's.  No
// second kernel, no workspace, and the order of the sum is the ranks'.
// What bounds it: 1.8K cycles of a pair of CTAs a tile (copies in flight, the weights' terms), and
// what an item does once, 10K cycles: first loads 4K (ids, table entries), first
// tile 2K, softmax's first references 1.6K, results 2.3K, join 4K.  Shared memory
// (a tile of 64 keys 36 KB, two of them) holds two CTAs, not three.  96 rows of 2 x
// 12 heads of 256 + 256, 1027 slots: 24.8 us, 3.6 TB/s; 1024 rows of 16 heads of 512 over
// documents of 341: 41.4 us; one row of 64 heads, 2048 slots: 12.6 us (the 64-head
// kernel and its join: 14.4).  With weights of one place of two E4M3 terms, which lost
// small ones: 20.8, 36.2 and 11.2 us.  Codes widened to bf16, weights in bf16 (eight gather warps,
// one tile buffer): 38.3, 56.8 and 15.5 us; only the values widened, a block of 128 dims at a
// time: 31.8, 63.5 and 16.2.
// Tried and slower: the first tile's copies or the query's conversion before the
// set-up barrier (36.7 and 36.4 us instead of 36.1 for the packed rows).
//
// Warps: 0..3 gather, 4..7 query conversion, softmax and epilogue, 8 MMA1, 9 MMA2.
#include "attention_kv8.cuh"

namespace {

using namespace dsa::kv8_attn;

constexpr int kHG = 16;
constexpr int kGatherWarps = 4;
constexpr int kGatherThreads = kGatherWarps * 32;
constexpr int kGatherKeys = kGatherThreads / 8;  // keys one gather step covers
constexpr int kGatherSteps = kKeys / kGatherKeys;
constexpr int kSoftWarps = 4;
constexpr int kSoftThreads = kSoftWarps * 32;
constexpr int kMmaWarp = kGatherWarps + kSoftWarps;
constexpr int kThreads = (kMmaWarp + 2) * 32;
constexpr uint32_t kQChunkBytes = 2 * kHG * 128;  // hi and lo of 16 heads x 128 codes
constexpr uint32_t kPBytes = kKeys * 2 * kHG;     // one term of P^T, both places
constexpr uint32_t kSwizzle32B = 6;
constexpr int kCols = 2 * kHG;  // TMEM columns of one S^T buffer or one block of O^T
constexpr int kOCol = 2 * kCols;
constexpr int kMaxCluster = 8;
// A reference moves when a tile passes it by more than this (powers of two).
// Weights then reach 14 * 2^5, E4M3's largest.
constexpr float kMoveR = 5.0f, kMoveM = 16.0f;
constexpr float kWeight = 14.0f;
constexpr float kLow = 0.015625f, kLowScale = 16384.0f;  // weights below 2^-6 go to the second place, times 2^14

template <int DQK, int DV, bool SEP>
struct Shape {
  static constexpr int kFull = DQK / 128;
  static constexpr bool kTail = DQK % 128 != 0;
  static constexpr int kNv = DV / 128;
  static constexpr uint32_t kVOff = SEP ? kFull * kChunkBytes : 0;
  static constexpr uint32_t kTailOff = kFull * kChunkBytes;
  static constexpr uint32_t kBuf = (kFull + (SEP ? kNv : 0)) * kChunkBytes + (kTail ? kKeys * 64 : 0);
  static constexpr int kStages = SEP ? 3 : 2;  // what two CTAs of an SM have room for
  static constexpr uint32_t kTmem = kOCol + kNv * kCols <= 128 ? 128 : 256;
  static constexpr uint32_t kKv = 0;
  static constexpr uint32_t kQ = kStages * kBuf;
  static constexpr uint32_t kQTail = kQ + kFull * kQChunkBytes;
  static constexpr uint32_t kP = kQTail + (kTail ? 2 * kHG * 64 : 0);  // [kPBufs][2 terms]
  static constexpr int kPBufs = SEP ? 1 : 2;
  // scale of each slot's key and, behind them, value (one number where they are one); 0: no slot
  static constexpr uint32_t kMeta = kP + kPBufs * 2 * kPBytes;
  static constexpr uint32_t kMetaStep = kKeys * (SEP ? 8 : 4);
  static constexpr uint32_t kWmax = kMeta + kStages * kMetaStep;  // float [4][16]
  static constexpr uint32_t kYmax = kWmax + 256;                  // float [4][16]
  static constexpr uint32_t kRed = kYmax + 256;                   // float [4][16] sums
  static constexpr uint32_t kRedM = kRed + 256;                   // float [4][16] maxima
  static constexpr uint32_t kAlpha = kRedM + 256;                 // float [16]
  static constexpr uint32_t kFac = kAlpha + 64;                   // float [16]
  static constexpr uint32_t kFacR = kFac + 64;                    // float [16]
  static constexpr uint32_t kStats = kFacR + 64;                  // float4 [16]: reference, sum, maximum, sink
  static constexpr uint32_t kSvm = kStats + 256;                  // float [4]
  static constexpr uint32_t kQexp = kSvm + 16;                    // uint8 [16]
  static constexpr uint32_t kBars = kQexp + 16;
  static constexpr uint32_t kMisc = kBars + 18 * 8;
  static constexpr uint32_t kTotal = kMisc + 16;
  static constexpr uint32_t kPart = kKv;  // float [16][DV]: a split's mean value, once its products have run
  static_assert(kTotal <= (228 * 1024) / 2 - 1024, "two CTAs' shared memory");
  static_assert(kHG * DV * 4 <= kStages * kBuf, "a split's mean value fits");
  static_assert(kBuf % 1024 == 0 && kQ % 1024 == 0 && kP % 1024 == 0, "alignment");
};

__device__ __forceinline__ void group_sync() {
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(kSoftThreads) : "memory");
}
__device__ __forceinline__ bool group_any(bool x) {
  __syncwarp();
  return dsa::named_bar_any(1, kSoftThreads, x);
}
// Every thread of every CTA of the cluster arrives, on every path.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ uint32_t of_rank(uint32_t smem_addr, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr), "r"(rank));
  return a;
}
__device__ __forceinline__ float4 ld_cluster(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

// Byte offset of 16-byte unit `u` of row `r` in rows of 32 bytes, 32-byte swizzle.
__device__ __forceinline__ uint32_t sw32_offset(uint32_t r, uint32_t u) { return r * 32u + ((u ^ ((r >> 2) & 1u)) << 4); }

// Combines v[0..3] (one value per head hb + i) over the 8 lanes that share
// lane & 3: lane keeps head hb + own_head(lane).
__device__ __forceinline__ int own_head(int lane) { return ((lane >> 4) & 1) * 2 + ((lane >> 3) & 1); }
template <class F>
__device__ __forceinline__ float fold4(const float (&v)[4], int lane, F f) {
  const bool up = (lane & 16) != 0;
  const float a = f(up ? v[2] : v[0], __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 16));
  const float b = f(up ? v[3] : v[1], __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 16));
  const bool up2 = (lane & 8) != 0;
  const float c = f(up2 ? b : a, __shfl_xor_sync(0xffffffffu, up2 ? a : b, 8));
  return f(c, __shfl_xor_sync(0xffffffffu, c, 4));
}

// What the sums of a head give: the factor of its weighted values and the statistics.
struct Norm {
  float f, lse, lse_kv;
};
__device__ __forceinline__ Norm norm_of(float m, float l, float sink) {
  Norm n{0.f, sink, INFINITY};
  if (l != 0.f) {  // true for NaN too
    const float sk = sink * kLog2e, M = fmaxf(m, sk);
    const float a = exp2f(m - M);
    const float z = l * a + exp2f(sk - M);
    n.f = a / z;
    n.lse = (M + log2f(z)) * kLn2;
    n.lse_kv = (m + log2f(l)) * kLn2;
  }
  return n;
}

template <int DQK, int DV, bool SEP>
__global__ void __launch_bounds__(kThreads, 2) attn_kv8_narrow_kernel(const Params p) {
  using S = Shape<DQK, DV, SEP>;
  constexpr int ST = S::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];  // the kernel has no other shared memory

  // the item: longest rows first (they are the last of a packed prompt)
  const int unit = blockIdx.x / p.splits, split = blockIdx.x - unit * p.splits;
  const int u = p.n_items - 1 - unit;
  const int per = p.Hc * p.G, group = p.H / p.Hc;
  const int t = u / per, r0 = u - t * per, kvh = r0 / p.G, g0 = (r0 - kvh * p.G) * kHG;
  const int h0 = kvh * group + g0, hv = min(kHG, group - g0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool aligned = (dsa::smem_u32(smem) & 1023u) == 0;  // else every swizzle breaks
  if (!aligned && threadIdx.x == 0) atomicOr(p.status, DSA_STATUS_CHECK_FAILED);
  // a row of padding behind the last sequence: nothing is read or written for it
  const bool dead = p.g.table && t >= __ldg(p.g.cu + p.g.n_seqs);
  int len = p.K;
  if (p.topk_length) {
    len = __ldg(p.topk_length + t);
    len = len < 0 ? 0 : (len > p.K ? p.K : len);
  }
  const int nt = aligned && !dead ? (len + kKeys - 1) / kKeys : 0;
  // (nt <= 2^25 and at most 8 splits: the products fit)
  const int i0 = split == 0 ? 0 : static_cast<int>(static_cast<uint32_t>(nt) * split / p.splits);
  const int i1 = static_cast<int>(static_cast<uint32_t>(nt) * (split + 1) / p.splits);

  float* wmax = reinterpret_cast<float*>(smem + S::kWmax);
  float* ymax = reinterpret_cast<float*>(smem + S::kYmax);
  float* red = reinterpret_cast<float*>(smem + S::kRed);
  float* redm = reinterpret_cast<float*>(smem + S::kRedM);
  float* alpha = reinterpret_cast<float*>(smem + S::kAlpha);
  float* fac = reinterpret_cast<float*>(smem + S::kFac);
  float* facr = reinterpret_cast<float*>(smem + S::kFacR);
  float4* stats = reinterpret_cast<float4*>(smem + S::kStats);
  float* svm = reinterpret_cast<float*>(smem + S::kSvm);
  uint8_t* qexp = smem + S::kQexp;  // exponents of the query scales (biased; 255: not finite)
  float* part = reinterpret_cast<float*>(smem + S::kPart);
  uint8_t* row16 = smem + S::kPart;  // [DV / 32] x 16 heads x 32 dims, 64-byte swizzle: the results of an undivided row
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBars);
  uint64_t* kv_full = bars;       // [3]
  uint64_t* kv_empty = bars + 3;  // [3]
  uint64_t* s_full = bars + 6;    // [2]
  uint64_t* s_empty = bars + 8;   // [2]
  uint64_t* p_full = bars + 10;   // [2]
  uint64_t* p_empty = bars + 12;  // [2]: MMA2 of the tile has run
  uint64_t* q_full = bars + 14;
  uint64_t* drain = bars + 15;    // [2]: the MMA issuers' exit commits
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kMisc + 4);

  // First loads, before the barriers and TMEM are there: the gather warps'
  // ids of two tiles and table entries of one, the softmax warps' query.
  static_assert(kGatherThreads == 8 * kHG, "eight threads a head");
  const int64_t orow = static_cast<int64_t>(t) * p.H + h0;
  const int32_t* irow = p.idx + static_cast<int64_t>(t) * p.K;
  auto slot_of = [&](int i, int kg) { return i * kKeys + kg * kGatherKeys + static_cast<int>(threadIdx.x >> 3); };
  const int32_t* trow = nullptr;
  auto load_block = [&](int x) {  // as the table holds it; -1 beyond the table
    const int page = x >> p.g.lb;
    return !trow || x < 0 ? page : page < p.g.max_blocks ? __ldg(trow + page) : -1;
  };
  int id[kGatherSteps], nid[kGatherSteps], blk[kGatherSteps];
  constexpr int kPieces = DQK / 64;  // 16-byte pieces of a head's row a thread converts
  const int st = threadIdx.x - kGatherThreads, hq = st >> 3, sub = st & 7;
  uint4 qv[kPieces];
  if (warp < kGatherWarps) {
#pragma unroll
    for (int kg = 0; kg < kGatherSteps; ++kg) {
      id[kg] = slot_of(i0, kg) < p.K ? __ldg(irow + slot_of(i0, kg)) : -1;
      nid[kg] = slot_of(i0 + 1, kg) < p.K ? __ldg(irow + slot_of(i0 + 1, kg)) : -1;
    }
    if (p.g.table) trow = p.g.table + static_cast<int64_t>(dsa::kv8_seq_warp(p.g.cu, p.g.n_seqs, t)) * p.g.max_blocks;
#pragma unroll
    for (int kg = 0; kg < kGatherSteps; ++kg) {
      id[kg] = slot_of(i0, kg) < len ? id[kg] : -1;
      nid[kg] = i0 + 1 < i1 && slot_of(i0 + 1, kg) < len ? nid[kg] : -1;
      blk[kg] = load_block(id[kg]);
    }
  } else if (warp < kMmaWarp) {
    const uint4* src = reinterpret_cast<const uint4*>(p.q + (orow + hq) * DQK) + sub;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) qv[k] = hq < hv ? __ldg(src + 8 * k) : make_uint4(0, 0, 0, 0);
  }

  if (aligned) {
    if (threadIdx.x == kThreads - 32) {  // (a warp that has nothing else to do)
      for (int b = 0; b < ST; ++b) {
        dsa::mbar_init(&kv_full[b], kGatherThreads);
        dsa::mbar_init(&kv_empty[b], 1);
      }
      for (int b = 0; b < 2; ++b) {
        dsa::mbar_init(&s_full[b], 1);
        dsa::mbar_init(&s_empty[b], kSoftWarps);
        dsa::mbar_init(&p_full[b], kSoftWarps);
        dsa::mbar_init(&p_empty[b], 1);
        dsa::mbar_init(&drain[b], 1);
      }
      dsa::mbar_init(q_full, kSoftWarps);
      *abort_flag = 0;
      dsa::fence_barrier_init();
    }
    __syncwarp();
    if (warp == kMmaWarp) dsa::tmem_alloc(tmem_slot, S::kTmem);
  }
  dsa::tc_fence_before();
  __syncthreads();
  dsa::tc_fence_after();
  const uint32_t tmem_base = aligned ? *tmem_slot : 0;
  const dsa::Waiter wt = dsa::make_waiter(abort_flag, p.status);

  if (i0 >= i1) {
    // no slots: sums of nothing
    if (threadIdx.x < kHG)
      stats[threadIdx.x] = make_float4(-INFINITY, 0.f, -INFINITY, p.sink && threadIdx.x < hv ? __ldg(p.sink + h0 + threadIdx.x) : -INFINITY);
    if (p.splits == 1 && !dead) {
      for (int h = 0; h < hv; ++h)
        for (int d = threadIdx.x; d < DV; d += kThreads) p.out[(orow + h) * DV + d] = __float2bfloat16_rn(0.f);
      if (threadIdx.x < hv) {
        p.lse[orow + threadIdx.x] = p.sink ? __ldg(p.sink + h0 + threadIdx.x) : -INFINITY;
        if (p.lse_kv) p.lse_kv[orow + threadIdx.x] = INFINITY;
        if (p.max_logits) p.max_logits[orow + threadIdx.x] = -INFINITY;
      }
    }
  } else if (warp < kGatherWarps) {
    // ------------------------------------------------------------ gather
    // Thread gt covers piece (gt & 7) (16 codes) of keys (gt >> 3) + 16 kg of
    // every chunk.  A row's place depends on its id and the block table: ids
    // are read two tiles ahead, the table one tile ahead.
    const int gt = threadIdx.x, piece = gt & 7, key0 = gt >> 3;
    const uint32_t kv_addr = dsa::smem_u32(smem) + S::kKv, meta_addr = dsa::smem_u32(smem) + S::kMeta;
    for (int i = i0, ctr = 0; i < i1; ++i, ++ctr) {
      const int stage = ctr % ST;
      int cur[kGatherSteps];
#pragma unroll
      for (int kg = 0; kg < kGatherSteps; ++kg) {
        cur[kg] = id[kg] >= 0 && blk[kg] >= 0 && blk[kg] < p.g.n_blocks
                      ? (blk[kg] << p.g.lb) + (id[kg] & ((1 << p.g.lb) - 1))
                      : -1;
        id[kg] = nid[kg];
        blk[kg] = load_block(nid[kg]);
        nid[kg] = i + 2 < i1 && slot_of(i + 2, kg) < len ? __ldg(irow + slot_of(i + 2, kg)) : -1;
      }
      const uint32_t ph = ((ctr / ST) & 1) ^ 1;
      if (!dsa::mbar_wait_warp(&kv_empty[stage], ph, wt)) break;
      const uint32_t buf = kv_addr + stage * S::kBuf;
      {
        // the scales: lanes with piece kg and kg + 4 take key kg's (with V, its key scale and its value scale)
        int r = cur[0];
#pragma unroll
        for (int kg = 1; kg < kGatherSteps; ++kg) r = (piece & 3) == kg ? cur[kg] : r;
        const int64_t at = static_cast<int64_t>((r >= 0 ? r : 0) >> p.g.lb) * p.Hc + kvh;
        const bool value = SEP && piece >= 4;
        if (dsa::check(r < (p.g.n_blocks << p.g.lb), p.status))
          cp_async4(meta_addr + stage * S::kMetaStep + (value ? kKeys * 4 : 0) + ((piece & 3) * kGatherKeys + key0) * 4,
                    (value ? p.v_scale : p.k_scale) + at, r >= 0 ? 4u : 0u);
      }
#pragma unroll
      for (int kg = 0; kg < kGatherSteps; ++kg) {
        const int key = kg * kGatherKeys + key0;
        const uint32_t nbytes = cur[kg] >= 0 ? 16u : 0u;
        const int64_t rh = static_cast<int64_t>(cur[kg] >= 0 ? cur[kg] : 0) * p.Hc + kvh;
        // checked build: the row is inside the cache
        if (!dsa::check(cur[kg] < (p.g.n_blocks << p.g.lb), p.status)) continue;
        const uint8_t* krow = p.k8 + rh * DQK + piece * 16;
        const uint32_t dst = buf + dsa::sw128_offset(key, piece * 16);
#pragma unroll
        for (int c = 0; c < S::kFull; ++c) cp_async16(dst + c * kChunkBytes, krow + c * 128, nbytes);
        if (SEP) {
          const uint8_t* vrow = p.v8 + rh * DV + piece * 16;
#pragma unroll
          for (int c = 0; c < S::kNv; ++c) cp_async16(dst + S::kVOff + c * kChunkBytes, vrow + c * 128, nbytes);
        }
      }
      if (S::kTail) {
        // the tail's four pieces: lanes with piece 0..3 take the even steps' keys, the others the odd ones'
#pragma unroll
        for (int kg = 0; kg < kGatherSteps; kg += 2) {
          const bool second = piece >= 4;
          const int key = (second ? kg + 1 : kg) * kGatherKeys + key0, r = second ? cur[kg + 1] : cur[kg];
          const int64_t rh = static_cast<int64_t>(r >= 0 ? r : 0) * p.Hc + kvh;
          if (dsa::check(r < (p.g.n_blocks << p.g.lb), p.status))
            cp_async16(buf + S::kTailOff + sw64_offset(key, piece & 3), p.k8 + rh * DQK + S::kFull * 128 + (piece & 3) * 16,
                       r >= 0 ? 16u : 0u);
        }
      }
      cp_async_arrive(&kv_full[stage]);
    }
    cp_async_wait_all();  // nothing of this thread is in flight when it leaves
  } else if (warp >= kMmaWarp) {
    // ------------------------------------------------------------ MMA issue
    // Two warps, one per product, each converged with one elected issuer.
    const bool leader = elect_sync();
    const uint32_t base = dsa::smem_u32(smem);
    if (warp == kMmaWarp) {
      constexpr uint32_t idesc1 = dsa::idesc_e4m3(kKeys, kCols);
      const uint64_t q_desc = dsa::smem_desc(base + S::kQ, 16, 1024, dsa::kSwizzle128B);
      const uint64_t kv_desc = dsa::smem_desc(base + S::kKv, 16, 1024, dsa::kSwizzle128B);
      const uint64_t qt_desc = dsa::smem_desc(base + S::kQTail, 16, 512, dsa::kSwizzle64B);
      const uint64_t kt_desc = dsa::smem_desc(base + S::kKv + S::kTailOff, 16, 512, dsa::kSwizzle64B);
      const bool go = dsa::mbar_wait_warp(q_full, 0, wt);
      for (int i = i0, ctr = 0; i < i1 && go; ++i, ++ctr) {
        const int b = ctr & 1, stage = ctr % ST;
        const bool got = dsa::mbar_wait(&s_empty[b], ((ctr >> 1) & 1) ^ 1, wt) &&
                         dsa::mbar_wait(&kv_full[stage], (ctr / ST) & 1, wt);
        // the gathered codes, before the tensor core reads them (MMA2's come
        // with the softmax warps' arrival, behind a fence of theirs)
        dsa::fence_proxy_async_smem();
        __syncwarp();
        dsa::tc_fence_after();
        const uint64_t a0 = kv_desc + stage * (S::kBuf >> 4);
        const uint32_t d = tmem_base + b * kCols;
#pragma unroll
        for (int c = 0; c < S::kFull; ++c) {
          const uint64_t ac = a0 + c * (kChunkBytes >> 4), bc = q_desc + c * (kQChunkBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            dsa::umma_f8_if(leader && got, d, ac + kk * 2, bc + kk * 2, idesc1, (c | kk) != 0);
        }
        if (S::kTail) {
          const uint64_t at = kt_desc + stage * (S::kBuf >> 4);
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) dsa::umma_f8_if(leader && got, d, at + kk * 2, qt_desc + kk * 2, idesc1, 1u);
        }
        if (leader && got) dsa::umma_commit(&s_full[b]);
        if (!__all_sync(0xffffffffu, got)) break;
      }
      if (leader) dsa::umma_drain(&drain[0], p.status);
      __syncwarp();
    } else {
      constexpr uint32_t idesc_hi = dsa::idesc_e4m3(128, kCols) | (1u << 15) | (1u << 16);  // both MN-major
      constexpr uint32_t idesc_lo = idesc_hi | (1u << 10);                                  // the weights' term in E5M2
      const uint64_t v_desc = dsa::smem_desc(base + S::kKv + S::kVOff, kChunkBytes, 1024, dsa::kSwizzle128B);
      // P^T rows are 32 bytes (hi and lo of 16 heads): 32-byte swizzle, groups of 8 keys 256 bytes apart
      const uint64_t p_desc = dsa::smem_desc(base + S::kP, kPBytes, 256, kSwizzle32B);
      for (int i = i0, ctr = 0; i < i1; ++i, ++ctr) {
        const int b = ctr & 1, stage = ctr % ST;
        const bool got = dsa::mbar_wait(&p_full[b], (ctr >> 1) & 1, wt);
        __syncwarp();
        dsa::tc_fence_after();
        const uint64_t a0 = v_desc + stage * (S::kBuf >> 4), b0 = p_desc + (S::kPBufs == 2 ? b : 0) * (2 * kPBytes >> 4);
#pragma unroll
        for (int mb = 0; mb < S::kNv; ++mb) {
#pragma unroll
          for (int kk = 0; kk < kKeys / 32; ++kk) {
            const uint32_t d = tmem_base + kOCol + mb * kCols;
            const uint64_t av = a0 + mb * (kChunkBytes >> 4) + kk * (32 * 128 >> 4), bp = b0 + kk * (32 * kCols >> 4);
            dsa::umma_f8_if(leader && got, d, av, bp, idesc_hi, (i > i0 || kk > 0) ? 1u : 0u);
            dsa::umma_f8_if(leader && got, d, av, bp + (kPBytes >> 4), idesc_lo, 1u);
          }
        }
        if (leader && got) {
          dsa::umma_commit(&p_empty[b]);
          dsa::umma_commit(&kv_empty[stage]);
        }
        if (!__all_sync(0xffffffffu, got)) break;
      }
      if (leader) dsa::umma_drain(&drain[1], p.status);
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ query, softmax, epilogue
    const int quarter = warp & 3;  // TMEM lane quarter
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    // the query: eight threads per head, pieces of 8 values sub, sub + 8, ...
    // Head 4 c + 2 j + e is row 8 j + 2 c + e of the operand (its second term
    // 16 rows on), which gives each softmax thread four consecutive heads.
    {
      const int row = ((hq >> 1) & 1) * 8 + (hq >> 2) * 2 + (hq & 1);
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < kPieces; ++k) m = dsa::amax_bf16x8(qv[k], m);
      m = dsa::max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = dsa::max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 2));
      m = dsa::larger_half(dsa::max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 4)));
      // a head with infinity or NaN: its scores are NaN
      const bool finite = m < 0x7F80u;
      const float s = finite ? dsa::kv8_scale_of(__uint_as_float(m << 16)) : 1.f;
      const float inv = dsa::pow2_inverse(s);
      if (sub == 0) qexp[hq] = finite ? static_cast<uint8_t>(__float_as_uint(s) >> 23) : 255;
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const uint32_t wd[4] = {qv[k].x, qv[k].y, qv[k].z, qv[k].w};
        uint16_t hi[4], lo[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) split_query(wd[n], inv, hi[n], lo[n]);
        const int unit16 = (sub + 8 * k) >> 1;  // 16 codes of the row
        const uint32_t half = (sub & 1) * 8;
        const bool tail = unit16 >= S::kFull * 8;
        const uint32_t at = tail ? S::kQTail + sw64_offset(row, unit16 - S::kFull * 8)
                                 : S::kQ + (unit16 >> 3) * kQChunkBytes + dsa::sw128_offset(row, (unit16 & 7) * 16);
        // (16 rows on leaves either swizzle's phase as it is)
        *reinterpret_cast<uint2*>(smem + at + half) = pack4(hi);
        *reinterpret_cast<uint2*>(smem + at + half + kHG * (tail ? 64 : 128)) = pack4(lo);
      }
      dsa::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) dsa::mbar_arrive(q_full);
    }
    // S^T registers 4j + e (key kA) and 4j + 2 + e (key kB) hold head hb + 2j + e
    const int kA = quarter * 16 + (lane >> 2), kB = kA + 8;
    const int hb = 4 * (lane & 3);
    // Per head hb + h: the references (of the sum and of the weighted values), this thread's keys' sum and maximum.
    float m[4], rr[4], l_part[4], qs[4], top[4];
    bool unset = true;  // no valid slot so far
#pragma unroll
    for (int h = 0; h < 4; ++h) l_part[h] = 0.f, m[h] = 0.f, rr[h] = 0.f, qs[h] = 0.f, top[h] = -INFINITY;
    bool ok = true;
    // A wait of this thread gave up: the four warps leave together, at a
    // point that reduces the flag (see the bf16 kernel).
    bool failed = false;
    int ctr = 0;
    for (int i = i0; i < i1; ++i, ++ctr) {
      const int b = ctr & 1, stage = ctr % ST;
      const uint32_t par = (ctr >> 1) & 1;
      // the slots' scales come with the gathered tile
      if (!failed) failed = !dsa::mbar_wait(&kv_full[stage], (ctr / ST) & 1, wt);
      const float* meta = reinterpret_cast<const float*>(smem + S::kMeta + stage * S::kMetaStep);
      const float skA = meta[kA], skB = meta[kB];
      const bool vA = skA > 0.f, vB = skB > 0.f;
      // the values' scales as 2^ek * fk, fk in (1/2, 1]
      const float svA = SEP ? meta[kKeys + kA] : skA, svB = SEP ? meta[kKeys + kB] : skB;
      const float2 eA = scale_parts(vA ? svA : 1.f), eB = scale_parts(vB ? svB : 1.f);
      if (!failed) failed = !dsa::mbar_wait(&s_full[b], par, wt);
      __syncwarp();
      dsa::tc_fence_after();
      float x[8];
      {
        uint32_t v[16];
        dsa::tmem_ld16x256b_x4(tmem_base + lane_off + b * kCols, v);
        dsa::tmem_wait_ld();
#pragma unroll
        for (int r = 0; r < 8; ++r) x[r] = fmaf(__uint_as_float(v[8 + r]), 0.0625f, __uint_as_float(v[r]));
      }
      if (i == i0) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {  // (255: a head with infinity or NaN)
          const uint8_t e = qexp[hb + h];
          qs[h] = __uint_as_float(static_cast<uint32_t>(e) << 23) * (e == 255 ? NAN : p.scale_log2);
        }
      }
      dsa::tc_fence_before();
      __syncwarp();
      if (lane == 0) dsa::mbar_arrive(&s_empty[b]);
      // scores in powers of two against the references; -inf where there is no slot
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int h = 2 * j + e;
          x[4 * j + e] = vA ? fmaf(x[4 * j + e], qs[h] * skA, -m[h]) : -INFINITY;
          x[4 * j + 2 + e] = vB ? fmaf(x[4 * j + 2 + e], qs[h] * skB, -m[h]) : -INFINITY;
        }
      }
      // y: with the value's scale, against the other reference
      float y[8], v[4], u[4], most = -INFINITY, most_y = -INFINITY;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int a = 4 * (h >> 1) + (h & 1);
        const float d = m[h] - rr[h];
        y[a] = x[a] + (d + eA.x), y[a + 2] = x[a + 2] + (d + eB.x);
        v[h] = fmaxf(x[a], x[a + 2]), u[h] = fmaxf(y[a], y[a + 2]);
        most = fmaxf(most, v[h]), most_y = fmaxf(most_y, u[h]);
        top[h] = fmaxf(top[h], v[h] + m[h]);
      }
      const bool ex = unset || most > kMoveM || most_y > kMoveR;
      bool need_rescale = false;
      if (i == i0 || group_any(ex || failed)) {
        // move the references: the tile's maxima per head over its 64 keys
        const auto larger = [](float a, float c) { return fmaxf(a, c); };
        wmax[quarter * kHG + hb + own_head(lane)] = fold4(v, lane, larger);
        ymax[quarter * kHG + hb + own_head(lane)] = fold4(u, lane, larger);
        const bool some = __any_sync(0xffffffffu, vA || vB);
        if (lane == 0) svm[quarter] = some ? 1.f : 0.f;
        if (group_any(failed)) {  // the group leaves together
          ok = false;
          break;
        }
        float4 t4 = *reinterpret_cast<const float4*>(wmax + hb), y4 = *reinterpret_cast<const float4*>(ymax + hb);
#pragma unroll
        for (int q4 = 1; q4 < 4; ++q4) {
          const float4 o = *reinterpret_cast<const float4*>(wmax + q4 * kHG + hb);
          t4.x = fmaxf(t4.x, o.x), t4.y = fmaxf(t4.y, o.y), t4.z = fmaxf(t4.z, o.z), t4.w = fmaxf(t4.w, o.w);
          const float4 r = *reinterpret_cast<const float4*>(ymax + q4 * kHG + hb);
          y4.x = fmaxf(y4.x, r.x), y4.y = fmaxf(y4.y, r.y), y4.z = fmaxf(y4.z, r.z), y4.w = fmaxf(y4.w, r.w);
        }
        const float tm[4] = {t4.x, t4.y, t4.z, t4.w}, ty[4] = {y4.x, y4.y, y4.z, y4.w};
        bool moved = false;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          // by how much each moves: to the next whole number above the tile's maximum, if
          // that passes it by enough or is the first
          const int a = 4 * (h >> 1) + (h & 1);
          const float up = (unset ? tm[h] > -INFINITY : tm[h] > kMoveM) ? ceilf(tm[h]) : 0.f;
          const float upr = (unset ? ty[h] > -INFINITY : ty[h] > kMoveR) ? ceilf(ty[h]) : 0.f;
          moved |= upr != 0.f;
          l_part[h] *= unset ? 1.f : ex2(-up);
          m[h] += up, rr[h] += upr;
          x[a] -= up, x[a + 2] -= up;
          y[a] -= upr, y[a + 2] -= upr;
          if (lane < 4) alpha[hb + h] = unset ? 1.f : ex2(-upr);  // (the four warps write the same ones)
        }
        unset = unset && !(fmaxf(fmaxf(svm[0], svm[1]), fmaxf(svm[2], svm[3])) > 0.f);
        need_rescale = __any_sync(0xffffffffu, moved) && i > i0;
      }
      // P^T rows kA and kB, both terms: the thread's four heads are bytes hb .. hb + 3 of each place
      if (!failed) failed = !dsa::mbar_wait(&p_empty[b], par ^ 1, wt);  // MMA2 of two tiles ago has read the buffer
      if (S::kPBufs == 1 && i > i0 && !failed) failed = !dsa::mbar_wait(&p_empty[b ^ 1], ((ctr - 1) >> 1) & 1, wt);
      {
        uint8_t* pb = smem + S::kP + (S::kPBufs == 2 ? b : 0) * 2 * kPBytes;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int key = k ? kB : kA;
          const float fk = (k ? eB.y : eA.y) * kWeight;
          uint16_t hi[2], lo[2];
          uint32_t low = 0;  // the bytes of the weights that go to the second place
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int a = 4 * j + 2 * k;
            l_part[2 * j] += ex2(x[a]);
            l_part[2 * j + 1] += ex2(x[a + 1]);
            float w0 = ex2(y[a]) * fk, w1 = ex2(y[a + 1]) * fk;
            if (w0 < kLow) w0 *= kLowScale, low |= 0xFFu << (16 * j);
            if (w1 < kLow) w1 *= kLowScale, low |= 0xFFu << (16 * j + 8);
            split_weights(w0, w1, hi[j], lo[j]);
          }
          const uint32_t h4 = hi[0] | (static_cast<uint32_t>(hi[1]) << 16), l4 = lo[0] | (static_cast<uint32_t>(lo[1]) << 16);
          const uint32_t at0 = sw32_offset(key, 0) + hb, at1 = sw32_offset(key, 1) + hb;
          *reinterpret_cast<uint32_t*>(pb + at0) = h4 & ~low;
          *reinterpret_cast<uint32_t*>(pb + at1) = h4 & low;
          *reinterpret_cast<uint32_t*>(pb + kPBytes + at0) = l4 & ~low;
          *reinterpret_cast<uint32_t*>(pb + kPBytes + at1) = l4 & low;
        }
      }
      if (need_rescale) {
        // MMA2 of the previous tile must have landed before O^T is scaled
        if (!failed) failed = !dsa::mbar_wait(&p_empty[b ^ 1], ((ctr - 1) >> 1) & 1, wt);
        __syncwarp();  // (and alpha, written by four lanes of this warp)
        dsa::tc_fence_after();
#pragma unroll 1
        for (int mb = 0; mb < S::kNv; ++mb) {
          const uint32_t ta = tmem_base + lane_off + kOCol + mb * kCols;
          uint32_t o[32];
          __syncwarp();
          dsa::tmem_ld32(ta, o);
          dsa::tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha[c & 15]);
          dsa::tmem_st32(ta, o);
        }
        dsa::tmem_wait_st();
      }
      dsa::fence_proxy_async_smem();
      dsa::tc_fence_before();
      __syncwarp();
      if (lane == 0) dsa::mbar_arrive(&p_full[b]);
    }

    // ---------------------------------------------------------- epilogue
    if (ok) {
      // The sums' norm, while the last tile's MMA2 runs.
      const float sink = p.sink && st < hv ? __ldg(p.sink + h0 + st) : -INFINITY;
      red[quarter * kHG + hb + own_head(lane)] = fold4(l_part, lane, [](float a, float c) { return a + c; });
      redm[quarter * kHG + hb + own_head(lane)] = fold4(top, lane, [](float a, float c) { return fmaxf(a, c); });
      if (quarter == 0 && lane < 4) {
#pragma unroll
        for (int h = 0; h < 4; ++h) fac[hb + h] = m[h], facr[hb + h] = rr[h];
      }
      group_sync();
      if (st < kHG) {
        const float l = red[st] + red[kHG + st] + red[2 * kHG + st] + red[3 * kHG + st];
        const float mc = fac[st];
        const float mx = fmaxf(fmaxf(redm[st], redm[kHG + st]), fmaxf(redm[2 * kHG + st], redm[3 * kHG + st]));
        stats[st] = make_float4(mc, l, mx, sink);
        // (in two steps: 2^(R - m) alone may pass fp32's range)
        const float half = floorf(0.5f * (facr[st] - mc)), e0 = exp2f(half) * (1.f / kWeight), e1 = exp2f(facr[st] - mc - half);
        fac[st] = l != 0.f ? e0 / l * e1 : 0.f;  // of a split's mean value, which stays in range where the sum might not
        if (p.splits == 1) {
          const Norm n = norm_of(mc, l, sink);
          fac[st] = n.f * e0 * e1;
          if (st < hv) {
            p.lse[orow + st] = n.lse;
            if (p.lse_kv) p.lse_kv[orow + st] = n.lse_kv;
            if (p.max_logits) p.max_logits[orow + st] = l != 0.f ? mx * kLn2 : -INFINITY;
          }
        }
      }
      // O^T is complete with the last tile's MMA2 (each phase of p_empty has
      // been waited for in turn, so the parity names that tile)
      if (!failed) failed = !dsa::mbar_wait(&p_empty[(ctr - 1) & 1], ((ctr - 1) >> 1) & 1, wt);
      group_sync();
      dsa::tc_fence_after();
      const uint32_t tm_o = tmem_base + lane_off + kOCol;
      if (p.splits > 1) {
        float f[kHG];
#pragma unroll
        for (int h = 0; h < kHG; h += 4) {
          const float4 f4 = *reinterpret_cast<const float4*>(fac + h);
          f[h] = f4.x, f[h + 1] = f4.y, f[h + 2] = f4.z, f[h + 3] = f4.w;
        }
#pragma unroll 1
        for (int mb = 0; mb < S::kNv; ++mb) {
          uint32_t v[32];
          __syncwarp();
          dsa::tmem_ld32(tm_o + mb * kCols, v);
          dsa::tmem_wait_ld();
          const int d = mb * 128 + quarter * 32 + lane;
#pragma unroll
          for (int h = 0; h < kHG; ++h) part[h * DV + d] = fmaf(__uint_as_float(v[kHG + h]), 1.f / kLowScale, __uint_as_float(v[h])) * f[h];
        }
      } else {
        // transposed by the store of 8 x 8 matrices, 16 heads x 32 dims at a
        // time: 64 consecutive bytes a head (two bytes a lane straight to
        // memory: 7K cycles of an item's 16K)
        float f[4];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float2 f2 = *reinterpret_cast<const float2*>(fac + 8 * c + 2 * (lane & 3));
          f[2 * c] = f2.x, f[2 * c + 1] = f2.y;
        }
        const int mrow = 8 * (lane >> 4) + (lane & 7), munit = (lane >> 3) & 1;  // matrices: 8 heads x 8 dims
        __nv_bfloat16* o0 = p.out + (orow + (lane >> 2)) * DV + quarter * 32 + (lane & 3) * 8;
#pragma unroll
        for (int mb = 0; mb < S::kNv; ++mb) {
          uint8_t* rows = row16 + (mb * 4 + quarter) * 1024;
          uint32_t v[2][16];
          __syncwarp();
          dsa::tmem_ld16x256b_x4(tm_o + mb * kCols, v[0]);
          dsa::tmem_ld16x256b_x4(tm_o + mb * kCols + (16u << 16), v[1]);
          dsa::tmem_wait_ld();
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint32_t r[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {  // 8 heads n / 2, 8 dims n % 2
              const float* fn = f + 2 * (n >> 1);
              const float a = fmaf(__uint_as_float(v[g][8 + 2 * n]), 1.f / kLowScale, __uint_as_float(v[g][2 * n]));
              const float b = fmaf(__uint_as_float(v[g][8 + 2 * n + 1]), 1.f / kLowScale, __uint_as_float(v[g][2 * n + 1]));
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(a * fn[0], b * fn[1]);
              r[n] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            dsa::stmatrix_x4_trans(dsa::smem_u32(rows) + sw64_offset(mrow, 2 * g + munit), r[0], r[1], r[2], r[3]);
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int h = k * 8 + (lane >> 2);
            if (h < hv)
              __stcs(reinterpret_cast<uint4*>(o0 + mb * 128 + k * 8 * DV),
                     *reinterpret_cast<const uint4*>(rows + sw64_offset(h, lane & 3)));
          }
        }
      }
      dsa::tc_fence_before();
    }
  }

  __syncwarp();
  if (p.splits > 1) {
    // Joins the splits: with M the largest reference and a_s = 2^(m_s - M) l_s, out = sum_s a_s O_s / z of their
    // mean values O_s.
    cluster_arrive();
    cluster_wait();
    const int dims = DV / p.splits, quads = dims / 4, d0 = split * dims;
    const uint32_t stats_at = dsa::smem_u32(stats), part_at = dsa::smem_u32(part);
    for (int x = threadIdx.x; x < (dead ? 0 : hv * quads); x += kThreads) {
      const int h = x / quads, d = d0 + (x - h * quads) * 4;
      float4 sm[kMaxCluster], o[kMaxCluster];
#pragma unroll
      for (int s = 0; s < kMaxCluster; ++s) {
        if (s < p.splits) {
          sm[s] = ld_cluster(of_rank(stats_at + h * 16, s));
          o[s] = ld_cluster(of_rank(part_at + (h * DV + d) * 4, s));
        } else {
          sm[s] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
        }
      }
      float M = -INFINITY, mx = -INFINITY, l = 0.f;
#pragma unroll
      for (int s = 0; s < kMaxCluster; ++s)
        if (sm[s].y != 0.f) M = fmaxf(M, sm[s].x), mx = fmaxf(mx, sm[s].z);
      float share[kMaxCluster];
#pragma unroll
      for (int s = 0; s < kMaxCluster; ++s) {
        share[s] = sm[s].y != 0.f ? sm[s].y * exp2f(sm[s].x - M) : 0.f;
        l += share[s];
      }
      const Norm n = norm_of(M, l, sm[0].w);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int s = 0; s < kMaxCluster; ++s) {
        if (sm[s].y == 0.f) continue;  // a split without a valid slot: it may have left no values
        const float a = share[s] * n.f;  // at most 1: a mean of means stays in range
        acc.x = fmaf(a, o[s].x, acc.x), acc.y = fmaf(a, o[s].y, acc.y), acc.z = fmaf(a, o[s].z, acc.z), acc.w = fmaf(a, o[s].w, acc.w);
      }
      *reinterpret_cast<uint2*>(p.out + (orow + h) * DV + d) = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
      if (d == 0) {
        p.lse[orow + h] = n.lse;
        if (p.lse_kv) p.lse_kv[orow + h] = n.lse_kv;
        if (p.max_logits) p.max_logits[orow + h] = l != 0.f ? mx * kLn2 : -INFINITY;
      }
    }
  }
  if (p.splits > 1) cluster_arrive();  // this thread has read the others' sums
  __syncwarp();
  __syncthreads();
  if (warp == kMmaWarp && aligned) {
    dsa::tc_fence_after();
    dsa::tmem_dealloc(tmem_base, S::kTmem);
  }
  if (p.splits > 1) cluster_wait();
}

int64_t units_of(int T, int H, int Hc) { return static_cast<int64_t>(T) * Hc * ((H / Hc + kHG - 1) / kHG); }

// Splits of each row's slots, one to eight CTAs of a cluster: the number that
// makes the last CTA earliest, in fifths of a tile: kItemTiles for what an item
// does once, 7 instead of 5 a tile where SMs have two CTAs, 13 and one per
// split for the join.  Measured (2048 slots, latent rows of 576; microseconds
// with 1, 2, 4, 8 splits): one row of 64 heads 43, 28, 17.2, 12.5; 64 rows of 32
// heads 46.7, 39.2, 44.8, 61.7; 1024 rows of 16 heads of 512 220, 243.
constexpr int kItemTiles = 5;

int plan_splits(int64_t units, int K) {
  const int nt = (K + kKeys - 1) / kKeys;
  int best = 1;
  int64_t cost = INT64_MAX;
  for (int s = 1; s <= kMaxCluster && s <= nt; s *= 2) {
    const int64_t waves = (units * s + 2 * kPlanSms - 1) / (2 * kPlanSms);
    const int64_t c = waves * ((nt + s - 1) / s + kItemTiles) * (units * s > kPlanSms ? 7 : 5) + (s > 1 ? 13 + s : 0);
    if (c < cost) cost = c, best = s;
  }
  return best;
}

template <int DQK, int DV, bool SEP>
int launch_form(const Params& p, cudaStream_t stream) {
  using S = Shape<DQK, DV, SEP>;
  auto kernel = attn_kv8_narrow_kernel<DQK, DV, SEP>;
  static std::atomic<uint64_t> ready{0};  // devices where the kernel's shared memory is allowed
  int dev = 0;
  cudaGetDevice(&dev);  // below 64: check_device
  if (!(ready.load(std::memory_order_acquire) >> dev & 1)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kTotal) != cudaSuccess)
      return dsa::launch_error("attn_kv8_narrow_kernel smem attribute");
    ready.fetch_or(uint64_t{1} << dev, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.n_items) * p.splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kTotal;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = p.splits;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = p.splits > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) return dsa::launch_error("attn_kv8_narrow_kernel");
  return DSA_OK;
}

}  // namespace

namespace dsa {
namespace kv8_attn {

// KV heads of at most 32 query heads, and calls of little work: up to 10 tiles
// of 16 heads an SM.  Measured (microseconds, this kernel against the other):
// 1024 rows of 16 heads of 512, 512 slots 68 / 125; 32 heads: 32 rows, 2048 slots 24.2 / 27.7,
// 1000 rows, 1000 slots 218 / 261; 48 heads, 500 slots: 40 rows 15.4 / 17.6, 1000 rows 180 / 149;
// 64 heads, 256 slots: 64 rows 13.3 / 14.7, 128 rows 23.5 / 17.6; 8 rows of 128 heads, 2048 slots
// 23.0 / 18.7.  Rows of more than 2^20 slots go to the other kernel, whose weights have no
// smallest step: here what lies below it could add up to 2^-9 of the largest.
bool narrow_takes(int T, int H, int Hc, int K) {
  const int groups = (H / Hc + kHG - 1) / kHG;
  return K <= (1 << 20) && (groups <= 2 || units_of(T, H, Hc) * ((K + kKeys - 1) / kKeys) <= 10 * kPlanSms);
}

int launch_narrow(Params p, int T, int Dqk, cudaStream_t stream) {
  p.G = (p.H / p.Hc + kHG - 1) / kHG;
  const int64_t units = units_of(T, p.H, p.Hc);
  p.splits = plan_splits(units, p.K);
  p.n_items = static_cast<int>(units);
  if (Dqk == 256) return launch_form<256, 256, true>(p, stream);
  return Dqk == 576 ? launch_form<576, 512, false>(p, stream) : launch_form<512, 512, false>(p, stream);
}

}  // namespace kv8_attn
}  // namespace dsa
