// attention_kv8.cu -- sparse attention over the 8-bit block cache.
//
// For row t, head h (of KV head h / (H / Hc)) and valid slot j, with row r_j
// in block b_j: s_j = scale * k_scale[b_j] * (q . e4m3(kv8[r_j])),
// out = sum_j exp(s_j) v_scale[b_j] e4m3(v8[r_j]) / (sum_j exp(s_j) + exp(sink)).
#include <climits>

#include "kv8.cuh"

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kKeys = 32;    // keys per tile, one per lane
constexpr int kHeads = 8;    // heads per CTA, one per warp
constexpr int kThreads = kHeads * 32;
constexpr int kPad = 16;     // bytes added to a staged row (bank conflicts)

struct Params {
  const __nv_bfloat16* q;
  const uint8_t* k8;
  const float* k_scale;
  const uint8_t* v8;  // == k8 when V is the first Dv dims of the row
  const float* v_scale;
  const int32_t* idx;
  const int32_t* topk_length;
  const float* sink;
  dsa::Kv8Geom g;
  __nv_bfloat16* out;
  float* lse;
  float* lse_kv;
  float* max_logits;
  int H, Hc, Dqk, Dv, K;
  bool separate;
  float scale_log2;
};

__global__ void __launch_bounds__(kThreads) attn_kv8_kernel(const Params p) {
  extern __shared__ uint8_t smem[];
  __shared__ int rows[kKeys];
  __shared__ float ks[kKeys], vs[kKeys];
  const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = p.H / p.Hc, per = (group + kHeads - 1) / kHeads;
  const int kvh = blockIdx.y / per, hg = (blockIdx.y - kvh * per) * kHeads + warp;
  const bool real = hg < group;
  const int h = kvh * group + min(hg, group - 1);
  if (p.g.table && t >= __ldg(p.g.cu + p.g.n_seqs)) return;
  const int b = p.g.table ? dsa::kv8_seq(p.g.cu, p.g.n_seqs, t) : 0;
  const int kst = p.Dqk + kPad, vst = p.separate ? p.Dv + kPad : 0;
  uint8_t* kt = smem;
  uint8_t* vt = p.separate ? smem + kKeys * kst : smem;
  const int vld = p.separate ? vst : kst;
  float* qs = reinterpret_cast<float*>(smem + kKeys * (kst + vst)) + warp * p.Dqk;
  const int64_t orow = static_cast<int64_t>(t) * p.H + h;
  for (int c = lane; c < p.Dqk; c += 32) qs[c] = __bfloat162float(p.q[orow * p.Dqk + c]);
  int len = p.K;
  if (p.topk_length) len = min(max(__ldg(p.topk_length + t), 0), p.K);
  float m = -INFINITY, l = 0.f, acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  for (int j0 = 0; j0 < len; j0 += kKeys) {
    __syncthreads();
    if (threadIdx.x < kKeys) {
      const int j = j0 + threadIdx.x;
      const int id = j < len ? __ldg(p.idx + static_cast<int64_t>(t) * p.K + j) : -1;
      const int r = id >= 0 ? dsa::kv8_row(p.g, b, id) : -1;
      rows[threadIdx.x] = r;
      const int64_t sb = static_cast<int64_t>(r >> p.g.lb) * p.Hc + kvh;
      ks[threadIdx.x] = r >= 0 ? __ldg(p.k_scale + sb) : 0.f;
      vs[threadIdx.x] = r >= 0 ? __ldg(p.v_scale + sb) : 0.f;
    }
    __syncthreads();
    const int pk = p.Dqk >> 4, pv = p.separate ? p.Dv >> 4 : 0;
    for (int i = threadIdx.x; i < kKeys * (pk + pv); i += kThreads) {
      const int j = i / (pk + pv), c = i - j * (pk + pv);
      uint4 v = make_uint4(0, 0, 0, 0);
      if (rows[j] >= 0) {
        const int64_t rh = static_cast<int64_t>(rows[j]) * p.Hc + kvh;
        v = c < pk ? __ldg(reinterpret_cast<const uint4*>(p.k8 + rh * p.Dqk) + c)
                   : __ldg(reinterpret_cast<const uint4*>(p.v8 + rh * p.Dv) + (c - pk));
      }
      *reinterpret_cast<uint4*>(c < pk ? kt + j * kst + c * 16 : vt + j * vst + (c - pk) * 16) = v;
    }
    __syncthreads();
    float dot = 0.f;
    for (int c = 0; c < p.Dqk; c += 4) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(kt + lane * kst + c);
      const float2 a = dsa::f2_of_e4m3x2(static_cast<uint16_t>(w)), e = dsa::f2_of_e4m3x2(static_cast<uint16_t>(w >> 16));
      const float4 qv = *reinterpret_cast<const float4*>(qs + c);
      dot = fmaf(qv.x, a.x, fmaf(qv.y, a.y, fmaf(qv.z, e.x, fmaf(qv.w, e.y, dot))));
    }
    const bool valid = rows[lane] >= 0;
    const float x = valid ? dot * (ks[lane] * p.scale_log2) : -INFINITY;
    float mx = x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(m, mx);
    const float mr = mn == -INFINITY ? 0.f : mn;
    const float alpha = exp2f(m - mr);
    const float e = valid ? exp2f(x - mr) : 0.f;
    float sum = e;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * alpha + sum;
    m = mn;
    const float w = valid ? e * vs[lane] : 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] *= alpha;
    for (int j = 0; j < kKeys; ++j) {
      if (rows[j] < 0) continue;
      const float wj = __shfl_sync(0xffffffffu, w, j);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = i * 128 + lane * 4;
        if (d < p.Dv) {
          const uint32_t u = *reinterpret_cast<const uint32_t*>(vt + j * vld + d);
          const float2 a = dsa::f2_of_e4m3x2(static_cast<uint16_t>(u)), c = dsa::f2_of_e4m3x2(static_cast<uint16_t>(u >> 16));
          acc[4 * i] = fmaf(wj, a.x, acc[4 * i]);
          acc[4 * i + 1] = fmaf(wj, a.y, acc[4 * i + 1]);
          acc[4 * i + 2] = fmaf(wj, c.x, acc[4 * i + 2]);
          acc[4 * i + 3] = fmaf(wj, c.y, acc[4 * i + 3]);
        }
      }
    }
  }
  if (!real) return;
  const float sink = p.sink ? __ldg(p.sink + h) : -INFINITY, sk = sink * kLog2e;
  const bool any = m > -INFINITY || l != 0.f;  // l != 0 also when it is NaN
  const float M = fmaxf(m, sk), Mr = M == -INFINITY ? 0.f : M;
  const float a = any ? exp2f(m - Mr) : 0.f;
  const float z = l * a + exp2f(sk - Mr);
  const float f = any ? a / z : 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int d = (i >> 2) * 128 + lane * 4 + (i & 3);
    if (d < p.Dv) p.out[orow * p.Dv + d] = __float2bfloat16_rn(acc[i] * f);
  }
  if (lane == 0) {
    p.lse[orow] = any ? (Mr + log2f(z)) * kLn2 : sink;
    if (p.lse_kv) p.lse_kv[orow] = any ? (m + log2f(l)) * kLn2 : INFINITY;
    if (p.max_logits) p.max_logits[orow] = m * kLn2;
  }
}

}  // namespace

extern "C" size_t dsa_sparse_attn_fwd_kv8_workspace_size(int T, int H, int Hc, int Dqk, int Dv, int K) {
  (void)T, (void)H, (void)Hc, (void)Dqk, (void)Dv, (void)K;
  return 0;
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
  if (T < 0 || H < 1 || Hc < 1 || Hc > DSA_KV8_MAX_HEADS || H % Hc != 0 || H / Hc > 128 || K < 0)
    return dsa::set_error(DSA_ERR_VALUE, "%s: need T >= 0, K >= 0, 1 <= Hc <= %d, H a multiple of Hc, H / Hc <= 128", fn,
                          DSA_KV8_MAX_HEADS);
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
  int rc = dsa::check_device(nullptr);
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
  p.Dqk = Dqk;
  p.Dv = Dv;
  p.K = K;
  p.separate = separate;
  p.scale_log2 = scale * kLog2e;
  const int per = (H / Hc + kHeads - 1) / kHeads;
  const int smem = kKeys * (Dqk + kPad + (separate ? Dv + kPad : 0)) + kHeads * Dqk * 4;
  attn_kv8_kernel<<<dim3(T, Hc * per), kThreads, smem, stream>>>(p);
  return dsa::launch_error("attn_kv8_kernel");
}
