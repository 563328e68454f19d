"""One small, self-contained invocation of one stage of the DSA forward path,
for profiling a single kernel launch (ncu ``-k <kernel> -s 1 -c 1``).

    python -m sparse_attention_gemm_gb300.profile_case CASE [--T N] [--k K]

Every case runs its call twice (the first launch warms up; profile the second)
on a single document of T tokens shaped like the long-context workload
(H = 64 heads, indexer Hi = 64, d = 128, latent 576/512, top-k k), with
seeded device-side draws: qi, ki ~ N(0, 1), head weights U(0, 1) / 8, q, kv
~ N(0, 1) * 0.1 in bf16, sink N(0, 1).  At the default T = 16384 every case
holds a few GB on the device and its inputs exceed the 129 MB L2.

Cases (kernel to select with -k in parentheses):
  indexer_dense   dsa_indexer_scores, scores [T, T] fp32       (indexer_kernel)
  indexer_fused   stage 1 of dsa_indexer_topk                   (indexer_kernel)
  indexer_mxfp8   dsa_indexer_scores_mxfp8 on E4M3 codes with E8M0 scales per 32
                  elements (drawn codes and scales), scores [T, T] fp32
                                                                (indexer_kernel)
  select          stage 2 of dsa_indexer_topk                   (fused_select_multi_kernel)
  topk            dsa_topk on the dense causal scores           (topk_stream_kernel)
  attention       dsa_sparse_attn_fwd on the fused top-k ids    (sparse_attn_kernel)
  gqa             dsa_sparse_attn_fwd, block-routed GQA, B = 8 x S = T / 8 packed
                  tokens, Hq = 12, D = 256, routes as the GQA workload draws them
                                                                (sparse_attn_kernel)
  backward        dsa_sparse_attn_bwd on the fused top-k ids, dout ~ N(0, 1) * 0.1
                  (bwd_prep_kernel, bwd_dq_kernel, bwd_dkv_kernel, bwd_reduce_*);
                  with --atomic the variant whose dkv goes through fp32 atomics
  kv8_write       dsa_kv8_write of T latent rows into pages of 64 tokens (kv8_write_kernel)
  kv8_read        dsa_kv8_read of them                          (kv8_read_kernel)
  attention_kv8   dsa_sparse_attn_fwd_kv8 over those pages, ids drawn evenly
                  from the causal rows                          (attn_cache_kernel)
  attention_kv8_narrow  the same with H = 16                    (attn_kv8_narrow_kernel)
  rms_norm        dsa_rms_norm_fwd of T rows of 4096, residual added (rms_fwd_kernel)
  rms_norm_bwd    dsa_rms_norm_bwd of them                      (rms_bwd_kernel, rms_dw_kernel)
  rotary          dsa_rotary of the last 64 of H heads of 576   (rotary_kernel)
  kv4_write       dsa_kv4_write of T latent rows into pages of 64 tokens (kv4_write_kernel)
  kv4_read        dsa_kv4_read of them                          (kv4_read_kernel)
  attention_kv4   dsa_sparse_attn_fwd_kv4 over a cache of T * k / 8 rows, ids drawn
                  evenly: too many rows to be widened once      (attn_cache_kernel)
  attention_kv4_widened  the same over T rows                   (kv4_widen_kernel, kv4_rows_kernel, sparse_attn_kernel)
  attention_kv4_narrow   the first with H = 16 heads, k at most 1024 (attn_kv4_narrow_kernel)
"""
from __future__ import annotations

import argparse
import math
import sys

import numpy as np
import torch

CASES = ("indexer_dense", "indexer_fused", "indexer_mxfp8", "select", "topk", "attention", "gqa", "backward",
         "kv8_write", "kv8_read", "attention_kv8", "attention_kv8_narrow", "rms_norm", "rms_norm_bwd", "rotary", "kv4_write",
         "kv4_read", "attention_kv4", "attention_kv4_widened", "attention_kv4_narrow")


def _bf16(shape, sigma, g, dev):
    return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * sigma).to(torch.bfloat16)


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("case", choices=CASES)
    ap.add_argument("--T", type=int, default=16384)
    ap.add_argument("--k", type=int, default=2048)
    ap.add_argument("--atomic", action="store_true", help="backward: dkv by fp32 atomics")
    args = ap.parse_args(argv)

    import os

    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    from sparse_attention_gemm_gb300 import build, ops

    build.build()
    dev = torch.device("cuda:0")
    T, K, H, Hi, d = args.T, args.k, 64, 64, 128
    g = torch.Generator(device=dev)
    g.manual_seed(1234)
    cu = torch.tensor([0, T], dtype=torch.int32, device=dev)
    stream = torch.cuda.current_stream(dev)

    def twice(fn):
        for _ in range(2):
            fn()
        torch.cuda.synchronize()

    if args.case == "gqa":
        from sparse_attention_gemm_gb300 import workloads as W

        B, S, Hq, D = 8, T // 8, 12, 256
        wl = W.gqa_routes()
        wl.B, wl.S, wl.T = B, S, B * S
        routes = torch.from_numpy(wl.routes()).to(dev)
        idx = ops.pack_routes(routes)
        q = _bf16((B * S, Hq, D), 0.1, g, dev)
        k = _bf16((B * S, D), 0.1, g, dev)
        v = _bf16((B * S, D), 0.1, g, dev)
        twice(lambda: ops.sparse_attn_fwd(q, k, idx, 1.0 / 16.0, v=v))
        print(f"gqa: B={B} S={S} Hq={Hq} D={D} width={idx.shape[1]}")
        return 0

    if args.case in ("kv8_write", "kv8_read", "attention_kv8", "attention_kv8_narrow"):
        pages = (T + 63) // 64
        table = torch.randperm(pages, generator=g, device=dev).to(torch.int32)[None]
        rows = _bf16((T, 1, 576), 1.0, g, dev)
        kv8 = torch.zeros((pages, 64, 1, 576), dtype=torch.uint8, device=dev)
        scale = torch.ones((pages, 1), device=dev)
        ops.kv8_write(rows, kv8, scale, cu, block_table=table)
        if args.case == "kv8_write":
            twice(lambda: ops.kv8_write(rows, kv8, scale, cu, block_table=table))
        elif args.case == "kv8_read":
            twice(lambda: ops.kv8_read(kv8, scale, cu, T, block_table=table, out=rows))
        else:
            q = _bf16((T, 64 if args.case == "attention_kv8" else 16, 576), 1.0, g, dev)
            u = torch.rand((T, K), generator=g, device=dev) * torch.arange(1, T + 1, device=dev)[:, None]
            idx = u.to(torch.int32).sort(1)[0].contiguous()
            twice(lambda: ops.sparse_attn_fwd_kv8(q, kv8, scale, idx, 1.0 / 24.0, cu_seqlens=cu, block_table=table))
        status = ops.device_status(clear=True)
        print(f"{args.case}: T={T} k={K} status={status:#x}")
        return 1 if status else 0

    if args.case in ("rms_norm", "rms_norm_bwd", "rotary"):
        if args.case == "rotary":
            q, k = _bf16((T, H, 576), 1.0, g, dev), _bf16((T, 1, 576), 1.0, g, dev)
            f, mul = ops.rotary_inv_freq(64, scaling="yarn", factor=40.0, device=dev)
            twice(lambda: ops.rotary(q[..., 512:], f, cu, x2=k[..., 512:], mul=mul, out=q[..., 512:], out2=k[..., 512:]))
        else:
            x, r, dy = (_bf16((T, 4096), 1.0, g, dev) for _ in range(3))
            weight = torch.ones(4096, device=dev)
            fwd = ops.rms_norm_fwd(x, weight, 1e-6, residual=r, want_rstd=True)
            if args.case == "rms_norm":
                twice(lambda: ops.rms_norm_fwd(x, weight, 1e-6, residual=r, want_rstd=True))
            else:
                twice(lambda: ops.rms_norm_bwd(dy, fwd["sum"], weight, fwd["rstd"], d_sum=r))
        torch.cuda.synchronize()
        print(f"{args.case}: T={T}")
        return 0

    if args.case in ("kv4_write", "kv4_read", "attention_kv4", "attention_kv4_widened", "attention_kv4_narrow"):
        narrow = args.case == "attention_kv4_narrow"
        K = min(K, 1024) if narrow else K
        n = T * K // 8 if args.case in ("attention_kv4", "attention_kv4_narrow") else T
        pages = (n + 63) // 64
        table = torch.randperm(pages, generator=g, device=dev).to(torch.int32)[None]
        kv4 = torch.randint(0, 256, (pages, 64, 1, 288), generator=g, device=dev, dtype=torch.int32).to(torch.uint8)
        scale = torch.full((pages, 64, 1, 18), 125, dtype=torch.uint8, device=dev)
        if args.case in ("kv4_write", "kv4_read"):
            rows = _bf16((T, 1, 576), 1.0, g, dev)
            if args.case == "kv4_write":
                twice(lambda: ops.kv4_write(rows, kv4, scale, cu, block_table=table))
            else:
                twice(lambda: ops.kv4_read(kv4, scale, cu, T, block_table=table, out=rows))
        else:
            q = _bf16((T, 16 if narrow else 64, 576), 1.0, g, dev)
            idx = torch.randint(0, n, (T, K), generator=g, device=dev, dtype=torch.int32).sort(1)[0].contiguous()
            twice(lambda: ops.sparse_attn_fwd_kv4(q, kv4, scale, idx, 1.0 / 24.0, cu_seqlens=cu, block_table=table))
        status = ops.device_status(clear=True)
        print(f"{args.case}: T={T} k={K} status={status:#x}")
        return 1 if status else 0

    if args.case == "indexer_mxfp8":
        # E4M3 codes of N(0,1) draws with scale bytes around 2^-2 (no NaN codes)
        q8 = torch.randn((T, Hi, d), generator=g, device=dev).to(torch.float8_e4m3fn).view(torch.uint8)
        k8 = torch.randn((T, d), generator=g, device=dev).to(torch.float8_e4m3fn).view(torch.uint8)
        qs = torch.randint(123, 128, (T, Hi, d // 32), generator=g, device=dev, dtype=torch.int32).to(torch.uint8)
        ks = torch.randint(123, 128, (T, d // 32), generator=g, device=dev, dtype=torch.int32).to(torch.uint8)
        w = torch.rand((T, Hi), generator=g, device=dev, dtype=torch.float32) / 8.0
        scores = torch.empty((T, T), dtype=torch.float32, device=dev)
        twice(lambda: ops.indexer_scores_mxfp8(q8, k8, qs, ks, w, cu, cu, None, 1, T, out=scores))
        print(f"{args.case}: T={T} status={ops.device_status(clear=True):#x}")
        return 0
    qi = _bf16((T, Hi, d), 1.0, g, dev)
    ki = _bf16((T, d), 1.0, g, dev)
    w = torch.rand((T, Hi), generator=g, device=dev, dtype=torch.float32) / 8.0
    if args.case in ("indexer_dense", "topk"):
        scores = torch.empty((T, T), dtype=torch.float32, device=dev)
        if args.case == "indexer_dense":
            twice(lambda: ops.indexer_scores(qi, ki, w, cu, T, out=scores))
        else:
            ops.indexer_scores(qi, ki, w, cu, T, out=scores)
            start, length = ops.thd_metadata(cu, T)
            twice(lambda: ops.topk(scores, length, K, row_start=start))
        print(f"{args.case}: T={T} k={K}")
        return 0
    ws = torch.empty(ops.indexer_topk_workspace_size(T, Hi, d, K, T), dtype=torch.uint8, device=dev)
    if args.case == "indexer_fused":
        twice(lambda: ops.indexer_candidates(qi, ki, w, cu, K, T, workspace=ws))
    elif args.case == "select":
        ops.indexer_candidates(qi, ki, w, cu, K, T, workspace=ws)
        twice(lambda: ops.select_candidates(cu, T, Hi, d, K, T, ws))
    else:  # attention, backward
        idx, tl = ops.indexer_topk(qi, ki, w, cu, K, T, workspace=ws)
        del ws, qi, ki, w
        q = _bf16((T, H, 576), 0.1, g, dev)
        kv = _bf16((T, 576), 0.1, g, dev)
        sink = torch.randn(H, generator=g, device=dev, dtype=torch.float32)
        scale = 1.0 / math.sqrt(576.0)
        if args.case == "attention":
            twice(lambda: ops.sparse_attn_fwd(q, kv, idx, scale, topk_length=tl, sink=sink))
        else:
            fwd = ops.sparse_attn_fwd(q, kv, idx, scale, topk_length=tl, sink=sink, want_lse_kv=True)
            dout = _bf16((T, H, 512), 0.1, g, dev)
            det = not args.atomic
            bws = torch.empty(ops.sparse_attn_bwd_workspace_size(T, T, H, K, det), dtype=torch.uint8, device=dev)
            twice(lambda: ops.sparse_attn_bwd(q, kv, fwd["out"], dout, fwd["lse_kv"], idx, scale, topk_length=tl,
                                              sink=sink, workspace=bws, deterministic=det))
    status = ops.device_status(clear=True)
    print(f"{args.case}: T={T} k={K} status={status:#x}")
    return 1 if status else 0


if __name__ == "__main__":
    sys.exit(main())
