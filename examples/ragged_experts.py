"""Experts with a body of their own, trained in bf16 and served in 4 bits.

The layer's kernels run SwiGLU experts; this example builds squared-ReLU ones
from the grouped products:

  train   grouped_linear on the ragged rows that the offsets call lays out
          (moe_grouped_gemm, its data gradient, moe_grouped_wgrad)
  serve   the trained weights quantised once (moe_quantize_fp4), then per batch:
          token rows quantised into expert order, moe_grouped_gemm_fp4, the
          activation, quantised again, moe_grouped_gemm_fp4 with the routing
          weights, moe_combine

  python examples/ragged_experts.py [--tokens T] [--steps N] [--format mx|nv]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import routing_permute_grouped_gb300 as moe  # noqa: E402


def layout(cfg, topk_idx, topk_w):
    """Group offsets, the permutation and the routing weights of unpadded rows."""
    A, dev = cfg.T * cfg.k, topk_idx.device
    i32 = dict(dtype=torch.int32, device=dev)
    counts, offsets = torch.empty(cfg.E, **i32), torch.empty(cfg.E + 1, **i32)
    perm, src = torch.empty(A, **i32), torch.empty(A, **i32)
    gate = torch.empty(A, dtype=torch.float32, device=dev)
    ws = torch.zeros(moe.moe_offsets_workspace_size(cfg), dtype=torch.uint8, device=dev)
    moe.moe_build_offsets_unpadded(cfg, topk_idx, topk_w, counts, offsets, perm, src, gate, ws)
    return offsets, perm, src, gate


def quantize(w, fmt):
    """[E, N, K] -> codes, scales, tensor scales [E] (None for MX)."""
    E, N, K = w.shape
    codes = torch.empty((E, N, K // 2), dtype=torch.uint8, device=w.device)
    scales = torch.empty((E, N, moe.moe_fp4_scale_stride(fmt, K)), dtype=torch.uint8, device=w.device)
    g = (w.abs().amax((1, 2)).float() / 2688).clamp(min=1e-30) if fmt == moe.FP4_NV else None
    for e in range(E):
        moe.moe_quantize_fp4(fmt, w[e], codes[e], scales[e], tensor_scale=None if g is None else g[e:e + 1])
    return codes, scales, g


def serve(cfg, fmt, x, w1q, w2q, offsets, perm, src, gate):
    A, d, de, dev = cfg.T * cfg.k, cfg.d, cfg.d_e, x.device

    def rows(K):
        return (torch.empty((A, K // 2), dtype=torch.uint8, device=dev),
                torch.empty((A, moe.moe_fp4_scale_stride(fmt, K)), dtype=torch.uint8, device=dev))

    xq, xs = rows(d)
    moe.moe_quantize_fp4(fmt, x, xq, xs, src=src, src_div=cfg.k)
    u = torch.empty((A, de), dtype=torch.bfloat16, device=dev)
    moe.moe_grouped_gemm_fp4(fmt, xq, xs, w1q[0], w1q[1], offsets, u, w_scale=w1q[2])
    h = torch.relu(u).square_()
    hq, hs = rows(de)
    moe.moe_quantize_fp4(fmt, h, hq, hs)
    y = torch.empty((A, d), dtype=torch.bfloat16, device=dev)
    moe.moe_grouped_gemm_fp4(fmt, hq, hs, w2q[0], w2q[1], offsets, y, w_scale=w2q[2], row_scale=gate)
    out = torch.empty((cfg.T, d), dtype=torch.bfloat16, device=dev)
    moe.moe_combine(cfg, y, perm, None, out)
    return out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--d", type=int, default=1024)
    ap.add_argument("--d-e", type=int, default=512)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--k", type=int, default=2)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--format", choices=sorted(moe.FP4_FORMATS), default="mx")
    a = ap.parse_args(argv)
    cfg = moe.config_of(T=a.tokens, d=a.d, d_e=a.d_e, E=a.experts, k=a.k)
    gen = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * std

    # a batch, its routing and what the experts shall learn
    x = normal(cfg.T, cfg.d).bfloat16()
    top = normal(cfg.T, cfg.E).topk(cfg.k)
    topk_idx, topk_w = top.indices.to(torch.int32).contiguous(), top.values.softmax(-1).contiguous()
    offsets, perm, src, gate = layout(cfg, topk_idx, topk_w)
    token = (src // cfg.k).long()
    goal = normal(cfg.E, cfg.d, cfg.d, std=cfg.d ** -0.5).bfloat16()
    target = moe.grouped_linear(x[token], goal, offsets)

    w1 = normal(cfg.E, cfg.d_e, cfg.d, std=cfg.d ** -0.5).bfloat16().requires_grad_()
    w2 = normal(cfg.E, cfg.d, cfg.d_e, std=cfg.d_e ** -0.5).bfloat16().requires_grad_()
    opt = torch.optim.Adam([w1, w2], lr=3e-3)
    losses = []
    for _ in range(a.steps):
        u = moe.grouped_linear(x[token], w1, offsets)
        y = moe.grouped_linear(torch.relu(u).square(), w2, offsets)
        loss = (y.float() - target.float()).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} over {a.steps} steps")

    # the trained layer in bf16, and in 4 bits
    with torch.no_grad():
        u = moe.grouped_linear(x[token], w1, offsets)
        y = torch.empty((cfg.T * cfg.k, cfg.d), dtype=torch.bfloat16, device="cuda")
        moe.moe_grouped_gemm(torch.relu(u).square(), w2.detach(), offsets, y, row_scale=gate)
        ref = torch.empty_like(x)
        moe.moe_combine(cfg, y, perm, None, ref)
        fmt = moe.FP4_FORMATS[a.format]
        out = serve(cfg, fmt, x, quantize(w1.detach(), fmt), quantize(w2.detach(), fmt), offsets, perm, src, gate)
    rel = ((out.float() - ref.float()).norm() / ref.float().norm()).item()
    print(f"4-bit ({a.format}) against bf16: relative error {rel:.3f}")
    return losses, rel


if __name__ == "__main__":
    main()
