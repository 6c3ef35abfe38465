"""GPU tests of the 4-bit layer, of grouped_linear and of the example that runs
the grouped products together.  Every stage of the layer is checked against
fp64 arithmetic on the previous stage's own output, so each bound is that
stage's (see test_gpu_ragged.py)."""
import numpy as np
import pytest
import torch

import routing_permute_grouped_gb300 as moe
from tests.test_gpu_ragged import BLOCK, E2M1, E4M3, _check, _gen, _quant_ref, _rand

pytestmark = pytest.mark.gpu


def _values(codes, scales, fmt, g=None):
    """fp64 values of 4-bit rows."""
    K = codes.shape[-1] * 2
    lut = torch.from_numpy(np.concatenate([E2M1, -E2M1])).cuda()
    v = lut[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    s = scales[..., :K // BLOCK[fmt]]
    s = torch.exp2(s.double() - 127) if fmt == moe.FP4_MX else torch.from_numpy(E4M3).cuda()[s.int()]
    v = (v.unflatten(-1, (s.shape[-1], -1)) * s[..., None]).flatten(-2)
    return v if g is None else v * g.double().reshape(-1, *[1] * (v.dim() - 1))


def _layer(name, T, E, k, d_shared, seed=3, prerouted=False, d=512, d_e=256):
    cfg = moe.config_of(T=T, d=d, d_e=d_e, E=E, k=k, d_shared=d_shared)
    w = dict(W1=_rand((E, d, d_e), seed, std=d ** -0.5), W3=_rand((E, d, d_e), seed + 1, std=d ** -0.5),
             W2=_rand((E, d_e, d), seed + 2, std=d_e ** -0.5))
    if d_shared:
        w.update(Ws1=_rand((d, d_shared), seed + 3, std=d ** -0.5), Ws3=_rand((d, d_shared), seed + 4, std=d ** -0.5),
                 Ws2=_rand((d_shared, d), seed + 5, std=d_shared ** -0.5))
    if not prerouted:
        w["Wg"] = _rand((d, E), seed + 6, std=d ** -0.5)
    scales = (None, None)
    if name == "nv":
        scales = tuple(torch.tensor([s], device="cuda") for s in (0.002, 0.003))
    return cfg, moe.MoeLayer(cfg, fp4=name, fp4_scales=scales, **w), _rand((T, d), seed + 7)


def _mlp_stages(layer, fmt, rows, d, width, off, x, gate, bufs, packed):
    """Checks quantise, gate/up, SwiGLU + quantise and down of one expert MLP;
    the fp64 values of its result are those of the buffer y itself."""
    buf = layer.buffer
    W13q, s13, g13, W2q, s2, g2 = packed
    E = W13q.shape[0]
    gx, gh = layer.fp4_scales
    xq, xs, gu, hq, hs, y = bufs
    u8, bf = torch.uint8, torch.bfloat16
    stride = lambda K: moe.moe_fp4_scale_stride(fmt, K)  # noqa: E731
    xq, xs = buf(xq, u8, (rows, d // 2)), buf(xs, u8, (rows, stride(d)))
    gu = buf(gu, bf, (rows, 2 * width))
    hq, hs, y = buf(hq, u8, (rows, width // 2)), buf(hs, u8, (rows, stride(width))), buf(y, bf, (rows, d))
    one = torch.ones(1, device="cuda")
    # rows: exact
    code, byte, _ = _quant_ref(x.double().cpu().numpy(), fmt, 1.0 if gx is None else gx.item())
    assert np.array_equal(xs.cpu().numpy()[:, :byte.shape[1]], byte)
    xv = _values(xq, xs, fmt, one if gx is None else gx)
    # gate/up of the stored rows, down of the stored h
    w13, w2 = _values(W13q, s13, fmt, g13), _values(W2q, s2, fmt, g2)
    hv = _values(hq, hs, fmt, one if gh is None else gh)
    for a, w, got, n, gates in ((xv, w13, gu, d, None), (hv, w2, y, width, gate)):
        ref = torch.zeros(got.shape, dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(ref)
        for e in range(E):
            lo, hi = off[e], off[e + 1]
            ref[lo:hi] = a[lo:hi] @ w[e].T
            mag[lo:hi] = a[lo:hi].abs() @ w[e].abs().T
        if gates is not None:
            ref, mag = ref * gates[:, None].double(), mag * gates[:, None].double()
        _check(got, ref, mag, n, bf)
    # SwiGLU: silu(gate) * up rounded to bf16 may land one bf16 value off, and
    # its code one step of the grid (amax / 3 at most) off where that crosses
    v = gu.double().reshape(rows, width // 128, 2, 128)
    h = (v[:, :, 0] * torch.sigmoid(v[:, :, 0]) * v[:, :, 1]).reshape(rows, width).bfloat16()
    _, _, ref = _quant_ref(h.double().cpu().numpy(), fmt, 1.0 if gh is None else gh.item())
    ref = torch.from_numpy(ref).cuda()
    top = h.double().abs().reshape(rows, -1, BLOCK[fmt]).amax(-1).repeat_interleave(BLOCK[fmt], 1)
    off_by = (hv - ref).abs()
    assert (off_by <= 1.1 * top / 3 + 1e-30).all()
    assert (off_by > 1e-6 * top).double().mean() < 2e-3
    return y


@pytest.mark.parametrize("name", ["mx", "nv"])
@pytest.mark.parametrize("T,E,k,d_shared,prerouted", [(200, 8, 2, 128, False), (1, 4, 1, 0, False), (64, 64, 8, 256, False),
                                                      (333, 5, 3, 0, True)])
def test_layer_stages(name, T, E, k, d_shared, prerouted):
    fmt = moe.FP4_FORMATS[name]
    cfg, layer, x = _layer(name, T, E, k, d_shared, prerouted=prerouted)
    kw = {}
    if prerouted:
        kw = dict(topk_idx=torch.randint(0, E, (T, k), generator=_gen(1), device="cuda").to(torch.int32),
                  topk_w=torch.rand((T, k), generator=_gen(2), device="cuda"))
    out = layer(x, **kw)
    torch.cuda.synchronize()
    assert layer.device_status() == 0
    A = T * k
    off = layer.buffer("group_offsets", torch.int32, (E + 1,)).tolist()
    assert off[0] == 0 and off[-1] == A
    src = layer.buffer("row_src", torch.int32, (A,)).long()
    gate = layer.buffer("row_gate", torch.float32, (A,))
    if prerouted:
        assert torch.equal(gate, kw["topk_w"].flatten()[src])
    y = _mlp_stages(layer, fmt, A, cfg.d, cfg.d_e, off, x[src // k], gate, ("xq", "xs", "gu", "hq", "hs", "y"),
                    layer.packed)
    perm = layer.buffer("perm_row", torch.int32, (T, k)).long()
    terms = y.double()[perm]
    if d_shared:
        ys = _mlp_stages(layer, fmt, T, cfg.d, d_shared, [0, T], x, None, ("sxq", "sxs", "sgu", "shq", "shs", "ys"),
                         layer.shared_packed)
        terms = torch.cat([terms, ys.double()[:, None]], 1)
    _check(out, terms.sum(1), terms.abs().sum(1), k + 1, torch.bfloat16)


def test_layer_on_another_stream_and_in_a_graph():
    cfg, layer, x = _layer("mx", 100, 8, 2, 128)
    first = layer(x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = torch.zeros_like(x)
    torch.cuda.synchronize()
    layer.forward(x, out, stream=s)
    s.synchronize()
    assert torch.equal(out, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        layer.forward(x, out)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)


def test_layer_skips_ids_out_of_range():
    cfg, layer, x = _layer("mx", 40, 4, 2, 0, prerouted=True)
    idx = torch.randint(0, 4, (40, 2), generator=_gen(1), device="cuda").to(torch.int32)
    w = torch.rand((40, 2), generator=_gen(2), device="cuda")
    bad = idx.clone()
    bad[3, 1] = 4
    bad[7, 0] = -1
    out = layer(x, topk_idx=bad, topk_w=w).clone()
    assert layer.device_status() == moe.DEVERR_EXPERT_RANGE
    ref = layer(x, topk_idx=idx, topk_w=w)
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[[3, 7]] = False
    assert torch.equal(out[keep], ref[keep])
    assert torch.isfinite(out.float()).all()


def test_empty_batch():
    cfg, layer, _ = _layer("nv", 0, 4, 2, 128)
    x = torch.empty((0, cfg.d), dtype=torch.bfloat16, device="cuda")
    assert layer(x).shape == (0, cfg.d)


def test_dense_group_without_offsets():
    x, w = _rand((70, 64), 1), _rand((1, 72, 64), 2)
    off = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
    y, z = (torch.empty((70, 72), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    moe.moe_grouped_gemm(x, w, off, y)
    moe.moe_grouped_gemm(x, w, None, z)
    assert torch.equal(y, z)
    a, b = (torch.empty((1, 72, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    moe.moe_grouped_wgrad(y, x, off, a)
    moe.moe_grouped_wgrad(y, x, None, b)
    assert torch.equal(a, b)


def test_grouped_linear_gradients():
    """Autograd through grouped_linear gives the formula's gradients, for rows
    outside every group zero, and from a transposed dy."""
    off = [2, 40, 40, 99]
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    x, w = _rand((104, 64), 1).requires_grad_(), _rand((3, 72, 64), 2, std=1 / 8).requires_grad_()
    y = moe.grouped_linear(x, w, offsets)
    assert (y[:2] == 0).all() and (y[99:] == 0).all()
    dy = _rand((72, 104), 3).t()
    y.backward(dy)
    d, xd, wd = dy.double(), x.detach().double(), w.detach().double()
    assert (x.grad[:2] == 0).all() and (x.grad[99:] == 0).all()
    for e in range(3):
        s = slice(off[e], off[e + 1])
        _check(x.grad[s], d[s] @ wd[e], d[s].abs() @ wd[e].abs(), 72, torch.bfloat16)
        _check(w.grad[e], d[s].T @ xd[s], d[s].abs().T @ xd[s].abs(), 59, torch.bfloat16)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_example_runs(fmt):
    from examples import ragged_experts

    losses, rel = ragged_experts.main(["--tokens", "300", "--d", "256", "--d-e", "128", "--experts", "6", "--steps", "12",
                                       "--format", fmt])
    assert losses[-1] < losses[0] and np.isfinite(losses).all()
    assert 0 < rel < 1
