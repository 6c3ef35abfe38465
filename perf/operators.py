"""Cases for timing the grouped-product operators and checking their outputs.

Four operators, each on token rows sorted by expert (group e owns rows
offsets[e] .. offsets[e + 1]), with whatever sizes the routing gave:

  product    y[r] = row_scale[r] * x[r] W[e]^T with W [E, N, K], or the data
             gradient dx[r] = dy[r] W[e] of the same W; bf16 or fp16
  wgrad      dW[e] = sum over e's rows of a[r]^T b[r]; bf16 or fp16
  quantize   rows to 4-bit codes with block scales (OCP MX: 32 elements and a
             power of two; NV: 16 elements, an e4m3 scale and one fp32 scale
             for the tensor), gathered into expert order; returned as values
  product4   product on 4-bit rows and 4-bit weights with their block scales

With ``own`` false, ``run`` computes them with elementary torch operations in
fp32; with ``own`` true, through the library's entry points.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the tiny layer's gate/up product: launch latency
        dict(name="product tiny", op="product", dtype="bf16", R=512, E=8, K=512, N=512, grad=False, gated=False, skew=0.0),
        # a decode step's down projection over 256 experts, two rows each: weight bytes
        dict(name="product decode", op="product", dtype="bf16", R=512, E=256, K=2048, N=7168, grad=False, gated=True, skew=0.0),
        # the default layer's gate/up product: tensor throughput
        dict(name="product default", op="product", dtype="bf16", R=32768, E=8, K=7168, N=4096, grad=False, gated=False, skew=0.2),
        # data gradient of a 64-expert layer whose hottest expert has about four times the mean load
        dict(name="dgrad imbalance", op="product", dtype="bf16", R=98304, E=64, K=2048, N=4096, grad=True, gated=False, skew=0.33),
        # weight gradient of the same layer
        dict(name="wgrad imbalance", op="wgrad", dtype="bf16", R=98304, E=64, M=2048, N=4096, skew=0.33),
        # a small fp16 training step with odd sizes: ragged in every direction
        dict(name="wgrad odd fp16", op="wgrad", dtype="fp16", R=3001, E=32, M=1000, N=712, skew=0.3),
        # a prefill batch's activations quantised into expert order, each token to 4 experts
        dict(name="quantize default mx", op="quantize", fmt="mx", T=8192, k=4, K=7168),
        # a decode step's activations: launch latency
        dict(name="quantize decode nv", op="quantize", fmt="nv", T=64, k=8, K=7168),
        # a short prompt on small 4-bit experts, ragged sizes
        dict(name="product4 small nv", op="product4", fmt="nv", R=300, E=8, K=512, N=520, gated=False, skew=0.3),
        # a decode step's gate/up product over 256 4-bit experts: weight bytes
        dict(name="product4 decode nv", op="product4", fmt="nv", R=512, E=256, K=7168, N=4096, gated=False, skew=0.0),
        # the 64-expert layer's down projection with routing weights: short sums
        dict(name="product4 down mx", op="product4", fmt="mx", R=98304, E=64, K=1024, N=4096, gated=True, skew=0.33),
        # the default layer's gate/up product on 4-bit experts: tensor throughput
        dict(name="product4 default mx", op="product4", fmt="mx", R=32768, E=8, K=7168, N=4096, gated=False, skew=0.2),
    ]


def draw(rng):
    def size(lo, hi, unit):
        return max(1, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / unit)) * unit

    op = rng.choice(("product", "wgrad", "quantize", "product4"))
    if op == "quantize":
        k = rng.randint(1, 8)
        return dict(op=op, fmt=rng.choice(("mx", "nv")), T=size(1, 32768 // k, 1), k=k, K=size(64, 7168, 32))
    unit = 32 if op == "product4" else 8
    a, b = size(64, 7168, unit), size(64, 7168, 8)
    E = min(size(1, 256, 1), max(1, 3_700_000_000 // (a * b)))
    R = min(size(1, 98304, 1), max(1, int(0.9e12 / (a * b))))
    case = dict(op=op, R=R, E=E, skew=round(rng.uniform(0.0, 0.33), 3))
    if op == "wgrad":
        return dict(case, dtype=rng.choice(("bf16", "fp16")), M=b, N=a)
    case = dict(case, K=a, N=b, gated=rng.random() < 0.5)
    if op == "product4":
        return dict(case, fmt=rng.choice(("mx", "nv")))
    return dict(case, dtype=rng.choice(("bf16", "fp16")), grad=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs --
def _sizes(case, seed):
    """Rows per expert: a Zipf profile over a random order of the experts; one in ten has none."""
    rng = np.random.default_rng(seed)
    E = case["E"]
    p = np.arange(1, E + 1, dtype=np.float64) ** -case["skew"]
    if E > 4:
        p[rng.permutation(E)[: E // 10]] = 0.0
    p = rng.permutation(p)
    return rng.multinomial(case["R"], p / p.sum())


def _normal(shape, gen, std, dtype):
    """N(0, std), drawn in slices of the leading dimension."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    step = max(1, (1 << 28) // max(1, out[0].numel())) if len(shape) > 1 else shape[0]
    for i in range(0, shape[0], step):
        part = out[i:i + step]
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda").mul_(std))
    return out


def _activations(rows, K, gen, dtype):
    """N(0, 1) rows with a few channels of larger magnitude."""
    x = _normal((rows, K), gen, 1.0, torch.float32)
    wide = torch.rand((K,), generator=gen, device="cuda") < 0.01
    return x.mul_(torch.where(wide, 8.0, 1.0)).to(dtype)


def _quantized(w, fmt, tscale):
    """Codes [.., K / 2], scales [.., stride] of w [.., K] and what they stand for."""
    v, s = _levels(w, fmt, tscale)
    mag = v.abs()
    code = (mag * 2).to(torch.uint8)                      # 0, 1, 2, 3, 4, 6, 8, 12
    code = torch.where(mag > 3, 6 + (mag > 5).to(torch.uint8), torch.where(mag > 2, 5, code)).to(torch.uint8)
    code |= (v < 0).to(torch.uint8) << 3
    codes = code[..., 0::2] | (code[..., 1::2] << 4)
    scales = torch.zeros((*s.shape[:-1], (s.shape[-1] + 15) // 16 * 16), dtype=torch.uint8, device=w.device)
    scales[..., : s.shape[-1]] = s
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, st = case["op"], dict(case=case)
    if op == "quantize":
        T, k, K = case["T"], case["k"], case["K"]
        st["x"] = _activations(T, K, gen, torch.bfloat16)
        st["src"] = torch.randperm(T * k, generator=gen, device="cuda").to(torch.int32)
        # a calibrated scale with one percent of headroom over these rows
        st["tscale"] = (st["x"].abs().amax().float() * (1.01 / (6 * 448))).reshape(1) if case["fmt"] == "nv" else None
        return st
    R, E = case["R"], case["E"]
    sizes = _sizes(case, seed)
    st["longest"] = int(sizes.max())
    st["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).cuda()
    st["gates"] = torch.rand((R,), generator=gen, device="cuda") * 0.95 + 0.05 if case.get("gated") else None
    if op == "wgrad":
        st["a"] = _normal((R, case["M"]), gen, 1.0, DT[case["dtype"]])
        st["b"] = _normal((R, case["N"]), gen, 1.0, DT[case["dtype"]])
        return st
    K, N = case["K"], case["N"]
    if op == "product":
        st["x"] = _activations(R, K, gen, DT[case["dtype"]])
        # a data gradient multiplies by the forward's own weights, [E, K, N] as it sees them
        st["w"] = _normal((E, K, N) if case["grad"] else (E, N, K), gen, K ** -0.5, DT[case["dtype"]])
        return st
    fmt = case["fmt"]
    x = _activations(R, K, gen, torch.bfloat16).float()
    st["xt"] = (x.abs().amax() / (6 * 448)).reshape(1) if fmt == "nv" else None
    st["xq"], st["xs"] = _quantized(x, fmt, st["xt"])
    st["wt"] = torch.empty((E,), device="cuda") if fmt == "nv" else None
    stride = (K // (32 if fmt == "mx" else 16) + 15) // 16 * 16
    st["wq"] = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    st["ws"] = torch.empty((E, N, stride), dtype=torch.uint8, device="cuda")
    for e in range(E):
        w = (torch.randn((N, K), generator=gen, device="cuda") * K ** -0.5).bfloat16().float()
        if fmt == "nv":
            st["wt"][e] = w.abs().amax() / (6 * 448)
        st["wq"][e], st["ws"][e] = _quantized(w, fmt, st["wt"][e:e + 1] if fmt == "nv" else None)
    return st


# -------------------------------------------------------------- plain form --
def _levels(x, fmt, tscale):
    """x [.., K] fp32 -> e2m1 values [.., K] and scale codes [.., K / block]."""
    block = 32 if fmt == "mx" else 16
    v = x.unflatten(-1, (-1, block))
    amax = v.abs().amax(-1)
    if fmt == "mx":  # the smallest power of two that keeps the block within 6; 1 for a zero block
        m, e = torch.frexp(amax)
        e = torch.where(amax > 0, e - torch.where(m <= 0.75, 3, 2), 0).clamp(min=-127)
        s = (e + 127).to(torch.uint8)
        scale = torch.ldexp(torch.ones_like(amax), e)
    else:
        q = (amax / (tscale * 6)).clamp(max=448).to(torch.float8_e4m3fn)
        s = q.view(torch.uint8)
        scale = q.float() * tscale
    t = torch.where(scale[..., None] > 0, v / scale[..., None], 0.0)
    a = t.abs()
    # nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6; ties to the even code
    r = 0.5 * ((a > 0.25).float() + (a >= 0.75).float() + (a > 1.25).float() + (a >= 1.75).float())
    r = r + (a > 2.5).float() + (a >= 3.5).float() + 2 * (a > 5).float()
    return torch.copysign(r, t).flatten(-2), s


def _values(codes, scales, fmt, K):
    """fp32 values of codes [.., K / 2] and scales [.., stride], without the tensor scale."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    byte = torch.arange(256, device=codes.device)
    pairs = torch.stack([lut[byte & 15], lut[byte >> 4]], -1)
    v = pairs[codes.int()].flatten(-2)
    block = 32 if fmt == "mx" else 16
    s = scales[..., : K // block]
    s = (s.int() << 23).view(torch.float32) if fmt == "mx" else s.contiguous().view(torch.float8_e4m3fn).float()
    v.unflatten(-1, (-1, block)).mul_(s[..., None])
    return v


def _padded(x, st):
    """x [R, C] fp32 as [E, longest, C], zeros past a group's end, and where its rows are."""
    lo, hi = st["offsets"][:-1, None].long(), st["offsets"][1:, None].long()
    rows = lo + torch.arange(st["longest"], device=x.device)
    inside = rows < hi
    rows = rows.clamp(max=x.shape[0] - 1)
    return x[rows].mul_(inside[..., None]), rows[inside], inside


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "quantize":
        x = st["x"].float()
        v, s = _levels(x, case["fmt"], st["tscale"])
        block = 32 if case["fmt"] == "mx" else 16
        scale = torch.ldexp(torch.ones_like(s, dtype=torch.float32), s.int() - 127) if case["fmt"] == "mx" \
            else s.view(torch.float8_e4m3fn).float()
        v = (v.unflatten(-1, (-1, block)) * scale[..., None]).flatten(-2)
        v = v * st["tscale"] if st["tscale"] is not None else v
        return v.bfloat16()[(st["src"] // case["k"]).long()]
    if op == "wgrad":
        a, _, _ = _padded(st["a"].float(), st)
        b, _, _ = _padded(st["b"].float(), st)
        return torch.bmm(a.transpose(1, 2), b).to(st["a"].dtype)
    if op == "product":
        x, dtype = st["x"].float(), st["x"].dtype
        w = st["w"].float()
        w = w if case["grad"] else w.transpose(1, 2)
    else:
        x, dtype = _values(st["xq"], st["xs"], case["fmt"], case["K"]), torch.bfloat16
        w = _values(st["wq"], st["ws"], case["fmt"], case["K"]).transpose(1, 2)
    xp, rows, inside = _padded(x, st)
    y = torch.bmm(xp, w)
    if op == "product4" and st["xt"] is not None:
        y = y * (st["xt"] * st["wt"])[:, None, None]
    out = torch.empty((case["R"], case["N"]), device=x.device)
    out[rows] = y[inside]
    if st["gates"] is not None:
        out.mul_(st["gates"][:, None])
    return out.to(dtype)


# ------------------------------------------------------- the library's calls --
def _own(st):
    import routing_permute_grouped_gb300 as moe

    case = st["case"]
    op = case["op"]
    if op == "quantize":
        fmt, K = moe.FP4_FORMATS[case["fmt"]], case["K"]
        rows, dev = case["T"] * case["k"], st["x"].device
        codes = torch.empty((rows, K // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((rows, moe.moe_fp4_scale_stride(fmt, K)), dtype=torch.uint8, device=dev)
        moe.moe_quantize_fp4(fmt, st["x"], codes, scales, tensor_scale=st["tscale"], src=st["src"], src_div=case["k"])
        out = torch.empty((rows, K), dtype=torch.bfloat16, device=dev)
        moe.moe_dequantize_fp4(fmt, codes, scales, out, tensor_scale=st["tscale"])
        return out
    if op == "wgrad":
        out = torch.empty((case["E"], case["M"], case["N"]), dtype=st["a"].dtype, device=st["a"].device)
        moe.moe_grouped_wgrad(st["a"], st["b"], st["offsets"], out)
        return out
    if op == "product":
        out = torch.empty((case["R"], case["N"]), dtype=st["x"].dtype, device=st["x"].device)
        moe.moe_grouped_gemm(st["x"], st["w"], st["offsets"], out, row_scale=st["gates"], w_transposed=case["grad"])
        return out
    out = torch.empty((case["R"], case["N"]), dtype=torch.bfloat16, device=st["xq"].device)
    moe.moe_grouped_gemm_fp4(moe.FP4_FORMATS[case["fmt"]], st["xq"], st["xs"], st["wq"], st["ws"], st["offsets"], out,
                             x_scale=st["xt"], w_scale=st["wt"], row_scale=st["gates"])
    return out


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op = case["op"]
    if op == "quantize":
        T, K = case["T"], case["K"]
        return dict(bytes=T * K * 2 + T * case["k"] * (4 + K * 2), flops=2 * T * K)
    R, E, N = case["R"], case["E"], case["N"]
    if op == "wgrad":
        return dict(bytes=2 * R * (case["M"] + N) + 2 * E * case["M"] * N, flops=2 * R * case["M"] * N)
    K = case["K"]
    used = min(E, R)  # experts that can have rows
    el = 2 if op == "product" else 0.5 + 1 / (32 if case["fmt"] == "mx" else 16)
    return dict(bytes=el * K * (R + used * N) + 2 * R * N + (4 * R if case["gated"] else 0), flops=2 * R * K * N)


# ------------------------------------------------------ the definition in fp64 --
def _nearest(v, grid):
    """The index of the value of `grid` nearest to v >= 0, ties to the even index."""
    g = torch.tensor(grid, dtype=torch.float64, device=v.device)
    mid = (g[1:] + g[:-1]) / 2
    i = torch.searchsorted(mid, v.contiguous())
    tie = mid[i.clamp(max=len(mid) - 1)] == v
    return torch.where(tie & (i < len(mid)) & (i % 2 == 1), i + 1, i)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = st["x"].double()
        block = 32 if case["fmt"] == "mx" else 16
        v = x.reshape(x.shape[0], -1, block)
        top = v.abs().amax(-1, keepdim=True)
        if case["fmt"] == "mx":
            scale = torch.exp2(torch.ceil(torch.log2(torch.where(top > 0, top, 6.0) / 6)))
            scale = torch.where(top > 6 * scale, 2 * scale, torch.where(top <= 3 * scale, scale / 2, scale))
            scale = torch.where(top > 0, scale, 1.0)
        else:
            g = st["tscale"].double()
            e4m3 = [(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127]
            scale = torch.tensor(e4m3, dtype=torch.float64, device=x.device)[_nearest(top / (6 * g), e4m3)] * g
        level = torch.tensor(E2M1, dtype=torch.float64, device=x.device)[_nearest(torch.where(scale > 0, v.abs() / scale, 0.0), E2M1)]
        return (torch.copysign(level, v) * scale).reshape(x.shape)[(st["src"] // case["k"]).long()]
    bounds = st["offsets"].tolist()
    dev = st["offsets"].device
    if op == "wgrad":
        out = torch.zeros((case["E"], case["M"], case["N"]), dtype=torch.float64, device=dev)
        for e in range(case["E"]):
            lo, hi = bounds[e], bounds[e + 1]
            if hi > lo:
                out[e] = st["a"][lo:hi].double().T @ st["b"][lo:hi].double()
        return out
    out = torch.zeros((case["R"], case["N"]), dtype=torch.float64, device=dev)

    def widen(codes, scales):
        nibble = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
        mag = torch.tensor(E2M1, dtype=torch.float64, device=dev)[(nibble & 7).int()]
        v = torch.where(nibble > 7, -mag, mag)
        s = scales[:, : case["K"] // (32 if case["fmt"] == "mx" else 16)]
        if case["fmt"] == "mx":
            s = torch.exp2(s.double() - 127)
        else:
            e, m = (s >> 3).double(), (s & 7).double()
            s = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m / 8 * 2.0 ** -6)
        return v * s.repeat_interleave(case["K"] // s.shape[1], 1)

    for e in range(case["E"]):
        lo, hi = bounds[e], bounds[e + 1]
        if hi == lo:
            continue
        if op == "product":
            w = st["w"][e].double()
            out[lo:hi] = st["x"][lo:hi].double() @ (w if case["grad"] else w.T)
        else:
            y = widen(st["xq"][lo:hi], st["xs"][lo:hi]) @ widen(st["wq"][e], st["ws"][e]).T
            out[lo:hi] = y * (st["xt"].double() * st["wt"][e].double()) if st["xt"] is not None else y
    if st["gates"] is not None:
        out *= st["gates"][:, None].double()
    return out
