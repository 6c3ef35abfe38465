"""Cases for timing the router's scores and the 4-bit weight-only products.

Four operators:

  route      logits [T, E] to the k experts of each token and their weights:
             softmax or sigmoid scores, a bias that only the choice sees, a
             limit to the best groups of experts, weights renormalised and
             scaled; for training also the experts' loads and two losses
  route_bwd  the gradient of the weights and of the losses in the logits
  quantize   rows to unsigned 4-bit codes with a 16-bit scale (and, if asked
             for, a zero point) per group of elements; returned as values
  product    y[r] = row_scale[r] * x[token of r] W[e]^T on such weights, rows
             sorted by expert; or silu(gate) * up of 2 N weight rows that hold
             gate and up interleaved per 128

The choice of experts is that of the exact keys (score + bias; without a bias
the logits' order), ties to the lower index: keys are formed in 64 bits here,
the rest in 32.  With ``own`` true, ``run`` goes through the library's entry
points.
"""
import math

import numpy as np
import torch

own = False

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
FLT_MAX = 3.4028234663852886e38


def listed():
    return [
        # a decode step of the 256-expert layer: launch latency
        dict(name="route decode", op="route", dtype="fp32", T=64, E=256, k=8, score="sigmoid", bias=True, groups=8,
             topk_groups=4, group_top=2, renorm=True, scale=2.5, losses=False),
        # a long prompt on the 64-expert layer, logits as a bf16 product left them
        dict(name="route prompt bf16", op="route", dtype="bf16", T=16384, E=64, k=6, score="softmax", bias=False, groups=0,
             topk_groups=0, group_top=1, renorm=False, scale=1.0, losses=False),
        # a training batch on 256 experts with loads and losses
        dict(name="route train", op="route", dtype="fp32", T=32768, E=256, k=8, score="sigmoid", bias=True, groups=8,
             topk_groups=4, group_top=2, renorm=True, scale=2.5, losses=True),
        # gradient of a small batch on the 8-expert layer: launch latency
        dict(name="route_bwd small", op="route_bwd", dtype="bf16", T=1000, E=8, k=2, score="softmax", renorm=True,
             scale=1.0, losses=False),
        # gradient of the training batch
        dict(name="route_bwd train", op="route_bwd", dtype="fp32", T=32768, E=256, k=8, score="sigmoid", renorm=True,
             scale=2.5, losses=True),
        # down projections of the 64-expert layer, quantised when a model is loaded
        dict(name="quantize experts", op="quantize", dtype="bf16", rows=64 * 4096, K=1024, group=128, zeros=True),
        # one small fp16 matrix whose last group is short
        dict(name="quantize odd fp16", op="quantize", dtype="fp16", rows=520, K=480, group=64, zeros=False),
        # one token through a small dense matrix: launch latency
        dict(name="product row fp16", op="product", dtype="fp16", T=1, k=1, E=1, K=4096, N=1024, group=32, zeros=False,
             swiglu=False, gated=False, skew=0.0),
        # one token's gate/up product over 8 of 256 experts: weight bytes, few rows to split
        dict(name="product one token", op="product", dtype="bf16", T=1, k=8, E=256, K=7168, N=2048, group=128, zeros=True,
             swiglu=True, gated=False, skew=0.0),
        # a decode step's down projection over 256 experts, two rows each: weight bytes
        dict(name="product decode", op="product", dtype="bf16", T=64, k=8, E=256, K=2048, N=7168, group=128, zeros=True,
             swiglu=False, gated=True, skew=0.0),
        # 64 sequences on 8 experts: 32 rows to an expert, weight bytes and products both count
        dict(name="product batch", op="product", dtype="bf16", T=64, k=4, E=8, K=7168, N=2048, group=128, zeros=False,
             swiglu=True, gated=False, skew=0.2),
        # a short prompt on the 64-expert layer with uneven loads, some experts idle
        dict(name="product imbalance", op="product", dtype="bf16", T=500, k=6, E=64, K=4096, N=1024, group=64, zeros=True,
             swiglu=True, gated=False, skew=0.33),
    ]


def draw(rng):
    def size(lo, hi, unit=1):
        return max(1, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / unit)) * unit

    op = rng.choice(("route", "route_bwd", "quantize", "product", "product"))
    if op in ("route", "route_bwd"):
        groups = rng.choice((0, 0, 2, 4, 8))
        if groups:
            E = groups * size(2, 256 // groups)
            tg = rng.randint(1, groups)
            k = rng.randint(1, min(8, tg * (E // groups)))
        else:
            E, tg = size(2, 256), 0
            k = rng.randint(1, min(8, E))
        case = dict(op=op, dtype=rng.choice(("fp32", "bf16", "fp16")), T=size(1, 32768), E=E, k=k,
                    score=rng.choice(("softmax", "sigmoid")), renorm=rng.random() < 0.6,
                    scale=rng.choice((1.0, 1.0, 2.5)), losses=rng.random() < 0.4)
        if op == "route":
            case.update(bias=rng.random() < 0.6, groups=groups, topk_groups=tg, group_top=rng.choice((1, 2)))
        return case
    if op == "quantize":
        K = size(32, 7168, 32)
        return dict(op=op, dtype=rng.choice(("bf16", "fp16")), rows=size(1, min(262144, 268435456 // K)), K=K,
                    group=rng.choice((32, 64, 128)), zeros=rng.random() < 0.5)
    swiglu = rng.random() < 0.4
    K, N = size(64, 7168, 32), size(128, 4096, 128) if swiglu else size(64, 7168, 8)
    E = min(size(1, 256), max(1, 3_700_000_000 // (K * N * (2 if swiglu else 1))))
    k = rng.randint(1, min(8, E))
    most = min(4096, 64 * E, int(7.4e9 / (K * N * (2 if swiglu else 1))) + 1)  # rows
    return dict(op=op, dtype=rng.choice(("bf16", "fp16")), T=size(1, max(1, most // k)), k=k, E=E, K=K, N=N,
                group=rng.choice((32, 64, 128)), zeros=rng.random() < 0.5, swiglu=swiglu,
                gated=rng.random() < 0.5, skew=round(rng.uniform(0.0, 0.33), 3))


# ------------------------------------------------------------------ inputs --
def _popularity(E, skew, gen):
    """Log-odds of the experts: a Zipf profile in a random order."""
    z = -skew * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    return z[torch.randperm(E, generator=gen, device="cuda")]


def _logits(case, gen):
    T, E = case["T"], case["E"]
    x = torch.randn((T, E), generator=gen, device="cuda") * 1.5 + _popularity(E, 0.3, gen)
    return x.to(DT[case["dtype"]])


def _rows(case, gen):
    """Rows in expert order of T tokens with k different experts each: offsets, row -> token * k + choice."""
    T, k, E = case["T"], case["k"], case["E"]
    odds = _popularity(E, case["skew"], gen)
    if E > 4 and case["skew"] > 0:
        odds[torch.randperm(E, generator=gen, device="cuda")[: min(E // 10, E - k)]] = -1e9  # idle experts
    noise = -torch.log(-torch.log(torch.rand((T, E), generator=gen, device="cuda").clamp(1e-7, 1 - 1e-7)))
    idx = (odds + noise).topk(k, dim=1).indices.flatten()
    src = torch.sort(idx, stable=True).indices.to(torch.int32)
    sizes = torch.bincount(idx, minlength=E)
    offsets = torch.zeros((E + 1,), dtype=torch.int32, device="cuda")
    offsets[1:] = sizes.cumsum(0)
    return offsets, src, int(sizes.max())


def _quantized(w, group, zeros):
    """Codes 0..15 of the rows of w (as uint8), scales and zero points of their groups."""
    K = w.shape[-1]
    pad = (-K) % group
    v = torch.nn.functional.pad(w.float(), (0, pad)).unflatten(-1, (-1, group))
    if zeros:
        hi, lo = v.amax(-1).clamp(min=0), v.amin(-1).clamp(max=0)
        scale = ((0.5 * hi - 0.5 * lo) / 7.5).to(w.dtype)
        s = scale.float()
        zero = torch.where(s > 0, (-lo / s).round().clamp(0, 15), 0.0)
        code = torch.where(s[..., None] > 0, (v / s[..., None]).round() + zero[..., None], 0.0).clamp(0, 15)
        zero = zero.to(torch.uint8)
    else:
        scale = (v.abs().amax(-1) / 7).to(w.dtype)
        s = scale.float()
        code = 8 + torch.where(s[..., None] > 0, (v / s[..., None]).round(), 0.0).clamp(-8, 7)
        zero = None
    return code.to(torch.uint8).flatten(-2)[..., :K], scale, zero


def _packed(code):
    """Eight codes to a 32-bit word: element 2 i in bits 4 i, element 2 i + 1 in bits 16 + 4 i."""
    c = code.unflatten(-1, (-1, 4, 2))                      # [.., word, i, parity]
    low = c[..., 0::2, :] | (c[..., 1::2, :] << 4)          # bytes 0, 1 (even elements) and 2, 3 (odd ones)
    return low.transpose(-1, -2).flatten(-3).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, st = case["op"], dict(case=case)
    if op in ("route", "route_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        st["logits"] = _logits(case, gen)
        if op == "route":
            # a balancing bias moves in steps of a thousandth
            st["bias"] = (torch.randn((E,), generator=gen, device="cuda") * 30).round() / 1000 if case["bias"] else None
            return st
        _, idx = _choose(st["logits"].double(), dict(case, groups=0))
        st["idx"] = idx.to(torch.int32)
        st["dw"] = torch.randn((T, k), generator=gen, device="cuda")
        if case["losses"]:
            st["counts"] = torch.bincount(idx.flatten(), minlength=E).to(torch.int32)
            # the coefficients that a training step gives its losses
            st["dlosses"] = torch.tensor([0.01, 0.001], device="cuda")
        return st
    if op == "quantize":
        w = torch.randn((case["rows"], case["K"]), generator=gen, device="cuda")
        # rows of different magnitude, a few of them zero
        size = torch.rand((case["rows"], 1), generator=gen, device="cuda")
        st["x"] = w.mul_(case["K"] ** -0.5 * (0.5 + size)).mul_(size > 0.001).to(DT[case["dtype"]])
        return st
    T, k, E, K, group = case["T"], case["k"], case["E"], case["K"], case["group"]
    rows = case["N"] * (2 if case["swiglu"] else 1)
    dtype = DT[case["dtype"]]
    offsets, src, st["longest"] = _rows(case, gen)
    R = T * k
    st["offsets"] = offsets
    x = torch.randn((T if case["swiglu"] else R, K), generator=gen, device="cuda")
    wide = torch.rand((K,), generator=gen, device="cuda") < 0.01
    st["x"] = x.mul_(torch.where(wide, 8.0, 1.0)).to(dtype)
    st["src"] = src if case["swiglu"] else None   # a gate/up product gathers the tokens, others have their rows
    st["gates"] = torch.rand((R,), generator=gen, device="cuda") * 0.95 + 0.05 if case["gated"] else None
    groups = -(-K // group)
    st["codes"] = torch.empty((E, rows, K // 2), dtype=torch.uint8, device="cuda")
    st["scales"] = torch.empty((E, rows, groups), dtype=dtype, device="cuda")
    st["zeros"] = torch.empty((E, rows, groups), dtype=torch.uint8, device="cuda") if case["zeros"] else None
    for e in range(E):
        w = (torch.randn((rows, K), generator=gen, device="cuda") * K ** -0.5).to(dtype)
        code, st["scales"][e], zero = _quantized(w, group, case["zeros"])
        st["codes"][e] = _packed(code)
        if zero is not None:
            st["zeros"][e] = zero
    return st


# -------------------------------------------------------------- plain form --
def _live(x):
    """Logits with -inf for what is not a number, and finite at the top."""
    return torch.where(x > -math.inf, x, -math.inf).clamp(max=FLT_MAX)


def _scores(x, score):
    """Scores of live logits (any float type) and the sum that softmax divides by, with its maximum."""
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    top = x.amax(1, keepdim=True).clamp(min=-FLT_MAX)
    e = torch.exp(x - top)
    return e / e.sum(1, keepdim=True).clamp(min=1e-30)


def _choose(x, case, bias=None):
    """Keys and the k experts of largest key, in descending order, ties to the lower index."""
    x = _live(x)
    T, E = x.shape
    need = bias is not None or (case.get("groups") and case["group_top"] == 2)
    s = _scores(x, case["score"]) if need else x
    key = s if bias is None else s + bias.to(x.dtype)
    key = torch.where(x > -math.inf, key, -math.inf)
    pick = key if bias is not None else x
    if case.get("groups"):
        g = key.unflatten(1, (case["groups"], -1))
        best, at = g.max(2)
        if case["group_top"] == 2 and g.shape[2] > 1:
            second = g.scatter(2, at[..., None], -math.inf).amax(2)
            best = torch.where(second > -math.inf, best + second, best)
        kept = torch.zeros_like(best, dtype=torch.bool)
        for _ in range(case["topk_groups"]):
            free = torch.where(kept, -math.inf, best)
            # a group that is taken cannot be taken again, even where every score is -inf
            i = torch.where(kept, 2, (free < free.amax(1, keepdim=True)).int()).argmin(1)
            kept.scatter_(1, i[:, None], True)
        allowed = kept.repeat_interleave(E // case["groups"], 1)
    else:
        allowed = torch.ones_like(pick, dtype=torch.bool)
    idx = torch.empty((T, case["k"]), dtype=torch.int64, device=x.device)
    for j in range(case["k"]):
        free = torch.where(allowed, pick, -math.inf)
        i = torch.where(allowed, (free < free.amax(1, keepdim=True)).int(), 2).argmin(1)
        idx[:, j] = i
        allowed = allowed.scatter(1, i[:, None], False)
    return pick, idx


def _route(st):
    case = st["case"]
    T, E, k = case["T"], case["E"], case["k"]
    _, idx = _choose(st["logits"].double(), case, st["bias"])
    x = _live(st["logits"].float())
    s = _scores(x, case["score"])
    w = s.gather(1, idx)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    out = [idx.to(torch.int32), w * case["scale"]]
    if case["losses"]:
        counts = torch.bincount(idx.flatten(), minlength=E)
        p = s if case["score"] == "softmax" else s / s.sum(1, keepdim=True)
        top = x.amax(1)
        lse = top + torch.log(torch.exp(x - top[:, None]).sum(1))
        balance = (counts.float() * p.mean(0)).sum() * (E / (k * T))
        out += [counts.to(torch.int32), torch.stack([balance, lse.square().mean()])]
    return out


def _route_bwd(st):
    case = st["case"]
    T, E, k = case["T"], case["E"], case["k"]
    idx, x = st["idx"].long(), _live(st["logits"].float())
    s = _scores(x, case["score"])
    chosen, dw = s.gather(1, idx), st["dw"] * case["scale"]
    if case["renorm"]:
        total = chosen.sum(1, keepdim=True)
        dw = (dw - (dw * chosen).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(s).scatter_(1, idx, dw)
    if case["losses"]:
        a = st["dlosses"][0] * (E / (k * T * T)) * st["counts"].float()
    if case["score"] == "softmax":
        if case["losses"]:
            ds = ds + a
        dx = s * (ds - (s * ds).sum(1, keepdim=True))
    else:
        if case["losses"]:
            total = s.sum(1, keepdim=True)
            ds = ds + (a - (s * a).sum(1, keepdim=True) / total) / total
        dx = ds * s * (1 - s)
    if case["losses"]:
        top = x.amax(1, keepdim=True)
        e = torch.exp(x - top)
        total = e.sum(1, keepdim=True)
        dx = dx + st["dlosses"][1] * (2 / T) * (top + torch.log(total)) * (e / total)
    return dx.to(st["logits"].dtype)


def _values(codes, scales, zeros, group):
    """fp32 values of packed codes [.., K / 2]."""
    even, odd = codes.unflatten(-1, (-1, 2, 2)).unbind(-2)                # two bytes of four even, of four odd elements
    pair = torch.stack([even, odd], -1)                                   # [.., word, byte, parity]
    v = torch.stack([pair & 15, pair >> 4], -2).flatten(-4).float()       # element 4 byte + 2 nibble + parity
    K = v.shape[-1]
    zero = 8.0 if zeros is None else zeros.repeat_interleave(group, -1)[..., :K].float()
    return v.sub_(zero).mul_(scales.repeat_interleave(group, -1)[..., :K].float())


def _unpaired(w, dim):
    """Rows of gate and up, interleaved per 128 along dim, as two halves."""
    w = w.unflatten(dim, (-1, 2, 128))
    return w.select(dim + 1, 0).flatten(dim, dim + 1), w.select(dim + 1, 1).flatten(dim, dim + 1)


def _product(st):
    case = st["case"]
    E, K, rows = case["E"], case["K"], st["codes"].shape[1]
    R = case["T"] * case["k"]
    x = st["x"].float()
    x = x if st["src"] is None else x[(st["src"] // case["k"]).long()]
    out = torch.zeros((R, rows), device=x.device)
    ids = torch.arange(R, device=x.device)
    z = st["zeros"]
    if R < E:  # each row with its own expert's weights
        e = torch.searchsorted(st["offsets"][1:].contiguous(), ids.to(torch.int32), right=True)
        w = _values(st["codes"][e], st["scales"][e], None if z is None else z[e], case["group"])
        out = torch.bmm(w, x[:, :, None])[:, :, 0]
    else:      # every expert's weights, a few at a time, on its rows padded to the longest
        step = max(1, (1 << 28) // (rows * K))
        for lo in range(0, E, step):
            hi = min(E, lo + step)
            w = _values(st["codes"][lo:hi], st["scales"][lo:hi], None if z is None else z[lo:hi], case["group"])
            at = st["offsets"][lo:hi, None].long() + torch.arange(st["longest"], device=x.device)
            inside = at < st["offsets"][lo + 1:hi + 1, None]
            y = torch.bmm(x[at.clamp(max=R - 1)], w.transpose(1, 2))
            out[at[inside]] = y[inside]
    if case["swiglu"]:
        gate, up = _unpaired(out, 1)
        out = gate / (1 + torch.exp(-gate)) * up
    if st["gates"] is not None:
        out = out * st["gates"][:, None]
    return out.to(st["x"].dtype)


def _plain(st):
    case = st["case"]
    if case["op"] == "route":
        return _route(st)
    if case["op"] == "route_bwd":
        return _route_bwd(st)
    if case["op"] == "quantize":
        code, scale, zero = _quantized(st["x"], case["group"], case["zeros"])
        zero = 8.0 if zero is None else zero.repeat_interleave(case["group"], 1)[:, :case["K"]].float()
        s = scale.repeat_interleave(case["group"], 1)[:, :case["K"]].float()
        return ((code.float() - zero) * s).to(st["x"].dtype)
    return _product(st)


# ------------------------------------------------------- the library's calls --
def _own(st):
    import routing_permute_grouped_gb300 as moe

    case = st["case"]
    op, dev = case["op"], torch.device("cuda")
    if op in ("route", "route_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        rule = moe.score_rule(E=E, k=k, score=case["score"], n_groups=case.get("groups", 0),
                              topk_groups=case.get("topk_groups", 0), group_top=case.get("group_top", 1),
                              renormalize=case["renorm"], scale=case["scale"])
        if op == "route_bwd":
            out = torch.empty((T, E), dtype=st["logits"].dtype, device=dev)
            moe.moe_route_scores_bwd(rule, st["logits"], st["idx"], out, dw=st["dw"], counts=st.get("counts"),
                                     dlosses=st.get("dlosses"))
            return out
        idx = torch.empty((T, k), dtype=torch.int32, device=dev)
        w = torch.empty((T, k), dtype=torch.float32, device=dev)
        if not case["losses"]:
            moe.moe_route_scores(rule, st["logits"], idx, w, bias=st["bias"])
            return [idx, w]
        counts = torch.empty((E,), dtype=torch.int32, device=dev)
        losses = torch.empty((2,), dtype=torch.float32, device=dev)
        ws = torch.empty((moe.moe_route_scores_workspace_size(rule, T),), dtype=torch.uint8, device=dev)
        moe.moe_route_scores(rule, st["logits"], idx, w, bias=st["bias"], counts=counts, losses=losses, ws=ws)
        return [idx, w, counts, losses]
    group = case["group"]
    if op == "quantize":
        rows, K, dtype = case["rows"], case["K"], st["x"].dtype
        codes = torch.empty((rows, K // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((rows, -(-K // group)), dtype=dtype, device=dev)
        zeros = torch.empty(scales.shape, dtype=torch.uint8, device=dev) if case["zeros"] else None
        moe.moe_quantize_int4(group, st["x"], codes, scales, zeros=zeros)
        out = torch.empty((rows, K), dtype=dtype, device=dev)
        moe.moe_dequantize_int4(group, codes, scales, out, zeros=zeros)
        return out
    out = torch.empty((case["T"] * case["k"], case["N"]), dtype=st["x"].dtype, device=dev)
    moe.moe_grouped_gemm_int4(group, st["x"], st["codes"], st["scales"], st["offsets"], out, w_zeros=st["zeros"],
                              src=st["src"], src_div=case["k"], row_scale=st["gates"], swiglu=case["swiglu"])
    return out


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op = case["op"]
    el = 4 if case["dtype"] == "fp32" else 2
    if op in ("route", "route_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        loads = 4 * E if case["losses"] else 0
        if op == "route":
            return dict(bytes=T * E * el + T * k * 8 + (4 * E if case["bias"] else 0) + loads, flops=8 * T * E)
        return dict(bytes=2 * T * E * el + T * k * 8 + loads, flops=10 * T * E)
    per = 0.5 + (3 if case["zeros"] else 2) / case["group"]   # bytes of a weight
    if op == "quantize":
        n = case["rows"] * case["K"]
        return dict(bytes=4 * n, flops=3 * n)
    E, K, R = case["E"], case["K"], case["T"] * case["k"]
    rows = case["N"] * (2 if case["swiglu"] else 1)
    used = E * (1 - (1 - case["k"] / E) ** case["T"])         # experts with rows, loads being even
    x = case["T"] if case["swiglu"] else R
    return dict(bytes=used * rows * K * per + 2 * x * K + 2 * R * case["N"] + (4 * R if case["gated"] else 0),
                flops=2 * R * rows * K)


# ------------------------------------------------------ the definition in fp64 --
def _ranked(key):
    """Indices in descending order of the keys, ties in ascending order of the index."""
    return torch.sort(key, dim=1, descending=True, stable=True).indices


def _exact_route(st):
    case = st["case"]
    T, E, k = case["T"], case["E"], case["k"]
    x = st["logits"].double()
    dead = ~(x > -math.inf)
    x = x.masked_fill(dead, -math.inf).clamp(max=FLT_MAX)
    s = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
    bias = torch.zeros(E, dtype=torch.float64, device=x.device) if st["bias"] is None else st["bias"].double()
    key = (s + bias).masked_fill(dead, -math.inf)
    order = x if st["bias"] is None else key  # scores rise with the logits, which separate them where they round alike
    if case["groups"]:
        n = case["groups"]
        by = order if case["group_top"] == 1 else key
        top = by.reshape(T, n, E // n).sort(2, descending=True).values[:, :, :case["group_top"]]
        value = torch.where(top[:, :, 0] > -math.inf, top.masked_fill(top == -math.inf, 0).sum(2), -math.inf)
        kept = torch.zeros((T, n), dtype=torch.bool, device=x.device)
        kept.scatter_(1, _ranked(value)[:, :case["topk_groups"]], True)
        group = torch.arange(E, device=x.device) // (E // n)
        # within the kept groups first, then by key
        first = _ranked(order)
        inside = kept[:, group].gather(1, first)
        idx = first.gather(1, torch.sort(inside.int(), dim=1, descending=True, stable=True).indices)[:, :k]
    else:
        idx = _ranked(order)[:, :k]
    w = s.gather(1, idx)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    out = [idx.to(torch.int32), w * case["scale"]]
    if case["losses"]:
        counts = (idx[..., None] == torch.arange(E, device=x.device)).sum((0, 1))
        out += [counts.to(torch.int32), _exact_losses(x, counts, case)]
    return out


def _exact_losses(x, counts, case):
    T, E, k = case["T"], case["E"], case["k"]
    s = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
    share = (s / s.sum(1, keepdim=True)).mean(0)
    load = counts.double() / (k * T)
    return torch.stack([E * (share * load).sum(), torch.logsumexp(x, 1).pow(2).mean()])


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(st)
    if op == "route_bwd":
        x = st["logits"].double().requires_grad_()
        s = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
        w = s.gather(1, st["idx"].long())
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        total = (w * case["scale"] * st["dw"].double()).sum()
        if case["losses"]:
            total = total + (_exact_losses(x, st["counts"], case) * st["dlosses"].double()).sum()
        return torch.autograd.grad(total, x)[0]
    if op == "quantize":
        x, group = st["x"], case["group"]
        v = x.double()
        out = torch.empty_like(v)
        for lo in range(0, case["K"], group):
            part = v[:, lo:lo + group]
            if case["zeros"]:
                top = part.max(1, keepdim=True).values.clamp(min=0)
                low = part.min(1, keepdim=True).values.clamp(max=0)
                s = ((top - low) / 15).to(x.dtype).double()
                z = torch.where(s > 0, torch.round(-low / s), 0).clamp(0, 15)
                q = torch.where(s > 0, torch.round(part / s) + z, 0).clamp(0, 15)
            else:
                s = (part.abs().max(1, keepdim=True).values / 7).to(x.dtype).double()
                z = 8
                q = torch.where(s > 0, torch.round(part / s), 0).clamp(-8, 7) + z
            out[:, lo:lo + group] = (q - z) * s
        return out
    bounds = st["offsets"].tolist()
    group, K = case["group"], case["K"]
    place = torch.arange(K, device="cuda")
    word, byte = place // 8 * 4, (place % 8) // 4 + (place % 2) * 2   # a byte holds elements of one parity
    shift = (place % 4) // 2 * 4
    out = torch.zeros((case["T"] * case["k"], case["N"]), dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        lo, hi = bounds[e], bounds[e + 1]
        if hi == lo:
            continue
        w = ((st["codes"][e][:, word + byte] >> shift.to(torch.uint8)) & 15).double()
        w -= 8 if st["zeros"] is None else st["zeros"][e][:, place // group].double()
        w *= st["scales"][e][:, place // group].double()
        x = st["x"][lo:hi] if st["src"] is None else st["x"][(st["src"][lo:hi] // case["k"]).long()]
        y = x.double() @ w.T
        if case["swiglu"]:
            column = torch.arange(case["N"], device="cuda")
            gate = column // 128 * 256 + column % 128
            y = torch.nn.functional.silu(y[:, gate]) * y[:, gate + 128]
        out[lo:hi] = y
    if st["gates"] is not None:
        out *= st["gates"][:, None].double()
    return out
