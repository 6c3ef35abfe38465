"""GPU tests of the routing by scores and of its gradient against plain fp64
arithmetic (scores_ref.py).

Bounds, u = 2^-24 (half a step of fp32).  exp is off by 2 u (1 + |argument|) at
most (its own error and its rounded argument), a division or product by u, a sum
of E <= 256 positive terms in a tree by 13 u: a score, a share or a weight is off
by (2 d + 40) u of itself, d the spread of a token's logits (for sigmoids: their
largest magnitude).  A gradient is a sum of at most five products of such factors
with the incoming gradients, so its error is (4 d + 200) u times the sum of the
terms' magnitudes; a 16-bit one adds half a step of its type."""
import pytest
import torch

import routing_permute_grouped_gb300 as moe
from tests import scores_ref as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: (0.0, 0.0), torch.bfloat16: (2.0 ** -8, 2.0 ** -134), torch.float16: (2.0 ** -11, 2.0 ** -25)}
INF, NAN = float("inf"), float("nan")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _logits(T, E, dtype=torch.float32, seed=0, std=2.0):
    return (torch.randn((T, E), generator=_gen(seed), device="cuda") * std).to(dtype)


def _bias(E, seed=1, step=0.001):
    return (torch.randn((E,), generator=_gen(seed), device="cuda") * 0.05 / step).round() * step


def _route(rule, logits, bias=None, losses=False, **kw):
    T = logits.shape[0]
    idx = torch.full((T, rule.k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, rule.k), NAN, device="cuda")
    if not losses:
        moe.moe_route_scores(rule, logits, idx, w, bias=bias, **kw)
        return idx, w
    counts = torch.full((rule.E,), -1, dtype=torch.int32, device="cuda")
    both = torch.full((2,), NAN, device="cuda")
    ws = torch.full((moe.moe_route_scores_workspace_size(rule, T),), 0xFF, dtype=torch.uint8, device="cuda")
    moe.moe_route_scores(rule, logits, idx, w, bias=bias, counts=counts, losses=both, ws=ws, **kw)
    return idx, w, counts, both


def _reach(logits, rule):
    d, mag = ref.spread(logits)
    return mag if rule.score else d


def _check_weights(w, logits, idx, rule):
    want = ref.weights(logits, idx, rule)
    tol = (2 * _reach(logits, rule)[:, None] + 40) * 2 * U * want.abs() + 2.0 ** -140
    assert torch.isfinite(w).all()
    assert ((w.double() - want).abs() <= tol).all(), (w.double() - want).abs().max()


def _check_losses(both, logits, counts, rule):
    want = ref.losses(logits, counts, rule)
    d, mag = ref.spread(logits)
    reach = _reach(logits, rule).max().item()
    # sums over tokens: at most 2^11 terms one after the other in a warp's part, then trees
    n = 60 + min(logits.shape[0], 2048)
    assert abs(both[0].item() - want[0].item()) <= (2 * reach + 40 + n) * U * want[0].item() + 1e-30
    # log-sum-exp: off by u times its terms and 2 u of the exponentials' own
    lse_off = (mag.max().item() + reach + 40) * U
    lse = want[1].sqrt().item()
    assert abs(both[1].item() - want[1].item()) <= 2 * lse * lse_off + lse_off ** 2 + (n + 4) * U * want[1].item()


RULES = [  # E, k, groups, kept, best of a group
    (1, 1, 0, 0, 1), (2, 1, 0, 0, 1), (3, 3, 0, 0, 1), (8, 2, 0, 0, 1), (8, 8, 4, 4, 1), (24, 3, 8, 2, 2), (30, 4, 5, 3, 2),
    (33, 5, 3, 2, 1), (64, 6, 0, 0, 1), (64, 6, 32, 3, 2), (65, 7, 5, 2, 2), (100, 8, 10, 1, 1), (128, 4, 16, 4, 2),
    (160, 6, 8, 3, 1), (250, 8, 10, 4, 2), (256, 8, 8, 4, 2), (256, 8, 8, 4, 1), (256, 8, 1, 1, 2), (256, 3, 32, 20, 2),
]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("E,k,groups,kept,top", RULES)
def test_choice_and_weights(E, k, groups, kept, top, with_bias, score):
    for i, dtype in enumerate((torch.float32, torch.bfloat16, torch.float16)):
        for renorm in (False, True):
            rule = moe.score_rule(E, k, score, groups, kept, top, renorm, 1.0 if renorm else 2.5)
            logits = _logits(131, E, dtype, seed=E + i)
            bias = _bias(E) if with_bias else None
            idx, w = _route(rule, logits, bias)
            assert torch.equal(idx.cpu(), ref.choose(logits, rule, bias))
            _check_weights(w, logits, idx, rule)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,kept,top", [r for r in RULES if r[0] in (8, 64, 65, 256)])
def test_losses(E, k, groups, kept, top, score):
    for T, dtype in ((1, torch.float32), (16, torch.bfloat16), (301, torch.float32), (6000, torch.float16)):
        rule = moe.score_rule(E, k, score, groups, kept, top)
        logits = _logits(T, E, dtype, seed=T)
        bias = _bias(E)
        idx, w, counts, both = _route(rule, logits, bias, losses=True)
        again = _route(rule, logits, bias, losses=True)
        assert all(torch.equal(a, b) for a, b in zip((idx, w, counts, both), again))  # the same bits every time
        plain = _route(rule, logits, bias)
        assert torch.equal(plain[0], idx) and torch.equal(plain[1], w)
        if T <= 301:
            assert torch.equal(idx.cpu(), ref.choose(logits, rule, bias))
        assert torch.equal(counts.long(), torch.bincount(idx.flatten().long(), minlength=E))
        _check_losses(both, logits, counts, rule)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,kept,top", [(0, 0, 1), (8, 3, 1), (8, 3, 2)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_ties_go_to_the_lower_index(score, groups, kept, top, with_bias):
    E, T = 64, 200
    logits = _logits(T, E, seed=3, std=1.0).mul(2).round().div(2).add(0.0)  # a handful of values
    logits[:20] = 0.25
    logits[20:30, ::2] = -0.0  # equal to 0
    logits[20:30, 1::2] = 0.0
    bias = _bias(E, step=0.05) if with_bias else None
    for k in (1, 5, 8):
        rule = moe.score_rule(E, k, score, groups, kept, top)
        idx, w = _route(rule, logits, bias)
        assert torch.equal(idx.cpu(), ref.choose(logits, rule, bias))
        _check_weights(w, logits, idx, rule)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(64, 0), (64, 8), (256, 8), (60, 6)])
def test_keys_that_fp32_cannot_separate(score, E, groups):
    """Biases that undo the scores' differences but for parts of 1e-9: the exact order counts."""
    T, k = 64, 8
    gen = _gen(9)
    logits = torch.randn((1, E), generator=gen, device="cuda").repeat(T, 1)
    rule = moe.score_rule(E, k, score, groups, max(groups // 2, 0), 2)
    s = ref.scores(ref.tame(logits), rule)[0]
    bias = (1.0 - s).float()  # keys within 2^-24 of 1, in an order that only fp64 sees
    logits = logits + torch.randint(0, 2, (T, E), generator=gen, device="cuda") * 2.0 ** -22
    idx, w = _route(rule, logits, bias)
    assert torch.equal(idx.cpu(), ref.choose(logits, rule, bias))
    _check_weights(w, logits, idx, rule)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top", [(0, 1), (4, 1), (4, 2)])
def test_masked_and_infinite_logits(dtype, score, groups, top):
    E, k, T = 24, 4, 40
    lowest = torch.finfo(dtype).min
    logits = _logits(T, E, dtype, seed=5)
    logits[0] = -INF
    logits[1] = NAN
    logits[2, 3:] = -INF
    logits[3, :23] = NAN
    logits[4, 7] = INF
    logits[5, [2, 9]] = INF
    logits[6] = INF
    logits[7] = lowest
    logits[8, ::2] = lowest
    logits[9, :6] = -INF      # a whole group of four
    logits[10, 1:6] = -INF    # one left in it
    logits[11] = torch.finfo(dtype).max
    bias = _bias(E)
    bias[3], bias[10], bias[20] = -INF, NAN, INF
    for renorm in (False, True):
        rule = moe.score_rule(E, k, score, groups, 2 if groups else 0, top, renorm)
        for b in (None, bias):
            idx, w, counts, both = _route(rule, logits, b, losses=True)
            assert torch.equal(idx.cpu(), ref.choose(logits, rule, b)), b is None
            plain = _route(rule, logits, b)
            assert torch.equal(plain[0], idx) and torch.equal(plain[1], w)
            rows = [t for t in range(T) if t not in (7, 8, 11)] if rule.score == 0 else list(range(T))
            # (2 d + 40) u is no bound where d passes 2^20: there exp is 0 or 1
            _check_weights(w[rows][6:], logits[rows][6:], idx[rows][6:], rule)
            want = ref.weights(logits, idx, rule)
            assert torch.allclose(w.double(), want, rtol=1e-4, atol=1e-6)
            assert not torch.isnan(both[0]) and torch.equal(counts.sum(), torch.tensor(T * k, device="cuda"))


def test_sigmoids_of_very_small_scores_renormalise():
    logits = _logits(50, 16, std=3.0) - 90.0  # scores around 1e-39
    rule = moe.score_rule(16, 4, "sigmoid")
    idx, w, counts, both = _route(rule, logits, losses=True)
    assert torch.equal(idx.cpu(), ref.choose(logits, rule))
    _check_weights(w, logits, idx, rule)
    _check_losses(both, logits, counts, rule)


@pytest.mark.parametrize("E", [5, 8, 31, 64, 130, 256])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_strides_and_alignment(E, dtype):
    T, rule = 70, moe.score_rule(E, 2)
    dense = _logits(T, E, dtype)
    want = _route(rule, dense)
    for pad, first in ((1, 0), (8, 0), (8, 1), (3, 2), (16, 8)):
        wide = torch.full((T, E + pad + first), 9.0, dtype=dtype, device="cuda")
        view = wide[:, first:first + E]
        view.copy_(dense)
        got = _route(rule, view)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        out = torch.full((T, E + pad + first), 5.0, dtype=dtype, device="cuda")
        dw = torch.randn((T, 2), generator=_gen(2), device="cuda")
        moe.moe_route_scores_bwd(rule, view, got[0], out[:, first:first + E], dw=dw)
        plain = torch.empty_like(dense)
        moe.moe_route_scores_bwd(rule, dense, got[0], plain, dw=dw)
        assert torch.equal(out[:, first:first + E], plain)
        out[:, first:first + E] = 5.0
        assert (out == 5.0).all()


# --------------------------------------------------------------- gradient --
def _grad_ref(logits, idx, rule, dw, counts, dlosses):
    x = logits.double().requires_grad_()
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    if dw is not None:
        total = total + (ref.weights(x, idx, rule) * dw.double()).sum()
    if dlosses is not None:
        total = total + (ref.losses(x, counts, rule) * dlosses.double()).sum()
    return torch.autograd.grad(total, x)[0]


def _grad_scale(logits, rule, dw, counts, dlosses):
    """Per token, the magnitude of the terms that its gradient sums."""
    T, E, k = logits.shape[0], rule.E, rule.k
    m = torch.zeros((T,), dtype=torch.float64, device="cuda")
    if dw is not None:
        m += 2 * abs(rule.scale) * dw.double().abs().amax(1)
    if dlosses is not None:
        m += 2 * abs(dlosses[0].item()) * E / (k * T * T) * counts.max().item()
        m += abs(dlosses[1].item()) * 2 / T * torch.logsumexp(ref.tame(logits), 1).abs()
    return m


def _check_grad(got, logits, idx, rule, dw, counts, dlosses):
    want = _grad_ref(logits, idx, rule, dw, counts, dlosses)
    rel, tiny = HALF[logits.dtype]
    tol = ((4 * _reach(logits, rule) + 200) * U * _grad_scale(logits, rule, dw, counts, dlosses))[:, None]
    assert torch.isfinite(got).all()
    off = (got.double() - want).abs()
    assert (off <= tol + rel * (want.abs() + tol) + tiny + 1e-30).all(), (off - tol).max()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("terms", ["weights", "losses", "both"])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (8, 2), (33, 5), (64, 6), (100, 8), (256, 8)])
def test_gradient(E, k, score, renorm, terms):
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        for T in (1, 77, 700):
            rule = moe.score_rule(E, k, score, renormalize=renorm, scale=1.0 if renorm else 2.5)
            logits = _logits(T, E, dtype, seed=T)
            idx, _, counts, _ = _route(rule, logits, _bias(E), losses=True)
            dw = torch.randn((T, k), generator=_gen(11), device="cuda") if terms != "losses" else None
            dl = torch.tensor([0.7, -0.3], device="cuda") if terms != "weights" else None
            c = counts if terms != "weights" else None
            out = torch.full((T, E), NAN, dtype=dtype, device="cuda")
            moe.moe_route_scores_bwd(rule, logits, idx, out, dw=dw, counts=c, dlosses=dl)
            _check_grad(out, logits, idx, rule, dw, counts, dl)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(score, renorm):
    T, E, k, h = 5, 12, 3, 1e-6
    rule = moe.score_rule(E, k, score, renormalize=renorm, scale=1.5)
    logits = _logits(T, E, seed=21)
    idx, _, counts, _ = _route(rule, logits, losses=True)
    dw, dl = torch.randn((T, k), generator=_gen(4), device="cuda"), torch.tensor([0.5, 0.25], device="cuda")
    out = torch.empty_like(logits)
    moe.moe_route_scores_bwd(rule, logits, idx, out, dw=dw, counts=counts, dlosses=dl)

    def value(x):
        return ((ref.weights(x, idx, rule) * dw.double()).sum() + (ref.losses(x, counts, rule) * dl.double()).sum()).item()

    for t in range(T):
        for e in range(E):
            step = torch.zeros_like(logits, dtype=torch.float64)
            step[t, e] = h
            slope = (value(logits.double() + step) - value(logits.double() - step)) / (2 * h)
            # a difference is off by h^2 times a third derivative (below 20) and rounding over h
            assert abs(out[t, e].item() - slope) <= 1e-8 + 3e-5 * (abs(slope) + dw.abs().max().item()) * 0.1


def test_gradient_of_masked_rows_and_of_indices_that_repeat_or_do_not_exist():
    E, k = 16, 4
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            rule = moe.score_rule(E, k, score, renormalize=renorm)
            logits = _logits(6, E, seed=8)
            logits[0] = -INF
            logits[1, 2:] = NAN
            idx = torch.tensor([[0, 1, 2, 3], [0, 1, 2, 3], [5, 5, 5, 5], [5, 7, 5, 7], [-1, 4, 16, 6], [-5, 99, 1 << 30, -1]],
                               dtype=torch.int32, device="cuda")
            dw = torch.randn((6, k), generator=_gen(3), device="cuda")
            counts = torch.arange(E, dtype=torch.int32, device="cuda")
            dl = torch.tensor([0.5, 0.25], device="cuda")
            out = torch.full((6, E), NAN, device="cuda")
            moe.moe_route_scores_bwd(rule, logits, idx, out, dw=dw, counts=counts, dlosses=dl)
            again = torch.full((6, E), NAN, device="cuda")
            moe.moe_route_scores_bwd(rule, logits, idx, again, dw=dw, counts=counts, dlosses=dl)
            assert torch.equal(out, again) and torch.isfinite(out).all()
            assert (out[0] == 0).all() and (out[1, 2:] == 0).all()
            # the rows of numbers: known choices alone, each as often as it is named
            for t in range(2, 6):
                known = [j for j in range(k) if 0 <= idx[t, j] < E]
                x = logits[t:t + 1].double().requires_grad_()
                total = (ref.losses(torch.cat([logits[:t].double(), x, logits[t + 1:].double()]), counts, rule)
                         * dl.double()).sum()
                if known:
                    total = total + (ref.weights(x, idx[t:t + 1, known], rule) * dw[t:t + 1, known].double()).sum()
                want = torch.autograd.grad(total, x)[0][0]
                assert ((out[t].double() - want).abs() <= 400 * U * (2 * dw[t].abs().max().item() + 1)).all()


# ------------------------------------------------------------------ calls --
def test_no_tokens():
    rule = moe.score_rule(8, 2)
    empty = torch.empty((0, 8), device="cuda")
    idx, w, counts, both = _route(rule, empty, losses=True)
    assert (counts == 0).all() and (both == 0).all()
    _route(rule, empty)
    moe.moe_route_scores_bwd(rule, empty, idx, torch.empty_like(empty), dw=w)
    x = torch.empty((0, 8), device="cuda", requires_grad=True)
    (moe.route_scores(x, rule)[0].sum()).backward()
    assert x.grad.shape == (0, 8)


def test_autograd():
    T, E, k = 50, 32, 4
    rule = moe.score_rule(E, k, "sigmoid", scale=2.0)
    base = _logits(T, 2 * E, seed=2)
    bias = _bias(E)
    for view in (lambda b: b[:, :E], lambda b: b[:, ::2], lambda b: b.t().reshape(2 * E, T).t()[:, :E],
                 lambda b: b[:1, :E].expand(T, E)):
        leaf = base.clone().requires_grad_()
        w, idx, both, counts = moe.route_scores(view(leaf), rule, bias, losses=True)
        g = torch.randn((k, T), generator=_gen(6), device="cuda").t()  # a gradient of another layout
        ((w * g).sum() + both @ torch.tensor([0.5, 0.1], device="cuda")).backward()
        x = view(base).contiguous()
        out = torch.empty_like(x)
        moe.moe_route_scores_bwd(rule, x, idx, out, dw=g.contiguous(), counts=counts,
                                 dlosses=torch.tensor([0.5, 0.1], device="cuda"))
        leaf2 = base.clone().requires_grad_()
        view(leaf2).backward(out)
        assert torch.equal(leaf.grad, leaf2.grad)
        leaf3 = base.clone().requires_grad_()
        w, idx = moe.route_scores(view(leaf3), rule, bias)
        w.sum().backward()
        assert torch.isfinite(leaf3.grad).all()
    leaf = base[:, :E].clone().requires_grad_()
    both = moe.route_scores(leaf, rule, losses=True)[2]
    both[1].backward()  # the weights unused
    assert leaf.grad.abs().sum() > 0
    w = moe.route_scores(leaf, rule)[0]
    g, = torch.autograd.grad(w.square().sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_captured_and_replayed_and_on_another_stream():
    T, E = 300, 64
    rule = moe.score_rule(E, 6, "sigmoid", 8, 4, 2)
    bias = _bias(E)
    logits = _logits(T, E)
    idx = torch.empty((T, 6), dtype=torch.int32, device="cuda")
    w = torch.empty((T, 6), device="cuda")
    counts, both = torch.empty((E,), dtype=torch.int32, device="cuda"), torch.empty((2,), device="cuda")
    ws = torch.empty((moe.moe_route_scores_workspace_size(rule, T),), dtype=torch.uint8, device="cuda")
    dw, dl, out = torch.randn((T, 6), device="cuda"), torch.tensor([0.1, 0.2], device="cuda"), torch.empty_like(logits)

    def step():
        moe.moe_route_scores(rule, logits, idx, w, bias=bias, counts=counts, losses=both, ws=ws)
        moe.moe_route_scores_bwd(rule, logits, idx, out, dw=dw, counts=counts, dlosses=dl)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        logits.copy_(_logits(T, E, seed=seed))
        graph.replay()
        got = [t.clone() for t in (idx, w, counts, both, out)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, (idx, w, counts, both, out)))
        assert torch.equal(idx.cpu(), ref.choose(logits, rule, bias))


def test_many_tokens():
    T, E = 70001, 256
    rule = moe.score_rule(E, 8, "sigmoid", 8, 4, 2)
    logits, bias = _logits(T, E), _bias(E)
    idx, w, counts, both = _route(rule, logits, bias, losses=True)
    some = torch.randperm(T, generator=_gen(1), device="cuda")[:300]
    assert torch.equal(idx[some].cpu(), ref.choose(logits[some], rule, bias))
    _check_weights(w, logits, idx, rule)
    _check_losses(both, logits, counts, rule)
    dw, dl = torch.randn((T, 8), device="cuda"), torch.tensor([0.5, 0.25], device="cuda")
    out = torch.empty_like(logits)
    moe.moe_route_scores_bwd(rule, logits, idx, out, dw=dw, counts=counts, dlosses=dl)
    _check_grad(out, logits, idx, rule, dw, counts, dl)
