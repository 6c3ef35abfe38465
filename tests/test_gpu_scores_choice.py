"""GPU tests of the choice of experts where equal keys, masked experts or keys at the
end of fp32's range meet the last place, against plain fp64 arithmetic (scores_ref.py).

What is compared are indices: they have to be equal.  The inputs' exact keys are far
enough apart in fp64 (by 2^-40 of themselves at least, or equal) for its own rounding
not to matter."""
import pytest
import torch

import routing_permute_grouped_gb300 as moe
from tests import scores_ref as ref

pytestmark = pytest.mark.gpu

INF = float("inf")


def _route(rule, logits, bias=None, losses=False):
    T = logits.shape[0]
    idx = torch.full((T, rule.k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, rule.k), float("nan"), device="cuda")
    kw = {}
    if losses:
        kw = dict(counts=torch.empty((rule.E,), dtype=torch.int32, device="cuda"), losses=torch.empty((2,), device="cuda"),
                  ws=torch.empty((moe.moe_route_scores_workspace_size(rule, T),), dtype=torch.uint8, device="cuda"))
    moe.moe_route_scores(rule, logits, idx, w, bias=bias, **kw)
    return idx, w


def _check(rule, logits, bias):
    logits = logits.cuda()
    bias = None if bias is None else bias.cuda()
    want = ref.choose(logits, rule, bias)
    for losses in (False, True):
        idx, w = _route(rule, logits, bias, losses)
        off = (idx.cpu() != want).any(1).nonzero().flatten()
        assert not len(off), (off[0].item(), idx[off[0]].tolist(), want[off[0]].tolist())
        assert torch.isfinite(w).all()


# ------------------------------------------- equal keys at the last place --
def test_a_larger_exact_key_behind_two_equal_ones():
    """Sigmoids of 17 and 18, and of 20 and 20.125, are 1 in fp32; 3 and its neighbour are
    not told apart under a bias of 100."""
    up = torch.nextafter(torch.tensor(3.0), torch.tensor(4.0)).item()
    rows = torch.tensor([[17.0, 17.0, 18.0], [20.0, 20.0, 20.125], [18.0, 17.0, 17.0], [17.0, 18.0, 17.0], [3.0, 3.0, up]])
    for bias in (0.0, 100.0):
        for k in (1, 2):
            _check(moe.score_rule(3, k, "sigmoid"), rows, torch.full((3,), bias))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept,top", [(16, 0, 0, 1), (64, 0, 0, 1), (256, 0, 0, 1), (64, 8, 4, 1), (64, 8, 4, 2),
                                               (60, 6, 3, 2), (256, 8, 4, 2)])
@pytest.mark.parametrize("ties", [2, 3, 7, 40])
@pytest.mark.parametrize("k", [1, 5, 8])
def test_equal_keys_over_the_last_place(score, E, groups, kept, top, ties, k):
    """`ties` experts of one logit hold the last place, one or two others have a key that is
    larger or smaller but the same, or next to it, in fp32."""
    if ties > E // 2:
        ties = E // 2
    T = 120
    gen = torch.Generator().manual_seed(E + 10 * ties + k + top)
    rule = moe.score_rule(E, k, score, groups, kept, top)
    for kind in ("saturated", "large bias"):
        if kind == "saturated":  # scores of 1, or of 0, in fp32
            base = 18.0 if score == "sigmoid" else -30.0
            rest, step = base - 16.0 + torch.randn((T, E), generator=gen) * 0.3, 0.125
            bias = torch.zeros(E)
        else:
            base = 0.5
            rest, step = -4.0 + torch.randn((T, E), generator=gen) * 0.3, 2.0 ** -16
            bias = torch.full((E,), 100.0)
        logits = rest
        # k - 1 or fewer clear ones, the ties, and strangers a step away, at random places
        for t in range(T):
            order = torch.randperm(E, generator=gen)
            clear = int(torch.randint(max(0, k - ties), k, (1,), generator=gen))
            logits[t, order[:clear]] = base + 4.0 + 0.25 * torch.arange(clear)
            logits[t, order[clear:clear + ties]] = base
            strangers = order[clear + ties:clear + ties + 1 + t % 2]
            logits[t, strangers] = base + step * (1 if t % 3 else -1)
        if score == "softmax" and kind == "saturated":
            logits[:, 0] = 0.0  # takes all of the softmax
        _check(rule, logits, bias)


def test_equal_logits_under_unequal_biases():
    """More experts than lanes share a logit; their biases differ by less than fp32 keys can."""
    E, T = 256, 64
    gen = torch.Generator().manual_seed(5)
    logits = torch.zeros((T, E))
    logits[1::2] = 0.25
    bias = 1.0 + torch.randint(0, 3, (E,), generator=gen) * 2.0 ** -23
    logits[:, 7] += 2.0 ** -22
    for score in ("softmax", "sigmoid"):
        for k in (1, 8):
            for groups, kept, top in ((0, 0, 1), (8, 4, 2)):
                _check(moe.score_rule(E, k, score, groups, kept, top), logits, bias)
                _check(moe.score_rule(E, k, score, groups, kept, top), torch.zeros((T, E)), torch.full((E,), 0.25))


# ---------------------------------------------- masks and the ends of fp32 --
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_sums_of_a_group_that_pass_fp32(score):
    """Two best keys whose sum is past fp32's largest number, or below its lowest: their
    order counts all the same, and a group that has them is not one without experts."""
    half = torch.finfo(torch.float32).max
    cases = [
        ([0.0] * 4, [2e38, 2e38, 3e38, 3e38], 2),
        ([0.0] * 4, [3e38, 3e38, INF, INF], 2),
        ([0.0] * 4, [INF, 1e38, INF, 2e38], 2),
        ([0.0] * 4, [-3e38, -3e38, -2e38, -2e38], 2),
        ([-INF, -INF, 0.0, 0.0], [0.0, 0.0, -3e38, -3e38], 2),
        ([-INF, -INF, 0.0, 0.0, 0.0, 0.0], [0.0, 0.0, -half, -half, -half, -2e38], 3),
        ([0.0, -INF, 0.0, 0.0], [-2e38, 0.0, -half, -half], 2),
        ([0.0, -INF, 0.0, 0.0], [half, 0.0, 1e38, 1e38], 2),
        ([0.0, -INF, 0.0, 0.0], [2e38, 0.0, half, -half], 2),
        ([0.0] * 6, [3e38, 3e38, INF, INF, 3.1e38, 3.1e38], 3),
    ]
    for logits, bias, groups in cases:
        for kept in range(1, groups):
            for k in (1, 2):
                rule = moe.score_rule(len(logits), k, score, groups, kept, 2)
                _check(rule, torch.tensor([logits]), torch.tensor(bias))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,kept,top", [(0, 0, 1), (4, 3, 1), (4, 3, 2)])
def test_biases_of_the_lowest_value_and_masked_logits(score, groups, kept, top):
    """An expert whose bias is the type's lowest number still comes before one without a score."""
    E, k = 16, 8
    lowest = torch.finfo(torch.float32).min
    gen = torch.Generator().manual_seed(3)
    rows, biases = [], []
    for _ in range(60):
        order = torch.randperm(E, generator=gen)
        live, low = (int(torch.randint(0, 7, (1,), generator=gen)) for _ in range(2))
        logits, bias = torch.full((E,), -INF), torch.zeros(E)
        logits[order[:live + low]] = torch.randn(live + low, generator=gen)
        bias[order[live:live + low]] = lowest
        bias[order[live + low:]] = torch.randint(-2, 8, (E - live - low,), generator=gen).float()
        rows.append(logits)
        biases.append(bias)
    for logits, bias in zip(rows, biases):
        _check(moe.score_rule(E, k, score, groups, kept, top), logits[None], bias)


# ----------------------------------------------------------------- weights --
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [8, 64, 256])
def test_equal_scores_have_equal_weights_to_the_bit(score, E):
    """2, 4 or 8 chosen experts of one score: their sum is that many times it exactly, and so
    is the quotient, at any logit."""
    T = 4000
    gen = torch.Generator().manual_seed(E)
    for spread in (1.0, 20.0):
        logits = (torch.randn((T, 1), generator=gen) * spread).expand(T, E).contiguous().cuda()
        for k in (2, 4, 8):
            _, w = _route(moe.score_rule(E, k, score), logits)
            assert (w == 1.0 / k).all()
