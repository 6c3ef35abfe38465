"""Plain fp64 arithmetic of the routing by scores, a token at a time, and the
error that fp32 may make in it.  Tests only."""
import math

import torch

FLT_MAX = torch.finfo(torch.float32).max


def tame(v):
    """What the library takes a logit or a bias for."""
    v = v.double()
    return torch.where(v > -math.inf, v.clamp(max=FLT_MAX), -math.inf)


def scores(x, rule):
    """Scores of tame logits [T, E]; 0 where the logit is -infinity, also in a row of nothing else."""
    if rule.score:
        return torch.where(x >= 0, 1 / (1 + torch.exp(-x)), torch.exp(x) / (1 + torch.exp(x)))
    top = x.amax(1, keepdim=True)
    e = torch.where(x > -math.inf, torch.exp(x - top), 0.0)
    total = e.sum(1, keepdim=True)
    return torch.where(total > 0, e / total, 0.0)


def choose(logits, rule, bias=None):
    """The k experts of every token, in order."""
    x = tame(logits).cpu()
    s = scores(x, rule)
    b = None if bias is None else tame(bias).cpu()
    idx = []
    for t in range(x.shape[0]):
        live = (x[t] > -math.inf).tolist()
        plain = x[t].tolist()
        score = s[t].tolist()
        key = [(v if b is None else v + b[e].item()) if live[e] else -math.inf for e, v in enumerate(score)]
        order = plain if b is None else key
        allowed = range(rule.E)
        if rule.n_groups:
            size = rule.E // rule.n_groups
            value = []
            for g in range(rule.n_groups):
                of = order if rule.group_top == 1 else key
                top = sorted(of[g * size:(g + 1) * size], reverse=True)[:rule.group_top]
                numbers = [v for v in top if v > -math.inf]
                value.append(sum(numbers) if numbers else -math.inf)
            best = sorted(range(rule.n_groups), key=lambda g: (-value[g], g))[:rule.topk_groups]
            allowed = [e for e in range(rule.E) if e // size in best]
        idx.append(sorted(allowed, key=lambda e: (-order[e], e))[:rule.k])
    return torch.tensor(idx, dtype=torch.int32).reshape(-1, rule.k)


def weights(logits, idx, rule):
    s = scores(tame(logits), rule).gather(1, idx.long())
    if rule.renormalize:
        # on a common factor, so that small scores of a whole token do not vanish
        x = tame(logits).gather(1, idx.long())
        top = x.amax(1, keepdim=True)
        m = top.clamp(max=0) if rule.score else top
        part = torch.where(x > -math.inf, torch.exp(x - m) / (1 + torch.exp(x)) if rule.score else torch.exp(x - m), 0.0)
        if rule.score:
            part = torch.where(x > 0, torch.exp(-m) / (1 + torch.exp(-x)), part)
        total = part.sum(1, keepdim=True)
        s = torch.where(total > 0, part / total, 0.0)
    return s * rule.scale


def losses(logits, counts, rule):
    """Balance and z; a token without a finite logit adds nothing."""
    x = tame(logits)
    T = x.shape[0]
    some = (x > -math.inf).any(1)
    y = torch.where(some[:, None], x, 0.0)
    s = scores(y, rule)
    if rule.score:  # ratios of sigmoids on a common factor
        m = y.amax(1, keepdim=True).clamp(max=0)
        s = torch.where(y > 0, torch.exp(-m) / (1 + torch.exp(-y)), torch.exp(y - m) / (1 + torch.exp(y)))
    p = s / s.sum(1, keepdim=True) * some[:, None]
    lse = torch.logsumexp(y, 1) * some
    balance = rule.E / (rule.k * T) * (counts.double() * p.sum(0) / T).sum()
    return torch.stack([balance, lse.square().sum() / T])


def spread(logits):
    """The largest difference of finite logits of a token, and their largest magnitude."""
    x = tame(logits)
    ok = x > -math.inf
    hi = torch.where(ok, x, -math.inf).amax(1)
    lo = torch.where(ok, x, math.inf).amin(1)
    d = torch.where(hi > -math.inf, hi - lo, 0.0)
    mag = torch.where(ok, x.abs(), 0.0).amax(1)
    return d, mag
