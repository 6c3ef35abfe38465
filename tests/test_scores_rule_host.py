"""The rule of a differentiable routing belongs to its forward pass, without a GPU: the two
calls are recorded in place of the kernels."""
import torch

import routing_permute_grouped_gb300 as moe


def test_a_rule_changed_after_the_forward_pass_is_the_old_one_in_the_gradient(monkeypatch):
    seen = []

    def fields(rule):
        return tuple(getattr(rule, name) for name, _ in rule._fields_)

    def forward(rule, logits, idx, w, bias=None, counts=None, losses=None, ws=None, stream=None):
        idx.zero_()
        w.zero_()
        for t in (counts, losses):
            if t is not None:
                t.zero_()
        seen.append(fields(rule))

    def backward(rule, logits, idx, dlogits, dw=None, counts=None, dlosses=None, stream=None):
        dlogits.zero_()
        seen.append(fields(rule))

    monkeypatch.setattr(moe, "moe_route_scores", forward)
    monkeypatch.setattr(moe, "moe_route_scores_bwd", backward)
    monkeypatch.setattr(moe, "moe_route_scores_workspace_size", lambda rule, T: 16)
    for losses in (False, True):
        rule = moe.score_rule(8, 2, "sigmoid", 4, 2, 2, scale=2.5)
        x = torch.zeros((3, 8), requires_grad=True)
        w = moe.route_scores(x, rule, losses=losses)[0]
        rule.scale, rule.score, rule.renormalize, rule.n_groups = 1.0, 0, 0, 0  # an annealed scale, say
        w.sum().backward()
        assert seen[0] == seen[1] == fields(moe.score_rule(8, 2, "sigmoid", 4, 2, 2, scale=2.5))
        seen.clear()
