"""CPU tests of grouped_linear's autograd side: the two library calls are replaced
by plain ones that keep the library's rules on layouts."""
import pytest
import torch

import routing_permute_grouped_gb300 as moe


def _check_rows(t):
    """The library's rules for a matrix of rows."""
    assert t.stride(1) == 1 and t.data_ptr() % 16 == 0
    assert t.shape[0] <= 1 or (t.stride(0) >= t.shape[1] and t.stride(0) % 8 == 0), t.stride()


def _gemm(x, w, offsets, y, row_scale=None, w_transposed=False, status=None, stream=None):
    _check_rows(x)
    _check_rows(y)
    for e in range(w.shape[0]):
        s = slice(int(offsets[e]), int(offsets[e + 1]))
        y[s] = x[s] @ (w[e] if w_transposed else w[e].T)


def _wgrad(a, b, offsets, out, status=None, stream=None):
    _check_rows(a)
    _check_rows(b)
    for e in range(out.shape[0]):
        s = slice(int(offsets[e]), int(offsets[e + 1]))
        out[e] = a[s].T @ b[s]


@pytest.fixture
def plain_calls(monkeypatch):
    monkeypatch.setattr(moe, "moe_grouped_gemm", _gemm)
    monkeypatch.setattr(moe, "moe_grouped_wgrad", _wgrad)


OFF = [2, 9, 9, 20]  # 21 rows: two before the first group, one past the last


def _reference(x, w):
    parts = [x[:OFF[0]] @ torch.zeros_like(w[0]).T]
    parts += [x[OFF[e]:OFF[e + 1]] @ w[e].T for e in range(3)]
    return torch.cat(parts + [x[OFF[-1]:] @ torch.zeros_like(w[0]).T])


def _odd_address(y):
    """A gradient 2 elements into its allocation: that of a part of a concatenated vector."""
    return torch.cat([y.new_zeros(2), y.flatten()])


LOSSES = {
    "sum over rows": lambda y, c: (y.sum(0) * c[0]).sum(),      # dy has strides (0, 1)
    "sum over columns": lambda y, c: (y.sum(1) * c[:, 0]).sum(),  # (1, 0)
    "sum": lambda y, c: y.sum(),                                # (0, 0)
    "transposed": lambda y, c: (y.t() * c.t().contiguous()).sum(),
    "row slice": lambda y, c: (y[3:18] * c[3:18]).sum(),
    "column slice": lambda y, c: (y[:, 8:16] * c[:, 8:16]).sum(),
    "odd address": lambda y, c: (_odd_address(y) * torch.arange(y.numel() + 2)).sum(),
}


@pytest.mark.parametrize("loss", LOSSES)
def test_any_gradient_layout(plain_calls, loss):
    g = torch.Generator().manual_seed(1)
    offsets = torch.tensor(OFF, dtype=torch.int32)
    x = torch.randn((21, 16), generator=g).requires_grad_()
    w = torch.randn((3, 24, 16), generator=g).requires_grad_()
    c = torch.randn((21, 24), generator=g)
    got = torch.autograd.grad(LOSSES[loss](moe.grouped_linear(x, w, offsets), c), (x, w))
    want = torch.autograd.grad(LOSSES[loss](_reference(x, w), c), (x, w))
    for a, b in zip(got, want):
        assert torch.allclose(a, b, rtol=1e-5, atol=1e-4)


def test_any_input_layout(plain_calls):
    g = torch.Generator().manual_seed(2)
    offsets = torch.tensor(OFF, dtype=torch.int32)
    w = torch.randn((3, 24, 16), generator=g)
    one, t = torch.randn((16,), generator=g), torch.randn((16, 21), generator=g)
    odd = torch.randn((21 * 16 + 1,), generator=g)[1:].view(21, 16)
    wide = torch.randn((21, 21), generator=g)[:, :16]
    for x in (one.expand(21, 16), t.t(), odd, wide):
        x = x.detach().requires_grad_()
        y = moe.grouped_linear(x, w, offsets)
        assert torch.allclose(y, _reference(x, w), rtol=1e-5, atol=1e-5)
        (dx,) = torch.autograd.grad(y.square().sum(), x)
        (want,) = torch.autograd.grad(_reference(x, w).square().sum(), x)
        assert torch.allclose(dx, want, rtol=1e-5, atol=1e-4)


def test_second_derivatives_are_refused(plain_calls):
    """The gradients carry no graph of their own: asking for one raises instead of
    leaving a gradient penalty's term out."""
    g = torch.Generator().manual_seed(3)
    offsets = torch.tensor(OFF, dtype=torch.int32)
    x = torch.randn((21, 16), generator=g).requires_grad_()
    w = torch.randn((3, 24, 16), generator=g).requires_grad_()
    y = moe.grouped_linear(x, w, offsets)
    dx, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (y.sum() + dx.square().sum()).backward()
    # first derivatives in the same graph are what they were
    dx, dw = torch.autograd.grad(moe.grouped_linear(x, w, offsets).square().sum(), (x, w))
    want = torch.autograd.grad(_reference(x, w).square().sum(), (x, w))
    assert torch.allclose(dx, want[0], rtol=1e-5, atol=1e-4) and torch.allclose(dw, want[1], rtol=1e-5, atol=1e-4)
