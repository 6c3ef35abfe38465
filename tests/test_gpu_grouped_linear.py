"""GPU tests of grouped_linear on the layouts that torch hands it.  The gradients
of one row-major and one odd layout of the same values are equal bit for bit."""
import pytest
import torch

import routing_permute_grouped_gb300 as moe
from tests.test_gpu_ragged import _check, _gen, _rand

pytestmark = pytest.mark.gpu

OFF = [2, 40, 40, 99]  # 104 rows


def _operands(dtype):
    offsets = torch.tensor(OFF, dtype=torch.int32, device="cuda")
    return _rand((104, 64), 1, dtype), _rand((3, 72, 64), 2, dtype, 1 / 8), offsets


def _expanded_rows(shape, dtype):
    return _rand((1, shape[1]), 5, dtype).expand(shape)


def _expanded(shape, dtype):
    return torch.full((), 0.375, dtype=dtype, device="cuda").expand(shape)


def _transposed(shape, dtype):
    return _rand(shape[::-1], 6, dtype).t()


def _odd_address(shape, dtype):
    return _rand((shape[0] * shape[1] + 1,), 7, dtype)[1:].view(shape)


def _odd_stride(shape, dtype):
    return _rand((shape[0], shape[1] + 5), 8, dtype)[:, :shape[1]]


def _columns(shape, dtype):
    return _rand((shape[0], shape[1] + 16), 9, dtype)[:, 8:8 + shape[1]]


LAYOUTS = [_expanded_rows, _expanded, _transposed, _odd_address, _odd_stride, _columns]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_any_gradient_layout(dtype, layout):
    x, w, offsets = _operands(dtype)
    x.requires_grad_(), w.requires_grad_()
    dy = layout((104, 72), dtype)
    dense = dy.clone(memory_format=torch.contiguous_format)
    want = torch.autograd.grad(moe.grouped_linear(x, w, offsets), (x, w), dense)
    got = torch.autograd.grad(moe.grouped_linear(x, w, offsets), (x, w), dy)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    d, xd, wd = dense.double(), x.detach().double(), w.detach().double()
    for e in range(3):
        s = slice(OFF[e], OFF[e + 1])
        _check(got[0][s], d[s] @ wd[e], d[s].abs() @ wd[e].abs(), 72, dtype)
        _check(got[1][e], d[s].T @ xd[s], d[s].abs().T @ xd[s].abs(), 59, dtype)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_any_input_layout(layout):
    _, w, offsets = _operands(torch.bfloat16)
    x = layout((104, 64), torch.bfloat16)
    dense = x.clone(memory_format=torch.contiguous_format)
    assert torch.equal(moe.grouped_linear(x, w, offsets), moe.grouped_linear(dense, w, offsets))


def test_sum_over_rows():
    """The gradient of a sum over rows reaches backward with row stride 0."""
    x, w, offsets = _operands(torch.bfloat16)
    x.requires_grad_()
    c = torch.randn((72,), generator=_gen(3), device="cuda").bfloat16()
    moe.grouped_linear(x, w, offsets).sum(0).backward(c)
    assert (x.grad[:2] == 0).all() and (x.grad[99:] == 0).all()
    for e in range(3):
        want = (c.double() @ w[e].double()).expand(OFF[e + 1] - OFF[e], 64)
        mag = (c.double().abs() @ w[e].double().abs()).expand_as(want)
        _check(x.grad[OFF[e]:OFF[e + 1]], want, mag, 72, torch.bfloat16)
