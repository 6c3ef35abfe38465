"""GPU tests of 4-bit values and products at the ends of their types' ranges.  A value is
an exact product rounded once, so values are compared to the bit; of sums with an
infinite scale, the infinity's sign."""
import pytest
import torch

import routing_permute_grouped_gb300 as moe
from tests.test_gpu_int4 import NAN, TYPES, _codes_ref, _quantize, _rand, _values

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_values_of_quantised_extremes(dtype, zeros, group):
    """Rows from the type's largest numbers to its subnormal ones, and back."""
    info = torch.finfo(dtype)
    base = _rand((40, 256), group, dtype).float().clamp(-4, 4) / 4
    top = torch.tensor(info.max).log2()
    size = torch.cat([2.0 ** (top - torch.arange(20) / 2), torch.tensor([info.smallest_normal]) * 2.0 ** torch.arange(-4, 16)])
    x = (base.double() * size.double().cuda()[:, None]).to(dtype)
    x[0, ::2], x[0, 1::2] = info.max, -info.max
    x[1], x[2] = info.max, -info.max
    assert torch.isfinite(x).all()
    codes, scales, z = _quantize(group, x, zeros)
    assert torch.equal(scales.double(), _codes_ref(x, group, zeros)[1])
    out = torch.full_like(x, NAN)
    moe.moe_dequantize_int4(group, codes, scales, out, zeros=z)
    assert torch.equal(out, _values(codes, scales, z, group).to(dtype))


@pytest.mark.parametrize("dtype", TYPES)
def test_values_of_every_code_and_zero_point(dtype):
    """All codes with all zero points, under scales of any size and either sign."""
    info = torch.finfo(dtype)
    word = torch.arange(8, dtype=torch.int64).mul(4)
    first = int((torch.arange(8) << word).sum())         # codes 0 .. 7
    second = int(((torch.arange(8) + 8) << word).sum())  # codes 8 .. 15
    row = torch.tensor([first, second - (1 << 32)] * 2, dtype=torch.int32)
    for s in (info.max, info.max / 16, 2.0 ** 12, 1.0, info.smallest_normal, info.smallest_normal * info.eps, 0.0):
        for sign in (1.0, -1.0):
            codes = row.repeat(17, 1).cuda().view(torch.uint8)
            scales = torch.full((17, 1), sign * s, dtype=dtype, device="cuda")
            z = torch.arange(16, dtype=torch.uint8, device="cuda")[:, None].contiguous()
            for zz, n in ((z, 16), (None, 17)):
                out = torch.full((n, 32), NAN, dtype=dtype, device="cuda")
                moe.moe_dequantize_int4(32, codes[:n].contiguous(), scales[:n].contiguous(), out, zeros=zz)
                want = _values(codes[:n], scales[:n], zz, 32).to(dtype)
                assert torch.equal(out, want), (s, sign)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("with_zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_an_infinite_scale_gives_infinities(dtype, with_zeros, group):
    """A sum other than 0 times an infinite scale, in any group of a row and wherever the row
    ends: an infinity of the sum's sign."""
    for R, N in ((1, 16), (3, 40), (64, 1032)):
        for K in (32, 96, 128, 160, 256, 384) if R < 64 else (16384, 16544):
            n = -(-K // group)
            codes = torch.full((1, N, K // 2), 0xBB, dtype=torch.uint8, device="cuda")  # 11
            codes[:, ::2] = 0x33                                                        # 3
            z = torch.full((1, N, n), 8, dtype=torch.uint8, device="cuda") if with_zeros else None
            x = torch.ones((R, K), dtype=dtype, device="cuda")
            for at in {0, n - 1}:
                scales = torch.full((1, N, n), 2.0 ** -9, dtype=dtype, device="cuda")
                scales[:, :, at] = INF
                y = torch.full((R, N), NAN, dtype=dtype, device="cuda")
                moe.moe_grouped_gemm_int4(group, x, codes, scales, None, y, w_zeros=z)
                assert (y[:, ::2] == -INF).all() and (y[:, 1::2] == INF).all(), (R, K, at)
