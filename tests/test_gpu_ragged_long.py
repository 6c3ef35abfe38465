"""GPU test of a weight gradient whose one sum takes longer than the 2 s after which
a kernel's wait for its next step gives up."""
import pytest
import torch

import routing_permute_grouped_gb300 as moe

pytestmark = pytest.mark.gpu


def test_wgrad_of_two_to_the_thirty_rows():
    """All rows are one group's, among 64, so that one CTA pair runs 2^24 steps.  All
    but a few rows are zero and those hold small whole numbers: the result is exact."""
    R, n, e = 1 << 30, 8, 40
    a = torch.zeros((R, n), dtype=torch.bfloat16, device="cuda")
    rows = [0, 5, 63, 64, R // 2 + 3, R - 70, R - 7, R - 6]
    a[rows] = (torch.arange(len(rows) * n, device="cuda") % 7 - 3).reshape(len(rows), n).bfloat16()
    a[R - 5:] = float("nan")  # rows of no group, in the last step of the sum
    off = [0] * (e + 1) + [R - 5] * (64 - e)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    out = torch.full((64, n, n), 3.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(64, dtype=torch.int32, device="cuda")
    moe.moe_grouped_wgrad(a, a, offsets, out, status=status)
    assert moe.moe_get_device_status(status) == 0
    few = a[rows].double()
    assert torch.equal(out[e].double(), few.T @ few)
    out[e] = 0
    assert (out == 0).all()
