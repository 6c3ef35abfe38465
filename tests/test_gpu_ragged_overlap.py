"""GPU tests of the grouped products on offsets that run backwards: the group that
does is skipped and flagged, and of the groups after it the rows before the end of
an earlier group are left out, so that no row is written by two groups."""
import numpy as np
import pytest
import torch

import routing_permute_grouped_gb300 as moe
from tests.test_gpu_ragged import _check, _fp4_operand, _rand

pytestmark = pytest.mark.gpu


def _random(seed, E, R):
    """Ascending offsets of which a few are put anywhere."""
    rng = np.random.default_rng(seed)
    off = np.sort(rng.integers(0, R + 1, E + 1))
    at = rng.choice(E + 1, max(1, E // 8), replace=False)
    off[at] = rng.integers(-3, R + 4, len(at))
    return [int(v) for v in off]


# rows, offsets
CASES = [
    (64, [0, 40, 20, 64]), (1000, [0, 700, 300, 1000]), (1000, [0, 1000, 0, 1000]), (90, [50, 90, 10, 60, 5, 90]),
    (700, [0, 650] + [600 - i for i in range(30)] + [100, 640, 10, 700]),  # over more groups than a warp has lanes
    *[(R, _random(seed, E, R)) for seed, (E, R) in enumerate([(5, 200), (33, 900), (64, 3000), (200, 1500)])],
]


def _owners(R, off):
    """The group of each row, -1 for none, and whether a group was skipped."""
    owner, flagged, end = np.full(R, -1), False, 0
    for e in range(len(off) - 1):
        lo, hi = off[e], off[e + 1]
        if lo < 0 or hi < lo or hi > R:
            flagged = True
            continue
        owner[max(lo, end):hi] = e
        end = max(end, hi)
    return owner, flagged


def _check_rows(run, x, w, K, R, off):
    owner, flagged = _owners(R, off)
    status = torch.zeros(64, dtype=torch.int32, device="cuda")
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    first = None
    for _ in range(3):
        y = torch.full((R, w.shape[1]), 7.0, dtype=torch.bfloat16, device="cuda")
        run(offsets, y, status)
        assert moe.moe_get_device_status(status) == (moe.DEVERR_SEGMENT if flagged else 0)
        assert first is None or torch.equal(y, first)
        first = y
    for e in range(len(off) - 1):
        rows = torch.from_numpy(np.flatnonzero(owner == e)).cuda()
        a, b = x[rows].double(), w[e].double()
        _check(first[rows], a @ b.T, a.abs() @ b.abs().T, K, torch.bfloat16, (off, e))
    assert (first[torch.from_numpy(owner < 0).cuda()] == 7).all()


@pytest.mark.parametrize("K", [72, 1096])  # whole sums, and split over a cluster's pairs where there are few tiles
@pytest.mark.parametrize("case", range(len(CASES)))
def test_product(case, K):
    R, off = CASES[case]
    x, w = _rand((R, K), case), _rand((len(off) - 1, 136, K), case + 50, std=K ** -0.5)
    _check_rows(lambda o, y, s: moe.moe_grouped_gemm(x, w, o, y, status=s), x, w, K, R, off)


@pytest.mark.parametrize("fmt", [moe.FP4_MX, moe.FP4_NV])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_product_fp4(case, fmt):
    (R, off), K = CASES[case], 160
    xq, xs, x = _fp4_operand((R, K), case, fmt)
    wq, ws, w = _fp4_operand((len(off) - 1, 136, K), case + 50, fmt)
    _check_rows(lambda o, y, s: moe.moe_grouped_gemm_fp4(fmt, xq, xs, wq, ws, o, y, status=s), x, w, K, R, off)
