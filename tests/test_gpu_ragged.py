"""GPU tests of the grouped products on ragged row groups (16-bit and 4-bit),
their gradients and the 4-bit quantisation, against plain fp64 arithmetic.

Bounds.  A product of two 16-bit (or scaled 4-bit) values is exact in fp32;
a sum of n of them in fp32, in any order and with truncating adders, is off by
at most n * 2^-23 * S, S the sum of the magnitudes.  The result is multiplied
by up to three fp32 factors (2^-23 each) and rounded once to the output type
(half an ulp: 2^-8 of a bf16, 2^-11 of an f16 or 2^-25 below its normal
range).  Codes and scales of the quantisation are fixed by the inputs."""
import math

import numpy as np
import pytest
import torch

import routing_permute_grouped_gb300 as moe

pytestmark = pytest.mark.gpu

HALF_ULP = {torch.bfloat16: (2.0 ** -8, 0.0), torch.float16: (2.0 ** -11, 2.0 ** -25)}


def _offsets(sizes, start=0, gap=0):
    """offsets [E + 1] of consecutive groups; with a gap the rows between two
    groups belong to an extra group that the caller leaves out of the check."""
    off = [start]
    for s in sizes:
        off.append(off[-1] + s)
    return torch.tensor(off, dtype=torch.int32, device="cuda"), off


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(shape, seed, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(shape, generator=_gen(seed), device="cuda") * std).to(dtype)


def _check(got, ref, mag, n, dtype, what=""):
    rel, tiny = HALF_ULP[dtype]
    acc = (n + 8) * 2.0 ** -23 * mag
    bound = acc + rel * (ref.abs() + acc) + tiny
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), what
    worst = (err - bound).max().item() if err.numel() else -1.0
    assert worst <= 0, (what, worst, err.max().item())


def _product_ref(x, w, off, transposed, gate=None):
    R, E = x.shape[0], w.shape[0]
    N = w.shape[2] if transposed else w.shape[1]
    ref = torch.zeros((R, N), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        we = w[e].double() if transposed else w[e].double().T
        ref[lo:hi] = x[lo:hi].double() @ we
        mag[lo:hi] = x[lo:hi].double().abs() @ we.abs()
    if gate is not None:
        ref, mag = ref * gate[:, None].double(), mag * gate[:, None].double().abs()
    return ref, mag


SHAPES = [  # sizes per group, N, K
    ([1], 8, 8),
    ([0, 1, 0, 2], 40, 72),
    ([3, 0, 17, 33], 136, 64),
    ([257, 31, 0, 511, 1], 264, 200),
    ([600, 256, 255], 512, 1000),
    ([5] * 40 + [0] * 16 + [1] * 200, 96, 128),
    ([1000], 1032, 520),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_product(dtype, transposed, case):
    sizes, N, K = SHAPES[case]
    offsets, off = _offsets(sizes)
    R, E = off[-1], len(sizes)
    x = _rand((R, K), 1 + case, dtype)
    w = _rand((E, K, N) if transposed else (E, N, K), 100 + case, dtype, K ** -0.5)
    gate = torch.rand((R,), generator=_gen(7), device="cuda") if case % 2 else None
    y = torch.full((R, N), float("nan"), dtype=dtype, device="cuda")
    moe.moe_grouped_gemm(x, w, offsets, y, row_scale=gate, w_transposed=transposed)
    _check(y, *_product_ref(x, w, off, transposed, gate), K, dtype, (sizes, N, K))


LONG = [  # few rows and long sums: the sum is split over the pairs of a cluster
    ([1], 8, 1024), ([64], 512, 7168), ([0, 33, 2], 264, 4096), ([100], 2048, 2056), ([31, 32, 33], 1000, 1032),
    ([65, 0, 1, 64], 256, 3000), ([7] * 5, 1280, 1544), ([130], 4096, 1096),
    ([64], 4096, 7168), ([128], 4096, 4104), ([50, 0, 63], 4096, 3592),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("case", range(len(LONG)))
def test_product_long_sums(dtype, transposed, case):
    sizes, N, K = LONG[case]
    offsets, off = _offsets(sizes, start=case)
    R, E = off[-1], len(sizes)
    x = _rand((R, K), 1 + case, dtype)
    w = _rand((E, K, N) if transposed else (E, N, K), 100 + case, dtype, K ** -0.5)
    gate = torch.rand((R,), generator=_gen(7), device="cuda") if case % 2 else None
    ref, mag = _product_ref(x, w, off, transposed, gate)
    inside = slice(off[0], off[-1])
    first = None
    for _ in range(3):  # and the same bits every time
        y = torch.full((R, N), float("nan"), dtype=dtype, device="cuda")
        moe.moe_grouped_gemm(x, w, offsets, y, row_scale=gate, w_transposed=transposed)
        _check(y[inside], ref[inside], mag[inside], K, dtype, (sizes, N, K))
        assert first is None or torch.equal(y[inside], first)
        first = y[inside]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_wgrad(dtype, case):
    sizes, M, N = SHAPES[case]
    offsets, off = _offsets(sizes)
    R, E = off[-1], len(sizes)
    a, b = _rand((R, M), 3 + case, dtype), _rand((R, N), 200 + case, dtype)
    out = torch.full((E, M, N), float("nan"), dtype=dtype, device="cuda")
    moe.moe_grouped_wgrad(a, b, offsets, out)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        A, B = a[lo:hi].double(), b[lo:hi].double()
        _check(out[e], A.T @ B, A.abs().T @ B.abs(), hi - lo, dtype, (sizes, e))


MANY = [  # many rows and few outputs: the rows are split over the pairs of a cluster
    ([1024], 8, 8), ([1025], 264, 72), ([4100, 0], 128, 512), ([0, 0, 4300, 1], 96, 520), ([1087, 1089], 1000, 264),
    ([2048, 50, 63, 65, 4000, 127, 0, 2000], 256, 256), ([9000], 1032, 1544), ([3001], 2048, 1024),
    ([2048], 8, 8), ([2049], 264, 72), ([4300, 0, 1, 4400], 96, 520),
    ([7000, 0, 1, 63, 65, 129, 9100, 200], 256, 256), ([0, 5000, 129], 1000, 776),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_wgrad_many_rows(dtype, case):
    sizes, M, N = MANY[case]
    offsets, off = _offsets(sizes, start=3 * case)
    R, E = off[-1] + case, len(sizes)
    a, b = _rand((R, M), 3 + case, dtype), _rand((R, N), 200 + case, dtype)
    for t in (a, b):  # rows of no group
        t[:off[0]] = float("nan")
        t[off[-1]:] = float("nan")
    first = None
    for _ in range(3):  # and the same bits every time
        out = torch.full((E, M, N), float("nan"), dtype=dtype, device="cuda")
        moe.moe_grouped_wgrad(a, b, offsets, out)
        for e in range(E):
            lo, hi = off[e], off[e + 1]
            A, B = a[lo:hi].double(), b[lo:hi].double()
            _check(out[e], A.T @ B, A.abs().T @ B.abs(), hi - lo, dtype, (sizes, e))
        assert first is None or torch.equal(out, first)
        first = out


def test_groups_that_start_late_and_rows_outside():
    """Rows before the first and past the last group are neither read into a
    result nor written, whatever they hold."""
    offsets, off = _offsets([70, 0, 45], start=19)
    R, N, K = off[-1] + 37, 72, 136
    x, w = _rand((R, K), 1), _rand((3, N, K), 2, std=0.1)
    x[:19] = float("nan")
    x[off[-1]:] = float("inf")
    y = torch.full((R, N), 5.0, dtype=torch.bfloat16, device="cuda")
    w[1] = float("nan")  # the empty group's weights
    moe.moe_grouped_gemm(x, w, offsets, y)
    assert (y[:19] == 5).all() and (y[off[-1]:] == 5).all()
    ref, mag = _product_ref(x, w, off, False)
    for e in (0, 2):
        s = slice(off[e], off[e + 1])
        _check(y[s], ref[s], mag[s], K, torch.bfloat16)
    dw = torch.empty((3, N, K), dtype=torch.bfloat16, device="cuda")
    dy = _rand((R, N), 3)
    dy[:19] = float("inf")
    moe.moe_grouped_wgrad(dy, x, offsets, dw)
    for e in range(3):
        A, B = dy[off[e]:off[e + 1]].double(), x[off[e]:off[e + 1]].double()
        _check(dw[e], A.T @ B, A.abs().T @ B.abs(), 70, torch.bfloat16)


def test_nan_stays_in_its_row():
    offsets, off = _offsets([40, 41])
    x, w = _rand((81, 64), 1), _rand((2, 48, 64), 2)
    x[13, 5] = float("nan")
    x[50, 0] = float("inf")
    y = torch.empty((81, 48), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm(x, w, offsets, y)
    bad = ~torch.isfinite(y).all(1)
    assert bad.nonzero().flatten().tolist() == [13, 50]


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(seed):
    rng = np.random.default_rng(seed)
    E = int(rng.integers(1, 40))
    sizes = [int(v) for v in rng.choice([0, 1, 2, 7, 16, 33, 64, 100, 129, 300], E)]
    N, K = int(rng.integers(1, 90)) * 8, int(rng.integers(1, 90)) * 8
    dtype = (torch.bfloat16, torch.float16)[seed & 1]
    offsets, off = _offsets(sizes, start=int(rng.integers(0, 9)))
    R = off[-1] + int(rng.integers(1, 9))
    # strided rows: slices of wider matrices
    x = _rand((R, K + 24), seed, dtype)[:, 8:8 + K]
    dy = _rand((R, N + 8), seed + 50, dtype)[:, :N]
    w = _rand((E, N, K), seed + 90, dtype, K ** -0.5)
    y = torch.zeros((R, N + 16), dtype=dtype, device="cuda")[:, 8:8 + N]
    dx = torch.zeros((R, K), dtype=dtype, device="cuda")
    dw = torch.empty((E, N, K), dtype=dtype, device="cuda")
    moe.moe_grouped_gemm(x, w, offsets, y)
    moe.moe_grouped_gemm(dy, w, offsets, dx, w_transposed=True)
    moe.moe_grouped_wgrad(dy, x, offsets, dw)
    inside = slice(off[0], off[-1])
    ref, mag = _product_ref(x, w, off, False)
    _check(y[inside], ref[inside], mag[inside], K, dtype)
    ref, mag = _product_ref(dy, w, off, True)
    _check(dx[inside], ref[inside], mag[inside], N, dtype)
    for e in range(E):
        A, B = dy[off[e]:off[e + 1]].double(), x[off[e]:off[e + 1]].double()
        _check(dw[e], A.T @ B, A.abs().T @ B.abs(), sizes[e], dtype)


def test_gradients_against_differences():
    """L = sum(dy * y) is linear in x and W: its difference along D equals the
    gradient's product with D.  Operands are multiples of 1/8 small enough that
    x + D and W + D are bf16 values; the bound is six standard deviations of
    the independent roundings of y and of the gradient."""
    sizes = [30, 0, 65, 1]
    offsets, off = _offsets(sizes)
    R, N, K = off[-1], 64, 96
    g = _gen(11)

    def grid(shape):
        return (torch.randint(-8, 9, shape, generator=g, device="cuda") / 8).bfloat16()

    x, w, dy = grid((R, K)), grid((4, N, K)), grid((R, N))
    Dx, Dw = grid((R, K)), grid((4, N, K))

    def forward(x, w):
        y = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")
        moe.moe_grouped_gemm(x, w, offsets, y)
        return y.double()

    dx, dw = torch.empty_like(x), torch.empty_like(w)
    moe.moe_grouped_gemm(dy, w, offsets, dx, w_transposed=True)
    moe.moe_grouped_wgrad(dy, x, offsets, dw)
    y0, u = forward(x, w), 2.0 ** -8
    for y1, grad, D in ((forward(x + Dx, w), dx, Dx), (forward(x, w + Dw), dw, Dw)):
        diff = (dy.double() * (y1 - y0)).sum()
        along = (grad.double() * D.double()).sum()
        var = ((dy.double() * u) ** 2 * (y0 ** 2 + y1 ** 2)).sum() + ((D.double() * u * grad.double()) ** 2).sum()
        assert abs(diff - along) <= 6 * var.sqrt() / math.sqrt(3), (diff.item(), along.item())


def test_bad_offsets_are_flagged_and_skipped():
    x, w = _rand((64, 64), 1), _rand((3, 64, 64), 2)
    status = torch.zeros(64, dtype=torch.int32, device="cuda")
    for off in ([0, 40, 20, 64], [0, 20, 40, 65], [-1, 20, 40, 64]):
        offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
        y = torch.zeros((64, 64), dtype=torch.bfloat16, device="cuda")
        dw = torch.full((3, 64, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_grouped_gemm(x, w, offsets, y, status=status)
        assert moe.moe_get_device_status(status) == moe.DEVERR_SEGMENT
        moe.moe_grouped_wgrad(x, x, offsets, dw, status=status)
        assert moe.moe_get_device_status(status) == moe.DEVERR_SEGMENT
        for e in range(3):
            lo, hi = off[e], off[e + 1]
            if lo < 0 or hi < lo or hi > 64:
                assert (dw[e] == 0).all()
            else:
                A = x[lo:hi].double()
                _check(dw[e], A.T @ A, A.abs().T @ A.abs(), hi - lo, torch.bfloat16)


def test_no_rows():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = _rand((2, 72, 64), 1)
    offsets = torch.zeros(3, dtype=torch.int32, device="cuda")
    moe.moe_grouped_gemm(x, w, offsets, torch.empty((0, 72), dtype=torch.bfloat16, device="cuda"))
    dw = torch.full((2, 72, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_wgrad(torch.empty((0, 72), dtype=torch.bfloat16, device="cuda"), x, offsets, dw)
    assert (dw == 0).all()


def test_another_stream_and_repeats():
    """The same bits on any stream and on every call."""
    offsets, off = _offsets([300, 17, 0, 129])
    x, w = _rand((off[-1], 256), 1), _rand((4, 264, 256), 2, std=1 / 16)
    first = torch.empty((off[-1], 264), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm(x, w, offsets, first)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        y = torch.zeros_like(first)
        torch.cuda.synchronize()
        moe.moe_grouped_gemm(x, w, offsets, y, stream=s)
        s.synchronize()
        assert torch.equal(y, first)


def test_offsets_past_32_bits():
    """Rows whose element offsets exceed 2^31 and 2^32 (x and y far apart in
    a wide matrix)."""
    R, wide, N, K = 300_000, 16384, 64, 64
    buf = torch.zeros((R, wide), dtype=torch.bfloat16, device="cuda")
    x, y = buf[:, :K], buf[:, 8192:8192 + N]
    x.copy_(_rand((R, K), 1))
    w = _rand((2, N, K), 2, std=1 / 8)
    offsets, off = _offsets([R - 1000, 1000])
    moe.moe_grouped_gemm(x, w, offsets, y)
    for lo, hi, e in ((0, 500, 0), (R - 1500, R - 1000, 0), (R - 1000, R, 1)):
        ref = x[lo:hi].double() @ w[e].double().T
        _check(y[lo:hi], ref, x[lo:hi].double().abs() @ w[e].double().abs().T, K, torch.bfloat16)
    dw = torch.empty((2, N, K), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_wgrad(y, x, offsets, dw)
    A, B = y[R - 1000:].double(), x[R - 1000:].double()
    _check(dw[1], A.T @ B, A.abs().T @ B.abs(), 1000, torch.bfloat16)


# ------------------------------------------------------------ 4-bit rows ----
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])
BLOCK = {moe.FP4_MX: 32, moe.FP4_NV: 16}


def _nearest(v, grid):
    """Index of the nearest grid value (v >= 0), ties to the even index."""
    mid = (grid[1:] + grid[:-1]) / 2
    i = np.searchsorted(mid, v)
    j = np.minimum(i, len(mid) - 1)
    return i + ((mid[j] == v) & (i < len(mid)) & (i % 2 == 1))


def _quant_ref(x, fmt, g):
    """Codes, scale bytes and values of x [rows, K] (float64 of 16-bit values)."""
    v = x.reshape(x.shape[0], -1, BLOCK[fmt])
    bad = ~np.isfinite(v).all(-1)
    v = np.where(bad[..., None], 0.0, v)
    top = np.abs(v).max(-1)
    if fmt == moe.FP4_MX:
        m, e = np.frexp(np.where(top > 0, top, 0.75))
        byte = np.where(top > 0, np.maximum(e - np.where(m <= 0.75, 3, 2) + 127, 0), 127)
        scale = np.ldexp(1.0, byte - 127)
        q = v / scale[..., None]
    else:
        # amax / (6 g), the scale and the quotients: one fp32 operation each
        f = np.float32
        byte = _nearest(np.minimum(top.astype(f) / (f(g) * f(6)), f(448)).astype(np.float64), E4M3)
        scale = E4M3[byte].astype(f) * f(g)
        with np.errstate(divide="ignore", invalid="ignore"):
            q = np.where(scale[..., None] > 0, v.astype(f) / scale[..., None], 0).astype(np.float64)
    code = _nearest(np.minimum(np.abs(q), 6.0), E2M1)
    sign = np.signbit(q) & (scale[..., None] > 0)
    byte = np.where(bad, 255 if fmt == moe.FP4_MX else 127, byte)
    values = np.where(sign, -1, 1) * E2M1[code] * scale.astype(np.float64)[..., None]
    values[bad] = np.nan
    return (code + 8 * sign).reshape(x.shape), byte, values.reshape(x.shape)


def _quantize(fmt, x, K=None, **kw):
    K = K or x.shape[1]
    rows = kw["src"].numel() if kw.get("src") is not None else x.shape[0]
    codes = torch.full((rows, K // 2), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, moe.moe_fp4_scale_stride(fmt, K)), 0xAB, dtype=torch.uint8, device="cuda")
    moe.moe_quantize_fp4(fmt, x, codes, scales, **kw)
    return codes, scales


def _nibbles(codes):
    c = codes.cpu().numpy().astype(np.int64)
    return np.stack([c & 15, c >> 4], -1).reshape(c.shape[0], -1)


def _check_quantized(fmt, x, codes, scales, g):
    code, byte, values = _quant_ref(x.double().cpu().numpy(), fmt, g)
    nb = byte.shape[1]
    got = scales.cpu().numpy()
    assert np.array_equal(got[:, :nb], byte)
    assert (got[:, nb:] == 0).all()
    keep = np.repeat(byte != (255 if fmt == moe.FP4_MX else 127), BLOCK[fmt], 1)
    # -0 and 0 stand for the same value
    same = np.where(code == 8, 0, code) == np.where(_nibbles(codes) == 8, 0, _nibbles(codes))
    assert (same | ~keep).all()
    return values


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fmt", [moe.FP4_MX, moe.FP4_NV])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (7, 544), (64, 1024), (33, 7168), (1000, 64)])
def test_quantize(fmt, dtype, rows, K):
    x = _rand((rows, K + 8), rows + K, dtype, 3.0)[:, :K]
    x[0, :16] = 0
    if rows > 2:
        x[1] = 0
        x[2] *= 2.0 ** -12
    g = None
    if fmt == moe.FP4_NV:
        g = (x.abs().amax().float() * (1.01 / 2688)).reshape(1)
    codes, scales = _quantize(fmt, x, tensor_scale=g)
    values = _check_quantized(fmt, x, codes, scales, 1.0 if g is None else g.item())
    for out_dtype in (torch.bfloat16, torch.float16):
        out = torch.empty((rows, K), dtype=out_dtype, device="cuda")
        moe.moe_dequantize_fp4(fmt, codes, scales, out, tensor_scale=g)
        rel, tiny = HALF_ULP[out_dtype]
        ref = torch.from_numpy(values).cuda()
        assert ((out.double() - ref).abs() <= (rel + 2.0 ** -23) * ref.abs() + tiny).all()


@pytest.mark.parametrize("fmt", [moe.FP4_MX, moe.FP4_NV])
def test_quantize_ties_and_extremes(fmt):
    """Every tie of the code grid at every power of two, the largest and the
    smallest magnitudes, NaN and infinity, signed zeros."""
    rows = []
    for p in range(-133, 126):
        ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.2, 0.26, 0.74, 3.4, 5.5, 0.0, 3.0, 1.0])
        rows.append(np.concatenate([ties, -ties]) * 2.0 ** p)
    x = torch.from_numpy(np.stack(rows)).float().bfloat16().cuda()
    special = torch.zeros((6, 32), dtype=torch.bfloat16, device="cuda")
    special[0, 3] = float("nan")
    special[1, 20] = float("inf")
    special[2] = 3.3895313892515355e38  # the largest bf16
    special[3] = -0.0
    special[4, 7] = 9.183549615799121e-41  # the smallest bf16
    special[5, 31] = -float("inf")
    x = torch.cat([x, special])
    codes, scales = _quantize(fmt, x)
    values = _check_quantized(fmt, x, codes, scales, 1.0)
    out = torch.empty_like(x)
    moe.moe_dequantize_fp4(fmt, codes, scales, out)
    got = out.double().cpu().numpy()
    # 2 + 4 bits fit a bf16; the largest bf16 rounds up to 4 * 2^126, past every fp32
    ref = torch.from_numpy(values).float().bfloat16().double().numpy()
    assert np.array_equal(got, ref, equal_nan=True)


@pytest.mark.parametrize("fmt", [moe.FP4_MX, moe.FP4_NV])
def test_quantize_gathers_rows(fmt):
    x = _rand((50, 160), 1)
    src = torch.randint(0, 200, (333,), generator=_gen(2), device="cuda").to(torch.int32)
    src[5], src[6], src[7] = -1, 200, 2 ** 30  # no such row: zeros
    codes, scales = _quantize(fmt, x, src=src, src_div=4)
    ref = x[(src.long() // 4).clamp(0, 49)]
    ref[5:8] = 0
    _check_quantized(fmt, ref, codes, scales, 1.0)


@pytest.mark.parametrize("fmt", [moe.FP4_MX, moe.FP4_NV])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_quantize_swiglu(fmt, dtype):
    """silu(gate) * up is within 8 fp32 roundings of its fp64 value, then
    rounded to 16 bits: the values may differ where that crosses a boundary of
    the code grid, by one step of the grid."""
    rows, K = 37, 384
    x = _rand((rows, 2 * K), 3, dtype)
    codes, scales = _quantize(fmt, x, K=K, swiglu=True)
    v = x.double().reshape(rows, K // 128, 2, 128)
    h = (v[:, :, 0] * torch.sigmoid(v[:, :, 0]) * v[:, :, 1]).reshape(rows, K)
    h16 = h.to(dtype)
    out = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda")
    moe.moe_dequantize_fp4(fmt, codes, scales, out)
    _, byte, values = _quant_ref(h16.double().cpu().numpy(), fmt, 1.0)
    top = np.abs(h16.double().cpu().numpy()).reshape(rows, -1, BLOCK[fmt]).max(-1)
    step = np.repeat(top / 3, BLOCK[fmt], 1) * 1.1  # the widest gap of the grid, 4 to 6, of amax = 6
    got = out.double().cpu().numpy()
    assert (np.abs(got - values) <= step).all()
    assert (got != values).mean() < 1e-3
    assert (scales[:, :byte.shape[1]].cpu().numpy() != byte).mean() < 1e-3


def _fp4_operand(shape, seed, fmt):
    """Random codes and scales, their fp64 values."""
    g = _gen(seed)
    K = shape[-1]
    codes = torch.randint(0, 256, (*shape[:-1], K // 2), generator=g, device="cuda").to(torch.uint8)
    stride, nb = moe.moe_fp4_scale_stride(fmt, K), K // BLOCK[fmt]
    lo, hi = (118, 132) if fmt == moe.FP4_MX else (20, 100)
    # the padding may hold anything
    scales = torch.full((*shape[:-1], stride), 255, dtype=torch.uint8, device="cuda")
    scales[..., :nb] = torch.randint(lo, hi, (*shape[:-1], nb), generator=g, device="cuda").to(torch.uint8)
    lut = torch.from_numpy(np.concatenate([E2M1, -E2M1])).cuda()
    v = lut[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    s = scales[..., :nb]
    s = torch.exp2(s.double() - 127) if fmt == moe.FP4_MX else torch.from_numpy(E4M3).cuda()[s.int()]
    return codes, scales, (v.unflatten(-1, (nb, -1)) * s[..., None]).flatten(-2)


FP4_SHAPES = [  # sizes, N, K
    ([1], 8, 32),
    ([0, 1, 0, 2], 40, 96),
    ([3, 0, 17, 33], 136, 64),
    ([257, 31, 0, 511, 1], 264, 160),
    ([600, 256, 191, 193], 520, 1024),
    ([5] * 40 + [0] * 16 + [1] * 200, 96, 544),
    ([1000], 1032, 2080),
    ([150, 66], 256, 7168),
]


@pytest.mark.parametrize("fmt", [moe.FP4_MX, moe.FP4_NV])
@pytest.mark.parametrize("case", range(len(FP4_SHAPES)))
def test_product_fp4(fmt, case):
    sizes, N, K = FP4_SHAPES[case]
    offsets, off = _offsets(sizes, start=case)
    R, E = off[-1] + case, len(sizes)
    xq, xs, x = _fp4_operand((R, K), case, fmt)
    wq, ws, w = _fp4_operand((E, N, K), case + 30, fmt)
    gate = torch.rand((R,), generator=_gen(3), device="cuda") if case % 2 else None
    xg = torch.rand((1,), generator=_gen(4), device="cuda") if case % 3 else None
    wg = torch.rand((E,), generator=_gen(5), device="cuda") if case % 3 else None
    y = torch.full((R, N + 8), 7.0, dtype=torch.bfloat16, device="cuda")[:, :N]
    moe.moe_grouped_gemm_fp4(fmt, xq, xs, wq, ws, offsets, y, x_scale=xg, w_scale=wg, row_scale=gate)
    f = torch.ones((), device="cuda", dtype=torch.float64) if xg is None else xg.double()
    ref, mag = _product_ref(x * f, w if wg is None else w * wg.double()[:, None, None], off, False, gate)
    inside = slice(off[0], off[-1])
    _check(y[inside], ref[inside], mag[inside], K, torch.bfloat16, (sizes, N, K))
    assert (y[:off[0]] == 7).all() and (y[off[-1]:] == 7).all()


@pytest.mark.parametrize("fmt", [moe.FP4_MX, moe.FP4_NV])
def test_product_fp4_nan_scale_stays_in_its_row(fmt):
    offsets, off = _offsets([40, 41, 0])
    xq, xs, x = _fp4_operand((81, 160), 1, fmt)
    wq, ws, w = _fp4_operand((3, 48, 160), 2, fmt)
    nan = 255 if fmt == moe.FP4_MX else 127
    xs[13, 2] = nan
    xs[80, 4] = nan
    ws[2] = nan  # the empty group's weights
    ws[1, 7, 0] = nan
    y = torch.empty((81, 48), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm_fp4(fmt, xq, xs, wq, ws, offsets, y)
    bad = torch.zeros((81, 48), dtype=torch.bool, device="cuda")
    bad[13] = bad[80] = True
    bad[40:, 7] = True
    assert torch.equal(torch.isnan(y), bad)
    ref, mag = _product_ref(x, w, off, False)
    _check(y[~bad], ref[~bad], mag[~bad], 160, torch.bfloat16)


def test_product_fp4_flags_bad_offsets():
    status = torch.zeros(64, dtype=torch.int32, device="cuda")
    xq, xs, _ = _fp4_operand((64, 64), 1, moe.FP4_MX)
    wq, ws, _ = _fp4_operand((2, 64, 64), 2, moe.FP4_MX)
    y = torch.zeros((64, 64), dtype=torch.bfloat16, device="cuda")
    offsets = torch.tensor([0, 70, 64], dtype=torch.int32, device="cuda")
    moe.moe_grouped_gemm_fp4(moe.FP4_MX, xq, xs, wq, ws, offsets, y, status=status)
    assert moe.moe_get_device_status(status) == moe.DEVERR_SEGMENT
    assert (y == 0).all()
