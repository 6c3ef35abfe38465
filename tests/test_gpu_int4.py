"""GPU tests of the 4-bit weights (quantiser and values) and of their product
with 16-bit rows, against plain fp64 arithmetic.

Bounds.  Codes, zero points and scales are fixed by the inputs: the integer next
to a quotient of 16-bit numbers is that of the exact quotient.  Values are exact
products rounded once.  In the product, code - zero times a row's element is
exact; a group's sum of at most 128 of them is off by 128 * 2^-23 * S_g in any
order and with truncating adders, S_g the sum of their magnitudes; scaled (2^-24)
and summed over G groups, with the parts of a split sum among them, the result is
off by (128 + G + 16) * 2^-23 * S; up to two fp32 factors and one rounding to the
output type (half a step) follow.  silu(g) has a slope of at most 1.1."""
import pytest
import torch

import routing_permute_grouped_gb300 as moe

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: (2.0 ** -8, 2.0 ** -134), torch.float16: (2.0 ** -11, 2.0 ** -25)}
TYPES = [torch.bfloat16, torch.float16]
NAN = float("nan")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rand(shape, seed, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(shape, generator=_gen(seed), device="cuda") * std).to(dtype)


def _quantize(group, x, zeros):
    rows, K = x.shape
    n = -(-K // group)
    codes = torch.full((rows, K // 2), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, n), NAN, dtype=x.dtype, device="cuda")
    z = torch.full((rows, n), 77, dtype=torch.uint8, device="cuda") if zeros else None
    moe.moe_quantize_int4(group, x, codes, scales, zeros=z)
    return codes, scales, z


def _unpack(codes):
    """Element 2 i of a word in bits 4 i, element 2 i + 1 in bits 16 + 4 i."""
    word = codes.contiguous().view(torch.int32)
    at = [4 * (e // 2) + 16 * (e % 2) for e in range(8)]
    return torch.stack([(word >> s) & 15 for s in at], -1).flatten(-2)


def _per_element(t, group, K):
    return t.repeat_interleave(group, -1)[..., :K]


def _values(codes, scales, zeros, group):
    q = _unpack(codes).double()
    K = q.shape[-1]
    q = q - (8 if zeros is None else _per_element(zeros, group, K).double())
    return q * _per_element(scales, group, K).double()


def _codes_ref(x, group, zeros):
    K = x.shape[1]
    v = x.double()
    code, scale, zero = torch.zeros_like(v), [], []
    for lo in range(0, K, group):
        part = v[:, lo:lo + group]
        if zeros:
            top, low = part.amax(1).clamp(min=0), part.amin(1).clamp(max=0)
            s = ((top - low) / 15).to(x.dtype).double()
            z = torch.where(s > 0, (-low / s).round().clamp(0, 15), 0.0)
        else:
            s = (part.abs().amax(1) / 7).to(x.dtype).double()
            z = torch.full_like(s, 8.0)
        q = torch.where(s[:, None] > 0, (part / s[:, None]).round(), 0.0)
        q = (q + z[:, None]).clamp(0, 15)
        code[:, lo:lo + group] = q
        scale.append(s)
        zero.append(z)
    return code, torch.stack(scale, 1), torch.stack(zero, 1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (5, 96), (37, 160), (300, 256), (9, 1000 // 32 * 32), (17, 7168),
                                    (2, 40032)])
def test_quantize(rows, K, group, zeros, dtype):
    x = _rand((rows, K), rows + K, dtype, 0.02)
    x[0] = 0
    if rows > 2:
        x[1] = x[1].abs()       # one-sided groups
        x[2] = -x[2].abs()
        x[2, K // 2] = 30.0
    codes, scales, z = _quantize(group, x, zeros)
    code, scale, zero = _codes_ref(x, group, zeros)
    assert torch.equal(scales.double(), scale)
    if zeros:
        assert torch.equal(z.double(), zero)
    assert torch.equal(_unpack(codes).double(), code)
    out = torch.full((rows, K), NAN, dtype=dtype, device="cuda")
    moe.moe_dequantize_int4(group, codes, scales, out, zeros=z)
    assert torch.equal(out, _values(codes, scales, z, group).to(dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("zeros", [False, True])
def test_quantize_ties_and_extremes(dtype, zeros):
    """Quotients that are half integers, the ends of the type's range, subnormal scales."""
    K, group = 64, 32
    big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    half = torch.arange(-15, 16, device="cuda").double() / 2  # 0.5 steps around a scale of 1
    rows = []
    for unit in (1.0, 2.0 ** -9, 1.5, 2.0 ** -3 * 1.75, tiny, tiny / 32):
        r = torch.zeros(K, dtype=torch.float64, device="cuda")
        r[:31] = half.clamp(-7, 7) * unit
        r[32:63] = half.clamp(-3.5, 7) * unit
        r[31] = 7 * unit
        r[63] = -8 * unit
        rows.append(r)
    x = torch.stack(rows).to(dtype)
    x = torch.cat([x, torch.tensor([[big, -big] * 32, [big] * 64, [-big] * 64, [tiny] * 64, [-tiny, 0.0] * 32],
                                   dtype=dtype, device="cuda")])
    codes, scales, z = _quantize(group, x, zeros)
    code, scale, zero = _codes_ref(x, group, zeros)
    assert torch.equal(scales.double(), scale)
    if zeros:
        assert torch.equal(z.double(), zero)
    assert torch.equal(_unpack(codes).double(), code)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("zeros", [False, True])
def test_quantize_marks_what_is_not_a_number(dtype, zeros):
    x = _rand((4, 256), 1, dtype)
    x[0, 5], x[1, 70], x[2, 200] = NAN, float("inf"), -float("inf")
    for group in (32, 64, 128):
        codes, scales, z = _quantize(group, x, zeros)
        bad = torch.zeros_like(scales, dtype=torch.bool)
        bad[0, 5 // group] = bad[1, 70 // group] = bad[2, 200 // group] = True
        assert torch.equal(torch.isnan(scales), bad)
        out = torch.zeros_like(x)
        moe.moe_dequantize_int4(group, codes, scales, out, zeros=z)
        assert torch.equal(torch.isnan(out), _per_element(bad, group, 256))


def test_quantize_strides():
    for dtype in TYPES:
        wide = _rand((20, 512), 3, dtype)
        view = wide[:, 64:224]
        a, b = _quantize(32, view, True), _quantize(32, view.contiguous(), True)
        assert all(torch.equal(u, v) for u, v in zip(a, b))
        out = torch.full((20, 512), 3.0, dtype=dtype, device="cuda")
        moe.moe_dequantize_int4(32, *a[:2], out[:, 8:168], zeros=a[2])
        assert torch.equal(out[:, 8:168], _values(*a, 32).to(dtype))
        out[:, 8:168] = 3.0
        assert (out == 3.0).all()


# ---------------------------------------------------------------- product --
def _weights(E, rows, K, group, zeros, dtype, seed):
    """Codes, scales, zero points, and the values in fp64."""
    gen = _gen(seed)
    n = -(-K // group)
    codes = torch.randint(0, 256, (E, rows, K // 2), generator=gen, device="cuda").to(torch.uint8)
    scales = ((torch.rand((E, rows, n), generator=gen, device="cuda") + 0.25) * K ** -0.5 / 4).to(dtype)
    z = torch.randint(0, 16, (E, rows, n), generator=gen, device="cuda").to(torch.uint8) if zeros else None
    return codes, scales, z


def _silu(g):
    return g / (1 + torch.exp(-g))


def _product_check(y, x, codes, scales, z, group, off, src=None, div=1, gate=None, swiglu=False):
    dtype, K, G = x.dtype, x.shape[1], scales.shape[2]
    rel, tiny = HALF[dtype]
    E, N = codes.shape[0], y.shape[1]
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if hi <= lo:
            continue
        if src is None:
            xe = x[lo:hi].double()
        else:
            s = src[lo:hi].long()
            ok = (s >= 0) & (s // div < x.shape[0])
            xe = x[(s // div).clamp(0, x.shape[0] - 1)].double() * ok[:, None]
        w = _values(codes[e], scales[e], None if z is None else z[e], group)
        v, mag = xe @ w.T, xe.abs() @ w.abs().T
        acc = (128 + G + 16) * 2.0 ** -23 * mag
        if swiglu:
            v, acc = (t.unflatten(1, (-1, 2, 128)) for t in (v, acc))
            g, u = v[:, :, 0].flatten(1), v[:, :, 1].flatten(1)
            ag, au = acc[:, :, 0].flatten(1), acc[:, :, 1].flatten(1)
            v = _silu(g) * u
            # exp's argument, the quotient and the product add 2^-22 (|g| + 4) of the value
            acc = (1.1 * ag) * (u.abs() + au) + _silu(g).abs() * au + 2.0 ** -22 * (g.abs() + 4) * v.abs()
        if gate is not None:
            f = gate[lo:hi, None].double()
            v, acc = v * f, acc * f.abs()
        acc = acc + 2.0 ** -22 * v.abs()
        bound = acc + rel * (v.abs() + acc) + tiny
        got = y[lo:hi]
        assert torch.isfinite(got).all(), e
        worst = ((got.double() - v).abs() - bound).max().item()
        assert worst <= 0, (e, hi - lo, worst)


def _offsets(sizes, start=0):
    off = [start]
    for s in sizes:
        off.append(off[-1] + s)
    return torch.tensor(off, dtype=torch.int32, device="cuda"), off


CASES = [  # sizes per group, N, K
    ([1], 8, 32), ([0, 1, 0, 2], 40, 96), ([3, 0, 17, 33], 136, 64), ([8, 9, 7, 16, 15], 64, 160), ([1] * 8, 264, 7168),
    ([5] * 40 + [0] * 16 + [1] * 200, 96, 128), ([31, 32, 0, 64, 65], 72, 992), ([300], 1032, 544), ([2, 4], 4096, 2048),
    ([129, 0, 1], 8, 40032), ([600, 257], 264, 352),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_product(case, group, zeros, dtype):
    sizes, N, K = CASES[case]
    offsets, off = _offsets(sizes)
    R, E = off[-1], len(sizes)
    x = _rand((R, K), 1 + case, dtype)
    w = _weights(E, N, K, group, zeros, dtype, 100 + case)
    gate = torch.rand((R,), generator=_gen(7), device="cuda") if case % 2 else None
    y = torch.full((R, N), NAN, dtype=dtype, device="cuda")
    moe.moe_grouped_gemm_int4(group, x, w[0], w[1], offsets, y, w_zeros=w[2], row_scale=gate)
    _product_check(y, x, *w, group, off, gate=gate)
    again = torch.full((R, N), NAN, dtype=dtype, device="cuda")
    moe.moe_grouped_gemm_int4(group, x, w[0], w[1], offsets, again, w_zeros=w[2], row_scale=gate)
    assert torch.equal(y, again)


SWIGLU = [([1], 128, 32), ([0, 3, 1], 128, 416), ([8, 17, 0, 40], 384, 256), ([1] * 8, 2048, 1024), ([130, 5], 256, 7168)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("case", range(len(SWIGLU)))
def test_product_swiglu_gathered(case, group, zeros, dtype):
    sizes, N, K = SWIGLU[case]
    offsets, off = _offsets(sizes)
    R, E, k = off[-1], len(sizes), 3
    T = R // k + 1
    x = _rand((T, K), 1 + case, dtype)
    src = torch.randperm(T * k, generator=_gen(2), device="cuda")[:R].to(torch.int32)
    if R > 3:
        src[1], src[2] = -1, T * k  # a padding row, and a token that does not exist
    w = _weights(E, 2 * N, K, group, zeros, dtype, 100 + case)
    gate = torch.randn((R,), generator=_gen(7), device="cuda") if case % 2 else None
    y = torch.full((R, N), NAN, dtype=dtype, device="cuda")
    moe.moe_grouped_gemm_int4(group, x, w[0], w[1], offsets, y, w_zeros=w[2], src=src, src_div=k, row_scale=gate,
                              swiglu=True)
    _product_check(y, x, *w, group, off, src=src, div=k, gate=gate, swiglu=True)
    if R > 3:
        assert (y[1:3] == 0).all()


def test_one_dense_group_without_offsets():
    for dtype in TYPES:
        for R, N, K in ((1, 1024, 4096), (5, 264, 480), (40, 128, 7168)):
            x = _rand((R, K), 5, dtype)
            w = _weights(1, N, K, 128, True, dtype, 6)
            y = torch.full((R, N), NAN, dtype=dtype, device="cuda")
            moe.moe_grouped_gemm_int4(128, x, w[0], w[1], None, y, w_zeros=w[2])
            _product_check(y, x, *w, 128, [0, R])


def test_product_strides_and_rows_outside_the_groups():
    sizes, N, K = [4, 0, 11, 2], 72, 224
    offsets, off = _offsets(sizes, start=3)
    R = off[-1] + 9
    for dtype in TYPES:
        xs = _rand((R, K + 40), 1, dtype)
        x = xs[:, 8:8 + K]
        ys = torch.full((R, N + 24), 5.0, dtype=dtype, device="cuda")
        y = ys[:, 16:16 + N]
        w = _weights(4, N, K, 64, True, dtype, 8)
        moe.moe_grouped_gemm_int4(64, x, w[0], w[1], offsets, y, w_zeros=w[2])
        _product_check(y, x, *w, 64, off)
        assert (ys[:off[0]] == 5.0).all() and (ys[off[-1]:] == 5.0).all()
        assert (ys[:, :16] == 5.0).all() and (ys[:, 16 + N:] == 5.0).all()


@pytest.mark.parametrize("bad", [[-1, 4, 8, 12], [0, 4, 3, 12], [0, 4, 8, 99], [4, 0, 8, 12], [0, 8, 4, 12], [99, 4, 8, 12],
                                 [0, 12, 4, 8], [2 ** 31 - 1, -2 ** 31, 4, 8]])
def test_groups_outside_the_rows_are_skipped_and_reported(bad):
    R, N, K = 12, 64, 64
    offsets = torch.tensor(bad, dtype=torch.int32, device="cuda")
    x = _rand((R, K), 1)
    w = _weights(3, N, K, 32, False, torch.bfloat16, 8)
    y = torch.full((R, N), 5.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros((1,), dtype=torch.int32, device="cuda")
    moe.moe_grouped_gemm_int4(32, x, w[0], w[1], offsets, y, status=status)
    assert status.item() == moe.DEVERR_SEGMENT
    end, off = 0, [0]
    for e in range(3):
        lo, hi = bad[e], bad[e + 1]
        if lo < 0 or hi < lo or hi > R:
            continue
        lo = max(lo, end)  # no row is two groups'
        if lo < hi:
            _product_check(y[lo:hi], x[lo:hi], w[0][e:e + 1], w[1][e:e + 1], None, 32, [0, hi - lo])
            off.append((lo, hi))
        end = max(end, hi)
    inside = torch.zeros(R, dtype=torch.bool, device="cuda")
    for lo, hi in off[1:]:
        inside[lo:hi] = True
    assert (y[~inside] == 5.0).all()


def test_scales_that_are_not_numbers_and_infinite_rows():
    x = _rand((3, 64), 1)
    w = _weights(1, 16, 64, 32, True, torch.bfloat16, 8)
    w[1][0, 3, 1] = NAN
    x[1, 7] = float("inf")
    y = torch.zeros((3, 16), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm_int4(32, x, w[0], w[1], None, y, w_zeros=w[2])
    assert torch.isnan(y[:, 3]).all()
    keep = [n for n in range(16) if n != 3]
    assert not torch.isfinite(y[1, keep]).any()  # inf, or NaN where its code is the zero point
    ok = torch.isfinite(y)
    assert ok[0][keep].all() and ok[2][keep].all()


def test_captured_and_on_another_stream():
    sizes, N, K = [2, 0, 9, 1], 256, 512
    offsets, off = _offsets(sizes)
    x = _rand((12, K), 1)
    w = _weights(4, 2 * N, K, 128, True, torch.bfloat16, 8)
    y = torch.full((12, N), NAN, dtype=torch.bfloat16, device="cuda")

    def step():
        moe.moe_grouped_gemm_int4(128, x, w[0], w[1], offsets, y, w_zeros=w[2], swiglu=True)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for sizes in ([12, 0, 0, 0], [0, 5, 5, 2], [3, 3, 3, 3]):
        offsets.copy_(_offsets(sizes)[0])
        x.copy_(_rand((12, K), sum(sizes[:2])))
        y.fill_(NAN)
        graph.replay()
        got = y.clone()
        _product_check(got, x, *w, 128, _offsets(sizes)[1], swiglu=True)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            y.fill_(NAN)
            step()
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, y)


def test_no_rows():
    w = _weights(2, 16, 64, 32, True, torch.bfloat16, 8)
    empty = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    offsets = torch.zeros((3,), dtype=torch.int32, device="cuda")
    moe.moe_grouped_gemm_int4(32, empty, w[0], w[1], offsets, empty[:, :16])
    moe.moe_quantize_int4(32, empty, torch.empty((0, 32), dtype=torch.uint8, device="cuda"), empty[:, :2].contiguous())
    # rows, but in no group
    y = torch.full((4, 16), 5.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm_int4(32, _rand((4, 64), 1), w[0], w[1], offsets, y)
    assert (y == 5.0).all()


# -------------------------------------------- the operators as they are used --
@pytest.mark.parametrize("T,d,de,E,k", [(1, 256, 128, 16, 4), (13, 512, 256, 8, 2), (200, 256, 384, 24, 3)])
def test_a_layer_of_these_operators(T, d, de, E, k):
    """Scores to experts to offsets to 4-bit gate/up, down and combine, against the same steps in fp64."""
    from tests import scores_ref

    dtype = torch.bfloat16
    x = _rand((T, d), 1)
    wg = _rand((d, E), 2, torch.float32, d ** -0.5)
    bias = (torch.randn((E,), generator=_gen(3), device="cuda") * 50).round() / 1000
    w13 = _rand((E, 2 * de, d), 4, dtype, d ** -0.5)
    w2 = _rand((E, d, de), 5, dtype, de ** -0.5)

    def pack(w):
        rows, K = w.shape[0] * w.shape[1], w.shape[2]
        return [None if t is None else t.view(w.shape[0], w.shape[1], -1) for t in _quantize(128, w.view(rows, K), True)]

    q13, q2 = pack(w13), pack(w2)
    rule = moe.score_rule(E, k, "sigmoid", 4, 2, 2, scale=2.5)
    logits = x.float() @ wg
    topk_w, topk_idx = moe.route_scores(logits, rule, bias)
    assert torch.equal(topk_idx.cpu(), scores_ref.choose(logits, rule, bias))
    cfg = moe.config_of(T=T, d=d, d_e=de, E=E, k=k)
    A, i32 = T * k, dict(dtype=torch.int32, device="cuda")
    counts, offsets, perm, src = (torch.empty(n, **i32) for n in (E, E + 1, A, A))
    gate = torch.empty((A,), device="cuda")
    ws = torch.zeros(moe.moe_offsets_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    moe.moe_build_offsets_unpadded(cfg, topk_idx, topk_w, counts, offsets, perm, src, gate, ws)
    h = torch.empty((A, de), dtype=dtype, device="cuda")
    moe.moe_grouped_gemm_int4(128, x, q13[0], q13[1], offsets, h, w_zeros=q13[2], src=src, src_div=k, swiglu=True)
    off = offsets.tolist()
    _product_check(h, x, *q13, 128, off, src=src, div=k, swiglu=True)
    y = torch.empty((A, d), dtype=dtype, device="cuda")
    moe.moe_grouped_gemm_int4(128, h, q2[0], q2[1], offsets, y, w_zeros=q2[2], row_scale=gate)
    _product_check(y, h, *q2, 128, off, gate=gate)
    out = torch.empty((T, d), dtype=dtype, device="cuda")
    moe.moe_combine(cfg, y, perm, None, out)
    want = y.double()[perm.long()].view(T, k, d).sum(1)
    mag = y.double().abs()[perm.long()].view(T, k, d).sum(1)
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + 9 * 2.0 ** -24 * mag * 1.01).all()
