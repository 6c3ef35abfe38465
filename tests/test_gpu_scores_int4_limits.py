"""GPU tests of the score routing and the 4-bit product at their limits: the wide
tiles of the product (work of 2^30 products and more) over odd sizes, strides and
masks, offsets past 32 bits, alignments, and calls that run beside one another.
Bounds of the product as in test_gpu_int4; what is compared between two calls is
equal to the bit, as every token and every row is computed by itself."""
import pytest
import torch

import routing_permute_grouped_gb300 as moe
from tests import scores_ref
from tests.test_gpu_int4 import NAN, TYPES, _gen, _offsets, _product_check, _quantize, _rand, _weights

pytestmark = pytest.mark.gpu

WIDE = [  # sizes per group, N, K: sum of the sizes * N * K >= 2^30, more than 8 rows per group
    ([31, 32, 0, 64, 65], 1032, 5536), ([300], 1032, 3552), ([9, 17, 33, 49, 1, 0, 16, 48], 4104, 1568),
    ([129, 0, 1], 264, 40032), ([600, 257], 264, 5088), ([64], 1024, 16384), ([20] * 24 + [0] * 8, 8392, 288),
    ([9], 16384, 8192), ([8], 16384, 8192),  # either side of the rows that a narrow tile holds
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("case", range(len(WIDE)))
def test_wide_product(case, group, zeros, dtype):
    sizes, N, K = WIDE[case]
    assert sum(sizes) * N * K >= 2 ** 30
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


WIDE_SWIGLU = [([130, 5], 256, 16416), ([8, 17, 0, 40], 1152, 7200), ([70, 3, 90, 0, 0, 33], 1408, 2080)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("case", range(len(WIDE_SWIGLU)))
def test_wide_product_swiglu_gathered(case, group, zeros, dtype):
    sizes, N, K = WIDE_SWIGLU[case]
    offsets, off = _offsets(sizes)
    R, E, k = off[-1], len(sizes), 3
    assert R * 2 * N * K >= 2 ** 30 and R > 8 * E
    T = R // k + 1
    x = _rand((T, K), 1 + case, dtype)
    src = torch.randperm(T * k, generator=_gen(2), device="cuda")[:R].to(torch.int32)
    src[1], src[2], src[R - 1] = -1, T * k, -2 ** 31  # padding rows, and a token that does not exist
    src[3] = src[0]                                   # a token twice
    w = _weights(E, 2 * N, K, group, zeros, dtype, 100 + case)
    gate = torch.randn((R,), generator=_gen(7), device="cuda") if case % 2 else None
    y = torch.full((R, N), NAN, dtype=dtype, device="cuda")
    moe.moe_grouped_gemm_int4(group, x, w[0], w[1], offsets, y, w_zeros=w[2], src=src, src_div=k, row_scale=gate,
                              swiglu=True)
    _product_check(y, x, *w, group, off, src=src, div=k, gate=gate, swiglu=True)
    assert (y[1:3] == 0).all() and (y[R - 1] == 0).all()


def test_wide_product_strides_and_rows_outside_the_groups():
    sizes, N, K = [40, 0, 111, 52], 1032, 5344
    offsets, off = _offsets(sizes, start=3)
    R = off[-1] + 9
    for dtype in TYPES:
        xs = _rand((R, K + 40), 1, dtype)
        ys = torch.full((R, N + 24), 5.0, dtype=dtype, device="cuda")
        x, y = xs[:, 8:8 + K], ys[:, 16:16 + N]
        xs[:off[0]] = NAN  # what no group holds is not read into any
        xs[off[-1]:] = NAN
        w = _weights(4, N, K, 64, True, dtype, 8)
        moe.moe_grouped_gemm_int4(64, x, w[0], w[1], offsets, y, w_zeros=w[2])
        _product_check(y, x, *w, 64, off)
        assert (ys[:off[0]] == 5.0).all() and (ys[off[-1]:] == 5.0).all()
        assert (ys[:, :16] == 5.0).all() and (ys[:, 16 + N:] == 5.0).all()


@pytest.mark.parametrize("bad", [[-1, 40, 80, 120], [0, 40, 30, 120], [0, 40, 80, 990], [40, 0, 80, 120], [0, 120, 40, 80],
                                 [2 ** 31 - 1, -2 ** 31, 40, 80]])
def test_wide_product_skips_and_reports_groups_outside_the_rows(bad):
    R, N, K = 120, 1032, 8736
    x = _rand((R, K), 1)
    w = _weights(3, N, K, 128, False, torch.bfloat16, 8)
    y = torch.full((R, N), 5.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros((1,), dtype=torch.int32, device="cuda")
    moe.moe_grouped_gemm_int4(128, x, w[0], w[1], torch.tensor(bad, dtype=torch.int32, device="cuda"), y, status=status)
    assert status.item() == moe.DEVERR_SEGMENT
    end, inside = 0, torch.zeros(R, dtype=torch.bool, device="cuda")
    for e in range(3):
        lo, hi = bad[e], bad[e + 1]
        if lo < 0 or hi < lo or hi > R:
            continue
        lo = max(lo, end)  # no row is two groups'
        if lo < hi:
            _product_check(y[lo:hi], x[lo:hi], w[0][e:e + 1], w[1][e:e + 1], None, 128, [0, hi - lo])
            inside[lo:hi] = True
        end = max(end, hi)
    assert (y[~inside] == 5.0).all()


@pytest.mark.parametrize("sizes,N,K", [([2, 0, 9, 1], 264, 544), ([40, 0, 111, 52], 1032, 5344)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_parameters_at_any_alignment(sizes, N, K, group):
    offsets, off = _offsets(sizes)
    for dtype in TYPES:
        x = _rand((off[-1], K), 1, dtype)
        codes, scales, z = _weights(4, N, K, group, True, dtype, 8)
        want = torch.full((off[-1], N), NAN, dtype=dtype, device="cuda")
        moe.moe_grouped_gemm_int4(group, x, codes, scales, offsets, want, w_zeros=z)
        for so, zo in ((1, 0), (0, 1), (3, 3), (2, 2)):
            s2 = torch.empty((scales.numel() + 8,), dtype=dtype, device="cuda")[so:so + scales.numel()].view(scales.shape)
            z2 = torch.empty((z.numel() + 8,), dtype=torch.uint8, device="cuda")[zo:zo + z.numel()].view(z.shape)
            s2.copy_(scales)
            z2.copy_(z)
            y = torch.full((off[-1], N), NAN, dtype=dtype, device="cuda")
            moe.moe_grouped_gemm_int4(group, x, codes, s2, offsets, y, w_zeros=z2)
            _product_check(y, x, codes, scales, z, group, off)
            assert torch.equal(y, want)


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_and_scales_that_are_not_numbers(dtype):
    """A row's infinity or NaN stays in its row, a scale's in its column, in narrow and wide tiles."""
    for R, N, K in ((5, 72, 256), (100, 2056, 5248)):
        x = _rand((R, K), 1, dtype)
        codes, scales, z = _weights(1, N, K, 32, True, dtype, 8)
        scales[0, 3, 1] = NAN
        scales[0, 9, K // 32 - 1] = float("inf")
        x[1, 7], x[R - 1, K - 1] = float("inf"), NAN
        y = torch.zeros((R, N), dtype=dtype, device="cuda")
        moe.moe_grouped_gemm_int4(32, x, codes, scales, None, y, w_zeros=z)
        columns = [n for n in range(N) if n not in (3, 9)]
        assert torch.isnan(y[:, 3]).all() and not torch.isfinite(y[:, 9]).any()
        assert not torch.isfinite(y[1, columns]).any() and torch.isnan(y[R - 1, columns]).all()
        rows = [r for r in range(R) if r not in (1, R - 1)]
        assert torch.isfinite(y[rows][:, columns]).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept,top", [(256, 0, 0, 1), (256, 8, 4, 1), (256, 8, 4, 2), (60, 6, 3, 2), (64, 32, 9, 1),
                                               (256, 2, 1, 2)])
@pytest.mark.parametrize("bias_of", ["even", "odd", "large"])
def test_neighbours_at_the_last_place_of_the_choice(score, E, groups, kept, top, bias_of):
    """A stranger's logit one fp32 step from that of the last expert chosen, and a dropped group
    whose logits are the last kept one's but for one step: choices of fp64 among few experts."""
    T, k = 1500, 6
    rule = moe.score_rule(E, k, score, groups, kept, top)
    gen = torch.Generator().manual_seed(E + groups + top)
    logits = torch.randn((T, E), generator=gen) * 1.5
    bias = {"even": torch.full((E,), 0.25), "odd": (torch.randn((E,), generator=gen) * 3).round() / 64,
            "large": torch.where(torch.arange(E) % 3 == 0, 100.0, 100.25)}[bias_of]
    last = scores_ref.choose(logits.cuda(), rule, bias.cuda())[:, k - 1].long()
    t = torch.arange(T)
    up = torch.rand((T,), generator=gen) < 0.5
    step = torch.where(up, torch.inf, -torch.inf)
    if groups:  # every second token: another group like that of the last expert
        n = E // groups
        mine, other = last // n, torch.randint(0, groups, (T,), generator=gen)
        at = torch.arange(n)[None]
        copy = logits[t[:, None], mine[:, None] * n + at]
        big = copy.argmax(1)
        copy[t, big] = torch.nextafter(copy[t, big], step)
        rows = (t % 2 == 0) & (mine != other)
        logits[t[rows, None], (other[:, None] * n + at)[rows]] = copy[rows]
    odd = t % 2 == 1
    stranger = torch.randint(0, E, (T,), generator=gen)
    logits[t[odd], stranger[odd]] = torch.nextafter(logits[t, last], step)[odd]
    logits, bias = logits.cuda(), bias.cuda()
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), device="cuda")
    moe.moe_route_scores(rule, logits, idx, w, bias)
    assert torch.equal(idx.cpu(), scores_ref.choose(logits, rule, bias))


# ---------------------------------------------- calls beside one another --
def _calls():
    """Independent calls of every kernel: (run, outputs)."""
    made = []
    rule = moe.score_rule(64, 6, "sigmoid", 8, 3, 2)
    logits = torch.randn((5000, 64), generator=_gen(1), device="cuda")
    bias = torch.randn((64,), generator=_gen(2), device="cuda") * 0.01
    idx = torch.empty((5000, 6), dtype=torch.int32, device="cuda")
    w = torch.empty((5000, 6), device="cuda")
    counts = torch.empty((64,), dtype=torch.int32, device="cuda")
    losses = torch.empty((2,), device="cuda")
    ws = torch.empty((moe.moe_route_scores_workspace_size(rule, 5000),), dtype=torch.uint8, device="cuda")
    dlogits = torch.empty_like(logits)
    dl = torch.tensor([0.5, 0.25], device="cuda")

    def route():
        moe.moe_route_scores(rule, logits, idx, w, bias, counts, losses, ws)
        moe.moe_route_scores_bwd(rule, logits, idx, dlogits, dw=w, counts=counts, dlosses=dl)

    made.append((route, [idx, w, counts, losses, dlogits]))
    for seed, (sizes, N, K) in enumerate((([2, 0, 9, 1], 264, 4096), ([40, 0, 111, 52], 1032, 5344), ([64], 1024, 16384))):
        offsets, off = _offsets(sizes)
        x = _rand((off[-1], K), 10 + seed)
        q = _weights(len(sizes), N, K, 128, True, torch.bfloat16, 20 + seed)
        y = torch.empty((off[-1], N), dtype=torch.bfloat16, device="cuda")

        def product(x=x, q=q, offsets=offsets, y=y):
            moe.moe_grouped_gemm_int4(128, x, q[0], q[1], offsets, y, w_zeros=q[2])

        made.append((product, [y]))
    v = _rand((3000, 416), 30)
    codes, scales, z = _quantize(64, v, True)
    back = torch.empty_like(v)

    def pack():
        moe.moe_quantize_int4(64, v, codes, scales, zeros=z)
        moe.moe_dequantize_int4(64, codes, scales, back, zeros=z)

    made.append((pack, [codes, scales, z, back]))
    return made


def _wipe(made):
    for _, outs in made:
        for t in outs:
            t.view(torch.uint8).fill_(0xA5)


def test_calls_on_streams_of_their_own_and_two_graphs():
    made = _calls()
    for run, _ in made:
        run()
    torch.cuda.synchronize()
    want = [[t.clone() for t in outs] for _, outs in made]

    def same():
        torch.cuda.synchronize()
        for (_, outs), ts in zip(made, want):
            for got, t in zip(outs, ts):
                assert torch.equal(got.view(torch.uint8), t.view(torch.uint8))

    streams = [torch.cuda.Stream() for _ in made]
    _wipe(made)
    torch.cuda.synchronize()
    for _ in range(5):
        for (run, _), s in zip(made, streams):
            with torch.cuda.stream(s):
                run()
    same()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]  # the kernels in two graphs, replayed at once
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            for run, _ in made[i::2]:
                run()
    _wipe(made)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    same()


def test_forward_and_backward_captured_together():
    rule = moe.score_rule(64, 6, "sigmoid", 8, 4, 2)
    bias = torch.randn((64,), generator=_gen(2), device="cuda") * 0.01
    x = torch.randn((500, 64), generator=_gen(3), device="cuda")
    g = torch.randn((500, 6), generator=_gen(4), device="cuda")

    def loss(leaf):
        w, _, both, _ = moe.route_scores(leaf, rule, bias, losses=True)
        return (w * g).sum() + both[0] + 0.1 * both[1]

    leaf = x.clone().requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        loss(leaf).backward()
    torch.cuda.current_stream().wait_stream(side)
    leaf.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss(leaf).backward()
    for seed in (5, 6):
        new = torch.randn((500, 64), generator=_gen(seed), device="cuda")
        with torch.no_grad():
            leaf.copy_(new)
        graph.replay()
        other = new.clone().requires_grad_()
        loss(other).backward()
        assert torch.equal(leaf.grad, other.grad)


# -------------------------------------------------- offsets past 32 bits --
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_routing_of_more_than_2_31_logits(score):
    T, E, k, last = 2 ** 23 + 77, 256, 8, 1000
    rule = moe.score_rule(E, k, score, 8, 4, 2)
    logits = torch.randn((T, E), generator=_gen(1), device="cuda", dtype=torch.bfloat16)
    bias = torch.randn((E,), generator=_gen(2), device="cuda") * 0.01
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), device="cuda")
    counts = torch.empty((E,), dtype=torch.int32, device="cuda")
    losses = torch.empty((2,), device="cuda")
    ws = torch.empty((moe.moe_route_scores_workspace_size(rule, T),), dtype=torch.uint8, device="cuda")
    moe.moe_route_scores(rule, logits, idx, w, bias, counts, losses, ws)
    assert torch.equal(counts.long(), torch.bincount(idx.flatten(), minlength=E))
    dlogits = torch.empty_like(logits)
    moe.moe_route_scores_bwd(rule, logits, idx, dlogits, dw=w)
    for rows in (slice(T - last, T), slice(0, last)):
        part = logits[rows].clone()
        idx1, w1, d1 = torch.empty_like(idx[rows]), torch.empty_like(w[rows]), torch.empty_like(part)
        moe.moe_route_scores(rule, part, idx1, w1, bias)
        moe.moe_route_scores_bwd(rule, part, idx1, d1, dw=w1)
        assert torch.equal(idx[rows], idx1) and torch.equal(w[rows], w1) and torch.equal(dlogits[rows], d1)


def test_quantising_more_than_2_31_elements():
    rows, K, last = 2 ** 20 + 3, 2080, 100
    x = torch.randn((rows, K), generator=_gen(1), device="cuda", dtype=torch.bfloat16)
    codes, scales, z = _quantize(128, x, True)
    part = _quantize(128, x[-last:].clone(), True)
    assert all(torch.equal(a[-last:], b) for a, b in zip((codes, scales, z), part))
    out = torch.empty_like(x)
    moe.moe_dequantize_int4(128, codes, scales, out, zeros=z)
    back = torch.empty((last, K), dtype=x.dtype, device="cuda")
    moe.moe_dequantize_int4(128, *part[:2], back, zeros=part[2])
    assert torch.equal(out[-last:], back)


@pytest.mark.parametrize("sizes", [[1, 1], [3, 40]])
def test_product_of_operands_past_2_32_bytes(sizes):
    """Codes past 2^32 bytes, token rows and results past 2^31 elements; narrow and wide tiles."""
    N, K, pitch, tokens = 80000, 65536, 2 ** 26 + 8, 40000
    offsets, off = _offsets(sizes)
    R = off[-1]
    codes = torch.randint(0, 256, (2, N, K // 2), generator=_gen(1), device="cuda", dtype=torch.uint8)
    scales = ((torch.rand((2, N, K // 128), generator=_gen(2), device="cuda") + 0.25) / 1024).bfloat16()
    x = torch.empty((tokens, K), dtype=torch.bfloat16, device="cuda")
    x[-R:] = _rand((R, K), 3)
    src = torch.arange(tokens - R, tokens, dtype=torch.int32, device="cuda").flip(0).contiguous()
    y = torch.empty(((R - 1) * pitch + N,), dtype=torch.bfloat16, device="cuda").as_strided((R, N), (pitch, 1))
    moe.moe_grouped_gemm_int4(128, x, codes, scales, offsets, y, src=src)
    rows = x[src.long()]
    for cols in (slice(0, 136), slice(N - 136, N)):
        _product_check(y[:, cols], rows, codes[:, cols].contiguous(), scales[:, cols].contiguous(), None, 128, off)


def test_smallest_calls_and_an_index_that_repeats():
    rule = moe.score_rule(1, 1, "softmax")
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        logits = torch.tensor([[0.5]], dtype=dtype, device="cuda")
        idx = torch.full((1, 1), 9, dtype=torch.int32, device="cuda")
        w = torch.full((1, 1), NAN, device="cuda")
        moe.moe_route_scores(rule, logits, idx, w)
        assert idx.item() == 0 and w.item() == 1.0
    for dtype in TYPES:
        x = torch.ones((1, 32), dtype=dtype, device="cuda")
        codes, scales, z = _quantize(32, x, True)
        y = torch.full((1, 8), NAN, dtype=dtype, device="cuda")
        moe.moe_grouped_gemm_int4(32, x, codes.expand(1, 8, 16).contiguous(), scales.expand(1, 8, 1).contiguous(), None, y,
                                  w_zeros=z.expand(1, 8, 1).contiguous())
        # 32 codes of 15 with the scale 1 / 15, rounded to the type
        assert torch.equal(y, (480 * scales.double()).to(dtype).expand(1, 8))
