"""CPU tests of the refusals of the routing by scores and of the 4-bit weights:
every check fails before anything is enqueued, and what the bindings check of
their tensors (on stand-ins, see test_binding_host.py)."""
import ctypes

import pytest
import torch

import routing_permute_grouped_gb300 as moe
from routing_permute_grouped_gb300 import build as moe_build
from tests.test_binding_host import BF, F32, I32, U8, Fake, lib as fake_lib  # noqa: F401

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
P = ctypes.c_void_p(0x1000)    # never dereferenced
ODD = ctypes.c_void_p(0x1008)  # not 16-byte aligned
ONE = ctypes.c_void_p(0x1001)


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.load()


def _rule(**kw):
    return moe.score_rule(**{**dict(E=16, k=4), **kw})


BAD_RULES = [
    (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(E=257), UNSUPPORTED), (dict(E=64, k=9), UNSUPPORTED),
    (dict(E=4, k=5), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(n_groups=-1), INVALID), (dict(n_groups=3, topk_groups=1), INVALID), (dict(E=66, n_groups=33, topk_groups=9), INVALID),
    (dict(n_groups=4, topk_groups=0), INVALID), (dict(n_groups=4, topk_groups=5), INVALID),
    (dict(n_groups=8, topk_groups=1), INVALID), (dict(n_groups=4, topk_groups=2, group_top=3), INVALID),
    (dict(n_groups=4, topk_groups=2, group_top=0), INVALID),
]


def _route(lib, rule, dtype=2, T=8, logits=P, ld=16, bias=None, idx=P, w=P, counts=None, losses=None, ws=None, ws_bytes=0):
    return lib.moe_route_scores(None if rule is None else ctypes.byref(rule), dtype, T, logits, ld, bias, idx, w, counts,
                                losses, ws, ws_bytes, None)


def _bwd(lib, rule, dtype=2, T=8, logits=P, ld=16, idx=P, dw=P, counts=None, dlosses=None, out=P, ldd=16):
    return lib.moe_route_scores_bwd(None if rule is None else ctypes.byref(rule), dtype, T, logits, ld, idx, dw, counts,
                                    dlosses, out, ldd, None)


@pytest.mark.parametrize("kw,status", BAD_RULES)
def test_rules(lib, kw, status):
    rule = _rule(**kw)
    assert _route(lib, rule, ld=300) == status and lib.moe_last_error()
    assert _bwd(lib, rule, ld=300, ldd=300) == status
    assert moe.moe_route_scores_workspace_size(rule, 8) == 0


def test_no_rule(lib):
    assert _route(lib, None) == INVALID and _bwd(lib, None) == INVALID
    bad = _rule()
    bad.score = 2
    assert _route(lib, bad) == INVALID
    with pytest.raises(ValueError):
        moe.score_rule(8, 2, "tanh")


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(T=-1), INVALID), (dict(T=(1 << 28) + 1), UNSUPPORTED),
    (dict(logits=None), INVALID), (dict(idx=None), INVALID), (dict(w=None), INVALID), (dict(ld=15), INVALID),
    (dict(logits=ONE), INVALID), (dict(logits=ctypes.c_void_p(0x1002)), INVALID), (dict(counts=P), INVALID),
    (dict(losses=P), INVALID), (dict(counts=P, losses=P), WORKSPACE), (dict(counts=P, losses=P, ws=P, ws_bytes=100), WORKSPACE),
    (dict(counts=P, losses=P, ws=ODD, ws_bytes=1 << 20), WORKSPACE),
])
def test_route_refuses(lib, kw, status):
    assert _route(lib, _rule(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), INVALID), (dict(T=-1), INVALID), (dict(logits=None), INVALID), (dict(out=None), INVALID),
    (dict(idx=None), INVALID), (dict(ld=15), INVALID), (dict(ldd=15), INVALID), (dict(out=ONE), INVALID),
    (dict(counts=P), INVALID), (dict(dlosses=P), INVALID),
])
def test_gradient_refuses(lib, kw, status):
    assert _bwd(lib, _rule(), **kw) == status


def test_without_tokens_nothing_is_read(lib):
    assert _route(lib, _rule(), T=0, logits=None, idx=None, w=None) == 0
    assert _bwd(lib, _rule(), T=0, logits=None, idx=None, dw=None, out=None) == 0


def test_workspace_size(lib):
    sizes = [moe.moe_route_scores_workspace_size(_rule(E=256, k=8), T) for T in (0, 1, 8, 9, 4096, 4097, 1 << 20)]
    assert sizes == sorted(sizes) and sizes[-1] == sizes[-2] == sizes[-3] and sizes[1] == sizes[2] < sizes[3]
    assert moe.moe_route_scores_workspace_size(_rule(), -1) == 0


QUANT = dict(group=64, dtype=0, rows=8, K=128, x=P, ldx=128, codes=P, scales=P, zeros=P, stream=None)


def _call(fn, base, kw):
    assert not set(kw) - set(base)
    return fn(*{**base, **kw}.values())


@pytest.mark.parametrize("kw,status", [
    (dict(group=16), UNSUPPORTED), (dict(group=0), UNSUPPORTED), (dict(dtype=2), INVALID), (dict(rows=-1), INVALID),
    (dict(rows=(1 << 30) + 1), UNSUPPORTED), (dict(K=0), INVALID), (dict(K=48), UNSUPPORTED), (dict(x=None), INVALID),
    (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(x=ODD), INVALID), (dict(codes=ODD), INVALID),
    (dict(scales=ONE), INVALID), (dict(ldx=120), INVALID), (dict(ldx=132), INVALID),
])
def test_quantize_refuses(lib, kw, status):
    assert _call(lib.moe_quantize_int4, QUANT, kw) == status


VALUES = dict(group=64, dtype=0, rows=8, K=128, codes=P, scales=P, zeros=None, out=P, ldo=128, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(group=256), UNSUPPORTED), (dict(dtype=7), INVALID), (dict(K=16), UNSUPPORTED), (dict(codes=None), INVALID),
    (dict(scales=None), INVALID), (dict(out=None), INVALID), (dict(out=ODD), INVALID), (dict(ldo=64), INVALID),
    (dict(ldo=130), INVALID), (dict(scales=ONE), INVALID),
])
def test_values_refuse(lib, kw, status):
    assert _call(lib.moe_dequantize_int4, VALUES, kw) == status


PRODUCT = dict(group=64, dtype=0, R=8, N=128, K=128, E=4, x=P, x_rows=8, ldx=128, src=None, div=1, codes=P, scales=P,
               zeros=None, off=P, gate=None, swiglu=0, y=P, ldy=128, status=None, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(group=100), UNSUPPORTED), (dict(dtype=2), INVALID), (dict(R=-1), INVALID), (dict(N=0), INVALID),
    (dict(K=0), INVALID), (dict(E=0), INVALID), (dict(K=72), UNSUPPORTED), (dict(N=60), UNSUPPORTED),
    (dict(N=64, swiglu=1), UNSUPPORTED), (dict(N=(1 << 29) + 8, ldy=1 << 30), UNSUPPORTED), (dict(E=257), UNSUPPORTED),
    (dict(R=(1 << 30) + 1), UNSUPPORTED), (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(off=None), INVALID), (dict(y=None), INVALID), (dict(x=ODD), INVALID), (dict(codes=ODD), INVALID),
    (dict(y=ODD), INVALID), (dict(scales=ONE), INVALID), (dict(ldx=120), INVALID), (dict(ldx=132), INVALID),
    (dict(ldy=120), INVALID), (dict(ldy=132), INVALID), (dict(x_rows=7), INVALID), (dict(src=P, div=0), INVALID),
    (dict(src=P, x_rows=0), INVALID), (dict(ldx=(1 << 30) + 8), UNSUPPORTED), (dict(ldy=(1 << 30) + 8), UNSUPPORTED),
])
def test_product_refuses(lib, kw, status):
    assert _call(lib.moe_grouped_gemm_int4, PRODUCT, kw) == status


def test_empty_calls_enqueue_nothing(lib):
    assert _call(lib.moe_quantize_int4, QUANT, dict(rows=0, x=None, codes=None, scales=None)) == 0
    assert _call(lib.moe_dequantize_int4, VALUES, dict(rows=0, codes=None, out=None)) == 0
    assert _call(lib.moe_grouped_gemm_int4, PRODUCT, dict(R=0, x=None, codes=None, y=None, off=None)) == 0


# ---------------------------------------------------- what the bindings check --
RULE = moe.score_rule(16, 4)
CALLS = {
    "moe_route_scores": (dict(logits=(BF, 8, 16), topk_idx=(I32, 8, 4), topk_w=(F32, 8, 4), bias=(F32, 16), counts=(I32, 16),
                              losses=(F32, 2), ws=(U8, 1 << 20)), dict(rule=RULE)),
    "moe_route_scores_bwd": (dict(logits=(F32, 8, 16), topk_idx=(I32, 8, 4), dlogits=(F32, 8, 16), dw=(F32, 8, 4),
                                  counts=(I32, 16), dlosses=(F32, 2)), dict(rule=RULE)),
    "moe_quantize_int4": (dict(x=(BF, 8, 96), codes=(U8, 8, 48), scales=(BF, 8, 2), zeros=(U8, 8, 2)), dict(group=64)),
    "moe_dequantize_int4": (dict(codes=(U8, 8, 48), scales=(BF, 8, 2), out=(BF, 8, 96), zeros=(U8, 8, 2)), dict(group=64)),
    "moe_grouped_gemm_int4": (dict(x=(BF, 8, 96), w_codes=(U8, 2, 72, 48), w_scales=(BF, 2, 72, 2), w_zeros=(U8, 2, 72, 2),
                                   offsets=(I32, 3), y=(BF, 6, 72), src=(I32, 6), row_scale=(F32, 6), status=(I32, 1)),
                              dict(group=64, src_div=1)),
}
EACH = [(name, arg) for name, (tensors, _) in CALLS.items() for arg in tensors]


def _bind(name, **other):
    tensors, rest = CALLS[name]
    args = {n: Fake(*v) for n, v in tensors.items()}
    args.update(other)
    getattr(moe, name)(**args, **rest)


@pytest.mark.parametrize("name", CALLS)
def test_calls_pass_on_the_current_device(fake_lib, name):  # noqa: F811
    _bind(name)
    assert [n for n, _ in fake_lib.calls] == [name] and fake_lib.calls[0][1][-1] == 0x70


@pytest.mark.parametrize("name,arg", EACH)
def test_other_tensors_are_refused(fake_lib, name, arg):  # noqa: F811
    dtype, *shape = CALLS[name][0][arg]
    bad = [Fake(dtype, *shape, device=1), Fake(dtype, *shape, device=-1)]
    if arg not in ("status", "ws"):
        bad += [Fake(torch.int64, *shape), Fake(torch.complex64, *shape)]
        if len(shape) > 1:
            bad += [Fake(dtype, *shape, strides=tuple(range(1, len(shape) + 1)))]
        if arg not in ("logits", "x", "out", "y", "dlogits", "w_codes"):
            bad += [Fake(dtype, *shape[:-1], shape[-1] + 1)]
    if arg == "ws":
        bad += [Fake(dtype, *shape, strides=(2,))]
    for t in bad:
        with pytest.raises(ValueError):
            _bind(name, **{arg: t})
    assert not fake_lib.calls


@pytest.mark.parametrize("name,arg,bad", [
    ("moe_route_scores", "logits", Fake(BF, 8, 17)), ("moe_route_scores", "logits", Fake(BF, 128)),
    ("moe_route_scores_bwd", "dlogits", Fake(BF, 8, 16)), ("moe_route_scores_bwd", "dlogits", Fake(F32, 7, 16)),
    ("moe_quantize_int4", "scales", Fake(torch.float16, 8, 2)), ("moe_dequantize_int4", "scales", Fake(torch.float16, 8, 2)),
    ("moe_grouped_gemm_int4", "y", Fake(BF, 6, 80)), ("moe_grouped_gemm_int4", "y", Fake(torch.float16, 6, 72)),
    ("moe_grouped_gemm_int4", "w_codes", Fake(U8, 3, 72, 48)), ("moe_grouped_gemm_int4", "w_scales", Fake(BF, 2, 72, 3)),
])
def test_shapes_that_do_not_go_together(fake_lib, name, arg, bad):  # noqa: F811
    with pytest.raises(ValueError):
        _bind(name, **{arg: bad})
    assert not fake_lib.calls


def test_groups_of_no_elements_are_refused(fake_lib):  # noqa: F811
    for group in (0, -32):
        with pytest.raises(ValueError):
            moe.moe_quantize_int4(group, Fake(BF, 8, 96), Fake(U8, 8, 48), Fake(BF, 8, 2))
    assert not fake_lib.calls


def test_scores_of_another_number_of_dimensions_are_refused():
    for shape in ((16,), (2, 3, 16)):
        with pytest.raises(ValueError, match="logits"):
            moe.route_scores(torch.zeros(shape), moe.score_rule(16, 2))
