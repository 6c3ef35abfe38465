"""CPU tests of the refusals of the grouped products on ragged row groups and
of the 4-bit rows: every check fails before anything is enqueued."""
import ctypes

import pytest

import routing_permute_grouped_gb300 as moe
from routing_permute_grouped_gb300 import build as moe_build

INVALID, UNSUPPORTED = 1, 2
P = ctypes.c_void_p(0x1000)    # never dereferenced
ODD = ctypes.c_void_p(0x1008)  # not 16-byte aligned


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.load()


def _call(fn, order, base, kw):
    args = dict(base, **kw)
    assert not set(kw) - set(order.split())
    return fn(*[args[n] for n in order.split()])


PRODUCT = dict(dtype=0, R=64, N=64, K=64, E=4, x=P, ldx=64, w=P, wt=0, off=P, gate=None, y=P, ldy=64, status=None,
               stream=None)
BAD_PRODUCT = [
    (dict(dtype=2), INVALID), (dict(R=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID),
    (dict(E=0), INVALID), (dict(N=60), UNSUPPORTED), (dict(K=4), UNSUPPORTED), (dict(E=257), UNSUPPORTED),
    (dict(R=(1 << 30) + 1), UNSUPPORTED), (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID),
    (dict(off=None), INVALID), (dict(x=ODD), INVALID), (dict(w=ODD), INVALID), (dict(y=ODD), INVALID),
    (dict(ldx=56), INVALID), (dict(ldx=68), INVALID), (dict(ldy=56), INVALID), (dict(ldy=68), INVALID),
]


@pytest.mark.parametrize("kw,status", BAD_PRODUCT)
def test_product_refuses(lib, kw, status):
    assert _call(lib.moe_grouped_gemm, " ".join(PRODUCT), PRODUCT, kw) == status
    assert lib.moe_last_error()


def test_product_without_rows_reads_nothing(lib):
    kw = dict(R=0, x=None, w=None, y=None, off=None)
    assert _call(lib.moe_grouped_gemm, " ".join(PRODUCT), PRODUCT, kw) == 0


WGRAD = dict(dtype=0, R=64, M=64, N=64, E=4, a=P, lda=64, b=P, ldb=64, off=P, out=P, status=None, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=-1), INVALID), (dict(R=-1), INVALID), (dict(M=0), INVALID), (dict(M=12), UNSUPPORTED),
    (dict(N=12), UNSUPPORTED), (dict(E=300), UNSUPPORTED), (dict(a=None), INVALID), (dict(b=None), INVALID),
    (dict(off=None), INVALID), (dict(out=None), INVALID), (dict(a=ODD), INVALID), (dict(b=ODD), INVALID),
    (dict(out=ODD), INVALID), (dict(lda=60), INVALID), (dict(ldb=56), INVALID), (dict(R=0, out=None), INVALID),
])
def test_wgrad_refuses(lib, kw, status):
    assert _call(lib.moe_grouped_wgrad, " ".join(WGRAD), WGRAD, kw) == status


QUANT = dict(fmt=0, dtype=0, rows=8, K=128, x=P, x_rows=8, ldx=128, src=None, div=1, swiglu=0, g=None, codes=P,
             scales=P, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=2), INVALID), (dict(dtype=3), INVALID), (dict(rows=-1), INVALID), (dict(K=0), INVALID),
    (dict(K=40), UNSUPPORTED), (dict(K=96, swiglu=1), UNSUPPORTED), (dict(x=None), INVALID),
    (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(x=ODD), INVALID), (dict(codes=ODD), INVALID),
    (dict(scales=ODD), INVALID), (dict(ldx=120), INVALID), (dict(ldx=132), INVALID), (dict(swiglu=1), INVALID),
    (dict(x_rows=7), INVALID), (dict(src=P, div=0), INVALID), (dict(src=P, x_rows=0), INVALID),
])
def test_quantize_refuses(lib, kw, status):
    assert _call(lib.moe_quantize_fp4, " ".join(QUANT), QUANT, kw) == status


DEQUANT = dict(fmt=0, dtype=0, rows=8, K=128, codes=P, scales=P, g=None, out=P, ldo=128, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=-1), INVALID), (dict(dtype=2), INVALID), (dict(K=16), UNSUPPORTED), (dict(codes=None), INVALID),
    (dict(scales=None), INVALID), (dict(out=None), INVALID), (dict(out=ODD), INVALID), (dict(ldo=64), INVALID),
    (dict(ldo=130), INVALID),
])
def test_dequantize_refuses(lib, kw, status):
    assert _call(lib.moe_dequantize_fp4, " ".join(DEQUANT), DEQUANT, kw) == status


FP4 = dict(fmt=0, R=64, N=64, K=64, E=4, xq=P, xs=P, wq=P, ws=P, off=P, xg=None, wg=None, gate=None, y=P, ldy=64,
           status=None, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=2), INVALID), (dict(R=-1), INVALID), (dict(N=0), INVALID), (dict(E=0), INVALID),
    (dict(K=48), UNSUPPORTED), (dict(N=12), UNSUPPORTED), (dict(E=257), UNSUPPORTED), (dict(xq=None), INVALID),
    (dict(xs=None), INVALID), (dict(wq=None), INVALID), (dict(ws=None), INVALID), (dict(off=None), INVALID),
    (dict(y=None), INVALID), (dict(xq=ODD), INVALID), (dict(xs=ODD), INVALID), (dict(wq=ODD), INVALID),
    (dict(ws=ODD), INVALID), (dict(y=ODD), INVALID), (dict(ldy=56), INVALID), (dict(ldy=66), INVALID),
])
def test_product_fp4_refuses(lib, kw, status):
    assert _call(lib.moe_grouped_gemm_fp4, " ".join(FP4), FP4, kw) == status


def test_empty_calls_enqueue_nothing(lib):
    assert _call(lib.moe_quantize_fp4, " ".join(QUANT), QUANT, dict(rows=0, x=None, codes=None, scales=None)) == 0
    assert _call(lib.moe_dequantize_fp4, " ".join(DEQUANT), DEQUANT, dict(rows=0, codes=None, out=None)) == 0
    assert _call(lib.moe_grouped_gemm_fp4, " ".join(FP4), FP4, dict(R=0, xq=None, wq=None, y=None, off=None)) == 0


def test_scale_stride(lib):
    stride = moe.moe_fp4_scale_stride
    assert [stride(0, k) for k in (32, 512, 544, 7168)] == [16, 16, 32, 224]
    assert [stride(1, k) for k in (32, 256, 544, 7168)] == [16, 16, 48, 448]
    assert stride(0, 40) == 0 and stride(2, 64) == 0 and stride(1, 0) == 0
    for fmt in (-1, 0, 1, 2):
        for k in (-32, 0, 31, 32, 96, 160, 512, 544, 2080, 7168):
            assert stride(fmt, k) == lib.moe_fp4_scale_stride(fmt, k)


def _cfg(**kw):
    return moe.config_of(**{**dict(T=64, d=512, d_e=256, E=8, k=2), **kw})


W4 = dict(fmt=0, Wg_t=0x1000, W13q=0x1000, s13=0x1000, W2q=0x1000, s2=0x1000)


@pytest.mark.parametrize("cfg,weights,kw,status", [
    ({}, {}, dict(short=1), 3), ({}, dict(fmt=2), {}, INVALID), ({}, dict(s13=None), {}, INVALID),
    ({}, dict(W2q=None), {}, INVALID), ({}, dict(Wg_t=None), {}, INVALID), ({}, {}, dict(x=None), INVALID),
    ({}, {}, dict(out=None), INVALID), (dict(d_shared=128), {}, {}, INVALID), (dict(d=500), {}, {}, UNSUPPORTED),
    (dict(k=9, E=16), {}, {}, UNSUPPORTED), (dict(k=5, E=4), {}, {}, INVALID),
])
def test_layer_fp4_refuses(lib, cfg, weights, kw, status):
    c = _cfg(**cfg)
    w = moe.MoeWeightsFp4(**{**W4, **weights})
    need = moe.moe_workspace_size_fp4(c, 0)
    args = {**dict(x=P, out=P, ws=P), **kw}
    assert lib.moe_layer_fwd_fp4(ctypes.byref(c), ctypes.byref(w), args["x"], args["out"], args["ws"],
                                 need - kw.get("short", 0), None) == status
    assert lib.moe_last_error()


def test_layer_fp4_prerouted_refuses_and_empty_batch(lib):
    c, w = _cfg(), moe.MoeWeightsFp4(**W4)
    need = moe.moe_workspace_size_fp4(c, 0)
    pre = lib.moe_layer_fwd_fp4_prerouted
    assert pre(ctypes.byref(c), ctypes.byref(w), P, None, P, P, P, need, None) == INVALID
    assert pre(ctypes.byref(c), ctypes.byref(w), P, P, None, P, P, need, None) == INVALID
    none = _cfg(T=0)
    assert lib.moe_layer_fwd_fp4(ctypes.byref(none), ctypes.byref(w), None, None, P, need, None) == 0


def test_workspace_layout_fp4(lib):
    for fmt in (0, 1):
        c = _cfg(d_shared=128)
        L = moe.moe_workspace_layout_fp4(c, fmt)
        order = list(L)[1:]
        assert [L[n] for n in order] == sorted(L[n] for n in order) and all(L[n] % 1024 == 0 for n in order)
        assert L["total"] == moe.moe_workspace_size_fp4(c, fmt)
        assert L["xs"] - L["xq"] >= 128 * 256 and L["gu"] - L["xs"] >= 128 * moe.moe_fp4_scale_stride(fmt, 512)
    assert moe.moe_workspace_size_fp4(_cfg(), 2) == 0


def test_binding_refuses_what_c_cannot_see():
    import torch

    cpu = torch.zeros((4, 64), dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    w = torch.zeros((2, 64, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # host tensors
        moe.moe_grouped_gemm(cpu, w, off, cpu.clone())
    with pytest.raises(ValueError):  # another type of weights
        moe.moe_grouped_gemm(cpu, w.half(), off, cpu.clone())
    with pytest.raises(ValueError):  # offsets of another length
        moe.moe_grouped_gemm(cpu, w, off[:2], cpu.clone())
    with pytest.raises(ValueError):
        moe.moe_grouped_wgrad(cpu, cpu, off, torch.zeros((2, 64, 32), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        moe.moe_quantize_fp4(0, cpu, torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8))
