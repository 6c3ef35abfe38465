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
