"""CPU tests of the largest dimensions of the grouped products and of the 4-bit
rows: 2^30, so that the kernels' 32-bit index arithmetic has room; larger ones are
refused before anything is enqueued, in C and in the bindings (whose C arguments
are 32 bits wide)."""
import pytest
import torch

import routing_permute_grouped_gb300 as moe
from tests.test_binding_host import BF, CALLS, U8, Fake, lib  # noqa: F401
from tests.test_ragged_host import DEQUANT, FP4, PRODUCT, QUANT, UNSUPPORTED, WGRAD, _call
from tests.test_ragged_host import lib as library  # noqa: F401

MOST = 1 << 30


@pytest.mark.parametrize("fn,base,kw", [
    ("moe_grouped_gemm", PRODUCT, dict(N=MOST + 8, ldy=MOST + 8)),
    ("moe_grouped_gemm", PRODUCT, dict(K=MOST + 8, ldx=MOST + 8)),
    ("moe_grouped_gemm", PRODUCT, dict(K=2 ** 31 - 8, ldx=2 ** 31)),
    ("moe_grouped_wgrad", WGRAD, dict(M=MOST + 8, lda=MOST + 8)),
    ("moe_grouped_wgrad", WGRAD, dict(N=MOST + 8, ldb=MOST + 8)),
    ("moe_quantize_fp4", QUANT, dict(K=MOST + 32, ldx=MOST + 32)),
    ("moe_dequantize_fp4", DEQUANT, dict(K=MOST + 32, ldo=MOST + 32)),
    ("moe_grouped_gemm_fp4", FP4, dict(K=MOST + 32)),
    ("moe_grouped_gemm_fp4", FP4, dict(N=MOST + 8, ldy=MOST + 8)),
])
def test_larger_dimensions_are_refused(library, fn, base, kw):  # noqa: F811
    assert _call(getattr(library, fn), " ".join(base), base, kw) == UNSUPPORTED
    assert b"2^30" in library.moe_last_error()


WRAP = (1 << 32) + 64  # 64 in 32 bits


@pytest.mark.parametrize("name,tensors", [
    ("moe_grouped_gemm", dict(x=(BF, 8, WRAP), w=(BF, 2, 72, WRAP))),
    ("moe_grouped_gemm", dict(w=(BF, 2, WRAP, 64), y=(BF, 8, WRAP))),
    ("moe_grouped_wgrad", dict(a=(BF, 8, WRAP), out=(BF, 2, WRAP, 64))),
    ("moe_grouped_wgrad", dict(b=(BF, 8, WRAP), out=(BF, 2, 72, WRAP))),
    ("moe_quantize_fp4", dict(x=(BF, 8, WRAP), codes=(U8, 8, WRAP // 2), scales=(U8, 8, WRAP // 16 + 12))),
    ("moe_dequantize_fp4", dict(out=(BF, 8, WRAP), codes=(U8, 8, WRAP // 2), scales=(U8, 8, WRAP // 16 + 12))),
    ("moe_grouped_gemm_fp4", dict(x_codes=(U8, 8, WRAP // 2), x_scales=(U8, 8, WRAP // 16 + 12),
                                  w_codes=(U8, 2, 72, WRAP // 2), w_scales=(U8, 2, 72, WRAP // 16 + 12))),
])
def test_bindings_refuse_what_32_bits_do_not_hold(lib, name, tensors):  # noqa: F811
    every = {n: Fake(*v) for n, v in {**CALLS[name][0], **tensors}.items()}
    with pytest.raises(ValueError, match="2\\^30"):
        getattr(moe, name)(**every, **CALLS[name][1])
    assert not lib.calls


def test_scale_stride_past_32_bits():
    assert moe.moe_fp4_scale_stride(moe.FP4_NV, MOST) == MOST // 16
    assert moe.moe_fp4_scale_stride(moe.FP4_NV, WRAP) == moe.moe_fp4_scale_stride(moe.FP4_MX, MOST + 32) == 0
    assert torch.iinfo(torch.int32).max > MOST
