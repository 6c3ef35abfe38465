"""CPU tests of what the bindings of the grouped products and of the 4-bit rows
check of their tensors, on stand-ins for CUDA tensors: the library is replaced by
one that only counts calls."""
import pytest
import torch

import routing_permute_grouped_gb300 as moe

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class Fake:
    """As much of a CUDA tensor as the bindings look at."""

    def __init__(self, dtype, *shape, device=0, address=1 << 20, strides=None):
        self.dtype, self.shape, self.address = dtype, torch.Size(shape), address
        self.is_cuda, self.device = device >= 0, torch.device("cuda", device) if device >= 0 else torch.device("cpu")
        dense = [1] * len(shape)
        for i in range(len(shape) - 2, -1, -1):
            dense[i] = dense[i + 1] * shape[i + 1]
        self.dense, self.strides = tuple(dense), tuple(strides or dense)

    def get_device(self):
        return self.device.index if self.is_cuda else -1

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self.strides if i is None else self.strides[i]

    def is_contiguous(self):
        return self.strides == self.dense

    def data_ptr(self):
        return self.address

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0

        return call


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(moe, "_lib", lib)
    monkeypatch.setattr(moe, "_raw_stream", lambda dev: 0x70 + dev)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return lib


# each call's tensors by argument name, and the rest of its arguments
CALLS = {
    "moe_grouped_gemm": (dict(x=(BF, 8, 64), w=(BF, 2, 72, 64), offsets=(I32, 3), y=(BF, 8, 72), row_scale=(F32, 8),
                              status=(I32, 64)), {}),
    "moe_grouped_wgrad": (dict(a=(BF, 8, 72), b=(BF, 8, 64), offsets=(I32, 3), out=(BF, 2, 72, 64), status=(I32, 64)),
                          {}),
    "moe_quantize_fp4": (dict(x=(BF, 8, 64), codes=(U8, 8, 32), scales=(U8, 8, 16), tensor_scale=(F32, 1), src=(I32, 8)),
                         dict(fmt=1)),
    "moe_dequantize_fp4": (dict(codes=(U8, 8, 32), scales=(U8, 8, 16), out=(BF, 8, 64), tensor_scale=(F32, 1)),
                           dict(fmt=1)),
    "moe_grouped_gemm_fp4": (dict(x_codes=(U8, 8, 32), x_scales=(U8, 8, 16), w_codes=(U8, 2, 72, 32),
                                  w_scales=(U8, 2, 72, 16), offsets=(I32, 3), y=(BF, 8, 72), x_scale=(F32, 1),
                                  w_scale=(F32, 2), row_scale=(F32, 8), status=(I32, 64)), dict(fmt=1)),
}
EACH = [(name, arg) for name, (tensors, _) in CALLS.items() for arg in tensors]


def _call(name, lib, **other):
    tensors, rest = CALLS[name]
    args = {n: Fake(*v) for n, v in tensors.items()}
    args.update(other)
    getattr(moe, name)(**args, **rest)


@pytest.mark.parametrize("name", CALLS)
def test_calls_pass_on_the_current_device(lib, name):
    _call(name, lib)
    assert [n for n, _ in lib.calls] == [name]
    assert lib.calls[0][1][-1] == 0x70  # the current device's current stream


@pytest.mark.parametrize("name,arg", EACH)
@pytest.mark.parametrize("device", [-1, 1])
def test_a_tensor_elsewhere_is_refused(lib, name, arg, device):
    with pytest.raises(ValueError):
        _call(name, lib, **{arg: Fake(*CALLS[name][0][arg], device=device)})
    assert not lib.calls


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_device_than_the_current_are_refused(lib, name):
    with pytest.raises(ValueError):
        _call(name, lib, **{n: Fake(*v, device=1) for n, v in CALLS[name][0].items()})
    assert not lib.calls


# the 4-bit layer of T = 6 tokens to 2 experts each, d = 128
LAYER = dict(x=(BF, 6, 128), out=(BF, 6, 128), ws=(U8, 4096), topk_idx=(I32, 6, 2), topk_w=(F32, 6, 2))


def _layer(prerouted, **other):
    cfg = moe.config_of(T=6, d=128, d_e=128, E=4, k=2)
    args = {n: Fake(*v) for n, v in LAYER.items() if prerouted or not n.startswith("topk")}
    args.update(other)
    call = moe.moe_layer_fwd_fp4_prerouted if prerouted else moe.moe_layer_fwd_fp4
    call(cfg, moe.MoeWeightsFp4(), **args)


@pytest.mark.parametrize("prerouted", [False, True])
def test_layer_fp4_takes_whole_tensors_of_any_shape(lib, prerouted):
    _layer(prerouted)
    _layer(prerouted, x=Fake(BF, 2, 3, 128), out=Fake(BF, 7, 128))  # larger buffers too
    assert len(lib.calls) == 2


@pytest.mark.parametrize("name,other", [
    (n, dict(device=1)) for n in LAYER] + [(n, dict(device=-1)) for n in LAYER] + [
    ("x", dict(shape=(5, 128))), ("out", dict(shape=(6, 120))), ("topk_idx", dict(shape=(6, 1))),
    ("topk_w", dict(shape=(11,))), ("x", dict(dtype=torch.float16)), ("out", dict(dtype=F32)),
    ("topk_idx", dict(dtype=torch.int64)), ("topk_w", dict(dtype=BF)), ("x", dict(strides=(256, 1))),
    ("topk_idx", dict(strides=(1, 6)))])
def test_layer_fp4_refuses_other_tensors(lib, name, other):
    dtype, *shape = LAYER[name]
    bad = Fake(other.pop("dtype", dtype), *other.pop("shape", shape), **other)
    with pytest.raises(ValueError):
        _layer(True, **{name: bad})
    if not name.startswith("topk"):
        with pytest.raises(ValueError):
            _layer(False, **{name: bad})
    assert not lib.calls


@pytest.mark.parametrize("name", [n for n, (tensors, _) in CALLS.items() if "status" in tensors])
def test_status_is_a_whole_aligned_word(lib, name):
    _call(name, lib, status=Fake(U8, 4))
    _call(name, lib, status=Fake(torch.int64, 1))
    for bad in (Fake(U8, 3), Fake(I32, 0, address=0), Fake(U8, 8, address=(1 << 20) + 2), Fake(I32, 4, 2, strides=(1, 4))):
        with pytest.raises(ValueError):
            _call(name, lib, status=bad)
    assert len(lib.calls) == 2
