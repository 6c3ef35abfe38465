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
