"""CPU tests of the 4-bit layer's set-up: the library's calls and torch's streams
are replaced by ones that record on which stream work is queued."""
import contextlib

import pytest
import torch

import routing_permute_grouped_gb300 as moe
from routing_permute_grouped_gb300 import build as moe_build


class Handle:
    cuda_stream = 0x5150


@pytest.mark.parametrize("stream,handle", [(None, None), (0x77, 0x77), (0, 0), (Handle(), 0x5150)])
@pytest.mark.parametrize("name", ["mx", "nv"])
def test_setup_stays_on_the_callers_stream(monkeypatch, stream, handle, name):
    """Packing, the tensor scales (torch operations), quantising and the reuse of the
    packed temporaries are ordered on one stream, whatever form it is given in."""
    moe_build.build()
    current, seen = [None], []

    @contextlib.contextmanager
    def use(s):
        current.append(s.cuda_stream)
        yield
        current.pop()

    class External:
        def __init__(self, stream_ptr, device=None):
            self.cuda_stream = stream_ptr

    def queued(what, stream):
        seen.append((what, current[-1], None if stream is None else moe._stream(stream)))

    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(moe, "moe_pack_experts", lambda *a: queued("pack", a[-1]))
    monkeypatch.setattr(moe, "moe_pack_router", lambda *a: queued("router", a[-1]))
    monkeypatch.setattr(moe, "moe_quantize_fp4", lambda *a, stream=None, **kw: queued("quantize", stream))
    monkeypatch.setattr(moe.MoeLayer, "_init_ws", lambda self, cfg, dev: queued("workspace", stream))

    def w(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16)

    cfg = moe.config_of(T=4, d=128, d_e=128, E=2, k=1, d_shared=128)
    moe.MoeLayer(cfg, w(2, 128, 128), w(2, 128, 128), w(2, 128, 128), Wg=w(128, 2), Ws1=w(128, 128), Ws3=w(128, 128),
                 Ws2=w(128, 128), stream=stream, fp4=name)
    assert {s[0] for s in seen} == {"pack", "router", "quantize", "workspace"}
    assert {s[1:] for s in seen} == {(handle, handle)}
