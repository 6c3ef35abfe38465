"""GPU tests of the 4-bit layer's set-up: streams in any form, tensor scales of the MX format."""
import pytest
import torch

import routing_permute_grouped_gb300 as moe
from tests.test_gpu_ragged import _rand

pytestmark = pytest.mark.gpu


def _layer(name, scales=(None, None), stream=None):
    T, d, de, E, ds = 70, 512, 256, 5, 128
    cfg = moe.config_of(T=T, d=d, d_e=de, E=E, k=2, d_shared=ds)
    w = dict(W1=_rand((E, d, de), 1, std=d ** -0.5), W3=_rand((E, d, de), 2, std=d ** -0.5),
             W2=_rand((E, de, d), 3, std=de ** -0.5), Wg=_rand((d, E), 4, std=d ** -0.5),
             Ws1=_rand((d, ds), 5, std=d ** -0.5), Ws3=_rand((d, ds), 6, std=d ** -0.5),
             Ws2=_rand((ds, d), 7, std=ds ** -0.5))
    torch.cuda.synchronize()
    return moe.MoeLayer(cfg, fp4=name, fp4_scales=scales, stream=stream, **w), _rand((T, d), 8)


@pytest.mark.parametrize("name", ["mx", "nv"])
def test_setup_on_a_raw_handle(name):
    want, x = _layer(name)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        layer, _ = _layer(name, stream=stream)
        torch.cuda.synchronize()
        for a, b in zip((*layer.packed, *layer.shared_packed), (*want.packed, *want.shared_packed)):
            assert (a is None and b is None) or torch.equal(a, b)
        assert torch.equal(layer(x), want(x))


@pytest.mark.parametrize("scale", [0.5, 3.0, 0.0, float("nan")])
def test_mx_rows_have_no_tensor_scale(scale):
    """The MX quantiser ignores tensor scales, so the products of the layer's own
    activations do too: the same bits with and without."""
    want, x = _layer("mx")
    g = tuple(torch.tensor([s], device="cuda") for s in (scale, 2 * scale))
    layer, _ = _layer("mx", scales=g)
    assert torch.equal(layer(x), want(x))
