"""MoELayer.decode's outputs are the same bits whoever does a call's items, and in any batch: over outputs enough that a
remainder which is rounded differently in one value of a hundred is seen in some of them. (Such a value of h is off by 2^-17 of
itself, so y by 6 x 10^-7, which flips one of 6000 outputs.)"""
import pytest
import torch

from tests import gpu_helpers as G
from tests.test_gpu_decode import impatient, shape, tokens  # noqa: F401
from workload import make_inputs

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(120)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    G.ensure_built()
    yield


LAYERS = [dict(H=4096, Lt=2048, E=40, K=16, I=384, S=2, Is=256), dict(H=0, latent=False, S=0, Is=0, Lt=3584, E=40, K=12, I=512)]


@pytest.mark.parametrize("layer", LAYERS, ids=["latent", "plain"])
@pytest.mark.parametrize("n", [1, 2, 7, 16])
def test_helpers_bits(layer, n, impatient):          # noqa: F811
    from mxfp4_latent_mixture_sigmoid_amd import abi
    s = shape(T=16, **layer)
    inp = make_inputs(s)
    layer, x = G.make_layer(s, inp, T_max=16), tokens(inp)
    parts = [x[i:i + n].contiguous() for i in range(0, 16 - n + 1, n)]
    got = [layer.decode(p) for p in parts]
    torch.cuda.synchronize()
    abi.lib().moe_decode_patience(-1)
    want = [layer.decode(p) for p in parts]
    for r, w in zip(got, want):
        for a, b in zip(r, w):
            assert torch.equal(a, b), int((a != b).sum())


@pytest.mark.parametrize("layer", LAYERS, ids=["latent", "plain"])
@pytest.mark.parametrize("n", [1, 2, 3, 8, 9])
def test_batches_bits(layer, n):
    s = shape(T=16, **layer)
    inp = make_inputs(s)
    layer, x = G.make_layer(s, inp, T_max=16), tokens(inp)
    want = layer.decode(x)
    for i in range(0, 16 - n + 1, n):
        for a, b in zip(layer.decode(x[i:i + n]), want):
            assert torch.equal(a, b[i:i + n]), (i, int((a != b[i:i + n]).sum()))
