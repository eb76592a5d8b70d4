"""The bound that tests/test_gpu_decode_precision.py holds the few-token form to tells it from forms that round more."""
import numpy as np
import pytest
import torch

from tests import decode_parts as P
from workload import make_inputs
from workload.gen import LayerShape

SHAPES = [LayerShape("few", T, 256, 256, 40, 4, 128, S, 64, True, "uniform", 0.0, 7) for T, S in ((1, 1), (16, 1), (5, 2))]
SHAPES.append(LayerShape("few", 6, 0, 256, 40, 4, 128, 0, 0, False, "uniform", 0.0, 7))


def exact(s, inp, **kw):
    x = P.f64(inp["x"], "cpu")
    best = torch.sort(x @ P.f64(inp["w_router"], "cpu").t(), dim=1, descending=True, stable=True)
    p = torch.sigmoid(best.values[:, :s.K])
    return P.forward(s, inp, best.indices[:, :s.K], p / p.sum(1, keepdim=True), "cpu", **kw)


@pytest.mark.parametrize("s", SHAPES, ids=lambda s: f"{s.T}x{s.S}")
def test_one_rounding_at_the_end_is_near(s):
    ref = exact(s, make_inputs(s))
    assert P.beyond(ref.bfloat16(), ref) == (0.0, 0.0)
    off = torch.from_numpy(np.random.default_rng(0).standard_normal(tuple(ref.shape))) * ref.square().mean().sqrt()
    assert P.near((ref + P.SIGMA / 2 * off).bfloat16(), ref)


@pytest.mark.parametrize("s", SHAPES, ids=lambda s: f"{s.T}x{s.S}")
@pytest.mark.parametrize("value", ["z", "h", "hs", "zc"])
def test_a_value_in_one_part_is_not(s, value):
    if not s.has_latent and value != "h":
        pytest.skip("not in a layer without latent projections and shared experts")
    inp = make_inputs(s)
    if value == "hs":
        inp = P.loud(inp)
    assert not P.near(exact(s, inp, rounded=(value,)).bfloat16(), exact(s, inp))
