"""How far the activations of the BF16 product are off, relative to themselves. Without activations (x = 0) every sum is its bias, so
that the outputs are the activation of any FP32 value.

With u = 2^-24, relative to the result:
  gelu       v times Phi(v), for v < 0 the tail itself: 1 / (1 + p |v|) an argument's rounding u and a reciprocal 2 u, times the
             polynomial's slope d log / d log of at most 3.02: 9 u; eight fused steps u each, the fit 0.6 u, the product with t u; the exponential 2 u
             and its correction u, two products: 24 u. For v > 0 half of that at most, a difference and a product: within 24 u too
  silu       exponent's rounding 2 |v| u, exponential, sum and reciprocal 2 u each, product: (24 + 6 |v|) u
  gelu_tanh  the exponent q with 6 u of itself: (24 + 10 |q|) u
Results below FP32's normal numbers are allowed to be 0: at -87.3 and beyond, 2^-119, for the two whose exponential's reciprocal is."""
import numpy as np
import pytest
import torch

from tests import gpu_helpers as G

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(120)]
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    G.ensure_built()
    yield


def exact(v, act):
    """(the activation, what it may be off by)"""
    if act == "gelu":   # erfc of 64 bits keeps its relative precision
        a = v * torch.special.erfc(-v * 0.5 ** 0.5) / 2
        return a, 24 * U * a.abs() + 2.0 ** -125
    q = v if act == "silu" else (8 / np.pi) ** 0.5 * (v + 0.044715 * v ** 3)
    a = v * torch.sigmoid(q)
    return a, (24 + (6 if act == "silu" else 10) * q.abs()) * U * a.abs() + torch.where(q < -87, 2.0 ** -119, 2.0 ** -125)


def values():
    g = torch.Generator().manual_seed(0)
    v = torch.cat((torch.linspace(-14, 14, 3584), 10 ** torch.linspace(-30, 0, 256), -10 ** torch.linspace(-30, 0, 256),
                   torch.empty(992).uniform_(-95, 95, generator=g), torch.tensor([0.0, -0.0, 1e19, 3e38, -3e38, -1e19, 88.0, -88.0])))
    return v[torch.randperm(len(v), generator=g)]


@pytest.mark.parametrize("T", [1, 17, 64, 300, 2048])   # tiles of few tokens, and the large ones
@pytest.mark.parametrize("act", ["gelu", "silu", "gelu_tanh"])
@pytest.mark.parametrize("residual", [False, True])
def test_relative_error(T, act, residual):
    from mxfp4_latent_mixture_sigmoid_amd import Bf16Linear
    v = values().cuda()
    layer = Bf16Linear(torch.ones(len(v), 64, dtype=torch.bfloat16, device="cuda"), bias=v, activation=act, T_max=T, out_dtype=torch.float32)
    res = torch.zeros(T, len(v), device="cuda") if residual else None
    out = layer.forward(torch.zeros(T, 64, dtype=torch.bfloat16, device="cuda"), residual=res).double()
    ref, err = exact(v.double(), act)
    over = (out - ref).abs() - err
    assert not torch.isnan(out).any()
    worst = ((out - ref).abs() / ref.abs().clamp(min=2.0 ** -100)).amax(0)
    print(f"  {act} T={T}: {float(worst[v.abs() < 12].max()) / U:.1f} u within 12", flush=True)
    assert over.max() <= 0, (float(v[over.amax(0).argmax()]), float(over.max()))


@pytest.mark.parametrize("T", [1, 300])
def test_the_gates_relative_error(T):
    """gelu(g) * up, with whole numbers of eighths as g and powers of two as up."""
    from mxfp4_latent_mixture_sigmoid_amd import Bf16Linear
    n = 208
    g = (torch.arange(n) - 104).float() / 8
    w, up = torch.zeros(n, 64), torch.zeros(n, 64)
    w[:, 0], up[:, 1] = g, 1
    layer = Bf16Linear(w.bfloat16().cuda(), up_weight=up.bfloat16().cuda(), activation="gelu", T_max=T, out_dtype=torch.float32)
    x = torch.zeros(T, 64)
    x[:, 0], x[:, 1] = 1, 2.0 ** (torch.arange(T) % 7 - 3)
    out = layer.forward(x.bfloat16().cuda()).double().cpu()
    ref = g.double() * torch.special.erfc(-g.double() * 0.5 ** 0.5) / 2 * x[:, 1:2].double()
    assert ((out - ref).abs() <= 25 * U * ref.abs()).all()
