"""More rows than one launch of block_norm takes (2^21): each row's outputs are those of the same row in a small call."""
import pytest
import torch

from tests import gpu_helpers as G
from tests.test_gpu_dense import BF16, F32

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(120)]
LAUNCH = 1 << 21


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    G.ensure_built()
    yield


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gate", [None, "full", "row", "token", "spread"])
def test_both_sides_of_a_launch(dtype, gate):
    from mxfp4_latent_mixture_sigmoid_amd import block_norm
    T, H = LAUNCH + 3, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")          # noqa: E731
    x, y = randn(T, H).to(dtype), randn(T, H + 3).bfloat16()[:, 1:H + 1]
    post, w = [(1 + 0.1 * randn(H)).bfloat16() for _ in range(2)]
    if gate is not None:
        gate = randn(*{"full": (T, H), "row": (1, H)}.get(gate, (T, 1))).bfloat16().expand(-1, H if gate != "token" else 1)
    near = [slice(0, 5), slice(LAUNCH - 5, LAUNCH + 3)]
    kw = dict(gate_act=None if gate is None else "sigmoid", scale=0.5, residual_scale=0.75, codes=True)
    want = [block_norm(x[n].clone(), y[n].contiguous(), post, w, gate=gate if gate is None or gate.shape[0] == 1 else gate[n], **kw)
            for n in near]
    codes = torch.full((T + 1, H), 99, dtype=torch.int8, device="cuda")
    r = block_norm(x, y, post, w, gate=gate, sum=x, **dict(kw, codes=codes[:T]))
    assert r.sum is x and (codes[T] == 99).all()
    for n, few in zip(near, want):
        for a, b in zip(r, few):
            assert torch.equal(a[n], b)
