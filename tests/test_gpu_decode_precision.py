"""What MoELayer.decode keeps beyond BF16: its outputs are the exact ones, rounded once. Bounds: tests/decode_parts.py."""
import pytest
import torch

from tests import decode_parts as P
from tests import gpu_helpers as G
from tests.test_gpu_decode import SHAPES_FEW, shape, tokens
from workload import make_inputs

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(120)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    G.ensure_built()
    yield


def check(s, inp=None):
    inp = inp or make_inputs(s)
    layer = G.make_layer(s, inp, T_max=s.T)
    bias = inp.get("router_bias")
    bias = None if bias is None else torch.from_numpy(bias).cuda()
    logits = torch.empty(s.T, s.E, device="cuda")
    r = layer.decode(tokens(inp), logit_bias=bias, logits_out=logits)
    p = torch.sigmoid(torch.gather(logits.double(), 1, r.ids.long()))
    P.check(r.out, P.forward(s, inp, r.ids, p / p.sum(1, keepdim=True)), f"T={s.T}")


@pytest.mark.parametrize("s", SHAPES_FEW, ids=lambda s: f"{s.T}x{s.H}x{s.Lt}-{s.E}top{s.K}x{s.I}-{s.S}x{s.Is}")
def test_layers(s):
    check(s)


# channels of shared experts around the latent width, whose parts lie in the same room; widths of one step and of odd counts of
# steps, on both sides of what the output product holds at once (two tokens of about 3000 columns in all)
WIDTHS = [shape(T=T, H=384, Lt=128, S=S, Is=Is) for T in (1, 8, 9) for S, Is in ((1, 96), (1, 128), (1, 160), (3, 256))]
WIDTHS += [shape(T=T, H=512, Lt=Lt, S=S, Is=Is) for T in (1, 2, 3, 16) for Lt, S, Is in ((3584, 2, 384), (1280, 1, 32), (3456, 0, 0))]
WIDTHS += [shape(T=T, H=256, Lt=7168, S=1, Is=224, E=4, K=2) for T in (1, 2, 8, 16)]


@pytest.mark.parametrize("s", WIDTHS, ids=lambda s: f"{s.T}x{s.Lt}-{s.S}x{s.Is}")
def test_widths(s):
    inp = make_inputs(s)
    check(s, inp=P.loud(inp) if s.S else inp)


@pytest.mark.parametrize("T", [1, 2, 4, 7, 8, 9, 16])
def test_one_gpus_share(T):
    s = shape(T=T, H=7168, Lt=3584, E=48, K=16, I=384, S=2, Is=384)
    check(s)


def test_the_same_bits_in_any_batch_of_wide_rows():
    """Rows whose parts do not all fit in LDS at once, with shared experts: one operand or two, the sums are the same."""
    s = shape(T=16, H=512, Lt=1792, E=30, K=5, I=256, S=2, Is=384)
    inp = make_inputs(s)
    layer, x = G.make_layer(s, inp, T_max=16), tokens(inp)
    want = layer.decode(x)
    assert torch.isfinite(want.out).all()
    for first, n in ((0, 1), (4, 2), (5, 3), (8, 8), (2, 9), (15, 1)):
        for a, b in zip(layer.decode(x[first:first + n]), want):
            assert torch.equal(a, b[first:first + n])


@pytest.mark.parametrize("T", [1, 3, 12])
def test_nothing_of_the_workspace_is_read(T):
    """NaN wherever the call has not written."""
    from mxfp4_latent_mixture_sigmoid_amd import abi
    s = shape(T=T, H=512, Lt=384, S=3, Is=160, K=5)
    inp = make_inputs(s)
    layer, x = G.make_layer(s, inp, T_max=T), tokens(inp)
    want = layer.decode(x)
    size = abi.decode_query(layer.cfg, T)
    room = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
    got = [torch.empty_like(t) for t in want]
    stream = torch.cuda.current_stream().cuda_stream
    for _ in range(2):
        room.fill_(255)
        abi.check(abi.lib().moe_decode(layer.handle, x.data_ptr(), T, None, None, got[1].data_ptr(), got[2].data_ptr(),
                                       got[0].data_ptr(), room.data_ptr(), size, stream), "moe_decode")
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert (room[size:] == 255).all()
