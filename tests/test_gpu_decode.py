"""The whole layer for a few tokens in one kernel (MoELayer.decode). Bounds: tests/decode_ref.py."""
import os

import numpy as np
import pytest
import torch

from tests import decode_ref as D
from tests import gpu_helpers as G
from workload import SHAPES, make_inputs
from workload.gen import LayerShape

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(120)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    G.ensure_built()
    yield


def shape(T=16, H=256, Lt=256, E=40, K=4, I=128, S=1, Is=64, latent=True, routing="uniform", seed=7):
    return LayerShape("few", T, H, Lt, E, K, I, S, Is, latent, routing, 0.0, seed)


def tokens(inp):
    return torch.from_numpy(inp["x"].view(np.int16)).cuda().view(torch.bfloat16)


def check_decode(s, inp, layer, x=None, r=None):
    """Every output of one call; returns it."""
    x = tokens(inp) if x is None else x
    bias = inp.get("router_bias")
    logits = torch.full((s.T, s.E), float("nan"), device="cuda")
    r = r or layer.decode(x, logit_bias=None if bias is None else torch.from_numpy(bias).cuda(), logits_out=logits)
    want = D.logits(inp, bias)
    # sums of Hin products in FP32, and the bias
    size = D.bf16(inp["x"]).abs() @ D.bf16(inp["w_router"]).abs().t() + want.abs()
    assert ((logits.double() - want).abs() <= size * 2.0 ** -24 * 64).all(), "logits"
    key = torch.sort(logits.double(), dim=1, descending=True, stable=True)
    assert torch.equal(r.ids.long(), key.indices[:, :s.K]), "ids"
    p = torch.sigmoid(key.values[:, :s.K])
    p = p / p.sum(1, keepdim=True)
    assert ((r.weights.double() - p).abs() <= p * 1e-6).all(), "weights"
    D.check(r.out, D.forward(s, inp, r.ids, p), f"T={s.T}")
    return r


SHAPES_FEW = [
    shape(T=1), shape(T=2, E=5, K=5), shape(T=3, H=384, Lt=128, E=17, K=1), shape(T=4, E=64, K=16, I=256),
    shape(T=5, S=0, Is=0), shape(T=7, H=128, Lt=640, S=2, Is=96), shape(T=8, E=257, K=8), shape(T=9, E=300, K=32),
    shape(T=12, E=1024, K=3, H=512), shape(T=13, I=384, Lt=384), shape(T=16, E=33, K=32, I=256, S=3, Is=32),
    shape(T=16, H=1024, Lt=1152, E=100, K=6), shape(T=1, H=0, latent=False, S=0, Is=0, Lt=512),
    shape(T=6, H=0, latent=False, S=0, Is=0, E=61, K=6, I=512), shape(T=16, H=0, latent=False, S=0, Is=0, E=16, K=16),
    # more down items than places: two groups of columns to an item, the last one short, over one part of K and over two
    shape(T=8, Lt=896, E=260, K=32), shape(T=16, Lt=384, E=400, K=30, I=512),
    shape(T=16, E=90, routing="zipf"), shape(T=3, E=1, K=1), shape(T=16, E=1, K=1), shape(T=11, H=128, Lt=128, Is=32),
]


@pytest.mark.parametrize("s", SHAPES_FEW, ids=lambda s: f"{s.T}x{s.H}x{s.Lt}-{s.E}top{s.K}x{s.I}-{s.S}x{s.Is}")
def test_layers(s):
    inp = make_inputs(s)
    check_decode(s, inp, G.make_layer(s, inp, T_max=s.T))


@pytest.mark.parametrize("T", range(1, 17))
def test_every_token_count(T):
    s = SHAPES["tiny"].with_tokens(T)
    inp = make_inputs(s)
    check_decode(s, inp, G.make_layer(s, inp, T_max=T))


@pytest.mark.parametrize("T", [1, 4, 16])
def test_one_gpus_share(T):
    """The full widths, with few experts held (the rest would take a minute to draw)."""
    s = shape(T=T, H=7168, Lt=3584, E=48, K=16, I=384, S=2, Is=384)
    inp = make_inputs(s)
    check_decode(s, inp, G.make_layer(s, inp, T_max=T))


def test_shared_experts_on_a_second_stream():
    """That mode holds the shared rows apart; the call does not use the stream."""
    s = shape(T=6, S=2)
    inp = make_inputs(s)
    want = check_decode(s, inp, G.make_layer(s, inp, T_max=6))
    got = G.make_layer(s, inp, T_max=6, shared_stream=True).decode(tokens(inp))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_near_the_other_form():
    """route_forward rounds each expert's output once more: 0.0023 of it."""
    s = shape(T=16, H=512, Lt=512, E=64, K=8, S=1)
    inp = make_inputs(s)
    layer = G.make_layer(s, inp, T_max=16)
    r, x = layer.alloc_routing(16), tokens(inp)
    other = layer.route_forward(x, 16, r).double()
    got = layer.decode(x)
    assert torch.equal(got.ids, r["topk_ids"])
    err, rms = (got.out.double() - other), other.square().mean().sqrt()
    assert float(err.square().mean().sqrt() / rms) <= 1.25 * np.hypot(2 ** 0.5 * np.hypot(D.SIGMA, 0.0023), 0.0023)


def test_the_same_bits_every_time():
    s = shape(T=16, E=200, K=16, Lt=512, H=512)
    inp = make_inputs(s)
    layer, x = G.make_layer(s, inp, T_max=16), tokens(inp)
    want = layer.decode(x)
    for _ in range(20):
        for a, b in zip(layer.decode(x), want):
            assert torch.equal(a, b)


def test_the_same_bits_in_any_batch():
    s = shape(T=16, E=70, K=9, Lt=384, H=512, I=256, routing="zipf")
    inp = make_inputs(s)
    layer, x = G.make_layer(s, inp, T_max=16), tokens(inp)
    bias = torch.from_numpy(inp["router_bias"]).cuda()
    want = layer.decode(x, logit_bias=bias)
    for first, n in ((0, 1), (3, 2), (5, 8), (15, 1), (1, 15)):
        for a, b in zip(layer.decode(x[first:first + n], logit_bias=bias), want):
            assert torch.equal(a, b[first:first + n])


@pytest.mark.parametrize("kind", ["all equal", "ties", "one token repeated"])
def test_ties(kind):
    s = shape(T=10, E=130, K=7)
    inp = make_inputs(s)
    if kind == "all equal":
        inp["w_router"][:] = 0
    elif kind == "ties":
        inp["w_router"][:] = inp["w_router"][np.arange(s.E) // 5]
    else:
        inp["x"][:] = inp["x"][0]
    r = check_decode(s, inp, G.make_layer(s, inp, T_max=10))
    if kind == "all equal":
        assert torch.equal(r.ids.cpu(), torch.arange(7, dtype=torch.int32).repeat(10, 1))
    if kind == "one token repeated":
        for t in r:
            assert torch.equal(t, t[:1].expand_as(t))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_token_that_is_not_finite(bad):
    """It takes some experts in range, and no other token sees it."""
    s = shape(T=5, E=70, K=6)
    inp = make_inputs(s)
    layer, x = G.make_layer(s, inp, T_max=5), tokens(inp)
    want = layer.decode(x)
    x = x.clone()
    x[2, 17] = bad
    got = layer.decode(x)
    keep = [0, 1, 3, 4]
    for a, b in zip(got, want):
        assert torch.equal(a[keep], b[keep])
    assert not torch.isfinite(got.out[2]).any()
    assert ((got.ids[2] >= 0) & (got.ids[2] < s.E)).all() and len(set(got.ids[2].tolist())) == s.K


def test_logits_of_nan_with_every_bit_set():
    """A bias whose bits are all ones gives no expert past the last."""
    s = shape(T=2, E=9, K=4)
    inp = make_inputs(s)
    bias = torch.full((9,), -1, dtype=torch.int32, device="cuda").view(torch.float32)
    r = G.make_layer(s, inp, T_max=2).decode(tokens(inp), logit_bias=bias)
    assert ((r.ids >= 0) & (r.ids < 9)).all()


def test_an_expert_that_is_not_finite():
    """Weights with a NaN scale mark the tokens that chose the expert and no others."""
    s = shape(T=16, E=24, K=3)
    inp = make_inputs(s)
    want = G.make_layer(s, inp, T_max=16).decode(tokens(inp))
    e = int(want.ids[0, 0])
    inp["down_scales"][e] = 255
    got = G.make_layer(s, inp, T_max=16).decode(tokens(inp))
    chose = (got.ids == e).any(1)
    assert torch.isnan(got.out[chose]).all() and torch.equal(got.out[~chose], want.out[~chose]) and (~chose).any()


def test_given_outputs_and_no_tokens():
    s = shape(T=3)
    inp = make_inputs(s)
    layer, x = G.make_layer(s, inp, T_max=3), tokens(inp)
    want = layer.decode(x)
    buf = torch.full((5, s.H), 7.0, dtype=torch.bfloat16, device="cuda")
    ids = torch.full((5, s.K), -9, dtype=torch.int32, device="cuda")
    got = layer.decode(x, out=buf[1:4], ids=ids[1:4])
    assert torch.equal(got.out, want.out) and torch.equal(got.ids, want.ids)
    assert (buf[[0, 4]] == 7).all() and (ids[[0, 4]] == -9).all()
    none = layer.decode(x[:0])
    assert none.out.shape == (0, s.H) and none.ids.shape == (0, s.K)


def test_two_streams_at_once():
    """Each call has its own workspace."""
    s = shape(T=16, E=200, K=8, H=1024, Lt=1024)
    inp = make_inputs(s)
    layer, x = G.make_layer(s, inp, T_max=16), tokens(inp)
    other = x.flip(0).contiguous()
    want, back = layer.decode(x), layer.decode(other)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for i in range(20):
        for j, (st, t) in enumerate(zip(streams, (x, other))):
            got[j].append(layer.decode(t, stream=st))
    torch.cuda.synchronize()
    for rs, w in zip(got, (want, back)):
        for r in rs:
            for a, b in zip(r, w):
                assert torch.equal(a, b)


def test_captured_and_replayed():
    s = shape(T=4, E=100, K=8, H=512, Lt=512)
    inp = make_inputs(s)
    layer, x = G.make_layer(s, inp, T_max=4), tokens(inp).clone()
    layer.decode(x)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held = layer.decode(x)
        graphs.append((g, held))
    for i in range(6):
        x.copy_(torch.randn(4, 512, device="cuda").bfloat16())
        for g, held in graphs:
            g.replay()
        want = layer.decode(x)
        torch.cuda.synchronize()
        for g, held in graphs:
            for a, b in zip(held, want):
                assert torch.equal(a, b), i


def test_in_a_step_with_the_norms_and_a_projection():
    """block_norm -> projection onto the residual stream -> block_norm -> decode, as a decoder's step runs them, eagerly and
    replayed; each against its own 64-bit form on the inputs that the step gave it."""
    from mxfp4_latent_mixture_sigmoid_amd import Bf16Linear, block_norm
    from tests import block_ref as N
    from tests import dense_ref as R
    s = shape(T=5, H=512, Lt=512, E=50, K=4)
    inp = make_inputs(s)
    layer, g = G.make_layer(s, inp, T_max=5), torch.Generator().manual_seed(1)
    w = (torch.randn(512, 512, generator=g) / 512 ** 0.5).bfloat16().cuda()
    one = (1 + 0.1 * torch.randn(512, generator=g)).bfloat16().cuda()
    proj = Bf16Linear(w, activation="silu", T_max=5)
    x, y = [torch.randn(5, 512, generator=g).bfloat16().cuda() for _ in range(2)]

    def step():
        a = block_norm(x, y, one, one, gate=y, gate_act="sigmoid")
        b = proj.forward(a.out, residual=a.sum)
        c = block_norm(a.sum, b, one, None)
        return a, b, c, layer.decode(c.out)
    a, b, c, d = step()
    f = lambda t: t.double().cpu().numpy()          # noqa: E731
    ref, off, out, lost = N.block_norm(f(x), f(y), f(one), f(one), float(np.float32(1e-6)), f(y), "sigmoid")
    R.check(f(a.sum), ref, off * (1 + R.B) + N.bf16(ref), "first sum")
    R.check(f(a.out), out, lost * (1 + R.B) + N.bf16(out), "first norm")
    v = a.out.double() @ w.double().t()
    p = v * torch.sigmoid(v) + a.sum.double()
    # 512 products in FP32, at most 512 roundings of their magnitudes, through silu's slope of 1.1
    size = a.out.double().abs() @ w.double().abs().t()
    R.check(f(b), f(p), f(1.1 * 512 * R.U * size + p.abs() * R.B + 64 * R.U * (v.abs() + p.abs())), "projection")
    ref, off, out, lost = N.block_norm(f(a.sum), f(b), f(one), None, float(np.float32(1e-6)))
    R.check(f(c.out), out, lost * (1 + R.B) + N.bf16(out), "second norm")
    inp["x"] = c.out.view(torch.int16).cpu().numpy().view(np.uint16)
    logits = D.logits(inp)
    best = torch.sort(logits, dim=1, descending=True, stable=True)
    p = torch.sigmoid(best.values[:, :s.K])
    assert torch.equal(best.indices[:, :s.K], d.ids.long())
    D.check(d.out, D.forward(s, inp, d.ids, p / p.sum(1, keepdim=True)), "mixture")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(3):
        y.copy_(torch.randn(5, 512, generator=g).bfloat16())
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        assert torch.equal(held[3].out, eager[3].out) and torch.equal(held[2].sum, eager[2].sum)


@pytest.fixture
def impatient():
    """Workgroups ask once for what they wait for, and then do each other's work."""
    from mxfp4_latent_mixture_sigmoid_amd import abi
    abi.lib().moe_decode_patience(0)
    yield
    abi.lib().moe_decode_patience(-1)


@pytest.mark.parametrize("s", [shape(T=1, E=70, K=8), shape(T=4, S=2, K=16), shape(T=16, E=200, K=8, Lt=512),
                               shape(T=2, H=0, latent=False, S=0, Is=0, E=61, K=6)], ids=lambda s: f"{s.T}")
def test_helping(s, impatient):
    from mxfp4_latent_mixture_sigmoid_amd import abi
    inp = make_inputs(s)
    layer, x = G.make_layer(s, inp, T_max=s.T), tokens(inp)
    got = [layer.decode(x) for _ in range(3)]
    torch.cuda.synchronize()
    abi.lib().moe_decode_patience(-1)
    want = layer.decode(x)
    for r in got:
        for a, b in zip(r, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 5])
def test_the_example_runs(T, capsys):
    import runpy
    example = runpy.run_path(os.path.join(os.path.dirname(__file__), "..", "examples", "decode_step.py"))
    example["main"]([str(T), "tiny"])
    assert f"{T} tokens" in capsys.readouterr().out
