"""The norms between two blocks on the GPU against their plain 64-bit form. Bounds: tests/block_ref.py."""
import numpy as np
import pytest
import torch

from tests import block_ref as N
from tests import dense_ref as R
from tests import gpu_helpers as G
from tests.test_gpu_dense import BF16, F32, f64, gen, guarded, rows

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(120)]
EPS = float(np.float32(1e-5))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    G.ensure_built()
    yield


def make_gate(kind, T, H, g):
    if kind is None:
        return None, None
    shape = {"full": (T, H), "row": (1, H), "vector": (H,), "token": (T, 1), "spread": (T, 1)}[kind]
    gate = (2 * torch.randn(*shape, generator=g)).bfloat16().cuda()
    if kind == "spread":
        gate = gate.expand(T, H)
    if kind == "full":
        gate = rows(T, H, BF16, g, pad=7, offset=1, sigma=2.0)
    return gate, np.broadcast_to(f64(gate), (T, H))


def check(r, x, y, post, weight, gate, act, alpha, beta, dtype, eps=EPS):
    a, b = float(np.float32(alpha)), float(np.float32(beta))
    s, off, out, lost = N.block_norm(f64(x), f64(y), None if post is None else f64(post),
                                     None if weight is None else f64(weight), eps, gate, act, a, b)
    if r.sum is not None:
        R.check(f64(r.sum), s, off + (N.bf16(s) + R.B * off if dtype is BF16 else 0), "sum")
    if r.out is not None:
        R.check(f64(r.out), out, lost * (1 + R.B) + N.bf16(out), "out")
    if r.codes is not None:
        top = np.abs(out).max(1)
        slack = lost.max(1)
        R.check(f64(r.scales), top / 127, slack / 127 + 2 * R.U * top / 127, "scales")
        held = f64(r.codes) * f64(r.scales)[:, None]
        # half a step, the value's own error, and the scale's in up to 127 codes
        R.check(held, out, lost + (slack + (0.5 + 127 * 8 * R.U) * top / 127 + 4 * R.U * top)[:, None], "codes")


@pytest.mark.parametrize("H", [1, 7, 8, 100, 512, 513, 1025, 2048, 2049, 2561, 4096, 4097, 7168, 8193, 16384, 16391, 40001])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind,act", [("full", "sigmoid"), ("token", "tanh")])
def test_every_output(H, dtype, kind, act):
    from mxfp4_latent_mixture_sigmoid_amd import block_norm
    T, g = (3 if H > 512 else 9), gen(H)
    x, y = rows(T, H, dtype, g, pad=5, offset=1), rows(T, H, BF16, g, pad=1, offset=3, sigma=4.0)
    post, w = [(1 + 0.1 * torch.randn(H, generator=g)).bfloat16().cuda() for _ in range(2)]
    gate, gv = make_gate(kind, T, H, g)
    out, ok_o = guarded(T, H, BF16)
    codes, ok_q = guarded(T, H, torch.int8)
    total, ok_s = guarded(T, H, dtype)
    r = block_norm(x, y, post, w, 1e-5, gate=gate, gate_act=act, scale=0.7, residual_scale=1.3, sum=total, out=out,
                   codes=codes)
    check(r, x, y, post, w, gv, act, 0.7, 1.3, dtype)
    assert ok_o() and ok_q() and ok_s()


@pytest.mark.parametrize("kind", [None, "full", "row", "vector", "token", "spread"])
@pytest.mark.parametrize("act", [None, "sigmoid", "tanh"])
@pytest.mark.parametrize("T,H", [(1, 7168), (5, 300), (1100, 1500)])
def test_gates(kind, act, T, H):
    from mxfp4_latent_mixture_sigmoid_amd import block_norm
    if kind is None and act is not None:
        pytest.skip("no gate to activate")
    g = gen(T + H)
    x, y = rows(T, H, BF16, g), rows(T, H, BF16, g, sigma=0.1)
    gate, gv = make_gate(kind, T, H, g)
    r = block_norm(x, y, None, None, 1e-5, gate=gate, gate_act=act, codes=True)
    check(r, x, y, None, None, gv, act, 1.0, 1.0, BF16)


@pytest.mark.parametrize("act", ["sigmoid", "tanh"])
def test_gate_over_its_whole_range(act):
    """Every finite BF16 value and both infinities as a gate: s = alpha a(g) n with x = 0 and n near one."""
    from mxfp4_latent_mixture_sigmoid_amd import block_norm
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(BF16)
    g = bits[~torch.isnan(bits)].cuda()[:, None]
    T = g.shape[0]
    x, y = torch.zeros(T, 8, device="cuda"), torch.ones(T, 8, dtype=BF16, device="cuda")
    r = block_norm(x, y, eps=0.0, gate=g, gate_act=act, out=False)
    want = np.broadcast_to(N.gate_value(f64(g), act), (T, 8))
    # past 87 the sigmoid's low end is taken for 0; subnormal results are not held to their own size
    R.check(f64(r.sum), want, np.abs(want) * (N.GATE_REL + R.NORM_REL) + 2.0 ** -125, act)


def test_many_rows_and_sum_in_place():
    from mxfp4_latent_mixture_sigmoid_amd import block_norm
    g = gen(3)
    for dtype in (BF16, F32):
        for H in (130, 3000, 5000, 20000):
            x, y = rows(6, H, dtype, g), rows(6, H, BF16, g)
            gate, _ = make_gate("row", 6, H, g)
            apart = block_norm(x, y, gate=gate, gate_act="tanh", codes=True)
            r = block_norm(x, y, gate=gate, gate_act="tanh", codes=True, sum=x)
            assert r.sum is x
            for a, b in zip(r, apart):
                assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H", [256, 900, 2000, 2500, 3584, 5000, 7168, 12000])
def test_same_bits_in_any_batch(dtype, H):
    """Rows alone, among few and among many."""
    from mxfp4_latent_mixture_sigmoid_amd import block_norm
    g, T = gen(H), 1500
    x, y = rows(T, H, dtype, g), rows(T, H, BF16, g)
    gate, _ = make_gate("full", T, H, g)
    post, w = [(1 + 0.1 * torch.randn(H, generator=g)).bfloat16().cuda() for _ in range(2)]
    every = block_norm(x, y, post, w, gate=gate, gate_act="sigmoid", scale=0.3, residual_scale=0.9, codes=True)
    for first, n in ((0, 1), (7, 3), (1000, 200)):
        p = slice(first, first + n)
        some = block_norm(x[p], y[p], post, w, gate=gate[p], gate_act="sigmoid", scale=0.3, residual_scale=0.9, codes=True)
        for a, b in zip(some, every):
            assert torch.equal(a, b[p])


@pytest.mark.parametrize("H", [64, 3000, 20000])
def test_rows_at_the_ends_of_the_range(H):
    """Zero rows, NaN, infinities, and blocks and streams whose squares leave FP32's range."""
    from mxfp4_latent_mixture_sigmoid_amd import block_norm
    g = gen(5)
    x, y = rows(9, H, F32, g), rows(9, H, BF16, g)
    y[1] = 0
    y[2, H // 2] = float("nan")
    y[3, 0] = float("inf")
    y[4] *= 1e30
    y[5] *= 1e-30
    x[6] *= 1e30
    x[7] = 0
    y[7] = 0
    r = block_norm(x, y, eps=1e-5, codes=True)
    good = [0, 1, 4, 5, 6, 7, 8]
    sub = type(r)(r.out[good], r.codes[good], r.scales[good], r.sum[good])
    check(sub, x[good], y[good], None, None, None, None, 1.0, 1.0, F32)
    assert torch.isnan(r.out[2]).all() and torch.isnan(r.scales[2]) and not r.codes[2].any()
    assert torch.isnan(r.sum[3, 0]) and torch.isnan(r.sum[3]).sum() == 1 and torch.equal(r.sum[3, 1:], x[3, 1:])
    assert torch.isnan(r.out[3]).all() and torch.isnan(r.scales[3])
    assert not r.codes[7].any() and r.scales[7] == 0
    tiny = block_norm(x[:1] * 1e-30, y[:1] * 1e-30, eps=0.0, scale=1e-30)      # squares below FP32's range
    s, off, out, lost = N.block_norm(f64(x[:1] * 1e-30), f64(y[:1] * 1e-30), None, None, 0.0, None, None,
                                     float(np.float32(1e-30)))
    R.check(f64(tiny.out), out, np.abs(out) * (R.B + 4 * R.NORM_REL) + 4 * R.NORM_REL, "tiny")


def test_no_rows_and_single_outputs():
    from mxfp4_latent_mixture_sigmoid_amd import block_norm
    e = torch.empty(0, 96, dtype=BF16, device="cuda")
    r = block_norm(e, e, codes=True)
    assert r.out.shape == r.codes.shape == r.sum.shape == (0, 96) and r.scales.shape == (0,)
    x, y = rows(4, 1000, BF16, gen(1)), rows(4, 1000, BF16, gen(2))
    every = block_norm(x, y, codes=True)
    only = block_norm(x, y, out=False)
    assert only.out is None and only.codes is None and torch.equal(only.sum, every.sum)
    assert torch.equal(block_norm(x, y, sum=False).out, every.out)
    only = block_norm(x, y, sum=False, out=False, codes=True)
    assert torch.equal(only.codes, every.codes) and torch.equal(only.scales, every.scales)


def test_another_stream_and_a_graph():
    from mxfp4_latent_mixture_sigmoid_amd import block_norm
    g = gen(9)
    x, y = rows(33, 7168, BF16, g), rows(33, 7168, BF16, g)
    gate, _ = make_gate("full", 33, 7168, g)
    want = block_norm(x, y, gate=gate, gate_act="sigmoid", codes=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = block_norm(x, y, gate=gate, gate_act="sigmoid", codes=True, stream=side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = block_norm(x, y, gate=gate, gate_act="sigmoid", codes=True)
    for i in range(3):
        y.copy_(rows(33, 7168, BF16, g))
        graph.replay()
        eager = block_norm(x, y, gate=gate, gate_act="sigmoid", codes=True)
        torch.cuda.synchronize()
        for a, b in zip(held, eager):
            assert torch.equal(a, b), i
