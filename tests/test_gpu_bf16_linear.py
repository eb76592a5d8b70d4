"""The BF16 product with bias, activation and residual on the GPU.

Inputs are small whole numbers times powers of two, so that every sum (at most 64 K of the smallest unit, K <= 131072)
is exact in FP32 whatever its order: what is left is the epilogue's error. With u = 2^-24:
  none, relu   a = p + bias: u of it
  silu         exponent's rounding 2 |v| u, exponential, sum and reciprocal 2 u each, product: (24 + 6 |v|) u
  gelu         argument 2 u (times x erf'(x) < 0.5), erf 4 u, sum u, two products, all of |v|: 8 u |v|
  gelu_tanh    gate q = 2 sqrt(2 / pi) (v + 0.044715 v^3) with 6 u of itself: (24 + 10 |q|) u
  gated        a product more; the residual's sum u of both; BF16 adds half a unit (R.B)."""
import numpy as np
import pytest
import torch

from tests import dense_ref as R
from tests import gpu_helpers as G
from tests.test_gpu_dense import BF16, F32, f64, gen, guarded

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(120)]
ACTS = ["none", "silu", "gelu", "gelu_tanh", "relu"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    G.ensure_built()
    yield


def whole(*shape, g, scale=1.0):
    return torch.randint(-8, 9, shape, generator=g).float().mul_(scale).bfloat16()


def placed(t, pad=0, offset=0, fill=float("nan")):
    """t's rows on the GPU, `pad` values apart, `offset` values into a buffer of `fill`."""
    T, n = t.shape
    ld = n + pad
    buf = torch.full((offset + T * ld + 64,), fill, dtype=t.dtype, device="cuda")
    v = buf[offset:offset + T * ld].view(T, ld)[:, :n]
    v.copy_(t)
    return v


def act64(p, act):
    """(a(p), its allowed error)"""
    e = torch.special
    if act == "silu":
        a = p * torch.sigmoid(p)
        return a, a.abs() * (24 + 6 * p.abs()) * R.U + 2.0 ** -120
    if act == "gelu":
        return p * e.erfc(-p * 0.5 ** 0.5) / 2, 8 * R.U * p.abs()
    if act == "gelu_tanh":
        q = (8 / np.pi) ** 0.5 * (p + 0.044715 * p ** 3)
        a = p * torch.sigmoid(q)
        return a, a.abs() * (24 + 10 * q.abs()) * R.U + 2.0 ** -120
    if act == "relu":
        p = p.clamp(min=0)
    return p, 2 * R.U * p.abs()


def unit(K):
    """A power of two that brings sums of K products of numbers up to 8 (deviation 24 sqrt(K)) to a few units."""
    return 2.0 ** -round(np.log2(12 * K ** 0.5))


def reference(x, w, up, bias, residual, act, bf16):
    p = x.double().cuda() @ w.double().cuda().t().contiguous()
    if bias is not None:
        p = p + bias.double()
    a, err = act64(p, act)
    err = err + 2 * R.U * p.abs() * (bias is not None)
    if up is not None:
        u = x.double().cuda() @ up.double().cuda().t().contiguous()
        a, err = a * u, err * u.abs() + 2 * R.U * (a * u).abs()
    if residual is not None:
        a = a + residual.double()
        err = err + R.U * a.abs()
    if bf16:
        err = err * (1 + R.B) + a.abs() * R.B + 2.0 ** -133
    return a, err


def compare(out, ref, err, what):
    over = (out.double() - ref).abs() - err
    assert not torch.isnan(out).any(), what
    assert over.max() <= 0, (what, float(over.max()), int((over > 0).sum()))


SIZES = [  # T, N, K, pad of x, offset of x: both sides of 16-row and 64-value blocks and of the tiles
    (1, 1, 1, 0, 0), (1, 16, 64, 0, 0), (1, 700, 1792, 0, 0), (2, 17, 63, 0, 1), (3, 100, 65, 7, 0), (1, 40, 7, 0, 0),
    (15, 64, 32, 0, 0), (16, 65, 72, 0, 0), (17, 31, 500, 8, 0), (31, 96, 136, 0, 3), (33, 48, 128, 16, 16),
    (63, 200, 555, 0, 0), (64, 129, 1024, 0, 0), (65, 127, 320, 0, 0), (100, 333, 389, 5, 2), (128, 256, 256, 0, 0),
    (129, 257, 257, 0, 0), (200, 1000, 192, 0, 0), (256, 64, 2176, 0, 0), (300, 520, 48, 0, 0), (777, 1001, 767, 1, 0),
    (1500, 272, 80, 0, 0), (64, 3000, 3584, 0, 0), (40, 2064, 7168, 0, 0), (513, 515, 65, 0, 0),
    # rows at odd addresses: through registers (from 8 values on) in every tile, or laid out first
    (5, 40, 7, 0, 1), (5, 40, 8, 1, 1), (7, 33, 15, 0, 0), (1, 3500, 129, 0, 7), (16, 7000, 71, 0, 0),
    (16, 13000, 67, 2, 1), (32, 6200, 65, 0, 1), (30, 25000, 50, 3, 0), (64, 6300, 100, 1, 0), (64, 13000, 77, 1, 0),
    (60, 24600, 65, 1, 0), (130, 5000, 65, 0, 1), (300, 4200, 69, 4, 0), (1000, 4000, 71, 0, 3), (700, 6000, 39, 0, 2),
    (64, 14336, 4700, 1, 0),
]


@pytest.mark.parametrize("T,N,K,pad,offset", SIZES)
@pytest.mark.parametrize("kind", ["bf16", "f32+bias+res", "glu", "glu f32+res"])
def test_products(T, N, K, pad, offset, kind):
    """Behind every row of x lies NaN: nothing of it may reach a sum."""
    from mxfp4_latent_mixture_sigmoid_amd import Bf16Linear
    g = gen(T * 1000 + N + K)
    out_dtype, glu = F32 if "f32" in kind else BF16, "glu" in kind
    act = ACTS[(T + N + K) % 5]
    s = unit(K)
    x, w = whole(T, K, g=g), whole(N, K, g=g, scale=s)
    up = whole(N, K, g=g, scale=s) if glu else None
    bias = (torch.randint(-16, 17, (N,), generator=g) * 0.25).cuda() if "bias" in kind else None
    res_dtype = (BF16, F32)[N % 2]
    res = placed(torch.randn(T, N, generator=g).to(res_dtype), pad=3, offset=1) if "res" in kind else None
    layer = Bf16Linear(w.cuda(), bias=bias, up_weight=None if up is None else up.cuda(), activation=act, T_max=T,
                       out_dtype=out_dtype)
    out, ok = guarded(T, N, out_dtype)
    layer.forward(placed(x, pad, offset), residual=res, out=out)
    ref, err = reference(x, w, up, bias, res, act, out_dtype is BF16)
    compare(out, ref, err, f"{kind} {act} {T}x{N}x{K}")
    assert ok()


# (tokens, outputs, values): whole and ragged tiles of 128 x 64, 128 x 128, 256 x 128, 256 x 224 and 256 x 256, and
# sums of one to several 64-value stages
LARGE = [(2048, 4096, 320, 0), (4100, 4200, 136, 0), (2304, 2100, 192, 1), (1030, 1100, 512, 0), (8192, 500, 64, 0),
         (300, 9000, 128, 1), (2048, 7168, 32, 0), (2050, 7170, 50, 0), (3584, 4096, 576, 0), (1921, 6930, 257, 0),
         (2048, 3584, 128, 1), (2300, 3900, 65, 1), (2048, 3600, 1, 1), (4096, 3584, 192, 0), (257, 6000, 168, 0),
         (1793, 7169, 1650, 0), (2000, 7000, 750, 0), (1700, 7010, 2100, 0), (1000, 7000, 1281, 0), (2047, 3501, 850, 1),
         (1000, 3500, 1700, 1), (300, 3000, 150, 1), (2040, 7000, 2049, 0)]


@pytest.mark.parametrize("T,N,K,glu", LARGE)
@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("res", [None, BF16, F32])
def test_products_large(T, N, K, glu, out_dtype, res):
    from mxfp4_latent_mixture_sigmoid_amd import Bf16Linear
    g, act = gen(T + N), ACTS[(T + K) % 5]
    s = unit(K)
    x, w = whole(T, K, g=g), whole(N, K, g=g, scale=s)
    up = whole(N, K, g=g, scale=s) if glu else None
    bias = (torch.randint(-16, 17, (N,), generator=g) * 0.25).cuda() if not glu and N % 3 == 0 else None
    r = None if res is None else placed(torch.randn(T, N, generator=g).to(res), pad=N % 4, offset=T % 2)
    layer = Bf16Linear(w.cuda(), bias=bias, up_weight=None if up is None else up.cuda(), activation=act, T_max=T,
                       out_dtype=out_dtype)
    out, ok = guarded(T, N, out_dtype)
    layer.forward(placed(x), residual=r, out=out)
    assert ok()
    ref, err = reference(x, w, up, bias, r, act, out_dtype is BF16)
    compare(out, ref, err, f"{act} {T}x{N}x{K}")


@pytest.mark.parametrize("T", [1, 16, 33, 64, 65, 200])
def test_widest_sum(T):
    from mxfp4_latent_mixture_sigmoid_amd import Bf16Linear, abi
    K, N = abi.DENSE_MAX_K, 20
    w = torch.full((N, K), 8.0, dtype=BF16, device="cuda")
    w[1::2] = -7.0
    out = Bf16Linear(w, T_max=T, out_dtype=F32).forward(torch.full((T, K), 8.0, dtype=BF16, device="cuda"))
    assert (out[:, 0::2] == 64.0 * K).all() and (out[:, 1::2] == -56.0 * K).all()


@pytest.mark.parametrize("T,N,K", [(3, 50, 300), (70, 50, 300), (70, 500, 320), (1500, 2000, 192)])
@pytest.mark.parametrize("glu", [0, 1])
def test_a_row_that_is_not_finite(T, N, K, glu):
    """NaN and infinities mark their own rows and no others."""
    from mxfp4_latent_mixture_sigmoid_amd import Bf16Linear
    g = gen(5)
    w = [whole(N, K, g=g, scale=unit(K)).cuda() for _ in range(2)]
    layer = Bf16Linear(w[0], up_weight=w[1] if glu else None, activation="silu", T_max=T)
    x = whole(T, K, g=g).cuda()
    want = layer.forward(x)
    x[1, K // 2], x[2, 0], x[-1, -1] = float("nan"), float("inf"), -float("inf")
    out = layer.forward(x)
    odd = torch.zeros(T, dtype=torch.bool, device="cuda")
    odd[[1, 2, -1]] = True
    assert torch.equal(out[~odd], want[~odd])
    assert torch.isnan(out[1]).all() and not torch.isfinite(out[2][w[0][:, 0] > 0]).any()


@pytest.mark.parametrize("act", ACTS)
def test_activations_over_their_range(act):
    """A product with one input: a(v) of values from -120 to 120 and far out."""
    from mxfp4_latent_mixture_sigmoid_amd import Bf16Linear
    v = torch.cat([torch.linspace(-120, 120, 4001), torch.tensor([1e4, -1e4, 1e18, -1e18, 0.0, 1e-20, -1e-30])]).bfloat16()
    for T in (1, 33):
        out = Bf16Linear(v[:, None].cuda(), activation=act, out_dtype=F32).forward(torch.ones(T, 1, dtype=BF16, device="cuda"))
        ref, err = act64(v.double().cuda(), act)
        ref = torch.where(torch.isnan(ref), torch.zeros_like(ref), ref)
        for row in out:
            compare(row, ref, err + 2.0 ** -120, act)


def test_many_tokens_take_the_same_activations():
    """The large tiles' epilogue against the small ones'."""
    from mxfp4_latent_mixture_sigmoid_amd import Bf16Linear
    g = gen(8)
    w, x = whole(2000, 64, g=g, scale=unit(64)), whole(3000, 64, g=g)
    for act in ACTS:
        layer = Bf16Linear(w.cuda(), activation=act, out_dtype=F32)
        assert torch.equal(layer.forward(x.cuda())[:16], layer.forward(x[:16].cuda()))


@pytest.mark.parametrize("T,N,K", [(1, 1000, 256), (48, 700, 130), (300, 3000, 192), (2048, 2100, 128)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_onto_the_residual_itself(T, N, K, dtype):
    from mxfp4_latent_mixture_sigmoid_amd import Bf16Linear
    g = gen(T)
    layer = Bf16Linear(whole(N, K, g=g, scale=unit(K)).cuda(), T_max=T, out_dtype=dtype)
    x, res = whole(T, K, g=g).cuda(), torch.randn(T, N, generator=g).to(dtype).cuda()
    want = layer.forward(x, residual=res)
    got = layer.forward(x, residual=res, out=res)
    assert got is res and torch.equal(got, want)


def test_no_tokens_other_streams_and_a_graph():
    from mxfp4_latent_mixture_sigmoid_amd import Bf16Linear
    g = gen(2)
    layer = Bf16Linear(whole(900, 320, g=g, scale=unit(320)).cuda(), activation="gelu", T_max=2000)
    assert layer.forward(torch.empty(0, 320, dtype=BF16, device="cuda")).shape == (0, 900)
    for T, pad in ((5, 0), (1500, 1)):
        x = placed(whole(T, 320, g=g), pad)
        res = torch.randn(T, 900, generator=g).cuda()
        want = layer.forward(x, residual=res)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        got = layer.forward(x, residual=res, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = layer.forward(x, residual=res)
        for _ in range(3):
            x.copy_(whole(T, 320, g=g))
            graph.replay()
            eager = layer.forward(x, residual=res)
            torch.cuda.synchronize()
            assert torch.equal(held, eager)


def test_weights_in_any_order():
    from mxfp4_latent_mixture_sigmoid_amd import Bf16Linear
    g = gen(4)
    w, x = whole(130, 70, g=g, scale=unit(70)).cuda(), whole(9, 70, g=g).cuda()
    want = Bf16Linear(w).forward(x)
    assert torch.equal(Bf16Linear(w.t().contiguous().t()).forward(x), want)
    wide = torch.zeros(130, 200, dtype=BF16, device="cuda")
    wide[:, 3:73] = w
    assert torch.equal(Bf16Linear(wide[:, 3:73]).forward(x), want)


def test_outputs_past_32_bit_offsets():
    """More than 2^31 outputs: the last rows and those around the boundary."""
    from mxfp4_latent_mixture_sigmoid_amd import Bf16Linear
    g = gen(6)
    T, N, K = 70000, 32768, 64
    w, x = whole(N, K, g=g, scale=unit(K)).cuda(), whole(T, K, g=g).cuda()
    out = Bf16Linear(w, T_max=T).forward(x)
    for r in (0, 65535, 65536, T - 1):
        assert torch.equal(out[r], (x[r].float() @ w.float().t()).bfloat16()), r
