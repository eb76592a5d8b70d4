"""The dense 8-bit path on the GPU against plain 64-bit forms: norm, quantisation, products, gated
products, and the block that runs them together. Bounds: tests/dense_ref.py."""
import numpy as np
import pytest
import torch

from tests import dense_ref as R
from tests import gpu_helpers as G

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(120)]

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    G.ensure_built()
    yield


def f64(t):
    return t.detach().double().cpu().numpy()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows(T, n, dtype, g, pad=0, offset=0, sigma=1.0):
    """[T, n] normal rows on the GPU, `pad` elements apart, starting `offset` elements into a buffer."""
    ld = n + pad
    buf = torch.zeros(offset + T * ld + 8, dtype=dtype)
    t = buf[offset:offset + T * ld].view(T, ld)[:, :n]
    t.copy_(torch.randn(T, n, generator=g) * sigma)
    d = buf.cuda()
    return d[offset:offset + T * ld].view(T, ld)[:, :n]


def codes_rows(T, n, g, pad=0, offset=0):
    ld = n + pad
    buf = torch.randint(-128, 128, (offset + T * ld + 8,), generator=g, dtype=torch.int8).cuda()
    return buf[offset:offset + T * ld].view(T, ld)[:, :n]


def guarded(T, n, dtype, pad=3):
    """An output inside a larger buffer whose other elements must not change."""
    buf = torch.full((T * (n + pad) + 64,), 77, dtype=dtype, device="cuda")
    view = buf[32:32 + T * (n + pad)].view(T, n + pad)[:, :n]

    def untouched():
        b = buf.clone()
        b[32:32 + T * (n + pad)].view(T, n + pad)[:, :n] = 77
        return bool((b == 77).all())
    return view, untouched


# widths on both sides of every limit of few rows (512, 2048, 4096, 8192, 16384; 1024 and 2560 are below) and past the last
WIDTHS = [1, 7, 8, 100, 511, 512, 513, 2048, 2051, 4096, 4097, 7168, 8193, 16384, 16391, 40001]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_all_outputs(H, dtype):
    from mxfp4_latent_mixture_sigmoid_amd import rms_norm
    T, g = (3 if H > 512 else 9), gen(H)
    x, d = rows(T, H, dtype, g, pad=5, offset=1), rows(T, H, BF16, g, pad=1, offset=3)
    w = (1 + 0.1 * torch.randn(H, generator=g)).bfloat16().cuda()
    out, ok_o = guarded(T, H, BF16)
    codes, ok_q = guarded(T, H, torch.int8)
    total, ok_s = guarded(T, H, dtype)
    r = rms_norm(x, w, 1e-5, delta=d, sum=total, out=out, codes=codes)
    s, y = R.norm(f64(x), f64(d), f64(w), float(np.float32(1e-5)))
    size = R.B if dtype is BF16 else 0
    R.check(f64(r.sum), s, np.abs(s) * (size + 2 * R.U), "sum")
    # where x and delta cancel, y inherits the rounding of their sum: u of either
    lost = 2 * R.U * (np.abs(f64(x)) + np.abs(f64(d))) * np.abs(y) / np.maximum(np.abs(s), 1e-30)
    R.check(f64(r.out), y, np.abs(y) * (R.B + R.NORM_REL) + 2 * lost, "out")
    if np.all(lost <= 0.01 * R.scales(y)[:, None]):
        R.check_codes(r.codes.cpu().numpy(), f64(r.scales), y, R.NORM_REL + 2e-6, "codes")
    assert ok_o() and ok_q() and ok_s()


@pytest.mark.parametrize("T,H", [(5, 1024), (6, 1025), (3, 2560), (3, 2561), (1025, 1000), (1024, 2048), (1030, 2555),
                                 (1027, 2561), (1025, 4096), (1024, 4097), (1025, 5120), (1026, 5121), (1024, 8192),
                                 (1023, 5000)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_many_rows(T, H, dtype):
    """Both sides of the limits for many rows (1024), and of 1024, 2560 and 5120 columns."""
    from mxfp4_latent_mixture_sigmoid_amd import quantise, rms_norm
    g = gen(T + H)
    x, d = rows(T, H, dtype, g, pad=3, offset=1, sigma=2.0), rows(T, H, BF16, g, pad=8)
    w = (1 + 0.1 * torch.randn(H, generator=g)).bfloat16().cuda()
    out, ok_o = guarded(T, H, BF16)
    codes, ok_q = guarded(T, H, torch.int8)
    total, ok_s = guarded(T, H, dtype)
    r = rms_norm(x, w, 1e-5, delta=d, sum=total, out=out, codes=codes)
    s, y = R.norm(f64(x), f64(d), f64(w), float(np.float32(1e-5)))
    size = R.B if dtype is BF16 else 0
    R.check(f64(r.sum), s, np.abs(s) * (size + 2 * R.U), "sum")
    lost = 2 * R.U * (np.abs(f64(x)) + np.abs(f64(d))) * np.abs(y) / np.maximum(np.abs(s), 1e-30)
    R.check(f64(r.out), y, np.abs(y) * (R.B + R.NORM_REL) + 2 * lost, "out")
    assert ok_o() and ok_q() and ok_s()
    got, want = f64(r.codes) * f64(r.scales)[:, None], y   # half a step, and the value's and the scale's error
    assert (np.abs(got - want) <= R.scales(y)[:, None] * (0.5 + 127 * (R.NORM_REL + 4e-6)) + 2 * lost).all()
    q, sc = quantise(x)
    R.check_codes(q.cpu().numpy(), f64(sc), f64(x), 0.0, "quantise")


@pytest.mark.parametrize("T", [1, 2, 4, 5, 64, 1000])
@pytest.mark.parametrize("H", [256, 1000, 7168])
def test_norm_plain(T, H):
    """No residual, no weight; one output at a time gives the bits of all at once."""
    from mxfp4_latent_mixture_sigmoid_amd import rms_norm
    x = rows(T, H, BF16, gen(T + H), sigma=3.0)
    r = rms_norm(x, codes=True)
    _, y = R.norm(f64(x), None, None, float(np.float32(1e-6)))
    R.check(f64(r.out), y, np.abs(y) * (R.B + R.NORM_REL), "out")
    R.check_codes(r.codes.cpu().numpy(), f64(r.scales), y, R.NORM_REL, "codes")
    assert torch.equal(rms_norm(x).out, r.out)
    only = rms_norm(x, out=False, codes=True)
    assert only.out is None and only.sum is None
    assert torch.equal(only.codes, r.codes) and torch.equal(only.scales, r.scales)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H", [130, 3000, 20000])
def test_norm_sum_in_place(dtype, H):
    from mxfp4_latent_mixture_sigmoid_amd import rms_norm
    g = gen(H)
    x, d = rows(6, H, dtype, g), rows(6, H, BF16, g)
    apart = rms_norm(x, delta=d, sum=True, codes=True)
    r = rms_norm(x, delta=d, sum=x, codes=True)
    assert r.sum is x
    for a, b in zip(r, apart):
        assert torch.equal(a, b)


@pytest.mark.parametrize("H", [64, 3000, 20000])
def test_norm_rows_without_a_norm(H):
    """Zero rows, NaN, infinities and values at both ends of the type, each in a row of its own."""
    from mxfp4_latent_mixture_sigmoid_amd import rms_norm
    x = rows(8, H, F32, gen(1))
    x[1] = 0
    x[2, H // 2] = float("nan")
    x[3, 0] = float("inf")
    x[4] = 1e-30
    x[5] *= 1e15
    x[6, 3] = -float("inf")
    r = rms_norm(x, eps=1e-6, codes=True)
    good = [0, 1, 4, 5, 7]
    _, y = R.norm(f64(x)[good], None, None, float(np.float32(1e-6)))
    R.check(f64(r.out)[good], y, np.abs(y) * (R.B + R.NORM_REL), "out")
    R.check_codes(r.codes.cpu().numpy()[good], f64(r.scales)[good], y, R.NORM_REL, "codes")
    assert torch.isnan(r.out[2]).all()
    for row, col in ((3, 0), (6, 3)):     # inf / inf at the infinity, 0 elsewhere
        nan = torch.isnan(r.out[row])
        assert nan[col] and nan.sum() == 1 and (r.out[row][~nan] == 0).all()
    for row in (2, 3, 6):
        assert torch.isnan(r.scales[row]) and not r.codes[row].any()
    zero = rms_norm(torch.zeros(2, H, device="cuda"), eps=0.0, codes=True)      # 0 / 0
    assert torch.isnan(zero.out).all() and torch.isnan(zero.scales).all() and not zero.codes.any()


@pytest.mark.parametrize("K", [1, 9, 512, 777, 2048, 14336, 16385, 33000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantise_and_back(K, dtype):
    from mxfp4_latent_mixture_sigmoid_amd import dequantise, quantise
    T = 7
    x = rows(T, K, dtype, gen(K), pad=3, offset=1)
    x[1] = 0
    x[2] *= 1e-36                # the lifted range: 127 / max|x| would overflow
    x[3] *= 1e30
    if K > 8:
        x[4, 5] = float("nan")
        x[5, 6] = -float("inf")
    codes, ok_q = guarded(T, K, torch.int8)
    codes, scales = quantise(x, codes=codes)
    R.check_codes(codes.cpu().numpy(), f64(scales), f64(x), 0.0, "codes")
    out, ok_o = guarded(T, K, BF16)
    back = dequantise(codes, scales, out=out)
    v = f64(codes) * f64(scales)[:, None]
    R.check(f64(back), v, np.abs(v) * (R.B + R.U) + 2.0 ** -133, "values")
    assert ok_q() and ok_o()


def test_no_tokens():
    from mxfp4_latent_mixture_sigmoid_amd import Int8Linear, dequantise, quantise, rms_norm
    x = torch.empty(0, 96, dtype=BF16, device="cuda")
    r = rms_norm(x, delta=x, sum=True, codes=True)
    assert r.out.shape == r.codes.shape == (0, 96) and r.scales.shape == (0,)
    q, s = quantise(x)
    assert dequantise(q, s).shape == (0, 96)
    w = torch.ones(40, 96, dtype=torch.int8, device="cuda")
    assert Int8Linear(w, torch.ones(40, device="cuda"), T_max=0).forward(q, s).shape == (0, 40)


def make(N, K, glu, g, bias=False, **kw):
    from mxfp4_latent_mixture_sigmoid_amd import Int8Linear
    w = [torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8).cuda() for _ in range(1 + glu)]
    # products of a few units: codes of deviation ~74 each, so sums of ~5500 sqrt(K)
    s = [((0.5 + torch.rand(N, generator=g)) / (2000 * K ** 0.5)).cuda() for _ in range(1 + glu)]
    b = torch.randn(N, generator=g).cuda() if bias else None
    layer = Int8Linear(w[0], s[0], bias=b, up_codes=w[1] if glu else None, up_scales=s[1] if glu else None, **kw)
    return layer, [t.cpu().numpy() for t in w], [f64(t) for t in s], None if b is None else f64(b)


def reference(x, sx, w, s, b, bf16):
    """(result, allowed error). One rounding of the sum to FP32 and two of the scalings: 3 u of a product;
    the gate's error reaches silu through exp(-g), at most |g| times relative; the FP32 functions
    themselves a few units."""
    p = R.product(x, w[0], sx, s[0])
    if len(w) == 2:
        u = R.product(x, w[1], sx, s[1])
        ref = R.silu(p) * u
        err = np.abs(ref) * ((24 + 6 * np.abs(p)) * R.U) + np.abs(u) * 2.0 ** -120
    else:
        ref = p + (0 if b is None else b)
        err = 4 * R.U * (np.abs(p) + (0 if b is None else np.abs(b)))
    return ref, err + (np.abs(ref) * R.B + 2.0 ** -133 if bf16 else 0)


SIZES = [  # T, N, K, pad of x, offset of x: both sides of 16-row and 128-code blocks and of the tiles
    (1, 1, 1, 0, 0), (1, 16, 128, 0, 0), (1, 700, 3584, 0, 0), (2, 17, 127, 0, 1), (3, 100, 129, 7, 0),
    (15, 64, 64, 0, 0), (16, 65, 144, 0, 0), (17, 31, 1000, 8, 0), (31, 96, 272, 0, 3), (33, 48, 256, 16, 16),
    (63, 200, 1111, 0, 0), (64, 129, 2048, 0, 0), (65, 127, 640, 0, 0), (100, 333, 777, 5, 2), (128, 256, 512, 0, 0),
    (129, 257, 513, 0, 0), (200, 1000, 384, 0, 0), (256, 64, 4352, 0, 0), (300, 520, 96, 0, 0), (777, 1001, 1535, 1, 0),
    (1500, 272, 160, 0, 0), (64, 3000, 7168, 0, 0), (40, 2064, 14336, 0, 0), (513, 515, 130, 0, 0),
    # rows at odd addresses: through registers (from 16 codes on) in every tile, or restaged
    (5, 40, 15, 0, 1), (5, 40, 16, 1, 1), (7, 33, 31, 0, 0), (1, 3500, 257, 0, 7), (16, 7000, 143, 0, 0),
    (16, 13000, 131, 2, 1), (32, 6200, 129, 0, 1), (30, 25000, 100, 3, 0), (64, 6300, 200, 1, 0), (64, 13000, 155, 1, 0),
    (60, 24600, 130, 1, 0), (130, 5000, 129, 0, 1), (300, 4200, 137, 4, 0), (1000, 4000, 141, 0, 3), (700, 6000, 77, 0, 2),
    (64, 14336, 9400, 1, 0),
]


@pytest.mark.parametrize("T,N,K,pad,offset", SIZES)
@pytest.mark.parametrize("kind", ["bf16", "f32+bias", "glu", "glu f32"])
def test_products(T, N, K, pad, offset, kind):
    g = gen(T * 1000 + N + K)
    out_dtype = F32 if "f32" in kind else BF16
    layer, w, s, b = make(N, K, "glu" in kind, g, bias="bias" in kind, T_max=T, out_dtype=out_dtype)
    x = codes_rows(T, K, g, pad, offset)
    sx = (0.5 + torch.rand(T, generator=g)).cuda()
    out, ok = guarded(T, N, out_dtype)
    layer.forward(x, sx, out=out)
    ref, err = reference(x.cpu().numpy(), f64(sx), w, s, b, out_dtype is BF16)
    R.check(f64(out), ref, err, f"{kind} {T}x{N}x{K}")
    assert ok()


# (tokens, outputs, codes): whole and ragged tiles of 128 x 64, 128 x 128, 256 x 128, 256 x 224 and 256 x 256, and
# sums of one to several 128-code stages
LARGE = [(2048, 4096, 640, 0), (4100, 4200, 272, 0), (2304, 2100, 384, 1), (1030, 1100, 1024, 0), (8192, 500, 128, 0),
         (300, 9000, 256, 1), (2048, 7168, 64, 0), (2050, 7170, 100, 0), (3584, 4096, 1152, 0), (1921, 6930, 515, 0),
         (2048, 3584, 256, 1), (2300, 3900, 130, 1), (2048, 3600, 1, 1), (4096, 3584, 384, 0), (257, 6000, 336, 0),
         (1793, 7169, 3300, 0), (2000, 7000, 1500, 0), (1700, 7010, 4200, 0), (1000, 7000, 2561, 0), (2047, 3501, 1700, 1),
         (1000, 3500, 3400, 1), (300, 3000, 300, 1), (2040, 7000, 4097, 0)]


@pytest.mark.parametrize("T,N,K,glu", LARGE)
@pytest.mark.parametrize("out_dtype", [BF16, F32])
def test_products_large(T, N, K, glu, out_dtype):
    """The large tiles against exact sums in FP64 on the GPU."""
    g = gen(T + N)
    layer, w, s, b = make(N, K, glu, g, bias=not glu and N % 3 == 0, T_max=T, out_dtype=out_dtype)
    x, sx = codes_rows(T, K, g), (0.5 + torch.rand(T, generator=g)).cuda()
    buf, ok = guarded(T, N, out_dtype)
    out = layer.forward(x, sx, out=buf).double()
    assert ok()

    def product(w, s):
        w, s = torch.from_numpy(w).cuda().double(), torch.from_numpy(s).cuda()
        return (x.double() @ w.t().contiguous()) * sx.double()[:, None] * s
    p = product(w[0], s[0])
    if glu:
        u = product(w[1], s[1])
        ref = p * torch.sigmoid(p) * u
        allowed = ref.abs() * (24 + 6 * p.abs()) * R.U + u.abs() * 2.0 ** -120
    else:
        bias = 0 if b is None else torch.from_numpy(b).cuda()
        ref = p + bias
        allowed = 4 * R.U * (p.abs() + abs(bias))
    if out_dtype is BF16:
        allowed = allowed + ref.abs() * R.B + 2.0 ** -133
    over = (out - ref).abs() - allowed
    assert over.max() <= 0, (float(over.max()), int((over > 0).sum()))


@pytest.mark.parametrize("T", [1, 16, 33, 64, 65, 200])
def test_products_longest_sum(T):
    """The widest sum, every code at the end of its range: 2^31 - 2^14 does not wrap."""
    from mxfp4_latent_mixture_sigmoid_amd import Int8Linear, abi
    K, N = abi.LINEAR_MAX_K, 20
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    w[1::2] = 127
    layer = Int8Linear(w, torch.ones(N, device="cuda"), T_max=T, out_dtype=F32)
    x = torch.full((T, K), -128, dtype=torch.int8, device="cuda")
    out = f64(layer.forward(x, torch.ones(T, device="cuda")))
    assert np.array_equal(out[:, 0::2], np.full((T, N // 2), np.float64(np.float32(128 * 128 * K))))
    assert np.array_equal(out[:, 1::2], np.full((T, N // 2), np.float64(np.float32(-128 * 127 * K))))


@pytest.mark.parametrize("T", [3, 70])
@pytest.mark.parametrize("glu", [0, 1])
def test_products_of_a_row_without_scale(T, glu):
    """A NaN scale marks its own row and no other; a zero scale gives zeros (or the bias)."""
    g = gen(5)
    layer, w, s, b = make(50, 300, glu, g, bias=not glu, T_max=T, out_dtype=F32)
    x, sx = codes_rows(T, 300, g), torch.ones(T, device="cuda")
    sx[1], sx[2] = float("nan"), 0.0
    out = layer.forward(x, sx)
    assert torch.isnan(out[1]).all() and torch.isfinite(out[0]).all() and torch.isfinite(out[2:]).all()
    R.check(f64(out[2]), np.zeros(50) if glu else b, 0.0, "zero scale")


def test_gate_far_out():
    """Gates whose exponential overflows or vanishes: 0 and the gate itself."""
    from mxfp4_latent_mixture_sigmoid_amd import Int8Linear
    w = torch.tensor([[100], [-100]], dtype=torch.int8, device="cuda").repeat(8, 16)
    one = torch.ones(16, device="cuda")
    layer = Int8Linear(w, one, up_codes=w.abs(), up_scales=one, T_max=1, out_dtype=F32)
    out = layer.forward(torch.ones(1, 16, dtype=torch.int8, device="cuda"), one[:1])[0]
    assert (out[0::2] == 1600.0 * 1600.0).all() and (out[1::2] == 0).all()


def test_outputs_past_32_bit_offsets():
    """More than 2^31 outputs and code rows: the last rows and those around the boundary."""
    from mxfp4_latent_mixture_sigmoid_amd import dequantise, quantise, rms_norm
    N, K, T = 32768, 16, 66000
    g = gen(9)
    layer, w, s, _ = make(N, K, 0, g, T_max=T)
    x, sx = codes_rows(T, K, g), (0.5 + torch.rand(T, generator=g)).cuda()
    out = layer.forward(x, sx)
    pick = [0, 65535, 65536, 65537, T - 1]
    ref, err = reference(x[pick].cpu().numpy(), f64(sx[pick]), w, s, None, True)
    R.check(f64(out[pick]), ref, err, "out")
    codes, scales = quantise(out)
    y = f64(out[pick])
    R.check_codes(codes[pick].cpu().numpy(), f64(scales[pick]), y, 0.0, "codes")
    back = f64(dequantise(codes, scales)[pick])
    v = f64(codes[pick]) * f64(scales[pick])[:, None]
    R.check(back, v, np.abs(v) * (R.B + R.U) + 2.0 ** -133, "values")
    del codes, scales
    total = rms_norm(out, delta=out, sum=out).out
    s2, y2 = R.norm(2 * y, None, None, float(np.float32(1e-6)))
    R.check(f64(out[pick]), s2, np.abs(s2) * R.B, "sum")
    R.check(f64(total[pick]), y2, np.abs(y2) * (R.B + R.NORM_REL), "norm")


def test_more_rows_than_one_launch_takes():
    from mxfp4_latent_mixture_sigmoid_amd import dequantise, quantise, rms_norm
    T, H = 2 ** 21 + 5, 40
    g = gen(12)
    x = torch.randn(997, H, generator=g).bfloat16().cuda().repeat(T // 997 + 1, 1)[:T]
    pick = [0, 996, 2 ** 21 - 1, 2 ** 21, T - 1]
    r = rms_norm(x, delta=x, sum=True, codes=True)
    s, y = R.norm(2 * f64(x[pick]), None, None, float(np.float32(1e-6)))
    R.check(f64(r.sum[pick]), s, np.abs(s) * R.B, "sum")
    R.check(f64(r.out[pick]), y, np.abs(y) * (R.B + R.NORM_REL), "out")
    R.check_codes(r.codes[pick].cpu().numpy(), f64(r.scales[pick]), y, R.NORM_REL, "codes")
    codes, scales = quantise(x)
    assert torch.equal(codes[997:], codes[:-997]) and torch.equal(scales[997:], scales[:-997])
    assert torch.equal(dequantise(codes[:997], scales[:997]), dequantise(codes, scales)[:997])


def block(H, I, T_max, g):
    from mxfp4_latent_mixture_sigmoid_amd import Int8FeedForward
    mat = lambda n, k: (torch.randint(-127, 128, (n, k), generator=g, dtype=torch.int8).cuda(),      # noqa: E731
                        ((0.5 + torch.rand(n, generator=g)) / (73 * k ** 0.5)).cuda())
    m = (mat(I, H), mat(I, H), mat(H, I))
    nw = (1 + 0.1 * torch.randn(H, generator=g)).bfloat16().cuda()
    return Int8FeedForward(nw, *m, T_max=T_max), nw, m


@pytest.mark.parametrize("T", [1, 5, 64, 130])
def test_block(T):
    """norm -> gated product -> quantisation -> down product, each step against the plain form of the
    step's own inputs (codes may differ by one where a value lies between two)."""
    from mxfp4_latent_mixture_sigmoid_amd import quantise, rms_norm
    H, I, g = 384, 640, gen(T)
    ff, nw, (gate, up, down) = block(H, I, T, g)
    x, d = rows(T, H, BF16, g), rows(T, H, BF16, g)
    y, total = ff.forward(x, delta=d)
    r = rms_norm(x, nw, ff.eps, delta=d, sum=True, out=False, codes=True)
    assert torch.equal(total, r.sum)
    num = lambda p: (p[0].cpu().numpy(), f64(p[1]))                                                   # noqa: E731
    h = ff.gated.forward(r.codes, r.scales)
    ref, err = reference(r.codes.cpu().numpy(), f64(r.scales), [num(gate)[0], num(up)[0]], [num(gate)[1], num(up)[1]],
                         None, True)
    R.check(f64(h), ref, err, "h")
    q, s = quantise(h)
    ref, err = reference(q.cpu().numpy(), f64(s), [num(down)[0]], [num(down)[1]], None, True)
    R.check(f64(y), ref, err, "y")
    assert torch.equal(ff.forward(total)[0], ff.forward(total)[0])


@pytest.mark.parametrize("T", [2, 64, 150])
def test_block_on_another_stream(T):
    H, I, g = 512, 768, gen(T)
    ff, _, _ = block(H, I, T, g)
    x, d = rows(T, H, BF16, g), rows(T, H, BF16, g)
    want, _ = ff.forward(x, delta=d)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, _ = ff.forward(x, delta=d, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


@pytest.mark.parametrize("T", [1, 40, 200])
def test_block_in_a_graph(T):
    """One captured block, replayed on new inputs with eager work and synchronisations between."""
    H, I, g = 512, 768, gen(T)
    ff, _, _ = block(H, I, T, g)
    x, d = rows(T, H, BF16, g), rows(T, H, BF16, g)
    ff.forward(x, delta=d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, total = ff.forward(x, delta=d)
    for k in range(4):
        x.copy_(rows(T, H, BF16, g))
        graph.replay()
        if k % 2:
            torch.cuda.synchronize()
        got, got_total = y.clone(), total.clone()
        want, want_total = ff.forward(x, delta=d)
        assert torch.equal(got, want) and torch.equal(got_total, want_total), k


def test_calls_repeat_bit_for_bit_and_interleave():
    """Layers of different sizes called in turn on one stream, every result as on its own."""
    g = gen(77)
    made = []
    for T, N, K in [(64, 640, 2048), (1, 320, 4096), (300, 500, 600), (17, 1000, 1536)]:
        layer, *_ = make(N, K, 0, g, T_max=T)
        made.append((layer, codes_rows(T, K, g), torch.ones(T, device="cuda")))
    alone = []
    for layer, x, sx in made:
        alone.append(layer.forward(x, sx))
        torch.cuda.synchronize()
    for _ in range(3):
        again = [layer.forward(x, sx) for layer, x, sx in made]
        for a, b in zip(again, alone):
            assert torch.equal(a, b)


def test_smaller_calls_of_a_larger_layer():
    """Every T up to T_max in one workspace, some after larger calls left their data in it."""
    g = gen(3)
    T, N, K = 150, 200, 900
    layer, w, s, _ = make(N, K, 0, g, T_max=T)
    x, sx = codes_rows(T, K, g), (0.5 + torch.rand(T, generator=g)).cuda()
    ref, err = reference(x.cpu().numpy(), f64(sx), w, s, None, True)
    for t in (150, 1, 64, 65, 16, 17, 149, 33):
        R.check(f64(layer.forward(x[:t], sx[:t])), ref[:t], err[:t], f"T={t}")


# (tokens, outputs, gated, 128-code stages up to): one for each tile of few tokens and of the smaller ones of many
STAGES = [(1, 300, 0, 80), (16, 3000, 1, 90), (16, 13000, 0, 40), (16, 25000, 0, 16), (32, 3584, 0, 80), (32, 7168, 0, 60),
          (31, 6200, 1, 30), (30, 25000, 0, 12), (64, 7168, 0, 30), (63, 6500, 1, 30), (60, 24600, 0, 12), (20, 2000, 1, 90),
          (777, 1001, 0, 30), (150, 7168, 0, 12), (300, 6000, 0, 12), (600, 7000, 0, 12)]


@pytest.mark.parametrize("T,N,glu,most", STAGES)
def test_every_number_of_stages(T, N, glu, most):
    """K axes that end at each place of the loops over stages: sums that FP32 holds exactly, with direct and with
    unaligned rows. Gated: the up half, whose gate is a constant, against the same sums
    (the reciprocal is within 2 U, two products and the expectation round once each)."""
    from mxfp4_latent_mixture_sigmoid_amd import Int8Linear
    g = torch.Generator(device="cuda").manual_seed(T)
    for s in range(1, most + 1, 1 if most <= 16 else 1 + (T + N) % 2):
        K = 128 * s - 16 * (s % 3)
        w = torch.randint(-9, 10, (N, K), generator=g, dtype=torch.int8, device="cuda")
        x = torch.randint(-9, 10, (T, K + 5), generator=g, dtype=torch.int8, device="cuda")
        one, sx = torch.ones(N, device="cuda"), torch.ones(T, device="cuda")
        if glu:   # the gate's sums are 127 * 9 or more, times 2^-3: silu is the identity there
            x[:, 0] = 9
            gate = torch.zeros_like(w)
            gate[:, 0] = 127
            layer = Int8Linear(gate, one / 8, up_codes=w, up_scales=one, T_max=T, out_dtype=F32)
        else:
            layer = Int8Linear(w, one, T_max=T, out_dtype=F32)
        want = x[:, :K].float() @ w.t().float().contiguous()
        want *= 9 * 127 / 8 if glu else 1
        for rows in (x[:, :K].contiguous(), x[:, :K]):
            got = layer.forward(rows, sx)
            if glu:
                assert ((got - want).abs() <= 5 * R.U * want.abs()).all(), s
            else:
                assert torch.equal(got, want), s


@pytest.mark.parametrize("N,K,glu,out_dtype", [(7168, 400, 0, BF16), (7168, 272, 0, F32), (3584, 640, 1, BF16),
                                               (3601, 130, 1, F32), (300, 4000, 0, F32), (6200, 257, 0, F32)])
def test_a_token_in_any_batch(N, K, glu, out_dtype):
    """A token's outputs are the same bits whatever batch, tile and row address it comes with."""
    g = gen(N)
    layer, *_ = make(N, K, glu, g, bias=not glu, T_max=2304, out_dtype=out_dtype)
    x, sx = codes_rows(2304, K, g), (torch.rand(2304, generator=g) - 0.5).cuda()
    whole = layer.forward(x, sx)
    apart = codes_rows(1200, K, g, pad=3, offset=1)
    for first, T in ((0, 1), (5, 7), (100, 16), (33, 17), (800, 33), (64, 64), (7, 100), (1000, 129), (50, 300),
                     (11, 520), (0, 1100), (1200, 1104)):
        assert torch.equal(layer.forward(x[first:first + T], sx[first:first + T]), whole[first:first + T]), T
        if T <= 1200:
            apart[:T].copy_(x[first:first + T])
            assert torch.equal(layer.forward(apart[:T], sx[first:first + T]), whole[first:first + T]), (T, "unaligned")


@pytest.mark.parametrize("N,K,glu", [(7168, 4300, 0), (3584, 3000, 1), (6101, 4112, 0)])
@pytest.mark.parametrize("out_dtype", [BF16, F32])
def test_a_token_in_any_large_batch(N, K, glu, out_dtype):
    """The same with K axes long enough for every tile of many tokens."""
    g = gen(N + 1)
    layer, *_ = make(N, K, glu, g, bias=not glu, T_max=2304, out_dtype=out_dtype)
    x, sx = codes_rows(2304, K, g), (torch.rand(2304, generator=g) - 0.5).cuda()
    whole = layer.forward(x, sx)
    for first, T in ((3, 61), (1, 200), (77, 300), (640, 520), (200, 1000), (9, 1104), (500, 1700), (304, 2000)):
        assert torch.equal(layer.forward(x[first:first + T], sx[first:first + T]), whole[first:first + T]), T


def test_views_and_weights_in_any_order():
    """Activations and outputs that are columns of wider buffers, single rows with arbitrary strides,
    weights that are transposed views: the bits of contiguous ones."""
    from mxfp4_latent_mixture_sigmoid_amd import Int8Linear, quantise, rms_norm
    g = gen(21)
    w = torch.randint(-128, 128, (96, 320), generator=g, dtype=torch.int8).cuda()
    s = torch.rand(96, generator=g).cuda()
    a = Int8Linear(w, s, T_max=40)
    b = Int8Linear(w.t().contiguous().t(), s, T_max=40)
    big = torch.randint(-128, 128, (40, 400), generator=g, dtype=torch.int8).cuda()
    sx = torch.rand(40, generator=g).cuda()
    want = a.forward(big[:, 37:357].contiguous(), sx)
    wide = torch.zeros(40, 300, dtype=BF16, device="cuda")
    assert b.forward(big[:, 37:357], sx, out=wide[:, 100:196]) is not None
    assert torch.equal(wide[:, 100:196], want) and not wide[:, :100].any() and not wide[:, 196:].any()
    one = big[7:8, 37:357]
    assert torch.equal(a.forward(one, sx[7:8]), want[7:8])
    assert torch.equal(a.forward(one.as_strided((1, 320), (1, 1), one.storage_offset()), sx[7:8]), want[7:8])
    x = torch.randn(40, 400, generator=g).bfloat16().cuda()
    for f in (lambda t: rms_norm(t).out, lambda t: quantise(t)[0], lambda t: quantise(t)[1]):
        assert torch.equal(f(x[::2, 3:333]), f(x[::2, 3:333].contiguous()))


def test_python_refusals():
    from mxfp4_latent_mixture_sigmoid_amd import Int8Linear, dequantise, quantise, rms_norm
    x = torch.zeros(4, 32, dtype=BF16, device="cuda")
    q = torch.zeros(4, 32, dtype=torch.int8, device="cuda")
    s = torch.ones(4, device="cuda")
    bad = [lambda: rms_norm(x.half()), lambda: rms_norm(x.t()), lambda: rms_norm(x.cpu()), lambda: rms_norm(x[0]),
           lambda: rms_norm(x, weight=torch.ones(31, dtype=BF16, device="cuda")), lambda: rms_norm(x, delta=x[:3]),
           lambda: rms_norm(x, weight=torch.ones(32, device="cuda")), lambda: rms_norm(x, scales=s),
           lambda: rms_norm(x, out=x.float()), lambda: quantise(q), lambda: dequantise(x, s),
           lambda: dequantise(q, s[:3]), lambda: dequantise(q, s.double()),
           lambda: Int8Linear(x, s), lambda: Int8Linear(q, s[:3]), lambda: Int8Linear(q, s, up_codes=q),
           lambda: Int8Linear(q, s, out_dtype=torch.float16), lambda: Int8Linear(q, s, bias=s, up_codes=q, up_scales=s)]
    layer = Int8Linear(q, s, T_max=4)
    bad += [lambda: layer.forward(q[:, :31], s), lambda: layer.forward(torch.cat([q, q]), torch.cat([s, s])),
            lambda: layer.forward(q, s[:2]), lambda: layer.forward(x, s),
            lambda: layer.forward(q, s, out=torch.empty(4, 5, dtype=BF16, device="cuda"))]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"case {i} was accepted")
    layer.close()
    with pytest.raises(RuntimeError):
        layer.forward(q, s)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("K", [40, 500, 1000, 2500, 4000, 7168, 14336, 17000])
def test_codes_are_the_quotients_by_the_stored_scale(K, dtype):
    """scales = max|x| / 127 and codes = x / scale, each one FP32 division rounded once, bit for bit; many of the
    values lie as near to a half between two codes as their type allows."""
    from mxfp4_latent_mixture_sigmoid_amd import quantise
    T, g = 60, gen(K)
    top = torch.exp(2 * torch.randn(T, 1, generator=g)).to(dtype).float()
    half = torch.randint(-127, 127, (T, K), generator=g) + 0.5
    x = (top / 127 * half).to(dtype)
    bits = {BF16: torch.int16, F32: torch.int32}[dtype]
    x = (x.view(bits) + torch.randint(-1, 2, (T, K), generator=g).to(bits)).view(dtype)
    x[:, :1] = top.to(dtype)
    x[50:55] *= 2.0 ** -80       # rows that are lifted first
    x[55:60] *= 2.0 ** 90
    codes, scales = quantise(x.cuda())
    f = x.float().numpy()
    want = np.abs(f).max(1) / np.float32(127)
    assert want.dtype == np.float32 and np.array_equal(scales.cpu().numpy(), want)
    assert np.array_equal(codes.cpu().numpy(), np.rint(f / want[:, None]).astype(np.int8))


# one for each large tile, plain and gated: 128 x 64, 128 x 128, 256 x 128, 256 x 224, 256 x 256
TILES = [(500, 4090, 128, 0), (1000, 4090, 128, 0), (1000, 8000, 3000, 0), (1800, 6900, 4096, 0), (2040, 8190, 2500, 0),
         (500, 2040, 128, 1), (1000, 2040, 128, 1), (1020, 3500, 3400, 1), (2040, 3500, 3000, 1)]


@pytest.mark.parametrize("T,N,K,glu", TILES)
def test_every_output_of_the_large_tiles(T, N, K, glu):
    """Outputs change hands between a wave's lanes on their way out: every one exact, in both types, call after call.
    Gated: a gate of 127 * 9 / 8, whose silu is the value itself; 8 U for the hardware's exponential and
    reciprocal and the products (and half a BF16 unit)."""
    from mxfp4_latent_mixture_sigmoid_amd import Int8Linear
    g = torch.Generator(device="cuda").manual_seed(N)
    w = torch.randint(-9, 10, (N, K), generator=g, dtype=torch.int8, device="cuda")
    x = torch.randint(-9, 10, (T, K), generator=g, dtype=torch.int8, device="cuda")
    one, sx = torch.ones(N, device="cuda"), torch.ones(T, device="cuda")
    gate = torch.zeros_like(w)
    gate[:, 0] = 127
    if glu:
        x[:, 0] = 9
    want = (x.float() @ w.t().float().contiguous()) * (9 * 127 / 8 if glu else 1)   # whole numbers below 2^24
    for dtype in (F32, BF16):
        kw = dict(T_max=T, out_dtype=dtype)
        layer = Int8Linear(gate, one / 8, up_codes=w, up_scales=one, **kw) if glu else Int8Linear(w, one, **kw)
        out, ok = guarded(T, N, dtype)
        for _ in range(3):
            out.zero_()
            layer.forward(x, sx, out=out)
            if glu:
                assert ((out.float() - want).abs() <= (8 * R.U + (R.B if dtype is BF16 else 0)) * want.abs()).all()
            else:
                assert torch.equal(out, want.to(dtype))
        assert ok()


@pytest.mark.parametrize("given", [False, True])
def test_memory_of_a_layer_dropped_while_it_runs(given):
    """A layer built on one stream, called on a busy other one and dropped: its packed weights are not handed out
    again before that call is done, and its result is right."""
    g = gen(8)
    layer, w, s, _ = make(512, 1024, 0, g, T_max=64)
    x, sx = codes_rows(64, 1024, g), torch.ones(64, device="cuda")
    want = layer.forward(x, sx)
    torch.cuda.synchronize()
    at, size = layer.packed.data_ptr(), layer.packed.numel()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    if given:
        got = layer.forward(x, sx, stream=side)
    else:
        with torch.cuda.stream(side):
            got = layer.forward(x, sx)
    del layer
    taken = [torch.full((size,), 1, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(t.data_ptr() != at for t in taken)
    side.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("H", [600, 1000, 1024, 2040, 2561, 3000, 4096, 4097, 5120, 5121, 7168, 8192, 9000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_row_s_norm_in_any_batch(H, dtype):
    """A row's norm is the same bits whatever batch it comes with (1024 rows take other kernels than 1023)."""
    from mxfp4_latent_mixture_sigmoid_amd import quantise, rms_norm
    T, g = 1500, gen(H)
    x, d = rows(T, H, dtype, g, sigma=2.0), rows(T, H, BF16, g)
    w = (1 + 0.1 * torch.randn(H, generator=g)).bfloat16().cuda()
    whole, plain = rms_norm(x, w, delta=d, sum=True, codes=True), quantise(x)
    for first, n in ((0, 1), (7, 64), (300, 1023), (400, 1024), (100, 1400)):
        part = slice(first, first + n)
        for a, b in zip(rms_norm(x[part], w, delta=d[part], sum=True, codes=True), whole):
            assert torch.equal(a, b[part]), n
        for a, b in zip(quantise(x[part]), plain):
            assert torch.equal(a, b[part]), n


def test_a_block_s_token_in_any_batch():
    H, I, T, g = 3000, 1000, 1300, gen(4)
    ff, _, _ = block(H, I, T, g)
    x, d = rows(T, H, BF16, g), rows(T, H, BF16, g)
    y, total = ff.forward(x, delta=d)
    for first, n in ((0, 1), (5, 64), (200, 1000), (100, 1100)):
        a, b = ff.forward(x[first:first + n], delta=d[first:first + n])
        assert torch.equal(a, y[first:first + n]) and torch.equal(b, total[first:first + n]), n


@pytest.mark.parametrize("H", [64, 700, 1500, 3000, 7168, 9000, 20000])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6, 1e30])
def test_norm_of_rows_whose_squares_leave_the_range(H, dtype, eps):
    """Rows up to both ends of the type: their squares overflow or vanish, their norm does not. (Bounds as
    elsewhere, and a BF16 subnormal's half unit, 2^-134.)"""
    from mxfp4_latent_mixture_sigmoid_amd import rms_norm
    g, eps32 = gen(H), float(np.float32(eps))
    sizes = [1.0, 1e15, 2e17, 1e19, 1e25, 3e37, 1e-12, 1e-18, 1e-22, 1e-30, 1e-36, 1e-38, 3e-40, 1e-44]
    x = (torch.randn(len(sizes) + 2, H, generator=g).clamp(-9, 9).double()
         * torch.tensor(sizes + [1.0, 0.0]).double()[:, None]).to(dtype)
    x[len(sizes), 3] = 2.0 ** 120           # one value that is all of the row's norm
    for n in (1, 1100 if H in (3000, 7168) else 2):
        xs = x.cuda().repeat(n, 1)
        w = (1 + 0.1 * torch.randn(H, generator=g)).bfloat16().cuda()
        r = rms_norm(xs, w, eps, codes=True)
        _, y = R.norm(f64(x), None, f64(w), eps32)
        live = np.isfinite(y).all(1)         # 0 / 0 in a row of zeros, as the formula has it
        assert live.sum() >= len(sizes) - (dtype is BF16)
        for part in (slice(0, len(x)), slice((n - 1) * len(x), n * len(x))):
            out, scales, codes = f64(r.out[part]), f64(r.scales[part]), r.codes[part].cpu().numpy()
            R.check(out[live], y[live], np.abs(y[live]) * (R.B + R.NORM_REL) + 2.0 ** -133, "out")
            big = live & (np.abs(y).max(1) > 1e-30)      # scales with all their bits
            R.check_codes(codes[big], scales[big], y[big], R.NORM_REL, "codes")
            assert np.isnan(out[~live]).all()


def test_workspace_only_where_rows_are_laid_out_first():
    """Aligned rows need no workspace; many unaligned ones are refused without one, with nothing written."""
    from mxfp4_latent_mixture_sigmoid_amd import abi
    g, (T, N, K) = gen(31), (1000, 4000, 144)
    layer, w, s, _ = make(N, K, 0, g, T_max=8192)
    held = [v.numel() for v in vars(layer).values() if torch.is_tensor(v)]
    assert held == [abi.linear_query(layer.cfg, 8192)[0]]   # the packed weights, not T_max rows as well
    x, sx = codes_rows(T, K, g), torch.ones(T, device="cuda")
    apart = codes_rows(T, K, g, pad=1, offset=3)
    apart.copy_(x)
    out, ok = guarded(T, N, BF16)
    size = abi.linear_query(layer.cfg, T)[1]
    room = torch.empty(size, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream

    def call(rows, at, size):
        return abi.lib().moe_linear_forward(layer.handle, rows.data_ptr(), rows.stride(0), sx.data_ptr(), T, out.data_ptr(),
                                            out.stride(0), at, size, stream)
    for at, n, want in ((None, 0, abi.Status.BUFFER_TOO_SMALL), (room.data_ptr(), size - 1, abi.Status.BUFFER_TOO_SMALL),
                        (None, size, abi.Status.INVALID_ARG), (room.data_ptr() + 64, size, abi.Status.INVALID_ARG)):
        assert call(apart, at, n) == want
    torch.cuda.synchronize()
    assert (out == 77).all()
    assert call(x, None, 0) == abi.Status.OK
    aligned = out.clone()
    out.zero_()
    assert call(apart, room.data_ptr(), size) == abi.Status.OK
    assert torch.equal(out, aligned) and ok()
    ref, err = reference(x.cpu().numpy(), f64(sx), w, s, None, True)
    R.check(f64(aligned), ref, err, "aligned")


def test_unaligned_calls_of_one_layer_on_two_streams():
    """Calls that lay their rows out first, of one layer, overlapping on two streams: each has room of its own."""
    g, (T, N, K) = gen(32), (2000, 4000, 1001)
    layer, *_ = make(N, K, 0, g, T_max=T)
    xs, sx = [codes_rows(T, K, g) for _ in range(2)], torch.ones(T, device="cuda")
    want = [layer.forward(x, sx) for x in xs]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(10):
        for k, (x, side) in enumerate(zip(xs, sides)):
            got[k].append(layer.forward(x, sx, stream=side))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[k]) for k in (0, 1) for y in got[k])


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_codes_of_every_width(H, dtype):
    """Codes and scales of rows whose residual cancels nowhere (x and delta of one sign), so that they are known to
    the norm's own error at every width."""
    from mxfp4_latent_mixture_sigmoid_amd import rms_norm
    T, g = 5, gen(H + 1)
    x, d = rows(T, H, dtype, g, pad=3, offset=1), rows(T, H, BF16, g, pad=2)
    d.copy_(d.abs() * x.sign().to(BF16))
    w = (1 + 0.1 * torch.randn(H, generator=g)).bfloat16().cuda()
    codes, ok = guarded(T, H, torch.int8)
    r = rms_norm(x, w, 1e-5, delta=d, out=False, codes=codes)
    _, y = R.norm(f64(x), f64(d), f64(w), float(np.float32(1e-5)))
    R.check_codes(r.codes.cpu().numpy(), f64(r.scales), y, R.NORM_REL + 2 * R.U, "codes")
    assert ok()


@pytest.mark.parametrize("H", [70001, 2 ** 20, 2 ** 24 + 3])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_of_long_rows_of_equal_values(H, dtype):
    """The sum of very many squares is as exact as that of a few: scale = value / rms / 127 to the norm's error."""
    from mxfp4_latent_mixture_sigmoid_amd import rms_norm
    for value in (1.1, 0.3):
        x = torch.full((2, H), value, dtype=dtype, device="cuda")
        x[1, ::2] *= -2
        r = rms_norm(x, eps=1e-6, codes=True)
        v = f64(x[:, :2])                                     # each row repeats its first two values
        odd = H % 2
        mean = ((H + odd) // 2 * v[:, 0] ** 2 + (H // 2) * v[:, 1] ** 2) / H
        y = v / np.sqrt(mean + float(np.float32(1e-6)))[:, None]
        R.check_codes(r.codes[:, :2].cpu().numpy(), f64(r.scales), y, R.NORM_REL, "codes")
        R.check(f64(r.out[:, :2]), y, np.abs(y) * (R.B + R.NORM_REL), "out")
        assert torch.equal(r.codes[:, 2:4], r.codes[:, :2]) and torch.equal(r.out[:, -2:].sort(1)[0], r.out[:, :2].sort(1)[0])


@pytest.mark.parametrize("T,N,K", [(600, 4096, 2047), (5, 40, 15)])
def test_rows_laid_out_first_in_a_graph(T, N, K):
    """A captured call that allocates room for its rows, replayed on new codes with eager calls of the layer between."""
    g = gen(K)
    layer, *_ = make(N, K, 0, g, T_max=T)
    x, sx = codes_rows(T, K, g, pad=2, offset=1), torch.ones(T, device="cuda")
    layer.forward(x, sx)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.forward(x, sx)
    other = codes_rows(T, K, g, pad=2, offset=1)
    for k in range(4):
        x.copy_(codes_rows(T, K, g))
        graph.replay()
        noise = layer.forward(other, sx)
        if k % 2:
            torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, layer.forward(x, sx)) and torch.equal(noise, layer.forward(other, sx)), k
