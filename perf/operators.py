"""What is measured of the dense 8-bit path around the mixture layer: RMS norm with the residual's
addition, quantisation per token, the 8-bit product with scales, and the gated 8-bit product.

The four operators, for T tokens (codes are whole numbers in [-127, 127], one scale per row):

  norm      s = x + delta;  y = s * rsqrt(mean(s^2) + eps) * weight;  y in BF16 and / or in 8 bits
  quantise  scale[t] = max_k |x[t, k]| / 127;  codes[t, k] = round(x[t, k] / scale[t])
  linear    out[t, n] = sx[t] * sw[n] * sum_k codes[t, k] * w[n, k] + bias[n]
  glu       g, u: two such products over the same codes;  out = g / (1 + exp(-g)) * u

Values held in 8 bits are returned as the numbers they stand for (codes * scale, in BF16).
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token before the router: the latency of the call itself
        dict(name="norm_t1", op="norm", T=1, H=7168, stream="bf16", delta=True, weight=True, out="bf16", pad=0),
        # a decode batch, 8-bit input of the dense products
        dict(name="norm_i8_t64", op="norm", T=64, H=7168, stream="bf16", delta=True, weight=True, out="i8", pad=0),
        # a prompt, residual stream in 32 bits, both forms of the normalised rows
        dict(name="norm_both_t8192", op="norm", T=8192, H=7168, stream="f32", delta=True, weight=True, out="both", pad=0),
        # an odd width in a wider buffer, so that rows start at every alignment; no residual
        dict(name="norm_odd_t1000", op="norm", T=1000, H=3581, stream="bf16", delta=False, weight=True, out="both", pad=6),
        # the feed-forward's inner values of a decode batch
        dict(name="quantise_t64", op="quantise", T=64, H=14336, stream="bf16", pad=0),
        # ... and of a prompt
        dict(name="quantise_t8192", op="quantise", T=8192, H=14336, stream="bf16", pad=0),
        # latent down-projection of one token: a pass over the weights
        dict(name="linear_t1", op="linear", T=1, N=3584, K=7168, out="bf16", bias=False, pad=0),
        # output product of a decode batch (latent and shared columns side by side)
        dict(name="linear_t64", op="linear", T=64, N=7168, K=4352, out="bf16", bias=False, pad=0),
        # ragged in every size, with a bias, in 32 bits
        dict(name="linear_odd_t777", op="linear", T=777, N=1001, K=3583, out="f32", bias=True, pad=5),
        # down product of a prompt
        dict(name="linear_t8192", op="linear", T=8192, N=7168, K=14336, out="bf16", bias=False, pad=0),
        # gate and up of a decode batch
        dict(name="glu_t64", op="glu", T=64, N=14336, K=7168, out="bf16", bias=False, pad=0),
        # gate and up of a prompt
        dict(name="glu_t8192", op="glu", T=8192, N=14336, K=7168, out="bf16", bias=False, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Half of the widths any whole number, half multiples of 128, as a model's are."""
    w = _log(rng, lo, hi)
    return w if rng.random() < 0.5 else max(128, w // 128 * 128)


def draw(rng):
    op = rng.choice(["norm", "norm", "quantise", "linear", "linear", "glu", "glu"])
    T = _log(rng, 1, 8192)
    pad = rng.choice([0, 0, 0, rng.randrange(1, 64)])
    if op in ("norm", "quantise"):
        case = dict(op=op, T=T, H=_width(rng, 128, 14336), stream=rng.choice(["bf16", "f32"]), pad=pad)
        if op == "norm":
            case |= dict(delta=rng.random() < 0.7, weight=rng.random() < 0.8, out=rng.choice(["bf16", "i8", "both"]))
            case["T"] = max(1, min(T, 8192 * 7168 // case["H"]))
        return case
    N, K = _width(rng, 128, 14336), _width(rng, 128, 14336)
    most = 8192 * 14336 * 7168
    T = max(1, min(T, most // (N * K)))
    return dict(op=op, T=T, N=N, K=K, out=rng.choice(["bf16", "bf16", "f32"]) if op == "linear" else "bf16",
                bias=op == "linear" and rng.random() < 0.4, pad=pad)


def _rows(T, width, pad, fill, dtype, gen):
    """[T, width] rows of a buffer `pad` values wider."""
    t = torch.empty(T, width + pad, dtype=dtype, device="cuda")
    return fill(t, gen)[:, :width]


def _activations(t, gen):
    """Hidden states as they come: normal, a few channels an order of magnitude larger, rows of different size."""
    f = torch.randn(t.shape, generator=gen, device="cuda")
    f *= 1 + 15 * (torch.rand(t.shape[1], generator=gen, device="cuda") < 0.005)
    f *= torch.exp(0.5 * torch.randn(t.shape[0], 1, generator=gen, device="cuda"))
    return t.copy_(f)


def _codes(t, gen):
    """Codes of normal values quantised against their row's largest, about four deviations out."""
    f = torch.randn(t.shape, generator=gen, device="cuda")
    return t.copy_(f.mul_(32).round_().clamp_(-127, 127))


def _scales(n, mid, gen):
    return mid * torch.exp(0.3 * torch.randn(n, generator=gen, device="cuda"))


def _inputs(case, seed):
    """The case's inputs, from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, T, pad = case["op"], case["T"], case["pad"]
    d = {}
    if op in ("norm", "quantise"):
        H, dtype = case["H"], DTYPES[case["stream"]]
        d["x"] = _rows(T, H, pad, _activations, dtype, gen)
        if op == "norm":
            d["delta"] = _rows(T, H, pad, _activations, torch.bfloat16, gen) if case["delta"] else None
            d["weight"] = (1 + 0.2 * torch.randn(H, generator=gen, device="cuda")).bfloat16() if case["weight"] else None
        return d
    N, K = case["N"], case["K"]
    d["x"] = _rows(T, K, pad, _codes, torch.int8, gen)
    d["sx"] = _scales(T, 1 / 32, gen)
    d["w"] = _rows(N, K, 0, _codes, torch.int8, gen)
    d["sw"] = _scales(N, 1 / (32 * math.sqrt(K)), gen)
    if op == "glu":
        d["w_up"] = _rows(N, K, 0, _codes, torch.int8, gen)
        d["sw_up"] = _scales(N, 1 / (32 * math.sqrt(K)), gen)
    d["bias"] = 0.5 * torch.randn(N, generator=gen, device="cuda") if case["bias"] else None
    return d


def prepare(case, seed):
    state = dict(case=case, **_inputs(case, seed))
    if own and case["op"] in ("linear", "glu"):  # the layer that a program makes once of its weights
        from mxfp4_latent_mixture_sigmoid_amd import Int8Linear
        state["layer"] = Int8Linear(state.pop("w"), state.pop("sw"), up_codes=state.pop("w_up", None),
                                    up_scales=state.pop("sw_up", None), bias=state["bias"], T_max=case["T"],
                                    out_dtype=DTYPES[case["out"]])
    return state


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(state):
    from mxfp4_latent_mixture_sigmoid_amd import dequantise, quantise, rms_norm
    case = state["case"]
    if case["op"] == "norm":
        r = rms_norm(state["x"], state["weight"], EPS, delta=state["delta"], sum=case["delta"],
                     out=case["out"] != "i8", codes=case["out"] != "bf16")
        got = {}
        if case["delta"]:
            got["sum"] = r.sum
        if case["out"] != "i8":
            got["out"] = r.out
        if case["out"] != "bf16":
            got["held"], got["scales"] = dequantise(r.codes, r.scales), r.scales
        return got
    if case["op"] == "quantise":
        codes, scales = quantise(state["x"])
        return {"held": dequantise(codes, scales), "scales": scales}
    return {"out": state["layer"].forward(state["x"], state["sx"])}


def _held(y):
    """Rows in 8 bits with a scale each, as the numbers that they stand for; and the scales."""
    scales = y.abs().amax(1) / 127
    codes = torch.round(y / scales[:, None]).clamp(-127, 127)
    return (codes * scales[:, None]).bfloat16(), scales


def _run_plain(state):
    case = state["case"]
    if case["op"] in ("norm", "quantise"):
        s = state["x"].float()
        if case["op"] == "quantise":
            held, scales = _held(s)
            return {"held": held, "scales": scales}
        got = {}
        if case["delta"]:
            s = s + state["delta"].float()
            got["sum"] = s.to(DTYPES[case["stream"]])
        y = s * torch.rsqrt((s * s).mean(1, keepdim=True) + EPS)
        if case["weight"]:
            y = y * state["weight"].float()
        if case["out"] != "i8":
            got["out"] = y.bfloat16()
        if case["out"] != "bf16":
            got["held"], got["scales"] = _held(y)
        return got
    x = state["x"].float()
    out = (x @ state["w"].float().t()) * state["sx"][:, None] * state["sw"]
    if case["op"] == "glu":
        up = (x @ state["w_up"].float().t()) * state["sx"][:, None] * state["sw_up"]
        out = out / (1 + torch.exp(-out)) * up
    if case["bias"]:
        out = out + state["bias"]
    return {"out": out.to(DTYPES[case["out"]])}


def exact(case, seed):
    """The operators' definitions in 64 bits; what is rounded to 8 bits is rounded from those."""
    d = _inputs(case, seed)
    x = d["x"].double()

    def in_eight_bits(rows):
        top = rows.abs().max(dim=1).values
        codes = torch.round(rows * (127 / top).unsqueeze(1))
        return codes * (top / 127).unsqueeze(1), top / 127

    if case["op"] == "quantise":
        held, scales = in_eight_bits(x)
        return {"held": held, "scales": scales}
    if case["op"] == "norm":
        got = {}
        if case["delta"]:
            x = x + d["delta"].double()
            got["sum"] = x
        y = x / torch.sqrt(x.pow(2).sum(dim=1, keepdim=True) / case["H"] + EPS)
        if case["weight"]:
            y = y * d["weight"].double()
        if case["out"] in ("bf16", "both"):
            got["out"] = y
        if case["out"] in ("i8", "both"):
            got["held"], got["scales"] = in_eight_bits(y)
        return got

    def product(codes, scales):
        return torch.matmul(x * d["sx"].double().unsqueeze(1), (codes.double() * scales.double().unsqueeze(1)).t())

    y = product(d["w"], d["sw"])
    if case["op"] == "glu":
        y = y * torch.sigmoid(y) * product(d["w_up"], d["sw_up"])
    if case["bias"]:
        y = y + d["bias"].double()
    return {"out": y}


def work(case):
    """Each input read once, each result written once; additions and multiplications of the products (of the
    norm: the addition, square, sum and two scalings; of the quantisation: magnitude, comparison and scaling)."""
    op, T = case["op"], case["T"]
    if op in ("norm", "quantise"):
        H, size = case["H"], {"bf16": 2, "f32": 4}[case["stream"]]
        if op == "quantise":
            return {"bytes": T * H * (size + 1) + 4 * T, "flops": 3 * T * H}
        row = size + (2 + size if case["delta"] else 0)
        row += {"bf16": 2, "i8": 1, "both": 3}[case["out"]]
        return {"bytes": T * H * row + 2 * H * case["weight"] + (0 if case["out"] == "bf16" else 4 * T),
                "flops": T * H * (5 + 3 * (case["out"] != "bf16"))}
    N, K = case["N"], case["K"]
    mats = 2 if op == "glu" else 1
    out = {"bf16": 2, "f32": 4}[case["out"]]
    return {"bytes": T * K + mats * N * K + 4 * T + 4 * N * (mats + case["bias"]) + T * N * out,
            "flops": 2 * T * N * K * mats}
