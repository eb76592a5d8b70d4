"""What is measured of a decoder's step around the mixture layer: the norms after one block and before the next
with the gate and the residual scale between them, the dense BF16 product with bias, activation and residual in
its epilogue, and the whole mixture layer for a few tokens.

  block_norm  n = y / sqrt(mean(y^2) + eps) * post;  s = beta * x + alpha * act(gate) * n;
              out = s / sqrt(mean(s^2) + eps) * weight, in BF16 and / or in 8 bits with a scale per row
  linear      out = act(x . w^T + bias) + residual, or gated: act(x . w^T) * (x . w_up^T) + residual
  moe         logits = x . wr^T + bias;  ids = the K largest (ties to the lower index);  p = sigmoid / their sum;
              z = x . w_down^T;  y_e = (silu(z . gate_e^T) * (z . up_e^T)) . down_e^T, experts in MXFP4;
              out = (sum_e p_e y_e) . w_up^T + sum_s (silu(x . sg_s^T) * (x . su_s^T)) . sd_s^T
              (without latent projections z = x and out = sum_e p_e y_e)

Values held in 8 bits are returned as the numbers they stand for (codes * scale, in BF16).
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    share = dict(op="moe", H=7168, Lt=3584, E=896, K=16, I=384, S=2, Is=384, latent=True, bias=False)
    return [
        # one token between two blocks: the latency of the call itself
        dict(name="block_norm_t1", op="block_norm", T=1, H=7168, stream="bf16", post=True, gate="none", act="none",
             alpha=1.0, beta=1.0, out="bf16", pad=0),
        # a decode batch with a sigmoid gate for every value, 8-bit input of the next block
        dict(name="block_norm_gate_t64", op="block_norm", T=64, H=7168, stream="bf16", post=True, gate="full",
             act="sigmoid", alpha=0.5, beta=1.0, out="i8", pad=0),
        # a prompt, residual stream in 32 bits, one learned gate row, both forms of the normalised rows
        dict(name="block_norm_t8192", op="block_norm", T=8192, H=7168, stream="f32", post=True, gate="row", act="tanh",
             alpha=1.0, beta=0.8, out="both", pad=0),
        # an odd width in a wider buffer, so that rows start at every alignment; a gate for every token
        dict(name="block_norm_odd_t1000", op="block_norm", T=1000, H=3581, stream="bf16", post=False, gate="token",
             act="sigmoid", alpha=1.0, beta=1.0, out="both", pad=6),
        # attention's output projection of one token, added to the residual stream
        dict(name="linear_t1", op="linear", T=1, N=7168, K=4096, glu=False, act="none", bias=False, res="bf16", out="bf16",
             pad=0),
        # gate and up of a shared expert or dense block, a decode batch
        dict(name="glu_t64", op="linear", T=64, N=7168, K=7168, glu=True, act="silu", bias=False, res="none", out="bf16",
             pad=0),
        # ragged in every size, everything in the epilogue, in 32 bits
        dict(name="linear_odd_t777", op="linear", T=777, N=1001, K=3583, glu=False, act="gelu", bias=True, res="f32",
             out="f32", pad=5),
        # the projection of a prompt, onto the residual stream
        dict(name="linear_t8192", op="linear", T=8192, N=7168, K=7168, glu=False, act="none", bias=True, res="bf16",
             out="bf16", pad=0),
        # one token through one GPU's share of the layer
        dict(share, name="moe_t1", T=1),
        # a small batch of requests, skewed routing
        dict(share, name="moe_t4", T=4, bias=True),
        # the most tokens that one row of matrix-core tiles takes
        dict(share, name="moe_t16", T=16),
        # a small layer without latent projections, odd number of experts
        dict(name="moe_small_t3", op="moe", T=3, H=0, Lt=512, E=61, K=6, I=256, S=0, Is=0, latent=False, bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Half of the widths any whole number, half multiples of 128, as a model's are."""
    w = _log(rng, lo, hi)
    return w if rng.random() < 0.5 else max(128, w // 128 * 128)


def _blocks(rng, lo, hi):
    """A multiple of 128, as the layer's widths are."""
    return max(1, _log(rng, lo, hi) // 128) * 128


def draw(rng):
    op = rng.choice(["block_norm", "linear", "linear", "moe", "moe"])
    T = _log(rng, 1, 8192)
    pad = rng.choice([0, 0, 0, rng.randrange(1, 64)])
    if op == "block_norm":
        H = _width(rng, 128, 14336)
        gate = rng.choice(["none", "full", "row", "token"])
        return dict(op=op, T=max(1, min(T, 8192 * 7168 // H)), H=H, stream=rng.choice(["bf16", "f32"]),
                    post=rng.random() < 0.8, gate=gate,
                    act="none" if gate == "none" else rng.choice(["none", "sigmoid", "tanh"]),
                    alpha=rng.choice([1.0, 0.5]), beta=rng.choice([1.0, 0.8]),
                    out=rng.choice(["bf16", "i8", "both", "sum"]), pad=pad)
    if op == "linear":
        N, K, glu = _width(rng, 128, 7168), _width(rng, 128, 14336), rng.random() < 0.4
        T = max(1, min(T, 8192 * 7168 * 7168 // (N * K * (1 + glu))))
        return dict(op=op, T=T, N=N, K=K, glu=glu, act=rng.choice(["none", "silu", "gelu", "gelu_tanh", "relu"]),
                    bias=not glu and rng.random() < 0.5, res=rng.choice(["none", "bf16", "f32"]),
                    out=rng.choice(["bf16", "bf16", "f32"]), pad=pad)
    E, latent = _log(rng, 8, 896), rng.random() < 0.7
    S = rng.randrange(0, 3) if latent else 0
    return dict(op=op, T=rng.randint(1, 16), H=_blocks(rng, 512, 7168) if latent else 0, Lt=_blocks(rng, 256, 3584), E=E,
                K=min(E, rng.choice([1, 2, 4, 6, 8, 16])), I=_blocks(rng, 128, 512), S=S,
                Is=_blocks(rng, 128, 512) if S else 0, latent=latent, bias=rng.random() < 0.5)


def _randn(*shape, gen):
    return torch.randn(*shape, generator=gen, device="cuda")


def _rows(T, width, pad, fill, dtype, gen):
    """[T, width] rows of a buffer `pad` values wider."""
    t = torch.empty(T, width + pad, dtype=dtype, device="cuda")
    return fill(t, gen)[:, :width]


def _activations(t, gen):
    """Hidden states as they come: normal, a few channels an order of magnitude larger, rows of different size."""
    f = _randn(*t.shape, gen=gen)
    f *= 1 + 15 * (torch.rand(t.shape[1], generator=gen, device="cuda") < 0.005)
    f *= torch.exp(0.5 * _randn(t.shape[0], 1, gen=gen))
    return t.copy_(f)


def _normal(t, gen):
    return t.copy_(_randn(*t.shape, gen=gen))


def _weights(n, k, gen):
    return (_randn(n, k, gen=gen) / math.sqrt(k)).bfloat16()


def _norm_weight(n, gen):
    return (1 + 0.2 * _randn(n, gen=gen)).bfloat16()


def _inputs(case, seed):
    """The case's inputs, from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"block_norm": _norm_inputs, "linear": _linear_inputs, "moe": _moe_inputs}[case["op"]](case, gen)


def _norm_inputs(case, gen):
    T, H, pad = case["T"], case["H"], case["pad"]
    d = {"x": _rows(T, H, pad, _activations, DTYPES[case["stream"]], gen),
         "y": _rows(T, H, pad, _activations, torch.bfloat16, gen),
         "post": _norm_weight(H, gen) if case["post"] else None, "weight": _norm_weight(H, gen), "gate": None}
    if case["gate"] == "full":
        d["gate"] = _rows(T, H, pad, _normal, torch.bfloat16, gen)
    elif case["gate"] != "none":
        d["gate"] = _randn(*((1, H) if case["gate"] == "row" else (T, 1)), gen=gen).bfloat16()
    return d


def _linear_inputs(case, gen):
    T, N, K, pad = case["T"], case["N"], case["K"], case["pad"]
    return {"x": _rows(T, K, pad, _normal, torch.bfloat16, gen), "w": _weights(N, K, gen),
            "w_up": _weights(N, K, gen) if case["glu"] else None,
            "bias": 0.5 * _randn(N, gen=gen) if case["bias"] else None,
            "residual": _rows(T, N, pad, _normal, DTYPES[case["res"]], gen) if case["res"] != "none" else None}


def _moe_inputs(case, gen):
    T, H, Lt, E, K, I, S, Is = (case[k] for k in ("T", "H", "Lt", "E", "K", "I", "S", "Is"))
    Hin = H if case["latent"] else Lt
    w = {"w_router": _weights(E, Hin, gen)}
    if case["latent"]:
        w |= {"w_down": _weights(Lt, H, gen), "w_up": _weights(H, Lt, gen)}
    if S:
        w |= {"sh_gate": _weights(S * Is, H, gen).view(S, Is, H), "sh_up": _weights(S * Is, H, gen).view(S, Is, H),
              "sh_down": _weights(S * H, Is, gen).view(S, H, Is)}
    for name, n, k in (("gate", I, Lt), ("up", I, Lt), ("down", Lt, I)):
        w[name + "_codes"] = torch.randint(0, 256, (E, n, k // 2), dtype=torch.uint8, generator=gen, device="cuda")
        # scales that keep an expert's values near those of a trained one: products of unit variance
        mid = round(127 - math.log2(2.9 * math.sqrt(k)))
        w[name + "_scales"] = torch.randint(mid - 1, mid + 2, (E, n, k // 32), dtype=torch.uint8, generator=gen,
                                            device="cuda")
    bias = None
    if case["bias"]:   # experts of very different popularity
        rank = 1 + torch.randperm(E, generator=gen, device="cuda")
        bias = -1.1 * torch.log(rank.double())
        bias = (bias - torch.logsumexp(bias, 0)).float()
    # Which expert comes next has to be the same in any precision: tokens are taken whose K + 1 largest logits are apart.
    pool = _randn(T + 16, Hin, gen=gen).bfloat16()
    logits = pool.double() @ w["w_router"].double().t() + (0 if bias is None else bias.double())
    best = torch.sort(logits, dim=1, descending=True).values[:, :K + 1]
    close = ((best[:, :-1] - best[:, 1:]) < 2e-5).any(1)
    x = pool[torch.sort(close.int(), stable=True).indices[:T]]
    return {"x": x, "bias": bias, "weights": w}


def prepare(case, seed):
    state = dict(case=case, **_inputs(case, seed))
    if own and case["op"] == "linear":   # the layers that a program makes once of its weights
        from mxfp4_latent_mixture_sigmoid_amd import Bf16Linear
        state["layer"] = Bf16Linear(state.pop("w"), bias=state["bias"], up_weight=state.pop("w_up"), activation=case["act"],
                                    T_max=case["T"], out_dtype=DTYPES[case["out"]])
    if own and case["op"] == "moe":
        from mxfp4_latent_mixture_sigmoid_amd import MoELayer
        state["layer"] = MoELayer(case["H"] if case["latent"] else case["Lt"], case["Lt"], case["E"], case["K"], case["I"],
                                  case["S"], case["Is"], case["latent"], state["weights"], T_max=case["T"])
        torch.cuda.synchronize()
        del state["weights"]
    return state


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(state):
    case = state["case"]
    if case["op"] == "block_norm":
        from mxfp4_latent_mixture_sigmoid_amd import block_norm, dequantise
        r = block_norm(state["x"], state["y"], state["post"], state["weight"], EPS, gate=state["gate"],
                       gate_act=case["act"], scale=case["alpha"], residual_scale=case["beta"],
                       out=case["out"] in ("bf16", "both"), codes=case["out"] in ("i8", "both"))
        got = {"sum": r.sum}
        if r.out is not None:
            got["out"] = r.out
        if r.codes is not None:
            got["held"], got["scales"] = dequantise(r.codes, r.scales), r.scales
        return got
    if case["op"] == "linear":
        return {"out": state["layer"].forward(state["x"], residual=state["residual"])}
    r = state["layer"].decode(state["x"], logit_bias=state["bias"])
    return {"out": r.out, "ids": r.ids, "weights": r.weights}


def _act(v, name):
    if name == "sigmoid":
        return 1 / (1 + torch.exp(-v))
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "tanh":
        return torch.tanh(v)
    if name == "relu":
        return v * (v > 0)
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _held(y):
    """Rows in 8 bits with a scale each, as the numbers that they stand for; and the scales."""
    scales = y.abs().amax(1) / 127
    codes = torch.round(y / scales[:, None]).clamp(-127, 127)
    return (codes * scales[:, None]).bfloat16(), scales


def _plain_norm(state):
    case = state["case"]
    n = state["y"].float()
    n = n * torch.rsqrt((n * n).mean(1, keepdim=True) + EPS)
    if state["post"] is not None:
        n = n * state["post"].float()
    if state["gate"] is not None:
        n = n * _act(state["gate"].float(), case["act"])
    s = case["beta"] * state["x"].float() + case["alpha"] * n
    got = {"sum": s.to(DTYPES[case["stream"]])}
    if case["out"] == "sum":
        return got
    y = s * torch.rsqrt((s * s).mean(1, keepdim=True) + EPS) * state["weight"].float()
    if case["out"] != "i8":
        got["out"] = y.bfloat16()
    if case["out"] != "bf16":
        got["held"], got["scales"] = _held(y)
    return got


def _plain_linear(state):
    case, x = state["case"], state["x"].float()
    out = x @ state["w"].float().t()
    if case["bias"]:
        out = out + state["bias"]
    out = _act(out, case["act"])
    if case["glu"]:
        out = out * (x @ state["w_up"].float().t())
    if state["residual"] is not None:
        out = out + state["residual"].float()
    return {"out": out.to(DTYPES[case["out"]])}


def _expert(weights, name, ids):
    """The matrices of experts `ids` in 32 bits."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    codes = weights[name + "_codes"][ids].int()
    values = torch.stack((table[codes & 15], table[codes >> 4]), -1).flatten(-2)
    scales = torch.exp2(weights[name + "_scales"][ids].float() - 127)
    return (values.unflatten(-1, (-1, 32)) * scales.unsqueeze(-1)).flatten(-2)


def _plain_moe(state):
    case, w, x = state["case"], state["weights"], state["x"].float()
    T, K = case["T"], case["K"]
    logits = state["x"].double() @ w["w_router"].double().t()      # 64 bits: values next to a border
    if case["bias"]:
        logits = logits + state["bias"].double()
    best = torch.sort(logits, dim=1, descending=True, stable=True)
    ids, p = best.indices[:, :K], 1 / (1 + torch.exp(-best.values[:, :K]))
    p = (p / p.sum(1, keepdim=True)).float()
    z = x @ w["w_down"].float().t() if case["latent"] else x
    zc = torch.zeros_like(z)
    for t in range(T):
        g = torch.matmul(_expert(w, "gate", ids[t]), z[t])
        u = torch.matmul(_expert(w, "up", ids[t]), z[t])
        h = g / (1 + torch.exp(-g)) * u
        y = torch.matmul(_expert(w, "down", ids[t]), h.unsqueeze(-1)).squeeze(-1)
        zc[t] = (p[t][:, None] * y).sum(0)
    out = zc
    if case["latent"]:
        out = zc @ w["w_up"].float().t()
        for s in range(case["S"]):
            g = x @ w["sh_gate"][s].float().t()
            out = out + (g / (1 + torch.exp(-g)) * (x @ w["sh_up"][s].float().t())) @ w["sh_down"][s].float().t()
    return {"out": out.bfloat16(), "ids": ids.int(), "weights": p}


def _run_plain(state):
    return {"block_norm": _plain_norm, "linear": _plain_linear, "moe": _plain_moe}[state["case"]["op"]](state)


def exact(case, seed):
    """The operators' definitions in 64 bits; what is rounded to 8 bits is rounded from those."""
    return {"block_norm": _exact_norm, "linear": _exact_linear, "moe": _exact_moe}[case["op"]](case, _inputs(case, seed))


def _curve(name, v):
    if name == "sigmoid":
        return torch.sigmoid(v)
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "tanh":
        e = torch.expm1(2 * v.abs())
        return torch.sign(v) * e / (e + 2)
    if name == "relu":
        return v.clamp(min=0)
    if name == "gelu":
        return v * torch.erfc(-v / math.sqrt(2)) / 2
    if name == "gelu_tanh":
        return v * torch.sigmoid(math.sqrt(8 / math.pi) * (v + 0.044715 * v.pow(3)))
    return v


def _exact_norm(case, d):
    def normed(rows, weight):
        rows = rows / torch.sqrt(rows.pow(2).sum(dim=1, keepdim=True) / case["H"] + EPS)
        return rows if weight is None else rows * weight.double()
    added = normed(d["y"].double(), d["post"]) * case["alpha"]
    if case["gate"] != "none":
        added = added * _curve(case["act"], d["gate"].double())
    s = d["x"].double() * case["beta"] + added
    got = {"sum": s}
    if case["out"] != "sum":
        rows = normed(s, d["weight"])
        if case["out"] in ("bf16", "both"):
            got["out"] = rows
        if case["out"] in ("i8", "both"):
            top = rows.abs().max(dim=1).values
            got["held"] = torch.round(rows * (127 / top).unsqueeze(1)) * (top / 127).unsqueeze(1)
            got["scales"] = top / 127
    return got


def _exact_linear(case, d):
    def product(w):
        return torch.matmul(d["x"].double(), w.double().t())
    y = product(d["w"])
    if d["bias"] is not None:
        y += d["bias"].double()
    y = _curve(case["act"], y)
    if d["w_up"] is not None:
        y *= product(d["w_up"])
    if d["residual"] is not None:
        y += d["residual"].double()
    return {"out": y}


def _exact_moe(case, d):
    x, w, K = d["x"].double(), d["weights"], case["K"]
    logits = torch.matmul(x, w["w_router"].double().t())
    if d["bias"] is not None:
        logits += d["bias"].double()
    order = torch.argsort(-logits, dim=1, stable=True)[:, :K]
    p = torch.sigmoid(torch.gather(logits, 1, order))
    p /= p.sum(dim=1, keepdim=True)

    def matrix(name, e):
        codes = w[name + "_codes"][e].long()
        nibbles = torch.stack((codes % 16, codes // 16), dim=2).reshape(codes.shape[0], -1)
        level = nibbles % 8
        size = torch.where(level < 2, level / 2.0, (1 + level % 2 / 2.0) * 2.0 ** (level // 2 - 1).double()).double()
        scales = 2.0 ** (w[name + "_scales"][e].double() - 127)
        return size * (1 - 2 * (nibbles // 8)) * scales.repeat_interleave(32, dim=1)
    z = torch.matmul(x, w["w_down"].double().t()) if case["latent"] else x
    mixed = torch.zeros_like(z)
    for e in order.unique().tolist():   # expert by expert, with the tokens that chose it
        token, slot = torch.nonzero(order == e, as_tuple=True)
        rows = z[token]
        inner = _curve("silu", rows @ matrix("gate", e).t()) * (rows @ matrix("up", e).t())
        mixed.index_add_(0, token, (inner @ matrix("down", e).t()) * p[token, slot].unsqueeze(1))
    if case["latent"]:
        mixed = mixed @ w["w_up"].double().t()
        for s in range(case["S"]):
            inner = _curve("silu", x @ w["sh_gate"][s].double().t()) * (x @ w["sh_up"][s].double().t())
            mixed = mixed + inner @ w["sh_down"][s].double().t()
    return {"out": mixed, "ids": None, "weights": p}


def work(case):
    """Each input read once, each result written once; additions and multiplications of the products (of the norm:
    two squares, two sums, four scalings, the addition). Of the mixture, the experts that its tokens reach: of E
    equally likely ones, T * K choices reach E (1 - (1 - K / E)^T) on average."""
    op, T = case["op"], case["T"]
    size = {"bf16": 2, "f32": 4, "none": 0}
    if op == "block_norm":
        H = case["H"]
        row = 2 * size[case["stream"]] + 2 + {"bf16": 2, "i8": 1, "both": 3, "sum": 0}[case["out"]]
        row += 2 * (case["gate"] == "full")
        return {"bytes": T * H * row + 2 * H * (1 + case["post"]) + 4 * T * (case["out"] in ("i8", "both")),
                "flops": T * H * (6 if case["out"] == "sum" else 10)}
    if op == "linear":
        N, K, mats = case["N"], case["K"], 1 + case["glu"]
        return {"bytes": 2 * T * K + 2 * mats * N * K + 4 * N * case["bias"]
                + T * N * (size[case["out"]] + size[case["res"]]), "flops": 2 * T * N * K * mats}
    H, Lt, E, K, I, SI = case["H"], case["Lt"], case["E"], case["K"], case["I"], case["S"] * case["Is"]
    Hin = H if case["latent"] else Lt
    reached = E * (1 - (1 - K / E) ** T)
    dense = E * Hin + (2 * H * Lt + 3 * H * SI if case["latent"] else 0)
    return {"bytes": int(2 * dense + reached * 3 * I * Lt * 17 / 32 + 4 * T * Hin + 8 * T * K),
            "flops": 2 * T * (dense + K * 3 * I * Lt)}
