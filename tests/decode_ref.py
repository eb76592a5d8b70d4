"""Plain 64-bit form of the whole layer, on the GPU for its products, and how far the few-token form may be from it.

The form rounds to BF16 (8 significant bits, so by 2^-8 / sqrt(3) = 0.0023 in the mean square at most) z, each h, each shared
h_s, zc and out, and nothing else to fewer than 24 bits. z's rounding reaches the gate and the up value, each sums of many
independent errors, and with silu's slope of at most 1.1 their product: 0.0023 sqrt(1 + 1.1^2) = 0.0034 at most. All in
all sqrt(0.0034^2 + 3 x 0.0023^2) = 0.0052 of the output's root mean square for the independent errors, plus the last
rounding of each output."""
import numpy as np
import torch

SIGMA = 0.0052
TABLE = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def bf16(a):
    """uint16 bits -> float64 on the GPU."""
    return torch.from_numpy(a.view(np.int16)).cuda().view(torch.bfloat16).double()


def matrix(inp, name, e):
    codes = torch.from_numpy(inp[name + "_codes"][e]).cuda().long()
    v = TABLE.cuda()[torch.stack((codes % 16, codes // 16), -1).flatten(-2)]
    s = torch.from_numpy(inp[name + "_scales"][e]).cuda().double()
    return v * torch.exp2(s - 127).repeat_interleave(32, -1)


def silu(v):
    return v * torch.sigmoid(v)


def logits(inp, bias=None):
    l = bf16(inp["x"]) @ bf16(inp["w_router"]).t()
    return l if bias is None else l + torch.from_numpy(bias).cuda().double()


def forward(shape, inp, ids, p):
    """The layer's output for given experts ids and weights p [T, K]."""
    x = bf16(inp["x"])
    z = x @ bf16(inp["w_down"]).t() if shape.has_latent else x
    zc = torch.zeros_like(z)
    for e in sorted(set(ids.flatten().tolist())):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        h = silu(z[t] @ matrix(inp, "gate", e).t()) * (z[t] @ matrix(inp, "up", e).t())
        zc.index_add_(0, t, (h @ matrix(inp, "down", e).t()) * p[t, j, None])
    if not shape.has_latent:
        return zc
    out = zc @ bf16(inp["w_up"]).t()
    for s in range(shape.S):
        h = silu(x @ bf16(inp["sh_gate"][s]).t()) * (x @ bf16(inp["sh_up"][s]).t())
        out = out + h @ bf16(inp["sh_down"][s]).t()
    return out


def check(out, ref, what):
    err, rms = (out.double() - ref).abs(), ref.square().mean(1, keepdim=True).sqrt()
    assert torch.isfinite(out).all(), what
    norm = float((err / rms).square().mean().sqrt())
    worst = float(((err - 2.0 ** -8 * ref.abs()) / rms).max())
    print(f"  {what}: {norm:.5f} of the rms, worst {worst:.4f}", flush=True)
    assert norm <= 1.25 * np.hypot(SIGMA, 0.0023), (what, norm)   # a quarter for few outputs
    assert worst <= 7 * SIGMA, (what, worst)
