"""How near the few-token form of the layer is to the exact result, and a 64-bit form in which its roundings can be put back.

The form keeps z, each h, each h_s and zc in two BF16 parts: the first is off by at most half a step, 2^-8 of the value, the second by
as much of what the first left, so a value by at most 2^-16 and, over a step, 2^-16 / sqrt(3) = 8.8e-6 in the mean square. z's reaches the
gate and the up value and, with silu's slope of at most 1.1, their product; the others come on top: 8.8e-6 sqrt(1 + 1.1^2 + 3) = 2.1e-5 of the
output's root mean square. Sums are FP32: K products added in K / 32 instructions of 32 are off by at most (K / 32 + 6) 2^-24 of their
magnitudes' sum, which for independent terms is about sqrt(K) times the result's size; their errors are independent as well, so that
sqrt(K / 32 + 6) 2^-24 sqrt(K) remains in the mean square, with K = 8192 8.6e-5 at most (in earnest a third: a sum's rounding
is a half of a step at most and its partial sums are smaller than it). Three products follow each other: 1.7 x 8.6e-5 and 2.1e-5 make
SIGMA = 1.5e-4 of the output's root mean square.

Then the output is rounded once, by at most half a step at its size. So what an output is off by BEYOND that half step is within
those errors: its mean square below SIGMA, no output beyond 7 of them. Any of the four values rounded to BF16 alone, 2^-8 / sqrt(3) =
0.0023 of it at most and about half of that in the mean, is beyond: tests/test_decode_precision.py."""
import numpy as np
import torch

from tests.decode_ref import TABLE, silu

SIGMA = 1.5e-4


def f64(a, device):
    return torch.from_numpy(a.view(np.int16)).to(device).view(torch.bfloat16).double()


def matrix(inp, name, e, device):
    codes = torch.from_numpy(inp[name + "_codes"][e]).to(device).long()
    v = TABLE.to(device)[torch.stack((codes % 16, codes // 16), -1).flatten(-2)]
    return v * torch.exp2(torch.from_numpy(inp[name + "_scales"][e]).to(device).double() - 127).repeat_interleave(32, -1)


def loud(inp):
    """Shared experts that carry most of the output, so that what their values lose is seen in it."""
    v = torch.from_numpy(inp["sh_down"].view(np.int16)).view(torch.bfloat16) * 32
    return dict(inp, sh_down=v.view(torch.int16).numpy().view(np.uint16))


def forward(shape, inp, ids, p, device="cuda", rounded=()):
    """The layer's output for given experts and weights [T, K]; the values named in `rounded` (z, h, hs, zc) go through BF16."""
    def keep(name, v):
        return v.bfloat16().double() if name in rounded else v
    x = f64(inp["x"], device)
    z = keep("z", x @ f64(inp["w_down"], device).t()) if shape.has_latent else x
    zc = torch.zeros_like(z)
    for e in sorted(set(ids.flatten().tolist())):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        h = keep("h", silu(z[t] @ matrix(inp, "gate", e, device).t()) * (z[t] @ matrix(inp, "up", e, device).t()))
        zc.index_add_(0, t, (h @ matrix(inp, "down", e, device).t()) * p[t, j, None])
    if not shape.has_latent:
        return zc
    out = keep("zc", zc) @ f64(inp["w_up"], device).t()
    for s in range(shape.S):
        h = keep("hs", silu(x @ f64(inp["sh_gate"][s], device).t()) * (x @ f64(inp["sh_up"][s], device).t()))
        out = out + h @ f64(inp["sh_down"][s], device).t()
    return out


def beyond(out, ref):
    """What outputs are off by past the half step of their rounding, over the row's root mean square: (root mean square, largest)."""
    half = torch.exp2(torch.floor(torch.log2(ref.abs().clamp(min=2.0 ** -126))) - 8)
    over = ((out.double() - ref).abs() - half).clamp(min=0) / ref.square().mean(1, keepdim=True).sqrt()
    return float(over.square().mean().sqrt()), float(over.max())


def near(out, ref):
    norm, worst = beyond(out, ref)
    return bool(torch.isfinite(out).all()) and norm <= SIGMA and worst <= 7 * SIGMA


def check(out, ref, what):
    norm, worst = beyond(out, ref)
    print(f"  {what}: {norm:.2e} of the rms beyond the rounding, worst {worst:.2e}", flush=True)
    assert near(out, ref), (what, norm, worst)
