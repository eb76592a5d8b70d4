#!/usr/bin/env python3
"""A decode step around one residual stream, for 1 to 16 tokens on one GPU: a BF16 projection that adds itself to the
stream, the norm between two blocks with its per-token gate, and the whole MXFP4 latent mixture layer in one launch.

    python examples/decode_step.py [tokens [tiny]]

Weights and tokens are random. Prints what a step took, eagerly and replayed from one HIP graph."""
import os
import sys
import time

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch                                                                                # noqa: E402

from mxfp4_latent_mixture_sigmoid_amd import Bf16Linear, MoELayer, block_norm, rms_norm    # noqa: E402
from workload import SHAPES, make_inputs                                                    # noqa: E402


def device(a):
    t = torch.from_numpy(a)
    return (t.view(torch.int16) if a.dtype.name == "uint16" else t).cuda()


class Step:
    """projection + residual -> norm -> mixture layer -> norm, gate, scaled residual, norm."""

    def __init__(self, shape, T, seed=0):
        inp = make_inputs(shape)
        weights = {k: device(v) for k, v in inp.items() if k.startswith(("w_", "gate_", "up_", "down_", "sh_"))
                   and v is not None}
        self.mixture = MoELayer(shape.H, shape.Lt, shape.E, shape.K, shape.I, shape.S, shape.Is, shape.has_latent,
                                weights, T_max=T)
        g = torch.Generator().manual_seed(seed)
        H = shape.H
        self.norm = (1 + 0.1 * torch.randn(H, generator=g)).bfloat16().cuda()
        self.projection = Bf16Linear((torch.randn(H, H, generator=g) / H ** 0.5).bfloat16().cuda(), T_max=T,
                                     out_dtype=torch.float32)

    def __call__(self, stream, attended, gate):
        """The FP32 residual stream, the attention's output and a gate per token -> the stream and the next block's input."""
        stream = self.projection.forward(attended, residual=stream)
        x = rms_norm(stream, self.norm).out
        y = self.mixture.decode(x).out
        r = block_norm(stream, y, self.norm, self.norm, gate=gate, gate_act="sigmoid")
        return r.sum, r.out


def main(argv=None):
    argv = sys.argv[1:] if argv is None else argv
    T = int(argv[0]) if argv else 1
    shape = SHAPES["tiny" if "tiny" in argv[1:] else "tp8_decode_t64"].with_tokens(T)
    step = Step(shape, T)
    stream = torch.randn(T, shape.H, device="cuda")
    attended, gate = torch.randn(T, shape.H, device="cuda").bfloat16(), torch.randn(T, 1, device="cuda").bfloat16()
    got = step(stream, attended, gate)
    torch.cuda.synchronize()

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(stream, attended, gate)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, got)), "the graph's step differs"

    def us(f, n=50):
        for _ in range(5):
            f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(n):
            f()
        torch.cuda.synchronize()
        return (time.perf_counter() - t) / n * 1e6
    print(f"{T} tokens: stream rms {got[0].square().mean().sqrt():.3f}; a step "
          f"{us(lambda: step(stream, attended, gate)):.0f} us, replayed {us(graph.replay):.0f} us", flush=True)


if __name__ == "__main__":
    main()
