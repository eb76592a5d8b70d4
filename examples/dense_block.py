#!/usr/bin/env python3
"""Two sublayers of a decoder around one residual stream: an MXFP4 latent mixture layer and a dense 8-bit
feed-forward block, each behind its residual addition and RMS norm, for a batch of tokens on one GPU.

    python examples/dense_block.py [tokens]

Weights and tokens are random. Prints what a step took, eagerly and replayed from one HIP graph."""
import os
import sys
import time

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch                                                                              # noqa: E402

from mxfp4_latent_mixture_sigmoid_amd import Int8FeedForward, MoELayer, quantise, rms_norm  # noqa: E402
from workload import SHAPES, make_inputs                                                    # noqa: E402


def device(a):
    t = torch.from_numpy(a)
    return (t.view(torch.int16) if a.dtype.name == "uint16" else t).cuda()


class Decoder:
    """norm -> mixture layer, norm -> dense block (of `inter` inner channels)."""

    def __init__(self, shape, T, inter, seed=0):
        inp = make_inputs(shape)
        weights = {k: device(v) for k, v in inp.items() if k.startswith(("w_", "gate_", "up_", "down_", "sh_"))
                   and v is not None}
        self.mixture = MoELayer(shape.H, shape.Lt, shape.E, shape.K, shape.I, shape.S, shape.Is, shape.has_latent,
                                weights, T_max=T)
        g = torch.Generator().manual_seed(seed)

        def matrix(n, k):
            return quantise((torch.randn(n, k, generator=g) / k ** 0.5).bfloat16().cuda())
        H = shape.H
        self.norm_weight = torch.ones(H, dtype=torch.bfloat16, device="cuda")
        self.dense = Int8FeedForward(self.norm_weight, matrix(inter, H), matrix(inter, H), matrix(H, inter), T_max=T)
        self.T, self.routing = T, self.mixture.alloc_routing(T)

    def step(self, stream, delta):
        """The residual stream and the last sublayer's output -> the same after both sublayers."""
        r = rms_norm(stream, self.norm_weight, delta=delta, sum=True)
        delta = self.mixture.route_forward(r.out, self.T, self.routing)
        return self.dense.forward(r.sum, delta=delta)[::-1]


def main():
    T = int(sys.argv[1]) if len(sys.argv) > 1 else 64
    shape = SHAPES["tp8_decode_t64"].with_tokens(T)
    decoder = Decoder(shape, T, inter=2 * shape.H)
    x = torch.randn(T, shape.H, device="cuda").bfloat16()
    zero = torch.zeros_like(x)
    stream, delta = decoder.step(x, zero)
    torch.cuda.synchronize()

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = decoder.step(x, zero)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held[0], stream) and torch.equal(held[1], delta), "the graph's step differs"

    def ms(f, n=50):
        for _ in range(5):
            f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(n):
            f()
        torch.cuda.synchronize()
        return (time.perf_counter() - t) / n * 1e3
    print(f"{T} tokens: stream rms {stream.float().square().mean().sqrt():.3f}, last output rms "
          f"{delta.float().square().mean().sqrt():.3f}; a step {ms(lambda: decoder.step(x, zero)):.3f} ms, "
          f"replayed {ms(graph.replay):.3f} ms", flush=True)


if __name__ == "__main__":
    main()
