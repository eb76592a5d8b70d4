"""Plain 64-bit numpy form of the norms between two blocks, and the error each output may have.

With u = 2^-24 as in dense_ref: n = y's norm is off by NORM_REL; the gate's sigmoid and tanh by at most 8 u of
themselves (an exponential to 3 u, a sum, a reciprocal to 2 u, a product; the difference that ends tanh at least
doubles as it loses two bits); alpha g n adds three roundings, the sum with beta x two more. What s is off by reaches
the second norm directly and, through its mean square, at most by its root mean square relative to s's."""
import numpy as np

from tests.dense_ref import B, NORM_REL, U

GATE_REL = 8 * U


def gate_value(g, act):
    with np.errstate(over="ignore"):
        return {None: lambda v: v, "sigmoid": lambda v: 1 / (1 + np.exp(-v)), "tanh": np.tanh}[act](g)


def block_norm(x, y, post, weight, eps, gate=None, act=None, alpha=1.0, beta=1.0):
    """(s, its error, out, its error before rounding)"""
    with np.errstate(all="ignore"):
        n = y / np.sqrt((y * y).mean(1, keepdims=True) + eps) * (1 if post is None else post)
        added = alpha * n * (1 if gate is None else gate_value(gate, act))
        s = beta * x + added
        off = np.abs(added) * (NORM_REL + GATE_REL + 4 * U) + 2 * U * (np.abs(beta * x) + np.abs(added)) + 2.0 ** -124
        root = np.sqrt((s * s).mean(1, keepdims=True) + eps)
        w = 1 if weight is None else weight
        out = s / root * w
        lost = np.sqrt((off * off).mean(1, keepdims=True)) / root
        return s, off, out, np.abs(out) * (NORM_REL + 1.01 * lost) + 1.01 * off / root * np.abs(w)


def bf16(v):
    return np.abs(v) * B
