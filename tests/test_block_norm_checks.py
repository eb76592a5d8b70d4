"""What the norms between two blocks refuse before any GPU work, in Python and at the C ABI."""
import ctypes
import os
import re

import pytest
import torch

from mxfp4_latent_mixture_sigmoid_amd import abi, dense

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16 = torch.bfloat16
BAD, UNSUPPORTED = abi.Status.INVALID_ARG, abi.Status.UNSUPPORTED
A = 1 << 20      # an aligned address that no refused call touches


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(abi.LIB_PATH):
        from mxfp4_latent_mixture_sigmoid_amd import build
        build.build()


def call(**kw):
    a = dict(x=A, y=A, post_weight=None, weight=None, gate=None, sum=A, out=A, codes=None, scales=None, ldx=64, ldy=64, ldg=0,
             lds=64, ldo=64, ldc=64, T=4, H=64, x_type=abi.TYPE_BF16, gate_act=0, gate_width=0, eps=1e-6, scale=1.0,
             residual_scale=1.0)
    a.update(kw)
    return abi.lib().moe_block_norm(bytes(abi.BlockNormArgs(**a)), None)


def test_the_structure_follows_the_header():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mxmoe.h")).read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\}\s*moe_block_norm_args;", src).group(1)
    fields = [f.strip().lstrip("*") for decl in body.split(";") if decl.strip()
              for f in re.sub(r"^\s*(const\s+)?\w+\s", "", decl).split(",")]
    assert fields == [f for f, _ in abi.BlockNormArgs._fields_]
    assert abi.BLOCK_NORM_ARGS.size == ctypes.sizeof(abi.BlockNormArgs)


@pytest.mark.parametrize("change", [
    dict(x=None), dict(y=None), dict(x=A + 1), dict(y=A + 1), dict(ldx=63), dict(ldy=63), dict(lds=63), dict(ldo=63),
    dict(T=-1), dict(H=0), dict(x_type=2), dict(eps=-1.0), dict(eps=float("nan")), dict(scale=float("nan")),
    dict(residual_scale=float("inf")), dict(sum=None, out=None), dict(codes=A), dict(scales=A), dict(codes=A, scales=A + 2),
    dict(codes=A, scales=A, ldc=63), dict(sum=A, lds=128), dict(weight=A + 1), dict(post_weight=A + 1),
    dict(gate=A, gate_width=2), dict(gate=A, gate_width=0), dict(gate=A, gate_width=64, gate_act=3),
    dict(gate=A, gate_width=64, gate_act=-1), dict(gate=A, gate_width=64, ldg=63), dict(gate=A, gate_width=64, ldg=-64),
    dict(gate=A + 1, gate_width=64), dict(gate_act=1), dict(gate_width=64)])
def test_the_abi_refuses(change):
    assert call(**change) == BAD


def test_limits():
    assert call(H=abi.MAX_WIDTH + 1) == UNSUPPORTED
    assert call(T=0, x=None, y=None) == abi.Status.OK
    assert abi.lib().moe_block_norm(None, None) == BAD


def test_the_function_refuses(monkeypatch):
    """Tensors here have no GPU (index -1); no call reaches the library."""
    def reached():
        raise AssertionError("the call reached the library")
    monkeypatch.setattr(dense.abi, "lib", reached)
    x = torch.zeros(4, 6, dtype=BF16)

    def f(x=x, y=x, post=None, weight=None, gate=None, act=None, sum=True, out=True, codes=False, scales=None):
        return dense._block_norm(x, y, post, weight, 1e-6, gate, act, 1.0, 1.0, sum, out, codes, scales, -1, 0)
    gate = torch.zeros(4, 6, dtype=BF16)
    for bad in (dict(y=x.float()), dict(y=x[:3]), dict(x=x.half(), y=x), dict(post=torch.ones(6)),
                dict(weight=torch.ones(5, dtype=BF16)), dict(act="sigmoid"), dict(gate=gate, act="relu"),
                dict(gate=gate.float()), dict(gate=gate[:3]), dict(gate=gate[:, :5]), dict(gate=gate[:, 0]),
                dict(gate=gate.t().contiguous().t()), dict(gate=gate[None]), dict(sum=x.float()), dict(scales=torch.ones(4)),
                dict(gate=torch.zeros(30, dtype=BF16).as_strided((4, 6), (2, 1)))):
        with pytest.raises(ValueError):
            f(**bad)
    with pytest.raises(AssertionError, match="reached"):
        f(gate=gate, act="tanh")


@pytest.mark.parametrize("shape,want", [((4, 6), (6, 6)), ((4, 1), (1, 1)), ((1, 6), (6, 0)), ((6,), (6, 0)), ((1, 1), (1, 0))])
def test_gate_shapes(shape, want):
    assert dense._gate(torch.zeros(*shape, dtype=BF16), 4, 6, -1) == want


def test_a_gate_spread_over_columns_is_one_per_token():
    assert dense._gate(torch.zeros(4, 1, dtype=BF16).expand(4, 6), 4, 6, -1) == (1, 1)
