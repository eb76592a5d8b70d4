"""What the few-token form of the layer refuses before any GPU work, in Python and at the C ABI, and its sizes."""
import ctypes
import os
from types import SimpleNamespace

import pytest
import torch

from mxfp4_latent_mixture_sigmoid_amd import abi
from mxfp4_latent_mixture_sigmoid_amd.layer import MoELayer

BF16 = torch.bfloat16
BAD, UNSUPPORTED = abi.Status.INVALID_ARG, abi.Status.UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(abi.LIB_PATH):
        from mxfp4_latent_mixture_sigmoid_amd import build
        build.build()


def config(hidden=256, latent=256, E=40, K=4, I=128, S=1, Is=64, lat=True, **kw):
    return abi.make_config(hidden, latent, E, K, I, S, Is, lat, **kw)


def query(cfg, T):
    n = ctypes.c_size_t()
    return abi.lib().moe_decode_query(cfg and ctypes.byref(cfg), T, ctypes.byref(n)), n.value


def test_sizes():
    up = lambda v: (v + 255) // 256 * 256          # noqa: E731
    st, size = query(config(), 5)
    assert st == 0 and size == (up((20 + 3 * 64 + 20 + 1) * 32 * 4) + up((4 * 3 + 36 + 2 * (1 + 1) + 20 * (8 + 1)) * 4) + up(20 * 256 * 4)
                                + up(4 * 5 * 40 * 4) + 2 * up(5 * 4 * 4) + up(20 * 4) + up(20 * 16 * 2) + 2 * up(5 * 256 * 2)
                                + up(5 * 320 * 2) + up(2 * 20 * 128 * 2))
    assert query(config(), 0)[0] == 0 and query(config(), abi.DECODE_MAX_T)[0] == 0


def test_refused():
    assert query(config(), -1)[0] == BAD and query(None, 1)[0] == BAD and query(config(latent=100), 1)[0] == BAD
    assert abi.lib().moe_decode_query(ctypes.byref(config()), 1, None) == BAD
    assert query(config(), abi.DECODE_MAX_T + 1)[0] == UNSUPPORTED
    assert query(config(stage1_a4=True), 1)[0] == UNSUPPORTED and query(config(stage2_fp8=True), 1)[0] == UNSUPPORTED
    assert query(config(I=1 << 24), 16)[0] == UNSUPPORTED       # offsets and launches past 32 bits
    assert abi.lib().moe_decode(None, 0, 1, None, None, None, None, None, None, 0, None) == BAD
    assert "MOE_DECODE_MAX_T %d" % abi.DECODE_MAX_T in open(os.path.join(os.path.dirname(__file__), "..", "include",
                                                                         "mxmoe.h")).read()


@pytest.fixture
def layer(monkeypatch):
    """A layer without a GPU, whose calls end at the library."""
    l = object.__new__(MoELayer)
    l.handle, l.cfg, l.E, l.K, l.Lt, l.H = None, config(), 40, 4, 256, 256
    l._decode_bytes, l._streams = {}, {0}

    def reached(*a):
        raise AssertionError("the call reached the library")
    monkeypatch.setattr(abi, "decode_query", reached)
    return l


def test_the_method_refuses(layer):
    x = torch.zeros(3, 256, dtype=BF16)
    given = dict(out=torch.zeros(3, 256, dtype=BF16), ids=torch.zeros(3, 4, dtype=torch.int32), weights=torch.zeros(3, 4),
                 logit_bias=torch.zeros(40), logits_out=torch.zeros(3, 40))

    def call(x=x, **kw):
        a = {**given, **kw}
        layer._decode(x, a["out"], a["logit_bias"], a["logits_out"], a["ids"], a["weights"], -1, 0)
    for bad in (dict(x=x.float()), dict(x=x[0]), dict(x=x[:, :255]), dict(x=torch.zeros(17, 256, dtype=BF16)),
                dict(x=torch.zeros(3, 512, dtype=BF16)[:, ::2]), dict(out=torch.zeros(2, 256, dtype=BF16)),
                dict(out=torch.zeros(3, 256)), dict(ids=torch.zeros(3, 4, dtype=torch.int64)), dict(weights=torch.zeros(4, 3)),
                dict(logit_bias=torch.zeros(41)), dict(logit_bias=torch.zeros(40).double()), dict(logits_out=torch.zeros(40, 3)),
                dict(logits_out=torch.zeros(3, 80)[:, ::2])):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(AssertionError, match="reached"):
        call()


def test_a_stream_of_another_gpu_is_refused(layer):
    layer.packed = SimpleNamespace(get_device=lambda: 0)
    stream = SimpleNamespace(device_index=1, cuda_stream=3)
    with pytest.raises(ValueError, match="stream: on GPU 1, expected GPU 0"):
        layer.decode(torch.zeros(1, 256, dtype=BF16), stream=stream)
