"""What the BF16 product refuses before any GPU work, in Python and at the C ABI, and its sizes."""
import ctypes
import os
import re
from types import SimpleNamespace

import pytest
import torch

from mxfp4_latent_mixture_sigmoid_amd import abi, dense

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16 = torch.bfloat16
BAD, UNSUPPORTED, SMALL = abi.Status.INVALID_ARG, abi.Status.UNSUPPORTED, abi.Status.BUFFER_TOO_SMALL
A = 1 << 20      # an aligned address that no refused call touches


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(abi.LIB_PATH):
        from mxfp4_latent_mixture_sigmoid_amd import build
        build.build()


def config(**kw):
    return abi.DenseConfig(**{**dict(n=100, k=200, glu=0, act=0, out_type=0), **kw})


def query(cfg, T=8):
    pb, wb = ctypes.c_size_t(), ctypes.c_size_t()
    return abi.lib().moe_dense_query(cfg and ctypes.byref(cfg), T, ctypes.byref(pb), ctypes.byref(wb)), pb.value, wb.value


def create(cfg, w=A, w_up=None, bias=None, packed=A, size=1 << 40):
    h = ctypes.c_void_p(5)
    st = abi.lib().moe_dense_create(ctypes.byref(cfg), ctypes.byref(abi.DenseWeights(w, w_up, bias)), packed, size,
                                          None, ctypes.byref(h))
    assert not h.value
    return st


def test_structures_follow_the_header():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mxmoe.h")).read(), flags=re.S)
    for name, cls in (("moe_dense_config", abi.DenseConfig), ("moe_dense_weights", abi.DenseWeights)):
        body = re.search(r"typedef struct \{([^}]*)\}\s*%s;" % name, src).group(1)
        fields = [f.strip().lstrip("*") for decl in body.split(";") if decl.strip()
                  for f in re.sub(r"^\s*(const\s+)?\w+\s", "", decl).split(",")]
        assert fields == [f for f, _ in cls._fields_], name
    assert f"MOE_DENSE_MAX_K {abi.DENSE_MAX_K}" in src


def test_sizes():
    st, packed, room = query(config(n=100, k=200), 9)
    # 7 blocks of 16 rows, 4 stages of 64 values, then the bias; a row of 4 stages for each token
    assert (st, packed, room) == (0, 7 * 4 * 2048 + 512, 9 * 512)
    assert query(config(n=100, k=200, glu=1))[1] == 14 * 4 * 2048 + 512


@pytest.mark.parametrize("change", [dict(n=0), dict(k=0), dict(glu=2), dict(act=5), dict(act=-1), dict(out_type=2)])
def test_configurations_refused(change):
    assert query(config(**change))[0] == BAD and create(config(**change)) == BAD


def test_limits():
    assert query(None)[0] == BAD and query(config(), -1)[0] == BAD
    assert query(config(k=abi.DENSE_MAX_K + 1))[0] == UNSUPPORTED
    assert query(config(k=abi.DENSE_MAX_K))[0] == 0
    assert query(config(n=2 ** 31 - 1))[0] == UNSUPPORTED
    assert query(config(n=1 << 20, k=64), 2 ** 31 - 1)[0] == BAD


def test_weights_refused():
    c, g = config(), config(glu=1)
    for st in (create(c, w=None), create(c, w=A + 1), create(c, w_up=A), create(g), create(g, w_up=A, bias=A),
               create(g, w_up=A + 1), create(c, bias=A + 2), create(c, packed=None), create(c, packed=A + 128)):
        assert st == BAD
    assert create(c, size=100) == SMALL


def test_the_class_refuses():
    w = torch.zeros(4, 8, dtype=BF16)
    for kw in (dict(out_dtype=torch.float16), dict(activation="tanh"), dict(up_weight=w, bias=torch.zeros(4)),
               dict(T_max=-1), dict(T_max=2 ** 31)):
        with pytest.raises(ValueError):
            dense.Bf16Linear(w, **kw)
    with pytest.raises(ValueError, match="GPU"):
        dense.Bf16Linear(w)


@pytest.fixture
def layer(monkeypatch):
    """A layer without a GPU, and the calls that it makes."""
    calls = []

    def forward(*a):
        calls.append(a)
        return abi.Status.BUFFER_TOO_SMALL if calls[0] is None and a[10] < 512 else abi.Status.OK
    monkeypatch.setattr(dense, "_current_gpu", lambda: -1)
    monkeypatch.setattr(dense, "_raw_stream", lambda index: 5)
    monkeypatch.setattr(dense.abi, "lib", lambda: SimpleNamespace(moe_dense_forward=forward))
    monkeypatch.setattr(dense.abi, "dense_query", lambda cfg, T: (256, 128 * T))
    monkeypatch.setattr(dense.abi, "dense_create", lambda *a: None)
    l = object.__new__(dense.Bf16Linear)
    l.handle, l.T_max, l.out_dtype, l.activation, l.calls = None, 4, BF16, "silu", calls
    l._create(torch.zeros(6, 8, dtype=BF16), torch.zeros(6), None, -1, 5)
    return l


def test_calls_refused(layer):
    x = torch.zeros(4, 8, dtype=BF16)
    for a in ((x.float(),), (x[:, :7],), (torch.zeros(5, 8, dtype=BF16),), (x.t(),), (x, torch.zeros(4, 5)),
              (x, torch.zeros(3, 6)), (x, torch.zeros(4, 6).half()), (x, None, torch.zeros(4, 6)),
              (x, None, torch.zeros(4, 7, dtype=BF16))):
        with pytest.raises(ValueError):
            layer.forward(*a)
    assert not layer.calls


def test_room_is_allocated_only_when_the_library_asks(layer):
    x, r = torch.zeros(4, 8, dtype=BF16), torch.zeros(4, 6)
    layer.forward(x, r)
    assert layer.calls[0][3:7] == (r.data_ptr(), abi.TYPE_F32, 6, 4) and layer.calls[0][9:11] == (None, 0)
    layer.calls[0] = None
    layer.forward(x)
    assert len(layer.calls) == 3 and layer.calls[2][9] and layer.calls[2][10] == 512
    assert sum(v.numel() for v in vars(layer).values() if torch.is_tensor(v)) == 256


def test_a_stream_of_another_gpu_is_refused(layer):
    stream = SimpleNamespace(device_index=1, device=torch.device("cuda", 1), cuda_stream=3)
    layer.packed = SimpleNamespace(get_device=lambda: 0)
    with pytest.raises(ValueError, match="stream: on GPU 1, expected GPU 0"):
        layer.forward(torch.zeros(4, 8, dtype=BF16), stream=stream)
