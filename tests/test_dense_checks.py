"""Host-side checks of the dense 8-bit path's Python functions: what they refuse before any GPU work, and how they
treat streams. Tensors here have no GPU (device index -1) or are stand-ins; no call reaches the library."""
from types import SimpleNamespace

import pytest
import torch

from mxfp4_latent_mixture_sigmoid_amd import dense

BF16 = torch.bfloat16


def wide(T, K, dtype):
    """A [T, K] tensor without memory."""
    return torch.empty(T, K, dtype=dtype, device="meta")


@pytest.fixture
def no_library(monkeypatch):
    """Any call that gets past the checks ends here."""
    def reached():
        raise AssertionError("the call reached the library")
    monkeypatch.setattr(dense.abi, "lib", reached)


@pytest.mark.parametrize("T,K", [(2 ** 32 + 5, 1), (1, 2 ** 32 + 64), (2 ** 31, 3), (2, 2 ** 31)])
def test_sizes_past_32_bits_are_refused(T, K, no_library):
    """The ABI's sizes are 32-bit: 2^32 + 64 columns must not become 64."""
    x, q, s = wide(T, K, BF16), wide(T, K, torch.int8), torch.empty(T, device="meta")
    out, codes = wide(T, K, BF16), wide(T, K, torch.int8)
    for f in (lambda: dense._rms_norm(x, None, 1e-6, None, False, out, False, None, -1, 0),
              lambda: dense._quantise(x, codes, s, -1, 0), lambda: dense._dequantise(q, s, out, -1, 0),
              lambda: dense._rows("x", q, (torch.int8,), -1)):
        with pytest.raises(ValueError, match="rows and columns"):
            f()


@pytest.mark.parametrize("T_max", [2 ** 31, 2 ** 32 + 5, -1])
def test_token_limit_past_32_bits_is_refused(T_max):
    w, s = torch.zeros(4, 4, dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError, match="T_max"):
        dense.Int8Linear(w, s, T_max=T_max)


class Buffer:
    """Stands for a layer's own memory; keeps the streams it was recorded for."""

    def __init__(self):
        self.streams = []

    def get_device(self):
        return -1

    def record_stream(self, stream):
        self.streams.append(stream)


def test_a_layer_tells_the_allocator_which_streams_use_it(monkeypatch):
    """Built on stream 5, called under others: the packed weights are recorded for each of those, once."""
    current = [5]
    monkeypatch.setattr(dense, "_current_gpu", lambda: -1)
    monkeypatch.setattr(dense, "_raw_stream", lambda index: current[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index=None: f"stream {current[0]}")
    monkeypatch.setattr(dense.abi, "lib", lambda: SimpleNamespace(moe_linear_forward=lambda *a: 0))
    monkeypatch.setattr(dense.abi, "linear_query", lambda cfg, T: (256, 256))
    monkeypatch.setattr(dense.abi, "linear_create", lambda *a: None)
    layer = object.__new__(dense.Int8Linear)
    layer.handle, layer.T_max, layer.out_dtype = None, 4, torch.float32
    q, s = torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4)
    layer._create(q, s, None, None, None, -1, 5)
    layer.packed, layer.workspace = Buffer(), Buffer()
    for handle in (5, 7, 7, 5, 9, 7):
        current[0] = handle
        layer.forward(q, s)
    assert layer.packed.streams == ["stream 7", "stream 9"]


def test_a_stream_of_another_gpu_is_refused():
    x = SimpleNamespace(get_device=lambda: 0)
    stream = SimpleNamespace(device_index=1, device=torch.device("cuda", 1), cuda_stream=3)
    for f in (lambda: dense.rms_norm(x, stream=stream), lambda: dense.quantise(x, stream=stream),
              lambda: dense.dequantise(x, None, stream=stream)):
        with pytest.raises(ValueError, match="stream: on GPU 1, expected GPU 0"):
            f()


def test_room_is_allocated_only_when_the_library_asks(monkeypatch):
    """The first call offers no workspace; only where that is refused is one of the queried size allocated."""
    calls, needs = [], [False]

    def forward(handle, x, ldx, scales, T, out, ldo, room, size, stream):
        calls.append((room, size))
        return dense.abi.Status.BUFFER_TOO_SMALL if needs[0] and size < 512 else dense.abi.Status.OK
    monkeypatch.setattr(dense, "_current_gpu", lambda: -1)
    monkeypatch.setattr(dense, "_raw_stream", lambda index: 5)
    monkeypatch.setattr(dense.abi, "lib", lambda: SimpleNamespace(moe_linear_forward=forward))
    monkeypatch.setattr(dense.abi, "linear_query", lambda cfg, T: (256, 128 * T))
    monkeypatch.setattr(dense.abi, "linear_create", lambda *a: None)
    q, s = torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4)
    layer = object.__new__(dense.Int8Linear)
    layer.handle, layer.T_max, layer.out_dtype = None, 8192, torch.float32
    layer._create(q, s, None, None, None, -1, 5)
    held = sum(v.numel() for v in vars(layer).values() if torch.is_tensor(v))
    assert held == 256   # the packed weights alone
    layer.forward(q, s)
    needs[0] = True
    layer.forward(q, s)
    assert calls[:2] == [(None, 0), (None, 0)] and len(calls) == 3
    assert calls[2][0] and calls[2][1] == 512
