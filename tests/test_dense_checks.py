"""Host-side checks of the dense 8-bit path's Python functions: what they refuse before any GPU work, and how they
treat streams. Tensors here have no GPU (device index -1) or are stand-ins; no call reaches the library."""
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
