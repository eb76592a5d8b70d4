"""The dense 8-bit path around the mixture layer: RMS norm with the residual's addition, quantisation
per token, products of 8-bit codes (plain and gated), and a dense feed-forward block of them.

Torch provides device memory and the stream; all arithmetic runs in the HIP library. Codes are int8
[rows, width] tensors with one FP32 scale per row. Row-major inputs may be views with any row stride;
their last dimension has to be contiguous. Calls run on ``stream`` (default: the current stream).
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import abi

_TYPES = {torch.bfloat16: abi.TYPE_BF16, torch.float32: abi.TYPE_F32}
_byref = ctypes.byref


class Normed(NamedTuple):
    """What ``rms_norm`` was asked for; None for the rest."""
    out: torch.Tensor | None
    codes: torch.Tensor | None
    scales: torch.Tensor | None
    sum: torch.Tensor | None


def _rows(name, t, dtypes, device=None, shape=None):
    """Row stride of a [T, width] tensor, after checking it."""
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}: expected two dimensions with contiguous rows, got shape {tuple(t.shape)}, "
                         f"strides {t.stride()}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name}: on {t.device}, expected {device if device is not None else 'a GPU'}")
    # the stride of a single row means nothing to the caller (torch reports any value there)
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _vector(name, t, n, dtype, device):
    if t.dtype != dtype or t.shape != (n,) or (n > 1 and t.stride(0) != 1) or t.device != device:
        raise ValueError(f"{name}: expected a contiguous {dtype} [{n}] on {device}, got {t.dtype} {tuple(t.shape)} "
                         f"on {t.device}")


class _on:
    """Makes `device`, and `stream` when given, current around the allocation of outputs and the launch,
    and lets the allocator know that `stream` uses tensors of other streams."""

    def __init__(self, device, stream, *tensors):
        self.device, self.stream, self.tensors = device, stream, tensors

    def __enter__(self):
        self.guard = torch.cuda.stream(self.stream) if self.stream is not None else torch.cuda.device(self.device)
        self.guard.__enter__()
        return abi.stream_handle()

    def __exit__(self, *exc):
        self.guard.__exit__(*exc)
        if self.stream is not None:
            for t in self.tensors:
                if t is not None:
                    t.record_stream(self.stream)


def _output(name, want, T, width, dtype, device):
    """(tensor, row stride) of an output asked for by True, given as a tensor, or not wanted."""
    if want is None or want is False:
        return None, 0
    if want is True:
        return torch.empty(T, width, dtype=dtype, device=device), width
    return want, _rows(name, want, (dtype,), device, (T, width))


def rms_norm(x, weight=None, eps=1e-6, delta=None, sum=None, out=True, codes=False, scales=None, stream=None) -> Normed:
    """s = x + delta; y = s / sqrt(mean(s^2) + eps) * weight, row by row in FP32.

    x: [T, H] BF16 or FP32; delta, weight: BF16, optional. Each of ``sum`` (s in x's type), ``out`` (y in
    BF16) and ``codes`` (y as int8, with ``scales`` = max|y| / 127 per row) is False, True (allocated
    here) or a tensor to write into; ``sum`` may be x itself. A row of zeros has scale 0; a row with a
    NaN or an infinity has scale NaN and codes 0."""
    ldx = _rows("x", x, _TYPES)
    T, H = x.shape
    dev = x.device
    ldd = _rows("delta", delta, (torch.bfloat16,), dev, x.shape) if delta is not None else 0
    if weight is not None:
        _vector("weight", weight, H, torch.bfloat16, dev)
    with _on(dev, stream, x, delta, weight, *(t for t in (sum, out, codes, scales) if torch.is_tensor(t))) as st:
        s, lds = _output("sum", sum, T, H, x.dtype, dev)
        o, ldo = _output("out", out, T, H, torch.bfloat16, dev)
        q, ldc = _output("codes", codes, T, H, torch.int8, dev)
        if q is None:
            if scales is not None:
                raise ValueError("scales given without codes")
        elif scales is None:
            scales = torch.empty(T, dtype=torch.float32, device=dev)
        else:
            _vector("scales", scales, T, torch.float32, dev)
        a = abi.NormArgs(abi.ptr(x), abi.ptr(delta), abi.ptr(weight), abi.ptr(s), abi.ptr(o), abi.ptr(q),
                         abi.ptr(scales), ldx, ldd, lds, ldo, ldc, T, H, _TYPES[x.dtype], eps)
        abi.check(abi.lib().moe_norm(_byref(a), st), "moe_norm")
    return Normed(o, q, scales, s)


def quantise(x, codes=None, scales=None, stream=None):
    """Rows of x ([T, K] BF16 or FP32) as int8 codes with a scale each: scale = max|x| / 127,
    codes = x / scale rounded to nearest even. Returns (codes, scales), into the given tensors if any."""
    ldx = _rows("x", x, _TYPES)
    T, K = x.shape
    dev = x.device
    with _on(dev, stream, x, codes, scales) as st:
        q, ldc = _output("codes", True if codes is None else codes, T, K, torch.int8, dev)
        if scales is None:
            scales = torch.empty(T, dtype=torch.float32, device=dev)
        else:
            _vector("scales", scales, T, torch.float32, dev)
        abi.check(abi.lib().moe_quantise(abi.ptr(x), _TYPES[x.dtype], ldx, T, K, abi.ptr(q), ldc, abi.ptr(scales), st),
                  "moe_quantise")
    return q, scales


def dequantise(codes, scales, out=None, stream=None):
    """The values that codes stand for, bf16(codes * scales[:, None])."""
    ldc = _rows("codes", codes, (torch.int8,))
    T, K = codes.shape
    dev = codes.device
    _vector("scales", scales, T, torch.float32, dev)
    with _on(dev, stream, codes, scales, out) as st:
        o, ldo = _output("out", True if out is None else out, T, K, torch.bfloat16, dev)
        abi.check(abi.lib().moe_dequantise(abi.ptr(codes), ldc, abi.ptr(scales), T, K, abi.ptr(o), ldo, st),
                  "moe_dequantise")
    return o


class Int8Linear:
    """A dense product of 8-bit codes with weights packed once: out = (x . w^T) * sx * scales + bias, or
    with ``up_codes`` the gated form silu((x . w^T) * sx * scales) * ((x . w_up^T) * sx * up_scales).

    codes, up_codes: int8 [N, K]; scales, up_scales: FP32 [N]; bias: FP32 [N]. They are read only while
    the packing kernel runs on ``stream`` and may be dropped after construction. Calls of one layer
    that overlap on different streams share its workspace and have to be serialised by the caller."""

    def __init__(self, codes, scales, bias=None, up_codes=None, up_scales=None, T_max=8192, out_dtype=torch.bfloat16,
                 stream=None):
        self.handle = None
        if out_dtype not in _TYPES:
            raise ValueError(f"out_dtype: {out_dtype}, expected bfloat16 or float32")
        if (up_codes is None) != (up_scales is None):
            raise ValueError("up_codes and up_scales go together")
        if up_codes is not None and bias is not None:
            raise ValueError("the gated product takes no bias")
        _rows("codes", codes, (torch.int8,))
        self.N, self.K = codes.shape
        self.device, self.T_max, self.out_dtype = codes.device, T_max, out_dtype
        _vector("scales", scales, self.N, torch.float32, self.device)
        if up_codes is not None:
            _rows("up_codes", up_codes, (torch.int8,), self.device, codes.shape)
            _vector("up_scales", up_scales, self.N, torch.float32, self.device)
        if bias is not None:
            _vector("bias", bias, self.N, torch.float32, self.device)
        self.cfg = abi.LinearConfig(self.N, self.K, int(up_codes is not None), _TYPES[out_dtype])
        packed_bytes, ws_bytes = abi.linear_query(self.cfg, T_max)
        with _on(self.device, stream, codes, scales, bias, up_codes, up_scales):
            codes = codes.contiguous()
            up_codes = up_codes.contiguous() if up_codes is not None else None
            self.packed = torch.empty(packed_bytes, dtype=torch.uint8, device=self.device)
            self.workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=self.device)
            self.handle = abi.linear_create(self.cfg, codes, scales, up_codes, up_scales, bias, self.packed)

    def forward(self, x, scales, out=None, stream=None):
        """The product for codes x [T, K] with FP32 scales [T]; returns out [T, N]."""
        ldx = _rows("x", x, (torch.int8,), self.device)
        T = x.shape[0]
        if x.shape[1] != self.K or T > self.T_max:
            raise ValueError(f"x: shape {tuple(x.shape)}, expected at most {self.T_max} rows of {self.K}")
        _vector("scales", scales, T, torch.float32, self.device)
        with _on(self.device, stream, x, scales, out, self.packed, self.workspace) as st:
            o, ldo = _output("out", True if out is None else out, T, self.N, self.out_dtype, self.device)
            abi.check(abi.lib().moe_linear_forward(self.handle, abi.ptr(x), ldx, abi.ptr(scales), T, abi.ptr(o), ldo,
                                                   abi.ptr(self.workspace), self.workspace.numel(), st),
                      "moe_linear_forward")
        return o

    def close(self):
        if self.handle:
            abi.linear_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Int8FeedForward:
    """A dense feed-forward block in 8 bits, in the place of a mixture layer: residual addition and RMS
    norm, gated product, quantisation, down product.

    norm_weight: BF16 [H]; gate, up, down: (codes, scales) pairs, int8 [I, H], [I, H] and [H, I]."""

    def __init__(self, norm_weight, gate, up, down, T_max, eps=1e-6, stream=None):
        self.norm_weight, self.eps = norm_weight, eps
        self.gated = Int8Linear(*gate, up_codes=up[0], up_scales=up[1], T_max=T_max, stream=stream)
        self.down = Int8Linear(*down, T_max=T_max, stream=stream)

    def forward(self, x, delta=None, stream=None):
        """The residual stream x [T, H] and the last block's output delta (BF16, added to it first) ->
        (this block's output in BF16, the residual stream to add it to)."""
        r = rms_norm(x, self.norm_weight, self.eps, delta=delta, sum=delta is not None, out=False, codes=True,
                     stream=stream)
        h = self.gated.forward(r.codes, r.scales, stream=stream)
        codes, scales = quantise(h, stream=stream)
        return self.down.forward(codes, scales, stream=stream), r.sum if delta is not None else x

    def close(self):
        self.gated.close()
        self.down.close()
