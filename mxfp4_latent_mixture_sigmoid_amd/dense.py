"""The dense 8-bit path around the mixture layer: RMS norm with the residual's addition, quantisation
per token, products of 8-bit codes (plain and gated), and a dense feed-forward block of them.

Torch provides device memory and the stream; all arithmetic runs in the HIP library. Codes are int8
[rows, width] tensors with one FP32 scale per row. Row-major tensors may be views with any row stride of at
least their width; their last dimension has to be contiguous. Calls run on ``stream`` (default: the current stream).
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import abi

_TYPES = {torch.bfloat16: abi.TYPE_BF16, torch.float32: abi.TYPE_F32}
_BF16, _INT8 = (torch.bfloat16,), (torch.int8,)
_INT32_MAX = 2 ** 31 - 1   # rows and columns cross the C ABI as 32-bit integers, which ctypes cuts without a word
_pack = abi.NORM_ARGS.pack
_raw_stream = torch._C._cuda_getCurrentRawStream   # of a GPU: its handle, without an object around it
_current_gpu = torch._C._cuda_getDevice


def _ptr(t):
    return 0 if t is None else t.data_ptr()


class Normed(NamedTuple):
    """What ``rms_norm`` was asked for; None for the rest."""
    out: torch.Tensor | None
    codes: torch.Tensor | None
    scales: torch.Tensor | None
    sum: torch.Tensor | None


def _bad_rows(name, t, dtypes, index, shape):
    """Why `t` is not the matrix that _rows wants."""
    if t.dtype not in dtypes:
        return f"{name}: {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}"
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        return (f"{name}: expected two dimensions with contiguous rows, got shape {tuple(t.shape)}, "
                f"strides {t.stride()}")
    if shape is not None and t.shape != shape:
        return f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}"
    if max(t.shape) > _INT32_MAX:
        return f"{name}: shape {tuple(t.shape)}, expected at most {_INT32_MAX} rows and columns"
    return f"{name}: on {t.device}, expected GPU {index}"


def _rows(name, t, dtypes, index, shape=None):
    """Row stride of a [T, width] tensor on GPU `index`, after checking it."""
    strides, sizes = t.stride(), t.shape
    if (t.dtype not in dtypes or len(strides) != 2 or (strides[1] != 1 and sizes[1] > 1)
            or (shape is not None and sizes != shape) or sizes[0] > _INT32_MAX or sizes[1] > _INT32_MAX
            or t.get_device() != index):
        raise ValueError(_bad_rows(name, t, dtypes, index, shape))
    # the stride of a single row means nothing (torch reports any value there)
    return strides[0] if sizes[0] > 1 else sizes[1]


def _vector(name, t, n, dtype, index):
    if t.dtype != dtype or t.shape != (n,) or (n > 1 and t.stride(0) != 1) or t.get_device() != index:
        raise ValueError(f"{name}: expected a contiguous {dtype} [{n}] on GPU {index}, got {t.dtype} {tuple(t.shape)} "
                         f"on {t.device}")


def _call(x, stream, tensors, f, *args):
    """f(*args, GPU index, stream handle) with x's GPU current, on `stream` when one is given: outputs
    are then allocated for it, and the allocator learns that it uses tensors of other streams. (The public
    functions make the bare call themselves on the current GPU and stream: its latency counts for
    single tokens, and this one costs 0.5 us.)"""
    index = x.get_device()
    if index < 0:
        raise ValueError(f"expected tensors on a GPU, got one on {x.device}")
    if stream is None:
        with torch.cuda.device(index):
            return f(*args, index, _raw_stream(index))
    if stream.device_index != index:
        raise ValueError(f"stream: on GPU {stream.device_index}, expected GPU {index}")
    with torch.cuda.stream(stream):
        got = f(*args, index, stream.cuda_stream)
    for t in tensors:
        if torch.is_tensor(t):
            t.record_stream(stream)
    return got


def _output(name, want, x, dtype, index):
    """(tensor, row stride) of an output of x's shape asked for by True, given as a tensor, or not wanted."""
    if want is True:
        return torch.empty_like(x, dtype=dtype), x.shape[1]
    if want is None or want is False:
        return None, 0
    return want, _rows(name, want, (dtype,), index, x.shape)


def rms_norm(x, weight=None, eps=1e-6, delta=None, sum=None, out=True, codes=False, scales=None, stream=None) -> Normed:
    """s = x + delta; y = s / sqrt(mean(s^2) + eps) * weight, row by row in FP32.

    x: [T, H] BF16 or FP32; delta, weight: BF16, optional. Each of ``sum`` (s in x's type), ``out`` (y in
    BF16) and ``codes`` (y as int8, with ``scales`` = max|y| / 127 per row) is False, True (allocated
    here) or a tensor to write into; ``sum`` may be x itself. A row of zeros has scale 0; a row with a
    NaN or an infinity has scale NaN and codes 0."""
    if stream is None and (index := x.get_device()) >= 0 and index == _current_gpu():
        return _rms_norm(x, weight, eps, delta, sum, out, codes, scales, index, _raw_stream(index))
    return _call(x, stream, (x, weight, delta, sum, out, codes, scales), _rms_norm, x, weight, eps, delta, sum, out, codes,
                 scales)


def _rms_norm(x, weight, eps, delta, sum, out, codes, scales, index, stream):
    ldx = _rows("x", x, _TYPES, index)
    T, H = x.shape
    dtype, ldd = x.dtype, 0
    if delta is not None:
        ldd = _rows("delta", delta, _BF16, index, x.shape)
    if weight is not None:
        _vector("weight", weight, H, torch.bfloat16, index)
    s, lds = _output("sum", sum, x, dtype, index)
    o, ldo = _output("out", out, x, torch.bfloat16, index)
    q, ldc = _output("codes", codes, x, torch.int8, index)
    if scales is not None:
        if q is None:
            raise ValueError("scales given without codes")
        _vector("scales", scales, T, torch.float32, index)
    elif q is not None:
        scales = torch.empty(T, dtype=torch.float32, device=x.device)
    ptr = _ptr
    status = abi.lib().moe_norm(_pack(x.data_ptr(), ptr(delta), ptr(weight), ptr(s), ptr(o), ptr(q), ptr(scales), ldx, ldd,
                                      lds, ldo, ldc, T, H, _TYPES[dtype], eps), stream)
    if status:
        raise abi.MoEError(status, "moe_norm")
    return Normed(o, q, scales, s)


def quantise(x, codes=None, scales=None, stream=None):
    """Rows of x ([T, K] BF16 or FP32) as int8 codes with a scale each: scale = max|x| / 127,
    codes = x / scale rounded to nearest even. Returns (codes, scales), into the given tensors if any."""
    if stream is None and (index := x.get_device()) >= 0 and index == _current_gpu():
        return _quantise(x, codes, scales, index, _raw_stream(index))
    return _call(x, stream, (x, codes, scales), _quantise, x, codes, scales)


def _quantise(x, codes, scales, index, stream):
    ldx = _rows("x", x, _TYPES, index)
    T, K = x.shape
    q, ldc = _output("codes", True if codes is None else codes, x, torch.int8, index)
    if scales is None:
        scales = torch.empty(T, dtype=torch.float32, device=x.device)
    else:
        _vector("scales", scales, T, torch.float32, index)
    status = abi.lib().moe_quantise(x.data_ptr(), _TYPES[x.dtype], ldx, T, K, q.data_ptr(), ldc, scales.data_ptr(), stream)
    if status:
        raise abi.MoEError(status, "moe_quantise")
    return q, scales


def dequantise(codes, scales, out=None, stream=None):
    """The values that codes stand for, bf16(codes * scales[:, None])."""
    if stream is None and (index := codes.get_device()) >= 0 and index == _current_gpu():
        return _dequantise(codes, scales, out, index, _raw_stream(index))
    return _call(codes, stream, (codes, scales, out), _dequantise, codes, scales, out)


def _dequantise(codes, scales, out, index, stream):
    ldc = _rows("codes", codes, _INT8, index)
    T, K = codes.shape
    _vector("scales", scales, T, torch.float32, index)
    o, ldo = _output("out", True if out is None else out, codes, torch.bfloat16, index)
    status = abi.lib().moe_dequantise(codes.data_ptr(), ldc, scales.data_ptr(), T, K, o.data_ptr(), ldo, stream)
    if status:
        raise abi.MoEError(status, "moe_dequantise")
    return o


class Int8Linear:
    """A dense product of 8-bit codes with weights packed once: out = (x . w^T) * sx * scales + bias, or
    with ``up_codes`` the gated form silu((x . w^T) * sx * scales) * ((x . w_up^T) * sx * up_scales).

    codes, up_codes: int8 [N, K]; scales, up_scales: FP32 [N]; bias: FP32 [N]. They are read only while
    the packing kernel runs on ``stream`` and may be dropped after construction. Beside the packed weights a
    layer holds no device memory, and its calls may overlap on different streams; a call whose rows have to be laid
    out first (many unaligned ones) allocates room for them."""

    def __init__(self, codes, scales, bias=None, up_codes=None, up_scales=None, T_max=8192, out_dtype=torch.bfloat16,
                 stream=None):
        self.handle = None
        if out_dtype not in _TYPES:
            raise ValueError(f"out_dtype: {out_dtype}, expected bfloat16 or float32")
        if (up_codes is None) != (up_scales is None):
            raise ValueError("up_codes and up_scales go together")
        if up_codes is not None and bias is not None:
            raise ValueError("the gated product takes no bias")
        if not 0 <= T_max <= _INT32_MAX:
            raise ValueError(f"T_max: {T_max}, expected 0 to {_INT32_MAX}")
        self.T_max, self.out_dtype = T_max, out_dtype
        _call(codes, stream, (codes, scales, bias, up_codes, up_scales), self._create, codes, scales, bias, up_codes,
              up_scales)

    def _create(self, codes, scales, bias, up_codes, up_scales, index, stream):
        codes = codes.contiguous()   # weights may be views in any order
        _rows("codes", codes, _INT8, index)
        self.N, self.K = codes.shape
        _vector("scales", scales, self.N, torch.float32, index)
        if up_codes is not None:
            up_codes = up_codes.contiguous()
            _rows("up_codes", up_codes, _INT8, index, codes.shape)
            _vector("up_scales", up_scales, self.N, torch.float32, index)
        if bias is not None:
            _vector("bias", bias, self.N, torch.float32, index)
        self.cfg = abi.LinearConfig(self.N, self.K, int(up_codes is not None), _TYPES[self.out_dtype])
        packed_bytes, _ = abi.linear_query(self.cfg, self.T_max)
        self.packed = torch.empty(packed_bytes, dtype=torch.uint8, device=codes.device)
        self.handle = abi.linear_create(self.cfg, codes, scales, up_codes, up_scales, bias, self.packed, stream)
        self._two_rows = abi.linear_query(self.cfg, 2)[1]   # room for rows is in proportion to them, up to its alignment
        self._streams = {stream}   # that the allocator knows to use the weights: their own, and those of the calls

    def forward(self, x, scales, out=None, stream=None):
        """The product for codes x [T, K] with FP32 scales [T]; returns out [T, N]."""
        if stream is None and (index := self.packed.get_device()) == _current_gpu():
            return self._forward(x, scales, out, index, _raw_stream(index))
        return _call(self.packed, stream, (x, scales, out), self._forward, x, scales, out)

    def _forward(self, x, scales, out, index, stream):
        ldx = _rows("x", x, _INT8, index)
        T, K = x.shape
        if K != self.K or T > self.T_max:
            raise ValueError(f"x: shape {tuple(x.shape)}, expected at most {self.T_max} rows of {self.K}")
        _vector("scales", scales, T, torch.float32, index)
        if out is None:
            ldo = self.N   # the strided form is the cheaper call, by 0.35 us
            out = torch.empty_strided((T, ldo), (ldo, 1), dtype=self.out_dtype, device=x.device)
        else:
            ldo = _rows("out", out, (self.out_dtype,), index, (T, self.N))
        if stream not in self._streams:   # once for each: a layer dropped while it runs there keeps its memory that long
            self.packed.record_stream(torch.cuda.current_stream(index))
            self._streams.add(stream)
        forward = abi.lib().moe_linear_forward
        status = forward(self.handle, x.data_ptr(), ldx, scales.data_ptr(), T, out.data_ptr(), ldo, None, 0, stream)
        if status == abi.Status.BUFFER_TOO_SMALL:   # rows to be laid out first
            size = (T + 1) // 2 * self._two_rows   # asking again would take 1 us
            room = torch.empty(size, dtype=torch.uint8, device=x.device)
            status = forward(self.handle, x.data_ptr(), ldx, scales.data_ptr(), T, out.data_ptr(), ldo, room.data_ptr(),
                             size, stream)
        if status:
            raise abi.MoEError(status, "moe_linear_forward")
        return out

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
