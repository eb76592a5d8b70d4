"""MoELayer: owns the packed weights, workspace and routing buffers of one layer on one GPU and
calls the C ABI (torch provides device memory and the stream; all arithmetic runs in HIP)."""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import abi


class Decoded(NamedTuple):
    """What ``MoELayer.decode`` computes: the layer's output, and the experts of each token with their weights."""
    out: torch.Tensor       # BF16 [T, H] ([T, latent] without latent projections)
    ids: torch.Tensor       # int32 [T, K], in rank order
    weights: torch.Tensor   # FP32 [T, K]


def _dense(name, t, shape, dtype, index):
    """t, checked to be a contiguous tensor of that shape and type on GPU `index`; a new one where it is None."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", index))
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != index:
        raise ValueError(f"{name}: expected a contiguous {dtype} {list(shape)} on GPU {index}, got {t.dtype} "
                         f"{list(t.shape)} on {t.device}")
    return t


class MoELayer:
    """One MXFP4 latent-MoE layer on the current GPU.

    ``weights`` maps the canonical weight names of ``abi.WEIGHT_FIELDS`` to device tensors
    (BF16 bit patterns as int16/bfloat16, MXFP4 codes/scales as uint8); they are only read while
    the packing kernels run and may be dropped after the first synchronisation.

    ``stage2_fp8`` quantises h to MX FP8 for the down product (MOE_STAGE2_FP8); ``stage1_a4``
    quantises z to MX FP4 for the gate/up product (MOE_STAGE1_MXFP4, A4W4). Both default to the
    BF16 layer; each adds one packed copy of the weights it changes. ``shared_stream`` runs the
    shared experts' gate/up product on a second stream owned by the handle, concurrently with the
    routing and the routed experts (MOE_SHARED_STREAM); the outputs are the same bits.
    """

    def __init__(self, hidden, latent, n_experts, top_k, inter, n_shared, shared_inter,
                 has_latent_proj, weights: dict, T_max: int, device="cuda", stream=None,
                 stage2_fp8: bool = False, stage1_a4: bool = False, shared_stream: bool = False):
        self.cfg = abi.make_config(hidden, latent, n_experts, top_k, inter, n_shared, shared_inter,
                                   has_latent_proj, stage2_fp8, stage1_a4, shared_stream)
        self.E, self.K, self.Lt = n_experts, top_k, latent
        self.H = hidden if has_latent_proj else latent
        self.T_max = T_max
        packed_bytes, ws_bytes = abi.query(self.cfg, T_max)
        self.device = torch.device(device)
        self.packed = torch.empty(packed_bytes, dtype=torch.uint8, device=self.device)
        self.workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=self.device)
        self.handle = abi.create(self.cfg, weights, self.packed, stream)
        self._decode_bytes, self._streams = {}, set()   # decode's workspace by token count; streams that its calls ran on

    def alloc_routing(self, T: int) -> dict:
        d, P = self.device, max(T * self.K, 1)
        i32 = dict(dtype=torch.int32, device=d)
        return dict(topk_ids=torch.empty(max(T, 1), self.K, **i32),
                    topk_w=torch.empty(max(T, 1), self.K, dtype=torch.float32, device=d),
                    counts=torch.empty(self.E, **i32), offsets=torch.empty(self.E + 1, **i32),
                    sorted_pairs=torch.empty(P, **i32), inv=torch.empty(P, **i32))

    def _check_T(self, T):
        if T > self.T_max:
            raise ValueError(f"T={T} exceeds T_max={self.T_max}")

    def route(self, x, T, routing, logit_bias=None, logits_in=None, logits_out=None, stream=None):
        self._check_T(T)
        abi.route(self.handle, x, T, routing, self.workspace, logit_bias, logits_in, logits_out, stream)

    def forward(self, x, T, routing, out=None, stream=None):
        self._check_T(T)
        if out is None:
            out = torch.empty(max(T, 1), self.H, dtype=torch.bfloat16, device=self.device)
        abi.forward(self.handle, x, T, routing, out, self.workspace, stream)
        return out

    def route_forward(self, x, T, routing, out=None, logit_bias=None, logits_out=None, stream=None):
        """route + forward in one call, bitwise identical to the two calls."""
        self._check_T(T)
        if out is None:
            out = torch.empty(max(T, 1), self.H, dtype=torch.bfloat16, device=self.device)
        abi.route_forward(self.handle, x, T, routing, out, self.workspace, logit_bias, logits_out, stream)
        return out

    def route_forward_static(self, x, T, routing, out=None, logit_bias=None, logits_out=None, stream=None):
        """route + forward in the library's per-GPU scratch array instead of this layer's workspace
        (the call allocates nothing; bitwise identical to route_forward)."""
        if out is None:
            out = torch.empty(max(T, 1), self.H, dtype=torch.bfloat16, device=self.device)
        abi.route_forward_static(self.handle, x, T, routing, out, logit_bias, logits_out, stream)
        return out

    def decode(self, x, out=None, logit_bias=None, logits_out=None, ids=None, weights=None, stream=None) -> Decoded:
        """The whole layer for x [T, Hin] BF16 of at most 16 tokens, in one launch (and a small one that clears its
        counters): what route_forward computes, without its routing arrays, nearer to the exact result (z, the experts' inner
        values and the weighted sum are held in 16 bits, an expert's output in FP32, where route_forward rounds each to
        BF16's 8), and a token's outputs are the same bits whatever tokens come with it. Of one GPU's TP8 share 54 us for one
        token (route_forward 68), 75 for 4 (82), 99 for 8 (103), 122 for 9 (107), 166 for 16 (136): above eight tokens
        route_forward is the faster one. Outputs go into the given tensors if any (contiguous; logits_out FP32 [T, E]). The
        call allocates its own workspace, so that calls may overlap on different streams and in
        captured graphs."""
        index = self.packed.get_device()
        if stream is not None and stream.device_index != index:
            raise ValueError(f"stream: on GPU {stream.device_index}, expected GPU {index}")
        if stream is None:
            with torch.cuda.device(index):
                return self._decode(x, out, logit_bias, logits_out, ids, weights, index,
                                    torch.cuda.current_stream(index).cuda_stream)
        with torch.cuda.stream(stream):   # what is allocated here belongs to it
            got = self._decode(x, out, logit_bias, logits_out, ids, weights, index, stream.cuda_stream)
        for t in (x, out, logit_bias, logits_out, ids, weights):
            if t is not None:
                t.record_stream(stream)
        return got

    def _decode(self, x, out, logit_bias, logits_out, ids, weights, index, stream):
        Hin = self.H if self.cfg.has_latent_proj else self.Lt
        if x.dim() != 2 or x.shape[1] != Hin or x.shape[0] > abi.DECODE_MAX_T:
            raise ValueError(f"x: shape {tuple(x.shape)}, expected at most {abi.DECODE_MAX_T} rows of {Hin}")
        T = x.shape[0]
        x = _dense("x", x, (T, Hin), torch.bfloat16, index)
        out = _dense("out", out, (T, self.H), torch.bfloat16, index)
        ids = _dense("ids", ids, (T, self.K), torch.int32, index)
        weights = _dense("weights", weights, (T, self.K), torch.float32, index)
        if logit_bias is not None:
            _dense("logit_bias", logit_bias, (self.E,), torch.float32, index)
        if logits_out is not None:
            _dense("logits_out", logits_out, (T, self.E), torch.float32, index)
        size = self._decode_bytes.get(T)
        if size is None:
            size = self._decode_bytes[T] = abi.decode_query(self.cfg, T)
        room = torch.empty(size, dtype=torch.uint8, device=x.device)
        if stream not in self._streams:   # once for each: a layer dropped while it runs there keeps its memory that long
            self.packed.record_stream(torch.cuda.current_stream(index))
            self._streams.add(stream)
        abi.check(abi.lib().moe_decode(self.handle, x.data_ptr(), T, abi.ptr(logit_bias), abi.ptr(logits_out), ids.data_ptr(),
                                       weights.data_ptr(), out.data_ptr(), room.data_ptr(), size, stream), "moe_decode")
        return Decoded(out, ids, weights)

    def graph(self, x, T, routing, out, logit_bias=None, logits_out=None):
        """route_forward captured as one HIP graph on these buffers (see StepGraph)."""
        self._check_T(T)
        return StepGraph(self, abi.graph_create(self.handle, x, T, routing, out, self.workspace, logit_bias,
                                                logits_out), (x, routing, out, logit_bias, logits_out))

    def unpack_expert(self, e: int, which: int, stream=None):
        rows, cols = (self.cfg.inter, self.Lt) if which < 2 else (self.Lt, self.cfg.inter)
        out = torch.empty(rows, cols, dtype=torch.bfloat16, device=self.device)
        abi.unpack_expert(self.handle, e, which, out, stream)
        return out

    def workspace_view(self, T: int, region: str, shape, dtype):
        """Tensor view of a workspace region (test hook)."""
        off = abi.workspace_layout(self.cfg, T)[region]
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.empty(0, dtype=dtype).element_size()
        return self.workspace[off:off + nbytes].view(dtype).view(*shape)

    def close(self):
        if self.handle:
            abi.destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class StepGraph:
    """One captured route_forward: launch() replays it on the buffers it was captured with (write
    each step's tokens into the same x tensor). Holds references to those buffers and the layer."""

    def __init__(self, layer, g, buffers):
        self.layer, self.g, self.buffers = layer, g, buffers

    def launch(self, stream=None):
        if not self.g:
            raise RuntimeError("graph destroyed")
        abi.graph_launch(self.g, stream)

    def close(self):
        if self.g:
            abi.graph_destroy(self.g)
            self.g = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
