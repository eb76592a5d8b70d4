"""MI355X (gfx950) routed-expert forward of an MXFP4 Stable LatentMoE layer.

The compute path is the HIP library ``libmxmoe.so`` behind the C ABI in ``include/mxmoe.h``;
``abi`` binds it with ctypes and ``MoELayer`` manages device buffers with torch. ``dense`` is the dense
path around the layer: ``rms_norm``, ``block_norm``, ``quantise``, ``dequantise``, ``Int8Linear``, ``Bf16Linear``,
``Int8FeedForward``.
"""
from . import abi  # noqa: F401

_DENSE = ("rms_norm", "block_norm", "quantise", "dequantise", "Int8Linear", "Bf16Linear", "Int8FeedForward")
__all__ = ["abi", "MoELayer", *_DENSE]


def __getattr__(name):
    if name == "MoELayer":
        from .layer import MoELayer
        return MoELayer
    if name in _DENSE:
        from . import dense
        globals().update({n: getattr(dense, n) for n in _DENSE})
        return globals()[name]
    raise AttributeError(name)
