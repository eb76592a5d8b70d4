"""Host-side checks of the dense 8-bit path's C ABI: sizes, and refusals before any GPU work."""
import ctypes
import os
import re

import pytest

from mxfp4_latent_mixture_sigmoid_amd import abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, UNSUPPORTED, SMALL = abi.Status.INVALID_ARG, abi.Status.UNSUPPORTED, abi.Status.BUFFER_TOO_SMALL
A = 1 << 20      # an aligned address that no refused call touches


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(abi.LIB_PATH):
        from mxfp4_latent_mixture_sigmoid_amd import build
        build.build()


def test_structs_follow_the_header():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mxmoe.h")).read(), flags=re.S)
    for name, cls in (("moe_norm_args", abi.NormArgs), ("moe_linear_config", abi.LinearConfig),
                      ("moe_linear_weights", abi.LinearWeights)):
        body = re.search(r"typedef struct \{([^}]*)\}\s*%s;" % name, src).group(1)
        fields = [f.strip().lstrip("*") for decl in body.split(";") if decl.strip()
                  for f in re.sub(r"^\s*(const\s+)?\w+\s", "", decl).split(",")]
        assert fields == [f for f, _ in cls._fields_], name
    assert f"MOE_LINEAR_MAX_K {abi.LINEAR_MAX_K}" in src


def _norm(**kw):
    a = dict(x=A, delta=None, weight=None, sum=None, out=A, codes=None, scales=None, ldx=64, ldd=64, lds=64, ldo=64,
             ldc=64, T=4, H=64, x_type=abi.TYPE_BF16, eps=1e-6)
    a.update(kw)
    return abi.lib().moe_norm(bytes(abi.NormArgs(**a)), None)


def test_packed_norm_arguments_are_the_structure():
    a = abi.NormArgs(*range(1, 16), 0.5)
    assert abi.NORM_ARGS.pack(*range(1, 16), 0.5) == bytes(a)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(H=0), dict(x_type=2), dict(eps=-1.0), dict(eps=float("nan")), dict(x=None), dict(out=None),
    dict(ldx=63), dict(ldo=63), dict(x=A + 1), dict(out=A + 1), dict(codes=A), dict(scales=A), dict(codes=A, scales=A + 2),
    dict(codes=A, scales=A, ldc=63), dict(delta=A, ldd=63), dict(delta=A + 1), dict(weight=A + 1), dict(sum=A, lds=65),
    dict(sum=A + 2, lds=63), dict(x_type=abi.TYPE_F32, x=A + 2), dict(x_type=abi.TYPE_F32, sum=A + 2)])
def test_norm_refuses(kw):
    assert _norm(**kw) == BAD


def test_null_arguments():
    L = abi.lib()
    assert L.moe_norm(None, None) == BAD
    assert L.moe_quantise(None, 0, 64, 4, 64, A, 64, A, None) == BAD
    assert L.moe_quantise(A, 0, 64, 4, 64, None, 64, A, None) == BAD
    assert L.moe_quantise(A, 0, 64, 4, 64, A, 64, None, None) == BAD
    assert L.moe_dequantise(None, 64, A, 4, 64, A, 64, None) == BAD
    assert L.moe_dequantise(A, 64, None, 4, 64, A, 64, None) == BAD
    assert L.moe_dequantise(A, 64, A, 4, 64, None, 64, None) == BAD
    assert L.moe_linear_query(None, 1, None, None) == BAD
    assert L.moe_linear_forward(None, A, 64, A, 4, A, 64, A, 1 << 20, None) == BAD
    L.moe_linear_destroy(None)


@pytest.mark.parametrize("args", [(A, 2, 64, 4, 64, A, 64, A), (A, 0, 63, 4, 64, A, 64, A), (A, 0, 64, 4, 64, A, 63, A),
                                  (A, 0, 64, -1, 64, A, 64, A), (A, 0, 64, 4, 0, A, 64, A), (A + 1, 0, 64, 4, 64, A, 64, A),
                                  (A, 0, 64, 4, 64, A, 64, A + 1)])
def test_quantise_refuses(args):
    assert abi.lib().moe_quantise(*args, None) == BAD


@pytest.mark.parametrize("args", [(A, 63, A, 4, 64, A, 64), (A, 64, A, 4, 64, A, 63), (A, 64, A, -1, 64, A, 64),
                                  (A, 64, A, 4, 0, A, 64), (A, 64, A, 4, 64, A + 1, 64), (A, 64, A + 2, 4, 64, A, 64)])
def test_dequantise_refuses(args):
    assert abi.lib().moe_dequantise(*args, None) == BAD


def test_no_tokens_touch_nothing():
    L = abi.lib()
    assert _norm(T=0, x=None) == abi.Status.OK
    assert L.moe_quantise(None, 0, 0, 0, 64, None, 0, None, None) == abi.Status.OK
    assert L.moe_dequantise(None, 0, None, 0, 64, None, 0, None) == abi.Status.OK


def _cfg(n=64, k=64, glu=0, out_type=0):
    return abi.LinearConfig(n, k, glu, out_type)


@pytest.mark.parametrize("kw", [dict(n=0), dict(k=0), dict(n=-1), dict(glu=2), dict(out_type=2)])
def test_linear_refuses_configs(kw):
    c = _cfg(**kw)
    assert abi.lib().moe_linear_query(ctypes.byref(c), 1, None, None) == BAD
    h = ctypes.c_void_p(5)
    w = abi.LinearWeights(A, A)
    assert abi.lib().moe_linear_create(ctypes.byref(c), ctypes.byref(w), A, 1 << 40, None, ctypes.byref(h)) == BAD
    assert h.value is None


def test_linear_sum_limit_and_token_limits():
    L = abi.lib()
    assert L.moe_linear_query(ctypes.byref(_cfg(k=abi.LINEAR_MAX_K)), 1, None, None) == abi.Status.OK
    assert L.moe_linear_query(ctypes.byref(_cfg(k=abi.LINEAR_MAX_K + 1)), 1, None, None) == UNSUPPORTED
    assert abi.LINEAR_MAX_K * 128 * 128 < 2 ** 31 <= (abi.LINEAR_MAX_K + 1) * 128 * 128
    assert L.moe_linear_query(ctypes.byref(_cfg()), -1, None, None) == BAD
    # more than 2^32 threads: 128 x 128 tiles of 512, packing or restaging 16 codes each
    assert L.moe_linear_query(ctypes.byref(_cfg(n=2 ** 16)), 2 ** 20, None, None) == abi.Status.OK
    assert L.moe_linear_query(ctypes.byref(_cfg(n=2 ** 16)), 2 ** 22, None, None) == BAD
    assert L.moe_linear_query(ctypes.byref(_cfg(n=1, k=1)), 2 ** 31 - 1, None, None) == BAD
    assert L.moe_linear_query(ctypes.byref(_cfg(n=2 ** 20, k=2 ** 17 - 1)), 1, None, None) == UNSUPPORTED
    assert L.moe_linear_query(ctypes.byref(_cfg(n=2 ** 31 - 1)), 1, None, None) == UNSUPPORTED


@pytest.mark.parametrize("n,k,glu", [(1, 1, 0), (16, 128, 0), (17, 129, 0), (100, 1000, 1), (7168, 4352, 0)])
def test_linear_packed_size(n, k, glu):
    """Rows padded to 16 (gate and up apart), codes to 128, then two FP32 vectors of the padded rows."""
    pb, _ = abi.linear_query(_cfg(n, k, glu), 4)
    rows, width = -(-n // 16) * 16 * (1 + glu), -(-k // 128) * 128
    assert rows * (width + 8) <= pb < rows * (width + 8) + 3 * 256


@pytest.mark.parametrize("w,packed,size,want", [
    (dict(), A, 1 << 30, BAD), (dict(w=A), A, 1 << 30, BAD), (dict(scales=A), A, 1 << 30, BAD),
    (dict(w=A, scales=A), None, 1 << 30, BAD), (dict(w=A, scales=A), A + 128, 1 << 30, BAD),
    (dict(w=A, scales=A, w_up=A, scales_up=A), A, 1 << 30, BAD), (dict(w=A, scales=A, scales_up=A), A, 1 << 30, BAD),
    (dict(w=A, scales=A + 2), A, 1 << 30, BAD), (dict(w=A, scales=A, bias=A + 1), A, 1 << 30, BAD),
    (dict(w=A, scales=A), A, 4096, SMALL)])
def test_linear_create_refuses(w, packed, size, want):
    h = ctypes.c_void_p(5)
    lw = abi.LinearWeights(**w)
    assert abi.lib().moe_linear_create(ctypes.byref(_cfg()), ctypes.byref(lw), packed, size, None, ctypes.byref(h)) == want
    assert h.value is None


@pytest.mark.parametrize("w", [dict(w=A, scales=A), dict(w=A, scales=A, w_up=A),
                               dict(w=A, scales=A, w_up=A, scales_up=A, bias=A)])
def test_gated_create_refuses(w):
    h = ctypes.c_void_p()
    lw = abi.LinearWeights(**w)
    assert abi.lib().moe_linear_create(ctypes.byref(_cfg(glu=1)), ctypes.byref(lw), A, 1 << 30, None,
                                       ctypes.byref(h)) == BAD


@pytest.mark.parametrize("n,k,glu", [(100, 1000, 0), (7168, 14336, 0), (14336, 7168, 1), (33, 20000, 0)])
def test_workspace_serves_every_smaller_batch(n, k, glu):
    c = _cfg(n, k, glu)
    sizes = sorted({0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500, 512, 513, 1024, 3000, 8192})
    need = [abi.linear_query(c, T)[1] for T in sizes]
    assert need == sorted(need)


@pytest.mark.parametrize("width", [abi.MAX_WIDTH + 1, 2 ** 31 - 8, 2 ** 31 - 7, 2 ** 31 - 1])
@pytest.mark.parametrize("T", [0, 1])
def test_rows_wider_than_the_kernels_indexes(width, T):
    """Columns are 32-bit indexes that go up in steps of 8192: wider rows would wrap, and are refused by all three."""
    L = abi.lib()
    assert abi.MAX_WIDTH == 2 ** 31 - 8192
    assert f"MOE_MAX_WIDTH {abi.MAX_WIDTH}" in open(os.path.join(ROOT, "include", "mxmoe.h")).read()
    assert _norm(H=width, T=T, ldx=width, ldo=width) == UNSUPPORTED
    assert L.moe_quantise(A, 0, width, T, width, A, width, A, None) == UNSUPPORTED
    assert L.moe_dequantise(A, width, A, T, width, A, width, None) == UNSUPPORTED
    assert _norm(H=abi.MAX_WIDTH, T=0) == abi.Status.OK


@pytest.mark.parametrize("n,k,glu", [(100, 1000, 0), (16, 1, 0), (14336, 7168, 1), (33, 20000, 0), (7, 127, 1)])
def test_workspace_is_in_proportion_to_the_tokens(n, k, glu):
    """What callers scale from the size for two tokens serves any number of them."""
    c = _cfg(n, k, glu)
    two = abi.linear_query(c, 2)[1]
    for T in (1, 2, 3, 7, 64, 129, 1000, 8191):
        need = abi.linear_query(c, T)[1]
        assert need <= (T + 1) // 2 * two < need + two
