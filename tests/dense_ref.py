"""Plain 64-bit numpy forms of the dense 8-bit path, and the error each output may have.

Bounds, with u = 2^-24 (half an FP32 unit, 24 significant bits) and b = 2^-8 (half a BF16 unit, 8
significant bits): an FP32 result of n
roundings is off by at most about n u of its terms' magnitudes; one final rounding to BF16 adds b of
the result. Sums of squares are added by at most 1024 threads of at most 64 values and trees of 16
waves: under 128 u, halved by the square root."""
import numpy as np

U, B = 2.0 ** -24, 2.0 ** -8
NORM_REL = 80 * U        # y of the norm: 64 u from rstd, then its division, root and two products
TINY = 2.0 ** -148       # two units of the smallest FP32 subnormals


def norm(x, delta, weight, eps):
    s = x + (0 if delta is None else delta)
    with np.errstate(all="ignore"):
        y = s / np.sqrt((s * s).mean(1, keepdims=True) + eps)
        if weight is not None:
            y = y * weight
    return s, y


def scales(y):
    """max|y| / 127 per row, NaN where a value is not finite."""
    top = np.abs(y).max(1) if y.shape[0] else np.zeros(0)
    return np.where(np.isfinite(y).all(1), top / 127, np.nan)


def product(codes, w, sx, sw):
    return (codes.astype(np.int64) @ w.astype(np.int64).T).astype(np.float64) * sx[:, None] * sw


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g))


def check(got, ref, allowed, what):
    """|got - ref| <= allowed everywhere, with NaN and infinities where the reference has them."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN elsewhere than the reference's"
    inf = ~fine & ~np.isnan(ref)
    assert np.array_equal(got[inf], ref[inf]), f"{what}: infinities differ"
    over = np.abs(got - ref)[fine] - np.broadcast_to(allowed, ref.shape)[fine]
    assert over.size == 0 or over.max() <= 0, f"{what}: past the bound by {over.max()} at {int((over > 0).sum())} values"


def check_codes(codes, scale, y, rel, what):
    """codes and scales of rows y (64-bit), y known to `rel` by the kernel."""
    ref = scales(y)
    check(scale, ref, np.abs(ref) * (rel + 2 * U) + TINY, what + " scales")
    codes = codes.astype(np.float64)
    assert np.abs(codes).max(initial=0) <= 127, what
    dead = np.isnan(ref) | (ref == 0)
    assert not codes[dead].any(), f"{what}: codes of a row without a scale"
    live = ~dead
    # y / scale to within 127 (2 rel + 8 u), then half a code
    check(codes[live], y[live] / ref[live][:, None], 0.5 + 127 * (2 * rel + 8 * U), what + " codes")
