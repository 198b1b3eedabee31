"""The bounds of the cross-entropy tests reject gradients that are wrong (on the CPU: the mistakes are in what is compared)."""
import numpy as np
import pytest

import ops_bounds as bounds


def _rows(vocab, kind, seed=0):
    rng = np.random.default_rng(seed)
    x = 3.0 * rng.standard_normal((4, vocab))
    if kind == "peaked":
        x[:, 5] = 40.0
    elif kind == "equal":
        x[:] = 2.5
    elif kind == "far":
        x = np.float64(np.float32(x + 10000.0))
    return x, rng.integers(0, vocab, 4), rng.random(4) / 4


@pytest.mark.parametrize("vocab", [40, 1256, 9001, 131328])
@pytest.mark.parametrize("kind", ["plain", "equal", "far"])
@pytest.mark.parametrize("from_lse", [False, True])
def test_wrong_gradients_are_out_of_bounds(vocab, kind, from_lse):
    x, y, c = _rows(vocab, kind)
    for dtype, least in (("float32", 0.999), ("bfloat16", 0.999), ("float16", 0.4)):   # float16: most of a long row underflows
        ref, err = bounds.gradient(x, y, c, dtype, from_lse)
        sized = np.abs(ref) > 4 * bounds.rounding_floor(dtype)
        if dtype != "float16":
            assert sized.mean() > least
        assert (np.abs(ref) > err)[sized].all()                              # zeros
        if dtype == "float32":
            assert (0.01 * np.abs(ref) > err)[sized].mean() > 0.9999         # one per cent
        swapped = np.roll(ref, 1, axis=1)
        assert kind == "equal" or (np.abs(swapped - ref) > err)[sized].mean() > 0.8


def test_wrong_losses_are_out_of_bounds():
    for kind in ("plain", "equal", "far", "peaked"):
        x, y, _ = _rows(9001, kind)
        ref, err = bounds.loss(x, y)
        assert (1e-4 * np.maximum(ref, 1.0) > err).all()
        m = x.max(axis=1)
        lse = (m + np.log(np.exp(x - m[:, None]).sum(axis=1))).astype(np.float32).astype(np.float64)
        if kind == "far":
            assert (np.abs(lse - x[np.arange(4), y] - ref) > err).any()      # by way of the rounded lse
