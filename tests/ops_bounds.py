"""Bounds on the errors of the cross-entropy kernels, element by element, from their arithmetic (used by the tests).

u = 2^-24 is half a step of a 32-bit number, relative to it.
  exp(d): d = x - m rounds by u relative to d, its product with log2 e by u more: the power is off by 2 |d| u, and a step
      (2 u) of the hardware's power of two, one for the rounding of log2 e itself.
  s: a thread adds eight powers of a vector and rescales by a power when its maximum grows; then the sums of 64 lanes meet
      in six steps and those of 16 wavefronts in 15.  A step rounds by u for its sum, and by u for a product with a power that
      is itself off by 3 u and by 2 u for every unit that the maximum grew.  On any way through the row the maximum
      grows by no more than the finite logits' range.
  log(s): a step of the hardware's logarithm to base 2, its product with log 2, the addition."""
import numpy as np

from ops_plain import SMALLEST, rounding, type_name

U = 2.0 ** -24


def _finite(x):
    return np.where(np.isfinite(x), x, np.nan)


def parts(x, threads_vectors):
    """(m, p, relative error bound of s) per row of finite or -inf logits; rows of -inf alone give NaN."""
    with np.errstate(all="ignore"):
        m = x.max(axis=1, keepdims=True)
        d = m - x
        e = np.exp(-d)
        s = e.sum(axis=1, keepdims=True)
        p = e / s
        dd = np.where(np.isfinite(d), d, 0.0)
        low = np.nanmin(_finite(x), axis=1, keepdims=True)
        grown = np.clip(m - low, 0, 104)     # a power of less is zero
        own = (p * (2 * np.minimum(dd, 104) + 4)).sum(axis=1, keepdims=True)
    return m, s, p, U * (own + 2 * grown + 13 * threads_vectors + 5 * 21)


def threads_vectors(vocab):
    """Vectors of a thread, at the fewest threads of a row of this length (256 up to 8,192 elements, and for pieces of 8,192)."""
    return -(-vocab // 2048) if vocab <= 8192 else -(-vocab // 4096) if vocab <= 32768 else -(-vocab // 8192)


def loss(x, y):
    """(loss, its error bound) of rows x with targets y, none ignored, of which no row is -inf alone."""
    m, s, _, rel = parts(x, threads_vectors(x.shape[1]))
    at = x[np.arange(len(x)), y][:, None]
    ref = (m - at) + np.log(s)
    err = rel + 4 * U * (np.log(s) + 1) + U * np.abs(m - at) + U * np.abs(ref)
    return ref[:, 0], err[:, 0]


FAR = 128.0   # the gradient from lse forms the sums of a row again from this |lse| on


def gradient(x, y, c, dtype, from_lse):
    """(gradient, its error bound) of rows x, targets y (none ignored) and factors c; no row is -inf alone.

    Fused, p_j = exp(x_j - m) / s: the power, the sum, the reciprocal and the product.  From lse: exp(x_j - lse) with
    the lse's own error (that of log s, and a rounding relative to lse), by rows of 256 threads where |lse| is FAR or more.
    c rounds once as a product, and the difference from one at the target, the product with c and the
    result in the output's type round once each.  The hardware's power of two has no subnormal results."""
    m, s, p, rel = parts(x, threads_vectors(x.shape[1]))
    with np.errstate(all="ignore"):
        d = np.where(np.isfinite(x), np.minimum(m - x, 104), 0.0)
        own = rel + U * (2 * d + 4 + 2)
        if from_lse:
            z = m + np.log(s)
            below = np.where(np.isfinite(x), np.minimum(np.abs(z - x), 104), 0.0)
            near = rel + 4 * U * (np.log(s) + 1) + U * np.abs(z) + U * (2 * below + 4)
            wide = parts(x, -(-x.shape[1] // 2048))[3] + U * (2 * d + 4 + 2)
            own = np.where(np.abs(z) < FAR, near, np.where(np.abs(z) > FAR + 1, wide, np.maximum(near, wide)))
    c = np.asarray(c)[:, None]
    hit = np.zeros_like(x)
    hit[np.arange(len(x)), y] = 1.0
    ref = c * (p - hit)
    err = np.abs(c) * (p * own + hit * U * np.abs(p - hit) + 2.0 ** -126) + 2 * U * np.abs(ref)
    return ref, err + rounding(np.abs(ref) + err, dtype)


def rounding_floor(dtype):
    return max(SMALLEST[type_name(dtype)], 2.0 ** -126)
