"""Plain 64-bit implementations of the token operators, row by row (used by the tests), and the error
bounds that the kernels' arithmetic gives."""
import math

import numpy as np

HALF_STEP = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
# half the distance between the smallest numbers of the type: what rounding can lose below the normal range
SMALLEST = {"float32": 2.0 ** -150, "float16": 2.0 ** -25, "bfloat16": 2.0 ** -134}


def type_name(dtype):
    return str(dtype).replace("torch.", "")


def f64(t):
    """A tensor's values as a float64 array."""
    return t.detach().to("cpu").double().numpy()


def rounding(ref, dtype):
    """Error of one rounding to dtype of values near ref."""
    name = type_name(dtype)
    return HALF_STEP[name] * np.abs(ref) + SMALLEST[name]


def embed(table, ids, scale):
    ids = np.asarray(ids, dtype=np.int64)
    out = np.zeros((len(ids), table.shape[1]))
    for t, r in enumerate(ids):
        if 0 <= r < len(table):
            out[t] = scale * table[r]
    return out


def embed_backward(grad, ids, n_vocab, scale, base=None):
    """(gradient table, bound on the error of a 32-bit sum): every addition of a run of n rounds once, so the
    sum is off by at most n 2^-24 times the sum of magnitudes; scaling, and adding to the base, round once
    more each."""
    out = np.zeros((n_vocab, grad.shape[1]))
    size = np.zeros_like(out)
    count = np.zeros((n_vocab, 1))
    for t, r in enumerate(np.asarray(ids, dtype=np.int64)):
        if 0 <= r < n_vocab:
            out[r] += grad[t]
            size[r] += np.abs(grad[t])
            count[r] += 1
    out, size = scale * out, abs(scale) * size
    err = (count + 2) * 2.0 ** -24 * size
    if base is not None:
        err = err + 2.0 ** -24 * (np.abs(base) + size)
        out = out + base
    return out, err


def cross_entropy(x, y, c):
    """(loss, lse, gradient) of the rows of x for targets y (negative: ignored) and factors c."""
    rows, vocab = x.shape
    loss, lse, grad = np.zeros(rows), np.zeros(rows), np.zeros_like(x)
    for i in range(rows):
        row = x[i]
        bad = np.isnan(row).any() or np.isposinf(row).any()
        top = row.max() if not bad else math.nan
        if bad:
            lse[i] = math.nan
        elif np.isneginf(top):
            lse[i] = -math.inf
        else:
            lse[i] = top + math.log(np.exp(row - top).sum())
        if y[i] < 0 or y[i] >= vocab:
            continue
        if bad:
            loss[i], grad[i] = math.nan, math.nan
        elif np.isneginf(top):
            loss[i] = math.inf
        else:
            loss[i] = lse[i] - row[y[i]]
            grad[i] = np.exp(row - lse[i])
            grad[i, y[i]] -= 1.0
            grad[i] *= c[i]
    return loss, lse, grad


def cross_entropy_bounds(x, lse, grad, c, dtype, from_lse):
    """Bounds on the errors of lse (per row, absolute) and of the gradient.

    exp is one rounding of x - m, one of its product with log2 e (both relative to the exponent, so the
    power is off by their sum times |x - m|) and one step of the hardware's power of two; the sum of a row
    rounds once per addition along its longest chain (a thread's part, then the joins, which also
    multiply by powers of two of their own); the logarithm rounds by a step, and so do its product and
    the addition of m."""
    u = 2.0 ** -24
    rows, vocab = x.shape
    finite = np.where(np.isfinite(x), x, np.nan)
    with np.errstate(all="ignore"):
        top = np.nanmax(np.where(np.isfinite(finite), finite, -1e30), axis=1)
        depth = top - np.nanmin(np.where(np.isfinite(finite), finite, 1e30), axis=1)
    depth = np.clip(depth, 0, 104)             # below that the power is zero in 32 bits
    power = (2 * depth + 4) * u
    chain = vocab // 64 + 64
    total = power + 4 * chain * u
    mag = np.abs(np.where(np.isfinite(lse), lse, 0)) + np.abs(np.where(np.isfinite(top), top, 0))
    lse_err = total + 8 * u * (mag + math.log(vocab + 1) + 1)
    rel = (2 * total + power if not from_lse else lse_err + power + 4 * u * (np.abs(mag) + depth))[:, None]
    p = np.abs(grad) + np.abs(c)[:, None]
    g = np.where(np.isfinite(grad), grad, 0)
    return lse_err, rel * np.minimum(p, np.abs(c)[:, None]) + 4 * u * np.abs(c)[:, None] + rounding(g, dtype)


def sample(x, temperature, top_k, top_p, min_p, u, allowed=None):
    """(ID or -1, log-probability, weight of the ID relative to the largest) of one row of float64 logits."""
    x = np.where(np.isnan(x), -np.inf, x)
    if allowed is not None:
        x = np.where(allowed, x, -np.inf)
    order = [j for j in np.argsort(-x, kind="stable") if x[j] > -np.inf]
    if not order:
        return -1, -math.inf, 0.0
    if not temperature > 0:
        return int(order[0]), 0.0, 1.0
    order = np.array(order[:top_k] if top_k else order)
    with np.errstate(all="ignore"):
        w = np.exp((x[order] - x[order[0]]) / temperature)
    w = np.where(x[order] == x[order[0]], 1.0, np.nan_to_num(w))
    n = len(w)
    if top_p < 1:
        target, mass, n = top_p * w.sum(), 0.0, 0
        while n < len(w) and (n == 0 or mass < target):
            mass += w[n]
            n += 1
    if min_p > 0:
        n = max(1, min(n, int((w >= min(min_p, 1.0)).sum())))
    ids = np.sort(order[:n])
    weight = dict(zip(order[:n].tolist(), w[:n].tolist()))
    total, run = sum(weight.values()), 0.0
    u = 0.0 if not u > 0 else min(u, 1 - 2.0 ** -24)
    for j in ids.tolist():
        run += weight[j]
        if run > u * total:
            break
    return j, math.log(weight[j] / total), weight[j]
