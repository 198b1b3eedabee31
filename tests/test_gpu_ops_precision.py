"""Cross entropy against 64-bit results at bounds of single elements, and at logits far from zero."""
import numpy as np
import pytest
import torch

import ops_bounds as bounds
import ops_plain as plain
from test_gpu_ops import TYPES, _close, _dev, _dtype, _say, _view, _ws

pytestmark = pytest.mark.gpu
LOWEST = {"float32": -3.4028234663852886e38, "float16": -65504.0, "bfloat16": -3.3895313892515355e38}


def _far(rng, rows, vocab, dtype, kind):
    x = 3.0 * rng.standard_normal((rows, vocab))
    if kind == "lowest":         # the type's lowest value as a mask that leaves nothing
        x[:] = LOWEST[dtype]
    elif kind == "lowest but one":
        x[:] = LOWEST[dtype]
        x[:, vocab // 2] = 1.0
    elif kind == "largest":
        x[:] = -LOWEST[dtype]
    else:
        x += kind
    return x


KINDS = ["lowest", "lowest but one", "largest", 0.0, 200.0, 10000.0, -10000.0]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(5, 40), (4, 9001), (3, 70001), (161, 66000)])
def test_loss_of_logits_far_from_zero(tt, rows, vocab, dtype, kind):
    _say("loss far", rows, vocab, dtype, kind)
    rng = np.random.default_rng(vocab)
    logits, _ = _view(_far(rng, rows, vocab, dtype, kind), _dtype(dtype))
    y = rng.integers(0, vocab, rows)
    y[0] = vocab // 2
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    tt.toktier_cross_entropy(logits, _dev(y), loss, lse, _ws(tt.toktier_cross_entropy_workspace_bytes(rows, vocab)))
    ref, err = bounds.loss(plain.f64(logits), y)
    _close(plain.f64(loss), ref, err, "loss")


def _gradient(tt, x, dtype, from_lse, in_place=False, pad=0, lead=0):
    rows, vocab = x.shape
    rng = np.random.default_rng(rows + vocab)
    logits, _ = _view(x, _dtype(dtype), pad, lead)
    x = plain.f64(logits)
    y = rng.integers(0, vocab, rows)
    y[0] = vocab // 2
    c = _dev(rng.random(rows) + 0.5, "float32")
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    grad = logits if in_place else _view(np.full((rows, vocab), 5.0), _dtype(dtype), pad, lead)[0]
    ws = _ws(tt.toktier_cross_entropy_workspace_bytes(rows, vocab))
    if from_lse:
        tt.toktier_cross_entropy(logits, _dev(y), loss, lse, ws)
        tt.toktier_cross_entropy_backward(logits, _dev(y), lse, grad, grad_loss=c, grad_scale=0.5)
    else:
        tt.toktier_cross_entropy(logits, _dev(y), loss, lse, ws, grad_logits=grad, grad_loss=c, grad_scale=0.5)
    ref, err = bounds.gradient(x, y, 0.5 * plain.f64(c), _dtype(dtype), from_lse)
    _close(plain.f64(grad), ref, err, "gradient")


@pytest.mark.parametrize("rows,vocab,pad,lead", [
    (1, 1, 0, 0), (3, 7, 1, 1), (9, 1256, 0, 0), (5, 8191, 0, 0), (4, 8193, 3, 1), (3, 33024, 0, 0), (2, 65535, 0, 0), (2, 65536, 0, 0),
    (2, 131328, 0, 0), (170, 70001, 0, 0), (300, 515, 0, 0)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("from_lse", [False, True])
@pytest.mark.parametrize("kind", [0.0, "peaked", "equal", "masked"])
def test_gradient_element_by_element(tt, rows, vocab, pad, lead, dtype, from_lse, kind):
    _say("gradient", rows, vocab, dtype, from_lse, kind)
    rng = np.random.default_rng(vocab)
    x = 3.0 * rng.standard_normal((rows, vocab))
    if kind == "peaked":
        x[:, vocab // 2] = 40.0
    elif kind == "equal":
        x[:] = 2.5
    elif kind == "masked":
        x[:, 1::3] = -np.inf
        x[:, 2::5] = LOWEST[dtype]
    _gradient(tt, x, dtype, from_lse, pad=pad, lead=lead)


@pytest.mark.parametrize("kind", KINDS + [-110.0, 100.0])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("from_lse", [False, True])
@pytest.mark.parametrize("rows,vocab", [(5, 40), (4, 9001), (3, 70001)])
def test_gradient_of_logits_far_from_zero(tt, rows, vocab, dtype, from_lse, kind):
    _say("gradient far", rows, vocab, dtype, from_lse, kind)
    rng = np.random.default_rng(vocab)
    x = _far(rng, rows, vocab, dtype, kind)
    if rows > 3:
        x[1] = 3.0 * rng.standard_normal(vocab)    # an ordinary row among them
    _gradient(tt, x, dtype, from_lse)
    _gradient(tt, x, dtype, from_lse, in_place=True, pad=1)


@pytest.mark.parametrize("vocab", [50, 9001, 70001])
@pytest.mark.parametrize("from_lse", [False, True])
def test_gradient_matches_differences_of_the_64_bit_loss(tt, vocab, from_lse):
    """Central differences of a loss that shares nothing with the kernels."""
    rows, h = 3, 2.0 ** -10
    _say("differences", vocab, from_lse)
    rng = np.random.default_rng(vocab)
    x = torch.from_numpy(2.0 * rng.standard_normal((rows, vocab))).float().cuda()
    y = np.array([vocab // 2, 0, vocab - 1])
    loss, lse, grad = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty_like(x)
    ws = _ws(tt.toktier_cross_entropy_workspace_bytes(rows, vocab))
    tt.toktier_cross_entropy(x, _dev(y), loss, lse, ws, grad_logits=None if from_lse else grad)
    if from_lse:
        tt.toktier_cross_entropy_backward(x, _dev(y), lse, grad)
    x64, got = plain.f64(x), plain.f64(grad)
    bound = bounds.gradient(x64, y, np.ones(rows), torch.float32, from_lse)[1]
    ones = np.ones(rows)
    for j in [0, 1, vocab // 2, vocab - 1] + [int(v) for v in rng.integers(0, vocab, 6)]:
        up, down = x64.copy(), x64.copy()
        up[:, j] += h
        down[:, j] -= h
        slope = (plain.cross_entropy(up, y, ones)[0] - plain.cross_entropy(down, y, ones)[0]) / (2 * h)
        # the third derivative of the loss is p (1 - p) (1 - 2 p), at most p in size (p moves by less than h of itself);
        # two 64-bit losses below 32, each some 32 roundings off, over 2 h
        p = np.exp(x64[:, j] - plain.f64(lse)) * 1.01
        assert np.all(np.abs(slope - got[:, j]) <= bound[:, j] + p * h * h / 6 + 2 * 32 * 32 * 2.0 ** -53 / (2 * h))
