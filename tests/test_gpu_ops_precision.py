"""Cross entropy against 64-bit results at bounds of single elements, and at logits far from zero."""
import numpy as np
import pytest
import torch

import ops_bounds as bounds
import ops_plain as plain
from test_gpu_ops import TYPES, _close, _dev, _dtype, _say, _view, _ws, tt  # noqa: F401

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
def test_loss_of_logits_far_from_zero(tt, rows, vocab, dtype, kind):  # noqa: F811
    _say("loss far", rows, vocab, dtype, kind)
    rng = np.random.default_rng(vocab)
    logits, _ = _view(_far(rng, rows, vocab, dtype, kind), _dtype(dtype))
    y = rng.integers(0, vocab, rows)
    y[0] = vocab // 2
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    tt.toktier_cross_entropy(logits, _dev(y), loss, lse, _ws(tt.toktier_cross_entropy_workspace_bytes(rows, vocab)))
    ref, err = bounds.loss(plain.f64(logits), y)
    _close(plain.f64(loss), ref, err, "loss")
