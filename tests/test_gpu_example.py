"""The example of the token operators runs, learns and generates IDs of its vocabulary."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    import importlib.util
    spec = importlib.util.spec_from_file_location("next_token", os.path.join(ROOT, "examples", "next_token.py"))
    mod = importlib.util.module_from_spec(spec)
    sys.modules["next_token"] = mod
    spec.loader.exec_module(mod)
    return mod


def test_example_learns_and_generates():
    import math
    ex = _example()
    losses, ids, texts = ex.run(steps=30, chars=40_000, tokens=1000, dim=128, n_new=12)
    assert all(math.isfinite(v) for v in losses)
    assert abs(losses[0] - math.log(1256)) < 0.5      # a table of small numbers: nearly uniform
    assert losses[-1] < losses[0] - 0.5
    assert ids.shape == (12, 4) and int(ids.min()) >= 0 and int(ids.max()) < 1256
    assert len(texts) == 4


def test_example_gradient_is_the_models():
    """The gradient of the table against the one that torch finds for the same model in 64 bits: at most
    the roundings of the bfloat16 parts, three in a row and each relative to at most the largest gradient."""
    import torch
    ex = _example()
    g = torch.Generator(device="cuda").manual_seed(5)
    n, vocab, dim = 96, 300, 64
    m = ex.Model(vocab, dim, n, seed=1)
    ids = torch.randint(vocab, (n,), generator=g, device="cuda", dtype=torch.int32)
    targets = torch.randint(-1, vocab, (n,), generator=g, device="cuda", dtype=torch.int32)
    table = m.table.bfloat16().double().cpu()
    m.table.copy_(table.float())
    mean, got, _ = m.gradients(ids, targets)
    t = table.clone().requires_grad_(True)
    h = t[ids.long().cpu()] * dim ** 0.5
    loss = torch.nn.functional.cross_entropy(h @ t.t(), torch.where(targets < 0, -100, targets).long().cpu(), ignore_index=-100)
    loss.backward()
    assert abs(float(mean) - float(loss.detach())) <= 8 * 2.0 ** -8 * float(loss.detach())
    assert float((got.double().cpu() - t.grad).abs().max()) <= 8 * 2.0 ** -8 * float(t.grad.abs().max())
