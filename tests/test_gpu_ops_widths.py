"""The sorted gradient of the lookup where rows are no multiple of eight columns: the last vector of a row shares
columns with the one before, so rows that are added to depend on the order of a wavefront's loads and stores."""
import numpy as np
import pytest
import torch

from test_gpu_ops import _dev, _dtype, _gaps_kept, _ids, _say, _view, _ws

pytestmark = pytest.mark.gpu


def _sums(vals, ids, vocab):
    """Integer sums of the rows of `vals` per ID."""
    ok = (ids >= 0) & (ids < vocab)
    out = torch.zeros(vocab, vals.shape[1], dtype=torch.int64)
    return out.index_add_(0, torch.from_numpy(ids[ok]), torch.from_numpy(vals[ok])).numpy()


def _exact(tt, ids, vocab, dim, grad_type, table_type, accumulate, pad=0, lead=0):
    """Small integers sum exactly in 32 bits, whatever the order, so that only the rounding to the table's type is
    left, to nearest even as torch rounds."""
    tokens = len(ids)
    rng = np.random.default_rng(tokens + 7 * dim + vocab)
    vals = rng.integers(-3, 4, size=(tokens, dim))
    base = rng.integers(-40, 41, size=(vocab, dim))
    grad, _ = _view(vals.astype(np.float64), _dtype(grad_type), pad, lead)
    table, flat = _view(base.astype(np.float64), _dtype(table_type), pad, lead)
    ws = _ws(tt.toktier_embed_backward_workspace_bytes(tokens, vocab, dim))
    tt.toktier_embed_backward(grad, _dev(ids), table, ws, scale=2.0, accumulate=accumulate)
    ref = 2 * _sums(vals, ids, vocab) + (base if accumulate else 0)
    assert np.abs(ref).max() < 1 << 24   # so it is a float32
    assert torch.equal(table.cpu(), torch.from_numpy(ref).float().to(table.dtype))
    assert _gaps_kept(flat, table)


@pytest.mark.parametrize("dim", [9, 15, 513, 1001, 2047])
@pytest.mark.parametrize("grad_type,table_type", [("bfloat16", "float32"), ("float32", "bfloat16"), ("float16", "float16")])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("kind", ["text", "one row of many chunks", "runs across chunks"])
def test_sorted_gradient_of_odd_widths(tt, dim, grad_type, table_type, accumulate, kind):
    tokens, vocab = 6000, 900
    _say("sorted gradient", kind, dim, grad_type, table_type, accumulate)
    rng = np.random.default_rng(dim)
    ids = _ids(rng, tokens, vocab, 0.05)
    if kind == "one row of many chunks":       # a chunk has 64 tokens at most: 69 chunks or more
        ids[rng.permutation(tokens)[:4500]] = 77
    elif kind == "runs across chunks":
        ids = np.arange(tokens) // 90 * 13
    _exact(tt, ids, vocab, dim, grad_type, table_type, accumulate)
    if dim == 1001:
        _exact(tt, ids, vocab, dim, grad_type, table_type, accumulate, pad=3, lead=1)


@pytest.mark.parametrize("dim", [9, 15, 513, 1001])
@pytest.mark.parametrize("accumulate", [False, True])
def test_few_tokens_of_odd_widths(tt, dim, accumulate):
    _say("few tokens", dim, accumulate)
    rng = np.random.default_rng(dim + 1)
    ids = _ids(rng, 1500, 600, 0.05)
    ids[::3] = 5
    for types in (("bfloat16", "float32"), ("float32", "bfloat16")):
        _exact(tt, ids, 600, dim, *types, accumulate)
