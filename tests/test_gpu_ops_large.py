"""Token operators at their largest vocabularies, and with more data than the caches hold."""
import numpy as np
import pytest
import torch

import ops_bounds as bounds
import ops_plain as plain
from test_gpu_ops import TYPES, _close, _dev, _dtype, _say, _ws

pytestmark = pytest.mark.gpu
MOST = 1 << 21


def _kept(x, temperature, k, p, min_p):
    """(kept IDs ascending, their weights) of one row of finite float64 logits."""
    order = np.argsort(-x, kind="stable")[:k or None]
    w = np.exp((x[order] - x[order[0]]) / temperature)
    n = len(w)
    if p < 1:
        run = np.cumsum(w.astype(np.longdouble))
        n = 1 + int(np.searchsorted(run, np.longdouble(np.float32(p)) * run[-1]))
    n = max(1, min(n, int((w >= np.float32(min_p)).sum())))
    by_id = np.argsort(order[:n])
    return order[:n][by_id], w[:n][by_id]


@pytest.mark.parametrize("vocab", [1 << 18, (1 << 18) + 1, 1 << 19, (1 << 20) + 3, MOST])
@pytest.mark.parametrize("dtype", TYPES)
def test_sample_of_the_largest_vocabularies(tt, vocab, dtype):
    """IDs are aimed at: u is the middle of an ID's share of the kept mass, which is far wider than the sums' errors."""
    _say("sample large", vocab, dtype)
    rng = np.random.default_rng(vocab)
    settings = [(1.0, 0, 1.0, 0.0), (0.8, 0, 0.9, 0.0), (1.0, 50, 0.95, 0.0), (0.9, 3000, 0.8, 0.0), (1.2, 0, 1.0, 0.01),
                (1.0, vocab - 5, 0.99, 0.0), (1.0, 0, 1.0, 0.0), (1.0, 0, 0.5, 0.0)]
    rows = len(settings)
    x = 12.0 - 1.25 * np.log1p(rng.random((rows, vocab)) * vocab) + 0.3 * rng.standard_normal((rows, vocab))
    x[6:] = 0.75                                   # all equal: the largest sum of weights there is
    logits = torch.from_numpy(x).to(_dtype(dtype)).cuda()
    x = plain.f64(logits)
    aims, u, ref = [], [], []
    for r, (t, k, p, m) in enumerate(settings):
        ids, w = _kept(x[r], float(np.float32(t)), k, p, m)
        run = np.cumsum(w)
        large = np.nonzero(w >= 2e-7 * run[-1])[0]   # shares of several steps of a 32-bit u
        for i in (large[0], large[rng.integers(len(large))], large[-1]):
            aims.append(int(ids[i]))
            u.append((run[i] - 0.5 * w[i]) / run[-1])
            ref.append((float(np.log(w[i] / run[-1])), w[i]))
    pick = np.repeat(np.arange(rows), 3)
    s = np.array(settings)[pick]
    out, lp = torch.full((len(pick),), 77, dtype=torch.int32, device="cuda"), torch.full((len(pick),), 7.0, device="cuda")
    tt.toktier_sample(logits[torch.from_numpy(pick).cuda()], _dev(u, "float32"), out, lp, _ws(tt.toktier_sample_workspace_bytes(len(pick), vocab)),
                      temperature=_dev(s[:, 0], "float32"), top_k=_dev(s[:, 1].astype(np.int64)), top_p=_dev(s[:, 2], "float32"),
                      min_p=_dev(s[:, 3], "float32"))
    assert out.tolist() == aims
    for got, (want, w) in zip(lp.tolist(), ref):
        # a weight is a multiple of 2^-42 or less; the total is off by half of that for each of 2^21 IDs at most; one rounding
        assert abs(got - want) <= 2.0 ** -24 * abs(want) + 2.0 ** -43 / w + 2.0 ** -22


@pytest.mark.parametrize("vocab", [MOST, MOST - 5, 1 << 20])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows", [2, 160])
def test_cross_entropy_of_the_largest_vocabularies(tt, rows, vocab, dtype):
    _say("cross_entropy large", rows, vocab, dtype)
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x = (3 * torch.randn(rows, vocab, generator=g, device="cuda")).to(_dtype(dtype))
    y = torch.randint(vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    y[0] = vocab - 1
    c = torch.rand(rows, generator=g, device="cuda") + 0.5
    ws = _ws(tt.toktier_cross_entropy_workspace_bytes(rows, vocab))
    loss, lse, grad, later = torch.empty_like(c), torch.empty_like(c), torch.empty_like(x), torch.empty_like(x)
    tt.toktier_cross_entropy(x, y, loss, lse, ws, grad_logits=grad, grad_loss=c)
    tt.toktier_cross_entropy_backward(x, y, lse, later, grad_loss=c)
    for r in (0, rows - 1):
        row, at, f = plain.f64(x[r:r + 1]), y[r:r + 1].cpu().numpy(), plain.f64(c[r:r + 1])
        ref, err = bounds.loss(row, at)
        _close(plain.f64(loss[r:r + 1]), ref, err, "loss")
        for got, from_lse in ((grad, False), (later, True)):
            ref, err = bounds.gradient(row, at, f, _dtype(dtype), from_lse)
            _close(plain.f64(got[r:r + 1]), ref, err, "gradient")


@pytest.mark.parametrize("table_type,out_type", [("bfloat16", "bfloat16"), ("float32", "float16"), ("float16", "float32")])
@pytest.mark.parametrize("dim", [4096, 4099])
def test_lookup_larger_than_the_caches(tt, dim, table_type, out_type):
    tokens, vocab = 4500, 900
    _say("lookup large", dim, table_type, out_type)
    g = torch.Generator(device="cuda").manual_seed(dim)
    table = torch.randn(vocab, dim, generator=g, device="cuda").to(_dtype(table_type))
    ids = torch.randint(-1, vocab, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    out = torch.full((tokens, dim + 1), 7.0, device="cuda", dtype=_dtype(out_type))
    tt.toktier_embed(table, ids, out[:, :dim], scale=1.7)
    ref = table.float()[ids.clamp(min=0).long()] * torch.tensor(1.7, device="cuda") * (ids >= 0).unsqueeze(1)
    assert torch.equal(out[:, :dim], ref.to(out.dtype)) and bool((out[:, dim] == 7.0).all())


@pytest.mark.parametrize("dim", [2048, 2051])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_larger_than_the_caches(tt, dim, accumulate):
    tokens, vocab = 70000, 5000
    _say("gradient large", dim, accumulate)
    g = torch.Generator(device="cuda").manual_seed(dim)
    grad = torch.randint(-3, 4, (tokens, dim), generator=g, device="cuda").bfloat16()
    ids = ((vocab + 1.0) ** torch.rand(tokens, generator=g, device="cuda", dtype=torch.float64) - 2).floor().clamp(max=vocab - 1).int()
    table = torch.full((vocab, dim), 5.0, device="cuda")
    tt.toktier_embed_backward(grad, ids, table, _ws(tt.toktier_embed_backward_workspace_bytes(tokens, vocab, dim)),
                              accumulate=accumulate)
    ok = ids >= 0
    ref = torch.zeros(vocab, dim, device="cuda", dtype=torch.float64).index_add_(0, ids[ok].long(), grad[ok].double())   # integers
    assert bool(ok.any()) and not bool(ok.all())
    assert torch.equal(table.double(), ref + (5.0 if accumulate else 0.0))
