"""Token operators on the GPU against plain 64-bit implementations: element types, odd sizes, strides and
alignments, rows that a mask leaves empty, infinities and NaN, one row and many, streams, graphs."""
import math

import numpy as np
import pytest

import ops_plain as plain

pytestmark = pytest.mark.gpu

TYPES = ["float32", "float16", "bfloat16"]


def _say(*a):
    print("[gpu-case]", *a, flush=True)


@pytest.fixture(scope="module")
def tt():
    import torch
    import exact_bpe_tokenization_amd as tt
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    tt.lib()
    return tt


def _dtype(name):
    import torch
    return getattr(torch, name)


def _view(values, dtype, pad=0, lead=0):
    """`values` (float64 array) on the GPU in a view whose rows are `pad` elements apart and whose first element
    lies `lead` elements into its buffer; the gaps hold NaN.  Returns (view, buffer)."""
    import torch
    rows, cols = values.shape
    flat = torch.full((lead + rows * (cols + pad) + 8,), math.nan, dtype=dtype, device="cuda")
    view = flat[lead:lead + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] if rows else flat[:0].view(0, cols)
    view.copy_(torch.from_numpy(values).to(dtype))
    return view, flat


def _gaps_kept(flat, view):
    import torch
    n = int(torch.isnan(flat).sum())
    return n - int(torch.isnan(view).sum()) == flat.numel() - view.numel()


def _ws(nbytes):
    import torch
    return torch.full((max(int(nbytes), 1),), 0xA5, dtype=torch.uint8, device="cuda")


def _close(got, ref, err, what):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape
    same = (got == ref) | (np.isnan(got) & np.isnan(ref))
    with np.errstate(all="ignore"):
        off = np.abs(got - ref) > err
    bad = ~same & (off | ~np.isfinite(got) | ~np.isfinite(ref))
    if bad.any():
        i = tuple(int(v[0]) for v in np.nonzero(bad))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first at {i}: {got[i]} for {ref[i]}, "
                             f"allowed {np.broadcast_to(err, ref.shape)[i]}")


def _ids(rng, n, vocab, bad=0.0):
    ids = np.minimum((vocab + 1.0) ** rng.random(n) - 1, vocab - 1).astype(np.int64)
    other = rng.random(n) < bad
    ids[other] = rng.choice([-1, vocab, vocab + 7, 2 ** 31 - 1, -2 ** 31], size=int(other.sum()))
    return ids


def _dev(a, dtype="int32"):
    import torch
    return torch.from_numpy(np.asarray(a)).to(_dtype(dtype)).cuda()


# ---------------------------------------------------------------------------------------------
# embedding lookup

@pytest.mark.parametrize("tokens,vocab,dim,pad,lead", [
    (1, 1, 1, 0, 0), (1, 1256, 2048, 0, 0), (3, 5, 7, 0, 1), (65, 300, 64, 8, 0), (130, 33, 1001, 0, 0),
    (17, 1256, 2056, 3, 5), (1000, 257, 130, 0, 0), (5, 9, 5000, 1, 3)])
@pytest.mark.parametrize("table_type,out_type", [("bfloat16", "bfloat16"), ("float32", "bfloat16"), ("float16", "float32"),
                                                 ("float32", "float32"), ("bfloat16", "float16")])
def test_embed(tt, tokens, vocab, dim, pad, lead, table_type, out_type):
    import torch
    _say("embed", tokens, vocab, dim, pad, lead, table_type, out_type)
    rng = np.random.default_rng(tokens * 7919 + dim)
    table, _ = _view(rng.standard_normal((vocab, dim)), _dtype(table_type), pad, lead)
    ids = _ids(rng, tokens, vocab, 0.15 if tokens > 2 else 0.0)
    out, flat = _view(np.full((tokens, dim), 7.0), _dtype(out_type), pad, lead)
    tt.toktier_embed(table, _dev(ids), out, scale=1.7)
    ref = plain.embed(plain.f64(table), ids, float(np.float32(1.7)))
    _close(plain.f64(out), ref, 2.0 ** -24 * np.abs(ref) + plain.rounding(ref, out.dtype), "embed")
    assert _gaps_kept(flat, out)
    torch.cuda.synchronize()


def test_embed_zero_tokens(tt):
    import torch
    t = torch.ones(4, 8, device="cuda")
    tt.toktier_embed(t, _dev(np.zeros(0, np.int64)), torch.empty(0, 8, device="cuda"))


def test_embed_offsets_past_32_bits(tt):
    import torch
    vocab, dim = 1 << 21, 2056   # 4.3e9 elements
    _say("embed far rows")
    table = torch.empty(vocab, dim, dtype=torch.bfloat16, device="cuda")
    ids = np.array([vocab - 1, 0, vocab // 2 + 1, vocab])
    rows = torch.randn(3, dim, device="cuda").to(torch.bfloat16)
    for k, r in enumerate(ids[:3]):
        table[int(r)] = rows[k]
    out = torch.empty(4, dim, dtype=torch.bfloat16, device="cuda")
    tt.toktier_embed(table, _dev(ids), out)
    assert torch.equal(out[:3], rows) and not out[3].any()
    # and its gradient, into the same rows
    before = table[int(ids[0]) - 1].clone()
    ws = _ws(tt.toktier_embed_backward_workspace_bytes(4, vocab, dim))
    for r in ids[:3]:
        table[int(r)] = 0
    tt.toktier_embed_backward(out, _dev(ids), table, ws, accumulate=True)
    for k, r in enumerate(ids[:3]):
        assert torch.equal(table[int(r)], rows[k])
    assert torch.equal(table[int(ids[0]) - 1].view(torch.int16), before.view(torch.int16))


# ---------------------------------------------------------------------------------------------
# gradient of the lookup

def _embed_backward(tt, tokens, vocab, dim, grad_type, table_type, accumulate, pad=0, lead=0, ids=None, bad=0.1, scale=0.7):
    rng = np.random.default_rng(tokens * 31 + dim + vocab)
    grad, _ = _view(rng.standard_normal((tokens, dim)), _dtype(grad_type), pad, lead)
    ids = _ids(rng, tokens, vocab, bad) if ids is None else ids
    base = rng.standard_normal((vocab, dim)) if accumulate else np.full((vocab, dim), 9.0)
    table, flat = _view(base, _dtype(table_type), pad, lead)
    base = plain.f64(table) if accumulate else None
    ws = _ws(tt.toktier_embed_backward_workspace_bytes(tokens, vocab, dim))
    tt.toktier_embed_backward(grad, _dev(ids), table, ws, scale=scale, accumulate=accumulate)
    ref, err = plain.embed_backward(plain.f64(grad), ids, vocab, float(np.float32(scale)), base)
    _close(plain.f64(table), ref, err + plain.rounding(np.abs(ref) + err, table.dtype), "embed_backward")
    assert _gaps_kept(flat, table)


@pytest.mark.parametrize("tokens,vocab,dim,pad,lead", [
    (0, 40, 24, 0, 0), (1, 1, 1, 0, 0), (1, 1256, 320, 0, 0), (2, 300, 9, 1, 1), (63, 5, 33, 0, 0), (64, 1, 520, 0, 0),
    (65, 2, 8, 0, 0), (129, 4000, 1001, 3, 5), (777, 1256, 320, 0, 0), (1000, 3, 72, 8, 0), (4097, 33024, 40, 0, 0),
    (20000, 131328, 8, 0, 0)])
@pytest.mark.parametrize("grad_type,table_type", [("bfloat16", "bfloat16"), ("float16", "float32"), ("float32", "float32"),
                                                  ("float32", "float16")])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_backward(tt, tokens, vocab, dim, pad, lead, grad_type, table_type, accumulate):
    _say("embed_backward", tokens, vocab, dim, pad, lead, grad_type, table_type, accumulate)
    _embed_backward(tt, tokens, vocab, dim, grad_type, table_type, accumulate, pad, lead)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("kind", ["one row", "two rows in turn", "no row", "all different", "runs of 64", "first and last"])
def test_embed_backward_patterns(tt, kind, accumulate):
    n, vocab = 9001, 10000
    _say("embed_backward pattern", kind, accumulate)
    ids = {"one row": np.full(n, 77), "two rows in turn": np.arange(n) % 2 * (vocab - 1), "no row": np.full(n, -1),
           "all different": np.arange(n)[::-1].copy(), "runs of 64": np.arange(n) // 64 * 3,
           "first and last": np.where(np.arange(n) == n - 1, vocab - 1, 0)}[kind]
    _embed_backward(tt, n, vocab, 24, "bfloat16", "float32", accumulate, ids=ids.astype(np.int64))


@pytest.mark.parametrize("tokens,vocab", [(4096, 131328), (150000, 2000), (600000, 1 << 21)])
def test_embed_backward_large_is_exact_on_integers(tt, tokens, vocab):
    """Small integers sum exactly in 32 bits, whatever the order: the rows have to be equal to a histogram."""
    import torch
    _say("embed_backward integers", tokens, vocab)
    rng = np.random.default_rng(tokens)
    ids = _ids(rng, tokens, vocab, 0.05)
    vals = rng.integers(-3, 4, size=(tokens, 3))
    table = torch.full((vocab, 3), 5.0, device="cuda")
    ws = _ws(tt.toktier_embed_backward_workspace_bytes(tokens, vocab, 3))
    tt.toktier_embed_backward(_dev(vals, "bfloat16"), _dev(ids), table, ws)
    ok = (ids >= 0) & (ids < vocab)
    ref = np.stack([np.bincount(ids[ok], weights=vals[ok, k], minlength=vocab) for k in range(3)], axis=1)
    assert np.array_equal(plain.f64(table), ref)


def test_embed_backward_repeats_bit_for_bit(tt):
    import torch
    torch.manual_seed(3)
    n, vocab, dim = 30000, 500, 72
    grad, ids = torch.randn(n, dim, device="cuda"), torch.randint(vocab, (n,), device="cuda", dtype=torch.int32)
    ws = _ws(tt.toktier_embed_backward_workspace_bytes(n, vocab, dim))
    a, b = torch.empty(vocab, dim, device="cuda"), torch.empty(vocab, dim, device="cuda")
    tt.toktier_embed_backward(grad, ids, a, ws)
    ws.fill_(0x3C)
    tt.toktier_embed_backward(grad, ids, b, ws)
    assert torch.equal(a, b)


def test_embed_backward_matches_differences(tt):
    """The gradient of L = sum(weights * embed(table)) against central differences through the lookup."""
    import torch
    torch.manual_seed(5)
    vocab, dim, n, scale = 13, 6, 40, 0.75
    table = torch.randn(vocab, dim, device="cuda")
    ids = torch.randint(-1, vocab, (n,), device="cuda", dtype=torch.int32)
    weights = torch.randn(n, dim, device="cuda")
    out = torch.empty(n, dim, device="cuda")

    def value(t):
        tt.toktier_embed(t, ids, out, scale=scale)
        return float((out.double() * weights.double()).sum())

    grad = torch.empty(vocab, dim, device="cuda")
    tt.toktier_embed_backward(weights, ids, grad, _ws(tt.toktier_embed_backward_workspace_bytes(n, vocab, dim)), scale=scale)
    h = 0.5    # the lookup is linear: a large step loses nothing but the rounding of table +- h
    for r, c in [(0, 0), (3, 5), (12, 2), (7, 1)]:
        up, down = table.clone(), table.clone()
        up[r, c] += h
        down[r, c] -= h
        slope = (value(up) - value(down)) / (2 * h)
        # per token: the rounding of table +- h, of its product with scale, on values below 8, over 2 h
        count = int((ids == r).sum())
        bound = count * float(weights.abs().max()) * 8 * 4 * 2.0 ** -24 + (count + 3) * 2.0 ** -24 * count * float(weights.abs().max())
        assert abs(slope - float(grad[r, c])) <= bound


# ---------------------------------------------------------------------------------------------
# cross entropy

def _loss_case(rng, rows, vocab, kind, spread=3.0):
    x = spread * rng.standard_normal((rows, vocab))
    y = _ids(rng, rows, vocab, 0.2 if rows > 1 else 0.0)
    c = rng.random(rows) / rows
    if kind == "masked":
        x[:, ::3] = -np.inf
        x[:: 4] = -np.inf
    elif kind == "lowest":      # the type's lowest value as a mask
        x[:, ::3] = -65504.0
        x[::4] = -65504.0
    elif kind == "special":
        x[0, 0] = np.nan
        x[1 % rows, vocab // 2] = np.inf
        x[2 % rows, -1] = np.nan
        x[2 % rows, :-1] = -np.inf
        x[3 % rows] = -np.inf
        x[4 % rows, :] = np.inf
        x[5 % rows, 0] = np.nan
        y[5 % rows] = -1
    elif kind == "peaked":
        x[np.arange(rows), np.clip(y, 0, vocab - 1)] = 40.0
    elif kind == "equal":
        x[:] = 2.5
    return x, y, c


def _loss(tt, rows, vocab, dtype, kind, pad=0, lead=0, split=False, in_place=False, grad_loss=True, want_grad=True):
    import torch
    rng = np.random.default_rng(rows * 101 + vocab)
    x, y, c = _loss_case(rng, rows, vocab, kind)
    logits, flat = _view(x, _dtype(dtype), pad, lead)
    x = plain.f64(logits)
    c32 = _dev(c, "float32")
    scale = 0.5
    factors = scale * (plain.f64(c32) if grad_loss else np.ones(rows))
    loss, lse = torch.full((rows,), 3.0, device="cuda"), torch.full((rows,), 3.0, device="cuda")
    grad, gflat = (logits, flat) if in_place else _view(np.full((rows, vocab), 5.0), _dtype(dtype), (pad + 1) if pad else 0, lead)
    ws = _ws(tt.toktier_cross_entropy_workspace_bytes(rows, vocab))
    gl = c32 if grad_loss else None
    keep = logits.clone()
    if split or not want_grad:
        tt.toktier_cross_entropy(logits, _dev(y), loss, lse, ws)
        if want_grad:
            tt.toktier_cross_entropy_backward(logits, _dev(y), lse, grad, grad_loss=gl, grad_scale=scale)
    else:
        tt.toktier_cross_entropy(logits, _dev(y), loss, lse, ws, grad_logits=grad, grad_loss=gl, grad_scale=scale)
    rl, rz, rg = plain.cross_entropy(x, y, factors)
    ez, eg = plain.cross_entropy_bounds(x, rz, rg, np.abs(factors), _dtype(dtype), split)
    _close(plain.f64(lse), rz, ez, "lse")
    with np.errstate(all="ignore"):
        _close(plain.f64(loss), rl, ez + 2.0 ** -23 * np.abs(np.where(np.isfinite(rz), rz, 0)) +
               2.0 ** -23 * np.abs(np.where(np.isfinite(rl), rl, 0)), "loss")
    if want_grad:
        _close(plain.f64(grad), rg, eg, "gradient")
        if kind != "special":
            assert _gaps_kept(gflat, grad)
    if not in_place:
        assert torch.equal(keep.nan_to_num(nan=123.0), logits.nan_to_num(nan=123.0))


@pytest.mark.parametrize("rows,vocab,pad,lead", [
    (1, 1, 0, 0), (1, 2, 0, 0), (3, 7, 0, 1), (2, 8, 0, 0), (5, 255, 1, 0), (9, 1256, 0, 0), (33, 1001, 0, 0),
    (4, 8191, 5, 3), (6, 8193, 0, 0), (3, 33024, 0, 0), (2, 65537, 0, 0), (2, 131328, 0, 0), (2, 200019, 0, 1), (300, 515, 0, 0)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("split", [False, True])
def test_cross_entropy(tt, rows, vocab, pad, lead, dtype, split):
    _say("cross_entropy", rows, vocab, pad, lead, dtype, split)
    _loss(tt, rows, vocab, dtype, "plain", pad, lead, split=split)


@pytest.mark.parametrize("vocab", [40, 1000, 9001, 140001])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["masked", "lowest", "special", "peaked", "equal"])
@pytest.mark.parametrize("split", [False, True])
def test_cross_entropy_rows_out_of_the_ordinary(tt, vocab, dtype, kind, split):
    _say("cross_entropy", kind, vocab, dtype, split)
    _loss(tt, 8, vocab, dtype, kind, split=split)


@pytest.mark.parametrize("rows,vocab", [(7, 1003), (3, 131328), (2, 200019), (600, 520)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("split", [False, True])
def test_cross_entropy_in_place(tt, rows, vocab, dtype, split):
    _say("cross_entropy in place", rows, vocab, dtype, split)
    _loss(tt, rows, vocab, dtype, "plain", pad=3, split=split, in_place=True)


@pytest.mark.parametrize("dtype", TYPES)
def test_cross_entropy_optional_arguments(tt, dtype):
    _loss(tt, 20, 777, dtype, "plain", grad_loss=False)
    _loss(tt, 20, 777, dtype, "plain", want_grad=False)
    _loss(tt, 700, 130, dtype, "plain", want_grad=False)


def test_cross_entropy_offsets_past_32_bits(tt):
    import torch
    rows, vocab, stride = 2100, 300, (1 << 21) + 8
    _say("cross_entropy far rows")
    flat = torch.empty(rows * stride, dtype=torch.bfloat16, device="cuda")
    x = flat.view(rows, stride)[:, :vocab]
    small = (3 * torch.randn(rows, vocab, device="cuda")).to(torch.bfloat16)
    x.copy_(small)
    y = torch.randint(vocab, (rows,), device="cuda", dtype=torch.int32)
    outs = []
    for logits in (x, small.clone()):
        loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        tt.toktier_cross_entropy(logits, y, loss, lse, _ws(tt.toktier_cross_entropy_workspace_bytes(rows, vocab)),
                                 grad_logits=logits)
        outs.append((loss, lse, logits.clone()))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    ids, lp = torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, device="cuda")
    x.copy_(small)
    tt.toktier_sample(x, torch.zeros(rows, device="cuda"), ids, lp, _ws(tt.toktier_sample_workspace_bytes(rows, vocab)),
                      temperature=torch.zeros(rows, device="cuda"))
    assert torch.equal(ids.long(), small.float().argmax(1))


def test_cross_entropy_gradient_matches_differences(tt):
    """d loss / d logit against central differences of the kernel's own loss."""
    import torch
    torch.manual_seed(9)
    rows, vocab, h = 4, 50, 2.0 ** -4
    x = torch.randn(rows, vocab, device="cuda")
    y = torch.tensor([3, 49, 0, -1], dtype=torch.int32, device="cuda")
    ws = _ws(tt.toktier_cross_entropy_workspace_bytes(rows, vocab))
    lse, grad = torch.empty(rows, device="cuda"), torch.empty(rows, vocab, device="cuda")

    def value(z):
        loss = torch.empty(rows, device="cuda")
        tt.toktier_cross_entropy(z, y, loss, lse, ws)
        return loss.double()

    tt.toktier_cross_entropy(x, y, torch.empty(rows, device="cuda"), lse, ws, grad_logits=grad)
    for j in (0, 3, 25, 49):
        up, down = x.clone(), x.clone()
        up[:, j] += h
        down[:, j] -= h
        slope = (value(up) - value(down)) / (2 * h)
        # third derivative of the loss at most 1 (of p): h^2 / 6; and 32-bit losses below 16, each some 16
        # roundings off, over 2 h
        assert torch.all((slope - grad[:, j].double()).abs() <= h * h / 6 + 2 * 16 * 16 * 2.0 ** -24 / (2 * h))


# ---------------------------------------------------------------------------------------------
# sampling

def _sample(tt, x, dtype, temperature, top_k, top_p, min_p, u, allowed=None, pad=0, lead=0, shared=False, omit=()):
    import torch
    rows, vocab = x.shape
    logits, _ = _view(x, _dtype(dtype), pad, lead)
    x = plain.f64(logits)
    mask = None
    if allowed is not None:
        words = -(-vocab // 32)
        bits = np.zeros((allowed.shape[0], words * 32), dtype=np.uint8)
        bits[:, :vocab] = allowed
        mask = torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32).copy()).cuda()
    f = lambda v: torch.tensor(np.broadcast_to(v, (rows,)).copy(), dtype=torch.float32, device="cuda")  # noqa: E731
    t, p, m, uu = f(temperature), f(top_p), f(min_p), f(u)
    k = torch.tensor(np.broadcast_to(top_k, (rows,)).copy(), dtype=torch.int32, device="cuda")
    ids, lp = torch.full((rows,), 77, dtype=torch.int32, device="cuda"), torch.full((rows,), 7.0, device="cuda")
    ws = _ws(tt.toktier_sample_workspace_bytes(rows, vocab))
    kw = dict(temperature=t, top_k=k, top_p=p, min_p=m, mask=mask)
    for name in omit:
        kw[name] = None
    tt.toktier_sample(logits, uu, ids, lp, ws, **kw)
    for r in range(rows):
        ref, rlp, w = plain.sample(x[r], float(t[r]), int(k[r]), float(p[r]) if not math.isnan(float(p[r])) else 2.0,
                                   float(m[r]) if not math.isnan(float(m[r])) else 0.0, float(uu[r]),
                                   None if allowed is None else allowed[r if len(allowed) > 1 else 0].astype(bool))
        settings = (r, vocab, dtype, float(t[r]), int(k[r]), float(p[r]), float(m[r]), float(uu[r]))
        assert int(ids[r]) == ref, settings
        if ref < 0:
            assert float(lp[r]) == -math.inf
        else:
            # the weight is a multiple of 2^-45 (2^-42 at the most IDs); the logarithm is rounded once
            assert abs(float(lp[r]) - rlp) <= 2.0 ** -24 * abs(rlp) + 2.0 ** -42 / w + 1e-15, settings
    return ids, lp


def _logits(rng, rows, vocab, kind="power"):
    if kind == "power":
        return 12.0 - 1.25 * np.log1p(rng.random((rows, vocab)) * vocab) + 0.3 * rng.standard_normal((rows, vocab))
    return 2.0 * rng.standard_normal((rows, vocab))


SETTINGS = [(1.0, 0, 1.0, 0.0), (0.7, 50, 0.95, 0.0), (0.0, 5, 0.5, 0.1), (1.3, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.05),
            (0.9, 1000, 0.8, 0.02), (1.0, 1, 1.0, 0.0), (0.6, 2, 0.3, 0.0), (2.0, 300, 1.0, 0.0), (1.0, 0, 0.999, 0.001),
            (-1.0, 0, 1.0, 0.0), (1.0, 0, 0.0, 0.0), (1.0, 0, 1.0, 1.0), (5.0, 7, 1.5, 2.0)]


@pytest.mark.parametrize("vocab,pad,lead", [(1, 0, 0), (2, 0, 0), (7, 1, 1), (8, 0, 0), (63, 0, 0), (257, 0, 0), (1256, 0, 0),
                                            (8191, 3, 0), (8192, 0, 0), (8200, 0, 5), (33024, 0, 0), (131328, 0, 0),
                                            (200019, 0, 0)])
@pytest.mark.parametrize("dtype", TYPES)
def test_sample(tt, vocab, pad, lead, dtype):
    _say("sample", vocab, pad, lead, dtype)
    rng = np.random.default_rng(vocab)
    rows = len(SETTINGS) * (3 if vocab < 10000 else 1)
    s = np.array([SETTINGS[r % len(SETTINGS)] for r in range(rows)])
    _sample(tt, _logits(rng, rows, vocab), dtype, s[:, 0], s[:, 1].astype(np.int64), s[:, 2], s[:, 3], rng.random(rows),
            pad=pad, lead=lead)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 2, 3, 400])
def test_sample_one_row_and_many(tt, rows, dtype):
    _say("sample rows", rows, dtype)
    rng = np.random.default_rng(rows)
    for kind in ("power", "normal"):
        for temperature, k, p, m in SETTINGS[:6]:
            _sample(tt, _logits(rng, rows, 1256, kind), dtype, temperature, k, p, m, rng.random(rows))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [100, 8300, 40000])
def test_sample_ties(tt, vocab, dtype):
    """Few different values: what the filters keep ends inside a run of equals, lowest IDs first."""
    _say("sample ties", vocab, dtype)
    rng = np.random.default_rng(vocab)
    rows = 24
    x = rng.choice([0.0, -0.0, 1.0, -1.5, 2.0], size=(rows, vocab))
    x[::6] = 0.25                                   # all equal
    x[1::6] = np.where(rng.random((4, vocab)) < 0.5, 0.0, -0.0)
    _sample(tt, x, dtype, 1.0, rng.integers(0, vocab, rows), rng.choice([0.1, 0.5, 0.9, 1.0], rows), rng.choice([0.0, 0.2], rows),
            rng.choice([0.0, 0.25, 0.5, 0.999], rows))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [33, 1256, 131328])
def test_sample_masks_and_special_values(tt, vocab, dtype):
    _say("sample masks", vocab, dtype)
    rng = np.random.default_rng(vocab + 1)
    rows = 15
    x = _logits(rng, rows, vocab)
    allowed = rng.random((rows, vocab)) < 0.5
    allowed[1] = False                              # nothing allowed
    allowed[2] = False
    allowed[2, vocab - 1] = True                    # one ID
    x[3] = -np.inf
    x[4] = np.nan
    x[5, ::2] = np.nan
    x[6, ::2] = -np.inf
    x[7, vocab // 2] = np.inf
    x[8, [0, vocab - 1]] = np.inf
    allowed[7:9] = True
    x[9] = -65504.0                                 # the lowest value of a type as a mask
    x[10, 1:] = -65504.0
    allowed[11] = False
    allowed[11, :3] = True
    s = np.array([SETTINGS[r % 6] for r in range(rows)])
    for k in (0, 3):
        _sample(tt, x, dtype, 0.8, k, s[:, 2], s[:, 3], rng.random(rows), allowed=allowed)
        _sample(tt, x, dtype, 0.8, k, 0.9, 0.0, rng.random(rows))
    _sample(tt, x, dtype, 0.0, 0, 1.0, 0.0, rng.random(rows), allowed=allowed)
    _sample(tt, x, dtype, 1.0, 0, 1.0, 0.0, rng.random(rows), allowed=allowed[:1])   # one mask for all rows


def test_sample_settings_off_or_out_of_range(tt):
    rng = np.random.default_rng(4)
    x = _logits(rng, 12, 3000)
    u = np.array([0.0, 0.5, 1.0, 2.0, -1.0, math.nan, 0.999999, 1e-30, 0.3, 0.7, 0.1, 0.9])
    _sample(tt, x, "bfloat16", 1.0, 0, 1.0, 0.0, u, omit=("temperature", "top_k", "top_p", "min_p"))
    _sample(tt, x, "float32", 1.0, 2 ** 31 - 1, math.nan, math.nan, u)
    _sample(tt, x, "float32", 1e-30, 0, 0.9, 0.0, u)
    _sample(tt, x, "float16", 1e30, 0, 0.5, 0.0, u)
    _sample(tt, x, "float32", math.nan, 0, 0.5, 0.0, u)


def test_sample_frequencies(tt):
    """65,536 rows of the same 5 logits: the drawn shares follow the softmax (5 standard deviations)."""
    import torch
    n = 1 << 16
    x = torch.tensor([0.0, 1.0, -1.0, 2.0, -math.inf], device="cuda").expand(n, 5).contiguous()
    g = torch.Generator(device="cuda").manual_seed(1)
    ids, lp = torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(n, device="cuda")
    tt.toktier_sample(x, torch.rand(n, generator=g, device="cuda"), ids, lp, _ws(tt.toktier_sample_workspace_bytes(n, 5)))
    p = torch.softmax(x[0].double(), 0).cpu().numpy()
    share = np.bincount(ids.cpu().numpy(), minlength=5) / n
    assert np.all(np.abs(share - p) <= 5 * np.sqrt(p * (1 - p) / n))


# ---------------------------------------------------------------------------------------------
# streams and graphs

def _step(tt, b):
    """One training step's operators and one draw, on the current stream."""
    tt.toktier_embed(b["table"], b["ids"], b["h"], scale=2.0)
    tt.toktier_cross_entropy(b["logits"], b["targets"], b["loss"], b["lse"], b["ws_l"], grad_logits=b["dlogits"])
    tt.toktier_cross_entropy_backward(b["logits"], b["targets"], b["lse"], b["dlogits2"])
    tt.toktier_embed_backward(b["h"], b["ids"], b["dtable"], b["ws_e"])
    tt.toktier_sample(b["logits"], b["u"], b["out"], b["lp"], b["ws_s"], temperature=b["t"], top_k=b["k"], top_p=b["p"])


def _buffers(tt, seed, n=70, vocab=1256, dim=136):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    bf, dev = torch.bfloat16, "cuda"
    b = dict(table=torch.randn(vocab, dim, generator=g, device=dev).to(bf),
             ids=torch.randint(vocab, (n,), generator=g, device=dev, dtype=torch.int32),
             targets=torch.randint(-1, vocab, (n,), generator=g, device=dev, dtype=torch.int32),
             logits=(3 * torch.randn(n, vocab, generator=g, device=dev)).to(bf), u=torch.rand(n, generator=g, device=dev))
    b["t"], b["p"] = torch.full((n,), 0.8, device=dev), torch.full((n,), 0.9, device=dev)
    b["k"] = torch.full((n,), 40, dtype=torch.int32, device=dev)
    for name, shape, dt in (("h", (n, dim), bf), ("loss", (n,), torch.float32), ("lse", (n,), torch.float32),
                            ("dlogits", (n, vocab), bf), ("dlogits2", (n, vocab), bf), ("dtable", (vocab, dim), torch.float32),
                            ("out", (n,), torch.int32), ("lp", (n,), torch.float32)):
        b[name] = torch.zeros(shape, dtype=dt, device=dev)
    b["ws_l"] = _ws(tt.toktier_cross_entropy_workspace_bytes(n, vocab))
    b["ws_e"] = _ws(tt.toktier_embed_backward_workspace_bytes(n, vocab, dim))
    b["ws_s"] = _ws(tt.toktier_sample_workspace_bytes(n, vocab))
    return b


RESULTS = ("h", "loss", "lse", "dlogits", "dlogits2", "dtable", "out", "lp")


def test_on_another_stream(tt):
    import torch
    a, b = _buffers(tt, 1), _buffers(tt, 1)
    _step(tt, a)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        _step(tt, b)
    s.synchronize()
    for name in RESULTS:
        assert torch.equal(a[name], b[name]), name


def test_graph_replays(tt):
    import torch
    b, eager = _buffers(tt, 2), _buffers(tt, 3)
    _step(tt, b)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        _step(tt, b)
    for seed in (3, 4, 5, 3):
        other = _buffers(tt, seed)
        for name in ("table", "ids", "targets", "logits", "u"):
            b[name].copy_(other[name])
        for name in ("ws_l", "ws_e", "ws_s"):
            b[name].fill_(seed)
        _step(tt, eager)                 # other work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        _step(tt, other)
        torch.cuda.synchronize()
        for name in RESULTS:
            assert torch.equal(b[name], other[name]), (seed, name)


# ---------------------------------------------------------------------------------------------
# borders between one way of working and another

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [300, 9000, 131328])
def test_sample_crowded_borders(tt, vocab, dtype):
    """Many logits, equal or nearly so, where top-k and top-p end: more than are sorted at once."""
    _say("sample crowded", vocab, dtype)
    rng = np.random.default_rng(vocab + 7)
    rows = 10
    near = 1.0 + rng.random((rows, vocab)) * 2.0 ** -7
    same = np.where(rng.random((rows, vocab)) < 0.01, 2.5, 1.0)
    last = rng.permuted(np.arange(rows * vocab).reshape(rows, vocab) % vocab < 40, axis=1) * 1.0   # 40 of one, the rest of another
    k = np.array([0, 1, 2, 41, 63, 255, 700, vocab // 2, vocab - 1, vocab])
    for x in (near, same, last):
        for p in (1.0, 0.37):
            _sample(tt, x, dtype, 0.01 if x is near else 0.7, k, p, rng.choice([0.0, 0.5], rows), rng.random(rows))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [2000, 40000])
@pytest.mark.parametrize("scale,temperature", [(1e-6, 1e-6), (1e-3, 3e-4), (4000.0, 3000.0), (200.0, 40.0), (1e4, 1e30)])
def test_sample_scales(tt, vocab, dtype, scale, temperature):
    """Logits far smaller or larger than usual, whose weights do differ, and a temperature that makes them equal."""
    _say("sample scale", vocab, dtype, scale, temperature)
    rng = np.random.default_rng(vocab + 11)
    rows = 8
    x = scale * rng.standard_normal((rows, vocab))
    x[0] = -np.abs(x[0])
    x[1] = np.abs(x[1])
    k = np.array([0, 0, 50, 1500, 0, 20, vocab, 700])
    for p in (1.0, 0.9):
        _sample(tt, x, dtype, temperature, k, p, 0.0, rng.random(rows))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [500, 131328])
def test_sample_nan_beside_logits(tt, vocab, dtype):
    """NaN of either sign is never chosen, and changes nothing else."""
    import torch
    _say("sample nan", vocab, dtype)
    rng = np.random.default_rng(vocab + 13)
    rows = 12
    x = _logits(rng, rows, vocab)
    for r in range(rows):
        x[r, rng.integers(0, vocab, 1 + r)] = math.nan if r % 2 else -math.nan
    x[3, 0] = x[4, vocab - 1] = math.nan
    assert torch.isnan(torch.from_numpy(x)).any(dim=1).all()
    s = np.array([SETTINGS[r % 6] for r in range(rows)])
    allowed = rng.random((rows, vocab)) < 0.7
    allowed[:, 1] = True
    for mask in (None, allowed):
        _sample(tt, x, dtype, s[:, 0], s[:, 1].astype(np.int64), s[:, 2], s[:, 3], rng.random(rows), allowed=mask)
        _sample(tt, x, dtype, 0.9, 0, 1.0, 0.0, rng.random(rows), allowed=mask)


@pytest.mark.parametrize("rows,vocab", [(1, 65528), (1, 65536), (5, 65537), (159, 65536), (160, 65536)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_cross_entropy_few_long_rows(tt, rows, vocab, dtype):
    _say("cross_entropy few long rows", rows, vocab, dtype)
    _loss(tt, rows, vocab, dtype, "plain")


@pytest.mark.parametrize("tokens", [4095, 4096, 4097, 8191, 8192, 8193, 16385, 1200001])
@pytest.mark.parametrize("vocab", [5, 2048, 2049, 50000])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_backward_lengths_are_exact_on_integers(tt, tokens, vocab, accumulate):
    import torch
    _say("embed_backward lengths", tokens, vocab, accumulate)
    rng = np.random.default_rng(tokens + vocab)
    ids = _ids(rng, tokens, vocab, 0.05)
    vals = rng.integers(-3, 4, size=(tokens, 2))
    table = torch.full((vocab, 2), 5.0, device="cuda")
    ws = _ws(tt.toktier_embed_backward_workspace_bytes(tokens, vocab, 2))
    tt.toktier_embed_backward(_dev(vals, "float32"), _dev(ids), table, ws, accumulate=accumulate)
    ok = (ids >= 0) & (ids < vocab)
    ref = np.stack([np.bincount(ids[ok], weights=vals[ok, k], minlength=vocab) for k in range(2)], axis=1)
    assert np.array_equal(plain.f64(table), ref + 5.0 if accumulate else ref)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n", [17, 700, 2048, 2049, 4096])
@pytest.mark.parametrize("kind", ["one row", "two rows in turn", "no row", "all different", "runs of 64", "first and last", "mixed"])
def test_embed_backward_few_tokens(tt, kind, n, accumulate):
    """Rows of several blocks of columns, of one token and of many."""
    vocab, dim = 5000, 1100
    _say("embed_backward few", kind, n, accumulate)
    ids = {"one row": np.full(n, 77), "two rows in turn": np.arange(n) % 2 * (vocab - 1), "no row": np.full(n, -1),
           "all different": np.arange(n)[::-1].copy(), "runs of 64": np.arange(n) // 64 * 3,
           "first and last": np.where(np.arange(n) == n - 1, vocab - 1, 0),
           "mixed": np.where(np.arange(n) % 3 == 0, 5, np.where(np.arange(n) % 5 == 0, vocab, np.arange(n) // 2))}[kind]
    _embed_backward(tt, n, vocab, dim, "bfloat16", "float32", accumulate, ids=ids.astype(np.int64))


def test_embed_backward_few_tokens_of_a_large_table(tt):
    """A table that is zeroed by a launch of its own."""
    _embed_backward(tt, 900, 40000, 500, "float16", "float16", False)
    _embed_backward(tt, 900, 40000, 500, "float16", "float16", False, pad=3, lead=1)


@pytest.mark.parametrize("vocab", [1, 2, 3])
@pytest.mark.parametrize("tokens", [4097, 9000])
def test_embed_backward_many_tokens_of_few_ids(tt, tokens, vocab):
    _embed_backward(tt, tokens, vocab, 40, "bfloat16", "float32", False)
    _embed_backward(tt, tokens, vocab, 600, "float32", "bfloat16", True)


@pytest.mark.parametrize("tokens", [4096, 5000])
def test_embed_backward_offsets_past_32_bits(tt, tokens):
    """Gradient rows and table rows 2^20 elements apart, against the same rows side by side."""
    import torch
    dim, stride = 24, (1 << 20) + 8
    _say("embed_backward far rows", tokens)
    far = torch.empty(tokens * stride, dtype=torch.bfloat16, device="cuda").view(tokens, stride)[:, :dim]
    near = torch.randn(tokens, dim, device="cuda").to(torch.bfloat16)
    far.copy_(near)
    ids = torch.randint(tokens, (tokens,), device="cuda", dtype=torch.int32)
    ws = _ws(tt.toktier_embed_backward_workspace_bytes(tokens, tokens, dim))
    out = torch.empty(tokens, dim, device="cuda")
    far_out = torch.empty(tokens * stride, dtype=torch.float32, device="cuda").view(tokens, stride)[:, :dim]
    tt.toktier_embed_backward(near, ids, out, ws)
    tt.toktier_embed_backward(far, ids, far_out, ws)
    assert torch.equal(out, far_out)


def test_graph_replays_of_the_longer_paths(tt):
    """The sorted gradient with zeros beside the sort and with sums added, and the loss of few long rows."""
    import torch
    n, vocab, dim, rows, wide = 5000, 9000, 72, 3, 70000
    dev, bf = "cuda", torch.bfloat16

    def buffers(seed):
        g = torch.Generator(device=dev).manual_seed(seed)
        return dict(grad=torch.randn(n, dim, generator=g, device=dev).to(bf),
                    ids=torch.randint(-1, vocab, (n,), generator=g, device=dev, dtype=torch.int32),
                    logits=(3 * torch.randn(rows, wide, generator=g, device=dev)).to(bf),
                    targets=torch.randint(wide, (rows,), generator=g, device=dev, dtype=torch.int32),
                    dense=torch.empty(vocab, dim, device=dev), added=torch.randn(vocab, dim, generator=g, device=dev),
                    loss=torch.empty(rows, device=dev), lse=torch.empty(rows, device=dev),
                    dlogits=torch.empty(rows, wide, device=dev, dtype=bf),
                    ws=_ws(max(tt.toktier_embed_backward_workspace_bytes(n, vocab, dim),
                               tt.toktier_cross_entropy_workspace_bytes(rows, wide))))

    def step(b):
        tt.toktier_embed_backward(b["grad"], b["ids"], b["dense"], b["ws"])
        tt.toktier_embed_backward(b["grad"], b["ids"], b["added"], b["ws"], accumulate=True)
        tt.toktier_cross_entropy(b["logits"], b["targets"], b["loss"], b["lse"], b["ws"], grad_logits=b["dlogits"])

    b = buffers(1)
    step(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        step(b)
    for seed in (2, 3, 4, 2):
        other = buffers(seed)
        for name in ("grad", "ids", "logits", "targets", "added"):
            b[name].copy_(other[name])
        b["ws"].fill_(seed)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        step(other)
        torch.cuda.synchronize()
        for name in ("dense", "added", "loss", "lse", "dlogits"):
            assert torch.equal(b[name], other[name]), (seed, name)
