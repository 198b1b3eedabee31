"""Token operators on the GPU over the parts of their range between the ordinary sizes."""
import numpy as np
import pytest
import torch

from test_gpu_ops import _dev, _sample, _say, _ws

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("distinct", [1, 2, 3, 63, 64, 65])
@pytest.mark.parametrize("apart", [1, 64, 2048])
def test_sort_keeps_every_token(tt, distinct, apart):
    """Neighbouring tokens with equal digits of the sort, low or high: a column per bit of the token's position, so that the
    sums of an ID count the bits of all of its tokens."""
    tokens, vocab = 20000, 70 * 2048
    _say("sort", distinct, apart)
    ids = np.arange(tokens) % distinct * apart
    bits = (np.arange(tokens)[:, None] >> np.arange(16)) & 1
    bits = np.concatenate([bits, 1 - bits], axis=1)
    table = torch.full((vocab, 32), 5.0, device="cuda")
    tt.toktier_embed_backward(_dev(bits, "bfloat16"), _dev(ids), table, _ws(tt.toktier_embed_backward_workspace_bytes(tokens, vocab, 32)))
    ref = torch.zeros(vocab, 32, dtype=torch.int64).index_add_(0, torch.from_numpy(ids), torch.from_numpy(bits))
    assert torch.equal(table.cpu().long(), ref)


def test_loss_of_a_last_batch_in_the_workspace_of_the_others(tt):
    """One workspace for a batch and for the few rows left after it."""
    vocab, most = 70001, 300
    torch.manual_seed(1)
    ws = _ws(tt.toktier_cross_entropy_workspace_bytes(most, vocab))
    x = (3 * torch.randn(most, vocab, device="cuda")).bfloat16()
    y = torch.randint(vocab, (most,), device="cuda", dtype=torch.int32)
    outs = []
    for rows in (most, 159, 3):
        _say("loss workspace", rows)
        loss, lse, grad = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty_like(x[:rows])
        tt.toktier_cross_entropy(x[:rows], y[:rows], loss, lse, ws, grad_logits=grad)
        outs.append((loss, grad))
    for loss, grad in outs[1:]:   # split or whole: sums in another order, 32 roundings at most along a longest chain
        n = len(loss)
        assert torch.allclose(loss, outs[0][0][:n], rtol=0, atol=20 * 64 * 2.0 ** -24)
        assert torch.allclose(grad.float(), outs[0][1][:n].float(), rtol=2.0 ** -7, atol=1e-30)


def test_gradients_of_fewer_tokens_in_the_workspace_of_the_most(tt):
    """One workspace through lengths at which the chunks and the sort's blocks change; integers, so sums are exact."""
    vocab, dim, most = 3000, 64, 262145
    rng = np.random.default_rng(5)
    ids, vals = rng.integers(-1, vocab, most), rng.integers(-3, 4, (most, dim))
    ws = _ws(tt.toktier_embed_backward_workspace_bytes(most, vocab, dim))
    grad, dev = _dev(vals, "bfloat16"), _dev(ids)
    for n in (most, 262144, 65536, 65535, 32767, 16384, 16383, 4097, 100):
        _say("gradient workspace", n)
        table = torch.full((vocab, dim), 5.0, device="cuda")
        tt.toktier_embed_backward(grad[:n], dev[:n], table, ws)
        ok = torch.from_numpy(ids[:n] >= 0)
        ref = torch.zeros(vocab, dim, dtype=torch.int64)
        ref.index_add_(0, torch.from_numpy(ids[:n])[ok], torch.from_numpy(vals[:n])[ok])
        assert torch.equal(table.cpu().long(), ref)


ROWS = (1 << 24) + 3   # 256 threads each: 2^32 and more


def test_loss_of_more_rows_than_a_launch_takes(tt):
    _say("loss rows", ROWS)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(ROWS, 3, generator=g, device="cuda")
    y = torch.randint(-1, 3, (ROWS,), generator=g, device="cuda", dtype=torch.int32)
    c = torch.rand(ROWS, generator=g, device="cuda")
    loss, lse, grad = torch.full_like(c, 7.0), torch.full_like(c, 7.0), torch.full_like(x, 7.0)
    tt.toktier_cross_entropy(x, y, loss, lse, _ws(tt.toktier_cross_entropy_workspace_bytes(ROWS, 3)), grad_logits=grad, grad_loss=c)
    z = torch.logsumexp(x.double(), 1)
    kept, at = y >= 0, y.clamp(min=0).long().unsqueeze(1)
    ref = torch.where(kept, z - x.double().gather(1, at).squeeze(1), torch.zeros_like(z))
    # three exponentials and a logarithm of numbers below 16: 16 roundings of 16 at most
    assert float((lse.double() - z).abs().max()) <= 16 * 16 * 2.0 ** -24
    assert float((loss.double() - ref).abs().max()) <= 16 * 16 * 2.0 ** -24
    p = torch.exp(x.double() - z.unsqueeze(1))
    p.scatter_add_(1, at, -torch.ones_like(z).unsqueeze(1))
    p *= (c.double() * kept).unsqueeze(1)
    assert float((grad.double() - p).abs().max()) <= 64 * 2.0 ** -24


def test_sampling_of_more_rows_than_a_launch_takes(tt):
    _say("sample rows", ROWS)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(ROWS, 3, generator=g, device="cuda")
    ids, lp = torch.full((ROWS,), 7, dtype=torch.int32, device="cuda"), torch.full((ROWS,), 7.0, device="cuda")
    t = torch.zeros(ROWS, device="cuda")
    t[-5:] = 1.0
    u, k = torch.rand(ROWS, generator=g, device="cuda"), torch.zeros(ROWS, dtype=torch.int32, device="cuda")
    k[-2:] = 1
    p = torch.ones_like(u)
    p[-3] = 0.0
    mask = torch.full((ROWS, 1), 7, dtype=torch.int32, device="cuda")
    mask[-1] = 0
    tt.toktier_sample(x, u, ids, lp, _ws(tt.toktier_sample_workspace_bytes(ROWS, 3)), temperature=t, top_k=k, top_p=p,
                      min_p=torch.zeros_like(u), mask=mask)
    assert torch.equal(ids[:-5].long(), x[:-5].argmax(1)) and not lp[:-5].any()
    assert ids[-1] == -1 and lp[-1] == float("-inf")
    for r in (-5, -4):
        w = torch.exp(x[r].double() - x[r].max().double())
        run = w.cumsum(0)
        assert int(ids[r]) == int((run <= u[r].double() * run[-1]).sum())
    assert torch.equal(ids[-3:-1].long(), x[-3:-1].argmax(1))


def test_lookup_of_more_tokens_than_a_launch_takes(tt):
    """Four tokens to a workgroup of 256 threads: 2^26 tokens are 2^32 threads."""
    tokens, dim, vocab = (1 << 26) + 9, 1025, 50
    need = 2 * tokens * dim + (4 << 30)
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip(f"needs {need >> 30} GiB of device memory")
    _say("lookup tokens", tokens)
    table = torch.randn(vocab, dim, device="cuda").bfloat16()
    ids = torch.randint(vocab, (tokens,), device="cuda", dtype=torch.int32)
    out = torch.empty(tokens, dim, device="cuda", dtype=torch.bfloat16)
    rows = [slice(a, a + 20) for a in (0, 4090, (1 << 25) - 10, (1 << 26) - 15, tokens - 20)]
    for r in rows:
        out[r] = 7.0
    tt.toktier_embed(table, ids, out)
    for r in rows:
        assert torch.equal(out[r], table[ids[r].long()]), r
    del out
    torch.cuda.empty_cache()


def test_zeros_of_a_table_that_a_launch_does_not_hold(tt):
    """No tokens: all of a table of 138 GB becomes zeros, 512 threads for every 16 KiB."""
    vocab, dim = 1 << 21, 33000
    need = 2 * vocab * dim + (1 << 30)
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip(f"needs {need >> 30} GiB of device memory")
    _say("zeros", vocab, dim)
    table = torch.empty(vocab, dim, device="cuda", dtype=torch.bfloat16)
    rows = [slice(a, a + 3) for a in (0, 1000, vocab // 2, vocab - 3)]
    for r in rows:
        table[r] = 7.0
    tt.toktier_embed_backward(torch.empty(0, dim, device="cuda", dtype=torch.bfloat16), _dev(np.zeros(0, np.int64)), table, _ws(256))
    for r in rows:
        assert not table[r].any(), r
    del table
    torch.cuda.empty_cache()


@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_of_the_most_tokens(tt, accumulate):
    """2^32 - 2 tokens of one column, each ID 2,048 times (two of them once less): the chunks' wavefronts and the joins' workgroups
    are 2^32 threads, and the last chunk ends where 32 bits do."""
    tokens, vocab = (1 << 32) - 2, 1 << 21
    size = tt.toktier_embed_backward_workspace_bytes(tokens, vocab, 1)
    need = size + 6 * tokens + (4 << 30)
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip(f"needs {need >> 30} GiB of device memory")
    _say("gradient of the most tokens", accumulate)
    ids = torch.empty(tokens, dtype=torch.int32, device="cuda")
    part = torch.arange(vocab, device="cuda", dtype=torch.int64) * 1048573 % vocab   # odd: every ID once
    part = part.to(torch.int32).repeat(64)
    for a in range(0, tokens, len(part)):
        n = min(len(part), tokens - a)
        ids[a:a + n] = part[:n]
    grad = torch.ones(tokens, 1, device="cuda", dtype=torch.bfloat16)
    table = torch.full((vocab, 1), 5.0, device="cuda")
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    tt.toktier_embed_backward(grad, ids, table, ws, accumulate=accumulate)
    ref = torch.full((vocab, 1), 2048.0 + (5.0 if accumulate else 0.0), device="cuda")
    ref[part[vocab - 2:vocab].long()] -= 1.0
    assert torch.equal(table, ref)
    del ids, grad, ws
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("vocab", [40, 9000])
def test_sampling_at_an_endless_temperature(tt, vocab, dtype):
    """All finite logits weigh the same, and one of +inf still more than all of them."""
    _say("sample endless", vocab, dtype)
    rng = np.random.default_rng(vocab)
    rows = 8
    x = rng.standard_normal((rows, vocab))
    x[1, 7] = x[2, [3, vocab - 1]] = x[3, 0] = x[4, 5] = np.inf
    x[5, ::2] = -np.inf
    k = np.array([0, 0, 0, 3, 0, 0, 30, 0])
    p = np.array([1.0, 1.0, 1.0, 1.0, 0.5, 1.0, 0.7, 0.3])
    for u in (0.0, 0.5, 0.999):
        _sample(tt, x, dtype, np.inf, k, p, 0.0, u)
        _sample(tt, x, dtype, np.inf, k, p, 0.5, u)
        _sample(tt, x, dtype, 3.0e38, k, p, 0.0, u)
