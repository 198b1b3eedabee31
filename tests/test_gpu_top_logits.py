"""The top logits of rows on the GPU against a plain sort: types, sizes, short and long lists, equal logits, rows that a mask
leaves empty, values that are not finite, strides, streams and graphs; and the way from them to a student's gradient."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [BF16, F16, F32]
U = 2.0 ** -24


def _say(*a):
    print("[gpu-case]", *a, flush=True)


def plain(logits, k, temperature=1.0):
    """(IDs, logits, lse, bound on lse's error) by a stable sort in 64 bits; a row's NaN and -inf are not listed."""
    x = logits.detach().double().cpu().numpy()
    n, v = x.shape
    ids, out, lse, err = np.full((n, k), -1), np.full((n, k), -np.inf), np.empty(n), np.zeros(n)
    for r in range(n):
        row = np.where(np.isnan(x[r]), -np.inf, x[r])
        order = np.argsort(-row, kind="stable")[:k]
        order = order[row[order] > -np.inf]
        ids[r, :len(order)], out[r, :len(order)] = order, row[order]
        with np.errstate(all="ignore"):
            z = x[r] / temperature
            m = z.max()
            lse[r] = math.nan if np.isnan(m) or m == np.inf else -np.inf if m == -np.inf else m + np.log(np.exp(z - m).sum())
            if np.isfinite(lse[r]):   # the bounds of distill_plain, of s and its logarithm; m k rounds, by u of |m| in the argument
                d = np.minimum(m - z, 104)
                p = np.exp(z - lse[r])
                low = z[np.isfinite(z)].min()
                rel = (p * (5 * d + 4)).sum() + 5 * min(m - low, 104) + 13 * -(-v // 2048) + 105
                err[r] = U * (rel + abs(m) + 4 * (abs(lse[r] - m) + 1) + 3 * abs(m) + 2 * abs(lse[r]))
    return ids, out, lse, err


def call(tt, logits, k, temperature=1.0, with_lse=True, ws=None, out=None):
    n = logits.size(0)
    ids, top = out or (torch.full((n, k), 77, dtype=torch.int32, device="cuda"), torch.full((n, k), 77.0, device="cuda"))
    lse = torch.full((n,), 77.0, device="cuda") if with_lse else None
    if ws is None:
        ws = torch.full((tt.toktier_top_logits_workspace_bytes(n, logits.size(1), k),), 0xA5, dtype=torch.uint8, device="cuda")
    tt.toktier_top_logits(logits, ids, top, ws, lse=lse, temperature=temperature)
    return ids, top, lse


def check(tt, logits, k, temperature=1.0):
    ids, out, lse, err = plain(logits, k, temperature)
    got = call(tt, logits, k, temperature)
    assert np.array_equal(got[0].cpu().numpy(), ids)
    assert np.array_equal(got[1].double().cpu().numpy(), out)
    z = got[2].double().cpu().numpy()
    with np.errstate(all="ignore"):
        assert ((z == lse) | (np.isnan(z) & np.isnan(lse)) | (np.abs(z - lse) <= err)).all(), (z, lse, err)
    alone = call(tt, logits, k, with_lse=False)
    assert torch.equal(alone[0], got[0]) and torch.equal(alone[1], got[1])


def make(n, v, dtype, seed=0, size=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed + 31 * n + v)
    return (size * torch.randn(n, v, generator=g, device="cuda")).to(dtype)


FEW = [(1, 1), (3, 7), (5, 64), (4, 1256), (3, 2048), (3, 2049), (2, 8192), (2, 8193), (2, 33001), (1, 65535), (1, 65536), (1, 131328),
       (2, 500001)]
SIZES = ([(n, v, k) for n, v in FEW for k in (1, 3, 20, 64, 65, 200, 700, 1000, 1024)] +
         [(n, 65537, k) for n in (64, 65) for k in (3, 65, 1000)])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,k", SIZES)
def test_sizes(tt, n, v, k, dtype):
    _say("top", n, v, k, dtype)
    check(tt, make(n, v, dtype), k, 1.0 + k % 2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [500, 3000, 20000, 131328])
@pytest.mark.parametrize("k", [1, 20, 300, 1024])
def test_equal_logits(tt, v, k, dtype):
    """Rows of one value, of two, of few, and with a border of thousands of equals."""
    _say("top equals", v, k, dtype)
    g = torch.Generator(device="cuda").manual_seed(v + k)
    x = torch.zeros(6, v, device="cuda")
    x[1] = torch.randint(0, 2, (v,), generator=g, device="cuda").float()
    x[2] = torch.randint(-3, 3, (v,), generator=g, device="cuda").float()
    x[3, torch.randperm(v, generator=g, device="cuda")[:k // 2 + 1]] = 5.0
    x[4] = -3.5
    x[4, v - 1] = -3.0
    x[5, ::2] = -0.0
    check(tt, x.to(dtype), k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [1256, 30000, 131328])
def test_ordered_rows(tt, v, dtype):
    """Sorted rows, and large logits side by side: few threads hold all that is wanted."""
    _say("top ordered", v, dtype)
    x = torch.linspace(-8, 8, v, device="cuda").repeat(4, 1)
    x[1] = x[1].flip(0)
    x[2] = 0.001 * x[2]
    x[2, 700:1200] += 9
    x[3, ::1024] += 20
    for k in (10, 64, 500, 1024):
        check(tt, x.to(dtype), k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [700, 9000, 70000])
def test_rows_that_are_empty_or_not_finite(tt, v, dtype):
    _say("top odd rows", v, dtype)
    x = make(9, v, dtype)
    x[1] = -math.inf
    x[2, 3:] = -math.inf
    x[3, 5] = math.nan
    x[4, v - 1] = math.inf
    x[4, 7] = math.inf
    x[5] = math.nan
    x[6] = torch.finfo(dtype).min
    x[6, 9] = -math.inf
    x[7, ::3] = -math.nan
    x[8, 1::2] = -math.inf
    for k in (1, 20, 600, 1024):
        check(tt, x, k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [4000, 131328])
def test_any_bits(tt, v, dtype):
    """Every kind of number: random bit patterns, among them subnormal ones."""
    _say("top bits", v, dtype)
    g = torch.Generator(device="cuda").manual_seed(v)
    whole = torch.int32 if dtype == F32 else torch.int16
    lim = 2 ** 31 if dtype == F32 else 2 ** 15
    bits = torch.randint(-lim, lim, (4, v), generator=g, device="cuda").to(whole)
    x = bits.view(dtype).clone()
    x[1] = torch.where(x[1].abs().double() < 1e-30 if dtype != F16 else x[1].abs() < 1e-4, x[1], torch.zeros_like(x[1]))
    ids, out, _, _ = plain(x, 1000)
    for k in (5, 64, 1000):
        got = call(tt, x, k)
        assert np.array_equal(got[0].cpu().numpy(), ids[:, :k]) and np.array_equal(got[1].double().cpu().numpy(), out[:, :k])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,lead", [(1, 0), (0, 1), (5, 3), (64, 8)])
def test_strides(tt, pad, lead, dtype):
    _say("top strides", pad, lead, dtype)
    for n, v, k in ((7, 1255, 30), (3, 70001, 64), (3, 20001, 900)):
        flat = torch.full((lead + n * (v + pad) + 8,), math.inf, dtype=dtype, device="cuda")
        x = flat[lead:lead + n * (v + pad)].view(n, v + pad)[:, :v]
        x.copy_(make(n, v, dtype))
        ids, out, _, _ = plain(x, k)
        wide_ids = torch.full((n, k + 5), 9, dtype=torch.int32, device="cuda")
        wide = torch.full((n, k + 3), 9.0, device="cuda")
        got = call(tt, x, k, out=(wide_ids[:, 2:k + 2], wide[:, 1:k + 1]))
        assert np.array_equal(got[0].cpu().numpy(), ids) and np.array_equal(got[1].double().cpu().numpy(), out)
        assert bool((wide_ids[:, :2] == 9).all()) and bool((wide_ids[:, k + 2:] == 9).all())
        assert bool((wide[:, :1] == 9).all()) and bool((wide[:, k + 1:] == 9).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("temperature", [1e-30, 1e-4, 1e4, 1e30])
def test_temperatures_far_from_one(tt, temperature, dtype):
    _say("top temperature", temperature, dtype)
    check(tt, make(3, 1256, dtype), 20, temperature)
    check(tt, make(2, 33001, dtype), 300, temperature)


def test_no_rows_many_rows_and_far_offsets(tt):
    _say("top many rows")
    call(tt, torch.empty(0, 8, device="cuda"), 3)
    x = make(70000, 40, BF16)
    ids, top, _ = call(tt, x, 3)
    want = torch.sort(x.float(), dim=1, descending=True, stable=True)
    assert torch.equal(ids, want.indices[:, :3].to(torch.int32)) and torch.equal(top, want.values[:, :3])
    n, v = 33000, 131328   # 4.3e9 elements
    x = torch.zeros(n, v, dtype=BF16, device="cuda")
    at = torch.randint(0, v, (n, 1), device="cuda")
    x.scatter_(1, at, 2.0)
    ids, top, lse = call(tt, x, 2)
    assert torch.equal(ids[:, 0].long(), at[:, 0]) and torch.equal(ids[:, 1].long(), (at[:, 0] == 0).long())
    assert bool((top[:, 0] == 2).all()) and bool((top[:, 1] == 0).all())
    assert torch.allclose(lse, torch.full_like(lse, math.log(v - 1 + math.exp(2.0))), rtol=1e-5)


def test_streams_and_graphs(tt):
    _say("top graphs")
    xs, ks = [make(3, 131328, BF16), make(70, 3000, F16)], [20, 100]
    want = [call(tt, x, k) for x, k in zip(xs, ks)]
    ws = torch.empty(max(tt.toktier_top_logits_workspace_bytes(*x.shape, k) for x, k in zip(xs, ks)), dtype=torch.uint8, device="cuda")
    outs = [tuple(torch.empty_like(t) for t in w) for w in want]

    def go(i):
        tt.toktier_top_logits(xs[i], outs[i][0], outs[i][1], ws, lse=outs[i][2])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go(0)
        go(1)
    side.synchronize()
    graphs = []
    for i in (0, 1):
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i]))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            go(i)
        graphs.append(graph)
    for turn in range(4):
        for i in ((0, 1), (1, 0))[turn % 2]:
            for t in outs[i]:
                t.fill_(9)
            ws.fill_(turn * 41)
            graphs[i].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i]))


def test_from_a_teacher_to_a_students_gradient(tt):
    """The lists and log-sum-exps of a teacher go into the student's loss as they come, and where the list holds the whole
    vocabulary the loss is the divergence of the two rows."""
    _say("top and distill")
    n, v, t = 40, 300, 1.5
    teacher, student = make(n, v, F32, 1), make(n, v, F32, 2)
    ids, top, lse = call(tt, teacher, v, t)
    p = torch.log_softmax(student.double() / t, 1)
    q = torch.softmax(teacher.double() / t, 1)
    want = (q * (torch.log(q) - p)).sum(1)
    ws = torch.empty(tt.toktier_distill_workspace_bytes(n, v, v), dtype=torch.uint8, device="cuda")
    for own in (None, lse):
        loss, z, grad = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty(n, v, device="cuda")
        tt.toktier_distill(student, ids, top, loss, z, ws, temperature=t, teacher_lse=own, grad_logits=grad)
        assert torch.allclose(loss.double(), want, rtol=1e-4, atol=1e-5)
        assert torch.allclose(grad.double(), (torch.exp(p) - q) / t, rtol=1e-4, atol=1e-6)
