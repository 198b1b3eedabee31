"""The gradients of the cross entropy from hidden states in a later call, for rows whose log-sum-exp is far from zero: its
rounding does not show in the probabilities."""
import pytest
import torch

import linear_plain as plain
from test_gpu_linear_rounding import BF16, F16, F32, TYPES, U, one_hot, run

pytestmark = pytest.mark.gpu


def _say(*a):
    print("[gpu-case]", *a, flush=True)


def _inputs(n, v, d, dtype, far, seed=0):
    """Table, targets and factors; logits of row i are column i of the table: near zero, or `far` from it."""
    gen = torch.Generator(device="cuda").manual_seed(seed + n + v)
    w = 2.5 * torch.randn(v, d, generator=gen, device="cuda")
    y = torch.randint(0, v, (n,), generator=gen, device="cuda", dtype=torch.int32)
    c = torch.rand(n, generator=gen, device="cuda") + 0.5
    for col, shift in far.items():
        if abs(shift) >= 1e6:
            w[:, col] = shift                  # equal ones
        else:
            w[:, col] += shift
    return w.to(dtype), y, c


def _check(w, y, c, lse, gw, rows, dtype, what):
    x = w.double().t()[rows]
    y, c, lse = y[rows].long().unsqueeze(1), c[rows].double().unsqueeze(1), lse[rows].double().unsqueeze(1)
    p = torch.softmax(x, 1)
    hit = torch.zeros_like(p).scatter_(1, y, 1.0)
    g = c * (p - hit)
    away = (x.amax(1, keepdim=True) - x).clamp(max=104)
    near = torch.where(lse.abs() < 128, 2 * lse.abs(), torch.zeros_like(lse))
    rel = U * (5 * away + 3 * (40 + -(-w.size(0) // 16)) + 8 + near)
    err = c * p * rel + 3 * U * g.abs()
    err = err + plain.HALF_STEP[dtype] * (g.abs() + err) + plain.SMALLEST[dtype] * (2.0 ** -13 if dtype == F16 else 1.0) + 2.0 ** -126
    plain.close(gw.t()[rows], g, err, what)


FAR = {2: 1000.0, 7: -1000.0, 11: 129.0, 13: -400.0, 19: 30000.0, 23: -30000.0}
FURTHER = {3: 1e8, 5: -1e8, 17: 3e38, 21: -3e38}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,d", [(30, 500, 64), (60, 5001, 64), (100, 3000, 128), (250, 1256, 256), (300, 9000, 320), (700, 20000, 704)])
def test_rows_far_from_zero(tt, n, v, d, dtype):
    _say("linear later far", n, v, d, dtype)
    far = FAR if dtype == F16 else {**FAR, **FURTHER}
    w, y, c = _inputs(n, v, d, dtype, {**far, n - 1: 700.0})
    h = one_hot(n, d, dtype)
    _, lse, gh, gw = run(tt, h, w, y, c, later=True)
    _check(w, y, c, lse, gw, torch.arange(n, device="cuda"), dtype, "far")
    # the rows that are near have the same gradients whatever the others are
    calm, _, _ = _inputs(n, v, d, dtype, {})
    near = torch.tensor([i for i in range(n - 1) if i not in far], device="cuda")
    other = run(tt, h, calm, y, c, later=True)
    assert torch.equal(gw[:, near], other[3][:, near])


@pytest.mark.parametrize("n,v,d,dtype", [(200, 40000, 2049, BF16), (200, 40000, 2049, F16), (130, 20000, 2049, F32)])
def test_of_a_table_copied_in_pieces(tt, n, v, d, dtype):
    _say("linear later copied", n, v, d, dtype)
    far = {2: 1000.0, 150 if n > 150 else 100: -700.0}
    w, y, c = _inputs(n, v, d, dtype, far)
    _, lse, _, gw = run(tt, one_hot(n, d, dtype), w, y, c, later=True)
    _check(w, y, c, lse, gw, torch.arange(n, device="cuda"), dtype, "copied")


@pytest.mark.parametrize("dtype", TYPES)
def test_one_gradient_and_rows_that_take_no_part(tt, dtype):
    _say("linear later one gradient", dtype)
    n, v, d = 90, 3000, 128
    w, y, c = _inputs(n, v, d, dtype, FAR)
    y[::5] = -1
    y[2] = v
    h = one_hot(n, d, dtype)
    _, lse, gh, gw = run(tt, h, w, y, c, later=True)
    kept = torch.nonzero((y >= 0) & (y < v)).squeeze(1)
    _check(w, y, c, lse, gw, kept, dtype, "part")
    ws = torch.empty(tt.toktier_linear_cross_entropy_workspace_bytes(n, v, d, dtype), dtype=torch.uint8, device="cuda")
    alone = torch.full_like(gh, 3.0), torch.full_like(gw, 5.0)
    tt.toktier_linear_cross_entropy_backward(h, w, y, lse, ws, grad_hidden=alone[0], grad_loss=c)
    tt.toktier_linear_cross_entropy_backward(h, w, y, lse, ws, grad_weight=alone[1], grad_loss=c)
    assert torch.equal(alone[0], gh) and torch.equal(alone[1], gw)


def test_captured_and_replayed_on_other_rows(tt):
    """A captured call finds out itself which rows are far."""
    _say("linear later graph")
    n, v, d = 100, 3000, 128
    h = one_hot(n, d, BF16)
    w, y, c = _inputs(n, v, d, BF16, {})
    loss, lse, gw = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty(v, d, device="cuda")
    ws = torch.empty(tt.toktier_linear_cross_entropy_workspace_bytes(n, v, d, BF16), dtype=torch.uint8, device="cuda")
    call = lambda: tt.toktier_linear_cross_entropy_backward(h, w, y, lse, ws, grad_weight=gw, grad_loss=c)
    tt.toktier_linear_cross_entropy(h, w, y, loss, lse, ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for turn, far in enumerate(({}, FAR, {**FAR, **FURTHER}, {}, FURTHER)):
        w.copy_(_inputs(n, v, d, BF16, far, seed=turn)[0])
        tt.toktier_linear_cross_entropy(h, w, y, loss, lse, ws.fill_(turn))
        gw.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        _check(w, y, c, lse, gw, torch.arange(n, device="cuda"), BF16, f"replay {turn}")
