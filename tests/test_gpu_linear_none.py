"""Batches of the cross entropy from hidden states in which no row takes part, at sizes of every tile of the products: zeros, whatever
the workspace holds, and the next batch is as if it were the first."""
import math

import pytest
import torch

from test_gpu_linear_loss import BF16, TYPES, Case, _bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,d", [(1, 70, 64), (40, 5001, 100), (300, 6000, 1024), (1100, 9000, 576), (2100, 6500, 640)])
def test_no_row_takes_part(tt, n, v, d, dtype):
    print("[gpu-case]", "linear none", n, v, d, dtype, flush=True)
    case = Case(n, v, d, dtype)
    want = case.outputs()
    case.forward(tt, want, case.workspace(tt))
    targets, hidden = case.targets.clone(), case.hidden.clone()
    case.targets.fill_(-1)
    case.hidden.fill_(math.nan)
    ws = case.workspace(tt)
    o = case.outputs()
    case.forward(tt, o, ws)
    assert not any(bool(t.any()) for t in _bits(o))
    for lse in (0.0, 500.0, -math.inf, math.nan):   # of rows that take no part: not looked at
        o = case.outputs()
        o["lse"].fill_(lse)
        case.backward(tt, o, ws.fill_(0x7F))
        assert not bool(o["gh"][0].any()) and not bool(o["gw"][0].any())
    case.targets.copy_(targets)
    case.hidden.copy_(hidden)
    case.forward(tt, o, ws)
    assert all(torch.equal(a, b) for a, b in zip(_bits(o), _bits(want)))


def test_replayed_batches_with_and_without_rows(tt):
    print("[gpu-case]", "linear none graph", flush=True)
    case = Case(300, 6000, 256, BF16)
    want = case.outputs()
    case.forward(tt, want, case.workspace(tt))
    targets = case.targets.clone()
    ws, o = case.workspace(tt), case.outputs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        case.forward(tt, o, ws)
    for turn in range(4):
        if turn % 2:
            case.targets.copy_(targets)
        else:
            case.targets.fill_(6000 + turn)
        for t in _bits(o):
            t.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        if turn % 2:
            assert all(torch.equal(a, b) for a, b in zip(_bits(o), _bits(want)))
        else:
            assert not any(bool(t.any()) for t in _bits(o))
