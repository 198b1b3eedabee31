"""Distillation at the ends of the range that its arguments may have: temperatures, log-sum-exps beyond 32 bits, lists with
+inf; both the one call and the gradient from lse; and the top logits' temperatures."""
import math

import pytest
import torch

from distill_plain import vectors
from linear_plain import U, close
from test_gpu_distill import BF16, F16, F32, TYPES, Case
from test_gpu_top_logits import check, make

pytestmark = pytest.mark.gpu

SHAPES = [(7, 1256, 8), (3, 33001, 100), (2, 65537, 64)]


def _say(*a):
    print("[gpu-case]", *a, flush=True)


def _both(tt, case, t, what):
    case.scale = max(t, 1.0)    # so that c / temperature is no subnormal number
    # a temperature whose reciprocal is subnormal: half a step of that is up to 2^-22
    subnormal = 5 * U if t > 2.0 ** 126 else 0.0
    # a row that is summed again by 256 threads, as distill_plain counts it for large log-sum-exps
    again = U * (13 * vectors(case.v) + 105) if t > 2.0 ** 120 else 0.0
    p = torch.softmax(case.logits.double() / t, 1) * (case.grad_loss.double() * case.scale / t).abs().unsqueeze(1)
    o = case.outputs()
    case.forward(tt, o)
    for later in (False, True):
        if later:
            o["grad"].fill_(3)
            case.backward(tt, o)
        ref = case.reference(from_lse=later)
        ref["grad"] = ref["grad"][0], ref["grad"][1] + subnormal * ref["grad"][0].abs() + (again * p if later else 0.0)
        case.check(o, ref, what + (" later" if later else ""), ("grad",) if later else ("loss", "lse", "grad"))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,v,k", SHAPES)
@pytest.mark.parametrize("t", [4.3e-39, 1e-38, 1e-30, 1e-4, 1e4, 1e30, 2.0 ** 120, 1.4e36, 2e37, 1e38, 3.4e38])
def test_temperatures(tt, t, n, v, k, dtype):
    """Logits of the temperature's size where that is small, of ordinary size where it is large."""
    _say("distill range temperature", t, n, v, k, dtype)
    t = float(torch.tensor(t, dtype=torch.float32))
    _both(tt, Case(n, v, k, dtype, t, size=2.5 * min(t, 1.0), own_lse=n == 3 and t >= 1e-4), t, "ordinary")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,v,k", SHAPES)
@pytest.mark.parametrize("t", [1e30, 2.0 ** 120, 1e37, 2e37])
def test_logits_of_a_large_temperatures_size(tt, t, n, v, k, dtype):
    _say("distill range logits", t, n, v, k, dtype)
    t = float(torch.tensor(t, dtype=torch.float32))
    case = Case(n, v, k, dtype, t, size=2.0 * t)
    # differences of logits have to be numbers of 32 bits
    case.logits.clamp_(-1.6e38, 1.6e38)
    _both(tt, case, t, "large")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [1256, 30000, 70000])
@pytest.mark.parametrize("t", [1e-38, 1e-37])
def test_log_sum_exps_beyond_32_bits(tt, t, v, dtype):
    """lse is -inf or +inf because it has no number, not because the row is empty."""
    _say("distill range lse", t, v, dtype)
    n, t = 4, float(torch.tensor(t, dtype=torch.float32))
    x = torch.full((n, v), -60.0, dtype=dtype, device="cuda")
    x[1:, 100], x[1:, 700], x[1:, v - 1] = -50.0, -50.0, -50.0
    x[2] = x[2] + 100
    x[3] = -math.inf
    ids = torch.tensor([[700, 5, -1]] * n, dtype=torch.int32, device="cuda")
    top = torch.tensor([[1.0, 0.0, 0.0]] * n, device="cuda")
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    ws = torch.empty(tt.toktier_distill_workspace_bytes(n, v, 3), dtype=torch.uint8, device="cuda")
    one, later = torch.empty_like(x), torch.empty_like(x)
    tt.toktier_distill(x, ids, top, loss, lse, ws, temperature=t, grad_logits=one, grad_scale=t)
    tt.toktier_distill_backward(x, ids, top, lse, later, temperature=t, grad_scale=t)
    assert lse.tolist() == [-math.inf, -math.inf, math.inf, -math.inf]
    want = torch.zeros(n, v, dtype=torch.float64, device="cuda")
    want[0] = 1.0 / v
    want[1:3, 100], want[1:3, 700], want[1:3, v - 1] = 1 / 3, 1 / 3, 1 / 3
    want[:3, 700] -= 1.0
    for g in (one, later):
        close(g, want, 2.0 ** -7 * want.abs() + (2.0 ** -24 if dtype == F16 else 0.0), "gradient")
    x[3] = -50.0
    here = x.clone()
    tt.toktier_distill_backward(here, ids, top, lse, here, temperature=t, grad_scale=t)
    assert torch.equal(here[:3], later[:3])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [1256, 30000, 70000])
@pytest.mark.parametrize("own_lse", [False, True])
def test_infinite_logits_in_a_list(tt, own_lse, v, dtype):
    _say("distill range list", own_lse, v, dtype)
    n = 6
    case = Case(n, v, 20, dtype, own_lse=own_lse)
    good = case.outputs()
    case.forward(tt, good)
    case.top[1, 3] = math.inf
    case.top[2, 0] = math.nan
    case.top[4, 19] = math.inf
    case.ids[4, 19] = -1        # no entry, not looked at
    o = case.outputs()
    case.forward(tt, o)
    for later in (False, True):
        if later:
            o["grad"].fill_(3)
            case.backward(tt, o)
        assert bool(o["loss"][1:3].isnan().all()) and bool(o["grad"][1:3].isnan().all())
        assert torch.equal(o["lse"], good["lse"])
        rest = torch.tensor([0, 3, 4, 5], device="cuda")
        assert bool(o["loss"][rest].isfinite().all()) and bool(o["grad"][rest].isfinite().all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t", [4.3e-39, 1e-38, 2.0 ** 120, 1e38, 3.4e38])
def test_temperatures_of_top_logits(tt, t, dtype):
    _say("top range temperature", t, dtype)
    t = float(torch.tensor(t, dtype=torch.float32))
    check(tt, make(3, 1256, dtype, size=2.5 * min(t, 1.0)), 20, t)
    check(tt, make(2, 33001, dtype, size=2.5 * min(t, 1.0)), 300, t)
