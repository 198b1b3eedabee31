"""How often the cross entropy from hidden states rounds: hidden states that are rows of the identity make every logit an
element of the table, exactly, and every row of the table's gradient the rows' G, so that both can be told to the last bit; and rows whose
target is certain."""
import math

import pytest
import torch

import linear_plain as plain

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [BF16, F16, F32]
U = plain.U


def _say(*a):
    print("[gpu-case]", *a, flush=True)


def one_hot(n, d, dtype):
    h = torch.zeros(n, d, dtype=dtype, device="cuda")
    h[torch.arange(n, device="cuda"), torch.arange(n, device="cuda") % d] = 1.0
    return h


def run(tt, h, w, y, c=None, scale=1.0, later=False):
    """(loss, lse, grad_hidden, grad_weight in float32)"""
    (n, d), v = h.shape, w.size(0)
    loss, lse = torch.full((n,), 7.0, device="cuda"), torch.full((n,), 7.0, device="cuda")
    gh, gw = torch.full_like(h, 3.0), torch.full((v, d), 5.0, device="cuda")
    size = tt.toktier_linear_cross_entropy_workspace_bytes(n, v, d, h.dtype)
    ws = torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")
    grads = dict(grad_hidden=gh, grad_weight=gw, grad_loss=c, grad_scale=scale)
    tt.toktier_linear_cross_entropy(h, w, y, loss, lse, ws, **({} if later else grads))
    if later:
        tt.toktier_linear_cross_entropy_backward(h, w, y, lse, ws.fill_(0x5A), **grads)
    return loss, lse, gh, gw


# What an exponential that waits for its row's sum may be off by: half a step of 10 bits, or of 12 and then half of the last
# one's step below 2^-30.
KEPT = {BF16: (2.0 ** -10, 2.0 ** -126), F16: (2.0 ** -12, 2.0 ** -42), F32: (0.0, 0.0)}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,d", [(20, 3000, 64), (64, 5001, 64), (300, 9000, 320), (700, 20000, 704)])
@pytest.mark.parametrize("later", [False, True])
def test_gradients_of_logits_are_rounded_once(tt, later, n, v, d, dtype):
    """G has one rounding to the type; where its exponential was kept, a quarter of one more in bfloat16, half of one in
    float16, and none at the target."""
    _say("linear roundings", later, n, v, d, dtype)
    gen = torch.Generator(device="cuda").manual_seed(n + v)
    w = (2.5 * torch.randn(v, d, generator=gen, device="cuda")).to(dtype)
    h = one_hot(n, d, dtype)
    y = torch.randint(0, v, (n,), generator=gen, device="cuda", dtype=torch.int32)
    c = torch.rand(n, generator=gen, device="cuda") + 0.5
    _, lse, _, gw = run(tt, h, w, y, c, later=later)
    x = w.double().t()[:n]
    p = torch.softmax(x, 1)
    g = p.clone()
    g[torch.arange(n, device="cuda"), y.long()] -= 1.0
    g *= c.double().unsqueeze(1)
    # in 32 bits: 2.5 u of the distance to the maximum, the sums' roundings, and of lse where p comes from it
    away = (x.amax(1, keepdim=True) - x).clamp(max=104)
    rel = U * (5 * away + 3 * (40 + -(-v // 64)) + 8 + (2 * lse.double().abs().unsqueeze(1) if later else 0))
    hit = torch.zeros_like(g).scatter_(1, y.long().unsqueeze(1), 1.0)
    size = c.double().unsqueeze(1)
    half, least = (0.0, 0.0) if later else KEPT[dtype]
    smallest = plain.SMALLEST[dtype] * (2.0 ** -13 if dtype == F16 else 1.0)   # float16's G is kept times 2^14
    err = size * p * rel + size * (1 - hit) * (half * p + least) + 3 * U * g.abs()
    err = err + plain.HALF_STEP[dtype] * (g.abs() + err) + smallest + 2.0 ** -126
    plain.close(gw.t()[:n], g, err, "G")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,d", [(1, 70, 64), (16, 300, 64), (60, 5001, 64), (128, 3000, 128), (300, 9000, 320), (700, 20000, 704),
                                   (4200, 140001, 64)])   # more than is kept
@pytest.mark.parametrize("later", [False, True])
def test_rows_that_are_certain(tt, later, n, v, d, dtype):
    """All of the probability at the target, at any height of its logit: loss and gradients are zeros, not a rounding of the logit."""
    _say("linear certain", later, n, v, d, dtype)
    heights = torch.tensor([1.0, 5.3, 30.0, -3.7, 63.7, 100.2, 127.9, 128.5, -90.3, 1000.0, -20.1, 0.0], device="cuda")
    top = heights[torch.arange(d, device="cuda") % 12].to(dtype)
    w = (top.float() - 250.0).to(dtype).expand(v, d).contiguous()
    at = (torch.arange(d, device="cuda") * 7919) % v
    w[at, torch.arange(d, device="cuda")] = top
    y = at[torch.arange(n, device="cuda") % d].to(torch.int32)
    loss, lse, gh, gw = run(tt, one_hot(n, d, dtype), w, y, later=later)
    assert torch.equal(loss, torch.zeros_like(loss)), float(loss.abs().max())
    assert torch.equal(lse, top.float()[torch.arange(n, device="cuda") % d])
    assert not bool(gh.any()) and not bool(gw.any()), (float(gh.abs().max()), float(gw.abs().max()))


@pytest.mark.parametrize("dtype", TYPES)
def test_losses_are_not_negative(tt, dtype):
    _say("linear not negative", dtype)
    gen = torch.Generator(device="cuda").manual_seed(11)
    n, v, d = 500, 4000, 512
    w = torch.randn(v, d, generator=gen, device="cuda").to(dtype)
    y = torch.randint(0, v, (n,), generator=gen, device="cuda", dtype=torch.int32)
    lift = torch.linspace(0.0, 0.24, n, device="cuda").unsqueeze(1)   # logits of the targets up to 120
    h = (lift * w[y.long()].float()).to(dtype)
    loss = run(tt, h, w, y)[0]
    assert bool((loss >= 0).all()) and float(loss[-1]) < 1e-6 and math.isclose(float(loss[0]), math.log(v), rel_tol=1e-5)
