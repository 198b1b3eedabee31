"""Cross entropy from hidden states in 64 bits, and bounds on what the kernels may be off by (used by the tests).

u = 2^-24 is half a step of a 32-bit number.  A product of two elements is exact in 32 bits for the 16-bit types and rounds
once for float32; a sum of n products in 32 bits, in any order, is off by at most n steps of the sum of their magnitudes
(a step, 2 u, rather than half of one: the matrix cores' additions are not assumed to round to nearest).
  x     |dx| <= (dim + 1) 2u sum |h w|
  s     relative: the powers' arguments are off by dx of the element and of the maximum, 2 u per unit of their
        size for the product with log2 e, 4 u for the power and the sum's roundings: log2 of the IDs summed pairwise
        would do, but a lane adds up to 32 of them and wavefronts and tiles join in turn: (32 + 8 + tiles) steps, each of
        which may rescale (2 u a unit of the maximum's growth, which is no more than the logits' range)
  G     c (p - [j = y]), rounded to the type (half a step, and the type's smallest number over the scale for float16).  Where
        exponentials are kept, e = exp(x - m') is rounded to no fewer digits than the type's before it is multiplied by c exp(m' - m) / s: half a
        step of c p more (and float16's smallest number over 2^15), except at the target, which has its own logit
  dh    sum_j |dG| |w| and the sum's own error over the padded IDs; then one rounding to the type
  dW    the same over the rows, plus one addition and a rounding where it accumulates."""
import torch

U = 2.0 ** -24
HALF_STEP = {torch.float32: U, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
SMALLEST = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def rounding(x, dtype):
    return HALF_STEP[dtype] * x.abs() + SMALLEST[dtype]


def losses(hidden, weight, targets):
    """(loss, lse, x, kept) in 64 bits, on the tensors' device; 0 where the target is no ID."""
    v = weight.size(0)
    y = targets.long()
    kept = (y >= 0) & (y < v)
    at = torch.where(kept, y, torch.zeros_like(y)).unsqueeze(1)
    h = torch.where(kept.unsqueeze(1), hidden.double(), torch.zeros((), dtype=torch.float64, device=hidden.device))
    x = torch.mm(h, weight.double().t().contiguous())
    lse = torch.logsumexp(x, 1)
    loss = lse - x.gather(1, at).squeeze(1)
    zero = torch.zeros_like(lse)
    return torch.where(kept, loss, zero), torch.where(kept, lse, zero), h, x, kept, at


def gradients(h, weight, x, lse, kept, at, c):
    """(G, grad_hidden, grad_weight) in 64 bits."""
    g = torch.exp(x - lse.unsqueeze(1))
    g.scatter_add_(1, at, -torch.ones_like(at, dtype=torch.float64))
    g = torch.where(kept.unsqueeze(1), g * c.double().unsqueeze(1), torch.zeros((), dtype=torch.float64, device=h.device))
    w = weight.double()
    return g, torch.mm(g, w), torch.mm(g.t().contiguous(), h)


def bounds(h, weight, x, lse, kept, at, c, g, dtype, from_lse, base=None, exact=False):
    """Bounds on the errors of (loss, lse, grad_hidden, grad_weight), of the first two where g is None; grad_weight's without its
    rounding to the output's type.  exact: the logits' products and sums have no roundings in 32 bits."""
    w = weight.double().abs()
    n, dim = h.shape
    v = w.size(0)
    dx = (dim + 1) * 2 * U * torch.mm(h.abs(), w.t().contiguous())
    if exact:
        dx = torch.zeros_like(dx)
    top = x.amax(1, keepdim=True)
    most = dx.amax(1, keepdim=True)
    away = (top - x).clamp(max=104)
    p = torch.exp(x - lse.unsqueeze(1))
    spread = (top - x.amin(1, keepdim=True)).clamp(max=104)
    joins = 32 + 8 + -(-v // 64)
    # a tile's maximum may be off too, but cancels: exp(x - m') exp(m' - m) has errors of x and m alone, and roundings
    rel = (p * (dx + U * (2 * away + 4))).sum(1, keepdim=True) + most + U * (2 * spread + 3 * joins)
    log_s = (lse.unsqueeze(1) - top).abs()
    e_lse = (rel + 4 * U * (log_s + 1) + 2 * U * (top.abs() + lse.unsqueeze(1).abs()) + most).squeeze(1)
    e_loss = e_lse + dx.gather(1, at).squeeze(1) + 2 * U * (top - x.gather(1, at)).abs().squeeze(1)
    zero = torch.zeros_like(e_lse)
    e_loss, e_lse = torch.where(kept, e_loss, zero), torch.where(kept, e_lse, zero)
    if g is None:
        return e_loss, e_lse
    own = dx + most + rel + U * (2 * away + 8)
    if from_lse:
        own = own + e_lse.unsqueeze(1) + 2 * U * (lse.unsqueeze(1).abs() + (lse.unsqueeze(1) - x).abs().clamp(max=104))
    size = c.double().abs().unsqueeze(1)
    hit = torch.zeros_like(g).scatter_(1, at, 1.0)
    lost = SMALLEST[dtype] * (float(c.abs().max()) * 2.0 ** -14 if dtype == torch.float16 else 1.0)
    dg = size * (p * torch.expm1(own.clamp(max=50.0)) + 2.0 ** -126) + (3 * U + HALF_STEP[dtype]) * (g.abs() + size * (p + hit) * own) + lost
    if not from_lse:
        kept_lost = 2.0 ** -40 if dtype == torch.float16 else SMALLEST[dtype]
        dg = dg + size * (1 + HALF_STEP[dtype]) * ((1 - hit) * HALF_STEP[dtype] * p * (1 + own) + kept_lost)
    dg = torch.where(kept.unsqueeze(1), dg, torch.zeros_like(dg))
    ag = g.abs() + dg
    e_h = torch.mm(dg, w) + (v + 256 + 34) * 2 * U * torch.mm(ag, w)
    h = h.abs()
    e_w = torch.mm(dg.t().contiguous(), h) + (n + 64) * 2 * U * torch.mm(ag.t().contiguous(), h)
    ref_h = torch.mm(g, weight.double()).abs() + e_h
    e_h = e_h + 2 * U * ref_h + rounding(ref_h, dtype)
    ref_w = torch.mm(ag.t().contiguous(), h)
    if base is not None:
        ref_w = ref_w + base.double().abs()
    e_w = e_w + 3 * U * ref_w
    return e_loss, e_lse, e_h, e_w


def close(got, ref, err, what):
    got = got.double()
    assert got.shape == ref.shape, what
    off = ~((got - ref).abs() <= err) & ~((got == ref) | (got.isnan() & ref.isnan()))
    if bool(off.any()):
        i = tuple(int(k) for k in off.nonzero()[0])
        raise AssertionError(f"{what}: {int(off.sum())} of {off.numel()} off, first at {i}: {float(got[i])} for {float(ref[i])}, "
                             f"allowed {float(err[i])}")
