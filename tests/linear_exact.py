"""Wide hidden states whose products with the table and their sums are exact in 32 bits, in any order (used by the tests):
all elements are -1, 0 or 1 times a power of two, so that a logit is a whole number, of less than 24 bits, times another.  A logit
has no error then, and the bounds on what comes after it stay narrow at any width."""
import math

import torch

import linear_plain as plain


def inputs(n, v, d, dtype, device, seed=0, ignored=0.0):
    """(hidden, weight, targets, c): logits of about 2.5 in size, a target's one lifted."""
    gen = torch.Generator(device=device).manual_seed(seed * 1000003 + n * 7919 + v * 31 + d)
    step = 2.0 ** round(math.log2(2.5 / math.sqrt(d * 4.0 / 9.0)))
    w = torch.randint(-1, 2, (v, d), generator=gen, device=device).to(dtype) * step
    h = torch.randint(-1, 2, (n, d), generator=gen, device=device).to(dtype)
    y = torch.randint(0, v, (n,), generator=gen, device=device, dtype=torch.int32)
    # a share of a row's elements take the sign of the target's, for a logit of up to about 6
    u = torch.rand(n, 1, generator=gen, device=device) * 6.0 / (step * d * 2.0 / 3.0)
    like = torch.rand(n, d, generator=gen, device=device) < u
    h = torch.where(like, torch.sign(w[y.long()]), h).to(dtype)
    if ignored:
        y[torch.rand(n, generator=gen, device=device) < ignored] = -1
    c = (torch.rand(n, generator=gen, device=device) + 0.5) / n
    return h, w, y, c


def reference(h, w, y, c, dtype, from_lse):
    """{name: (value, bound)} in 64 bits, grad_weight's before its rounding."""
    loss, lse, hh, x, kept, at = plain.losses(h, w, y)
    g, gh, gw = plain.gradients(hh, w, x, lse, kept, at, c)
    e_loss, e_lse, e_h, e_w = plain.bounds(hh, w, x, lse, kept, at, c, g, dtype, from_lse, exact=True)
    e_h = torch.where(kept.unsqueeze(1), e_h, torch.zeros_like(e_h))
    return dict(loss=(loss, e_loss), lse=(lse, e_lse), gh=(gh, e_h), gw=(gw, e_w + plain.rounding(gw.abs() + e_w, dtype)))


def reject_wrong(h, w, y, c, ref):
    """Asserts that most of what is wrong lies outside the bounds: gradients of zeros, negated, twice as large, of the next row (of
    a sum of many terms of both signs some elements are small beside their terms' roundings); losses without the last tenth of the
    columns, or without the last 32 of them."""
    for key in ("gh", "gw"):
        value, err = ref[key]
        some = value.abs().amax(1) > 0
        for name, wrong in (("zeros", torch.zeros_like(value)), ("negated", -value), ("twice", 2 * value), ("rolled", value.roll(1, 0))):
            share = float(((wrong - value).abs() > err)[some].double().mean())
            assert share > 0.6, (key, name, share)
    d = h.size(1)
    for cut in (d - d // 10, d - 32):
        loss = plain.losses(h[:, :cut], w[:, :cut], y)[0]
        value, err = ref["loss"]
        kept = (y >= 0) & (y < w.size(0))
        share = float(((loss - value).abs() > err)[kept].double().mean())
        assert share > 0.9, ("loss", cut, share)
