"""The bounds of the GPU tests of wide hidden states, without a GPU: at every width that those tests use, the formula's results,
rounded, lie inside them, and wrong ones outside."""
import pytest
import torch

import linear_exact as exact
import linear_plain as plain


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,v,d", [(20, 3000, 4096), (300, 1256, 4096), (90, 3000, 4095), (100, 700, 4097), (60, 300, 16384), (5, 70, 65536),
                                   (33, 300, 65536), (33, 300, 65535)])
@pytest.mark.parametrize("from_lse", [False, True])
def test_bounds_reject_wrong_results(from_lse, n, v, d, dtype):
    h, w, y, c = exact.inputs(n, v, d, dtype, "cpu", ignored=0.1 if n > 5 else 0.0)
    ref = exact.reference(h, w, y, c, dtype, from_lse)
    for key, (value, err) in ref.items():
        plain.close(value.to(dtype if key in ("gh", "gw") else torch.float32), value, err, key)
    exact.reject_wrong(h, w, y, c, ref)
    x = torch.mm(h.double(), w.double().t())
    step = float(w.abs().max())
    assert bool((x / step == torch.round(x / step)).all()) and float(h.shape[1]) < 2 ** 24   # exact whatever the order
    assert 1.0 < float(x.std()) < 6.0


@pytest.mark.parametrize("d", [4096, 65536])
def test_bounds_of_inexact_products_would_not(d):
    """The bounds for any inputs grow with the width, so that they tell less and less: the reason for exact ones."""
    h, w, y, c = exact.inputs(20, 70, d, torch.float32, "cpu")
    loss, lse, hh, x, kept, at = plain.losses(h, w, y)
    loose = plain.bounds(hh, w, x, lse, kept, at, c, None, torch.float32, False)[0]
    tight = plain.bounds(hh, w, x, lse, kept, at, c, None, torch.float32, False, exact=True)[0]
    assert bool((tight < 1e-4).all()) and bool((loose > tight).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [1, 31, 33, 65, 100, 128, 192, 200, 256, 320, 512, 576, 640, 768, 1001, 1024, 2050, 2112])
@pytest.mark.parametrize("from_lse", [False, True])
def test_bounds_of_any_products_up_to_2112_columns(from_lse, d, dtype):
    """The widths at which the GPU tests compare inputs of any kind: zeros, negated, doubled and rolled gradients lie outside."""
    g = torch.Generator().manual_seed(d)
    n, v = 60, 300
    w = (torch.randn(v, d, generator=g) * (2.5 / d ** 0.5)).to(dtype)
    y = torch.randint(0, v, (n,), generator=g, dtype=torch.int32)
    h = (torch.randn(n, d, generator=g) + (6.0 / 2.5 ** 2) * w[y.long()].float()).to(dtype)
    loss, lse, hh, x, kept, at = plain.losses(h, w, y)
    c = torch.rand(n, generator=g) + 0.1
    gr, gh, gw = plain.gradients(hh, w, x, lse, kept, at, c)
    e_loss, e_lse, e_h, e_w = plain.bounds(hh, w, x, lse, kept, at, c, gr, dtype, from_lse)
    e_w = e_w + plain.rounding(gw.abs() + e_w, dtype)
    for key, ref, err in (("gh", gh, e_h), ("gw", gw, e_w)):
        plain.close(ref.to(dtype), ref, err, "rounded")
        for name, wrong in (("zeros", torch.zeros_like(ref)), ("negated", -ref), ("twice", 2 * ref), ("rolled", ref.roll(1, 0))):
            assert float(((wrong - ref).abs() > err).double().mean()) > 0.6, (key, name)
    assert float((e_loss / loss.clamp(min=1.0)).max()) < 0.15 and float(e_lse.max()) < 0.15
