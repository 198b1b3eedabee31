"""Cross entropy from hidden states on the GPU against 64 bits: types, odd sizes, strides and alignments, sizes around
the tiles and pieces, ignored positions, values that are not finite, accumulation, streams and graphs."""
import math

import pytest
import torch

import linear_plain as plain

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [BF16, F16, F32]


def _say(*a):
    print("[gpu-case]", *a, flush=True)


def _matrix(values, pad=0, lead=0):
    """`values` in a view whose rows lie `pad` elements further apart than they are long and which begins `lead`
    elements into its buffer; NaN around it."""
    rows, cols = values.shape
    flat = torch.full((lead + rows * (cols + pad) + 8,), math.nan, dtype=values.dtype, device="cuda")
    view = flat[lead:lead + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(values)
    return view, flat


def _around(flat, view):
    return int(torch.isnan(flat).sum()) - int(torch.isnan(view).sum()) == flat.numel() - view.numel()


class Case:
    """Inputs of one call, and what it has to give."""

    def __init__(self, n, v, d, dtype, ignored=0.0, pad=0, lead=0, size=2.5, seed=0, lift=6.0):
        self.gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + n * 7919 + v * 31 + d)
        r = lambda *s: torch.randn(*s, generator=self.gen, device="cuda")
        self.n, self.v, self.d, self.dtype = n, v, d, dtype
        w = (r(v, d) * (size / math.sqrt(d))).to(dtype)
        y = torch.randint(0, v, (n,), generator=self.gen, device="cuda", dtype=torch.int32)
        h = (r(n, d) + (lift / size ** 2) * w[y.long()].float()).to(dtype)
        if ignored:
            bad = torch.rand(n, generator=self.gen, device="cuda") < ignored
            odd = torch.tensor([-1, v, v + 7, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
            y = torch.where(bad, odd[torch.randint(0, 5, (n,), generator=self.gen, device="cuda")], y)
            h[bad] = math.nan    # what is ignored is not used
        self.hidden, self.weight = _matrix(h, pad, lead)[0], _matrix(w, pad, lead)[0]
        self.targets = y
        self.grad_loss = (torch.rand(n, generator=self.gen, device="cuda") + 0.1) / n
        self.scale = 1024.0 if dtype == F16 else 1.5
        self.pad, self.lead = pad, lead

    def outputs(self, weight_dtype=None, base=None):
        v = lambda: torch.full((self.n,), 7.0, device="cuda")
        gw = torch.full((self.v, self.d), 5.0, device="cuda") if base is None else base
        return dict(loss=v(), lse=v(), gh=_matrix(torch.full((self.n, self.d), 3.0, device="cuda").to(self.dtype), self.pad, self.lead),
                    gw=_matrix(gw.to(weight_dtype or self.dtype), self.pad, self.lead))

    def workspace(self, tt, grads=True):
        size = tt.toktier_linear_cross_entropy_workspace_bytes(self.n, self.v, self.d, self.dtype, grads)
        return torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")

    def forward(self, tt, o, ws, grads=True, **more):
        if grads:
            more = dict(grad_hidden=o["gh"][0], grad_weight=o["gw"][0], grad_loss=self.grad_loss, grad_scale=self.scale, **more)
        tt.toktier_linear_cross_entropy(self.hidden, self.weight, self.targets, o["loss"], o["lse"], ws, **more)

    def backward(self, tt, o, ws, **more):
        more = dict(dict(grad_hidden=o["gh"][0], grad_weight=o["gw"][0]), **more)
        tt.toktier_linear_cross_entropy_backward(self.hidden, self.weight, self.targets, o["lse"], ws, grad_loss=self.grad_loss,
                                                 grad_scale=self.scale, **more)

    def check(self, o, what, from_lse=False, hidden=True, weight=True, base=None, losses=True):
        c = self.grad_loss * self.scale
        loss, lse, h, x, kept, at = plain.losses(self.hidden, self.weight, self.targets)
        g, gh, gw = plain.gradients(h, self.weight, x, lse, kept, at, c)
        e_loss, e_lse, e_h, e_w = plain.bounds(h, self.weight, x, lse, kept, at, c, g, self.dtype, from_lse, base=base)
        if losses:
            plain.close(o["loss"], loss, e_loss, what + " loss")
            plain.close(o["lse"], lse, e_lse, what + " lse")
        if hidden:
            plain.close(o["gh"][0], gh, torch.where(kept.unsqueeze(1), e_h, torch.zeros_like(e_h)), what + " grad_hidden")
        if weight:
            ref = gw if base is None else gw + base.double()
            out = o["gw"][0]
            plain.close(out, ref, e_w + plain.rounding(ref.abs() + e_w, out.dtype), what + " grad_weight")
        for k in ("gh", "gw"):
            if self.pad:
                assert _around(o[k][1], o[k][0]), what


SIZES = [(1, 1, 1), (1, 2, 7), (3, 65, 64), (17, 300, 100), (64, 257, 128), (65, 1256, 320), (130, 63, 33), (255, 1001, 31),
         (257, 256, 65), (600, 5001, 1001), (16, 20000, 256)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,d", SIZES)
def test_loss_and_gradients(tt, n, v, d, dtype):
    _say("linear", n, v, d, dtype)
    case = Case(n, v, d, dtype, ignored=0.2 if n > 3 else 0.0)
    ws = case.workspace(tt)
    o = case.outputs()
    case.forward(tt, o, ws)
    case.check(o, "one call")
    later = case.outputs()
    later["loss"], later["lse"] = o["loss"], o["lse"].clone()
    case.backward(tt, later, ws.fill_(0x5A))
    case.check(later, "later", from_lse=True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,lead", [(1, 0), (0, 1), (64, 0), (64, 8), (3, 5)])
def test_strides_and_alignments(tt, pad, lead, dtype):
    _say("linear strides", pad, lead, dtype)
    case = Case(75, 700, 192, dtype, ignored=0.1, pad=pad, lead=lead)
    o = case.outputs()
    case.forward(tt, o, case.workspace(tt))
    case.check(o, "strides")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,d", [
    (300, 6000, 1024),        # several tiles of the middle size; dh in shares
    (1100, 9000, 576),
    (2100, 6500, 640),        # the largest tiles
    (600, 140001, 64),        # several pieces of the backward pass alone
    (4200, 140001, 64),       # more than is kept
])
def test_large_tiles_and_pieces(tt, n, v, d, dtype):
    _say("linear large", n, v, d, dtype)
    case = Case(n, v, d, dtype, ignored=0.1)
    ws = case.workspace(tt)
    o = case.outputs()
    case.forward(tt, o, ws)
    case.check(o, "large")


@pytest.mark.parametrize("n,v,d,dtype", [
    (300, 33124, 512, BF16), (300, 33124, 512, F16), (300, 33124, 256, F32),   # IDs too
    (640, 33001, 200, F16), (385, 33024, 320, BF16),
    (300, 131328, 768, BF16),                                                  # a table that the cache does not hold
    (1350, 66000, 64, BF16),                                                   # strips at the end too
])
def test_last_tiles_that_are_half_empty(tt, n, v, d, dtype):
    _say("linear halves", n, v, d, dtype)
    case = Case(n, v, d, dtype, ignored=0.05)
    ws = case.workspace(tt)
    o = case.outputs()
    case.forward(tt, o, ws)
    case.check(o, "one call")
    later = case.outputs()
    later["loss"], later["lse"] = o["loss"], o["lse"].clone()
    case.backward(tt, later, ws.fill_(0x5A))
    case.check(later, "later", from_lse=True)


def test_pieces_of_a_copied_table(tt):
    _say("linear copied pieces")
    case = Case(200, 40000, 2050, BF16, ignored=0.1, pad=1)   # 164 MB of table: two pieces for the loss
    o = case.outputs()
    case.forward(tt, o, case.workspace(tt))
    case.check(o, "copied pieces")


@pytest.mark.parametrize("extra", [0, 8])
def test_rows_four_mebibytes_apart(tt, extra):
    """The furthest apart that a table is read where it lies, and further; both pass 2^32 bytes."""
    _say("linear far apart", extra)
    case = Case(70, 1100, 64, BF16, ignored=0.1)
    flat = torch.full((1100, (1 << 21) + extra), math.nan, dtype=BF16, device="cuda")
    flat[:, :64] = case.weight
    case.weight = flat[:, :64]
    o = case.outputs()
    case.forward(tt, o, case.workspace(tt))
    case.check(o, "far apart")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,d", [(5, 70, 65536), (300, 300, 16384), (70000, 300, 16)])
def test_wide_and_tall(tt, n, v, d, dtype):
    _say("linear wide and tall", n, v, d, dtype)
    case = Case(n, v, d, dtype, ignored=0.3 if n > 5 else 0.0)
    ws = case.workspace(tt)
    o = case.outputs()
    case.forward(tt, o, ws)
    case.check(o, "one call")
    later = case.outputs()
    later["loss"], later["lse"] = o["loss"], o["lse"].clone()
    case.backward(tt, later, ws.fill_(0x5A))
    case.check(later, "later", from_lse=True)


@pytest.mark.parametrize("dtype", TYPES)
def test_one_gradient_alone(tt, dtype):
    _say("linear one gradient", dtype)
    case = Case(150, 3000, 256, dtype, ignored=0.1)
    ws = case.workspace(tt)
    o = case.outputs()
    case.forward(tt, o, case.workspace(tt, False), grads=False)
    case.check(o, "loss alone", hidden=False, weight=False)
    assert bool((o["gh"][0] == 3).all()) and bool((o["gw"][0] == 5).all())
    case.backward(tt, o, ws, grad_weight=None)
    case.check(o, "hidden alone", from_lse=True, weight=False)
    assert bool((o["gw"][0] == 5).all())
    o["gh"][0].fill_(3)
    case.backward(tt, o, ws, grad_hidden=None)
    case.check(o, "weight alone", from_lse=True, hidden=False)
    assert bool((o["gh"][0] == 3).all())


@pytest.mark.parametrize("dtype,weight_dtype", [(BF16, BF16), (BF16, F32), (F16, F32), (F32, F32)])
@pytest.mark.parametrize("pad", [0, 3])
def test_accumulation(tt, dtype, weight_dtype, pad):
    _say("linear accumulate", dtype, weight_dtype, pad)
    case = Case(90, 1256, 320, dtype, ignored=0.1, pad=pad)
    base = torch.randn(1256, 320, generator=case.gen, device="cuda").to(weight_dtype)
    o = case.outputs(weight_dtype, base)
    case.forward(tt, o, case.workspace(tt), accumulate=True)
    case.check(o, "accumulate", base=base)
    o = case.outputs(weight_dtype)
    case.forward(tt, o, case.workspace(tt))
    case.check(o, "written")


@pytest.mark.parametrize("dtype", TYPES)
def test_all_ignored_and_none_at_all(tt, dtype):
    _say("linear ignored", dtype)
    case = Case(40, 300, 64, dtype)
    case.targets.fill_(-1)
    case.hidden.fill_(math.nan)
    o = case.outputs()
    case.forward(tt, o, case.workspace(tt))
    assert not any(bool(t.any()) for t in (o["loss"], o["lse"], o["gh"][0], o["gw"][0]))
    base = torch.randn(300, 64, device="cuda")
    o = case.outputs(base=base)
    case.forward(tt, o, case.workspace(tt), accumulate=True)
    assert torch.equal(o["gw"][0], base.to(dtype))
    none = torch.empty(0, 64, dtype=dtype, device="cuda")
    empty, ids = torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    ws = torch.empty(tt.toktier_linear_cross_entropy_workspace_bytes(0, 300, 64, dtype), dtype=torch.uint8, device="cuda")
    gw = torch.full((300, 64), 5.0, device="cuda").to(dtype)
    tt.toktier_linear_cross_entropy(none, case.weight, ids, empty, empty, ws, grad_hidden=none, grad_weight=gw, accumulate=True)
    assert bool((gw == 5).all())
    tt.toktier_linear_cross_entropy(none, case.weight, ids, empty, empty, ws, grad_hidden=none, grad_weight=gw)
    assert not bool(gw.any())


@pytest.mark.parametrize("dtype", TYPES)
def test_not_finite_values_stay_in_their_rows(tt, dtype):
    _say("linear not finite", dtype)
    case = Case(70, 500, 128, dtype)
    good = case.outputs()
    case.forward(tt, good, case.workspace(tt))
    for row, value in ((3, math.nan), (40, math.inf), (69, -math.inf)):
        case.hidden[row, 5] = value
    o = case.outputs()
    case.forward(tt, o, case.workspace(tt))
    bad = torch.zeros(70, dtype=torch.bool, device="cuda")
    bad[[3, 40, 69]] = True
    assert bool(o["loss"][bad].isnan().all()) and bool(o["gh"][0][bad].isnan().all())
    for k in ("loss", "lse"):
        assert torch.equal(o[k][~bad], good[k][~bad])
    assert torch.equal(o["gh"][0][~bad], good["gh"][0][~bad])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size,lift", [(200.0, 0.0), (0.001, 0.0), (30.0, 900.0)])
def test_sizes_of_logits(tt, dtype, size, lift):
    _say("linear sizes", dtype, size, lift)
    case = Case(100, 800, 256, dtype, size=size, lift=lift)
    o = case.outputs()
    case.forward(tt, o, case.workspace(tt))
    case.check(o, "sizes")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,v,d", [(3, 500, 64), (300, 40000, 64)])
@pytest.mark.parametrize("size", [1.7e19, 3e14, 1e8, 1000.0, 200.0])
def test_logits_at_the_end_of_the_range(tt, size, n, v, d, dtype):
    """Logits up to -+3e38, whose product with log2(e) has no number or is off by more than a power's range: equal ones share the
    probability, far ones have none."""
    _say("linear range", size, n, v, d, dtype)
    h = torch.zeros(n, d, dtype=dtype, device="cuda")
    w = torch.zeros(v, d, dtype=dtype, device="cuda")
    big = torch.full((1,), size, dtype=dtype, device="cuda")
    w[:, 0], h[0, 0], h[1, 0] = -big, big, -big    # row 0: all logits -2.9e38, row 1: all 2.9e38
    w[v // 2:, 1], h[2, 1] = -big, big             # row 2: one half 0, the other -2.9e38
    y = torch.full((n,), 7, dtype=torch.int32, device="cuda")
    loss, lse, gw = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty(v, d, device="cuda")
    ws = torch.empty(tt.toktier_linear_cross_entropy_workspace_bytes(n, v, d, dtype), dtype=torch.uint8, device="cuda")
    tt.toktier_linear_cross_entropy(h, w, y, loss, lse, ws, grad_weight=gw, grad_scale=2.0 ** -40)
    x = torch.zeros(n, v, dtype=torch.float64, device="cuda")
    x[0], x[1], x[2, v // 2:] = -big.double() ** 2, big.double() ** 2, -big.double() ** 2
    z = torch.logsumexp(x, 1)
    plain.close(lse, z, 4 * plain.U * z.abs() + plain.U * (8 * 104 + 3 * (v // 16 + 64)), "range lse")
    ref = (x.amax(1) - x[:, 7]) + torch.log(torch.exp(x - x.amax(1, keepdim=True)).sum(1))
    plain.close(loss, ref, 4 * plain.U * ref.abs() + plain.U * (8 * 104 + 3 * (v // 16 + 64)), "range loss")
    p = torch.exp(x - x.amax(1, keepdim=True))
    g = p / p.sum(1, keepdim=True)
    g[:, 7] -= 1.0
    g *= 2.0 ** -40
    ref = torch.mm(g.t().contiguous(), h.double())
    # G is kept rounded, and so are the exponentials; the powers' and sums' errors are below 2^-12
    err = torch.mm(g.abs().t().contiguous(), h.double().abs()) * (2 * plain.rounding(torch.ones((), dtype=torch.float64, device="cuda"), dtype) + 2.0 ** -12)
    plain.close(gw, ref, err, "range grad_weight")


def test_float16_keeps_small_probabilities(tt):
    """131,072 equal logits: every probability is 2^-17, and times c far below float16's numbers."""
    _say("linear float16 small")
    n, v, d = 8, 131072, 64
    w = torch.zeros(v, d, dtype=F16, device="cuda")
    h = torch.ones(n, d, dtype=F16, device="cuda")
    y = torch.arange(n, dtype=torch.int32, device="cuda")
    loss, lse, gw = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty(v, d, device="cuda")
    ws = torch.empty(tt.toktier_linear_cross_entropy_workspace_bytes(n, v, d, F16), dtype=torch.uint8, device="cuda")
    tt.toktier_linear_cross_entropy(h, w, y, loss, lse, ws, grad_weight=gw, grad_scale=2.0 ** -30)
    ref = torch.full((v, d), n * 2.0 ** -47, dtype=torch.float64, device="cuda")
    ref[:n] -= 2.0 ** -30
    plain.close(gw, ref, 2.0 ** -10 * ref.abs(), "float16 small")


def test_offsets_past_32_bits(tt):
    _say("linear far rows")
    v, d, n = 1 << 21, 2112, 3
    w = torch.zeros(v, d, dtype=BF16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(5)
    h = torch.randn(n, d, generator=gen, device="cuda").to(BF16)
    at = torch.tensor([v - 1, v // 2 + 7, 2035000], device="cuda")
    w[at] = (torch.randn(n, d, generator=gen, device="cuda") * 0.3).to(BF16)
    y = at.to(torch.int32)
    loss, lse, gh = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty_like(h)
    ws = torch.empty(tt.toktier_linear_cross_entropy_workspace_bytes(n, v, d, BF16), dtype=torch.uint8, device="cuda")
    gw = torch.empty_like(w)
    tt.toktier_linear_cross_entropy(h, w, y, loss, lse, ws, grad_hidden=gh, grad_weight=gw)
    some = torch.zeros(n + 1, d, dtype=torch.float64, device="cuda")   # the three rows, and the others' zeros
    some[:n] = w[at].double()
    x = torch.mm(h.double(), some.t().contiguous())
    z = torch.logsumexp(torch.cat([x[:, :n], x[:, n:] + math.log(v - n)], 1), 1)
    p = torch.exp(x - z.unsqueeze(1))
    g = p[:, :n] - torch.eye(n, dtype=torch.float64, device="cuda")
    dx = (d + 1) * 2 * plain.U * torch.mm(h.double().abs(), some.abs().t().contiguous()).amax(1)
    ref = z - torch.diagonal(x[:, :n])
    err = 3 * dx + plain.U * (8 * 104 + 3 * (v // 256 + 64))
    plain.close(lse, z, err + 4 * plain.U * z.abs(), "far lse")
    plain.close(loss, ref, err + 4 * plain.U * (z.abs() + ref.abs()), "far loss")
    own = torch.expm1(2 * err).unsqueeze(1)
    dg = p[:, :n] * own + (2 ** -8 + 4 * plain.U) * g.abs()
    ref = torch.mm(g, some[:n])
    e = torch.mm(dg, some[:n].abs()) + 64 * plain.U * torch.mm(g.abs(), some[:n].abs())
    plain.close(gh, ref, e + plain.rounding(ref.abs() + e, BF16), "far grad_hidden")
    ref = torch.mm(g.t().contiguous(), h.double())
    e = torch.mm(dg.t().contiguous(), h.double().abs()) + 64 * plain.U * torch.mm(g.abs().t().contiguous(), h.double().abs())
    plain.close(gw[at], ref, e + plain.rounding(ref.abs() + e, BF16), "far grad_weight")
    rest = torch.mm(p[:, n:].t().contiguous(), h.double())
    e = 2.0 ** -7 * torch.mm(p[:, n:].t().contiguous(), h.double().abs()) + torch.mm((p[:, n:] * own).t().contiguous(), h.double().abs())
    others = torch.tensor([0, 1, v // 2, v - 2, 2034999], device="cuda")
    plain.close(gw[others], rest.expand(5, d), (e + plain.rounding(rest.abs() + e, BF16)).expand(5, d), "far zeros")


def test_more_tiles_than_one_launch_takes(tt):
    """2^19 rows and as many IDs that the tiles of all of them would have more than 2^32 threads."""
    _say("linear many tiles")
    n, v, d = 1 << 19, (1 << 20) + 300, 64
    gen = torch.Generator(device="cuda").manual_seed(6)
    w = (torch.randn(v, d, generator=gen, device="cuda") * 0.3).to(BF16)
    h = torch.randn(n, d, generator=gen, device="cuda").to(BF16)
    y = torch.randint(0, v, (n,), generator=gen, device="cuda", dtype=torch.int32)
    loss, lse = torch.full((n,), 7.0, device="cuda"), torch.full((n,), 7.0, device="cuda")
    ws = torch.empty(tt.toktier_linear_cross_entropy_workspace_bytes(n, v, d, BF16, grads=False), dtype=torch.uint8,
                     device="cuda")
    tt.toktier_linear_cross_entropy(h, w, y, loss, lse, ws)
    some = torch.cat([torch.arange(0, n, n // 61, device="cuda"), torch.tensor([n - 1, n - 257, n // 2 - 1], device="cuda")])
    x = torch.mm(h[some].double(), w.double().t().contiguous())
    z = torch.logsumexp(x, 1)
    ref = z - x.gather(1, y[some].long().unsqueeze(1)).squeeze(1)
    dx = (d + 1) * 2 * plain.U * torch.mm(h[some].double().abs(), w.double().abs().t().contiguous()).amax(1)
    err = 3 * dx + plain.U * (8 * 104 + 3 * (v // 256 + 64))
    plain.close(lse[some], z, err + 4 * plain.U * z.abs(), "many tiles lse")
    plain.close(loss[some], ref, err + 4 * plain.U * (z.abs() + ref.abs()), "many tiles loss")


def test_against_differences(tt):
    """The gradients' slopes along random directions against differences of the 64-bit loss."""
    _say("linear differences")
    case = Case(40, 600, 96, F32, ignored=0.2, size=1.0)
    o = case.outputs()
    case.forward(tt, o, case.workspace(tt))
    c = (case.grad_loss * case.scale).double()
    safe = torch.nan_to_num(case.hidden)
    total = lambda h, w: float((plain.losses(h, w, case.targets)[0] * c).sum())
    for k in range(4):
        dh = torch.randn(40, 96, generator=case.gen, device="cuda").double()
        dw = torch.randn(600, 96, generator=case.gen, device="cuda").double()
        eps = 1e-5
        slope = (total(safe + eps * dh, case.weight) - total(safe - eps * dh, case.weight)) / (2 * eps)
        own = (o["gh"][0].double() * dh).sum()
        # differences in the middle: off by eps^2 / 6 of the third derivative, and 2^-52 of the sum over eps
        size = float((o["gh"][0].double().abs() * dh.abs()).sum())
        assert abs(slope - float(own)) <= 1e-5 * size + 1e-8, k
        slope = (total(safe, case.weight + eps * dw) - total(safe, case.weight - eps * dw)) / (2 * eps)
        own = (o["gw"][0].double() * dw).sum()
        size = float((o["gw"][0].double().abs() * dw.abs()).sum())
        assert abs(slope - float(own)) <= 1e-5 * size + 1e-8, k


def _bits(o):
    return [o["loss"], o["lse"], o["gh"][0], o["gw"][0]]


def test_repeated_calls_give_the_same_bits(tt):
    _say("linear bits")
    for case in (Case(300, 6000, 1024, BF16, ignored=0.3), Case(90, 3000, 320, F32), Case(33, 70000, 512, F16)):
        ws = case.workspace(tt)
        first = None
        for fill in (0, 255, 0x7F):
            o = case.outputs()
            case.forward(tt, o, ws.fill_(fill))
            if first is not None:
                assert all(torch.equal(a, b) for a, b in zip(_bits(first), _bits(o)))
            first = o


def test_another_stream_and_graphs_that_share_a_workspace(tt):
    _say("linear graphs")
    cases = [Case(120, 3000, 256, BF16, ignored=0.2, seed=1), Case(40, 1256, 320, F16, ignored=0.2, seed=2)]
    want = []
    for c in cases:
        o = c.outputs()
        c.forward(tt, o, c.workspace(tt))
        want.append([t.clone() for t in _bits(o)])
    ws = torch.empty(max(c.workspace(tt).numel() for c in cases), dtype=torch.uint8, device="cuda")
    outs, graphs = [c.outputs() for c in cases], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c, o in zip(cases, outs):
            c.forward(tt, o, ws)
    side.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(_bits(o), w))
    for c, o in zip(cases, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.forward(tt, o, ws)
        graphs.append(graph)
    for turn in range(4):
        for i in (0, 1, 1, 0)[turn:turn + 2]:
            for t in _bits(outs[i]):
                t.fill_(9)
            ws.fill_(turn * 37)
            graphs[i].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(_bits(outs[i]), want[i])), (turn, i)
    # new inputs in the same places, other rows ignored
    c, o = cases[0], outs[0]
    c.hidden.copy_(torch.randn(120, 256, generator=c.gen, device="cuda"))
    c.targets.copy_(torch.randint(-900, 3000, (120,), generator=c.gen, device="cuda", dtype=torch.int32))
    graphs[0].replay()
    c.check(o, "replayed on new inputs")


def test_agrees_with_the_loss_of_kept_logits(tt):
    _say("linear and logits")
    case = Case(200, 2000, 128, F32, ignored=0.2)
    case.hidden.copy_(torch.nan_to_num(case.hidden))
    o = case.outputs()
    case.forward(tt, o, case.workspace(tt))
    x = torch.mm(case.hidden, case.weight.t())
    loss, lse, g = torch.empty(200, device="cuda"), torch.empty(200, device="cuda"), torch.empty_like(x)
    ws = torch.empty(tt.toktier_cross_entropy_workspace_bytes(200, 2000), dtype=torch.uint8, device="cuda")
    tt.toktier_cross_entropy(x, case.targets, loss, lse, ws, grad_logits=g, grad_loss=case.grad_loss, grad_scale=case.scale)
    assert torch.allclose(o["loss"], loss, rtol=1e-4, atol=1e-4)
    assert torch.allclose(o["gh"][0], torch.mm(g, case.weight), rtol=1e-3, atol=1e-6)
    assert torch.allclose(o["gw"][0], torch.mm(g.t(), case.hidden), rtol=1e-3, atol=1e-6)
