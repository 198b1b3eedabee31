"""Distillation from a teacher's top logits on the GPU against 64 bits: types, sizes, lists with gaps and with an ID twice,
strides, in place, values that are not finite, the gradient from lse, streams and graphs."""
import math

import pytest
import torch

import distill_plain as plain
from linear_plain import close

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [BF16, F16, F32]


def _say(*a):
    print("[gpu-case]", *a, flush=True)


def _matrix(values, pad=0, lead=0):
    rows, cols = values.shape
    flat = torch.full((lead + rows * (cols + pad) + 8,), math.nan, dtype=values.dtype, device="cuda")
    view = flat[lead:lead + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(values)
    return view, flat


class Case:
    def __init__(self, n, v, k, dtype, temperature=1.0, own_lse=False, gaps=0.0, pad=0, lead=0, size=2.5, shift=0.0, seed=0):
        self.gen = g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + n * 7919 + v * 31 + k)
        self.n, self.v, self.k, self.dtype, self.t, self.pad, self.lead = n, v, k, dtype, temperature, pad, lead
        x = shift + size * torch.randn(n, v, generator=g, device="cuda")
        teacher = x + torch.randn(n, v, generator=g, device="cuda")
        top, ids = torch.topk(teacher, min(k, v), dim=1)
        if k > v:   # lists longer than the vocabulary: nothing more in them
            ids = torch.cat([ids, torch.full((n, k - v), -1, device="cuda")], 1)
            top = torch.cat([top, torch.randn(n, k - v, device="cuda", generator=g)], 1)
        self.ids = ids.to(torch.int32).contiguous()
        if gaps:
            bad = torch.rand(n, k, generator=g, device="cuda") < gaps
            bad[:, 0] = False
            odd = torch.tensor([-1, v, v + 7, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
            self.ids = torch.where(bad, odd[torch.randint(0, 5, (n, k), generator=g, device="cuda")], self.ids)
            top = torch.where(bad, torch.full_like(top, math.nan), top)   # what is no entry is not used
        self.top = top.contiguous()
        self.teacher_lse = torch.logsumexp(teacher / temperature, 1) if own_lse else None
        self.logits, self.flat = _matrix(x.to(dtype), pad, lead)
        self.grad_loss = (torch.rand(n, generator=g, device="cuda") + 0.1) / n
        self.scale = 1024.0 if dtype == F16 else 1.5

    def outputs(self):
        v = lambda: torch.full((self.n,), 7.0, device="cuda")
        grad, flat = _matrix(torch.full((self.n, self.v), 3.0, device="cuda").to(self.dtype), self.pad, self.lead)
        return dict(loss=v(), lse=v(), grad=grad, flat=flat)

    def workspace(self, tt):
        return torch.full((tt.toktier_distill_workspace_bytes(self.n, self.v, self.k),), 0xA5, dtype=torch.uint8, device="cuda")

    def forward(self, tt, o, grad=True):
        more = dict(grad_logits=o["grad"], grad_loss=self.grad_loss, grad_scale=self.scale) if grad else {}
        tt.toktier_distill(self.logits, self.ids, self.top, o["loss"], o["lse"], self.workspace(tt), temperature=self.t,
                           teacher_lse=self.teacher_lse, **more)

    def backward(self, tt, o):
        tt.toktier_distill_backward(self.logits, self.ids, self.top, o["lse"], o["grad"], temperature=self.t, teacher_lse=self.teacher_lse,
                                    grad_loss=self.grad_loss, grad_scale=self.scale)

    def reference(self, x=None, from_lse=False):
        lse = None if self.teacher_lse is None else self.teacher_lse.double()
        return plain.distill((self.logits if x is None else x).double(), self.ids, self.top.double(), self.t, lse,
                             self.grad_loss.double() * self.scale, self.dtype, from_lse)

    def check(self, o, ref, what, keys=("loss", "lse", "grad")):
        for key in keys:
            close(o[key], *ref[key], f"{what} {key}")
        if self.pad:
            assert int(torch.isnan(o["flat"]).sum()) == o["flat"].numel() - o["grad"].numel(), what


SIZES = [(1, 1, 1), (2, 2, 5), (3, 7, 3), (17, 1256, 8), (33, 8192, 64), (9, 8193, 65), (5, 33001, 100), (3, 40000, 1024),
         (2, 65536, 64), (159, 65537, 7), (160, 65537, 7), (1, 131328, 300), (4, 200019, 64)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,k", SIZES)
def test_loss_and_gradient(tt, n, v, k, dtype):
    own_lse, t = (n + k) % 2 == 0, (1.0, 2.0, 0.75)[(n + v) % 3]
    _say("distill", n, v, k, dtype, own_lse, t)
    case = Case(n, v, k, dtype, t, own_lse, gaps=0.2)
    o = case.outputs()
    case.forward(tt, o)
    case.check(o, case.reference(), "one call")
    alone = case.outputs()
    case.forward(tt, alone, grad=False)
    assert torch.equal(alone["loss"], o["loss"]) and torch.equal(alone["lse"], o["lse"]) and bool((alone["grad"] == 3).all())
    later = case.outputs()
    later["lse"] = o["lse"]
    case.backward(tt, later)
    case.check(later, case.reference(from_lse=True), "later", ("grad",))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,pad,lead", [(20, 1256, 1, 0), (20, 1255, 0, 1), (7, 65539, 5, 3), (170, 65539, 3, 0), (4, 20000, 64, 8)])
def test_strides_and_in_place(tt, n, v, pad, lead, dtype):
    _say("distill strides", n, v, pad, lead, dtype)
    case = Case(n, v, 20, dtype, 1.5, pad=pad, lead=lead, gaps=0.1)
    wide = torch.full((n, 29), math.nan, device="cuda")
    wide[:, 3:23] = case.top
    case.top = wide[:, 3:23]
    wide = torch.full((n, 31), 5, dtype=torch.int32, device="cuda")
    wide[:, :20] = case.ids
    case.ids = wide[:, :20]
    ref, from_lse, x = case.reference(), case.reference(from_lse=True), case.logits.clone()
    o = case.outputs()
    case.forward(tt, o)
    case.check(o, ref, "strides")
    o["grad"], o["flat"] = case.logits, case.flat
    case.forward(tt, o)
    case.check(o, ref, "in place")
    case.logits.copy_(x)
    case.backward(tt, o)
    case.check(o, from_lse, "in place later", ("grad",))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,k", [(40, 1256, 64), (3, 70000, 64), (5, 40000, 1024)])
def test_an_id_twice(tt, n, v, k, dtype):
    _say("distill twice", n, v, k, dtype)
    case = Case(n, v, k, dtype)
    case.ids[:, k // 2] = case.ids[:, 0]
    case.ids[1::2, 1:k // 3] = case.ids[1::2, :1]
    ref = case.reference()
    first = None
    for _ in range(3):
        o = case.outputs()
        case.forward(tt, o)
        case.check(o, ref, "twice")
        if first is not None:
            assert torch.equal(first["grad"], o["grad"]) and torch.equal(first["loss"], o["loss"])
        first = o
    o = case.outputs()
    o["lse"] = first["lse"]
    case.backward(tt, o)
    case.check(o, case.reference(from_lse=True), "twice later", ("grad",))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v", [(12, 1256), (3, 70000), (12, 30000)])
@pytest.mark.parametrize("shift,size", [(1000.0, 2.5), (-1000.0, 2.5), (127.0, 1.0), (0.0, 60.0)])
def test_far_logits(tt, n, v, shift, size, dtype):
    _say("distill far", n, v, shift, size, dtype)
    case = Case(n, v, 30, dtype, 1.0, own_lse=False, shift=shift, size=size)
    o = case.outputs()
    case.forward(tt, o)
    case.check(o, case.reference(), "far")
    later = case.outputs()
    later["lse"] = o["lse"]
    case.backward(tt, later)
    case.check(later, case.reference(from_lse=True), "far later", ("grad",))
    case.logits.copy_(case.logits.clone())
    x = case.logits.clone()
    ref = case.reference(from_lse=True)
    later["grad"] = case.logits
    case.backward(tt, later)
    case.check(later, ref, "far later in place", ("grad",))
    case.logits.copy_(x)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [1256, 30000, 70000])
def test_rows_that_are_empty_or_not_finite(tt, v, dtype):
    _say("distill odd rows", v, dtype)
    n, k = 10, 20
    case = Case(n, v, k, dtype)
    good = case.outputs()
    case.forward(tt, good)
    x, ids, top = case.logits, case.ids, case.top
    x[1] = -math.inf                      # a mask that leaves nothing
    x[2, 5] = math.nan
    x[3, v - 1] = math.inf
    ids[4] = -1                           # no list
    top[5] = -math.inf                    # a list without weight
    x[6, int(ids[6, 3])] = -math.inf      # a listed ID that the row rules out
    top[6, 2] = -math.inf                 # and one that the list does
    top[7, 0] = math.nan
    x[8] = -math.inf
    ids[8] = -1
    x[9, 7] = math.nan
    ids[9] = v
    for later in (False, True):
        o = case.outputs()
        if later:
            o["lse"] = lse
            case.backward(tt, o)
        else:
            case.forward(tt, o)
            lse = o["lse"]
            loss = o["loss"]
            assert float(loss[1]) == math.inf and float(lse[1]) == -math.inf
            assert bool(loss[2:4].isnan().all()) and bool(lse[2:4].isnan().all())
            assert float(loss[4]) == 0 and float(loss[5]) == 0 and float(loss[6]) == math.inf
            assert bool(loss[7].isnan()) and float(lse[7]) == float(good["lse"][7])
            assert float(loss[8]) == 0 and float(lse[8]) == -math.inf and float(loss[9]) == 0 and bool(lse[9].isnan())
            assert torch.equal(loss[:1], good["loss"][:1]) and torch.equal(o["grad"][0], good["grad"][0])
        g = o["grad"].float()
        assert not bool(g[[1, 4, 5, 8, 9]].any())
        assert bool(g[2:4].isnan().all()) and bool(g[7].isnan().all())
        assert bool(g[6].isfinite().all()) and float(g[6, int(ids[6, 3])]) < 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,v,k", [(7, 1256, 8), (3, 33001, 100), (2, 65537, 64)])
@pytest.mark.parametrize("t", [1e-30, 1e-4, 1e4, 1e30])
def test_temperatures_far_from_one(tt, t, n, v, k, dtype):
    _say("distill temperature", t, n, v, k, dtype)
    case = Case(n, v, k, dtype, t)
    o = case.outputs()
    case.forward(tt, o)
    case.check(o, case.reference(), "one call")


def test_no_rows(tt):
    e, i = torch.empty(0, 8, device="cuda"), torch.empty(0, 3, dtype=torch.int32, device="cuda")
    v, t = torch.empty(0, device="cuda"), torch.empty(0, 3, device="cuda")
    ws = torch.empty(tt.toktier_distill_workspace_bytes(0, 8, 3), dtype=torch.uint8, device="cuda")
    tt.toktier_distill(e, i, t, v, v, ws, grad_logits=e)
    tt.toktier_distill_backward(e, i, t, v, e)


def test_against_differences(tt):
    _say("distill differences")
    case = Case(30, 500, 16, F32, 1.5, own_lse=True, gaps=0.2)
    o = case.outputs()
    case.forward(tt, o)
    c = (case.grad_loss * case.scale).double()
    total = lambda x: float((case.reference(x)["loss"][0] * c).sum())
    for k in range(4):
        d = torch.randn(30, 500, generator=case.gen, device="cuda").double()
        eps = 1e-5
        slope = (total(case.logits.double() + eps * d) - total(case.logits.double() - eps * d)) / (2 * eps)
        own = o["grad"].double() * d
        assert abs(slope - float(own.sum())) <= 1e-5 * float(own.abs().sum()) + 1e-8, k


def test_more_rows_than_a_grid_holds_and_far_offsets(tt):
    _say("distill many rows")
    n, v = 70000, 40
    case = Case(n, v, 3, BF16)
    o = case.outputs()
    case.forward(tt, o)
    case.check(o, case.reference(), "many rows")
    case.backward(tt, o)
    case.check(o, case.reference(from_lse=True), "many rows later", ("grad",))
    del case, o
    n, v = 33000, 131328   # 4.3e9 elements
    x = torch.zeros(n, v, dtype=BF16, device="cuda")
    ids = torch.randint(0, v, (n, 2), dtype=torch.int32, device="cuda")
    top = torch.zeros(n, 2, device="cuda")
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    ws = torch.empty(tt.toktier_distill_workspace_bytes(n, v, 2), dtype=torch.uint8, device="cuda")
    tt.toktier_distill(x, ids, top, loss, lse, ws, grad_logits=x)
    assert torch.allclose(lse, torch.full_like(lse, math.log(v)), rtol=1e-5)
    two = ids[:, 0] != ids[:, 1]
    assert torch.allclose(loss[two], torch.full_like(loss[two], math.log(v / 2)), rtol=1e-5)
    for r in (0, n // 2, n - 1):
        row = x[r].float()
        at = ids[r].long().unique()
        assert torch.allclose(row[at], torch.full_like(row[at], -1.0 / at.numel()), rtol=2 ** -7)
        row[at] = 1.0 / v
        assert torch.allclose(row, torch.full_like(row, 1.0 / v), rtol=2 ** -7)


def test_streams_graphs_and_bits(tt):
    _say("distill graphs")
    cases = [Case(6, 70000, 40, BF16, seed=1), Case(50, 3000, 9, F16, own_lse=True, seed=2)]
    want = [c.outputs() for c in cases]
    for c, o in zip(cases, want):
        c.forward(tt, o)
    ws = torch.empty(max(c.workspace(tt).numel() for c in cases), dtype=torch.uint8, device="cuda")

    def call(c, o):
        tt.toktier_distill(c.logits, c.ids, c.top, o["loss"], o["lse"], ws, temperature=c.t, teacher_lse=c.teacher_lse, grad_logits=o["grad"],
                           grad_loss=c.grad_loss, grad_scale=c.scale)

    same = lambda a, b: all(torch.equal(a[k], b[k]) for k in ("loss", "lse", "grad"))
    outs, graphs = [c.outputs() for c in cases], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c, o in zip(cases, outs):
            call(c, o)
    side.synchronize()
    assert all(same(a, b) for a, b in zip(outs, want))
    for c, o in zip(cases, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(c, o)
        graphs.append(graph)
    for turn in range(4):
        for i in ((0, 1), (1, 0))[turn % 2]:
            for key in ("loss", "lse", "grad"):
                outs[i][key].fill_(9)
            ws.fill_(turn * 41)
            graphs[i].replay()
            torch.cuda.synchronize()
            assert same(outs[i], want[i]), (turn, i)
