"""Distillation and top logits without a GPU: refusals before any device call, workspace sizes, and that the bounds of the
GPU tests reject wrong gradients."""
import ctypes

import numpy as np
import pytest
import torch

import distill_plain as plain
import exact_bpe_tokenization_amd as tt
from linear_plain import close

INVALID, CAPACITY, HIP = 1, 5, 6
BUF = np.zeros(1 << 20, dtype=np.uint8)
BASE = (BUF.ctypes.data + 255) & ~255


def at(offset):
    return ctypes.c_void_p(BASE + offset)


DISTILL = dict(logits=at(0), type=3, n_rows=4, n_vocab=10, stride=16, top_ids=at(4096), top_ids_stride=3, top_logits=at(8192),
               top_logits_stride=4, top_k=3, teacher_lse=at(12288), temperature=1.0, loss=at(16384), lse=at(16640), grad_loss=at(16896),
               grad_scale=1.0, grad=at(20480), grad_stride=10, workspace=at(65536), workspace_bytes=1 << 16, stream=None)
BACKWARD = {k: v for k, v in DISTILL.items() if k not in ("loss", "workspace", "workspace_bytes")}
TOP = dict(logits=at(0), type=3, n_rows=4, n_vocab=10, stride=16, k=3, temperature=1.0, out_ids=at(4096), out_ids_stride=3,
           out_logits=at(8192), out_logits_stride=4, lse=at(12288), workspace=at(65536), workspace_bytes=1 << 16, stream=None)
NAN, INF = float("nan"), float("inf")
SHARED = [dict(logits=None), dict(type=0), dict(type=4), dict(n_vocab=0), dict(n_vocab=(1 << 21) + 1), dict(n_rows=1 << 31), dict(stride=9),
          dict(logits=at(1)), dict(stride=1 << 62), dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=NAN), dict(temperature=INF),
          dict(temperature=1e-39)]
BOTH = SHARED + [dict(top_ids=None), dict(top_logits=None), dict(lse=None), dict(top_k=0), dict(top_k=1025), dict(top_ids_stride=2),
                 dict(top_logits_stride=2), dict(top_ids=at(4097)), dict(top_logits=at(8194)), dict(teacher_lse=at(12289)), dict(lse=at(16642)),
                 dict(grad_loss=at(16897)), dict(grad=at(20481)), dict(grad_stride=9), dict(grad_stride=1 << 62), dict(top_ids_stride=1 << 62),
                 dict(grad=at(0)), dict(grad=at(32), grad_stride=16), dict(grad=at(4096)), dict(grad=at(8192)), dict(grad=at(12288)),
                 dict(grad=at(16640)), dict(grad=at(16896))]
CASES = [("toktier_distill", DISTILL, BOTH + [
            dict(loss=None), dict(loss=at(16386)), dict(workspace=None), dict(workspace=at(65540)), dict(loss=at(0)), dict(lse=at(16384)),
            dict(loss=at(4096)), dict(loss=at(8192)), dict(lse=at(12288)), dict(loss=at(16896)), dict(loss=at(20480)), dict(workspace=at(0)),
            dict(workspace=at(4096)), dict(workspace=at(16384)), dict(workspace=at(20480))]),
         ("toktier_distill_backward", BACKWARD, BOTH + [dict(grad=None)]),
         ("toktier_top_logits", TOP, SHARED + [
            dict(out_ids=None), dict(out_logits=None), dict(k=0), dict(k=1025), dict(out_ids_stride=2), dict(out_logits_stride=2),
            dict(out_ids=at(4097)), dict(out_logits=at(8193)), dict(lse=at(12290)), dict(workspace=None), dict(workspace=at(65540)),
            dict(out_ids=at(0)), dict(out_logits=at(4)), dict(lse=at(16)), dict(out_logits=at(4096)), dict(lse=at(4096)), dict(lse=at(8192)),
            dict(workspace=at(0)), dict(workspace=at(4096)), dict(workspace=at(8192)), dict(workspace=at(12288))])]


def call(name, base, **changes):
    return getattr(tt.lib(), name)(*{**base, **changes}.values())


def _name(c):
    return ",".join(f"{k}={(v.value or 0) - BASE if isinstance(v, ctypes.c_void_p) else v}" for k, v in c.items())


@pytest.mark.parametrize("name,base,change", [pytest.param(n, b, c, id=f"{n}-{_name(c)}") for n, b, cs in CASES for c in cs])
def test_refusals(name, base, change):
    assert call(name, base, **change) == INVALID


def test_capacity_nothing_to_do_and_no_device():
    empty = dict(n_rows=0, logits=None, lse=None)
    assert call("toktier_distill", DISTILL, **empty, top_ids=None, top_logits=None, loss=None, grad=None) == 0
    assert call("toktier_distill_backward", BACKWARD, **empty, top_ids=None, top_logits=None) == 0
    assert call("toktier_top_logits", TOP, **empty, out_ids=None, out_logits=None) == 0
    for name, base in (("toktier_distill", DISTILL), ("toktier_top_logits", TOP)):
        assert call(name, base, workspace_bytes=255) == CAPACITY
    if not torch.cuda.is_available():
        for name, base, _ in CASES:
            assert call(name, base) == HIP
            assert tt.lib().toktier_last_hip_error() != b""
        assert call("toktier_distill", DISTILL, grad=at(0), grad_stride=16) == HIP   # in place
        assert call("toktier_distill", DISTILL, teacher_lse=None, grad_loss=None, grad=None) == HIP
        assert call("toktier_top_logits", TOP, lse=None) == HIP


def test_binding_refuses_tensors_of_another_kind():
    x, i, v, t = torch.zeros(4, 8), torch.zeros(4, 3, dtype=torch.int32), torch.zeros(4), torch.zeros(4, 3)
    ws = torch.zeros(4096, dtype=torch.uint8)
    for f in (lambda: tt.toktier_distill(x, i, t, v, v, ws), lambda: tt.toktier_distill_backward(x, i, t, v, x),
              lambda: tt.toktier_top_logits(x, i, t, ws)):
        with pytest.raises(tt.ToktierError) as e:
            f()
        assert e.value.status == INVALID


ROWS = [0, 1, 2, 63, 64, 65, 128, 158, 159, 160, 8192, (1 << 31) - 1]
VOCABS = [1, 1256, 65535, 65536, 65537, 131328, 1 << 21]
KS = [1, 8, 20, 120, 121, 300, 1024]


@pytest.mark.parametrize("f", [tt.toktier_distill_workspace_bytes, tt.toktier_top_logits_workspace_bytes])
def test_sizes_never_fall_and_hold_every_smaller_call(f):
    size = {(n, v, k): f(n, v, k) for n in ROWS for v in VOCABS for k in KS}
    for v in VOCABS:
        for k in KS:
            line = [size[n, v, k] for n in ROWS]
            assert line == sorted(line) and line[0] >= 256
    for n in ROWS:
        for k in KS:
            line = [size[n, v, k] for v in VOCABS]
            assert line == sorted(line)
        for v in VOCABS:
            line = [size[n, v, k] for k in KS]
            assert line == sorted(line)
    for bad in ((1, 0, 3), (1, (1 << 21) + 1, 3), (1, 8, 0), (1, 8, 1025), (1 << 31, 8, 3)):
        with pytest.raises(tt.ToktierError):
            f(*bad)


def _area(i):   # addresses 4 TiB apart: no argument lies on another
    return ctypes.c_void_p((i + 1) << 42)


@pytest.mark.parametrize("n,v,k", [(64, 131328, 20), (159, 1 << 21, 1024), (8192, 131328, 300), (60, 70000, 1024)])
def test_a_workspace_for_the_largest_call_is_enough(n, v, k):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the calls would touch their addresses")
    for name, sizes, args in (
            ("toktier_distill", tt.toktier_distill_workspace_bytes,
             lambda n, v, k, s: (_area(0), 3, n, v, v, _area(1), k, _area(2), k, k, None, 1.0, _area(3), _area(4), None, 1.0, None, 0, _area(5), s, None)),
            ("toktier_top_logits", tt.toktier_top_logits_workspace_bytes,
             lambda n, v, k, s: (_area(0), 3, n, v, v, k, 1.0, _area(1), k, _area(2), k, None, _area(3), s, None))):
        given = sizes(n, v, k)
        for a in [r for r in ROWS if 0 < r <= n] + [n]:
            for b in [x for x in VOCABS if x <= v] + [v]:
                for c in [x for x in KS if x <= k] + [k]:
                    assert getattr(tt.lib(), name)(*args(a, b, c, given)) == HIP, (name, a, b, c)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_bounds_reject_wrong_gradients(dtype):
    g = torch.Generator().manual_seed(1)
    n, v, k = 20, 300, 12
    x = (2.5 * torch.randn(n, v, generator=g)).to(dtype).double()
    top, ids = torch.topk(x + torch.randn(n, v, generator=g).double(), k, dim=1)
    c = torch.full((n,), 1.0, dtype=torch.float64)
    for from_lse in (False, True):
        r = plain.distill(x, ids.to(torch.int32), top, 1.5, None, c, dtype, from_lse)
        ref, err = r["grad"]
        close(ref.to(dtype), ref, err, "rounded")
        share = 0.02 if dtype == torch.bfloat16 else 0.005
        for wrong in (torch.zeros_like(ref), ref * (1 + share), ref.roll(1, 1)):
            assert float(((wrong - ref).abs() > err).double().mean()) > 0.8
        hot = torch.zeros_like(ref).scatter_(1, ids, 1.0) > 0
        unlisted = ref.clone()
        unlisted[hot] = 0.0
        assert bool(((unlisted - ref).abs() > err)[hot].all())
        assert float((r["loss"][1] / r["loss"][0].abs()).max()) < 1e-4 and float(r["lse"][1].max()) < 1e-4
