"""Cross entropy from hidden states without a GPU: refusals before any device call, workspace sizes, and that the bounds of
the GPU tests reject wrong gradients."""
import ctypes

import numpy as np
import pytest
import torch

import exact_bpe_tokenization_amd as tt
import linear_plain as plain

INVALID, CAPACITY, HIP = 1, 5, 6
BUF = np.zeros(1 << 22, dtype=np.uint8)
BASE = (BUF.ctypes.data + 255) & ~255


def at(offset):
    return ctypes.c_void_p(BASE + offset)


SIZE = tt.toktier_linear_cross_entropy_workspace_bytes(4, 10, 8, torch.bfloat16)
FORWARD = dict(hidden=at(0), type=3, n_rows=4, dim=8, hidden_stride=8, weight=at(4096), n_vocab=10, weight_stride=8, targets=at(8192),
               loss=at(8448), lse=at(8704), grad_loss=at(8960), grad_scale=1.0, grad_hidden=at(12288), grad_hidden_stride=8,
               grad_weight=at(16384), grad_weight_type=1, grad_weight_stride=8, accumulate=0, workspace=at(65536), workspace_bytes=SIZE,
               stream=None)
BACKWARD = {k: v for k, v in FORWARD.items() if k != "loss"}
BOTH = [dict(hidden=None), dict(weight=None), dict(targets=None), dict(lse=None), dict(workspace=None), dict(workspace=at(65537)),
        dict(type=0), dict(type=4), dict(dim=0), dict(dim=(1 << 16) + 1), dict(n_vocab=0), dict(n_vocab=(1 << 21) + 1),
        dict(n_rows=(1 << 20) + 1), dict(hidden_stride=7), dict(weight_stride=7), dict(grad_hidden_stride=7), dict(grad_weight_stride=7),
        dict(hidden=at(1)), dict(weight=at(4097)), dict(targets=at(8193)), dict(lse=at(8706)), dict(grad_loss=at(8961)),
        dict(grad_hidden=at(12289)), dict(grad_weight=at(16386)), dict(grad_weight_type=2), dict(grad_weight_type=0),
        dict(hidden_stride=1 << 62), dict(weight_stride=1 << 62), dict(grad_hidden_stride=1 << 62), dict(grad_weight_stride=1 << 62),
        dict(grad_hidden=at(0)), dict(grad_hidden=at(4096)), dict(grad_weight=at(4096)), dict(grad_weight=at(32)),
        dict(grad_hidden=at(16400)), dict(grad_hidden=at(8192)), dict(grad_weight=at(8704)), dict(grad_weight=at(8960)),
        dict(workspace=at(0)), dict(workspace=at(4096)), dict(workspace=at(8192)), dict(workspace=at(16384)), dict(grad_hidden=at(65536))]


def call(name, base, **changes):
    return getattr(tt.lib(), name)(*{**base, **changes}.values())


def _name(c):
    return ",".join(f"{k}={(v.value or 0) - BASE if isinstance(v, ctypes.c_void_p) else v}" for k, v in c.items())


@pytest.mark.parametrize("change", BOTH + [dict(loss=None), dict(loss=at(8449)), dict(loss=at(0)), dict(lse=at(8192)), dict(loss=at(8704)),
                                           dict(loss=at(65536))], ids=_name)
def test_refusals(change):
    assert call("toktier_linear_cross_entropy", FORWARD, **change) == INVALID


@pytest.mark.parametrize("change", BOTH, ids=_name)
def test_refusals_backward(change):
    assert call("toktier_linear_cross_entropy_backward", BACKWARD, **change) == INVALID


def test_capacity_and_nothing_to_do():
    for name, base in (("toktier_linear_cross_entropy", FORWARD), ("toktier_linear_cross_entropy_backward", BACKWARD)):
        assert call(name, base, workspace_bytes=SIZE - 1) == CAPACITY
        assert call(name, base, workspace_bytes=0) == CAPACITY
        empty = dict(n_rows=0, hidden=None, targets=None, lse=None, grad_loss=None, grad_hidden=None)
        assert call(name, base, **empty, accumulate=1) == 0
        assert call(name, base, **empty, grad_weight=None) == 0
        if not torch.cuda.is_available():
            assert call(name, base) == HIP
            assert tt.lib().toktier_last_hip_error() != b""
            assert call(name, base, **empty) == HIP   # zeros to write
    small = tt.toktier_linear_cross_entropy_workspace_bytes(4, 10, 8, torch.bfloat16, False)
    if not torch.cuda.is_available():
        assert call("toktier_linear_cross_entropy", FORWARD, grad_hidden=None, grad_weight=None, workspace_bytes=small) == HIP


def test_binding_refuses_tensors_of_another_kind():
    x, i, v = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    ws = torch.zeros(4096, dtype=torch.uint8)
    for f in (lambda: tt.toktier_linear_cross_entropy(x, x, i, v, v, ws), lambda: tt.toktier_linear_cross_entropy_backward(x, x, i, v, ws)):
        with pytest.raises(tt.ToktierError) as e:
            f()
        assert e.value.status == INVALID
    with pytest.raises(tt.ToktierError):
        tt.toktier_linear_cross_entropy_workspace_bytes(4, 10, 8, torch.float64)


ROWS = [0, 1, 255, 256, 257, 1500, 2048, 4096, 8192, 1 << 16, 1 << 20]
VOCABS = [1, 256, 257, 1256, 33001, 33024, 131328, 1 << 21]
DIMS = [1, 63, 64, 65, 320, 1001, 2048, 4096, 1 << 16]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("grads", [False, True])
def test_sizes_never_fall(dtype, grads):
    f = lambda n, v, d: tt.toktier_linear_cross_entropy_workspace_bytes(n, v, d, dtype, grads)
    size = {(n, v, d): f(n, v, d) for n in ROWS for v in VOCABS for d in DIMS}
    for (n, v, d), s in size.items():
        assert s % 256 == 0 and s >= 256
        if not grads:
            assert s <= tt.toktier_linear_cross_entropy_workspace_bytes(n, v, d, dtype, True)
    for seq, key in ((ROWS, lambda a, b, c: (a, b, c)), (VOCABS, lambda a, b, c: (b, a, c)), (DIMS, lambda a, b, c: (b, c, a))):
        others = [s for s in (ROWS, VOCABS, DIMS) if s is not seq]
        for x in others[0]:
            for y in others[1]:
                line = [size[key(a, x, y)] for a in seq]
                assert line == sorted(line), (x, y)


def test_workspace_is_much_smaller_than_kept_logits():
    n, v, d = 1 << 16, 131328, 4096
    assert tt.toktier_linear_cross_entropy_workspace_bytes(n, v, d, torch.bfloat16) < n * v * 2 / 4


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_bounds_reject_wrong_gradients(dtype):
    """Gradients that are zero, a twentieth off (bfloat16; a hundredth in the others), of the wrong row or without the target's
    part lie outside the bounds; the formula's, rounded, lie inside."""
    g = torch.Generator().manual_seed(3)
    n, v, d = 50, 400, 64
    w = (torch.randn(v, d, generator=g) * 0.3).to(dtype)
    y = torch.randint(0, v, (n,), generator=g, dtype=torch.int32)
    h = (torch.randn(n, d, generator=g) + w[y.long()].float()).to(dtype)
    loss, lse, hh, x, kept, t = plain.losses(h, w, y)
    c = torch.full((n,), 1.0)
    gr, gh, gw = plain.gradients(hh, w, x, lse, kept, t, c)
    e_loss, e_lse, e_h, e_w = plain.bounds(hh, w, x, lse, kept, t, c, gr, dtype, False)
    e_w = e_w + plain.rounding(gw, dtype)
    share = 0.05 if dtype == torch.bfloat16 else 0.01
    for ref, err in ((gh, e_h), (gw, e_w)):
        plain.close(ref.to(dtype), ref, err, "rounded")
        for wrong in (torch.zeros_like(ref), ref * (1 + share), ref.roll(1, 0)):
            off = (wrong - ref).abs() > err
            assert float(off.double().mean()) > 0.5
    untouched = gr + torch.zeros_like(gr).scatter_(1, t, 1.0)
    assert float(((torch.mm(untouched, w.double()) - gh).abs() > e_h).double().mean()) > 0.9
    assert float(e_loss.max()) < 1e-3 and float(e_lse.max()) < 1e-3
