"""Cross entropy from wide hidden states on the GPU, with logits that are exact in 32 bits: every column takes part, and no
bound grows with the width."""
import pytest
import torch

import linear_exact as exact
import linear_plain as plain

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [BF16, F16, F32]


def _say(*a):
    print("[gpu-case]", *a, flush=True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,d,pad", [
    (20, 3000, 4096, 0), (50, 1256, 4096, 0), (100, 2000, 4096, 0),   # tiles for few rows
    (300, 2500, 4096, 0), (700, 9000, 4096, 0),
    (1700, 8200, 4096, 0),                                            # the largest tiles
    (90, 3000, 4095, 1), (300, 5000, 4097, 0),                        # copied tables
    (300, 300, 16384, 0), (5, 70, 65536, 0), (130, 500, 65536, 0), (33, 700, 65535, 1)])
def test_wide_rows(tt, n, v, d, pad, dtype):
    _say("linear wide", n, v, d, pad, dtype)
    h, w, y, c = exact.inputs(n, v, d, dtype, "cuda", ignored=0.1 if n > 5 else 0.0)
    wide = torch.full((v, d + pad), float("nan"), dtype=dtype, device="cuda")
    wide[:, :d] = w
    scale = 1024.0 if dtype == F16 else 1.0    # a power of two
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    gh, gw = torch.empty_like(h), torch.empty_like(w)
    size = tt.toktier_linear_cross_entropy_workspace_bytes(n, v, d, dtype)
    ws = torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")
    for later in (False, True):
        gh.fill_(3), gw.fill_(5)
        grads = dict(grad_hidden=gh, grad_weight=gw, grad_loss=c, grad_scale=scale)
        if later:
            tt.toktier_linear_cross_entropy_backward(h, wide[:, :d], y, lse, ws.fill_(0x5A), **grads)
        else:
            tt.toktier_linear_cross_entropy(h, wide[:, :d], y, loss, lse, ws, **grads)
        ref = exact.reference(h, w, y, c * scale, dtype, later)
        for key, got in (("loss", loss), ("lse", lse), ("gh", gh), ("gw", gw)):
            plain.close(got, *ref[key], f"wide {key}" + (" later" if later else ""))
        exact.reject_wrong(h, w, y, c * scale, ref)
