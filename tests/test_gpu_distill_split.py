"""Distillation where rows begin or cease to be split over several workgroups: rows and IDs around the borders, of every type."""
import pytest
import torch

from test_gpu_distill import TYPES, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v", [(64, 65536), (65, 65537), (128, 65537), (129, 65536), (64, 65535), (65, 262143), (129, 262145), (66, 524289),
                                 (160, 524288)])
def test_around_the_borders(tt, n, v, dtype):
    print("[gpu-case]", "distill split", n, v, dtype, flush=True)
    case = Case(n, v, 20, dtype, 1.5, gaps=0.1)
    o = case.outputs()
    case.forward(tt, o)
    case.check(o, case.reference(), "one call")
    alone = case.outputs()
    case.forward(tt, alone, grad=False)
    assert torch.equal(alone["loss"], o["loss"]) and torch.equal(alone["lse"], o["lse"])
    later = case.outputs()
    later["lse"] = o["lse"]
    case.backward(tt, later)
    case.check(later, case.reference(from_lse=True), "later", ("grad",))
