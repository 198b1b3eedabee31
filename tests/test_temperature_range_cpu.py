"""Which temperatures distillation and the top logits take, without a GPU."""
import pytest
import torch

import test_distill_cpu as distill

CALLS = [(name, base) for name, base, _ in distill.CASES]


@pytest.mark.parametrize("name,base", CALLS, ids=[c[0] for c in CALLS])
@pytest.mark.parametrize("t", [2.95e-39, 3.5e-39, 4.2e-39, 1e-45, 0.0, -0.0, -1e38, float("inf"), float("nan")])
def test_refused(t, name, base):
    """Among them those whose reciprocal is finite, but not log2(e) / t, which every power is taken with."""
    assert distill.call(name, base, temperature=t) == distill.INVALID


@pytest.mark.parametrize("name,base", CALLS, ids=[c[0] for c in CALLS])
@pytest.mark.parametrize("t", [4.3e-39, 1.2e-38, 1.0, 2.0 ** 120, 3.4e38])
def test_taken(t, name, base):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the calls would touch their addresses")
    assert distill.call(name, base, temperature=t) == distill.HIP
