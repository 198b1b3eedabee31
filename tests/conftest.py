import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
for p in (ROOT, os.path.join(ROOT, "tests")):
    if p not in sys.path:
        sys.path.insert(0, p)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU; runs through the C ABI")
    config.addinivalue_line("markers", "slow: full-size CPU checks")


@pytest.fixture(scope="session")
def tt():
    """The package, with its library loaded, on a GPU."""
    import torch

    import exact_bpe_tokenization_amd as package
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    package.lib()
    return package
