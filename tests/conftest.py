import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

GOLDEN = os.path.join(ROOT, "tests", "golden")


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")
    config.addinivalue_line("markers", "slow: CPU test that takes more than a few seconds")


@pytest.fixture(scope="session", autouse=True)
def _vector_math_initialised():
    """torch's float64 logarithm and exponential on several threads at their very first use were
    off by 1e-10 in about one process of ten; once one thread has used them they are not."""
    import torch
    torch.logsumexp(torch.zeros(2, 3, 45, 45, dtype=torch.float64), -1)


def require_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
