import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (runs through the HIP library)")
    config.addinivalue_line("markers", "slow: long CPU test")


@pytest.fixture(autouse=True)
def _torch_seed(request):
    """torch seeds its GPU generator differently in every process: tests that
    draw from it get the same inputs in every run, whatever ran before them."""
    if request.node.get_closest_marker("gpu"):
        import torch

        torch.manual_seed(0)
