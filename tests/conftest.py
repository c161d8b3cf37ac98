import ctypes
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a)")
    config.addinivalue_line("markers", "slow: long-running CPU case")


@pytest.fixture(scope="session")
def cuda_device():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


@pytest.fixture(autouse=True)
def addressed_objects_live(request, monkeypatch):
    """What test_cache_refusals.py takes the address of lives until the test ends: its helpers address temporaries, and
    whether a freed structure's first field then reads as NULL depends on what else the heap holds.  No other test is
    given this, so that none hides an address that outlives its object."""
    if request.module.__name__ != "test_cache_refusals":
        return
    address, kept = ctypes.addressof, []
    monkeypatch.setattr(ctypes, "addressof", lambda x: (kept.append(x), address(x))[1])
