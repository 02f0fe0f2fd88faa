import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


LAUNCHES_ON_A_GPU = ("test_ops_abi.py::test_attn_range_of_scale[2e-30-None]",)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU")
    config.addinivalue_line("markers", "slow: takes more than a few seconds")


def pytest_collection_modifyitems(config, items):
    # A test marked gpu must never be silently satisfied by a CPU path: when no
    # GPU is visible it is skipped with a reason, never run.
    try:
        import torch
        have_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        have_gpu = False
    if have_gpu:
        # Calls that the C ABI accepts, on addresses that are no memory: without a
        # GPU they end at the device check, with one they would be launched.
        for it in items:
            if any(it.nodeid.endswith(n) for n in LAUNCHES_ON_A_GPU):
                it.add_marker(pytest.mark.skip(reason="a GPU is visible, and its addresses are no memory"))
        return
    skip = pytest.mark.skip(reason="no GPU visible")
    for it in items:
        if "gpu" in it.keywords:
            it.add_marker(skip)
