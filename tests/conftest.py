import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA device (B200, sm_100a)")


# Host tests that pass made-up addresses to a call which is accepted: only the missing device keeps the kernel from
# running on them, so they do not run where there is one (a test marked gpu makes the same calls with real tensors).
ONLY_WITHOUT_A_DEVICE = {"test_rope_refuses_tensors_of_a_call_that_share_elements"}


def pytest_collection_modifyitems(config, items):
    # tests marked gpu cannot run without a device; skip them instead of failing
    try:
        import torch
        has_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        has_gpu = False
    if has_gpu:
        skip = pytest.mark.skip(reason="passes made-up addresses to a call that would be launched here")
        for it in items:
            if it.name in ONLY_WITHOUT_A_DEVICE:
                it.add_marker(skip)
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for it in items:
        if "gpu" in it.keywords:
            it.add_marker(skip)
