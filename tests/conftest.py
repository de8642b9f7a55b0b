import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA device (B200) and the built CUDA library")
    config.addinivalue_line("markers", "slow: long-running case")


# Tests that hand made-up device addresses to a call which refuses nothing about them: they count on the call
# ending for want of a GPU, and on a machine with one it would launch kernels on those addresses.
MADE_UP_ADDRESSES = {("test_capi_cpu.py", "test_format_flags_are_validated"),
                     ("test_training_capi_cpu.py", "test_neighbouring_buffers_and_shared_gradients_are_not_refused")}


def pytest_collection_modifyitems(config, items):
    # Without a GPU, skip gpu-marked tests loudly instead of failing at import time.
    try:
        import torch
        has_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        has_gpu = False
    if has_gpu:
        skip = pytest.mark.skip(reason="made-up device addresses: runs only where there is no GPU")
        for item in items:
            if (item.path.name, getattr(item, "originalname", item.name)) in MADE_UP_ADDRESSES:
                item.add_marker(skip)
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for item in items:
        if "gpu" in item.keywords:
            item.add_marker(skip)
