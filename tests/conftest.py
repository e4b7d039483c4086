import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a B200 (sm_100a) GPU and the built CUDA library")
    config.addinivalue_line("markers", "slow: full-size case, minutes on the CPU")


# Tests that hand valid calls addresses of no memory: they check what happens up to
# the device and count on there being none. On a GPU their kernels would launch on
# those addresses, so there they never run.
WITHOUT_DEVICE = ("test_quant_ops_cpu.py::test_lists_that_are_allowed_reach_the_device",)


def pytest_collection_modifyitems(config, items):
    # GPU tests cannot run without a device: report them as skipped instead
    # of failing when the suite runs on a CPU-only machine with -m gpu.
    try:
        import torch
        has_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        has_gpu = False
    if has_gpu:
        skip = pytest.mark.skip(reason="hands the library addresses of no memory: only without a CUDA device")
        for it in items:
            if any(name in it.nodeid for name in WITHOUT_DEVICE):
                it.add_marker(skip)
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for it in items:
        if "gpu" in it.keywords:
            it.add_marker(skip)


GOLDEN = os.path.join(os.path.dirname(os.path.abspath(__file__)), "golden")
