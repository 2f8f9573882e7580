import gc
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built libpadoc")
    config.addinivalue_line("markers", "slow: long CPU test")


def _gpu_available():
    try:
        import torch
        return torch.cuda.is_available()
    except Exception:
        return False


def pytest_collection_modifyitems(config, items):
    if _gpu_available():
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for item in items:
        if "gpu" in item.keywords:
            item.add_marker(skip)


@pytest.fixture(scope="session")
def padoc_lib():
    """Builds (if stale) and loads libpadoc.so."""
    from tree_structured_shared_gb300 import build, padoc
    build.build()
    return padoc.lib()


@pytest.fixture(autouse=True)
def _collected_before(request):
    """Pools of earlier tests are collected now: freeing their block tables while
    a test captures a graph would end the capture."""
    if "gpu" in request.keywords:
        gc.collect()
