import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")
    config.addinivalue_line("markers", "slow: long-running oracle comparison")


def pytest_collection_modifyitems(config, items):
    have_gpu = False
    try:
        import torch

        have_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        pass
    if have_gpu:
        # calls with such addresses are refused, or end at the check of the GPU where there is none
        skip = pytest.mark.skip(reason="passes addresses of no memory: only where there is no CUDA device")
        for it in items:
            if "gpu" not in it.keywords and hasattr(getattr(it, "module", None), "FAKE"):
                it.add_marker(skip)
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for it in items:
        if "gpu" in it.keywords:
            it.add_marker(skip)
