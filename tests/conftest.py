"""Test configuration: the ``gpu`` marker and shared helpers.

``-m "not gpu"`` runs the oracle's pins, the generators and the host-side
checks of the C-ABI library (it loads and exports its symbols; argument
validation that returns before any CUDA call).  ``-m gpu`` runs the parity
tests of the CUDA path against the oracle through the C-ABI.
"""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a)")


def pytest_collection_modifyitems(config, items):
    # GPU tests fail loudly (not skip) when no GPU is present and they were selected.
    pass


# Host-side tests that hand made-up addresses to several entry points at once, of
# which one refuses and the others would launch: only where there is no GPU to
# launch on (with one, CUDA_VISIBLE_DEVICES= hides it).
WITHOUT_GPU = {"test_cache_entry_points_refuse"}


def pytest_runtest_setup(item):
    if getattr(item, "originalname", item.name) in WITHOUT_GPU and gpu_available():
        pytest.skip("made-up addresses: run it without a GPU")


def gpu_available() -> bool:
    try:
        import torch
        return torch.cuda.is_available()
    except Exception:
        return False
