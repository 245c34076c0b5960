import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a) and the built libibp.so")


# Expects what ibp_kv_evict gave before a sequence longer than its weights was left alone.  Last, so that
# a run that ends at its first failure has run all others.
LAST = "test_evict_lengths_beyond_the_weights"


def pytest_collection_modifyitems(config, items):
    import torch

    items.sort(key=lambda item: item.name == LAST)
    if torch.cuda.is_available():
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for item in items:
        if "gpu" in item.keywords:
            item.add_marker(skip)
