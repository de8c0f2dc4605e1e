import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU")


def pytest_collection_modifyitems(items):
    """Tests that call the library with made-up device addresses (modules with
    a FAKE one) stop at the device check where there is no GPU; on a GPU a
    call that passes the host checks would launch a kernel on them."""
    import torch
    if torch.cuda.device_count() == 0:
        return
    skip = pytest.mark.skip(reason="made-up device addresses: only where no GPU is visible")
    for item in items:
        if hasattr(getattr(item, "module", None), "FAKE") and not item.get_closest_marker("gpu"):
            item.add_marker(skip)
