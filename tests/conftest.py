import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a)")


def pytest_collection_modifyitems(config, items):
    try:
        import torch
        has_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        has_gpu = False
    if has_gpu:
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for item in items:
        if "gpu" in item.keywords:
            item.add_marker(skip)


@pytest.fixture(autouse=True)
def argument_blocks_live_as_long_as_the_test(request, monkeypatch):
    """test_packed_calls_are_the_same_calls views an attention problem by its address after the only reference to it
    has gone; the allocator may by then have put its own pointer, or null, into the first field.  The problems that
    a test of that module makes are held until it ends."""
    if request.module.__name__.rpartition(".")[2] != "test_attn_side_host":
        return
    from quant_packed_gemv_gb300 import plm
    held = []

    class Held(plm._AttnProblem):
        def __init__(self, *args, **fields):
            super().__init__(*args, **fields)
            held.append(self)

    monkeypatch.setattr(plm, "_AttnProblem", Held)
