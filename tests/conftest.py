import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")
    config.addinivalue_line("markers", "slow: oracle runs that take tens of seconds")


def pytest_collection_modifyitems(config, items):
    # GPU tests need a GPU; report them as skipped (not passed) where none is present.
    try:
        import torch
        have_gpu = torch.cuda.is_available()
    except Exception:
        have_gpu = False
    if have_gpu:
        return
    skip = pytest.mark.skip(reason="no CUDA GPU on this machine")
    for item in items:
        if "gpu" in item.keywords:
            item.add_marker(skip)


@pytest.fixture(autouse=True)
def latent_attention_record(request):
    """The latent attention's GPU tests each start with an empty device error record, so that what one expects is its own, and none may end
    with a wait that ran out; the other errors of a test are the test's to read."""
    if not request.module.__name__.startswith("test_gpu_mla") or "gpu" not in request.node.keywords:
        yield
        return
    from gpu_util import lib
    ql = lib()

    def message():
        try:
            ql.ql_check_device_error()
        except ql.QLError as e:
            return str(e)
        return ""
    message()
    yield
    left = message()
    assert "did not arrive" not in left, left
