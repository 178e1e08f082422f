import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a)")
    config.addinivalue_line("markers", "slow: full-size workloads")


@pytest.fixture(scope="module", autouse=True)
def _no_wait_gave_up(request):
    """After each module of GPU tests: no bounded wait inside a kernel has run out unnoticed
    (a test that makes one run out clears the count)."""
    yield
    marks = getattr(request.module, "pytestmark", None)
    if getattr(marks, "name", None) != "gpu":
        return
    import torch
    if torch.cuda.is_available():
        import paged_kv_cache_305_gb300 as pa
        assert pa.wait_timeout_count() == 0
