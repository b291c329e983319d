import ctypes
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    # the parity tests compare caches of gigabytes: large temporaries stay on the heap instead of being mapped and
    # faulted in anew each time (glibc's M_MMAP_MAX and M_TRIM_THRESHOLD; a sixth of the GPU suite's time)
    mallopt = getattr(ctypes.CDLL(None), "mallopt", None)
    if mallopt is not None:
        mallopt(-4, 0)
        mallopt(-1, 2**31 - 1)
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (runs the CUDA library through its C ABI)")


@pytest.fixture(scope="session")
def orc():
    import oracle

    oracle.lib()
    return oracle
