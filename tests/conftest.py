import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
TESTS = os.path.dirname(os.path.abspath(__file__))
if TESTS not in sys.path:
    sys.path.insert(0, TESTS)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA device (B200, sm_100a)")


# Tests that compare memory which nothing has written (rows past a sequence's end) before and
# after a call: a NaN that an earlier test left there would not equal itself.
_READS_FRESH_MEMORY = {"test_append_and_read_bad_ranges_are_reported"}


@pytest.fixture(autouse=True)
def _numbers_in_recycled_memory(request):
    """Zeros in every free small block of the allocator before such a test."""
    if request.node.name in _READS_FRESH_MEMORY:
        import torch

        torch.cuda.synchronize()
        held, reserved = [], torch.cuda.memory_reserved()
        while torch.cuda.memory_reserved() == reserved and len(held) < 100_000:
            held.append(torch.zeros(512, dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
        del held
    yield
