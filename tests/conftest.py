import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")
    config.addinivalue_line("markers", "slow: full-size workload (seconds to minutes)")


# Tests that hold a wrong value: they stay as they are, and their failing is what is expected.
WRONG = {
    "test_gpu_kv_attention.py::test_lengths_past_the_table":
        "two queries of a sequence of 70 keys stand at 68 and 69 and see all 64 keys of the table (include/kvcache.h); the test wants "
        "what two queries at 62 and 63 see, the first of them not key 63.  test_gpu_kv_attention_positions.py has the right values",
}


def pytest_collection_modifyitems(items):
    for item in items:
        for name, reason in WRONG.items():
            if item.nodeid.endswith(name):
                item.add_marker(pytest.mark.xfail(reason=reason, strict=True))
