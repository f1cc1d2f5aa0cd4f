import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a B200 (sm_100a) GPU")
    config.addinivalue_line("markers", "slow: full-size workloads")


# Expectations that do not hold, by the formula.  The tests stay as they are and run.
NOT_SO = {
    f"test_gpu_cache.py::test_nan_behind_the_causal_mask_of_a_few_rows[vs-{t}]":
        "expects NaN weights from a NaN value scale: weights are softmax(Q K^T), which V does not enter"
    for t in ("i8", "e4m3")
}


def pytest_collection_modifyitems(items):
    for item in items:
        for name, why in NOT_SO.items():
            if item.nodeid.endswith(name):
                item.add_marker(pytest.mark.xfail(reason=why, strict=True, raises=AssertionError))
