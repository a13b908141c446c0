import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU")
    config.addinivalue_line("markers", "slow: long-running CPU test")


# This test asks for y = 0 from the norm of a row whose 64 values (or more) are all 3.0e38:
# mean h^2 = 9e76, y = 3e38 / sqrt(9e76 + eps) = 1.  Its zero was the overflow of an
# fp32 sum.  The same rows and all its other checks are in
# test_gpu_norm_range.py::test_bad_rows_stay_alone_beside_the_largest.
HOLDS_A_WRONG_VALUE = "test_gpu_rms_norm.py::test_bad_rows_stay_alone["


def pytest_collection_modifyitems(items):
    for item in items:
        if HOLDS_A_WRONG_VALUE in item.nodeid:
            item.add_marker(pytest.mark.xfail(strict=True, raises=AssertionError,
                                              reason="asks for y = 0 where the formula gives 1"))
