import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")
    config.addinivalue_line("markers", "slow: long-running CPU test")


def pytest_collectstart(collector):
    # One module under both names that tests import it by: its compiled kernels are made once.
    if "test_codegen" in sys.modules:
        sys.modules.setdefault("tests.test_codegen", sys.modules["test_codegen"])
