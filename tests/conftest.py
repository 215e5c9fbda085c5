import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
HERE = os.path.dirname(os.path.abspath(__file__))
if HERE not in sys.path:
    sys.path.insert(0, HERE)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")


@pytest.fixture(autouse=True)
def no_give_up_left(request):
    """A give-up that a test provokes and does not ask for is not left for the next test to find: those of the gated
    recurrence are reported to the first query on the GPU."""
    yield
    if request.node.get_closest_marker("gpu"):
        import primitives_device_scan_amd as ds

        ds.query_timeout()
