import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")


def pytest_collection_modifyitems(items):
    # This test asserts the placement of launches that begin on XCD 0, as those of a process's first
    # queue do until further queues (streams) are made, which other tests do: it goes first.
    items.sort(key=lambda i: i.name != "test_remap_places_contiguous_tasks_on_one_xcd")


@pytest.fixture(scope="session")
def orc():
    import oracle
    oracle.lib()
    return oracle
