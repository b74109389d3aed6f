import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU; runs the HIP library")
    config.addinivalue_line("markers", "slow: longer CPU-side check")


@pytest.fixture(scope="session")
def oracle_lib():
    import oracle

    return oracle.lib()


@pytest.fixture(scope="session", autouse=True)
def built():
    """The library and the wrappers' tensor reader, built if either is missing."""
    from sparse_moe_02_amd import _build

    if not _build.built():
        import __graft_entry__

        __graft_entry__.build()
