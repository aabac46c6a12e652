import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")


@pytest.fixture
def monkeypatch(monkeypatch):
    """pytest's own; a GS_RECURRENCE_PATIENCE that a test sets goes to the library's entry for
    tests (the library itself reads no environment): polls that a recurrence call waits, 0 for
    the way without waiting."""
    from gaussian_splatting_tile_amd import _lib
    setenv, delenv, changed = monkeypatch.setenv, monkeypatch.delenv, []

    def patience(name, polls):
        if name == "GS_RECURRENCE_PATIENCE":
            polls = int(polls)
            changed.append(name)
            _lib.load().gs_test_recurrence_patience(polls)

    monkeypatch.setenv = lambda name, value, *a, **kw: (setenv(name, value, *a, **kw), patience(name, value))[0]
    monkeypatch.delenv = lambda name, *a, **kw: (delenv(name, *a, **kw), patience(name, -1))[0]
    yield monkeypatch
    if changed:
        _lib.load().gs_test_recurrence_patience(-1)


@pytest.fixture(scope="session")
def orc():
    import oracle
    oracle.lib()
    return oracle
