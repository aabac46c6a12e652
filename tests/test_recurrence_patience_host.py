"""How long a recurrence call waits is no business of the environment; tests set it through an
entry of the library that gs.h does not declare. Needs no GPU."""
import os

USUAL = 1 << 14


def _now():
    from gaussian_splatting_tile_amd import _lib
    lib = _lib.load()
    polls = lib.gs_test_recurrence_patience(-1)
    lib.gs_test_recurrence_patience(polls)
    return polls


def test_monkeypatch_reaches_the_entry(monkeypatch):
    assert _now() == USUAL
    monkeypatch.setenv("GS_RECURRENCE_PATIENCE", "0")
    assert _now() == 0
    monkeypatch.delenv("GS_RECURRENCE_PATIENCE")
    assert _now() == USUAL
    monkeypatch.setenv("GS_RECURRENCE_PATIENCE", "5")


def test_the_next_test_finds_the_usual_number():
    assert _now() == USUAL


def test_the_library_reads_no_environment():
    """No source of the library looks at it, so no variable changes a call."""
    import gaussian_splatting_tile_amd as pkg
    csrc = os.path.join(os.path.dirname(pkg.__file__), "csrc")
    for name in sorted(os.listdir(csrc)):
        assert "getenv" not in open(os.path.join(csrc, name)).read(), name
