"""gs_adam_step computes in float32: an eps that is 0 there would make 0 / 0 of an element that
has never had a gradient, one that is infinite there would stop every update. Refused before
anything is launched; needs no GPU."""
import ctypes

import pytest


@pytest.mark.parametrize("eps", [1e-50, 1e-46, 1e39, 1e300])
def test_eps_outside_float32_is_refused(eps):
    from gaussian_splatting_tile_amd import _lib
    gs = _lib.load()
    cfg = _lib.GsAdam(0.9, 0.999, eps, 0.0, 0)
    # misaligned on purpose: a call that got past eps is refused for it, not launched
    step = ctypes.c_void_p(260)
    one = (_lib.GsAdamTensor * 1)()
    assert gs.gs_adam_step(ctypes.byref(cfg), one, 1, step, None, ctypes.c_void_p(256), None) == _lib.GS_ERR_INVALID
    assert b"eps" in gs.gs_last_error()


def test_small_and_large_eps_are_taken():
    from gaussian_splatting_tile_amd import _lib
    gs = _lib.load()
    one = (_lib.GsAdamTensor * 1)()
    for eps in (1e-45, 1e-30, 1.0, 1e38):
        cfg = _lib.GsAdam(0.9, 0.999, eps, 0.0, 0)
        assert gs.gs_adam_step(ctypes.byref(cfg), one, 1, ctypes.c_void_p(260), None, ctypes.c_void_p(256), None)
        assert b"step" in gs.gs_last_error() and b"eps" not in gs.gs_last_error()
