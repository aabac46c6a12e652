"""Chunks that compute for themselves what the chunks before them have not given yet read the
inputs again at any later time: outputs of more than one chunk in an input's place are refused,
before anything is launched. Needs no GPU."""
import ctypes

P = ctypes.c_void_p
# distinct aligned addresses; none is looked at
GATE, X, G, DG, DX, CKPT, SCRATCH = (P(4096 * (k + 1)) for k in range(7))


def _rec(steps):
    from gaussian_splatting_tile_amd import _lib
    r = _lib.GsRecurrence()
    for k, v in dict(batch=1, steps=steps, channels=8, gate_batch=8 * steps, gate_step=8, x_batch=8 * steps,
                     x_step=8).items():
        setattr(r, k, v)
    return ctypes.byref(r)


def test_outputs_in_an_inputs_place_are_refused():
    from gaussian_splatting_tile_amd import _lib
    gs = _lib.load()
    for steps in (129, 100_000):
        r, bad = _rec(steps), _lib.GS_ERR_INVALID
        n = gs.gs_recurrence_scratch_bytes(r)
        for h in (GATE, X):
            assert gs.gs_recurrence_fwd(r, GATE, X, None, h, None, None, SCRATCH, n, None) == bad
            assert b"overlaps" in gs.gs_last_error()
        for dg, dx in ((GATE, DX), (X, DX), (G, DX), (DG, GATE), (DG, X), (DG, G)):
            assert gs.gs_recurrence_bwd(r, GATE, X, None, CKPT, G, None, dg, dx, None, SCRATCH, n, None) == bad
            assert b"overlaps" in gs.gs_last_error()
