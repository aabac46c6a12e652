"""Which sizes and strides calls of the recurrent block refuse, and which they must not. Needs no GPU."""
import ctypes
import os

import pytest
import torch

from test_blocks_host import D, P, _delta, on


@pytest.fixture(scope="module")
def gs():
    from gaussian_splatting_tile_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libgs.so is not built: run __graft_entry__.build()")
    return _lib.load()


@pytest.mark.parametrize("stride", ["q_step", "k_step", "v_step"])
def test_wide_steps(gs, stride):
    """Refused where a chunk's rows are addressed by them, only there. (The calls that pass are refused for an address
    that is not aligned, the last check.)"""
    from gaussian_splatting_tile_amd import _lib
    wide = {stride: (1 << 22) + 1}

    def fwd(**kw):
        assert gs.gs_delta_rule_fwd(ctypes.byref(_delta(**kw)), D, D, D, P(257), D, None, P(512), None, None, D, 1 << 40,
                                    None) == _lib.GS_ERR_INVALID
        return gs.gs_last_error()

    def bwd(**kw):
        assert gs.gs_delta_rule_bwd(ctypes.byref(_delta(**kw)), D, D, D, P(257), D, None, D, D, None, P(512), P(768),
                                    P(1024), P(1280), P(1536), None, D, 1 << 40, None) == _lib.GS_ERR_INVALID
        return gs.gs_last_error()

    few = _lib.GS_DELTA_FEW
    for steps in (0, 1, few):
        assert b"aligned" in fwd(steps=steps, **wide)
    assert b"stride" in fwd(steps=few + 1, **wide)
    for steps in (0, 1):
        assert b"aligned" in bwd(steps=steps, **wide)
    assert b"stride" in bwd(steps=2, **wide)
    size = lambda steps: gs.gs_delta_rule_scratch_bytes(ctypes.byref(_delta(steps=steps, **wide)), 1)  # noqa: E731
    assert size(1) > 0 and size(2) == 0


def test_sizes_past_32_bits(gs):
    """A dimension that a description's 32-bit fields cannot hold is refused, not cut to its low bits (1 and 3 here)."""
    import gaussian_splatting_tile_amd as g
    much = (1 << 32) + 1
    q, v, gates = on(0, 1, 1, 1, 1), on(0, 1, 1, 1, 1), on(0, 1, 1, 1)
    for shape in ((1, much, 1, 1), (much, 1, 1, 1), (1, 1, much, 1), (1, 1, 1, much)):
        with pytest.raises(ValueError, match="at most"):
            g.delta_rule_fwd(q.expand(shape), q.expand(shape), v.expand(shape), gates.expand(shape[:3]), gates.expand(shape[:3]))
        with pytest.raises(ValueError, match="at most"):
            g.delta_rule_bwd(q, q, v.expand(shape), gates, gates, v.expand(shape))
    y = on(0, 2, 1, 1).expand(2, much + 2, 1)
    for kw in (dict(), dict(residual=y)):
        with pytest.raises(ValueError, match="rows"):
            g.block_norm_fwd(y, **kw)
        with pytest.raises(ValueError, match="rows"):
            g.block_norm_bwd(y, y, **kw)
    with pytest.raises(ValueError, match="elements"):
        g.block_norm_fwd(on(0, 1, 1).expand(1, much))
    with pytest.raises(ValueError, match="elements"):
        g.block_norm_fwd(on(0, 1, 0))


def test_outputs_of_one_buffer(gs):
    """Refused, but for h_last in the place of h0."""
    from gaussian_splatting_tile_amd import _lib
    bad, big = _lib.GS_ERR_INVALID, 1 << 40
    a = [P(4096 * i) for i in range(1, 20)]

    def fwd(h0=a[5], o=a[6], last=a[7], ck=a[8], steps=100):
        return gs.gs_delta_rule_fwd(ctypes.byref(_delta(steps=steps)), *a[:5], h0, o, last, ck, a[9], big, None)

    def bwd(outs):
        return gs.gs_delta_rule_bwd(ctypes.byref(_delta()), *a[:9], *outs, a[18], big, None)

    for kw in (dict(o=a[3]), dict(o=a[5]), dict(ck=a[0]), dict(ck=a[5]), dict(last=a[4])):
        for steps in (3, 100):
            assert fwd(steps=steps, **kw) == bad and b"overlaps an input" in gs.gs_last_error(), kw
    for kw in (dict(o=a[7]), dict(o=a[8]), dict(ck=a[7])):
        assert fwd(**kw) == bad and b"one buffer" in gs.gs_last_error(), kw
    outs = a[9:15]
    for i in range(6):
        for j in range(i):
            same = list(outs)
            same[i] = same[j]
            assert bwd(same) == bad and b"one buffer" in gs.gs_last_error(), (i, j)
