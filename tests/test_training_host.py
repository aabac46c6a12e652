"""Host-side checks of the sequence and training entry points that need no
GPU: sizes, and refusals before anything is launched."""
import ctypes
import os

import pytest

P = ctypes.c_void_p
D = P(256)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def gs():
    from gaussian_splatting_tile_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libgs.so is not built: run __graft_entry__.build()")
    return _lib.load()


def _rec(**kw):
    from gaussian_splatting_tile_amd import _lib
    r = _lib.GsRecurrence()
    for k, v in dict(dict(batch=2, steps=100, channels=8, gate_batch=800, gate_step=8, x_batch=800, x_step=8), **kw).items():
        setattr(r, k, v)
    return r


def test_recurrence_refuses_before_launch(gs):
    from gaussian_splatting_tile_amd import _lib
    bad = _lib.GS_ERR_INVALID
    fwd = lambda r, gate=D, x=D, h0=None, h=D, last=None, ckpt=None, scratch=None, n=0: gs.gs_recurrence_fwd(
        ctypes.byref(r) if r is not None else None, gate, x, h0, h, last, ckpt, scratch, n, None)
    bwd = lambda r, ckpt=None, g=D, dg=D, dx=D, dh0=None, scratch=None, n=0: gs.gs_recurrence_bwd(
        ctypes.byref(r) if r is not None else None, D, D, None, ckpt, g, None, dg, dx, dh0, scratch, n, None)
    for call in (fwd, bwd):
        assert call(None) == bad and b"NULL" in gs.gs_last_error()
        for kw, word in ((dict(dtype=3), b"dtype"), (dict(dtype=-1), b"dtype"), (dict(gating=2), b"gating"),
                         (dict(batch=-1), b"batch"), (dict(steps=(1 << 30) + 1), b"steps"), (dict(channels=-5), b"channels"),
                         (dict(gate_step=-8), b"stride"), (dict(x_batch=-1), b"stride"),
                         (dict(batch=1 << 20, channels=1 << 20), b"too many"),
                         (dict(batch=1 << 30, channels=1 << 30, steps=1 << 30), b"too many"),
                         (dict(lengths=258), b"lengths")):
            assert call(_rec(**kw)) == bad and word in gs.gs_last_error(), kw
        # nothing to do
        assert call(_rec(batch=0)) == _lib.GS_OK
        assert call(_rec(channels=0)) == _lib.GS_OK
    for kw in (dict(gate=None), dict(x=None), dict(h=None)):
        assert fwd(_rec(), **kw) == bad and b"NULL" in gs.gs_last_error()
    for kw in (dict(gate=P(258)), dict(h0=P(258)), dict(last=P(257)), dict(ckpt=P(258))):
        assert fwd(_rec(), **kw) == bad and b"aligned" in gs.gs_last_error()
    assert fwd(_rec(dtype=_lib.GS_BF16), gate=P(257)) == bad
    for kw in (dict(g=None), dict(dg=None), dict(dx=None)):
        assert bwd(_rec(), **kw) == bad and b"NULL" in gs.gs_last_error()
    assert bwd(_rec(steps=129)) == bad and b"ckpt" in gs.gs_last_error()
    assert bwd(_rec(), dh0=P(258)) == bad


def test_recurrence_scratch_size(gs):
    size = lambda **kw: gs.gs_recurrence_scratch_bytes(ctypes.byref(_rec(**kw)))
    assert size(steps=128) == 0 and size(steps=0) == 0 and size(batch=0, steps=1000) == 0
    assert size(dtype=9, steps=1000) == 0 and size(steps=-1) == 0
    assert gs.gs_recurrence_scratch_bytes(None) == 0
    # a word per channel of each chunk and of each 8 chunks, a state per 64 chunks (channels in
    # rows of 128)
    assert size(batch=3, steps=129, channels=65) == 3 * (2 * 128 * 8 + 128 * 8 + 128 * 4)
    assert size(batch=1, steps=128 * 65, channels=64) == 65 * 128 * 8 + 9 * 128 * 8 + 2 * 128 * 4
    from gaussian_splatting_tile_amd import _lib
    r = _rec(steps=129, gate_batch=0, x_batch=0)
    need = gs.gs_recurrence_scratch_bytes(ctypes.byref(r))
    for scratch, n, word in ((None, need, b"smaller"), (D, need - 1, b"smaller"), (P(260), need, b"aligned")):
        assert gs.gs_recurrence_fwd(ctypes.byref(r), D, D, None, D, None, None, scratch, n, None) == _lib.GS_ERR_INVALID
        assert word in gs.gs_last_error()
        assert gs.gs_recurrence_bwd(ctypes.byref(r), D, D, None, D, D, None, D, D, None, scratch, n,
                                    None) == _lib.GS_ERR_INVALID
        assert word in gs.gs_last_error()


def test_recurrence_checkpoint_rows():
    from gaussian_splatting_tile_amd import recurrence_ckpt_rows
    assert [recurrence_ckpt_rows(t) for t in (0, 1, 128, 129, 256, 257)] == [0, 0, 0, 1, 1, 2]


def _list(ctype, n=2, **kw):
    a = (ctype * n)()
    for d in a:
        for k, v in kw.items():
            setattr(d, k, v)
    return a


def test_norm_and_clip_refuse_before_launch(gs):
    from gaussian_splatting_tile_amd import _lib
    bad = _lib.GS_ERR_INVALID
    good = dict(grad=256, out=256, count=4)
    L = lambda **kw: _list(_lib.GsGradTensor, **dict(good, **kw))
    assert gs.gs_grad_scratch_bytes() > 0
    for call in (lambda t, n=2, kind=0, norm=D, s=D: gs.gs_grad_norm(t, n, kind, norm, s, None),
                 lambda t, n=2, kind=0, norm=D, s=D: gs.gs_clip_grads(t, n, kind, 1.0, norm, s, None)):
        assert call(L(), n=-1) == bad and call(L(), n=16385) == bad and b"n_tensors" in gs.gs_last_error()
        assert call(None) == bad and b"tensors" in gs.gs_last_error()
        assert call(L(), kind=2) == bad and b"kind" in gs.gs_last_error()
        assert call(L(), norm=None) == bad and call(L(), norm=P(258)) == bad
        assert call(L(), s=None) == bad and call(L(), s=P(260)) == bad and b"scratch" in gs.gs_last_error()
        assert call(L(dtype=3)) == bad and b"dtype" in gs.gs_last_error()
        assert call(L(grad=None)) == bad and call(L(grad=257)) == bad
        assert call(L(count=-1)) == bad and call(L(count=1 << 38)) == bad and b"count" in gs.gs_last_error()
    clip = lambda t, m=1.0: gs.gs_clip_grads(t, 2, 0, m, D, D, None)
    assert clip(L(out=None)) == bad and clip(L(out=258)) == bad
    for m in (0.0, -1.0, float("nan"), float("inf")):
        assert clip(L(), m) == bad and b"max_norm" in gs.gs_last_error()


def test_adam_refuses_before_launch(gs):
    from gaussian_splatting_tile_amd import _lib
    bad = _lib.GS_ERR_INVALID
    good = dict(param=256, grad=256, m=256, v=256, count=4, lr=0.1)
    L = lambda **kw: _list(_lib.GsAdamTensor, **dict(good, **kw))

    def call(t=None, cfg=None, n=2, step=D, norm=None, s=D):
        c = _lib.GsAdam(0.9, 0.999, 1e-8, 0.0, 0)
        for k, v in (cfg or {}).items():
            setattr(c, k, v)
        return gs.gs_adam_step(ctypes.byref(c), L() if t is None else t, n, step, norm, s, None)

    assert gs.gs_adam_step(None, L(), 2, D, None, D, None) == bad and b"cfg" in gs.gs_last_error()
    nan, inf = float("nan"), float("inf")
    for cfg, word in ((dict(beta1=1.0), b"beta1"), (dict(beta2=-0.1), b"beta2"), (dict(beta1=nan), b"beta1"),
                      (dict(eps=0.0), b"eps"), (dict(eps=inf), b"eps"), (dict(max_norm=-1.0), b"max_norm"),
                      (dict(max_norm=nan), b"max_norm"), (dict(max_norm=inf), b"max_norm"), (dict(flags=2), b"flags")):
        assert call(cfg=cfg) == bad and word in gs.gs_last_error(), cfg
    assert call(n=-1) == bad and call(n=20000) == bad
    assert call(step=None) == bad and call(step=P(260)) == bad and b"step" in gs.gs_last_error()
    assert call(norm=P(258)) == bad and call(s=None) == bad and call(s=P(260)) == bad
    for kw in (dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(param=258), dict(m=258), dict(v=257),
               dict(param_dtype=3), dict(grad_dtype=-1), dict(lr=nan), dict(weight_decay=inf), dict(count=-1)):
        assert call(L(**kw)) == bad, kw
