"""Host-side checks of the delta rule and the block norms that need no GPU: sizes, and refusals before anything is
launched."""
import ctypes
import os
from types import SimpleNamespace

import pytest
import torch

P = ctypes.c_void_p
D = P(256)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def gs():
    from gaussian_splatting_tile_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libgs.so is not built: run __graft_entry__.build()")
    return _lib.load()


def _delta(**kw):
    from gaussian_splatting_tile_amd import _lib
    r = _lib.GsDeltaRule()
    base = dict(batch=2, steps=100, key_heads=2, heads=4, key_dim=64, value_dim=32, scale=0.125)
    for k, v in dict(base, **kw).items():
        setattr(r, k, v)
    return r


def test_delta_rule_refuses_before_launch(gs):
    from gaussian_splatting_tile_amd import _lib
    bad, big = _lib.GS_ERR_INVALID, 1 << 40
    fwd = lambda r, q=D, k=D, v=D, g=D, b=D, h0=None, o=P(512), last=None, ck=None, s=D, n=big: gs.gs_delta_rule_fwd(  # noqa: E731
        ctypes.byref(r) if r is not None else None, q, k, v, g, b, h0, o, last, ck, s, n, None)
    bwd = lambda r, ck=D, go=D, last=None, gq=P(512), gk=P(768), gv=P(1024), gg=P(1280), gb=P(1536), gh=None, s=D, n=big: gs.gs_delta_rule_bwd(  # noqa: E731
        ctypes.byref(r) if r is not None else None, D, D, D, D, D, None, ck, go, last, gq, gk, gv, gg, gb, gh, s, n, None)
    for call in (fwd, bwd):
        assert call(None) == bad and b"NULL" in gs.gs_last_error()
        for kw, word in ((dict(dtype=3), b"dtype"), (dict(batch=-1), b"batch"), (dict(steps=-1), b"batch"),
                         (dict(batch=1 << 20, steps=1 << 20), b"batch"), (dict(key_heads=0), b"heads"),
                         (dict(heads=3), b"heads"), (dict(heads=5000, key_heads=1), b"heads"),
                         (dict(key_dim=0), b"key_dim"), (dict(value_dim=129), b"value_dim"),
                         (dict(scale=float("nan")), b"scale"), (dict(scale=float("inf")), b"scale"),
                         (dict(q_step=-1), b"stride"), (dict(beta_batch=-4), b"stride"), (dict(lengths=258), b"lengths"),
                         (dict(batch=1 << 14, steps=1 << 16, heads=4096, key_heads=1), b"too many"),
                         (dict(batch=1 << 24, steps=1, heads=4, key_heads=1), b"too many")):
            assert call(_delta(**kw)) == bad and word in gs.gs_last_error(), kw
        assert call(_delta(batch=0)) == _lib.GS_OK
        for s, n, word in ((None, big, b"smaller"), (D, 16, b"smaller"), (P(264), big, b"aligned")):
            assert call(_delta(), s=s, n=n) == bad and word in gs.gs_last_error()
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(g=None), dict(b=None), dict(o=None)):
        assert fwd(_delta(), **kw) == bad and b"NULL" in gs.gs_last_error()
    for kw in (dict(q=P(258)), dict(g=P(257)), dict(h0=P(258)), dict(last=P(258)), dict(ck=P(257))):
        assert fwd(_delta(), **kw) == bad and b"aligned" in gs.gs_last_error()
    assert fwd(_delta(), o=D) == bad and b"overlaps" in gs.gs_last_error()
    for kw in (dict(go=None), dict(gq=None), dict(gk=None), dict(gv=None), dict(gg=None), dict(gb=None)):
        assert bwd(_delta(), **kw) == bad and b"NULL" in gs.gs_last_error()
    assert bwd(_delta(), ck=None) == bad and b"ckpt" in gs.gs_last_error()
    for kw in (dict(gq=D), dict(gv=D), dict(gb=D)):
        assert bwd(_delta(), **kw) == bad and b"overlaps" in gs.gs_last_error()


def test_delta_rule_sizes(gs):
    from gaussian_splatting_tile_amd import delta_rule_ckpt_rows, delta_rule_scratch_bytes
    size = lambda back, **kw: gs.gs_delta_rule_scratch_bytes(ctypes.byref(_delta(**kw)), back)  # noqa: E731
    assert size(0, key_dim=0) == 0 and size(1, dtype=7) == 0 and gs.gs_delta_rule_scratch_bytes(None, 0) == 0
    assert size(0, steps=0) == 0
    assert size(1) > size(0) > 0 and size(1, steps=200) == 2 * size(1)
    assert delta_rule_scratch_bytes(2, 100, 4, 64, 32, True, key_heads=2) == size(1)
    for back in (False, True):  # without the key heads: enough for any number of them
        assert delta_rule_scratch_bytes(2, 100, 4, 64, 32, back) >= max(size(back, key_heads=n) for n in (1, 2, 4))
    assert [delta_rule_ckpt_rows(t) for t in (0, 1, 64, 65, 128, 129)] == [0, 0, 0, 1, 1, 2]


def _norm(**kw):
    from gaussian_splatting_tile_amd import _lib
    d = _lib.GsBlockNorm()
    for k, v in dict(dict(inner=1, width=64, outer=10, eps=1e-6, post=1, pre=1, gating=2, y_outer=64, gate_outer=64,
                          residual_outer=64), **kw).items():
        setattr(d, k, v)
    return d


def test_block_norm_refuses_before_launch(gs):
    from gaussian_splatting_tile_amd import _lib
    bad = _lib.GS_ERR_INVALID
    fwd = lambda d, y=D, z=D, r=None, w=None, b=None, s=None, w2=None, b2=None, o=P(512), n=P(768): gs.gs_block_norm_fwd(  # noqa: E731
        ctypes.byref(d) if d is not None else None, y, z, r, w, b, s, w2, b2, o, n, None)
    bwd = lambda d, y=D, z=D, r=None, w=None, go=P(4096), gn=P(8192), gy=P(512), gz=None, gr=None, sw=None, sp=None, sc=None, n=0: gs.gs_block_norm_bwd(  # noqa: E731
        ctypes.byref(d) if d is not None else None, y, z, r, w, None, None, None, None, go, gn, gy, gz, gr, sw, None,
        None, sp, None, sc, n, None)
    for call in (fwd, bwd):
        assert call(None) == bad and b"NULL" in gs.gs_last_error()
        for kw, word in ((dict(dtype=5), b"dtype"), (dict(weight_dtype=-1), b"dtype"), (dict(post=3), b"norm"),
                         (dict(pre=-1), b"norm"), (dict(gating=9), b"gating"), (dict(outer=-1), b"outer"),
                         (dict(inner=0), b"inner"), (dict(outer=1 << 30, inner=2), b"rows"), (dict(width=0), b"width"),
                         (dict(width=16385), b"width"), (dict(eps=-1.0), b"eps"), (dict(eps=float("nan")), b"eps"),
                         (dict(y_outer=-64), b"stride")):
            assert call(_norm(**kw)) == bad and word in gs.gs_last_error(), kw
        assert call(_norm(outer=0)) == _lib.GS_OK
        assert call(_norm(), y=None) == bad and call(_norm(), z=None) == bad
        assert call(_norm(gating=0)) == bad and b"without gating" in gs.gs_last_error()
        assert call(_norm(post=0), w=D) == bad and b"without the post norm" in gs.gs_last_error()
        assert call(_norm(), y=P(258)) == bad and b"aligned" in gs.gs_last_error()
    assert fwd(_norm(pre=0), b2=D) == bad and b"without the pre norm" in gs.gs_last_error()
    assert fwd(_norm(), n=None) == bad and fwd(_norm(pre=0), o=None) == bad
    assert fwd(_norm(), n=P(512)) == bad and fwd(_norm(), n=D) == bad
    assert fwd(_norm(y_outer=128), o=D) == bad and b"contiguous" in gs.gs_last_error()
    assert bwd(_norm(), gn=None) == bad and bwd(_norm(pre=0), go=None) == bad and bwd(_norm(), gy=None) == bad
    assert bwd(_norm(pre=0), sp=D) == bad and bwd(_norm(post=0), sw=D) == bad
    assert bwd(_norm(), gy=D) == bad and bwd(_norm(), gz=P(512)) == bad
    assert bwd(_norm(), sw=D) == bad and b"smaller" in gs.gs_last_error()
    assert bwd(_norm(), sw=D, sc=P(258), n=1 << 40) == bad and b"aligned" in gs.gs_last_error()


class On(torch.Tensor):
    """A host tensor that says it is on cuda:`card` (views of one: on cuda:0)."""

    card = 0
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.card))

    def get_device(self):
        return self.card


def on(card, *shape, dtype=torch.float32):
    t = torch.zeros(shape, dtype=dtype).as_subclass(On)
    t.card = card
    return t


STREAM = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=12345)


def test_delta_rule_refuses_tensors():
    import gaussian_splatting_tile_amd as gs
    B, T, Hk, H, dk, dv = 2, 10, 1, 2, 8, 16
    good = lambda i=0: dict(q=on(i, B, T, Hk, dk), k=on(i, B, T, Hk, dk), v=on(i, B, T, H, dv),  # noqa: E731
                            log_decay=on(i, B, T, H), beta=on(i, B, T, H))
    shapes = {k: t.shape for k, t in good().items()}
    for name in shapes:
        for bad in (1, -1):
            if name != "q":
                with pytest.raises(TypeError, match="cuda:0"):
                    gs.delta_rule_fwd(**dict(good(), **{name: on(bad, *shapes[name])}))
        with pytest.raises(TypeError):
            gs.delta_rule_fwd(**dict(good(), **{name: on(0, *shapes[name], dtype=torch.float64)}))
    given = dict(o=on(0, B, T, H, dv), h_last=on(0, B, H, dk, dv))
    for kw in (dict(h0=on(1, B, H, dk, dv)), dict(lengths=on(1, B, dtype=torch.int32)),
               dict(restart=on(1, B, T, dtype=torch.uint8)), dict(out=dict(given, h_last=on(1, B, H, dk, dv))),
               dict(out=dict(given, o=on(1, B, T, H, dv)))):
        with pytest.raises(TypeError, match="cuda:0"):
            gs.delta_rule_fwd(**dict(dict(good(), out=given), **kw))
    for name, shape in (("k", (B, T, Hk, dk + 1)), ("v", (B, T + 1, H, dv)), ("beta", (B, T, Hk))):
        with pytest.raises(ValueError):
            gs.delta_rule_fwd(**dict(good(), **{name: on(0, *shape)}))
    with pytest.raises(ValueError, match="contiguous"):
        gs.delta_rule_fwd(**dict(good(), v=on(0, B, T, dv, H).transpose(2, 3)))
    with pytest.raises(ValueError, match="stream belongs to cuda:1"):
        gs.delta_rule_fwd(**good(), stream=STREAM)
    with pytest.raises(ValueError, match="stream belongs to cuda:1"):
        gs.delta_rule_bwd(**good(), grad_o=on(0, B, T, H, dv), stream=STREAM)


def test_block_norm_refuses_tensors():
    import gaussian_splatting_tile_amd as gs
    y = on(0, 6, 4, 8)
    for kw in (dict(residual=on(1, 6, 4, 8)), dict(gate=on(-1, 6, 4, 8)), dict(scale=on(1, 8))):
        with pytest.raises(TypeError, match="cuda:0"):
            gs.block_norm_fwd(y, **kw)
    with pytest.raises(TypeError):
        gs.block_norm_fwd(y, residual=on(0, 6, 4, 8, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        gs.block_norm_fwd(y, scale=on(0, 8), post=gs.BLOCK_NORM_RMS, post_weight=on(0, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        gs.block_norm_fwd(y, scale=on(0, 9))
    with pytest.raises(ValueError):
        gs.block_norm_fwd(on(0, 8))
    with pytest.raises(ValueError, match="one stride"):
        gs.block_norm_fwd(on(0, 3, 4, 5, 8).transpose(0, 2), residual=on(0, 5, 4, 3, 16)[..., :8])
    with pytest.raises(ValueError, match="stream belongs to cuda:1"):
        gs.block_norm_fwd(y, stream=STREAM)


def test_delta_rule_addresses(gs):
    """A chunk's rows are addressed in 32 bits: wider strides are refused, as is a workspace that is not aligned."""
    from gaussian_splatting_tile_amd import _lib
    wide = (1 << 22) + 1
    for kw in (dict(q_step=wide), dict(k_step=wide), dict(v_step=wide)):
        r = _delta(**kw)
        assert gs.gs_delta_rule_fwd(ctypes.byref(r), D, D, D, D, D, None, P(512), None, None, D, 1 << 40, None) == _lib.GS_ERR_INVALID
        assert b"stride" in gs.gs_last_error()
        assert gs.gs_delta_rule_scratch_bytes(ctypes.byref(r), 0) == 0


def test_block_norm_weights_type(gs):
    """Weights are float32 or of the rows' type."""
    from gaussian_splatting_tile_amd import _lib
    d = _norm(dtype=_lib.GS_BF16, weight_dtype=_lib.GS_F16)
    assert gs.gs_block_norm_fwd(ctypes.byref(d), D, D, None, None, None, None, None, None, P(512), P(768), None) == _lib.GS_ERR_INVALID
    assert b"weight_dtype" in gs.gs_last_error()


def test_constants_match_the_header(gs):
    import re
    from gaussian_splatting_tile_amd import _lib
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gs.h")) as f:
        header = dict(re.findall(r"#define (GS_(?:DELTA|BLOCK)_\w+) (\d+)", f.read()))
    for name, value in header.items():
        assert getattr(_lib, name, int(value)) == int(value), name
    assert {"GS_DELTA_CHUNK", "GS_DELTA_FEW", "GS_DELTA_MAX_DIM", "GS_BLOCK_NORM_RMS", "GS_BLOCK_GATE_SILU"} <= set(header)
